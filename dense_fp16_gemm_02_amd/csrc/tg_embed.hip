// tg_embed.hip — embedding lookup and its gradient.  See include/tg_embed.h for
// the contract.
//
// The lookup copies rows, 16 bytes a lane.
//
// The gradient sorts the tokens (a stable radix sort of (token, row of dY)
// pairs) and walks two sorted lists at once, the sorted tokens and
// the rows of dW, each row after its tokens: a token adds its row of dY to the sum
// in registers, a row stores the sum and clears it.  The walk is cut into equal
// pieces of the two lists taken together (the "merge path" partition of Merrill
// and Garland, Merge-based Parallel Sparse Matrix-Vector Multiplication, 2016), so
// that a wave's work is the same whether its piece holds rows without tokens, which
// are only zeroed, or one token a thousand times.  A row that begins in one
// piece and ends in another leaves fp32 sums in the workspace, which a last kernel
// adds in order.  No atomics: the order of every addition is fixed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "proj_tile.hpp"

#include "tg_embed.h"
#include "tg_gemm.h"

namespace {
using namespace pt;

template <typename E>
constexpr int VEC = 16 / (int)sizeof(E);  // elements of a lane

// 16 bytes at the alignment of an element, `n` elements of them inside the row.
// A store of aligned ones is spelled out: the compiler splits it otherwise where it
// knows the values (rows of zeros: 1 GB of them in 300 us instead of 220).
typedef float f32x4_row __attribute__((ext_vector_type(4)));
template <typename E>
__device__ inline void load_row(E (&x)[VEC<E>], const E *p, int n)
{
    if (n >= VEC<E>) {
        __builtin_memcpy(x, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            x[e] = e < n ? p[e] : (E)0.0f;
    }
}
// NT: past the caches.
template <bool NT = false, typename E>
__device__ inline void store_row(const E (&x)[VEC<E>], E *p, int n)
{
    if (n >= VEC<E> && (uintptr_t)p % 16 == 0) {
        f32x4_row v;
        __builtin_memcpy(&v, x, 16);
        if constexpr (NT)
            __builtin_nontemporal_store(v, reinterpret_cast<f32x4_row *>(p));
        else
            *reinterpret_cast<f32x4_row *>(p) = v;
    } else if (n >= VEC<E>) {
        __builtin_memcpy(p, x, 16);
    } else {
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            if (e < n)
                p[e] = x[e];
    }
}

// ------------------------------------------------------------------ lookup
constexpr int LOOK_THREADS = 256, LOOK_STEPS = 4;
struct LookArgs {
    const int64_t *tokens;
    const void *W;
    void *Y;
    int64_t M, V, K, ldw, ldy;
    int segments;  // of 64 lanes · LOOK_STEPS to a row
    float scale;
};
// A wave takes LOOK_STEPS·64 lanes of one row.  Bound by memory where a row fills them; of
// narrower rows some 3.4 a ns are looked up whatever their width (2^20 of them from 32000
// rows: 64, 128 and 256 fp32 314, 314 and 306 us, where a copy of the bytes would take 56, 110
// and 218; as many bf16 377-379 us).  NT: Y is too large
// to be kept for its reader anyway; without it Y displaces W from the last-level cache
// (65536 tokens of 32000×2048 fp16, 268 MB of Y: 64 us, 86 without; 8192 of
// 131072×4096 bf16, 64 MiB: 23.5 and 24.9).
constexpr int64_t NT_BYTES = (int64_t)64 << 20;
template <typename E, bool NT>
__global__ __launch_bounds__(LOOK_THREADS) void embedding_kernel(LookArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t units = a.M * a.segments, stride = (int64_t)gridDim.x * (LOOK_THREADS / 64);
    for (int64_t u = (int64_t)blockIdx.x * (LOOK_THREADS / 64) + uniform(threadIdx.x >> 6); u < units; u += stride) {
        const int64_t row = u / a.segments;
        const int64_t c0 = (u - row * a.segments) * (64 * LOOK_STEPS * VEC<E>) + lane * VEC<E>;
        const int64_t t = a.tokens[row];
        const bool in = t >= 0 && t < a.V;
        const E *src = reinterpret_cast<const E *>(a.W) + (in ? t : 0) * a.ldw;
        E *dst = reinterpret_cast<E *>(a.Y) + row * a.ldy;
        E x[LOOK_STEPS][VEC<E>];
#pragma unroll
        for (int k = 0; k < LOOK_STEPS; ++k) {
            const int64_t c = c0 + k * (64 * VEC<E>);
            load_row(x[k], src + c, in && c < a.K ? imin((int)(a.K - c), VEC<E>) : 0);
        }
#pragma unroll
        for (int k = 0; k < LOOK_STEPS; ++k) {
            const int64_t c = c0 + k * (64 * VEC<E>);
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
                x[k][e] = in ? (E)((float)x[k][e] * a.scale) : (E)NAN;
            if (c < a.K)
                store_row<NT>(x[k], dst + c, imin((int)(a.K - c), VEC<E>));
        }
    }
}

// -------------------------------------------------------------------- sort
// A stable radix sort in as few passes as digits of up to 9 bits allow (two for
// up to 2^18 rows).
constexpr int DIGIT_BITS = 9, DIGITS = 1 << DIGIT_BITS;
constexpr int FEW = 256, MANY = 1024;    // threads of a workgroup
// Pairs of a lane, which are ordered 64 to a round: half as many where small workgroups
// are there to spread the rounds over the chip (65536 tokens, lookup and gradient, 194 us,
// 198 with eight).  Bound by the latency of the rounds: a pass over 65536 pairs some 14 us,
// the two of one workgroup's 8192 22 us.
constexpr int sort_per(int threads) { return threads == FEW ? 4 : 8; }
struct SortArgs {
    const int64_t *tokens;          // first pass
    const uint32_t *key_in, *at_in; // later passes
    uint32_t *key, *at;
    uint32_t *count;                // [workgroup][digit], and behind them one sum for each digit
    bool scanned;                   // count holds sums over the workgroups before
    int M, V;
    int64_t padding;
    int tiles, shift, bits, passes;  // bits: of a digit
};
// A token that adds to no row sorts behind all rows.
__device__ inline uint32_t token_key(const SortArgs &a, int i)
{
    const int64_t t = a.tokens[i];
    return t >= 0 && t < a.V && t != a.padding ? (uint32_t)t : (uint32_t)a.V;
}
// Items of a wave, so that few are spread over all waves.
template <int THREADS>
__device__ inline int wave_items(int items)
{
    return 64 * ((items + THREADS - 1) / THREADS);
}
// Item r of this lane: a wave's items are consecutive, 64 to a round.  Past the
// wave's: INT_MAX.
__device__ inline int sort_item(int wave, int lane, int r, int per)
{
    return 64 * r < per ? wave * per + r * 64 + lane : 0x7fffffff;
}

template <int THREADS>
struct SortShared {
    static constexpr int WAVES = THREADS / 64;
    uint32_t wave_count[WAVES][DIGITS];  // of a digit in a wave, then where the wave's first of it goes
    uint32_t wave_sum[WAVES];
    uint32_t base[DIGITS];
};
// Exclusive sum of x over the workgroup's threads.
template <int THREADS>
__device__ inline uint32_t sum_before(uint32_t x, uint32_t *wave_sum)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    uint32_t upto = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = __shfl_up(upto, o);
        upto += lane >= o ? y : 0;
    }
    if (lane == 63)
        wave_sum[wave] = upto;
    __syncthreads();
    uint32_t before = upto - x;
    for (int w = 0; w < wave; ++w)
        before += wave_sum[w];
    __syncthreads();
    return before;
}
// For each of this lane's items its place among the workgroup's items, ordered
// by digit and, within one, as they came.  Lanes of a wave that hold the same
// digit find each other with one ballot per bit.
template <int THREADS>
__device__ inline void sort_places(SortShared<THREADS> &s, const uint32_t (&key)[sort_per(THREADS)], int items,
                                   int shift, int bits, uint32_t (&place)[sort_per(THREADS)])
{
    constexpr int WAVES = THREADS / 64, PER = sort_per(THREADS);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), per = wave_items<THREADS>(items);
    const uint32_t mask = (1u << bits) - 1;
    for (int d = lane; d < DIGITS; d += 64)
        s.wave_count[wave][d] = 0;
    __builtin_amdgcn_wave_barrier();
    volatile uint32_t *mine = s.wave_count[wave];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        place[r] = 0;
        if (sort_item(wave, 0, r, per) >= items)  // the same for the whole wave
            continue;
        const bool live = sort_item(wave, lane, r, per) < items;
        const uint32_t d = (key[r] >> shift) & mask;
        const uint64_t all = __ballot(live);
        uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
#pragma unroll
        for (int b = 0; b < DIGIT_BITS; ++b) {
            const uint32_t bit = (d >> b) & 1, flip = bit - 1;  // all ones where the bit is clear
            const uint64_t set = __ballot(bit);
            lo &= (uint32_t)set ^ flip;
            hi &= (uint32_t)(set >> 32) ^ flip;
        }
        const uint32_t before = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
        const uint32_t seen = mine[d];
        __builtin_amdgcn_wave_barrier();
        if (live && before == 0)
            mine[d] = seen + (uint32_t)(__popc(lo) + __popc(hi));
        __builtin_amdgcn_wave_barrier();
        place[r] = seen + before;
    }
    __syncthreads();
    // exclusive sums over (digit, wave): a thread takes all waves of some digits,
    // or some waves of one
    constexpr int EACH = WAVES * DIGITS / THREADS;  // counts of a thread: DIGITS / 64
    static_assert(EACH % WAVES == 0 || WAVES % EACH == 0, "whole digits, or one digit's waves");
    uint32_t c[EACH], sum = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        c[k] = s.wave_count[(tid * EACH + k) % WAVES][(tid * EACH + k) / WAVES];
        sum += c[k];
    }
    uint32_t at = sum_before<THREADS>(sum, s.wave_sum);
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        s.wave_count[(tid * EACH + k) % WAVES][(tid * EACH + k) / WAVES] = at;
        at += c[k];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < PER; ++r)
        place[r] += s.wave_count[wave][(key[r] >> shift) & mask];
}

// All passes of at most SORT_SMALL tokens, by one workgroup.
constexpr int SORT_SMALL = MANY * sort_per(MANY);
__global__ __launch_bounds__(MANY) void sort_small_kernel(SortArgs a)
{
    constexpr int PER = sort_per(MANY);
    __shared__ SortShared<MANY> s;
    __shared__ uint32_t keys[SORT_SMALL], ats[SORT_SMALL];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int per = wave_items<MANY>(a.M);
    uint32_t key[PER], at[PER], place[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = sort_item(wave, lane, r, per);
        key[r] = i < a.M ? token_key(a, i) : 0;
        at[r] = (uint32_t)i;
    }
    for (int p = 0; p < a.passes; ++p) {
        sort_places<MANY>(s, key, a.M, a.bits * p, a.bits, place);
#pragma unroll
        for (int r = 0; r < PER; ++r)
            if (sort_item(wave, lane, r, per) < a.M) {
                keys[place[r]] = key[r];
                ats[place[r]] = at[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            const int i = sort_item(wave, lane, r, per);
            if (i < a.M) {
                key[r] = keys[i];
                at[r] = ats[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = sort_item(wave, lane, r, per);
        if (i < a.M) {
            a.key[i] = key[r];
            a.at[i] = at[r];
        }
    }
}

// How often each digit occurs in each workgroup's pairs.
template <int THREADS, bool FIRST>
__global__ __launch_bounds__(THREADS) void sort_count_kernel(SortArgs a)
{
    constexpr int PER = sort_per(THREADS);
    __shared__ uint32_t count[DIGITS];
    const int tid = threadIdx.x;
    for (int d = tid; d < DIGITS; d += THREADS)
        count[d] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * (THREADS * PER);
    const uint32_t mask = (1u << a.bits) - 1;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int64_t i = i0 + r * THREADS + tid;
        if (i < a.M)
            atomicAdd(&count[((FIRST ? token_key(a, (int)i) : a.key_in[i]) >> a.shift) & mask], 1u);
    }
    __syncthreads();
    for (int d = tid; d < DIGITS; d += THREADS)
        a.count[(int64_t)blockIdx.x * DIGITS + d] = count[d];
}
// The counts of many workgroups into sums over the workgroups before each, so that the
// work stays linear in the pairs.  A workgroup takes SCAN_DIGITS digits, its threads
// runs of the counts.
constexpr int SCAN_DIGITS = 32, SCAN_RUNS = 1024 / SCAN_DIGITS;
__global__ __launch_bounds__(1024) void sort_scan_kernel(SortArgs a)
{
    __shared__ uint32_t sums[SCAN_RUNS][SCAN_DIGITS];
    const int d = (int)blockIdx.x * SCAN_DIGITS + threadIdx.x % SCAN_DIGITS, run = threadIdx.x / SCAN_DIGITS;
    const int len = (a.tiles + SCAN_RUNS - 1) / SCAN_RUNS, from = imin(run * len, a.tiles), to = imin(from + len, a.tiles);
    uint32_t sum = 0;
#pragma unroll 8
    for (int b = from; b < to; ++b)
        sum += a.count[(int64_t)b * DIGITS + d];
    sums[run][threadIdx.x % SCAN_DIGITS] = sum;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int r = 0; r < SCAN_RUNS; ++r) {
        const uint32_t x = sums[r][threadIdx.x % SCAN_DIGITS];
        before += r < run ? x : 0;
        all += x;
    }
#pragma unroll 8
    for (int b = from; b < to; ++b) {
        uint32_t *c = a.count + (int64_t)b * DIGITS + d;
        const uint32_t x = *c;
        *c = before;
        before += x;
    }
    if (run == 0)
        a.count[(int64_t)a.tiles * DIGITS + d] = all;
}
// One pass: each pair to its place.
template <int THREADS, bool FIRST>
__global__ __launch_bounds__(THREADS) void sort_scatter_kernel(SortArgs a)
{
    constexpr int PER = sort_per(THREADS);
    __shared__ SortShared<THREADS> s;
    __shared__ uint32_t part[2][THREADS > DIGITS ? THREADS : DIGITS];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t i0 = (int64_t)blockIdx.x * (THREADS * PER);
    const int items = (int)(a.M - i0 < THREADS * PER ? a.M - i0 : THREADS * PER), per = wave_items<THREADS>(items);
    uint32_t key[PER], at[PER], place[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = sort_item(wave, lane, r, per);
        key[r] = i < items ? (FIRST ? token_key(a, (int)(i0 + i)) : a.key_in[i0 + i]) : 0;
        at[r] = i < items ? (FIRST ? (uint32_t)(i0 + i) : a.at_in[i0 + i]) : 0;
    }
    // where this workgroup's first pair of each digit goes: behind all pairs of
    // smaller digits, and those of its digit in the workgroups before
    constexpr int SPLIT = THREADS > DIGITS ? THREADS / DIGITS : 1;  // threads that share a digit's counts
    for (int q = tid; q < DIGITS * SPLIT; q += THREADS) {
        const int d = q % DIGITS;
        part[0][q] = part[1][q] = 0;
        if (d >> a.bits)  // not a digit
            continue;
        if (a.scanned) {
            if (q < DIGITS) {
                part[0][q] = a.count[(int64_t)a.tiles * DIGITS + d];
                part[1][q] = a.count[(int64_t)blockIdx.x * DIGITS + d];
            }
            continue;
        }
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int b = q / DIGITS; b < a.tiles; b += SPLIT) {
            const uint32_t c = a.count[(int64_t)b * DIGITS + d];
            all += c;
            before += b < (int)blockIdx.x ? c : 0;
        }
        part[0][q] = all, part[1][q] = before;
    }
    __syncthreads();
    constexpr int EACH = DIGITS > THREADS ? DIGITS / THREADS : 1;  // consecutive digits of a thread
    uint32_t all[EACH], before[EACH], sum = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int d = tid * EACH + k;
        all[k] = before[k] = 0;
        if (d < DIGITS)
            for (int q = d; q < DIGITS * SPLIT; q += DIGITS)
                all[k] += part[0][q], before[k] += part[1][q];
        sum += all[k];
    }
    uint32_t base = sum_before<THREADS>(sum, s.wave_sum);
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        if (tid * EACH + k < DIGITS)
            s.base[tid * EACH + k] = base + before[k];
        base += all[k];
    }
    sort_places<THREADS>(s, key, items, a.shift, a.bits, place);
    // (behind sort_places wave_count[0][d] is the digit's first place in the workgroup)
#pragma unroll
    for (int r = 0; r < PER; ++r)
        if (sort_item(wave, lane, r, per) < items) {
            const uint32_t d = (key[r] >> a.shift) & ((1u << a.bits) - 1);
            const uint32_t to = s.base[d] + place[r] - s.wave_count[0][d];
            a.key[to] = key[r];
            a.at[to] = at[r];
        }
}

// ------------------------------------------------------------------ gradient
constexpr int WALK_THREADS = 256, WALK_WAVES = WALK_THREADS / 64, AHEAD = 4;
struct WalkArgs {
    const uint32_t *key, *at;  // sorted tokens, and their rows of dY
    const void *dY;
    void *dW;
    int M, V;
    int64_t K, lddy, lddw;
    int piece;     // items of a wave: tokens and rows
    int pieces, segments;
    float scale;
    int2 *carried; // per piece: the row that it ends and others began (-1: none), and the first of those
    float *head, *tail;  // per piece: its part of that row; its part of the row that it leaves open
};
// How many of the first d items of the two lists are tokens: the smallest i whose
// token does not come before item d.  64 probes at a time.
__device__ inline int walk_tokens(const uint32_t *key, int64_t M, int64_t V, int64_t d, int lane)
{
    int64_t lo = d > V ? d - V : 0, hi = d < M ? d : M;  // the answer is in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t i = lo + lane * step;
        const bool before = i < hi && (int64_t)key[i] <= d - 1 - i;  // token i is one of the first d items
        const int n = __popcll(__ballot(before));
        if (n == 0)
            hi = lo;
        else {
            const int64_t last = lo + (n - 1) * step;  // the last probe that holds
            hi = hi < last + step ? hi : last + step;
            lo = last + 1;
        }
    }
    return uniform((int)lo);
}
// Bound by memory: dW of 131072×4096 bf16 from 8192 rows 225 us (5.1 TB/s), of 32000×2048
// fp16 from 65536 rows 80 us (4.8 TB/s).  A piece of a row narrower than a wave's 64·VEC
// elements leaves lanes idle.
template <typename E>
__global__ __launch_bounds__(WALK_THREADS) void embedding_walk_kernel(WalkArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * WALK_WAVES + uniform(threadIdx.x >> 6);
    const int piece = (int)(unit / a.segments), segment = (int)(unit - (int64_t)piece * a.segments);
    if (piece >= a.pieces)
        return;
    const int64_t d0 = (int64_t)piece * a.piece, items = (int64_t)a.V + a.M;
    const int64_t d1 = d0 + a.piece < items ? d0 + a.piece : items;
    const int i0 = walk_tokens(a.key, a.M, a.V, d0, lane), i1 = walk_tokens(a.key, a.M, a.V, d1, lane);
    const int v0 = (int)(d0 - i0), v1 = (int)(d1 - i1);
    const int open = i0 > 0 && v0 < a.V && (int)a.key[i0 - 1] == v0 ? v0 : -1;
    const int64_t c = ((int64_t)segment * 64 + lane) * VEC<E>;
    const int n = c < a.K ? (int)(a.K - c < VEC<E> ? a.K - c : VEC<E>) : 0;
    if (segment == 0 && lane == 0) {
        int first = 0;
        if (open >= 0 && v1 > v0) {  // the piece with the row's first token
            int lo = 0, hi = i0 - 1;
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if ((int)a.key[mid] < open)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            first = (int)(((int64_t)lo + open) / a.piece);
        }
        a.carried[piece] = make_int2(open >= 0 && v1 > v0 ? open : -1, first);
    }
    const E *dY = reinterpret_cast<const E *>(a.dY) + c;
    E *dW = reinterpret_cast<E *>(a.dW) + c;
    float acc[VEC<E>];
    bool some = false;
#pragma unroll
    for (int e = 0; e < VEC<E>; ++e)
        acc[e] = 0.0f;
    int v = v0;
    const auto part = [&](float *to) {
        float *dst = to + (int64_t)piece * a.K + c;
        if (n == VEC<E>)
            __builtin_memcpy(dst, acc, sizeof acc);
        else
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
                if (e < n)
                    dst[e] = acc[e];
    };
    const auto close_before = [&](int k) {  // rows v .. k - 1 end
        if (v < k && (some || v == open)) {
            if (v == open) {
                part(a.head);
            } else {
                E x[VEC<E>];
#pragma unroll
                for (int e = 0; e < VEC<E>; ++e)
                    x[e] = (E)(acc[e] * a.scale);
                store_row(x, dW + (int64_t)v * a.lddw, n);
            }
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
                acc[e] = 0.0f;
            some = false;
            ++v;
        }
        const E zero[VEC<E>] = {};
        for (; v < k; ++v)
            store_row(zero, dW + (int64_t)v * a.lddw, n);
    };
    bool done = false;
    for (int b = i0; b < i1 && !done; b += 64) {
        const int cnt = imin(i1 - b, 64);
        const uint32_t keys = lane < cnt ? a.key[b + lane] : (uint32_t)a.V;
        const uint32_t ats = lane < cnt ? a.at[b + lane] : 0;
        const int live = __popcll(__ballot((int)keys < a.V));  // the others sorted behind all rows
        for (int u = 0; u < live; u += AHEAD) {
            E x[AHEAD][VEC<E>];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)ats, imin(u + q, live - 1));
                load_row(x[q], dY + row * a.lddy, n);
            }
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
                if (u + q < live) {
                    const int k = __builtin_amdgcn_readlane((int)keys, u + q);
                    close_before(k);
#pragma unroll
                    for (int e = 0; e < VEC<E>; ++e)
                        acc[e] += (float)x[q][e];
                    some = true;
                }
        }
        done = live < cnt;
    }
    close_before(v1);
    if (some)  // row v goes on in the next piece
        part(a.tail);
}

// A row that several pieces share: their parts in order.  A workgroup takes
// JOIN pieces' ends; a wave adds up a row of few parts by itself, all of them a
// long one, in WALK_WAVES runs of parts.
constexpr int JOIN = 4, LONG_ROW = 16;
template <typename E>
__global__ __launch_bounds__(WALK_THREADS) void embedding_join_kernel(WalkArgs a)
{
    __shared__ float runs[WALK_WAVES][64 * VEC<E>];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int group = (int)(blockIdx.x / a.segments), segment = (int)(blockIdx.x % a.segments);
    const int64_t c = ((int64_t)segment * 64 + lane) * VEC<E>;
    const int n = c < a.K ? (int)(a.K - c < VEC<E> ? a.K - c : VEC<E>) : 0;
    const int end = group * JOIN + (lane < JOIN ? lane : 0);
    const int2 mine = lane < JOIN && end < a.pieces ? a.carried[end] : make_int2(-1, 0);
    const auto add = [&](float (&acc)[VEC<E>], const float *from, int64_t piece) {
        const float *p = from + piece * a.K + c;
        float x[VEC<E>] = {};
        if (n == VEC<E>)
            __builtin_memcpy(x, p, sizeof x);
        else
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
                x[e] = e < n ? p[e] : 0.0f;
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            acc[e] += x[e];
    };
    const auto finish = [&](const float (&acc)[VEC<E>], int row) {
        E x[VEC<E>];
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            x[e] = (E)(acc[e] * a.scale);
        store_row(x, reinterpret_cast<E *>(a.dW) + (int64_t)row * a.lddw + c, n);
    };
    const uint64_t short_rows = __ballot(mine.x >= 0 && end - mine.y <= LONG_ROW);
    const uint64_t long_rows = __ballot(mine.x >= 0 && end - mine.y > LONG_ROW);
    for (int j = wave; j < JOIN; j += WALK_WAVES) {
        if (!(short_rows >> j & 1))
            continue;
        const int row = __builtin_amdgcn_readlane(mine.x, j), first = __builtin_amdgcn_readlane(mine.y, j);
        const int last = group * JOIN + j;
        float acc[VEC<E>] = {};
#pragma unroll 4
        for (int p = first; p < last; ++p)
            add(acc, a.tail, p);
        add(acc, a.head, last);
        finish(acc, row);
    }
    for (uint64_t left = long_rows; left; left &= left - 1) {
        const int j = __builtin_ctzll(left);
        const int row = __builtin_amdgcn_readlane(mine.x, j), first = __builtin_amdgcn_readlane(mine.y, j);
        const int last = group * JOIN + j, len = (last - first + WALK_WAVES - 1) / WALK_WAVES;
        float acc[VEC<E>] = {};
        const int from = first + wave * len, to = imin(from + len, last);
#pragma unroll 8
        for (int p = from; p < to; ++p)
            add(acc, a.tail, p);
        if (wave == WALK_WAVES - 1)
            add(acc, a.head, last);
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            runs[wave][e * 64 + lane] = acc[e];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
#pragma unroll
                for (int w = 1; w < WALK_WAVES; ++w)
                    acc[e] += runs[w][e * 64 + lane];
            finish(acc, row);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host
constexpr int64_t LIMIT = (int64_t)1 << 31, MOST = (int64_t)1 << 40;

template <typename E>
int lookup(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K, int64_t ldw, int64_t ldy,
           float scale, void *stream)
{
    if (M < 0 || V < 0 || K < 0 || (V > 1 && ldw < K) || (M > 1 && ldy < K))
        return TG_ERR_INVALID_ARG;
    if (M >= LIMIT || V >= LIMIT || K >= LIMIT || (V > 1 && ldw >= LIMIT) || (M > 1 && ldy >= LIMIT) || M * K >= MOST)
        return TG_ERR_TOO_LARGE;
    if (M == 0 || K == 0)
        return TG_OK;
    if (!tokens || !Y || (V > 0 && !W) || (uintptr_t)tokens % 8 || (uintptr_t)W % sizeof(E) || (uintptr_t)Y % sizeof(E))
        return TG_ERR_INVALID_ARG;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    LookArgs a = {tokens, W, Y, M, V, K, V > 1 ? ldw : 0, M > 1 ? ldy : 0, 0, scale};
    a.segments = (int)cdiv(K, 64 * LOOK_STEPS * VEC<E>);
    const int64_t grid = std::min(cdiv(M * a.segments, LOOK_THREADS / 64), (int64_t)1 << 20);
    const bool ok = M * K * (int64_t)sizeof(E) >= NT_BYTES ? launch(embedding_kernel<E, true>, grid, LOOK_THREADS, stream, a)
                                                           : launch(embedding_kernel<E, false>, grid, LOOK_THREADS, stream, a);
    return ok ? TG_OK : TG_ERR_LAUNCH;
}

// Of more workgroups than these, sums over their counts are made once, by a kernel of its
// own, and not by each of them.  Without and with it: 2^20 tokens of 256 columns (128
// workgroups) 704 and 709 us, 200000 of 1024 (196) 317 and 310, 2^22 of 64 (512) 2465 and
// 2448, 2^24 (2048) 9093 and 8720; what it saves grows with the square.
constexpr int SCAN_TILES = 128;
struct Plan {
    int passes, bits, tiles, threads;  // of the sort
    int piece, pieces;       // of the walk
    int64_t key, at, key2, at2, count, carried, head, tail, bytes;  // offsets in the workspace
};
// (M + V: the walk counts tokens 64 at a time in 32 bits, up to one step past the last)
int validate(int64_t M, int64_t V, int64_t K)
{
    if (M < 0 || V < 0 || K < 0)
        return TG_ERR_INVALID_ARG;
    return M >= LIMIT || V >= LIMIT || K >= LIMIT || M + V >= LIMIT - 64 || (M + V) * K >= MOST ? TG_ERR_TOO_LARGE : TG_OK;
}
// Pieces of 32 items where there are few, of 64 otherwise (with gradient: 333 tokens
// on 50001×1000 fp32 70 us with 32, 80 with 64; 65536 on 32000×2048 fp16 238 and 219,
// where every piece leaves two rows of fp32 sums; 128 are slower everywhere).  More
// only to keep the launch within its limit.
Plan make_plan(int64_t M, int64_t V, int64_t K)
{
    Plan p = {};
    int bits = 1;
    while ((int64_t)1 << bits < V + 1)
        ++bits;
    p.passes = (int)cdiv(bits, DIGIT_BITS);
    p.bits = (int)cdiv(bits, p.passes);
    // small workgroups spread a short sort over the chip; a long one takes large ones
    p.threads = M <= SORT_SMALL || M > 256 * FEW * sort_per(FEW) ? MANY : FEW;
    p.tiles = (int)cdiv(M, p.threads * sort_per(p.threads));
    const int64_t segments = cdiv(K, 64 * 4);  // of the widest type
    p.piece = cdiv(M + V, 32) * segments <= 16384 ? 32 : 64;
    while (p.piece < 256 && cdiv(M + V, p.piece) * segments > (int64_t)1 << 22)
        p.piece *= 2;
    p.pieces = (int)cdiv(M + V, p.piece);
    int64_t used = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t at = used;
        used += round_up(bytes, 256);
        return at;
    };
    p.key = take(4 * M), p.at = take(4 * M);
    if (p.tiles > 1) {
        p.key2 = take(4 * M), p.at2 = take(4 * M);
        p.count = take((int64_t)4 * DIGITS * (p.tiles + 1));
    }
    p.carried = take((int64_t)8 * p.pieces);
    if (M > 0) {
        p.head = take((int64_t)4 * p.pieces * K);
        p.tail = take((int64_t)4 * p.pieces * K);
    }
    p.bytes = used;
    return p;
}

template <typename E>
int gradient(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K, int64_t lddy,
             int64_t lddw, float scale, int64_t padding, void *ws, int64_t ws_bytes, void *stream)
{
    const int st = validate(M, V, K);
    if (st == TG_ERR_INVALID_ARG || (M > 1 && lddy < K) || (V > 1 && lddw < K))
        return TG_ERR_INVALID_ARG;
    if (st != TG_OK || (M > 1 && lddy >= LIMIT) || (V > 1 && lddw >= LIMIT))
        return TG_ERR_TOO_LARGE;
    if (V == 0 || K == 0)
        return TG_OK;
    const Plan p = make_plan(M, V, K);
    if (!dW || (uintptr_t)dW % sizeof(E) || (M > 0 && (!tokens || !dY || (uintptr_t)tokens % 8 || (uintptr_t)dY % sizeof(E))) ||
        !ws || (uintptr_t)ws % 256 || ws_bytes < p.bytes)
        return TG_ERR_INVALID_ARG;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    char *const base = reinterpret_cast<char *>(ws);
    const auto words = [&](int64_t at) { return reinterpret_cast<uint32_t *>(base + at); };
    bool ok = true;
    SortArgs s = {};
    s.tokens = tokens, s.M = (int)M, s.V = (int)V, s.padding = padding;
    s.key = words(p.key), s.at = words(p.at);
    s.tiles = p.tiles, s.bits = p.bits, s.passes = p.passes;
    if (p.tiles == 1) {
        ok = launch(sort_small_kernel, 1, MANY, stream, s);
    } else if (p.tiles > 1) {
        s.count = words(p.count);
        s.scanned = p.tiles > SCAN_TILES;
        const auto pass = [&](auto threads, auto first) {
            constexpr int T = decltype(threads)::value;
            constexpr bool F = decltype(first)::value;
            return launch(sort_count_kernel<T, F>, p.tiles, T, stream, s) &&
                   (!s.scanned || launch(sort_scan_kernel, DIGITS / SCAN_DIGITS, 1024, stream, s)) &&
                   launch(sort_scatter_kernel<T, F>, p.tiles, T, stream, s);
        };
        // the pairs go back and forth so that the last pass ends in (key, at)
        for (int q = 0; ok && q < p.passes; ++q) {
            const bool to_first = (p.passes - 1 - q) % 2 == 0;
            s.key = words(to_first ? p.key : p.key2), s.at = words(to_first ? p.at : p.at2);
            s.key_in = words(to_first ? p.key2 : p.key), s.at_in = words(to_first ? p.at2 : p.at);
            s.shift = p.bits * q;
            if (p.threads == FEW)
                ok = q == 0 ? pass(std::integral_constant<int, FEW>{}, std::true_type{})
                            : pass(std::integral_constant<int, FEW>{}, std::false_type{});
            else
                ok = q == 0 ? pass(std::integral_constant<int, MANY>{}, std::true_type{})
                            : pass(std::integral_constant<int, MANY>{}, std::false_type{});
        }
    }
    WalkArgs w = {};
    w.key = words(p.key), w.at = words(p.at);
    w.dY = dY, w.dW = dW, w.M = (int)M, w.V = (int)V, w.K = K;
    w.lddy = M > 1 ? lddy : 0, w.lddw = V > 1 ? lddw : 0;
    w.piece = p.piece, w.pieces = p.pieces, w.segments = (int)cdiv(K, 64 * VEC<E>);
    w.scale = scale;
    w.carried = reinterpret_cast<int2 *>(base + p.carried);
    w.head = reinterpret_cast<float *>(base + p.head), w.tail = reinterpret_cast<float *>(base + p.tail);
    ok = ok && launch(embedding_walk_kernel<E>, cdiv((int64_t)p.pieces * w.segments, WALK_WAVES), WALK_THREADS, stream, w);
    if (M > 0)  // a single token, too, may lie in the piece before its row's
        ok = ok && launch(embedding_join_kernel<E>, cdiv(p.pieces, JOIN) * w.segments, WALK_THREADS, stream, w);
    return ok ? TG_OK : TG_ERR_LAUNCH;
}
}  // namespace

extern "C" int tg_embedding_f32(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K,
                                int64_t ldw, int64_t ldy, float scale, void *stream)
{
    return lookup<float>(tokens, W, Y, M, V, K, ldw, ldy, scale, stream);
}

extern "C" int tg_embedding_f16(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K,
                                int64_t ldw, int64_t ldy, float scale, void *stream)
{
    return lookup<_Float16>(tokens, W, Y, M, V, K, ldw, ldy, scale, stream);
}

extern "C" int tg_embedding_bf16(const int64_t *tokens, const void *W, void *Y, int64_t M, int64_t V, int64_t K,
                                 int64_t ldw, int64_t ldy, float scale, void *stream)
{
    return lookup<__bf16>(tokens, W, Y, M, V, K, ldw, ldy, scale, stream);
}

extern "C" int64_t tg_embedding_bwd_workspace_bytes(int64_t M, int64_t V, int64_t K)
{
    if (validate(M, V, K) != TG_OK)
        return -1;
    return V == 0 || K == 0 ? 0 : make_plan(M, V, K).bytes;
}

extern "C" int tg_embedding_bwd_f32(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K,
                                    int64_t lddy, int64_t lddw, float scale, int64_t padding, void *workspace,
                                    int64_t workspace_bytes, void *stream)
{
    return gradient<float>(tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace, workspace_bytes, stream);
}

extern "C" int tg_embedding_bwd_f16(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K,
                                    int64_t lddy, int64_t lddw, float scale, int64_t padding, void *workspace,
                                    int64_t workspace_bytes, void *stream)
{
    return gradient<_Float16>(tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace, workspace_bytes, stream);
}

extern "C" int tg_embedding_bwd_bf16(const int64_t *tokens, const void *dY, void *dW, int64_t M, int64_t V, int64_t K,
                                     int64_t lddy, int64_t lddw, float scale, int64_t padding, void *workspace,
                                     int64_t workspace_bytes, void *stream)
{
    return gradient<__bf16>(tokens, dY, dW, M, V, K, lddy, lddw, scale, padding, workspace, workspace_bytes, stream);
}
