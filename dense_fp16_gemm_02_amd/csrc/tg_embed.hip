// tg_embed.hip — embedding lookup and its gradient.  See include/tg_embed.h for
// the contract.
//
// The lookup copies rows, 16 bytes a lane.
//
// The gradient sorts the tokens (a stable radix sort of (token, row of dY)
// pairs, 8 bits a pass) and walks two sorted lists at once, the sorted tokens and
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

// 16 bytes at the alignment of an element, `n` elements of them inside the row
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
template <typename E>
__device__ inline void store_row(const E (&x)[VEC<E>], E *p, int n)
{
    if (n >= VEC<E>) {
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
// A wave takes LOOK_STEPS·64 lanes of one row.
template <typename E>
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
            load_row(x[k], src + c, in && c < a.K ? (int)imin((int)(a.K - c), VEC<E>) : 0);
        }
#pragma unroll
        for (int k = 0; k < LOOK_STEPS; ++k) {
            const int64_t c = c0 + k * (64 * VEC<E>);
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
                x[k][e] = in ? (E)((float)x[k][e] * a.scale) : (E)NAN;
            if (c < a.K)
                store_row(x[k], dst + c, (int)imin((int)(a.K - c), VEC<E>));
        }
    }
}

// -------------------------------------------------------------------- sort
constexpr int SORT_THREADS = 1024, SORT_WAVES = SORT_THREADS / 64, SORT_PER = 8;
constexpr int SORT_TILE = SORT_THREADS * SORT_PER;  // pairs of a workgroup
constexpr int DIGITS = 256;
struct SortArgs {
    const int64_t *tokens;          // first pass
    const uint32_t *key_in, *at_in; // later passes
    uint32_t *key, *at;
    uint32_t *count;                // [digit][workgroup]
    int M, V;
    int64_t padding;
    int tiles, shift, passes;
};
// A token that adds to no row sorts behind all rows.
__device__ inline uint32_t token_key(const SortArgs &a, int i)
{
    const int64_t t = a.tokens[i];
    return t >= 0 && t < a.V && t != a.padding ? (uint32_t)t : (uint32_t)a.V;
}
// Item r of this lane: a wave's items are consecutive, 64 to a round.
__device__ inline int sort_item(int wave, int lane, int r) { return wave * (64 * SORT_PER) + r * 64 + lane; }

struct SortShared {
    uint32_t wave_count[SORT_WAVES][DIGITS];  // of a digit in a wave, then where the wave's first of it goes
    uint32_t wave_sum[SORT_WAVES];
    uint32_t base[DIGITS];
};
// For each of this lane's items its place among the workgroup's items, ordered
// by digit and, within one, as they came.  Lanes of a wave that hold the same
// digit find each other with one ballot per bit.
__device__ inline void sort_places(SortShared &s, const uint32_t (&key)[SORT_PER], int items, int shift,
                                   uint32_t (&place)[SORT_PER])
{
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    for (int d = lane; d < DIGITS; d += 64)
        s.wave_count[wave][d] = 0;
    __builtin_amdgcn_wave_barrier();
    volatile uint32_t *mine = s.wave_count[wave];
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r) {
        const bool live = sort_item(wave, lane, r) < items;
        const uint32_t d = (key[r] >> shift) & (DIGITS - 1);
        uint64_t same = __ballot(live);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const uint64_t set = __ballot((d >> b) & 1);
            same &= (d >> b) & 1 ? set : ~set;
        }
        const uint32_t before = (uint32_t)__popcll(same & ((1ull << lane) - 1));
        const uint32_t seen = mine[d];
        __builtin_amdgcn_wave_barrier();
        if (live && before == 0)
            mine[d] = seen + (uint32_t)__popcll(same);
        __builtin_amdgcn_wave_barrier();
        place[r] = seen + before;
    }
    __syncthreads();
    // exclusive sums over (digit, wave), four waves of one digit to a thread
    constexpr int QUADS = SORT_WAVES / 4;
    static_assert(DIGITS * QUADS == SORT_THREADS, "a thread for four counts");
    const int d = tid / QUADS, w0 = 4 * (tid % QUADS);
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        c[w] = s.wave_count[w0 + w][d];
        sum += c[w];
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t x = __shfl_up(upto, o);
        upto += lane >= o ? x : 0;
    }
    if (lane == 63)
        s.wave_sum[wave] = upto;
    __syncthreads();
    uint32_t at = upto - sum;
    for (int w = 0; w < wave; ++w)
        at += s.wave_sum[w];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        s.wave_count[w0 + w][d] = at;
        at += c[w];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r)
        place[r] += s.wave_count[wave][(key[r] >> shift) & (DIGITS - 1)];
}

// All passes of at most SORT_TILE tokens, by one workgroup.
__global__ __launch_bounds__(SORT_THREADS) void sort_small_kernel(SortArgs a)
{
    __shared__ SortShared s;
    __shared__ uint32_t keys[SORT_TILE], ats[SORT_TILE];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    uint32_t key[SORT_PER], at[SORT_PER], place[SORT_PER];
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r) {
        const int i = sort_item(wave, lane, r);
        key[r] = i < a.M ? token_key(a, i) : 0;
        at[r] = (uint32_t)i;
    }
    for (int p = 0; p < a.passes; ++p) {
        sort_places(s, key, a.M, 8 * p, place);
#pragma unroll
        for (int r = 0; r < SORT_PER; ++r)
            if (sort_item(wave, lane, r) < a.M) {
                keys[place[r]] = key[r];
                ats[place[r]] = at[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < SORT_PER; ++r) {
            const int i = sort_item(wave, lane, r);
            if (i < a.M) {
                key[r] = keys[i];
                at[r] = ats[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r) {
        const int i = sort_item(wave, lane, r);
        if (i < a.M) {
            a.key[i] = key[r];
            a.at[i] = at[r];
        }
    }
}

// How often each digit occurs in each workgroup's pairs.
template <bool FIRST>
__global__ __launch_bounds__(SORT_THREADS) void sort_count_kernel(SortArgs a)
{
    __shared__ uint32_t count[DIGITS];
    const int tid = threadIdx.x;
    if (tid < DIGITS)
        count[tid] = 0;
    __syncthreads();
    const int i0 = (int)blockIdx.x * SORT_TILE;
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r) {
        const int i = i0 + r * SORT_THREADS + tid;
        if (i < a.M)
            atomicAdd(&count[((FIRST ? token_key(a, i) : a.key_in[i]) >> a.shift) & (DIGITS - 1)], 1u);
    }
    __syncthreads();
    if (tid < DIGITS)
        a.count[(int64_t)tid * a.tiles + blockIdx.x] = count[tid];
}
// One pass: each pair to its place.
template <bool FIRST>
__global__ __launch_bounds__(SORT_THREADS) void sort_scatter_kernel(SortArgs a)
{
    __shared__ SortShared s;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int i0 = (int)blockIdx.x * SORT_TILE, items = imin(a.M - i0, SORT_TILE);
    uint32_t key[SORT_PER], at[SORT_PER], place[SORT_PER];
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r) {
        const int i = sort_item(wave, lane, r);
        key[r] = i < items ? (FIRST ? token_key(a, i0 + i) : a.key_in[i0 + i]) : 0;
        at[r] = i < items ? (FIRST ? (uint32_t)(i0 + i) : a.at_in[i0 + i]) : 0;
    }
    // where this workgroup's first pair of each digit goes: behind all pairs of
    // smaller digits, and those of its digit in the workgroups before
    constexpr int PARTS = SORT_THREADS / DIGITS;
    const int d = tid / PARTS, part = tid % PARTS;
    uint32_t all = 0, before = 0;
    const uint32_t *row = a.count + (int64_t)d * a.tiles;
    for (int b = part; b < a.tiles; b += PARTS) {
        const uint32_t c = row[b];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
    }
#pragma unroll
    for (int o = 1; o < PARTS; o <<= 1) {
        all += __shfl_xor(all, o);
        before += __shfl_xor(before, o);
    }
    uint32_t upto = part == PARTS - 1 ? all : 0;
    const uint32_t own = upto;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t x = __shfl_up(upto, o);
        upto += lane >= o ? x : 0;
    }
    if (lane == 63)
        s.wave_sum[wave] = upto;
    __syncthreads();
    uint32_t base = upto - own + before;
    for (int w = 0; w < wave; ++w)
        base += s.wave_sum[w];
    if (part == PARTS - 1)
        s.base[d] = base;
    __syncthreads();
    sort_places(s, key, items, a.shift, place);
    // (behind sort_places wave_count[0][d] is the digit's first place in the workgroup)
#pragma unroll
    for (int r = 0; r < SORT_PER; ++r)
        if (sort_item(wave, lane, r) < items) {
            const uint32_t dig = (key[r] >> a.shift) & (DIGITS - 1);
            const uint32_t to = s.base[dig] + place[r] - s.wave_count[0][dig];
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
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            if (e < n)
                dst[e] = acc[e];
    };
    const auto close = [&] {  // row v ends
        if (v == open) {
            part(a.head);
        } else {
            E x[VEC<E>];
#pragma unroll
            for (int e = 0; e < VEC<E>; ++e)
                x[e] = some ? (E)(acc[e] * a.scale) : (E)0.0f;
            store_row(x, dW + (int64_t)v * a.lddw, n);
        }
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            acc[e] = 0.0f;
        some = false;
        ++v;
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
                    while (v < k)
                        close();
#pragma unroll
                    for (int e = 0; e < VEC<E>; ++e)
                        acc[e] += (float)x[q][e];
                    some = true;
                }
        }
        done = live < cnt;
    }
    while (v < v1)
        close();
    if (some)  // row v goes on in the next piece
        part(a.tail);
}

// A row that several pieces share: their parts in order.  A workgroup takes
// JOIN pieces' ends; a wave adds up a row of few parts by itself, all of them a
// long one, in WALK_WAVES runs of parts.
constexpr int JOIN = 16, LONG_ROW = 32;
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
#pragma unroll
        for (int e = 0; e < VEC<E>; ++e)
            acc[e] += e < n ? p[e] : 0.0f;
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
    return launch(embedding_kernel<E>, grid, LOOK_THREADS, stream, a) ? TG_OK : TG_ERR_LAUNCH;
}

struct Plan {
    int passes, tiles;       // of the sort
    int piece, pieces;       // of the walk
    int64_t key, at, key2, at2, count, carried, head, tail, bytes;  // offsets in the workspace
};
int validate(int64_t M, int64_t V, int64_t K)
{
    if (M < 0 || V < 0 || K < 0)
        return TG_ERR_INVALID_ARG;
    return M >= LIMIT || V >= LIMIT || K >= LIMIT || M + V >= LIMIT || (M + V) * K >= MOST ? TG_ERR_TOO_LARGE : TG_OK;
}
// Pieces of 32 items where there are few, so that some 32768 waves share the work; of
// up to 256 where there are many, as every piece has room for two rows of fp32 sums.
Plan make_plan(int64_t M, int64_t V, int64_t K)
{
    Plan p = {};
    for (int64_t keys = V + 1; keys > 1; keys = cdiv(keys, DIGITS))
        ++p.passes;
    p.tiles = (int)cdiv(M, SORT_TILE);
    const int64_t segments = cdiv(K, 64 * 4);  // of the widest type
    p.piece = 32;
    while (p.piece < 256 && cdiv(M + V, p.piece) * segments > 65536)
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
        p.count = take((int64_t)4 * DIGITS * p.tiles);
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
    SortArgs s = {tokens, nullptr, nullptr, words(p.key), words(p.at), nullptr, (int)M, (int)V, padding, p.tiles, 0, p.passes};
    if (p.tiles == 1) {
        ok = launch(sort_small_kernel, 1, SORT_THREADS, stream, s);
    } else if (p.tiles > 1) {
        s.count = words(p.count);
        // the pairs go back and forth so that the last pass ends in (key, at)
        for (int q = 0; ok && q < p.passes; ++q) {
            const bool to_first = (p.passes - 1 - q) % 2 == 0;
            s.key = words(to_first ? p.key : p.key2), s.at = words(to_first ? p.at : p.at2);
            s.key_in = words(to_first ? p.key2 : p.key), s.at_in = words(to_first ? p.at2 : p.at);
            s.shift = 8 * q;
            ok = q == 0 ? launch(sort_count_kernel<true>, p.tiles, SORT_THREADS, stream, s) &&
                              launch(sort_scatter_kernel<true>, p.tiles, SORT_THREADS, stream, s)
                        : launch(sort_count_kernel<false>, p.tiles, SORT_THREADS, stream, s) &&
                              launch(sort_scatter_kernel<false>, p.tiles, SORT_THREADS, stream, s);
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
    if (M > 1)
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
