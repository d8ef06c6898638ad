// tg_xent.hip — softmax cross entropy of the vocabulary projection and its
// gradients.  See include/tg_xent.h for the contract.
//
// Forward: the logits tile z = H·Wᵀ stays in the accumulators; per row of a tile
// the kernel keeps only the maximum m and s = Σ exp(z − m), so M·V logits
// shrink to M·(V/256) pairs.  Two pairs join as
// m = max(m1, m2), s = s1·exp(m1 − m) + s2·exp(m2 − m); a second kernel joins a
// row's pairs and subtracts the target's logit, which the one lane that held
// it has written out.
//
// Backward, per piece of the vocabulary: the logits tile is computed again and
// turned into G = c·exp(z − lse) − c'·[target] while it is in registers (no
// second pass for the softmax: lse is known); then dH += G·W and dW = Gᵀ·H take
// G, W and H as they lie, through transposed LDS reads.
//
// Tokens that are ignored are taken out first: the rows of H that count are
// gathered, so that a batch of mostly masked tokens costs what its live tokens
// cost, and whatever the ignored rows hold (NaN included) reaches nothing.
#include "proj_tile.hpp"

#include <algorithm>
#include <math.h>
#include <stdio.h>

#include "tg_gemm.h"
#include "tg_xent.h"

namespace {
using namespace pt;

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

// What the first kernel finds out, at the start of a workspace.
struct Head {
    int live;          // tokens not ignored
    float alpha;       // what G was divided by (backward)
    unsigned arrived;  // workgroups of the join that are done (forward)
};

// G is stored in the operands' type; binary16 stores it times 2^14, bfloat16 as
// it is (its exponent range holds any probability of note).
template <typename E>
constexpr float g_scale()
{
    return std::is_same_v<E, _Float16> ? 16384.0f : 1.0f;
}

// exp through the hardware's base-2 exponential (1 ulp)
__device__ inline float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }

// ------------------------------------------------------------------ gather
// Numbers the live tokens and copies their rows of H to consecutive rows, K
// columns padded with zeros to K8; for the backward pass also each live token's
// coefficients, and zeros for the ignored tokens' rows of dH.  A workgroup counts
// the live tokens before its own itself (8·M bytes from the caches): one launch,
// no pass over the targets in between.  So there are at most two workgroups to a
// compute unit, which take their tokens PREP_ROWS at a time.
constexpr int PREP_THREADS = 256, PREP_ROWS = 256;
struct PrepArgs {
    const int64_t *target;
    int64_t M, V, ignore;
    int rows;        // tokens per workgroup
    Head *head;
    int *map;        // live row -> token
    int *col;        // live row -> target, -1 if out of range
    float *loss;     // per-token loss and lse: zeroed for ignored tokens
    float *lse_out;
    const uint16_t *H;
    int64_t ldh;
    uint16_t *hc;
    int64_t K, K8;
    bool vec;        // 16-byte aligned rows of H, K % 8 == 0
    // backward
    int reduction;
    const float *dloss, *dlse, *lse;
    float *lse_c, *cp, *ct;  // per live row: lse, and the coefficients of the softmax and of the target
    uint16_t *dH;
    int64_t lddh;
};
template <typename X>
__device__ inline X wave_sum(X x)
{
    for (int o = 32; o; o >>= 1)
        x += __shfl_xor(x, o);
    return x;
}
template <bool BWD>
__global__ __launch_bounds__(PREP_THREADS) void xent_prep_kernel(PrepArgs a)
{
    constexpr int WAVES = PREP_THREADS / 64;
    __shared__ int before_w[WAVES], all_w[WAVES];
    __shared__ float top_w[WAVES];
    __shared__ int place[PREP_ROWS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t r0 = (int64_t)blockIdx.x * a.rows;
    const int rows = (int)(a.M - r0 < a.rows ? a.M - r0 : a.rows);
    int before = 0, all = 0;
#pragma unroll 8
    for (int64_t i = tid; i < a.M; i += PREP_THREADS) {
        const int live = a.target[i] != a.ignore;
        all += live;
        before += i < r0 ? live : 0;
    }
    before = wave_sum(before), all = wave_sum(all);
    if (lane == 0)
        before_w[wave] = before, all_w[wave] = all;
    __syncthreads();
    before = all = 0;
    for (int w = 0; w < WAVES; ++w)
        before += before_w[w], all += all_w[w];
    float scale = 1.0f, top = 0.0f;
    if constexpr (BWD) {
        if (a.reduction == TG_XENT_MEAN)
            scale = 1.0f / (float)imax(all, 1);
        // the largest coefficient (a NaN or an infinity among them reaches its own
        // row through its coefficient, not the others through the maximum)
        const auto size = [](float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.0f; };
        if (a.reduction != TG_XENT_NONE && !a.dlse) {
            top = size(a.dloss[0] * scale);
        } else {
            for (int64_t i = tid; i < a.M; i += PREP_THREADS)
                if (a.target[i] != a.ignore) {
                    const float g = (a.reduction == TG_XENT_NONE ? a.dloss[i] : a.dloss[0]) * scale;
                    top = fmaxf(top, fmaxf(size(g), a.dlse ? size(g + a.dlse[i]) : 0.0f));
                }
            for (int o = 32; o; o >>= 1)
                top = fmaxf(top, __shfl_xor(top, o));
            if (lane == 0)
                top_w[wave] = top;
            __syncthreads();
            for (int w = 0; w < WAVES; ++w)
                top = fmaxf(top, top_w[w]);
        }
        if (!(top > 0.0f))
            top = 1.0f;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.head->live = all;
        a.head->alpha = top;
    }
    const int per = (int)(a.K8 / 8);
    for (int64_t first = r0; first < r0 + rows; first += PREP_ROWS) {
        const int n = (int)(r0 + rows - first < PREP_ROWS ? r0 + rows - first : PREP_ROWS);
        // numbered 64 at a time by the first wave
        if (wave == 0)
            for (int c = 0; c < n; c += 64) {
                const int64_t i = first + c + lane;
                const int64_t t = c + lane < n ? a.target[i] : a.ignore;
                const bool live = c + lane < n && t != a.ignore;
                const unsigned long long votes = __ballot(live);
                const int at = before + __popcll(votes & ((1ull << lane) - 1));
                before += __popcll(votes);
                if (c + lane >= n)
                    continue;
                place[c + lane] = live ? at : -1;
                if (live) {
                    const bool in = t >= 0 && t < a.V;
                    a.map[at] = (int)i;
                    a.col[at] = in ? (int)t : -1;
                    if constexpr (BWD) {
                        const float g = (a.reduction == TG_XENT_NONE ? a.dloss[i] : a.dloss[0]) * scale;
                        a.lse_c[at] = a.lse[i];
                        a.cp[at] = in ? (g + (a.dlse ? a.dlse[i] : 0.0f)) / top : NAN;
                        a.ct[at] = g / top;
                    }
                } else if constexpr (!BWD) {
                    if (a.loss)
                        a.loss[i] = 0.0f;
                    if (a.lse_out)
                        a.lse_out[i] = 0.0f;
                }
            }
        __syncthreads();
        for (int r = wave; r < n; r += WAVES) {
            const int at = place[r];
            if (at >= 0) {
                const uint16_t *src = a.H + (first + r) * a.ldh;
                uint4 *dst = reinterpret_cast<uint4 *>(a.hc + at * a.K8);
#pragma unroll 4
                for (int c = lane; c < per; c += 64)
                    dst[c] = load8(src, 8 * (int64_t)c, a.K, a.vec);
            } else if (BWD && a.dH) {
                uint16_t *dst = a.dH + (first + r) * a.lddh;
                for (int64_t c = lane; c < a.K; c += 64)
                    dst[c] = 0;
            }
        }
        __syncthreads();  // every wave has read `place`
    }
}

// Rows of W padded with zeros to K8 columns (W whose rows are not aligned).  Bound
// by memory: with nothing of W in the caches 60000×2047 in 138 us (492 MB, 3.6 TB/s;
// 164 with loads of one element each), 20000×1001 in 23 (31).
__global__ __launch_bounds__(256) void xent_pack_kernel(const uint16_t *src, int64_t ld, uint16_t *dst, int64_t rows,
                                                        int64_t K, int64_t K8)
{
    const int64_t per = K8 / 8, total = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        *reinterpret_cast<uint4 *>(dst + r * K8 + c) = load8(src + r * ld, c, K, false);
    }
}
// dW, and the total, of no tokens
__global__ __launch_bounds__(256) void xent_zero_kernel(uint16_t *dst, int64_t ld, int64_t rows, int64_t cols)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256)
            dst[r * ld + c] = 0;
}

// ---------------------------------------------------------- logits, forward
// One workgroup per BM×BN block of logits.  Bound by the matrix cores (the
// epilogue's BM·BN/256 exponentials per lane cost some 5% of a K = 4096 block),
// or for few tokens by streaming W.
struct StatsArgs {
    Operand h, w;
    int K, M;           // M: rows of h, or an upper bound where head is given
    const Head *head;   // live rows (null: all M)
    int V, v0;          // columns of this piece, its first vocabulary entry
    const int *col;     // live row -> target (compacted rows)
    const int64_t *target;
    int64_t Vall;
    float2 *part;       // [column of tiles][row]
    int64_t part_ld;
    float *at_target;   // row -> logit of its target
    unsigned *arrived;  // for the join
    int tiles_n;
};
__device__ inline void join(float2 &a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    const float from = m == -INFINITY ? 0.0f : m;
    // a NaN in either sum stays one
    a.y = a.y * fast_exp(a.x - from) + b.y * fast_exp(b.x - from);
    a.x = m;
}
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void xent_stats_kernel(
    StatsArgs a)
{
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const int M = a.head ? a.head->live : a.M;
    const int tiles_m = (M + T::BM - 1) / T::BM, total = tiles_m * a.tiles_n;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *a.arrived = 0;
    if ((int)blockIdx.x >= total)
        return;
    int tm, tn;
    grouped_tile<4>(xcd_contiguous(blockIdx.x, total), tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    Operand h = a.h;
    h.extent = M;
    T::run(smem, h, a.w, m0, n0, a.K, acc);

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int row0 = m0 + wm * T::WTM + (lane & 15);
    const int col0 = n0 + wn * T::WTN + 4 * (lane >> 4);
    const bool whole = n0 + wn * T::WTN + T::WTN <= a.V;
    barrier_lds();
    float2 *pairs = reinterpret_cast<float2 *>(smem);  // [WN][BM]
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
        const int row = row0 + 16 * i;
        int at = -1;
        if (row < M) {
            if (a.col) {
                at = a.col[row];
            } else {
                const int64_t t = a.target[row];
                at = t >= 0 && t < a.Vall ? (int)t : -1;
            }
        }
        at -= a.v0;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (col0 + 16 * j + v >= a.V)
                        acc[i][j][v] = -INFINITY;
        }
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                m = fmaxf(m, acc[i][j][v]);
                if (col0 + 16 * j + v == at)
                    a.at_target[row] = acc[i][j][v];
            }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float from = m == -INFINITY ? 0.0f : m;  // nothing but −∞: the sum is 0, not NaN
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                s += fast_exp(acc[i][j][v] - from);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lane < 16)
            pairs[wn * T::BM + wm * T::WTM + 16 * i + lane] = make_float2(m, s);
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r < T::BM && m0 + r < M) {
        float2 p = pairs[r];
#pragma unroll
        for (int w = 1; w < T::WN; ++w)
            join(p, pairs[w * T::BM + r]);
        a.part[(int64_t)(a.v0 / T::BN + tn) * a.part_ld + m0 + r] = p;
    }
}

// Joins each row's pairs: 16 rows per workgroup, 64 threads to a row, which take
// every 64th tile.  Reads 8·M bytes per column of tiles, 128 at a time.  For SUM
// and MEAN each workgroup leaves its own sum, and the one that arrives last adds
// them all, in their order: which one that is changes nothing in the result.
constexpr int JOIN_ROWS = 16;
struct JoinArgs {
    const float2 *part;
    int64_t part_ld;
    int tiles, M, reduction;  // tiles: columns of tiles, the pairs of a row
    const Head *head;
    const int *map, *col;
    const int64_t *target;
    int64_t V, ignore;
    const float *at_target;
    float *loss, *lse;   // per token (loss null unless TG_XENT_NONE)
    float2 *block_sum;   // per workgroup: sum of losses, tokens counted (null for NONE)
    unsigned *arrived;   // set to 0 by the kernel before
    float *total;
};
__device__ inline float reduced(float sum, float count, int reduction)
{
    return reduction == TG_XENT_MEAN ? sum / fmaxf(count, 1.0f) : sum;
}
__global__ __launch_bounds__(1024) void xent_join_kernel(JoinArgs a)
{
    constexpr int ROWS = JOIN_ROWS, PER_ROW = 1024 / ROWS;
    __shared__ float2 sh[PER_ROW][ROWS];
    __shared__ bool last;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int M = a.head ? a.head->live : a.M;
    const int row = blockIdx.x * ROWS + threadIdx.x % ROWS;
    float2 p = make_float2(-INFINITY, 0.0f);
    if (row < M)
#pragma unroll 4
        for (int s = threadIdx.x / ROWS; s < a.tiles; s += PER_ROW)
            join(p, a.part[(int64_t)s * a.part_ld + row]);
    sh[threadIdx.x / ROWS][threadIdx.x % ROWS] = p;
    __syncthreads();
    if (wave == 0) {
        // four lanes to a row, then across them (a fixed order)
        p = sh[lane / ROWS][lane % ROWS];
#pragma unroll
        for (int w = 64 / ROWS; w < PER_ROW; w += 64 / ROWS)
            join(p, sh[w + lane / ROWS][lane % ROWS]);
#pragma unroll
        for (int o = ROWS; o < 64; o *= 2) {
            const float2 q = make_float2(__shfl_xor(p.x, o), __shfl_xor(p.y, o));
            join(p, q);
        }
        float loss = 0.0f, count = 0.0f;
        if (row < M && lane < ROWS) {
            float lse = p.x + LN2 * __builtin_amdgcn_logf(p.y);
            bool live = true, in;
            if (a.col) {
                in = a.col[row] >= 0;
            } else {
                const int64_t t = a.target[row];
                live = t != a.ignore;
                in = t >= 0 && t < a.V;
            }
            const int out = a.map ? a.map[row] : row;
            if (live) {
                loss = in ? lse - a.at_target[row] : NAN;
                count = 1.0f;
            } else {
                lse = 0.0f;
            }
            if (a.lse)
                a.lse[out] = lse;
            if (a.loss)
                a.loss[out] = loss;
        }
        if (a.block_sum) {
            loss = wave_sum(loss), count = wave_sum(count);
            if (lane == 0) {
                // the sum is out before the arrival is: release at device scope
                float2 *b = a.block_sum + blockIdx.x;
                __hip_atomic_store(&b->x, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                __hip_atomic_store(&b->y, count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                last = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                       gridDim.x - 1;
            }
        }
    }
    if (!a.block_sum)
        return;
    __syncthreads();
    if (!last)
        return;
    __syncthreads();
    float2 s = make_float2(0.0f, 0.0f);
    for (unsigned i = threadIdx.x; i < gridDim.x; i += 1024) {
        s.x += __hip_atomic_load(&a.block_sum[i].x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s.y += __hip_atomic_load(&a.block_sum[i].y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    s.x = wave_sum(s.x), s.y = wave_sum(s.y);
    if (lane == 0)
        sh[wave][0] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) {
            s.x += sh[w][0].x;
            s.y += sh[w][0].y;
        }
        a.total[0] = reduced(s.x, s.y, a.reduction);
    }
}

// --------------------------------------------------------- logits, backward
// G of one piece, live rows × Gld columns (zeros from the piece's width on, to
// a multiple of 64 as the product with W reads it).
struct GradArgs {
    Operand h, w;
    int K;
    const Head *head;
    int V, v0;
    const int *col;
    const float *lse, *cp, *ct;
    void *G;
    int64_t Gld;
    int tiles_n;
};
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void xent_grad_kernel(
    GradArgs a)
{
    using V4 = typename El<E>::v4;
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const int M = a.head->live;
    const int tiles_m = (M + T::BM - 1) / T::BM, total = tiles_m * a.tiles_n;
    if ((int)blockIdx.x >= total)
        return;
    int tm, tn;
    grouped_tile<4>(xcd_contiguous(blockIdx.x, total), tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    Operand h = a.h;
    h.extent = M;
    T::run(smem, h, a.w, m0, n0, a.K, acc);

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    barrier_lds();
    E *stg = smem + wave * T::WTM * T::WTN;
    const int fr = lane & 15, fc = 4 * (lane >> 4);
    const int col0 = n0 + wn * T::WTN + fc;
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
        const int row = m0 + wm * T::WTM + 16 * i + fr;
        float lse = 0.0f, cp = 0.0f, ct = 0.0f;
        int at = -1;
        if (row < M) {
            lse = a.lse[row];
            cp = a.cp[row] * g_scale<E>();
            ct = a.ct[row] * g_scale<E>();
            at = a.col[row] - a.v0;
        }
#pragma unroll
        for (int j = 0; j < T::TN; ++j) {
            V4 g;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int c = col0 + 16 * j + v;
                float x = cp * fast_exp(acc[i][j][v] - lse);
                if (c == at)
                    x -= ct;
                // the one rounding of the gradient's factor (see tg_xent.h)
                g[v] = (E)(c < a.V ? x : 0.0f);
            }
            *reinterpret_cast<V4 *>(stg + stage_off<T::WTN>(16 * i + fr, 16 * j + fc)) = g;
        }
    }
    store_block<E, T::WTM, T::WTN, true>(stg, reinterpret_cast<E *>(a.G), a.Gld, m0 + wm * T::WTM, n0 + wn * T::WTN, M,
                                   (int)a.Gld, true, nullptr, lane);
}

// ------------------------------------------------------------ dH (+)= G·W
// A: G, K-major; B: W of the piece, transposed.  dH has live·K outputs and a
// contraction over the whole vocabulary: fp32 sums, added to what earlier
// pieces left, and where the tiles are few the contraction is split, each split
// with sums of its own.  How many splits is decided here, from the number of
// live tokens, which the host does not know; the last kernel joins them.
struct DhArgs {
    Operand g, w;
    int V;              // contraction length
    const Head *head;
    float *acc;         // [splits][live][K8], room for `room` rows
    int64_t room, K8;
    bool add;
    const int *map;
    void *dH;
    int64_t lddh;
    int K;
    bool vec;
    int bm, tiles_n, slots, piece;  // tile rows, columns of tiles, workgroups to fill, vocabulary per piece
};
// Splits of the contraction: as many as fill the slots and the room, each of at
// least 8 K-tiles (the same for every piece).
__device__ inline int dh_splits(const DhArgs &a, int live)
{
    const int t = imax((live + a.bm - 1) / a.bm * a.tiles_n, 1);
    const int64_t room = a.room / imax(live, 1);
    return imax(imin(imin(a.slots / t, (int)(room < 1024 ? room : 1024)), a.piece / (8 * BK)), 1);
}
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void xent_dh_kernel(
    DhArgs a)
{
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const int M = a.head->live;
    const int splits = dh_splits(a, M);
    const int tiles_m = (M + T::BM - 1) / T::BM, tiles = tiles_m * a.tiles_n, total = tiles * splits;
    if ((int)blockIdx.x >= total)
        return;
    const int logical = xcd_contiguous(blockIdx.x, total);
    const int z = logical / tiles;
    int tm, tn;
    grouped_tile<4>(logical - z * tiles, tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    const int split = (a.piece + splits * BK - 1) / (splits * BK) * BK;
    const int from = z * split, len = imax(imin(split, a.V - from), 0);
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    Operand g = a.g, w = a.w;
    g.extent = M;
    g.p = reinterpret_cast<const E *>(g.p) + from;
    w.p = reinterpret_cast<const E *>(w.p) + (int64_t)from * w.ld;
    T::run(smem, g, w, m0, n0, len, acc);

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int fr = lane & 15, fc = 4 * (lane >> 4);
    const int r0 = m0 + wm * T::WTM, c0 = n0 + wn * T::WTN;
    // three columns of blocks ahead: their sums are being loaded while one is
    // added and stored
    constexpr int DEPTH = 4;
    float *out = a.acc + ((int64_t)z * M + r0 + fr) * a.K8 + c0 + fc;
    f32x4 old[DEPTH][T::TM];
    auto fetch = [&](int j) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            old[j % DEPTH][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (a.add && r0 + 16 * i + fr < M && c0 + 16 * j + fc < a.K8)
                old[j % DEPTH][i] = *reinterpret_cast<const f32x4 *>(out + (int64_t)(16 * i) * a.K8 + 16 * j);
        }
    };
#pragma unroll
    for (int j = 0; j < DEPTH - 1 && j < T::TN; ++j)
        fetch(j);
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
        if (j + DEPTH - 1 < T::TN)
            fetch(j + DEPTH - 1);
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
            if (r0 + 16 * i + fr < M && c0 + 16 * j + fc < a.K8)
                *reinterpret_cast<f32x4 *>(out + (int64_t)(16 * i) * a.K8 + 16 * j) = old[j % DEPTH][i] + acc[i][j];
    }
}
// The splits' sums, in order, scaled, rounded and scattered.
template <typename E>
__global__ __launch_bounds__(256) void xent_dh_finish_kernel(DhArgs a)
{
    const int64_t live = a.head->live, per = a.K8 / 4, total = live * per;
    const int splits = dh_splits(a, (int)live);
    const float alpha = a.head->alpha / g_scale<E>();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 4;
        f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int z = 0; z < splits; ++z)
            s += *reinterpret_cast<const f32x4 *>(a.acc + (z * live + r) * a.K8 + c);
        E *dst = reinterpret_cast<E *>(a.dH) + (int64_t)a.map[r] * a.lddh + c;
        typename El<E>::v4 d;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            d[v] = (E)(s[v] * alpha);
        if (a.vec && c + 4 <= a.K) {
            *reinterpret_cast<typename El<E>::v4 *>(dst) = d;
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (c + v < a.K)
                    dst[v] = d[v];
        }
    }
}

// -------------------------------------------------------------- dW = Gᵀ·H
struct DwArgs {
    Operand g, h;       // both transposed: K rows are live tokens
    const Head *head;
    void *dW;           // rows of the piece
    int64_t lddw;
    int V, K;
    bool vec;
    int tiles_m, tiles_n;
};
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void xent_dw_kernel(
    DwArgs a)
{
    using V4 = typename El<E>::v4;
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    int tm, tn;
    grouped_tile<4>(xcd_contiguous(blockIdx.x, a.tiles_m * a.tiles_n), a.tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    T::run(smem, a.g, a.h, m0, n0, a.head->live, acc);
    const float alpha = a.head->alpha / g_scale<E>();
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int fr = lane & 15, fc = 4 * (lane >> 4);
    barrier_lds();
    E *stg = smem + wave * T::WTM * T::WTN;
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) {
            V4 d;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                d[v] = (E)(acc[i][j][v] * alpha);
            *reinterpret_cast<V4 *>(stg + stage_off<T::WTN>(16 * i + fr, 16 * j + fc)) = d;
        }
    store_block<E, T::WTM, T::WTN>(stg, reinterpret_cast<E *>(a.dW), a.lddw, m0 + wm * T::WTM, n0 + wn * T::WTN, a.V,
                                   a.K, a.vec, nullptr, lane);
}

// ------------------------------------------------------------------- plans
// Tile classes: one workgroup per CU at 256×256 and 192×192, two of the smaller
// ones; 64×128 for at most 64 tokens, so that W is read once.
enum Class { C256, C192, C128, C64, C64X128, CLASSES };
const char *const CLASS_NAME[] = {"256x256", "192x192", "128x128", "64x64", "64x128"};
constexpr TileClass CLASS[] = {{256, 256, 1, 1.50, 1.50, 16.0},
                               {192, 192, 1, 1.15, 1.15, 9.0},
                               {128, 128, 2, 1.10, 0.50, 6.0},
                               {64, 64, 2, 0.50, 0.27, 4.0},
                               {64, 128, 2, 0.80, 0.45, 5.0}};
// `stream`: one row of tiles and a W larger than the 256 MB last-level cache, so
// that each element of W comes from memory, once (a forward call of 100×50001×4096
// 106 -> 91 us, 250×131072×2048 165 -> 132; a W that the cache still holds is read
// faster without: 200×50001×1000 42 against 50).
template <typename E, bool TA, bool TB, typename F>
bool with_tile(Class c, bool stream, F f)
{
    if constexpr (!TA && !TB) {
        if (stream && c == C256)
            return f(Tile<E, 256, 256, 2, 2, 2, TA, TB, true>{});
        if (stream && c == C128)
            return f(Tile<E, 128, 128, 2, 2, 2, TA, TB, true>{});
    }
    switch (c) {
    case C256:
        return f(Tile<E, 256, 256, 2, 2, 2, TA, TB>{});
    case C192:  // (not dH's: its splits fill the chip at any tile size)
        if constexpr (TA == TB)
            return f(Tile<E, 192, 192, 2, 2, 2, TA, TB>{});
        [[fallthrough]];
    case C128:
        return f(Tile<E, 128, 128, 2, 2, 2, TA, TB>{});
    case C64X128:
        if constexpr (!TA)
            return f(Tile<E, 64, 128, 1, 4, 3, TA, TB, !TB>{});
        [[fallthrough]];
    default:
        return f(Tile<E, 64, 64, 2, 2, 3, TA, TB>{});
    }
}
int64_t tiles(Class c, int64_t m, int64_t n) { return cdiv(m, CLASS[c].bm) * cdiv(n, CLASS[c].bn); }
Class best_class(int64_t m, int64_t n, int64_t k, bool dh = false)
{
    int c = 0;
    for (int i = 1; i < C64X128; ++i)
        if (!(dh && i == C192) && tile_time(CLASS[i], tiles((Class)i, m, n), cdiv(k, BK)) < tile_time(CLASS[c], tiles((Class)c, m, n), cdiv(k, BK)))
            c = i;
    return (Class)c;
}
Class logits_class(int64_t M, int64_t V, int64_t K)
{
    return M <= 64 && tiles(C64X128, M, V) >= NUM_CU / 4 ? C64X128 : best_class(M, V, K);
}
constexpr int64_t G_BYTES = (int64_t)512 << 20;  // of G at a time
constexpr int64_t G_COLS = 768 * 1365;           // and so many columns (a row is walked with 32-bit offsets)
constexpr int64_t COMPACT_FLOP = (int64_t)1 << 38;

struct Plan {
    bool pack_w, compact;
    int64_t K8, piece, pieces;
    Class logits, dh, dw;
    bool stream;   // the logits' products
    int slots;     // workgroups that fill the chip, of dH's class
    int64_t room;  // rows of fp32 sums for dH
};
bool rows_ok(const void *p, int64_t ld, int64_t K)
{
    return (uintptr_t)p % 16 == 0 && ld % 8 == 0 && K % 8 == 0 && ld <= MAX_DMA_LD;
}
Plan make_plan(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw, bool bwd)
{
    Plan p;
    p.K8 = round_up(K, 8);
    p.pack_w = !rows_ok(W, ldw, K);
    // the forward pass gathers the live tokens where the product is long
    // enough (2^38 flop, some 200 us) that the two extra launches cost nothing
    p.compact = bwd || !rows_ok(H, ldh, K) || 2.0 * (double)M * (double)V * (double)K >= (double)COMPACT_FLOP;
    int64_t most = V;
    if (bwd)
        most = std::min(std::min(V, G_COLS), std::max(G_BYTES / 2 / M, (int64_t)8192));
    if (p.pack_w)
        most = std::min(most, std::max(G_BYTES / 2 / p.K8, (int64_t)1024));
    p.piece = most >= V ? V : round_up(most, 768);  // whole tiles of 256 and of 192
    p.pieces = cdiv(V, p.piece);
    p.logits = logits_class(M, p.piece, K);
    p.stream = M <= CLASS[p.logits].bm && V * K * 2 > (int64_t)256 << 20;
    p.dw = best_class(p.piece, K, M);
    // dH's contraction is long, so its class is the one that runs a K-tile
    // fastest; the splits (dh_splits) take care of few tiles
    // (up to 64 of them there is nothing to split)
    p.dh = M <= 64 ? C64X128 : p.piece <= 64 * BK ? best_class(M, K, p.piece, true) : M * K >= (int64_t)1 << 20 ? C256 : C128;
    p.slots = NUM_CU * CLASS[p.dh].per_cu;
    const int64_t t = tiles(p.dh, M, K), most_splits = std::max((int64_t)1, p.piece / (8 * BK));
    p.room = M * std::max((int64_t)2, std::min(most_splits, cdiv(p.slots, t)));
    return p;
}

// workspace: a bump allocator in 256-byte steps
struct Space {
    char *base;
    int64_t used = 0;
    template <typename X>
    X *take(int64_t n)
    {
        X *p = base ? reinterpret_cast<X *>(base + used) : nullptr;
        used += round_up(n * (int64_t)sizeof(X), 256);
        return p;
    }
};
struct Buffers {
    Head *head;
    int *map, *col;
    void *hc, *wp, *G;
    float2 *part, *block_sum;
    float *at_target, *lse, *cp, *ct, *acc;
    int64_t Gld;
};
Buffers lay_out(Space &s, const Plan &p, int64_t M, int64_t V, bool bwd)
{
    Buffers b = {};
    b.head = s.take<Head>(1);
    b.map = s.take<int>(M);
    b.col = s.take<int>(M);
    if (p.compact)
        b.hc = s.take<uint16_t>(M * p.K8);
    if (p.pack_w)
        b.wp = s.take<uint16_t>(p.piece * p.K8);
    if (!bwd) {
        b.part = s.take<float2>(cdiv(V, CLASS[p.logits].bn) * M);
        b.at_target = s.take<float>(M);
        b.block_sum = s.take<float2>(cdiv(M, JOIN_ROWS));
    } else {
        b.lse = s.take<float>(M);
        b.cp = s.take<float>(M);
        b.ct = s.take<float>(M);
        b.Gld = round_up(p.piece, BK);
        b.G = s.take<uint16_t>(M * b.Gld);
        b.acc = s.take<float>(p.room * p.K8);
    }
    return b;
}

// The kernels' own limits beside the interface's: a row of a packed or gathered
// operand is K8 elements (a descriptor's offsets are 32-bit), and a launch holds
// fewer than 2^32 threads.
int validate(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw, bool bwd)
{
    if (M < 0 || V < 0 || K < 0 || ldh < K || ldw < K)
        return TG_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 31;
    if (M >= lim / 64 || V >= lim / 2 || K > MAX_DMA_LD || ldh >= lim || ldw >= lim)
        return TG_ERR_TOO_LARGE;
    if (M == 0)
        return TG_OK;
    if (V == 0 || K == 0 || !H || !W)
        return TG_ERR_INVALID_ARG;
    const Plan p = make_plan(H, W, M, V, K, ldh, ldw, bwd);
    int64_t most = tiles(p.logits, M, p.piece);
    if (bwd)
        most = std::max(most, std::max(tiles(p.dh, M, K), tiles(p.dw, p.piece, K)));
    return most >= MAX_GRID ? TG_ERR_TOO_LARGE : TG_OK;
}
bool reduction_ok(int r) { return r == TG_XENT_NONE || r == TG_XENT_SUM || r == TG_XENT_MEAN; }

int64_t workspace_bytes(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
                        bool bwd)
{
    if (validate(H, W, M, V, K, ldh, ldw, bwd) != TG_OK)
        return -1;
    if (M == 0)
        return 0;
    Space s = {nullptr};
    lay_out(s, make_plan(H, W, M, V, K, ldh, ldw, bwd), M, V, bwd);
    return s.used;
}

int64_t copy_grid(int64_t chunks)
{
    const int64_t g = cdiv(chunks, 256);
    return g < 1 ? 1 : g < 8 * NUM_CU ? g : 8 * NUM_CU;
}
// W rows [v0, v0 + n) as the kernels take them
bool w_piece(const Plan &p, const Buffers &b, const void *W, int64_t ldw, int64_t v0, int64_t n, int64_t K,
             void *stream, Operand &w)
{
    const uint16_t *src = reinterpret_cast<const uint16_t *>(W) + v0 * ldw;
    if (!p.pack_w) {
        w = {src, ldw, (int)n};
        return true;
    }
    w = {b.wp, p.K8, (int)n};
    return launch(xent_pack_kernel, copy_grid(n * p.K8 / 8), 256, stream, src, ldw, (uint16_t *)b.wp, n, K, p.K8);
}
// the workgroups' share of the tokens
void split_rows(PrepArgs &a, int64_t &grid)
{
    a.rows = (int)std::max((int64_t)4, cdiv(a.M, 2 * NUM_CU));
    grid = cdiv(a.M, a.rows);
}

template <typename E>
int forward(const void *H, const void *W, const int64_t *target, float *loss, float *lse, int64_t M, int64_t V,
            int64_t K, int64_t ldh, int64_t ldw, int64_t ignore, int reduction, void *ws, int64_t ws_bytes,
            void *stream)
{
    int st = validate(H, W, M, V, K, ldh, ldw, false);
    if (st != TG_OK)
        return st;
    if (!reduction_ok(reduction) || (M > 0 && !target) || (!loss && (M > 0 || reduction != TG_XENT_NONE)))
        return TG_ERR_INVALID_ARG;
    Plan p;
    if (M > 0) {
        p = make_plan(H, W, M, V, K, ldh, ldw, false);
        const int64_t need = workspace_bytes(H, W, M, V, K, ldh, ldw, false);
        if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < need)
            return TG_ERR_INVALID_ARG;
    }
    if (M == 0 && reduction == TG_XENT_NONE)
        return TG_OK;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    if (M == 0) {
        return launch(xent_zero_kernel, 1, 256, stream, (uint16_t *)loss, (int64_t)2, (int64_t)1, (int64_t)2)
                   ? TG_OK
                   : TG_ERR_LAUNCH;
    }
    Space s = {reinterpret_cast<char *>(ws)};
    const Buffers b = lay_out(s, p, M, V, false);
    float *row_loss = reduction == TG_XENT_NONE ? loss : nullptr;
    bool ok = true;
    if (p.compact) {
        PrepArgs a = {};
        a.target = target, a.M = M, a.V = V, a.ignore = ignore;
        a.head = b.head, a.map = b.map, a.col = b.col, a.loss = row_loss, a.lse_out = lse;
        a.H = (const uint16_t *)H, a.ldh = ldh, a.hc = (uint16_t *)b.hc, a.K = K, a.K8 = p.K8, a.vec = rows_ok(H, ldh, K);
        int64_t grid;
        split_rows(a, grid);
        ok = launch(xent_prep_kernel<false>, grid, PREP_THREADS, stream, a);
    }
    for (int64_t v0 = 0; ok && v0 < V; v0 += p.piece) {
        const int64_t n = v0 + p.piece < V ? p.piece : V - v0;
        StatsArgs a = {};
        ok = w_piece(p, b, W, ldw, v0, n, K, stream, a.w);
        a.h = p.compact ? Operand{b.hc, p.K8, (int)M} : Operand{H, ldh, (int)M};
        a.K = (int)(p.pack_w || p.compact ? p.K8 : K);
        a.M = (int)M;
        a.head = p.compact ? b.head : nullptr;
        a.V = (int)n, a.v0 = (int)v0;
        a.col = p.compact ? b.col : nullptr;
        a.target = target, a.Vall = V;
        a.part = b.part, a.part_ld = M, a.at_target = b.at_target, a.arrived = &b.head->arrived;
        a.tiles_n = (int)cdiv(n, CLASS[p.logits].bn);
        ok = ok && with_tile<E, false, false>(p.logits, p.stream, [&](auto t) {
            return launch(xent_stats_kernel<E, decltype(t)>, tiles(p.logits, M, n), t.THREADS, stream, a);
        });
    }
    JoinArgs j = {};
    j.part = b.part, j.part_ld = M;
    j.tiles = (int)cdiv(V, CLASS[p.logits].bn);
    j.M = (int)M, j.reduction = reduction;
    j.head = p.compact ? b.head : nullptr;
    j.map = p.compact ? b.map : nullptr;
    j.col = p.compact ? b.col : nullptr;
    j.target = target, j.V = V, j.ignore = ignore;
    j.at_target = b.at_target, j.loss = row_loss, j.lse = lse;
    j.block_sum = reduction == TG_XENT_NONE ? nullptr : b.block_sum;
    j.arrived = &b.head->arrived, j.total = loss;
    ok = ok && launch(xent_join_kernel, cdiv(M, JOIN_ROWS), 1024, stream, j);
    return ok ? TG_OK : TG_ERR_LAUNCH;
}

template <typename E>
int backward(const void *H, const void *W, const int64_t *target, const float *lse, const float *dloss,
             const float *dlse, void *dH, void *dW, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
             int64_t lddh, int64_t lddw, int64_t ignore, int reduction, void *ws, int64_t ws_bytes, void *stream)
{
    int st = validate(H, W, M, V, K, ldh, ldw, true);
    if (st != TG_OK)
        return st;
    if (!reduction_ok(reduction) || (dH && lddh < K) || (dW && lddw < K) ||
        (M > 0 && (!target || !lse || !dloss)))
        return TG_ERR_INVALID_ARG;
    if (lddh >= ((int64_t)1 << 31) || lddw >= ((int64_t)1 << 31))
        return TG_ERR_TOO_LARGE;
    Plan p;
    if (M > 0) {
        p = make_plan(H, W, M, V, K, ldh, ldw, true);
        const int64_t need = workspace_bytes(H, W, M, V, K, ldh, ldw, true);
        if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < need)
            return TG_ERR_INVALID_ARG;
    }
    if ((M == 0 && (!dW || V == 0 || K == 0)) || (!dH && !dW))
        return TG_OK;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    if (M == 0)
        return launch(xent_zero_kernel, std::min(V, (int64_t)8 * NUM_CU), 256, stream, (uint16_t *)dW, lddw, V, K)
                   ? TG_OK
                   : TG_ERR_LAUNCH;
    Space s = {reinterpret_cast<char *>(ws)};
    const Buffers b = lay_out(s, p, M, V, true);
    PrepArgs q = {};
    q.target = target, q.M = M, q.V = V, q.ignore = ignore;
    q.head = b.head, q.map = b.map, q.col = b.col;
    q.H = (const uint16_t *)H, q.ldh = ldh, q.hc = (uint16_t *)b.hc, q.K = K, q.K8 = p.K8, q.vec = rows_ok(H, ldh, K);
    q.reduction = reduction, q.dloss = dloss, q.dlse = dlse, q.lse = lse;
    q.lse_c = b.lse, q.cp = b.cp, q.ct = b.ct, q.dH = (uint16_t *)dH, q.lddh = lddh;
    int64_t grid;
    split_rows(q, grid);
    bool ok = launch(xent_prep_kernel<true>, grid, PREP_THREADS, stream, q);
    DhArgs d = {};
    for (int64_t v0 = 0; ok && v0 < V; v0 += p.piece) {
        const int64_t n = v0 + p.piece < V ? p.piece : V - v0;
        Operand w;
        ok = w_piece(p, b, W, ldw, v0, n, K, stream, w);
        GradArgs a = {};
        a.h = {b.hc, p.K8, (int)M};
        a.w = w;
        a.K = (int)p.K8;
        a.head = b.head, a.V = (int)n, a.v0 = (int)v0, a.col = b.col;
        a.lse = b.lse, a.cp = b.cp, a.ct = b.ct;
        a.G = b.G, a.Gld = round_up(n, BK);
        a.tiles_n = (int)cdiv(n, CLASS[p.logits].bn);
        ok = ok && with_tile<E, false, false>(p.logits, p.stream, [&](auto t) {
            return launch(xent_grad_kernel<E, decltype(t)>, tiles(p.logits, M, n), t.THREADS, stream, a);
        });
        if (dH) {
            d.g = {b.G, a.Gld, (int)M};
            d.w = {w.p, w.ld, (int)K};
            d.V = (int)n, d.piece = (int)p.piece, d.head = b.head;
            d.acc = b.acc, d.room = p.room, d.K8 = p.K8, d.add = v0 > 0;
            d.map = b.map, d.dH = dH, d.lddh = lddh, d.K = (int)K;
            d.vec = lddh % 8 == 0 && (uintptr_t)dH % 16 == 0;
            d.bm = CLASS[p.dh].bm, d.tiles_n = (int)cdiv(K, CLASS[p.dh].bn), d.slots = p.slots;
            const int64_t g = std::max(tiles(p.dh, M, K), (int64_t)p.slots);
            ok = ok && with_tile<E, false, true>(p.dh, false, [&](auto t) {
                return launch(xent_dh_kernel<E, decltype(t)>, g, t.THREADS, stream, d);
            });
        }
        if (dW) {
            DwArgs x = {};
            x.g = {b.G, a.Gld, (int)n};
            x.h = {b.hc, p.K8, (int)K};
            x.head = b.head;
            x.dW = reinterpret_cast<uint16_t *>(dW) + v0 * lddw, x.lddw = lddw;
            x.V = (int)n, x.K = (int)K;
            x.vec = lddw % 8 == 0 && (uintptr_t)dW % 16 == 0;
            x.tiles_m = (int)cdiv(n, CLASS[p.dw].bm), x.tiles_n = (int)cdiv(K, CLASS[p.dw].bn);
            ok = ok && with_tile<E, true, true>(p.dw, false, [&](auto t) {
                return launch(xent_dw_kernel<E, decltype(t)>, tiles(p.dw, n, K), t.THREADS, stream, x);
            });
        }
    }
    if (ok && dH)
        ok = launch(xent_dh_finish_kernel<E>, copy_grid(M * p.K8 / 4), 256, stream, d);
    return ok ? TG_OK : TG_ERR_LAUNCH;
}

}  // namespace

extern "C" int64_t tg_xent_workspace_bytes(const void *H, const void *W, int64_t M, int64_t V, int64_t K,
                                           int64_t ldh, int64_t ldw)
{
    return workspace_bytes(H, W, M, V, K, ldh, ldw, false);
}

extern "C" int64_t tg_xent_bwd_workspace_bytes(const void *H, const void *W, int64_t M, int64_t V, int64_t K,
                                               int64_t ldh, int64_t ldw)
{
    return workspace_bytes(H, W, M, V, K, ldh, ldw, true);
}

extern "C" int tg_xent_f16(const void *H, const void *W, const int64_t *target, float *loss, float *lse, int64_t M,
                           int64_t V, int64_t K, int64_t ldh, int64_t ldw, int64_t ignore_index, int reduction,
                           void *workspace, int64_t workspace_bytes, void *stream)
{
    return forward<_Float16>(H, W, target, loss, lse, M, V, K, ldh, ldw, ignore_index, reduction, workspace,
                             workspace_bytes, stream);
}

extern "C" int tg_xent_bf16(const void *H, const void *W, const int64_t *target, float *loss, float *lse, int64_t M,
                            int64_t V, int64_t K, int64_t ldh, int64_t ldw, int64_t ignore_index, int reduction,
                            void *workspace, int64_t workspace_bytes, void *stream)
{
    return forward<__bf16>(H, W, target, loss, lse, M, V, K, ldh, ldw, ignore_index, reduction, workspace,
                           workspace_bytes, stream);
}

extern "C" int tg_xent_bwd_f16(const void *H, const void *W, const int64_t *target, const float *lse,
                               const float *dloss, const float *dlse, void *dH, void *dW, int64_t M, int64_t V,
                               int64_t K, int64_t ldh, int64_t ldw, int64_t lddh, int64_t lddw, int64_t ignore_index,
                               int reduction, void *workspace, int64_t workspace_bytes, void *stream)
{
    return backward<_Float16>(H, W, target, lse, dloss, dlse, dH, dW, M, V, K, ldh, ldw, lddh, lddw, ignore_index,
                              reduction, workspace, workspace_bytes, stream);
}

extern "C" int tg_xent_bwd_bf16(const void *H, const void *W, const int64_t *target, const float *lse,
                                const float *dloss, const float *dlse, void *dH, void *dW, int64_t M, int64_t V,
                                int64_t K, int64_t ldh, int64_t ldw, int64_t lddh, int64_t lddw,
                                int64_t ignore_index, int reduction, void *workspace, int64_t workspace_bytes,
                                void *stream)
{
    return backward<__bf16>(H, W, target, lse, dloss, dlse, dH, dW, M, V, K, ldh, ldw, lddh, lddw, ignore_index,
                            reduction, workspace, workspace_bytes, stream);
}

extern "C" int tg_xent_plan(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
                            int backward_pass, char *name, int64_t name_len, int64_t *pieces)
{
    if (name && name_len > 0)
        name[0] = 0;
    if (pieces)
        *pieces = 0;
    const int st = validate(H, W, M, V, K, ldh, ldw, backward_pass != 0);
    if (st != TG_OK || M == 0)
        return st;
    const Plan p = make_plan(H, W, M, V, K, ldh, ldw, backward_pass != 0);
    if (pieces)
        *pieces = p.pieces;
    if (name && name_len > 0) {
        const char *pre = p.compact ? "gather " : "", *pack = p.pack_w ? "pack " : "";
        const char *how = p.stream && (p.logits == C256 || p.logits == C128) ? "_stream" : "";
        if (backward_pass)
            snprintf(name, (size_t)name_len, "%s%sgrad_%s%s dh_%s dw_%s", pre, pack, CLASS_NAME[p.logits], how,
                     CLASS_NAME[p.dh], CLASS_NAME[p.dw]);
        else
            snprintf(name, (size_t)name_len, "%s%sstats_%s%s", pre, pack, CLASS_NAME[p.logits], how);
    }
    return TG_OK;
}
