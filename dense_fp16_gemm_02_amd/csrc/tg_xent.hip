// tg_xent.hip — softmax cross entropy of the vocabulary projection and its
// gradients.  See include/tg_xent.h for the contract.
//
// Forward: the logits tile z = H·Wᵀ stays in the accumulators; per row and
// per wave column strip the kernel keeps only the running maximum m and
// s = Σ exp(z − m), so M·V logits shrink to M·(V/strip) pairs.  Two pairs join as
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

// What the index kernel finds out, at the start of a workspace.
struct Head {
    int live;     // tokens not ignored
    float alpha;  // what G was divided by (backward)
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

// ------------------------------------------------------------ index, gather
// One workgroup: numbers the live tokens, and for the backward pass their
// coefficients.  A few microseconds at 8192 tokens; it reads 8·M bytes.
struct IndexArgs {
    const int64_t *target;
    int64_t M, V, ignore;
    Head *head;
    int *map;        // live row -> token
    int *col;        // live row -> target, -1 if out of range
    float *loss;     // per-token loss and lse: zeroed for ignored tokens
    float *lse_out;
    // backward
    int reduction;
    const float *dloss, *dlse, *lse;
    float *lse_c, *cp, *ct;  // per live row: lse, and the coefficients of the softmax and of the target
};
constexpr int INDEX_THREADS = 1024;
template <bool BWD>
__global__ __launch_bounds__(INDEX_THREADS) void xent_index_kernel(IndexArgs a)
{
    __shared__ int wave_count[16];
    __shared__ float wave_max[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto live_at = [&](int64_t i) { return i < a.M && a.target[i] != a.ignore; };
    float scale = 1.0f, top = 0.0f;
    if constexpr (BWD) {
        if (a.reduction == TG_XENT_MEAN) {
            int n = 0;
            for (int64_t i = tid; i < a.M; i += INDEX_THREADS)
                n += live_at(i);
            for (int o = 32; o; o >>= 1)
                n += __shfl_xor(n, o);
            if (lane == 0)
                wave_count[wave] = n;
            __syncthreads();
            n = 0;
            for (int w = 0; w < 16; ++w)
                n += wave_count[w];
            __syncthreads();
            scale = 1.0f / (float)imax(n, 1);
        }
        // the largest coefficient (a NaN among them reaches its own row through
        // its coefficient, not through the maximum)
        for (int64_t i = tid; i < a.M; i += INDEX_THREADS)
            if (live_at(i)) {
                const float g = (a.reduction == TG_XENT_NONE ? a.dloss[i] : a.dloss[0]) * scale;
                top = fmaxf(top, fmaxf(fabsf(g), a.dlse ? fabsf(g + a.dlse[i]) : 0.0f));
            }
        for (int o = 32; o; o >>= 1)
            top = fmaxf(top, __shfl_xor(top, o));
        if (lane == 0)
            wave_max[wave] = top;
        __syncthreads();
        top = 0.0f;
        for (int w = 0; w < 16; ++w)
            top = fmaxf(top, wave_max[w]);
        if (!(top > 0.0f))
            top = 1.0f;
    }
    int base = 0;
    for (int64_t i0 = 0; i0 < a.M; i0 += INDEX_THREADS) {
        const int64_t i = i0 + tid;
        const bool live = live_at(i);
        const unsigned long long votes = __ballot(live);
        if (lane == 0)
            wave_count[wave] = __popcll(votes);
        __syncthreads();
        int at = base, all = 0;
        for (int w = 0; w < 16; ++w) {
            at += w < wave ? wave_count[w] : 0;
            all += wave_count[w];
        }
        at += __popcll(votes & ((1ull << lane) - 1));
        __syncthreads();
        base += all;
        if (live) {
            const int64_t t = a.target[i];
            const bool in = t >= 0 && t < a.V;
            a.map[at] = (int)i;
            a.col[at] = in ? (int)t : -1;
            if constexpr (BWD) {
                const float g = (a.reduction == TG_XENT_NONE ? a.dloss[i] : a.dloss[0]) * scale;
                const float l = a.dlse ? a.dlse[i] : 0.0f;
                a.lse_c[at] = a.lse[i];
                a.cp[at] = in ? (g + l) / top : NAN;
                a.ct[at] = g / top;
            }
        } else if (i < a.M) {
            if constexpr (!BWD) {
                if (a.loss)
                    a.loss[i] = 0.0f;
                if (a.lse_out)
                    a.lse_out[i] = 0.0f;
            }
        }
    }
    if (tid == 0) {
        a.head->live = base;
        a.head->alpha = top;
    }
}

// Rows map[0 .. *live) of src (all of the first `rows` where map is null) to
// consecutive rows of dst, K columns padded with zeros to K8 (a multiple of
// 8).  Rows of `zero` (dH) whose token is ignored are cleared: zero_target.
struct GatherArgs {
    const void *src;
    int64_t ld;
    void *dst;
    int64_t rows, K, K8;
    const int *map;
    const Head *head;
    bool vec;  // 16-byte aligned source rows, K % 8 == 0
};
__global__ __launch_bounds__(256) void xent_gather_kernel(GatherArgs a)
{
    const int64_t rows = a.map ? a.head->live : a.rows;
    const int64_t per = a.K8 / 8, total = rows * per;
    const uint16_t *src = reinterpret_cast<const uint16_t *>(a.src);
    uint16_t *dst = reinterpret_cast<uint16_t *>(a.dst);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        const uint16_t *s = src + (a.map ? (int64_t)a.map[r] : r) * a.ld + c;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (a.vec) {
            v = *reinterpret_cast<const uint4 *>(s);
        } else {
            union {
                uint4 u;
                uint16_t h[8];
            } w;
            w.u = v;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < a.K)
                    w.h[e] = s[e];
            v = w.u;
        }
        *reinterpret_cast<uint4 *>(dst + r * a.K8 + c) = v;
    }
}
// dH rows of ignored tokens, or a whole matrix (target null), set to zero
__global__ __launch_bounds__(256) void xent_zero_kernel(uint16_t *dst, int64_t ld, int64_t rows, int64_t cols,
                                                        const int64_t *target, int64_t ignore)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        if (!target || target[r] == ignore)
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
    float2 *part;       // [strip][row]
    int64_t part_ld;
    float *at_target;   // row -> logit of its target
    int tiles_n;
};
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void xent_stats_kernel(
    StatsArgs a)
{
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const int M = a.head ? a.head->live : a.M;
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
    const int row0 = m0 + wm * T::WTM + (lane & 15);
    const int col0 = n0 + wn * T::WTN + 4 * (lane >> 4);
    float2 *part = a.part + (int64_t)(a.v0 / T::WTN + tn * T::WN + wn) * a.part_ld;
    const bool whole = n0 + wn * T::WTN + T::WTN <= a.V;
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
        if (lane < 16 && row < M)
            part[row] = make_float2(m, s);
    }
}

// Joins each row's pairs: 64 rows per workgroup, 16 waves taking every 16th
// strip.  Reads 8·strips·M bytes, coalesced along rows.
struct JoinArgs {
    const float2 *part;
    int64_t part_ld;
    int strips, M, reduction;
    const Head *head;
    const int *map, *col;
    const int64_t *target;
    int64_t V, ignore;
    const float *at_target;
    float *loss, *lse;   // per token (loss null unless TG_XENT_NONE)
    float2 *block_sum;   // per workgroup: sum of losses, tokens counted
    float *total;        // SUM, MEAN with one workgroup
};
__device__ inline void join(float2 &a, float2 b)
{
    const float m = fmaxf(a.x, b.x);
    const float from = m == -INFINITY ? 0.0f : m;
    // a NaN in either sum stays one
    a.y = a.y * fast_exp(a.x - from) + b.y * fast_exp(b.x - from);
    a.x = m;
}
__device__ inline float reduced(float sum, float count, int reduction)
{
    return reduction == TG_XENT_MEAN ? sum / fmaxf(count, 1.0f) : sum;
}
__global__ __launch_bounds__(1024) void xent_join_kernel(JoinArgs a)
{
    __shared__ float2 sh[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int M = a.head ? a.head->live : a.M;
    const int row = blockIdx.x * 64 + lane;
    float2 p = make_float2(-INFINITY, 0.0f);
    if (row < M)
        for (int s = wave; s < a.strips; s += 16)
            join(p, a.part[(int64_t)s * a.part_ld + row]);
    sh[wave][lane] = p;
    __syncthreads();
    if (wave)
        return;
#pragma unroll
    for (int w = 1; w < 16; ++w)
        join(p, sh[w][lane]);
    float loss = 0.0f, count = 0.0f;
    if (row < M) {
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
        for (int o = 32; o; o >>= 1) {
            loss += __shfl_xor(loss, o);
            count += __shfl_xor(count, o);
        }
        if (lane == 0) {
            if (a.total)
                a.total[0] = reduced(loss, count, a.reduction);
            else
                a.block_sum[blockIdx.x] = make_float2(loss, count);
        }
    }
}
__global__ __launch_bounds__(1024) void xent_total_kernel(const float2 *block_sum, int blocks, int reduction,
                                                          float *total)
{
    __shared__ float2 sh[16];
    float2 s = make_float2(0.0f, 0.0f);
    for (int i = threadIdx.x; i < blocks; i += 1024) {
        s.x += block_sum[i].x;
        s.y += block_sum[i].y;
    }
    for (int o = 32; o; o >>= 1) {
        s.x += __shfl_xor(s.x, o);
        s.y += __shfl_xor(s.y, o);
    }
    if ((threadIdx.x & 63) == 0)
        sh[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) {
            s.x += sh[w].x;
            s.y += sh[w].y;
        }
        total[0] = reduced(s.x, s.y, reduction);
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
// A: G, K-major; B: W of the piece, transposed.  With `acc` the product goes
// to fp32 sums (one per split of the contraction, added to what earlier
// pieces left), otherwise it is scaled, rounded and scattered to dH.
struct DhArgs {
    Operand g, w;
    int V, split;       // contraction length, and how much of it a split takes
    const Head *head;
    float *acc;         // [splits][M][K8]
    int64_t acc_rows, K8;
    bool add;
    const int *map;
    void *dH;
    int64_t lddh;
    int K;
    bool vec;
    int tiles_n, splits;
};
template <typename E, typename T, bool ACC>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void xent_dh_kernel(
    DhArgs a)
{
    using V4 = typename El<E>::v4;
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const int M = a.head->live;
    const int tiles_m = (M + T::BM - 1) / T::BM, tiles = tiles_m * a.tiles_n, total = tiles * a.splits;
    if ((int)blockIdx.x >= total)
        return;
    const int logical = xcd_contiguous(blockIdx.x, total);
    const int z = logical / tiles;
    int tm, tn;
    grouped_tile<4>(logical - z * tiles, tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    const int from = z * a.split, len = imax(imin(a.split, a.V - from), 0);
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
    if constexpr (ACC) {
        // a column of blocks ahead: the next one's sums are being loaded while
        // one is added and stored
        float *out = a.acc + ((int64_t)z * a.acc_rows + r0 + fr) * a.K8 + c0 + fc;
        f32x4 old[2][T::TM];
        auto fetch = [&](int j) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < T::TM; ++i) {
                old[j & 1][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (a.add && r0 + 16 * i + fr < M && c0 + 16 * j + fc < a.K8)
                    old[j & 1][i] = *reinterpret_cast<const f32x4 *>(out + (int64_t)(16 * i) * a.K8 + 16 * j);
            }
        };
        fetch(0);
#pragma unroll
        for (int j = 0; j < T::TN; ++j) {
            if (j + 1 < T::TN)
                fetch(j + 1);
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
                if (r0 + 16 * i + fr < M && c0 + 16 * j + fc < a.K8)
                    *reinterpret_cast<f32x4 *>(out + (int64_t)(16 * i) * a.K8 + 16 * j) = old[j & 1][i] + acc[i][j];
        }
        return;
    }
    const float alpha = a.head->alpha / g_scale<E>();
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
    store_block<E, T::WTM, T::WTN>(stg, reinterpret_cast<E *>(a.dH), a.lddh, r0, c0, M, a.K, a.vec, a.map, lane);
}
// The splits' sums, in order, scaled, rounded and scattered.
template <typename E>
__global__ __launch_bounds__(256) void xent_dh_finish_kernel(DhArgs a)
{
    const int64_t live = a.head->live, per = a.K8 / 4, total = live * per;
    const float alpha = a.head->alpha / g_scale<E>();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per, c = (i - r * per) * 4;
        f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int z = 0; z < a.splits; ++z)
            s += *reinterpret_cast<const f32x4 *>(a.acc + ((int64_t)z * a.acc_rows + r) * a.K8 + c);
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
// Tile classes.  256×256 (one workgroup per CU) from 5/8 of the CUs on;
// 128×128 (two per CU) below; 64×64 where even those are few; 64×128 for at
// most 64 tokens, so that W is read once.
enum Class { C256, C128, C64, C64X128 };
const char *const CLASS_NAME[] = {"256x256", "128x128", "64x64", "64x128"};
constexpr int CLASS_BM[] = {256, 128, 64, 64}, CLASS_BN[] = {256, 128, 64, 128};
template <typename E, bool TA, bool TB>
using T256 = Tile<E, 256, 256, 2, 2, 2, TA, TB>;
template <typename E, bool TA, bool TB>
using T128 = Tile<E, 128, 128, 2, 2, 2, TA, TB>;
template <typename E, bool TA, bool TB>
using T64 = Tile<E, 64, 64, 2, 2, 3, TA, TB>;
template <typename E, bool TA, bool TB>
using T64x128 = Tile<E, 64, 128, 1, 4, 3, TA, TB>;

int64_t tiles(Class c, int64_t m, int64_t n) { return cdiv(m, CLASS_BM[c]) * cdiv(n, CLASS_BN[c]); }
Class logits_class(int64_t M, int64_t V)
{
    if (M <= 64)
        return tiles(C64X128, M, V) >= NUM_CU / 4 ? C64X128 : C64;
    return tiles(C256, M, V) >= 160 ? C256 : tiles(C128, M, V) >= 80 ? C128 : C64;
}
// strip width (columns per pair) of the logits tiles
int strip_of(Class c) { return c == C256 ? 128 : c == C128 ? 64 : 32; }

constexpr int64_t G_BYTES = (int64_t)512 << 20;  // of G at a time
constexpr int64_t COMPACT_FLOP = (int64_t)1 << 38;

struct Plan {
    bool pack_w, compact;
    int64_t K8, piece, pieces;
    Class logits, dh, dw;
    int splits;
    int64_t split;  // contraction per split of dH
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
        most = std::min(V, std::max(G_BYTES / 2 / M, (int64_t)8192));
    if (p.pack_w)
        most = std::min(most, std::max(G_BYTES / 2 / p.K8, (int64_t)1024));
    p.piece = most >= V ? V : round_up(most, 256);
    p.pieces = cdiv(V, p.piece);
    p.logits = logits_class(M, p.piece);
    p.dh = M <= 64 ? C64X128 : tiles(C256, M, K) >= 160 ? C256 : C128;
    p.dw = tiles(C256, p.piece, K) >= 160 ? C256 : tiles(C128, p.piece, K) >= 80 ? C128 : C64;
    // dH has M·K outputs and a contraction over the piece: few tiles are split
    // along it until some 512 workgroups run, each with at least 8 K-tiles
    p.splits = 1;
    p.split = round_up(p.piece, BK);
    const int64_t t = tiles(p.dh, M, K);
    if (p.dh != C256 && t < 256) {
        const int64_t want = cdiv(512, t), can = cdiv(p.piece, 8 * BK);
        const int64_t s = want < can ? want : can;
        p.split = round_up(cdiv(p.piece, s), BK);
        p.splits = (int)cdiv(p.piece, p.split);
    }
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
    int64_t strips, Gld;
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
        b.strips = cdiv(V, strip_of(p.logits)) + 8;  // the last tile's strips past V included
        b.part = s.take<float2>(b.strips * M);
        b.at_target = s.take<float>(M);
        b.block_sum = s.take<float2>(cdiv(M, 64));
    } else {
        b.lse = s.take<float>(M);
        b.cp = s.take<float>(M);
        b.ct = s.take<float>(M);
        b.Gld = round_up(p.piece, BK);
        b.G = s.take<uint16_t>(M * b.Gld);
        if (p.pieces > 1 || p.splits > 1)
            b.acc = s.take<float>(p.splits * M * p.K8);
    }
    return b;
}

int validate(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw)
{
    if (M < 0 || V < 0 || K < 0 || ldh < K || ldw < K)
        return TG_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 31;
    if (M >= lim || V >= lim || K >= lim || ldh >= lim || ldw >= lim)
        return TG_ERR_TOO_LARGE;
    if (M == 0)
        return TG_OK;
    if (V == 0 || K == 0 || !H || !W)
        return TG_ERR_INVALID_ARG;
    if (cdiv(M, 64) * cdiv(V, 64) >= lim || cdiv(M, 64) * cdiv(K, 64) * 64 >= lim ||
        cdiv(V, 64) * cdiv(K, 64) >= lim || M > lim - 1024 || V > lim - 1024 || K > lim - 1024)
        return TG_ERR_TOO_LARGE;
    return TG_OK;
}
bool reduction_ok(int r) { return r == TG_XENT_NONE || r == TG_XENT_SUM || r == TG_XENT_MEAN; }

int64_t workspace_bytes(const void *H, const void *W, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
                        bool bwd)
{
    if (validate(H, W, M, V, K, ldh, ldw) != TG_OK)
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
    return launch(xent_gather_kernel, copy_grid(n * p.K8 / 8), 256, stream,
                  GatherArgs{src, ldw, b.wp, n, K, p.K8, nullptr, nullptr, false});
}
bool gather_h(const Plan &p, const Buffers &b, const void *H, int64_t ldh, int64_t M, int64_t K, void *stream)
{
    return launch(xent_gather_kernel, copy_grid(M * p.K8 / 8), 256, stream,
                  GatherArgs{H, ldh, b.hc, M, K, p.K8, b.map, b.head, rows_ok(H, ldh, K)});
}

template <typename E>
int forward(const void *H, const void *W, const int64_t *target, float *loss, float *lse, int64_t M, int64_t V,
            int64_t K, int64_t ldh, int64_t ldw, int64_t ignore, int reduction, void *ws, int64_t ws_bytes,
            void *stream)
{
    int st = validate(H, W, M, V, K, ldh, ldw);
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
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    if (M == 0) {
        if (reduction == TG_XENT_NONE)
            return TG_OK;
        return launch(xent_total_kernel, 1, 1024, stream, (const float2 *)nullptr, 0, reduction, loss)
                   ? TG_OK
                   : TG_ERR_LAUNCH;
    }
    Space s = {reinterpret_cast<char *>(ws)};
    const Buffers b = lay_out(s, p, M, V, false);
    float *row_loss = reduction == TG_XENT_NONE ? loss : nullptr;
    bool ok = true;
    if (p.compact) {
        IndexArgs ia = {};
        ia.target = target, ia.M = M, ia.V = V, ia.ignore = ignore;
        ia.head = b.head, ia.map = b.map, ia.col = b.col, ia.loss = row_loss, ia.lse_out = lse;
        ok = ok && launch(xent_index_kernel<false>, 1, INDEX_THREADS, stream, ia);
        ok = ok && gather_h(p, b, H, ldh, M, K, stream);
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
        a.part = b.part, a.part_ld = M, a.at_target = b.at_target;
        const int64_t grid = tiles(p.logits, M, n);
        a.tiles_n = (int)cdiv(n, CLASS_BN[p.logits]);
        switch (p.logits) {
        case C256:
            ok = ok && launch(xent_stats_kernel<E, T256<E, false, false>>, grid, 256, stream, a);
            break;
        case C128:
            ok = ok && launch(xent_stats_kernel<E, T128<E, false, false>>, grid, 256, stream, a);
            break;
        case C64X128:
            ok = ok && launch(xent_stats_kernel<E, T64x128<E, false, false>>, grid, 256, stream, a);
            break;
        default:
            ok = ok && launch(xent_stats_kernel<E, T64<E, false, false>>, grid, 256, stream, a);
        }
    }
    JoinArgs j = {};
    j.part = b.part, j.part_ld = M;
    j.strips = (int)cdiv(V, strip_of(p.logits));
    j.M = (int)M, j.reduction = reduction;
    j.head = p.compact ? b.head : nullptr;
    j.map = p.compact ? b.map : nullptr;
    j.col = p.compact ? b.col : nullptr;
    j.target = target, j.V = V, j.ignore = ignore;
    j.at_target = b.at_target, j.loss = row_loss, j.lse = lse;
    const int64_t blocks = cdiv(M, 64);
    j.block_sum = reduction == TG_XENT_NONE ? nullptr : b.block_sum;
    j.total = reduction != TG_XENT_NONE && blocks == 1 ? loss : nullptr;
    ok = ok && launch(xent_join_kernel, blocks, 1024, stream, j);
    if (reduction != TG_XENT_NONE && blocks > 1)
        ok = ok && launch(xent_total_kernel, 1, 1024, stream, (const float2 *)b.block_sum, (int)blocks, reduction, loss);
    return ok ? TG_OK : TG_ERR_LAUNCH;
}

template <typename E>
int backward(const void *H, const void *W, const int64_t *target, const float *lse, const float *dloss,
             const float *dlse, void *dH, void *dW, int64_t M, int64_t V, int64_t K, int64_t ldh, int64_t ldw,
             int64_t lddh, int64_t lddw, int64_t ignore, int reduction, void *ws, int64_t ws_bytes, void *stream)
{
    int st = validate(H, W, M, V, K, ldh, ldw);
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
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    const auto zero = [&](void *d, int64_t ld, int64_t rows, const int64_t *t) {
        return launch(xent_zero_kernel, rows < 8 * NUM_CU ? rows : 8 * NUM_CU, 256, stream, (uint16_t *)d, ld, rows, K,
                      t, ignore);
    };
    if (M == 0)
        return !dW || V == 0 || K == 0 || zero(dW, lddw, V, nullptr) ? TG_OK : TG_ERR_LAUNCH;
    Space s = {reinterpret_cast<char *>(ws)};
    const Buffers b = lay_out(s, p, M, V, true);
    IndexArgs ia = {};
    ia.target = target, ia.M = M, ia.V = V, ia.ignore = ignore;
    ia.head = b.head, ia.map = b.map, ia.col = b.col;
    ia.reduction = reduction, ia.dloss = dloss, ia.dlse = dlse, ia.lse = lse;
    ia.lse_c = b.lse, ia.cp = b.cp, ia.ct = b.ct;
    bool ok = launch(xent_index_kernel<true>, 1, INDEX_THREADS, stream, ia);
    ok = ok && gather_h(p, b, H, ldh, M, K, stream);
    if (dH)
        ok = ok && zero(dH, lddh, M, target);
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
        a.tiles_n = (int)cdiv(n, CLASS_BN[p.logits]);
        const int64_t grid = tiles(p.logits, M, n);
        switch (p.logits) {
        case C256:
            ok = ok && launch(xent_grad_kernel<E, T256<E, false, false>>, grid, 256, stream, a);
            break;
        case C128:
            ok = ok && launch(xent_grad_kernel<E, T128<E, false, false>>, grid, 256, stream, a);
            break;
        case C64X128:
            ok = ok && launch(xent_grad_kernel<E, T64x128<E, false, false>>, grid, 256, stream, a);
            break;
        default:
            ok = ok && launch(xent_grad_kernel<E, T64<E, false, false>>, grid, 256, stream, a);
        }
        if (dH) {
            d = {};
            d.g = {b.G, a.Gld, (int)M};
            d.w = {w.p, w.ld, (int)K};
            d.V = (int)n, d.split = (int)p.split, d.head = b.head;
            d.acc = b.acc, d.acc_rows = M, d.K8 = p.K8, d.add = v0 > 0;
            d.map = b.map, d.dH = dH, d.lddh = lddh, d.K = (int)K;
            d.vec = lddh % 8 == 0 && (uintptr_t)dH % 16 == 0;
            d.tiles_n = (int)cdiv(K, CLASS_BN[p.dh]), d.splits = p.splits;
            const int64_t g = tiles(p.dh, M, K) * p.splits;
            switch (p.dh) {
            case C256:
                ok = ok && launch(b.acc ? xent_dh_kernel<E, T256<E, false, true>, true> : xent_dh_kernel<E, T256<E, false, true>, false>, g, 256, stream, d);
                break;
            case C128:
                ok = ok && launch(b.acc ? xent_dh_kernel<E, T128<E, false, true>, true> : xent_dh_kernel<E, T128<E, false, true>, false>, g, 256, stream, d);
                break;
            default:
                ok = ok && launch(b.acc ? xent_dh_kernel<E, T64x128<E, false, true>, true> : xent_dh_kernel<E, T64x128<E, false, true>, false>, g, 256, stream, d);
            }
        }
        if (dW) {
            DwArgs x = {};
            x.g = {b.G, a.Gld, (int)n};
            x.h = {b.hc, p.K8, (int)K};
            x.head = b.head;
            x.dW = reinterpret_cast<uint16_t *>(dW) + v0 * lddw, x.lddw = lddw;
            x.V = (int)n, x.K = (int)K;
            x.vec = lddw % 8 == 0 && (uintptr_t)dW % 16 == 0;
            x.tiles_m = (int)cdiv(n, CLASS_BM[p.dw]), x.tiles_n = (int)cdiv(K, CLASS_BN[p.dw]);
            const int64_t g = tiles(p.dw, n, K);
            switch (p.dw) {
            case C256:
                ok = ok && launch(xent_dw_kernel<E, T256<E, true, true>>, g, 256, stream, x);
                break;
            case C128:
                ok = ok && launch(xent_dw_kernel<E, T128<E, true, true>>, g, 256, stream, x);
                break;
            default:
                ok = ok && launch(xent_dw_kernel<E, T64<E, true, true>>, g, 256, stream, x);
            }
        }
    }
    if (ok && dH && b.acc)
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
    const int st = validate(H, W, M, V, K, ldh, ldw);
    if (st != TG_OK || M == 0)
        return st;
    const Plan p = make_plan(H, W, M, V, K, ldh, ldw, backward_pass != 0);
    if (pieces)
        *pieces = p.pieces;
    if (name && name_len > 0) {
        const char *pre = p.compact ? "gather " : "", *pack = p.pack_w ? "pack " : "";
        if (backward_pass)
            snprintf(name, (size_t)name_len, "%s%sgrad_%s dh_%s_s%d dw_%s", pre, pack, CLASS_NAME[p.logits],
                     CLASS_NAME[p.dh], p.splits, CLASS_NAME[p.dw]);
        else
            snprintf(name, (size_t)name_len, "%s%sstats_%s", pre, pack, CLASS_NAME[p.logits]);
    }
    return TG_OK;
}
