// tg_ortho.hip — Newton–Schulz orthogonalisation of a projection's update.  See
// include/tg_ortho.h for the contract.
//
// With s the shorter and l the longer side, a step is three products:
//
//   gram     A = X·Xᵀ (tall: Xᵀ·X)   s×s over l   symmetric
//   square   B = b·A + c·A²          s×s over s   symmetric
//   update   X ← a·X + B·X (X·B)     s×l over s
//
// The symmetric products compute the tiles of the lower triangle and store
// each twice, as it is and transposed: s·(s+1)·l instead of 2·s²·l flop.
// X is never transposed: its row-major image is the K-major operand of X·Xᵀ
// and X·B and the transposed one of Xᵀ·X and B·X.
//
// Numbers.  An early step multiplies small singular values by a ≈ 3.4, so an
// error made in X then is amplified by up to 3.4⁵ ≈ 485 where the value it
// perturbs is small beside the norm; X is therefore carried in fp32, and only
// the products' operands are rounded.  Near convergence B ≈ −2.4·I plus a small
// remainder; rounding B as a whole would put an error of 2.4·2⁻¹² on every
// row, so the diagonals of A and B are kept in fp32 (d, e) and the products
// run on the off-diagonal parts O and P alone:
//
//   A² = d_i² or (d_i + d_j)·O_ij, plus O·O        B = diag(e) + P
//   X ← (a + e_i)·X + P·X
//
// Measured against 64 bits on Gaussian, low-rank-plus-noise and 1/k spectra:
// 1.66e-3 to 1.85e-3 (relative, 2-norm) for the bfloat16 result, 1.66e-3 being
// the rounding of the result itself; with B rounded whole 2.1e-3 to 2.7e-3,
// with X carried in 16 bits up to 4.4e-3, with bfloat16 operands 1e-2 to 3e-2.
// Where many directions are far below the norm, or the rank is low, the rounding of
// the operands shows more (include/tg_ortho.h has the figures): up to 64 rows they
// are held in two parts, above in one, as two would take three times the products.
//
// Operands are binary16 times 2^14 (X) and 2^12 (O, P): entries of X start near
// (rows·cols)^-1/2 and of O near 1/s·l^-1/2, far below binary16's 2^-14, and the
// scales keep 11 bits down to 2^-28 and 2^-26.
#include "proj_tile.hpp"

#include <algorithm>
#include <math.h>
#include <stdio.h>

#include "tg_gemm.h"
#include "tg_ortho.h"

namespace {
using namespace pt;

typedef _Float16 half_t;
typedef half_t half4 __attribute__((ext_vector_type(4)));

constexpr float X_SCALE = 16384.0f, S_SCALE = 4096.0f;  // of X, and of O and P

// ------------------------------------------------------------- norm, scaling
constexpr int NORM_BLOCKS = 1024;  // most partial sums per matrix
// Sums of squares in 64 bits: fp32 squares would overflow or vanish for
// elements beyond 1e19 or below 1e-23.  Reads G once, 16 bytes per lane where
// rows follow each other without gaps.
template <typename G>
__global__ __launch_bounds__(256) void ns_norm_kernel(const G *g, int64_t rows, int64_t cols, int64_t ld,
                                                      int64_t stride, int blocks, double *part)
{
    __shared__ double sh[4];
    const int m = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    const G *p = g + (int64_t)m * stride;
    double s = 0.0;
    const auto add = [&](G v) {
        const double x = (double)(float)v;
        s += x * x;
    };
    const int64_t total = rows * cols;
    if (ld == cols) {
        constexpr int N = 16 / sizeof(G);
        typedef G vec __attribute__((ext_vector_type(N)));
        const int64_t chunks = total / N;
#pragma unroll 4
        for (int64_t i = (int64_t)blk * 256 + threadIdx.x; i < chunks; i += (int64_t)blocks * 256) {
            vec v;
            __builtin_memcpy(&v, p + i * N, 16);  // at an element's alignment
#pragma unroll
            for (int e = 0; e < N; ++e)
                add(v[e]);
        }
        for (int64_t i = chunks * N + (int64_t)blk * 256 + threadIdx.x; i < total; i += (int64_t)blocks * 256)
            add(p[i]);
    } else {
        for (int64_t r = blk; r < rows; r += blocks)
            for (int64_t c = threadIdx.x; c < cols; c += 256)
                add(p[r * ld + c]);
    }
    for (int o = 32; o; o >>= 1)
        s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0)
        sh[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        part[blockIdx.x] = ((sh[0] + sh[1]) + sh[2]) + sh[3];
}

// 1 / (norm + eps): 0 for a zero matrix without eps, which stays zero; NaN where
// the norm is not finite, so that the whole result is.
__device__ inline double inverse(double by)
{
    return by == 0.0 ? 0.0 : by < (double)INFINITY ? 1.0 / by : (double)NAN;
}

// X0 = G / (norm + eps) in fp32, and its binary16 image padded with zeros to
// ldx columns.  With `out` (no steps) the result itself.  Bound by memory: 66 us
// for 8×1024×4096 fp32 (335 MB, the rate of a copy; loads element by element
// took 84).
template <typename G>
__global__ __launch_bounds__(256) void ns_scale_kernel(const G *g, int64_t rows, int64_t cols, int64_t ld,
                                                       int64_t stride, int norm_blocks, const double *part, float eps,
                                                       int blocks, float *x, half_t *xh, int64_t ldx, __bf16 *out,
                                                       int64_t ldo, int64_t o_stride)
{
    const int m = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    const G *p = g + (int64_t)m * stride;
    const int64_t per = ldx / 4, total = rows * per, step = (int64_t)blocks * 256;
    typedef G four __attribute__((ext_vector_type(4)));
    const auto load = [&](int64_t r, int64_t c) {
        four v = {(G)0.0f, (G)0.0f, (G)0.0f, (G)0.0f};
        if (c + 4 <= cols) {
            __builtin_memcpy(&v, p + r * ld + c, sizeof v);  // at an element's alignment
            return v;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < cols)
                v[e] = p[r * ld + c + e];
        return v;
    };
    // the first elements are on their way while the norm is added up
    int64_t i = (int64_t)blk * 256 + threadIdx.x;
    int64_t r = i / per, c = (i - r * per) * 4;
    four next = {(G)0.0f, (G)0.0f, (G)0.0f, (G)0.0f};
    if (i < total)
        next = load(r, c);
    double s = 0.0;
    for (int z = threadIdx.x & 63; z < norm_blocks; z += 64)
        s += part[m * norm_blocks + z];
    for (int o = 32; o; o >>= 1)
        s += __shfl_xor(s, o);
    const double inv = inverse(sqrt(s) + (double)eps);
    for (; i < total; i += step) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = c + e < cols ? (float)((double)(float)next[e] * inv) : 0.0f;
        const int64_t at_r = r, at_c = c;
        if (i + step < total) {
            r = (i + step) / per, c = (i + step - r * per) * 4;
            next = load(r, c);
        }
        if (out) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at_c + e < cols)
                    out[(int64_t)m * o_stride + at_r * ldo + at_c + e] = (__bf16)v[e];
            continue;
        }
        half4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = (half_t)(v[e] * X_SCALE);
        const int64_t at = ((int64_t)m * rows + at_r) * ldx + at_c;
        *reinterpret_cast<f32x4 *>(x + at) = v;
        *reinterpret_cast<half4 *>(xh + at) = h;
    }
}

// -------------------------------------------------------- symmetric products
// One workgroup per BM×BM tile of a lower triangle.  gram: SQUARE false, the
// product of X with itself; square: the product of O with itself, joined with
// O's own tile and the diagonal.
struct SymArgs {
    Operand x;           // one operand on both sides
    int64_t x_stride;    // elements between matrices
    int K, s;
    half_t *out;         // s × lds, zero columns from s on
    int64_t lds;
    float *diag;         // lds per matrix, s of them set
    const half_t *o;     // square: A's off-diagonal part and diagonal
    const float *d;
    float b, c;
    int tri, total;      // tiles per matrix, workgroups
    float *part;         // gram in splits: [matrix][tile][split], each a tile in the accumulators' order
    int splits, per_split;  // and the K of one (a multiple of 64)
};
template <typename T, bool SQUARE>
__device__ __attribute__((always_inline)) void sym_epilogue(const SymArgs &a, half_t *smem, int m, int tm, int tn,
                                                            f32x4 (&acc)[T::TM][T::TN])
{
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int fr = lane & 15, fc = 4 * (lane >> 4);
    const int r0 = tm * T::BM + wm * T::WTM, c0 = tn * T::BN + wn * T::WTN;
    half_t *out = a.out + (int64_t)m * a.s * a.lds;
    float *__restrict__ diag = a.diag + (int64_t)m * a.lds;
    const half_t *__restrict__ o = SQUARE ? a.o + (int64_t)m * a.s * a.lds : nullptr;
    const float *__restrict__ d = SQUARE ? a.d + (int64_t)m * a.lds : nullptr;
    barrier_lds();
    half_t *stg = smem + wave * T::WTM * T::WTN;
    // Rows and columns past s hold copies of the last ones' products here (and
    // their loads are clamped alike); they are cleared in the staged block.
    // Columns outside, rows inside, so that a column's loads (O, d) are all in
    // flight before they are used.
    float dr[T::TM];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
        dr[i] = SQUARE ? d[imin(r0 + 16 * i + fr, a.s - 1)] : 0.0f;
    // the diagonal: in fp32, and out of the staged block (below)
    if (r0 == c0 && fr >= fc && fr < fc + 4)
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            float y = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                y = fr == fc + v ? acc[i][i][v] : y;
            if (r0 + 16 * i + fr < a.s)
                diag[r0 + 16 * i + fr] = SQUARE
                                             ? a.b * dr[i] + a.c * (dr[i] * dr[i] + y * (1.0f / (S_SCALE * S_SCALE)))
                                             : y * (1.0f / (X_SCALE * X_SCALE));
        }
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
        const int col = imin(c0 + 16 * j + fc, (a.s - 1) & ~3);
        f32x4 dc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        half4 oh[T::TM];
        if constexpr (SQUARE) {
            dc = *reinterpret_cast<const f32x4 *>(d + col);
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
                oh[i] = *reinterpret_cast<const half4 *>(o + (int64_t)imin(r0 + 16 * i + fr, a.s - 1) * a.lds + col);
        }
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            half4 h;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float y = acc[i][j][v] * (SQUARE ? 1.0f / S_SCALE : S_SCALE / (X_SCALE * X_SCALE));
                if constexpr (SQUARE) {
                    const float f = (float)oh[i][v];
                    y = a.b * f + a.c * ((dr[i] + dc[v]) * f + y);
                }
                h[v] = (half_t)y;  // the rounding of the next product's operand
            }
            *reinterpret_cast<half4 *>(stg + stage_off<T::WTN>(16 * i + fr, 16 * j + fc)) = h;
        }
    }
    if (r0 == c0 && fr >= fc && fr < fc + 4)
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
            stg[stage_off<T::WTN>(16 * i + fr, 16 * i + fr)] = (half_t)0.0f;
    if (imax(r0, c0) + T::WTM > a.s)
        clear_outside<half_t, T::WTM, T::WTN>(stg, a.s - r0, a.s - c0, lane);
    store_block<half_t, T::WTM, T::WTN, true>(stg, out, a.lds, r0, c0, a.s, (int)a.lds, true, nullptr, lane);
    if (tm != tn)
        store_block_transposed<half_t, T::WTM, T::WTN>(stg, out, a.lds, c0, r0, a.s, (int)a.lds, lane);
}
__device__ inline void sym_tile(const SymArgs &a, int logical, int &m, int &tm, int &tn)
{
    m = logical / a.tri;
    triangle_tile(logical - m * a.tri, tm, tn);
    tm = uniform(tm), tn = uniform(tn);
}
template <typename T, bool SQUARE>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void ns_sym_kernel(
    SymArgs a)
{
    static_assert(T::BM == T::BN && T::WTM == T::WTN, "symmetric tiles");
    __shared__ __attribute__((aligned(1024))) half_t smem[T::LDS_ELEMS];
    int m, tm, tn;
    sym_tile(a, xcd_contiguous(blockIdx.x, a.total), m, tm, tn);
    Operand x = a.x;
    x.p = reinterpret_cast<const half_t *>(x.p) + (int64_t)m * a.x_stride;
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    T::run(smem, x, x, tm * T::BM, tn * T::BN, a.K, acc);
    sym_epilogue<T, SQUARE>(a, smem, m, tm, tn, acc);
}
// A short side of few tiles and a long one: the contraction in splits, one
// workgroup each, and a second kernel that adds them in order and stores the tile.
template <typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(2) void ns_gram_split_kernel(SymArgs a)
{
    __shared__ __attribute__((aligned(1024))) half_t smem[T::LDS_ELEMS];
    const int logical = xcd_contiguous(blockIdx.x, a.total);
    const int z = logical % a.splits;
    int m, tm, tn;
    sym_tile(a, logical / a.splits, m, tm, tn);
    const int from = z * a.per_split, len = imax(imin(a.per_split, a.K - from), 0);
    Operand x = a.x;
    x.p = reinterpret_cast<const half_t *>(x.p) + (int64_t)m * a.x_stride + (T::TA ? (int64_t)from * x.ld : from);
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    if (len > 0)
        T::run(smem, x, x, tm * T::BM, tn * T::BN, len, acc);
    f32x4 *out = reinterpret_cast<f32x4 *>(a.part + (int64_t)logical * T::BM * T::BN) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            out[(i * T::TN + j) * T::THREADS] = acc[i][j];
}
template <typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(2) void ns_gram_join_kernel(SymArgs a)
{
    __shared__ __attribute__((aligned(1024))) half_t smem[T::BM * T::BN];
    int m, tm, tn;
    sym_tile(a, blockIdx.x, m, tm, tn);
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    const f32x4 *in =
        reinterpret_cast<const f32x4 *>(a.part + (int64_t)blockIdx.x * a.splits * T::BM * T::BN) + threadIdx.x;
#pragma unroll 2
    for (int z = 0; z < a.splits; ++z, in += T::BM * T::BN / 4)
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
                acc[i][j] += in[(i * T::TN + j) * T::THREADS];
    sym_epilogue<T, false>(a, smem, m, tm, tn, acc);
}

// ------------------------------------------------------------------- update
// X ← (a + e)·X + P·X, or with the factors on the right for a tall X.  Reads
// and writes X in fp32 in place (each element by the one lane that owns it)
// and writes the next operand; the last step writes the bfloat16 result.
struct UpdateArgs {
    Operand l, r;           // left and right operand
    int64_t l_stride, r_stride;
    int K, rows, cols;
    float *x;
    half_t *xh;
    int64_t ldx;
    const float *e;
    int64_t lds;
    float a;
    __bf16 *out;
    int64_t ldo, o_stride;
    bool vec;
    int tiles_m, tiles_n, total;
};
template <typename T, bool TALL, bool LAST>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(T::BM *T::BN > 128 * 128 ? 1 : 2) void ns_update_kernel(
    UpdateArgs a)
{
    __shared__ __attribute__((aligned(1024))) half_t smem[T::LDS_ELEMS];
    const int tiles = a.tiles_m * a.tiles_n;
    const int logical = xcd_contiguous(blockIdx.x, a.total);
    const int m = logical / tiles;
    int tm, tn;
    grouped_tile<4>(logical - m * tiles, a.tiles_m, a.tiles_n, tm, tn);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    Operand l = a.l, r = a.r;
    l.p = reinterpret_cast<const half_t *>(l.p) + (int64_t)m * a.l_stride;
    r.p = reinterpret_cast<const half_t *>(r.p) + (int64_t)m * a.r_stride;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int fr = lane & 15, fc = 4 * (lane >> 4);
    const int r0 = m0 + wm * T::WTM, c0 = n0 + wn * T::WTN;
    const float *__restrict__ e = a.e + (int64_t)m * a.lds;
    float *x = a.x + (int64_t)m * a.rows * a.ldx;
    // X some columns of blocks ahead of its use, the first of them before the
    // last K-tile: their loads (1 KiB each) are what the epilogue waits for,
    // and with one column ahead it waited 35 us of a 4096×4096 step's 150.
    // Loads are clamped; what lies past cols is cleared in the staged block.
    constexpr int DEPTH = 4, EARLY = T::BM * T::BN >= 256 * 256 ? (LAST ? 0 : 1) : DEPTH - 1;
    f32x4 xs[DEPTH][T::TM];
    auto fetch = [&](int j) __attribute__((always_inline)) {
        const int col = imin(c0 + 16 * j + fc, (a.cols - 1) & ~3);
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
            xs[j % DEPTH][i] = *reinterpret_cast<const f32x4 *>(x + (int64_t)imin(r0 + 16 * i + fr, a.rows - 1) * a.ldx + col);
    };
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    T::run(smem, l, r, m0, n0, a.K, acc, [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < EARLY && j < T::TN; ++j)
            fetch(j);
    });
    barrier_lds();
    half_t *stg = smem + wave * T::WTM * T::WTN;
    float er[T::TM];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
        er[i] = TALL ? 0.0f : e[imin(r0 + 16 * i + fr, a.rows - 1)];
#pragma unroll
    for (int j = EARLY; j < DEPTH - 1 && j < T::TN; ++j)
        fetch(j);
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
        const int col = c0 + 16 * j + fc;
        if (j + DEPTH - 1 < T::TN)
            fetch(j + DEPTH - 1);
        f32x4 ec = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (TALL)
            ec = *reinterpret_cast<const f32x4 *>(e + imin(col, (a.cols - 1) & ~3));
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            f32x4 v = xs[j % DEPTH][i];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = (a.a + (TALL ? ec[k] : er[i])) * v[k] + acc[i][j][k] * (1.0f / (S_SCALE * X_SCALE));
            const int at = stage_off<T::WTN>(16 * i + fr, 16 * j + fc);
            if constexpr (LAST) {
                typename El<__bf16>::v4 h;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[k] = (__bf16)v[k];
                *reinterpret_cast<typename El<__bf16>::v4 *>(reinterpret_cast<__bf16 *>(stg) + at) = h;
            } else {
                half4 h;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[k] = (half_t)(v[k] * X_SCALE);
                if (r0 + 16 * i + fr < a.rows && col < a.cols)
                    *reinterpret_cast<f32x4 *>(x + (int64_t)(r0 + 16 * i + fr) * a.ldx + col) = v;
                *reinterpret_cast<half4 *>(stg + at) = h;
            }
        }
    }
    if (!LAST && c0 + T::WTN > a.cols)
        clear_outside<half_t, T::WTM, T::WTN>(stg, T::WTM, a.cols - c0, lane);
    if constexpr (LAST)
        store_block<__bf16, T::WTM, T::WTN>(reinterpret_cast<const __bf16 *>(stg), a.out + (int64_t)m * a.o_stride,
                                            a.ldo, r0, c0, a.rows, a.cols, a.vec, nullptr, lane);
    else
        store_block<half_t, T::WTM, T::WTN, true>(stg, a.xh + (int64_t)m * a.rows * a.ldx, a.ldx, r0, c0, a.rows,
                                            (int)a.ldx, true, nullptr, lane);
}

// --------------------------------------------------- short sides of up to 128
// With s at most 128 the s×s operands fit one workgroup's LDS, and launches, not
// arithmetic, are what the chain of products above costs (some 4 us each for well
// under one of work).  Two forms:
//
//   both sides at most 128   one workgroup runs the whole iteration, X (fp32)
//                            in registers, the operands in LDS: 128x128 25 us
//                            with the chain 65, 64x128 19, 64x64 14;
//   a long side              two launches per step, and X read and written once
//                            in it.  The strip kernel takes X in strips of 64
//                            columns: update, store, and the strip's part of the
//                            next Gram matrix, from the image it already holds.
//                            The core kernel adds the parts and, in the workgroup
//                            that finishes last, does the square: 1x64x4096 60 us
//                            with the chain 87, of which the core's wait for
//                            memory, three trips there one after the other, is
//                            the longest part (6 us of each step's 11).
//
// X is held with the shorter side as rows (`flip`: G and the result are
// transposed on the way), so that no other form is needed.  Images are IM rows,
// 64 or 128.
//
// The rounding of X's operand spreads evenly over the s directions of the
// short side, and a direction whose singular value is small beside the norm is
// amplified by up to 485 afterwards: with many directions that stays below the
// result's own rounding for most spectra, with a few it does not (a 2×2 matrix of condition
// 100 came out 6e-3 off, one of 2×100 and rank one 3e-2).  The forms for 64 rows
// of the short side, however long the other, therefore hold each operand as
// the sum of two binary16 values and take three products for each (the fourth,
// of the two low parts, is below fp32).
//
// LDS images are row-major, C columns; chunk c of row r at c ^ swz(r), so that the
// sixteen rows of a K-major fragment read fall on sixteen bank groups; the
// transposed reads of X (two rows to a 32-byte group) take two passes.
using V8h = El<half_t>::v8;
template <int C>
__host__ __device__ constexpr int image_off(int r, int c)
{
    return r * C + (((c >> 3) ^ (C == 128 ? r & 15 : (r >> 1) & 7)) << 3) + (c & 7);
}
template <int C>
__device__ inline V8h image_kmajor(const half_t *img, int row, int kk, int fr, int fh)
{
    return *reinterpret_cast<const V8h *>(img + image_off<C>(row + fr, kk * 32 + 8 * fh));
}
template <int C>
__device__ inline V8h image_trans(const half_t *img, int col, int kk, int fr, int fh)
{
    const int k = kk * 32 + 8 * fh + (fr >> 2), c = col + 4 * (fr & 3);
    union {
        s16x4 h[2];
        V8h v;
    } u;
    u.h[0] = lds_read_tr(img + image_off<C>(k, c));
    u.h[1] = lds_read_tr(img + image_off<C>(k + 4, c));
    return u.v;
}
// acc += the block at row r0, column c0 of A·Bᵀ (B K-major) or A·B (TRANS), over
// 32·KK of K; a_part, b_part: where the low parts begin.
template <int PARTS, int CA, int CB, bool TRANS, int KK, int TM, int TN>
__device__ inline void image_product(const half_t *ai, int a_part, const half_t *bi, int b_part, int r0, int c0,
                                     int fr, int fh, f32x4 (&acc)[TM][TN])
{
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
        V8h fa[PARTS][TM], fb[PARTS][TN];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fa[p][i] = image_kmajor<CA>(ai + p * a_part, r0 + 16 * i, kk, fr, fh);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[p][j] = TRANS ? image_trans<CB>(bi + p * b_part, c0 + 16 * j, kk, fr, fh)
                                 : image_kmajor<CB>(bi + p * b_part, c0 + 16 * j, kk, fr, fh);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                acc[i][j] = El<half_t>::mfma(fb[0][j], fa[0][i], acc[i][j]);
                if constexpr (PARTS == 2) {
                    acc[i][j] = El<half_t>::mfma(fb[1][j], fa[0][i], acc[i][j]);
                    acc[i][j] = El<half_t>::mfma(fb[0][j], fa[1][i], acc[i][j]);
                }
            }
    }
}
// v at row r, columns c .. c+3 as the operand's image holds it; returns the value
// held.
template <int PARTS, int C>
__device__ inline f32x4 image_put(half_t *img, int part, int r, int c, const f32x4 &v)
{
    half4 h;
    f32x4 held;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = (half_t)v[k];
        held[k] = (float)h[k];
    }
    *reinterpret_cast<half4 *>(img + image_off<C>(r, c)) = h;
    if constexpr (PARTS == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = (half_t)(v[k] - held[k]);
            held[k] += (float)h[k];
        }
        *reinterpret_cast<half4 *>(img + part + image_off<C>(r, c)) = h;
    }
    return held;
}
template <int TM, int TN>
__device__ inline void zero_blocks(f32x4 (&acc)[TM][TN])
{
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// The s×s part of a step for one workgroup: waves 2 × WN over the IM×IM image.
template <int IM>
struct Small {
    static constexpr int WM = 2, WN = IM == 128 ? 4 : 2, WAVES = WM * WN;
    static constexpr int TM = IM / WM / 16, TN = IM / WN / 16;
    static constexpr int PARTS = IM == 128 ? 1 : 2, PART = IM * IM;
    static_assert(IM == 128 || IM == 64, "two forms");
    struct Core {
        half_t oi[PARTS * PART], pi[PARTS * PART];
        float d[IM], e[IM];
    };
    // acc: X·Xᵀ of the X_SCALE images.  Leaves P and e in `m`; two barriers, and
    // the caller passes one before it reads them.
    __device__ static void square(Core &m, f32x4 (&acc)[TM][TN], float kb, float kc, int r0, int c0, int fr, int fh)
    {
        f32x4 o[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    o[i][j][v] = acc[i][j][v] * (S_SCALE / (X_SCALE * X_SCALE));
                if (r0 + 16 * i == c0 + 16 * j)  // a block of the diagonal
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (fr == 4 * fh + v) {
                            m.d[r0 + 16 * i + fr] = acc[i][j][v] * (1.0f / (X_SCALE * X_SCALE));
                            o[i][j][v] = 0.0f;
                        }
                o[i][j] = image_put<PARTS, IM>(m.oi, PART, r0 + 16 * i + fr, c0 + 16 * j + 4 * fh, o[i][j]);
            }
        __syncthreads();
        zero_blocks(acc);
        image_product<PARTS, IM, IM, false, IM / 32>(m.oi, PART, m.oi, PART, r0, c0, fr, fh, acc);
        float dr[TM];
        f32x4 dc[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            dr[i] = m.d[r0 + 16 * i + fr];
#pragma unroll
        for (int j = 0; j < TN; ++j)
            dc[j] = *reinterpret_cast<const f32x4 *>(m.d + c0 + 16 * j + 4 * fh);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                f32x4 h;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float f = o[i][j][v], y = acc[i][j][v] * (1.0f / S_SCALE);
                    h[v] = kb * f + kc * ((dr[i] + dc[j][v]) * f + y);
                }
                if (r0 + 16 * i == c0 + 16 * j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (fr == 4 * fh + v) {
                            m.e[r0 + 16 * i + fr] =
                                kb * dr[i] + kc * (dr[i] * dr[i] + acc[i][j][v] * (1.0f / (S_SCALE * S_SCALE)));
                            h[v] = 0.0f;
                        }
                image_put<PARTS, IM>(m.pi, PART, r0 + 16 * i + fr, c0 + 16 * j + 4 * fh, h);
            }
        __syncthreads();
    }
};
struct SmallArgs {
    const void *g;
    int64_t ld, stride;
    __bf16 *out;
    int64_t ldo, o_stride;
    int s, l;      // rows and columns of the image
    bool flip;     // the image is G transposed
    int steps;
    float eps;
    float k[3 * TG_NS_MAX_STEPS];
};
// X is IM rows of L columns: 64×64 and 64×128 in two parts, 128×128 in one.  Two
// parts of 64 rows are no more work than one of 128: 1x64x128 takes 19 us, as
// 128×128 in one part 23, 512x64x128 33 and 50.
template <typename G, int IM, int L>
__global__ __launch_bounds__(Small<IM>::WAVES * 64) void ns_small_kernel(SmallArgs a)
{
    using S = Small<IM>;
    constexpr int TM = S::TM, TN = L / S::WN / 16, PARTS = S::PARTS;  // a wave's blocks of X
    constexpr int XPART = IM * L;
    __shared__ __attribute__((aligned(1024))) half_t xi[PARTS * XPART];
    __shared__ __attribute__((aligned(1024))) typename S::Core m;
    __shared__ double sums[S::WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fh = lane >> 4;
    const int r0 = wave / S::WN * (IM / S::WM), c0 = wave % S::WN * (L / S::WN);
    const int g0 = wave % S::WN * (IM / S::WN);  // the wave's columns of the Gram matrix
    const G *g = reinterpret_cast<const G *>(a.g) + (int64_t)blockIdx.x * a.stride;

    // X in the accumulators' layout: block (i, j), row fr, columns 4·fh .. +3
    f32x4 x[TM][TN];
    double s2 = 0.0;
    typedef G four __attribute__((ext_vector_type(4)));
    const bool rows4 = !a.flip && a.ld % 4 == 0 && (uintptr_t)g % sizeof(four) == 0;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int r = r0 + 16 * i + fr, c = c0 + 16 * j + 4 * fh;
            x[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (rows4 && r < a.s && c + 4 <= a.l) {
                const four v = *reinterpret_cast<const four *>(g + r * a.ld + c);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[i][j][k] = (float)v[k];
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r < a.s && c + k < a.l)
                        x[i][j][k] = (float)g[a.flip ? (c + k) * a.ld + r : r * a.ld + c + k];
            }
        }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                s2 += (double)x[i][j][v] * (double)x[i][j][v];
    for (int o = 32; o; o >>= 1)
        s2 += __shfl_xor(s2, o);
    if (lane == 0)
        sums[wave] = s2;
    __syncthreads();
    s2 = 0.0;
    for (int w = 0; w < S::WAVES; ++w)
        s2 += sums[w];
    const double inv = inverse(sqrt(s2) + (double)a.eps);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                x[i][j][v] = (float)((double)x[i][j][v] * inv);

#pragma unroll 1
    for (int t = 0; t < a.steps; ++t) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                f32x4 v;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = x[i][j][k] * X_SCALE;
                image_put<PARTS, L>(xi, XPART, r0 + 16 * i + fr, c0 + 16 * j + 4 * fh, v);
            }
        __syncthreads();
        f32x4 gram[TM][S::TN];
        zero_blocks(gram);
        image_product<PARTS, L, L, false, L / 32>(xi, XPART, xi, XPART, r0, g0, fr, fh, gram);
        S::square(m, gram, a.k[3 * t + 1], a.k[3 * t + 2], r0, g0, fr, fh);
        f32x4 acc[TM][TN];
        zero_blocks(acc);
        image_product<PARTS, IM, L, true, IM / 32>(m.pi, S::PART, xi, XPART, r0, c0, fr, fh, acc);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const float f = a.k[3 * t] + m.e[r0 + 16 * i + fr];
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    x[i][j][v] = f * x[i][j][v] + acc[i][j][v] * (1.0f / (S_SCALE * X_SCALE));
        }
        __syncthreads();  // every wave has read X's image
    }
    __bf16 *out = a.out + (int64_t)blockIdx.x * a.o_stride;
    const bool out4 = !a.flip && a.ldo % 4 == 0 && (uintptr_t)out % 8 == 0;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int r = r0 + 16 * i + fr, c = c0 + 16 * j + 4 * fh;
            El<__bf16>::v4 h;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[k] = (__bf16)x[i][j][k];
            if (out4 && r < a.s && c + 4 <= a.l) {
                *reinterpret_cast<El<__bf16>::v4 *>(out + r * a.ldo + c) = h;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (r < a.s && c + k < a.l)
                        out[a.flip ? (c + k) * a.ldo + r : r * a.ldo + c + k] = h[k];
            }
        }
}

// ------------------------------------------------- a short and a long side
constexpr int STRIP = 64;  // columns
struct ThinArgs {
    const void *g;
    int64_t ld, g_stride;
    __bf16 *out;
    int64_t ldo, o_stride;
    int s, l;
    bool flip;
    const double *part;      // sums of squares
    int norm_blocks;
    float eps;
    float *x;                // [matrix][s][lp], lp = l rounded up to whole strips
    int64_t lp;
    int strips, per, groups; // strips per matrix, per workgroup, workgroups per matrix
    float *gram;             // [matrix][group][IM·IM], the accumulators' order
    float *sum;              // [matrix][IM·IM]
    half_t *p;               // [matrix][PARTS·IM·IM], the image's order
    float *e;                // [matrix][IM]
    unsigned *arrived;       // [matrix]
    int reducers;            // core workgroups per matrix
    float ka, kb, kc;
};
// FIRST: X from G.  LAST: the result, and no Gram matrix.  (Both: no steps.)
template <typename G, int IM, bool FIRST, bool LAST>
__global__ __launch_bounds__(Small<IM>::WAVES * 64) void ns_strip_kernel(ThinArgs a)
{
    using S = Small<IM>;
    constexpr int PARTS = S::PARTS, THREADS = S::WAVES * 64;
    constexpr int TM = S::TM, TN = STRIP / S::WN / 16;  // a wave's blocks of a strip
    __shared__ __attribute__((aligned(1024))) half_t xi[PARTS * IM * STRIP];
    __shared__ __attribute__((aligned(1024))) half_t pi[FIRST ? 8 : PARTS * IM * IM];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fh = lane >> 4;
    const int m = blockIdx.x / a.groups, group = blockIdx.x % a.groups;
    const int r0 = wave / S::WN * (IM / S::WM), c0 = wave % S::WN * (STRIP / S::WN);
    const int g0 = wave % S::WN * (IM / S::WN);  // the wave's columns of the Gram matrix
    if (threadIdx.x == 0 && group == 0)
        a.arrived[m] = 0;
    double inv = 0.0;
    if constexpr (FIRST) {
        double s2 = 0.0;
        for (int i = lane; i < a.norm_blocks; i += 64)
            s2 += a.part[m * a.norm_blocks + i];
        for (int o = 32; o; o >>= 1)
            s2 += __shfl_xor(s2, o);
        inv = inverse(sqrt(s2) + (double)a.eps);
    } else {
        const uint4 *src = reinterpret_cast<const uint4 *>(a.p + (int64_t)m * PARTS * IM * IM);
#pragma unroll
        for (int i = 0; i < PARTS * IM * IM / 8 / THREADS; ++i)
            reinterpret_cast<uint4 *>(pi)[i * THREADS + threadIdx.x] = src[i * THREADS + threadIdx.x];
    }
    float er[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i)
        er[i] = FIRST ? 0.0f : a.ka + a.e[m * IM + r0 + 16 * i + fr];
    const G *g = reinterpret_cast<const G *>(a.g) + (int64_t)m * a.g_stride;
    float *xm = a.x + (int64_t)m * a.s * a.lp;
    __bf16 *out = a.out + (int64_t)m * a.o_stride;
    typedef G four __attribute__((ext_vector_type(4)));
    const bool out4 = !a.flip && a.ldo % 4 == 0 && (uintptr_t)out % 8 == 0;
    f32x4 gram[S::TM][S::TN];
    zero_blocks(gram);
#pragma unroll 1
    for (int q = group * a.per; q < imin((group + 1) * a.per, a.strips); ++q) {
        f32x4 x[TM][TN];
        zero_blocks(x);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int r = r0 + 16 * i + fr;
                const int64_t c = (int64_t)q * STRIP + c0 + 16 * j + 4 * fh;
                if (r >= a.s)
                    continue;
                if constexpr (!FIRST) {
                    x[i][j] = *reinterpret_cast<const f32x4 *>(xm + r * a.lp + c);
                } else if (!a.flip && c + 4 <= a.l) {
                    four v;
                    __builtin_memcpy(&v, g + r * a.ld + c, sizeof v);  // at an element's alignment
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[i][j][k] = (float)((double)(float)v[k] * inv);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (c + k < a.l)
                            x[i][j][k] = (float)((double)(float)g[a.flip ? (c + k) * a.ld + r : r * a.ld + c + k] * inv);
                }
            }
        auto put = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    f32x4 v;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = x[i][j][k] * X_SCALE;
                    image_put<PARTS, STRIP>(xi, IM * STRIP, r0 + 16 * i + fr, c0 + 16 * j + 4 * fh, v);
                }
        };
        if constexpr (!FIRST) {
            put();
            __syncthreads();
            f32x4 acc[TM][TN];
            zero_blocks(acc);
            image_product<PARTS, IM, STRIP, true, IM / 32>(pi, IM * IM, xi, IM * STRIP, r0, c0, fr, fh, acc);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[i][j][k] = er[i] * x[i][j][k] + acc[i][j][k] * (1.0f / (S_SCALE * X_SCALE));
            __syncthreads();  // every wave has read the image
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int r = r0 + 16 * i + fr;
                const int64_t c = (int64_t)q * STRIP + c0 + 16 * j + 4 * fh;
                if (r >= a.s)
                    continue;
                if constexpr (!LAST) {
                    *reinterpret_cast<f32x4 *>(xm + r * a.lp + c) = x[i][j];
                } else {
                    El<__bf16>::v4 h;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = (__bf16)x[i][j][k];
                    if (out4 && c + 4 <= a.l) {
                        *reinterpret_cast<El<__bf16>::v4 *>(out + r * a.ldo + c) = h;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (c + k < a.l)
                                out[a.flip ? (c + k) * a.ldo + r : r * a.ldo + c + k] = h[k];
                    }
                }
            }
        if constexpr (!LAST) {
            put();
            __syncthreads();
            image_product<PARTS, STRIP, STRIP, false, STRIP / 32>(xi, IM * STRIP, xi, IM * STRIP, r0, g0, fr, fh, gram);
            __syncthreads();
        }
    }
    if constexpr (!LAST) {
        f32x4 *dst = reinterpret_cast<f32x4 *>(a.gram + ((int64_t)m * a.groups + group) * IM * IM) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
                dst[(i * S::TN + j) * THREADS] = gram[i][j];
    }
}
// Adds the groups' Gram matrices (each workgroup a range of elements, in the
// groups' order), and in the workgroup that arrives last squares the sum.
template <int IM>
__global__ __launch_bounds__(Small<IM>::WAVES * 64) void ns_core_kernel(ThinArgs a)
{
    using S = Small<IM>;
    constexpr int THREADS = S::WAVES * 64, PARTS = S::PARTS;
    __shared__ __attribute__((aligned(1024))) typename S::Core core;
    __shared__ bool last;
    const int m = blockIdx.x / a.reducers, part = blockIdx.x % a.reducers;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fh = lane >> 4;
    const int r0 = wave / S::WN * (IM / S::WM), c0 = wave % S::WN * (IM / S::WN);
    const f32x4 *in = reinterpret_cast<const f32x4 *>(a.gram + (int64_t)m * a.groups * IM * IM);
    constexpr int n = IM * IM / 4;
    f32x4 acc[S::TM][S::TN];
    if (a.reducers == 1) {
        zero_blocks(acc);
        for (int z = 0; z < a.groups; ++z)
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
                    acc[i][j] += in[(int64_t)z * n + (i * S::TN + j) * THREADS + threadIdx.x];
    } else {
        // this workgroup's elements, the groups in `slices` parts side by side
        unsigned long long *sum = reinterpret_cast<unsigned long long *>(a.sum) + (int64_t)m * n * 2;
        const int each = n / a.reducers, width = imin(each, THREADS), slices = THREADS / width;
        const int slice = threadIdx.x / width, z0 = slice * a.groups / slices, z1 = (slice + 1) * a.groups / slices;
        f32x4 *joined = reinterpret_cast<f32x4 *>(core.oi);
        for (int i = part * each + threadIdx.x % width; i < (part + 1) * each; i += width) {
            f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (int z = z0; z < z1; ++z)
                v += in[(int64_t)z * n + i];
            if (slices > 1) {  // then each thread has one element
                joined[threadIdx.x] = v;
                __syncthreads();
                if (slice)
                    break;
                for (int q = 1; q < slices; ++q)
                    v += joined[q * width + threadIdx.x];
            }
            // past the caches: another workgroup reads it
            union {
                f32x4 f;
                unsigned long long u[2];
            } w = {v};
            for (int h = 0; h < 2; ++h)
                __hip_atomic_store(sum + 2 * i + h, w.u[h], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        wait_vmem<0>();  // each wave's sums are out before the arrival is
        __syncthreads();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(a.arrived + m, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   (unsigned)a.reducers - 1;
        __syncthreads();
        if (!last)
            return;
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j) {
                union {
                    unsigned long long u[2];
                    f32x4 f;
                } w;
                for (int h = 0; h < 2; ++h)
                    w.u[h] = __hip_atomic_load(sum + 2 * ((i * S::TN + j) * THREADS + threadIdx.x) + h, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
                acc[i][j] = w.f;
            }
    }
    S::square(core, acc, a.kb, a.kc, r0, c0, fr, fh);
    uint4 *dst = reinterpret_cast<uint4 *>(a.p + (int64_t)m * PARTS * IM * IM);
#pragma unroll
    for (int i = 0; i < PARTS * IM * IM / 8 / THREADS; ++i)
        dst[i * THREADS + threadIdx.x] = reinterpret_cast<const uint4 *>(core.pi)[i * THREADS + threadIdx.x];
    if (threadIdx.x < IM)
        a.e[m * IM + threadIdx.x] = core.e[threadIdx.x];
}

// -------------------------------------------------------------------- plans
// Tile classes, chosen by tile_time for the whole batch.  One 256×256 or
// 192×192 workgroup per CU, two of the smaller ones.  192×192 is there for the
// counts that leave most of a round of 256×256 tiles empty: the lower triangle
// of 4096×4096 is 136 tiles of 256 (or 528 of 128, one round of 512 and 16 more)
// but 253 of 192, one round of the 256 CUs.
enum Class { C256, C192, C128, C64, CLASSES };
const char *const CLASS_NAME[] = {"256x256", "192x192", "128x128", "64x64"};
constexpr TileClass SYM_CLASS[] = {{256, 256, 1, 1.40, 1.40, 14.0},
                                   {192, 192, 1, 1.15, 1.15, 5.0},
                                   {128, 128, 2, 1.10, 0.50, 5.0},
                                   {64, 64, 2, 0.50, 0.27, 4.0}};
// the update's epilogue reads and writes X in fp32 besides
constexpr TileClass UPD_CLASS[] = {{256, 256, 1, 1.50, 1.50, 35.0},
                                   {192, 192, 1, 1.25, 1.25, 18.0},
                                   {128, 128, 2, 1.10, 0.50, 14.0},
                                   {64, 64, 2, 0.50, 0.27, 4.5}};
template <bool TA, bool TB>
using T256 = Tile<half_t, 256, 256, 2, 2, 2, TA, TB>;
template <bool TA, bool TB>
using T192 = Tile<half_t, 192, 192, 2, 2, 2, TA, TB>;
template <bool TA, bool TB>
using T128 = Tile<half_t, 128, 128, 2, 2, 2, TA, TB>;
template <bool TA, bool TB>
using T64 = Tile<half_t, 64, 64, 2, 2, 3, TA, TB>;

struct Plan {
    int64_t s, l, ldx, lds;
    bool tall, small, thin;
    int image;        // rows of the short side's image (small, thin)
    int columns;      // of X's image (small)
    int strips, per, groups, reducers;  // thin
    Class gram, square, upd;
    int splits;       // of the gram product's contraction
    int64_t per_split;
    int norm_blocks;
};
int64_t triangle(int64_t s, int b)
{
    const int64_t t = cdiv(s, b);
    return t * (t + 1) / 2;
}
Plan make_plan(int64_t batch, int64_t rows, int64_t cols)
{
    Plan p;
    p.tall = rows > cols;
    p.small = std::max(rows, cols) <= 128;
    p.s = std::min(rows, cols), p.l = std::max(rows, cols);
    p.ldx = round_up(cols, BK), p.lds = round_up(p.s, BK);
    p.image = p.s <= 64 ? 64 : 128, p.columns = p.l <= 64 ? 64 : 128;
    // Up to 64 rows always take the strips: the operands in two parts are right
    // where one is not, and nothing was slower (1x64x200 59 -> 48 us, 1x16x14336
    // 124 -> 73, 1x64x131072 676 -> 162, 32x64x14336 502 -> 316, 300x64x300
    // 164 -> 136).  Up to 128 rows a workgroup's Gram matrix is twice a strip's
    // bytes, which pays for one matrix (1x100x200 69 -> 63, 1x128x14336
    // 171 -> 132) and for long ones (8x128x4096 160 -> 140, 32x128x14336
    // 1013 -> 730), and not for several short ones (16x128x1024 99 with the
    // chain, 135 with strips; 32x100x1000 126 and 143).
    p.thin = !p.small && (p.s <= 64 || (p.s <= 128 && (batch == 1 || p.l >= 2048)));
    // Workgroups: with 512 and 256 in all, 32x64x14336 takes 313 and 432 us and
    // 1x64x131072 158 and 178; for 128 rows 8x128x4096 154 and 139, 1x128x131072
    // 281 and 259, 128x128x2048 402 and 390.
    p.strips = (int)cdiv(p.l, STRIP);
    const int64_t most = std::max((int64_t)1, std::min((int64_t)p.strips, (p.image == 64 ? 512 : 256) / batch));
    p.per = (int)cdiv(p.strips, most);
    p.groups = (int)cdiv(p.strips, p.per);
    // Workgroups that add up one matrix's parts: each costs a write past the
    // caches and an arrival, so few where the matrices are many (8x64x4096 with
    // 32 each 109 us, with 8 each 95; 1x64x131072 with 16 171, with 32 157).
    p.reducers = 1;
    while (p.groups > 4 && p.reducers < (p.groups <= 16 ? 8 : 32) && 2 * p.reducers * batch <= 64)
        p.reducers *= 2;
    const auto best = [&](const TileClass *cls, auto count, int64_t k) {
        int c = 0;
        for (int i = 1; i < CLASSES; ++i)
            if (tile_time(cls[i], count(cls[i].bm), cdiv(k, BK)) < tile_time(cls[c], count(cls[c].bm), cdiv(k, BK)))
                c = i;
        return (Class)c;
    };
    const auto sym = [&](int b) { return batch * triangle(p.s, b); };
    p.gram = best(SYM_CLASS, sym, p.l);
    p.square = best(SYM_CLASS, sym, p.s);
    // splits that fill the slots of a small class, at least 4 K-tiles each, where
    // with the second kernel (some 5 us and the partial tiles twice through the
    // caches) they are faster than the best class without.  (The larger classes and
    // the square product are not split: their split forms are not built, and what
    // they would take is not measured.)
    p.splits = 1, p.per_split = p.l;
    const int64_t kt = cdiv(p.l, BK);
    double t = tile_time(SYM_CLASS[p.gram], sym(SYM_CLASS[p.gram].bm), kt);
    for (const Class c : {C128, C64}) {
        const TileClass &k = SYM_CLASS[c];
        const int64_t n = sym(k.bm), splits = std::min((int64_t)NUM_CU * k.per_cu / n, kt / 4);
        if (splits < 2)
            continue;
        const int64_t per = cdiv(kt, splits), used = cdiv(kt, per);
        const double with = tile_time(k, n * used, per) + 5.0 + (double)(n * used * k.bm * k.bm) * 8.0 / 4e6;
        if (with < t)
            t = with, p.gram = c, p.splits = (int)used, p.per_split = per * BK;
    }
    p.upd = best(UPD_CLASS, [&](int b) { return batch * cdiv(rows, b) * cdiv(cols, b); }, p.s);
    const int64_t want = cdiv(rows * cols, 8192);
    p.norm_blocks = (int)std::max((int64_t)1, std::min(want, std::max((int64_t)1, std::min((int64_t)NORM_BLOCKS, 4096 / batch))));
    return p;
}
struct Buffers {
    double *part;
    float *x, *d, *e, *gram, *sum;
    half_t *xh[2], *o, *p;
    unsigned *arrived;
    int64_t used = 0;
};
Buffers lay_out(char *base, const Plan &p, int64_t batch, int64_t rows)
{
    Buffers b = {};
    if (p.small)
        return b;
    const auto take = [&](auto *&ptr, int64_t n) {
        using X = std::remove_reference_t<decltype(*ptr)>;
        ptr = base ? reinterpret_cast<X *>(base + b.used) : nullptr;
        b.used += round_up(n * (int64_t)sizeof(X), 256);
    };
    take(b.part, batch * p.norm_blocks);
    if (p.thin) {
        const int64_t im2 = (int64_t)p.image * p.image;
        take(b.x, batch * p.s * p.strips * STRIP);
        take(b.gram, batch * p.groups * im2);
        take(b.sum, batch * im2);
        take(b.p, batch * im2 * 2);
        take(b.e, batch * p.image);
        take(b.arrived, batch);
        return b;
    }
    take(b.x, batch * rows * p.ldx);
    take(b.xh[0], batch * rows * p.ldx);
    take(b.xh[1], batch * rows * p.ldx);
    take(b.o, batch * p.s * p.lds);
    take(b.p, batch * p.s * p.lds);
    take(b.gram, p.splits > 1 ? batch * triangle(p.s, SYM_CLASS[p.gram].bm) * p.splits * SYM_CLASS[p.gram].bm *
                                    SYM_CLASS[p.gram].bm
                              : 0);
    take(b.d, batch * p.lds);
    take(b.e, batch * p.lds);
    return b;
}

int validate_sizes(int64_t batch, int64_t rows, int64_t cols)
{
    if (batch < 0 || rows < 0 || cols < 0)
        return TG_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 31;
    if (rows >= MAX_DMA_LD - BK || cols >= MAX_DMA_LD - BK || batch >= lim)
        return TG_ERR_TOO_LARGE;
    if (batch * cdiv(rows, 64) >= lim || batch * cdiv(rows, 64) * cdiv(cols, 64) >= MAX_GRID)
        return TG_ERR_TOO_LARGE;
    return TG_OK;
}

template <typename T>
int64_t update_grid(UpdateArgs &u, int64_t batch)
{
    u.tiles_m = (int)cdiv(u.rows, T::BM), u.tiles_n = (int)cdiv(u.cols, T::BN);
    u.total = (int)(batch * u.tiles_m * u.tiles_n);
    return u.total;
}
template <template <bool, bool> class T, bool TALL>
bool launch_step(UpdateArgs u, bool last, int64_t batch, void *stream)
{
    // wide: P (K-major) · X (transposed); tall: X (K-major) · P (K-major, symmetric)
    using Tl = T<false, !TALL>;
    const int64_t g = update_grid<Tl>(u, batch);
    return last ? launch(ns_update_kernel<Tl, TALL, true>, g, Tl::THREADS, stream, u)
                : launch(ns_update_kernel<Tl, TALL, false>, g, Tl::THREADS, stream, u);
}
template <bool TALL>
bool launch_step_class(Class c, const UpdateArgs &u, bool last, int64_t batch, void *stream)
{
    return c == C256   ? launch_step<T256, TALL>(u, last, batch, stream)
           : c == C192 ? launch_step<T192, TALL>(u, last, batch, stream)
           : c == C128 ? launch_step<T128, TALL>(u, last, batch, stream)
                       : launch_step<T64, TALL>(u, last, batch, stream);
}
template <template <bool, bool> class T, bool SQUARE, bool TRANS>
bool launch_sym(SymArgs a, int64_t batch, void *stream)
{
    using Tl = T<TRANS, TRANS>;
    a.tri = (int)triangle(a.s, Tl::BM);
    a.total = (int)(batch * a.tri);
    return launch(ns_sym_kernel<Tl, SQUARE>, a.total, Tl::THREADS, stream, a);
}
template <template <bool, bool> class T, bool TRANS>
bool launch_gram_split(SymArgs a, int64_t batch, void *stream)
{
    using Tl = T<TRANS, TRANS>;
    a.tri = (int)triangle(a.s, Tl::BM);
    a.total = (int)(batch * a.tri * a.splits);
    return launch(ns_gram_split_kernel<Tl>, a.total, Tl::THREADS, stream, a) &&
           launch(ns_gram_join_kernel<T<false, false>>, batch * a.tri, Tl::THREADS, stream, a);
}
template <bool SQUARE, bool TRANS>
bool launch_sym_class(Class c, const SymArgs &a, int64_t batch, void *stream)
{
    return c == C256   ? launch_sym<T256, SQUARE, TRANS>(a, batch, stream)
           : c == C192 ? launch_sym<T192, SQUARE, TRANS>(a, batch, stream)
           : c == C128 ? launch_sym<T128, SQUARE, TRANS>(a, batch, stream)
                       : launch_sym<T64, SQUARE, TRANS>(a, batch, stream);
}

template <typename G, int IM>
bool thin_steps(const Plan &p, ThinArgs a, int64_t batch, int steps, const float *coefficients, void *stream)
{
    constexpr int THREADS = Small<IM>::WAVES * 64;
    const int64_t grid = batch * p.groups;
    if (steps == 0)
        return launch(ns_strip_kernel<G, IM, true, true>, grid, THREADS, stream, a);
    bool ok = launch(ns_strip_kernel<G, IM, true, false>, grid, THREADS, stream, a);
    for (int t = 0; ok && t < steps; ++t) {
        a.ka = coefficients[3 * t], a.kb = coefficients[3 * t + 1], a.kc = coefficients[3 * t + 2];
        ok = launch(ns_core_kernel<IM>, batch * p.reducers, THREADS, stream, a) &&
             (t == steps - 1 ? launch(ns_strip_kernel<G, IM, false, true>, grid, THREADS, stream, a)
                             : launch(ns_strip_kernel<G, IM, false, false>, grid, THREADS, stream, a));
    }
    return ok;
}

template <typename G>
int newton_schulz(const void *g, void *o, int64_t batch, int64_t rows, int64_t cols, int64_t ldg, int64_t g_stride,
                  int64_t ldo, int64_t o_stride, int steps, const float *coefficients, float eps, void *ws,
                  int64_t ws_bytes, void *stream)
{
    const int st = validate_sizes(batch, rows, cols);
    if (st != TG_OK)
        return st;
    if (steps < 0 || steps > TG_NS_MAX_STEPS || !(eps >= 0.0f) || ldg < cols || ldo < cols || g_stride < 0)
        return TG_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || cols == 0)
        return TG_OK;
    if (batch > 1 && o_stride < (rows - 1) * ldo + cols)
        return TG_ERR_INVALID_ARG;
    const Plan p = make_plan(batch, rows, cols);
    const Buffers b = lay_out(reinterpret_cast<char *>(ws), p, batch, rows);
    if (!g || !o || (b.used > 0 && (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < b.used)))
        return TG_ERR_INVALID_ARG;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    const G *src = reinterpret_cast<const G *>(g);
    __bf16 *out = reinterpret_cast<__bf16 *>(o);
    float k[3 * TG_NS_MAX_STEPS] = {};
    for (int i = 0; i < 3 * steps; ++i) {
        static const float standard[3] = {3.4445f, -4.7750f, 2.0315f};
        k[i] = coefficients ? coefficients[i] : standard[i % 3];
    }
    if (p.small) {
        SmallArgs a = {g, ldg, g_stride, out, ldo, o_stride, (int)p.s, (int)p.l, p.tall, steps, eps, {}};
        memcpy(a.k, k, sizeof k);
        const bool ok = p.columns == 64 ? launch(ns_small_kernel<G, 64, 64>, batch, Small<64>::WAVES * 64, stream, a)
                        : p.image == 64 ? launch(ns_small_kernel<G, 64, 128>, batch, Small<64>::WAVES * 64, stream, a)
                                        : launch(ns_small_kernel<G, 128, 128>, batch, Small<128>::WAVES * 64, stream, a);
        return ok ? TG_OK : TG_ERR_LAUNCH;
    }
    bool ok = launch(ns_norm_kernel<G>, batch * p.norm_blocks, 256, stream, src, rows, cols, ldg, g_stride,
                     p.norm_blocks, b.part);
    if (p.thin) {
        ThinArgs a = {};
        a.g = g, a.ld = ldg, a.g_stride = g_stride, a.out = out, a.ldo = ldo, a.o_stride = o_stride;
        a.s = (int)p.s, a.l = (int)p.l, a.flip = p.tall;
        a.part = b.part, a.norm_blocks = p.norm_blocks, a.eps = eps;
        a.x = b.x, a.lp = (int64_t)p.strips * STRIP, a.strips = p.strips, a.per = p.per, a.groups = p.groups;
        a.gram = b.gram, a.sum = b.sum, a.p = b.p, a.e = b.e, a.arrived = b.arrived, a.reducers = p.reducers;
        ok = ok && (p.image == 64 ? thin_steps<G, 64>(p, a, batch, steps, k, stream)
                                  : thin_steps<G, 128>(p, a, batch, steps, k, stream));
        return ok ? TG_OK : TG_ERR_LAUNCH;
    }
    const int64_t chunks = cdiv(rows * p.ldx / 4, 256);
    const int scale_blocks = (int)std::max((int64_t)1, std::min(chunks, std::max((int64_t)1, 8 * NUM_CU / batch)));
    ok = ok && launch(ns_scale_kernel<G>, batch * scale_blocks, 256, stream, src, rows, cols, ldg, g_stride,
                      p.norm_blocks, (const double *)b.part, eps, scale_blocks, b.x, b.xh[0], p.ldx,
                      steps == 0 ? out : nullptr, ldo, o_stride);
    for (int t = 0; ok && t < steps; ++t) {
        const half_t *xh = b.xh[t & 1];
        SymArgs a = {};
        a.x = {xh, p.ldx, (int)p.s};
        a.x_stride = rows * p.ldx;
        a.K = (int)(p.tall ? rows : round_up(cols, 8));
        a.s = (int)p.s, a.out = b.o, a.lds = p.lds, a.diag = b.d;
        a.part = b.gram, a.splits = p.splits, a.per_split = (int)p.per_split;
        if (p.splits > 1 && p.gram == C128)
            ok = p.tall ? launch_gram_split<T128, true>(a, batch, stream) : launch_gram_split<T128, false>(a, batch, stream);
        else if (p.splits > 1)
            ok = p.tall ? launch_gram_split<T64, true>(a, batch, stream) : launch_gram_split<T64, false>(a, batch, stream);
        else
            ok = p.tall ? launch_sym_class<false, true>(p.gram, a, batch, stream)
                        : launch_sym_class<false, false>(p.gram, a, batch, stream);
        SymArgs q = {};
        q.x = {b.o, p.lds, (int)p.s};
        q.x_stride = p.s * p.lds;
        q.K = (int)round_up(p.s, 8);
        q.s = (int)p.s, q.out = b.p, q.lds = p.lds, q.diag = b.e, q.o = b.o, q.d = b.d;
        q.b = k[3 * t + 1], q.c = k[3 * t + 2];
        ok = ok && launch_sym_class<true, false>(p.square, q, batch, stream);
        UpdateArgs u = {};
        const Operand x = {xh, p.ldx, (int)(p.tall ? rows : cols)}, pm = {b.p, p.lds, (int)p.s};
        u.l = p.tall ? x : pm, u.r = p.tall ? pm : x;
        u.l_stride = p.tall ? rows * p.ldx : p.s * p.lds, u.r_stride = p.tall ? p.s * p.lds : rows * p.ldx;
        u.K = (int)(p.tall ? round_up(p.s, 8) : p.s);
        u.rows = (int)rows, u.cols = (int)cols, u.x = b.x, u.xh = b.xh[(t + 1) & 1], u.ldx = p.ldx;
        u.e = b.e, u.lds = p.lds, u.a = k[3 * t];
        u.out = out, u.ldo = ldo, u.o_stride = o_stride;
        u.vec = ldo % 8 == 0 && o_stride % 8 == 0 && (uintptr_t)out % 16 == 0;
        const bool last = t == steps - 1;
        ok = ok && (p.tall ? launch_step_class<true>(p.upd, u, last, batch, stream)
                           : launch_step_class<false>(p.upd, u, last, batch, stream));
    }
    return ok ? TG_OK : TG_ERR_LAUNCH;
}

}  // namespace

extern "C" int64_t tg_newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols)
{
    if (validate_sizes(batch, rows, cols) != TG_OK)
        return -1;
    if (batch == 0 || rows == 0 || cols == 0)
        return 0;
    return lay_out(nullptr, make_plan(batch, rows, cols), batch, rows).used;
}

extern "C" int tg_newton_schulz_f32(const void *G, void *O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                                    int64_t g_stride, int64_t ldo, int64_t o_stride, int steps,
                                    const float *coefficients, float eps, void *workspace, int64_t workspace_bytes,
                                    void *stream)
{
    return newton_schulz<float>(G, O, batch, rows, cols, ldg, g_stride, ldo, o_stride, steps, coefficients, eps,
                                workspace, workspace_bytes, stream);
}

extern "C" int tg_newton_schulz_f16(const void *G, void *O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                                    int64_t g_stride, int64_t ldo, int64_t o_stride, int steps,
                                    const float *coefficients, float eps, void *workspace, int64_t workspace_bytes,
                                    void *stream)
{
    return newton_schulz<_Float16>(G, O, batch, rows, cols, ldg, g_stride, ldo, o_stride, steps, coefficients, eps,
                                   workspace, workspace_bytes, stream);
}

extern "C" int tg_newton_schulz_bf16(const void *G, void *O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                                     int64_t g_stride, int64_t ldo, int64_t o_stride, int steps,
                                     const float *coefficients, float eps, void *workspace, int64_t workspace_bytes,
                                     void *stream)
{
    return newton_schulz<__bf16>(G, O, batch, rows, cols, ldg, g_stride, ldo, o_stride, steps, coefficients, eps,
                                 workspace, workspace_bytes, stream);
}

extern "C" int tg_newton_schulz_plan(int64_t batch, int64_t rows, int64_t cols, char *name, int64_t name_len)
{
    if (name && name_len > 0)
        name[0] = 0;
    const int st = validate_sizes(batch, rows, cols);
    if (st != TG_OK || batch == 0 || rows == 0 || cols == 0)
        return st;
    const Plan p = make_plan(batch, rows, cols);
    if (name && name_len > 0 && p.small)
        snprintf(name, (size_t)name_len, "small_%d", p.columns);
    else if (name && name_len > 0 && p.thin)
        snprintf(name, (size_t)name_len, "thin_%d", p.image);
    else if (name && name_len > 0)
        snprintf(name, (size_t)name_len, "%s gram_%s%s square_%s update_%s", p.tall ? "tall" : "wide",
                 CLASS_NAME[p.gram], p.splits > 1 ? "_split" : "", CLASS_NAME[p.square], CLASS_NAME[p.upd]);
    return TG_OK;
}
