// tg_grouped.hip — products of rows grouped by expert.  See include/tg_grouped.h
// for the contract.
//
// One launch covers all experts: the output is cut into tiles expert by expert,
// and a workgroup finds its tile from `ends` itself (a scan over the experts, 64
// at a time), so that nothing of the routing passes through the host.  The grid is
// an upper bound: experts' last tile rows are partly empty, so that E of them
// may be added to M rows' tiles; workgroups past the last tile leave at once.
//
// The tile product is that of proj_tile.hpp; with few rows an expert it is bound by
// streaming W, with many by the matrix cores.
#include "proj_tile.hpp"

#include <algorithm>
#include <math.h>
#include <stdio.h>

#include "tg_gemm.h"
#include "tg_grouped.h"

namespace {
using namespace pt;

// ------------------------------------------------------------------- groups
// Workgroup id → tile where tiles differ in length, as those of weights with few
// and many rows do: each XCD takes 32 consecutive tiles (one for each of its compute
// units) of every 256, so that all eight work on the same experts at a time.  (With one
// eighth of all tiles for each XCD, the XCD with the largest expert ends last: dW of
// 16384 rows in 8 experts of 14336×4096, the largest with 1.8 times the mean,
// 2633 us instead of 1707; Y 1580 instead of 1529, as its tiles share more.)
__host__ __device__ constexpr int xcd_chunks(int bid, int total)
{
    constexpr int EACH = NUM_CU / NUM_XCD;
    const int whole = total / NUM_CU * NUM_CU;
    if (bid >= whole)
        return whole + xcd_contiguous(bid - whole, total - whole);
    const int xcd = bid % NUM_XCD, local = bid / NUM_XCD;
    return (local / EACH * NUM_XCD + xcd) * EACH + local % EACH;
}

// Inclusive scan of values >= 0 over a wave, in DPP moves: within rows of 16 lanes,
// then each row's last value on to the rows behind it (0 comes in from outside).
template <typename Op>
__device__ inline int scan64(int x, Op op)
{
#if defined(__HIP_DEVICE_COMPILE__)
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));  // row_shr:1, 2, 4, 8
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));  // row_bcast:15 to rows 1 and 3
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));  // row_bcast:31 to rows 2 and 3
#endif
    return x;
}
// Where expert idx's rows end (past the experts: 0, which changes nothing).
__device__ inline int group_end(const int64_t *ends, int E, int M, int idx)
{
    if (idx >= E)
        return 0;
    const int64_t x = ends[idx];
    return (int)(x < 0 ? 0 : x > M ? M : x);
}
// 64 experts from `base` on, one to a lane: first row, end, and the tile rows up to
// and with it.  `row` and `tiles`: the end and the tile rows of the experts before.
template <int BM>
__device__ inline void scan_groups(const int64_t *ends, int E, int M, int base, int lane, int row, int tiles,
                                   int &lo, int &hi, int &upto)
{
    hi = scan64(imax(group_end(ends, E, M, base + lane), row), [](int x, int y) { return imax(x, y); });
    lo = __shfl_up(hi, 1);
    lo = lane == 0 ? row : lo;
    upto = tiles + scan64((hi - lo + BM - 1) / BM, [](int x, int y) { return x + y; });
}
// The experts' tile rows, as far as a wave's registers hold them: the last 64.
struct Groups {
    int lo, hi, upto;  // of this lane's expert
    int row, tiles;    // where the rows behind the experts begin; tile rows of the experts
    int all;           // tile rows with the rows behind
};
template <int BM>
__device__ inline Groups find_groups(const int64_t *ends, int E, int M)
{
    Groups g = {};
    for (int base = 0; base < E; base += 64) {
        scan_groups<BM>(ends, E, M, base, lane_id(), g.row, g.tiles, g.lo, g.hi, g.upto);
        g.row = __builtin_amdgcn_readlane(g.hi, 63), g.tiles = __builtin_amdgcn_readlane(g.upto, 63);
    }
    g.all = g.tiles + (M - g.row + BM - 1) / BM;
    return g;
}
struct Tile2d {
    int e, lo, rows;  // expert (E: the rows behind), its first row and their number
    int tm, tn;
};
// Tile `logical` of all: expert by expert, in groups of four tile rows.
template <int BM>
__device__ inline Tile2d find_tile(Groups g, const int64_t *ends, int E, int M, int tiles_n, int logical)
{
    const int tile_row = logical / tiles_n;
    Tile2d t = {E, g.row, M - g.row, 0, 0};
    int first = g.tiles;
    if (tile_row < g.tiles) {
        int base = 0;
        if (E > 64) {  // otherwise the registers still hold the only scan
            g.row = g.tiles = 0;
            for (;; base += 64) {
                scan_groups<BM>(ends, E, M, base, lane_id(), g.row, g.tiles, g.lo, g.hi, g.upto);
                if (__builtin_amdgcn_readlane(g.upto, 63) > tile_row)
                    break;
                g.row = __builtin_amdgcn_readlane(g.hi, 63), g.tiles = __builtin_amdgcn_readlane(g.upto, 63);
            }
        }
        const int at = uniform(__builtin_ctzll(__ballot(g.upto > tile_row)));
        t.e = base + at;
        t.lo = __builtin_amdgcn_readlane(g.lo, at);
        t.rows = __builtin_amdgcn_readlane(g.hi, at) - t.lo;
        first = __builtin_amdgcn_readlane(g.upto, at) - (t.rows + BM - 1) / BM;
    }
    grouped_tile<4>(logical - first * tiles_n, (t.rows + BM - 1) / BM, tiles_n, t.tm, t.tn);
    return t;
}
// The last round of a launch: where its tiles are at most half of the workgroups that
// run at once, each is cut into parts along the sum, whose fp32 sums go to the
// workspace and are added by a kernel behind it, in order.
constexpr int MIN_PART = 8, MAX_PARTS = 32;  // K-tiles of a part, and parts
struct Split {
    int full, rest, parts;  // tiles of whole rounds; the others; parts of each of those
};
__device__ inline Split split_tiles(int total, int slots, int ktiles)
{
    Split s;
    s.full = total / slots * slots;
    s.rest = total - s.full;
    s.parts = s.rest > 0 ? imax(imin(imin(slots / s.rest, ktiles / MIN_PART), MAX_PARTS), 1) : 1;
    return s;
}
// Expert e's rows.
__device__ inline void find_rows(const int64_t *ends, int M, int e, int &lo, int &rows)
{
    const int lane = lane_id(), end = group_end(ends, e + 1, M, e);
    int before = 0;
    for (int i = lane; i < e; i += 64)
        before = imax(before, group_end(ends, e, M, i));
    lo = __builtin_amdgcn_readlane(scan64(before, [](int x, int y) { return imax(x, y); }), 63);
    rows = uniform(imax(end - lo, 0));
}

// ------------------------------------------------------------------ products
// The tile product with one stage of LDS instead of rings: 128×128 in 32 KiB and at
// most 128 registers, so that four workgroups run on a compute unit.  A workgroup
// waits for each K-tile; the others' products, loads and stores fill the time.  For
// short sums, where a tile's first loads and its stores take longer than its
// products (dW from 128 rows in 8 experts of 14336×4096, 940 MB: 156 us, 302 with the
// rings; from 4096 rows in 64 experts of 1024×2048 69 and 102, in 8 of 4096×4096 159 and
// 190; dX of 8192 rows in the 64 85 and 92).
template <typename E, bool TA, bool TB>
struct OneStage : Tile<E, 128, 128, 2, 2, 2, TA, TB> {
    using T = Tile<E, 128, 128, 2, 2, 2, TA, TB>;
    using V8 = typename El<E>::v8;
    static constexpr int LDS_ELEMS = T::STAGE_A + T::STAGE_B;
    static constexpr bool FIRST = false;  // the partial K-tile comes last, masked
    static_assert(T::BM * T::BN <= LDS_ELEMS, "the block's 16-bit image fits the stage");

    // K a multiple of 8 where an operand is K-major
    __device__ static __attribute__((always_inline)) void run(E *smem, const Operand &a, const Operand &b, int x0a,
                                                              int x0b, int K, f32x4 (&acc)[T::TM][T::TN])
    {
        x0a = uniform(x0a), x0b = uniform(x0b), K = uniform(K);
        const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), wm = wave / T::WN, wn = wave % T::WN;
        E *const sa = smem, *const sb = smem + T::STAGE_A;
        uint32_t a_off[T::PA], b_off[T::PB];
        T::template dma_offsets<TA, T::BM>(a_off, a.ld, x0a, a.extent, lane, wave);
        T::template dma_offsets<TB, T::BN>(b_off, b.ld, x0b, b.extent, lane, wave);
        const char *const a_base = uniform(reinterpret_cast<const char *>(a.p) + 2 * (TA ? (int64_t)x0a : x0a * a.ld));
        const char *const b_base = uniform(reinterpret_cast<const char *>(b.p) + 2 * (TB ? (int64_t)x0b : x0b * b.ld));
        // a transposed operand's buffer ends with its last K row; a K-major one's
        // chunks past K are masked
        const auto rsrc = [](const char *base, int64_t ld, bool trans, int t, int k, int x0) {
            return __builtin_amdgcn_make_buffer_rsrc((void *)(base + t * (trans ? 2 * BK * ld : 2 * BK)), (short)0,
                                                     trans ? imax(k * (2 * (int)ld) - 2 * x0, 0) : DMA_RANGE, BUFFER_WORD3);
        };
        const int kc = 8 * ((lane & 7) ^ kmajor_swz(8 * wave + (lane >> 3)));
        const auto read = [&](const E *st, auto trans, auto bx, int x, int kk) {
            constexpr int BX = decltype(bx)::value;
            if constexpr (decltype(trans)::value) {
                const E *from = st + trans_off<BX>(8 * (lane >> 4) + ((lane & 15) >> 2), x + 4 * (lane & 3)) + kk * 32 * BX;
                union {
                    s16x4 h[2];
                    V8 v;
                } u;
                u.h[0] = lds_read_tr(from);
                u.h[1] = lds_read_tr(from + 4 * BX);
                return u.v;
            } else {
                return *reinterpret_cast<const V8 *>(st + kmajor_off(x + (lane & 15), kk * 4 + (lane >> 4)));
            }
        };
        for (int t = 0; t * BK < K; ++t) {
            const int k = imin(K - t * BK, BK);
            const auto ra = rsrc(a_base, a.ld, TA, t, k, x0a), rb = rsrc(b_base, b.ld, TB, t, k, x0b);
            const bool past = kc >= k;
            if (t > 0)
                barrier_lds();  // every wave has read the K-tile before
#pragma unroll
            for (int p = 0; p < T::PA; ++p)
                dma16(ra, sa + (p * T::NW + wave) * 512, !TA && past ? DMA_OOB : a_off[p]);
#pragma unroll
            for (int p = 0; p < T::PB; ++p)
                dma16(rb, sb + (p * T::NW + wave) * 512, !TB && past ? DMA_OOB : b_off[p]);
            wait_vmem<0>();
            barrier_lds();
            for (int kk = 0; kk < (k > 32 ? 2 : 1); ++kk) {
                V8 fa[T::TM], fb[T::TN];
#pragma unroll
                for (int q = 0; q < T::TM; ++q)
                    fa[q] = read(sa, std::bool_constant<TA>{}, std::integral_constant<int, T::BM>{}, wm * T::WTM + q * 16, kk);
#pragma unroll
                for (int q = 0; q < T::TN; ++q)
                    fb[q] = read(sb, std::bool_constant<TB>{}, std::integral_constant<int, T::BN>{}, wn * T::WTN + q * 16, kk);
#pragma unroll
                for (int i = 0; i < T::TM; ++i)
#pragma unroll
                    for (int j = 0; j < T::TN; ++j)
                        acc[i][j] = El<E>::mfma(fb[j], fa[i], acc[i][j]);
            }
        }
    }
};
// Waves of a tile's kernels on each SIMD unit.
template <typename T>
constexpr int waves_of()
{
    return T::LDS_ELEMS <= 128 * 128 ? 4 : T::BM * T::BN > 128 * 128 ? 1 : 2;
}

template <typename E, typename T>
__device__ inline void store_tile(E *smem, const f32x4 (&acc)[T::TM][T::TN], E *D, int64_t ld, int m0, int n0, int rows,
                                  int cols, bool vec, bool nt)
{
    using V4 = typename El<E>::v4;
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
                d[v] = (E)acc[i][j][v];
            *reinterpret_cast<V4 *>(stg + stage_off<T::WTN>(16 * i + fr, 16 * j + fc)) = d;
        }
    if (nt)
        store_block<E, T::WTM, T::WTN, false, true>(stg, D, ld, m0 + wm * T::WTM, n0 + wn * T::WTN, rows, cols, vec,
                                                    nullptr, lane);
    else
        store_block<E, T::WTM, T::WTN>(stg, D, ld, m0 + wm * T::WTM, n0 + wn * T::WTN, rows, cols, vec, nullptr, lane);
}
// Zeros where a tile's product is over nothing.
template <typename E, int BM, int BN, int THREADS>
__device__ inline void zero_tile(E *D, int64_t ld, int m0, int n0, int rows, int cols)
{
    const int r1 = imin(rows, m0 + BM), c1 = imin(cols, n0 + BN);
    for (int r = m0 + (int)threadIdx.x / 64; r < r1; r += THREADS / 64)
        for (int c = n0 + lane_id(); c < c1; c += 64)
            D[r * ld + c] = (E)0.0f;
}

// A tile's fp32 sums, as the lanes hold them, to place `at` of the workspace's parts.
template <typename T>
__device__ inline void store_part(const f32x4 (&acc)[T::TM][T::TN], float *parts, int64_t at)
{
    f32x4 *to = reinterpret_cast<f32x4 *>(parts + at * (T::BM * T::BN)) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            to[(i * T::TN + j) * T::THREADS] = acc[i][j];
}
// `n` parts of a tile added in order, `step` places apart: of the 16-row strips that the
// tile's waves hold, strip i.
template <typename E, typename T>
__device__ inline void join_parts(const float *parts, int64_t at, int64_t step, int n, int i, E *D, int64_t ld, int m0,
                                  int n0, int rows, int cols, bool vec)
{
    using V4 = typename El<E>::v4;
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6);
    const int row = m0 + wave / T::WN * T::WTM + 16 * i + (lane & 15);
    const int col0 = n0 + wave % T::WN * T::WTN + 4 * (lane >> 4);
    E *d = D + (int64_t)row * ld;
    const f32x4 *from = reinterpret_cast<const f32x4 *>(parts + at * (T::BM * T::BN)) + threadIdx.x;
    f32x4 sum[T::TN];
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
        sum[j] = from[(i * T::TN + j) * T::THREADS];
    for (int z = 1; z < n; ++z) {
        from += step * (T::BM * T::BN / 4);
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            sum[j] += from[(i * T::TN + j) * T::THREADS];
    }
    if (row >= rows)
        return;
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
        const int col = col0 + 16 * j;
        V4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (E)sum[j][e];
        if (vec && col + 4 <= cols) {
            *reinterpret_cast<V4 *>(d + col) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < cols)
                    d[col + e] = v[e];
        }
    }
}

// Y (K-major W) and dX (transposed W): tiles of rows of one expert.
struct RowsArgs {
    const void *a, *w;
    const int64_t *ends;
    void *d;
    int64_t lda, ldw, w_stride, ldd;
    int M, E;
    int inner;     // K (Y) or N (dX): what is summed over
    int w_extent;  // rows (Y) or columns (dX) of a weight
    int cols;      // of d
    bool vec;      // d's rows are 16-byte aligned
    bool nt;       // d is written past the caches
    int tiles_n;
    float *parts;  // SPLIT: sums of the last round's parts, BM·BN to each of `slots`
    int slots;     // workgroups that run at once
};
template <typename T>
__device__ inline Operand weight_of(const RowsArgs &a, int e, int k0)
{
    return {reinterpret_cast<const uint16_t *>(a.w) + (int64_t)e * a.w_stride + (T::TB ? k0 * a.ldw : k0), a.ldw, a.w_extent};
}
__device__ inline Operand rows_of(const RowsArgs &a, const Tile2d &t, int k0)
{
    return {reinterpret_cast<const uint16_t *>(a.a) + (int64_t)t.lo * a.lda + k0, a.lda, t.rows};
}
// SPLIT: all whole rounds; the last one too where it is not cut into parts.  16384 rows of 8
// experts of 14336×4096 bf16: Y 1500-1540 us, dX 1320-1400 and 145 for its last round,
// matrix cores busy 0.78 of the waves' time under the power limit.
template <typename E, typename T, bool SPLIT>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(waves_of<T>()) void grouped_rows_kernel(
    RowsArgs a)
{
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const Groups g = find_groups<T::BM>(a.ends, a.E, a.M);
    const int total = g.all * a.tiles_n;
    int here = total;
    if constexpr (SPLIT) {
        const Split s = split_tiles(total, a.slots, (a.inner + BK - 1) / BK);
        here = s.parts > 1 ? s.full : total;
    }
    if ((int)blockIdx.x >= here)
        return;
    const Tile2d t = find_tile<T::BM>(g, a.ends, a.E, a.M, a.tiles_n, xcd_chunks(blockIdx.x, total));
    const int m0 = t.tm * T::BM, n0 = t.tn * T::BN;
    E *d = reinterpret_cast<E *>(a.d) + (int64_t)t.lo * a.ldd;
    if (t.e >= a.E) {
        zero_tile<E, T::BM, T::BN, T::THREADS>(d, a.ldd, m0, n0, t.rows, a.cols);
        return;
    }
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    T::run(smem, rows_of(a, t, 0), weight_of<T>(a, t.e, 0), m0, n0, a.inner, acc);
    store_tile<E, T>(smem, acc, d, a.ldd, m0, n0, t.rows, a.cols, a.vec, a.nt);
}
// The last round's parts, where it is cut into some: their fp32 sums, as the lanes
// hold them.  (A kernel of its own: both ends of the tile product in one spill
// registers at 256×256.)
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(waves_of<T>()) void grouped_parts_kernel(
    RowsArgs a)
{
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const Groups g = find_groups<T::BM>(a.ends, a.E, a.M);
    const int ktiles = (a.inner + BK - 1) / BK, part = (int)blockIdx.x;
    const Split s = split_tiles(g.all * a.tiles_n, a.slots, ktiles);
    if (s.parts < 2 || part >= s.rest * s.parts)
        return;
    const Tile2d t = find_tile<T::BM>(g, a.ends, a.E, a.M, a.tiles_n, s.full + part % s.rest);
    const int m0 = t.tm * T::BM, n0 = t.tn * T::BN;
    if (t.e >= a.E) {
        if (part < s.rest)
            zero_tile<E, T::BM, T::BN, T::THREADS>(reinterpret_cast<E *>(a.d) + (int64_t)t.lo * a.ldd, a.ldd, m0, n0, t.rows,
                                                   a.cols);
        return;
    }
    // K-tiles in memory order; the K-major product's partial one comes first
    const int z = part / s.rest, shift = T::FIRST ? a.inner - ktiles * BK : 0;
    const int k0 = imax(ktiles * z / s.parts * BK + shift, 0), k1 = imin(ktiles * (z + 1) / s.parts * BK + shift, a.inner);
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    T::run(smem, rows_of(a, t, k0), weight_of<T>(a, t.e, k0), m0, n0, k1 - k0, acc);
    store_part<T>(acc, a.parts, part);
}
// The parts' sums: a workgroup takes one of the 16-row strips that a tile's waves hold.
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) void grouped_join_kernel(RowsArgs a)
{
    const Groups g = find_groups<T::BM>(a.ends, a.E, a.M);
    const Split s = split_tiles(g.all * a.tiles_n, a.slots, (a.inner + BK - 1) / BK);
    const int tile = (int)blockIdx.x / T::TM, i = (int)blockIdx.x % T::TM;
    if (s.parts < 2 || tile >= s.rest)
        return;
    const Tile2d t = find_tile<T::BM>(g, a.ends, a.E, a.M, a.tiles_n, s.full + tile);
    if (t.e >= a.E)
        return;  // the rows behind: written as zeros
    join_parts<E, T>(a.parts, tile, s.rest, s.parts, i, reinterpret_cast<E *>(a.d) + (int64_t)t.lo * a.ldd, a.ldd,
                     t.tm * T::BM, t.tn * T::BN, t.rows, a.cols, a.vec);
}

// Y of a few rows an expert where a tile of W for each compute unit is not there:
// 16 rows × 32 columns to a workgroup, whose eight waves take every eighth 128-K piece of
// the sum straight from memory to registers, all loads of two pieces ahead of their
// products, and add up in LDS at the end.  Bound by the latency of its few
// dependent steps (8 of 64 experts of 1024×2048 with a row each, weights not in the
// caches: 12 us, 19 with 64×64 tiles; 16 rows of 8192×8192 35 and 43).
constexpr int FEW_M = 16, FEW_N = 32, FEW_WAVES = 8, FEW_K = 128, FEW_AHEAD = 2;
template <typename E>
__device__ inline typename El<E>::v8 load_chunk(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    union {
        uint32_t __attribute__((ext_vector_type(4))) u;
        typename El<E>::v8 v;
    } x = {};
#if defined(__HIP_DEVICE_COMPILE__)
    x.u = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
#else
    (void)r, (void)off;
#endif
    return x.v;
}
template <typename E>
__global__ __launch_bounds__(64 * FEW_WAVES) void grouped_few_kernel(RowsArgs a)
{
    __shared__ f32x4 sums[FEW_WAVES][FEW_N / 16][64];
    const Groups groups = find_groups<FEW_M>(a.ends, a.E, a.M);
    if ((int)blockIdx.x >= groups.all * a.tiles_n)
        return;
    const Tile2d t = find_tile<FEW_M>(groups, a.ends, a.E, a.M, a.tiles_n, xcd_chunks(blockIdx.x, groups.all * a.tiles_n));
    const int m0 = t.tm * FEW_M, n0 = t.tn * FEW_N;
    E *d = reinterpret_cast<E *>(a.d) + (int64_t)t.lo * a.ldd;
    if (t.e >= a.E) {
        zero_tile<E, FEW_M, FEW_N, 64 * FEW_WAVES>(d, a.ldd, m0, n0, t.rows, a.cols);
        return;
    }
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const auto rsrc = [](const void *p) {
        return __builtin_amdgcn_make_buffer_rsrc((void *)uniform(reinterpret_cast<const char *>(p)), (short)0, DMA_RANGE,
                                                 BUFFER_WORD3);
    };
    const auto rx = rsrc(reinterpret_cast<const E *>(a.a) + (int64_t)(t.lo + m0) * a.lda);
    const auto rw = rsrc(reinterpret_cast<const E *>(a.w) + (int64_t)t.e * a.w_stride + (int64_t)n0 * a.ldw);
    // rows past the last one read it again: they feed only outputs that are not stored
    const uint32_t x_off = (uint32_t)(2 * imin(r, t.rows - 1 - m0) * a.lda);
    uint32_t w_off[FEW_N / 16];
    f32x4 acc[FEW_N / 16];
#pragma unroll
    for (int j = 0; j < FEW_N / 16; ++j) {
        w_off[j] = (uint32_t)(2 * imin(16 * j + r, a.w_extent - 1 - n0) * a.ldw);
        acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int k0 = wave * FEW_K; k0 < a.inner; k0 += FEW_AHEAD * FEW_WAVES * FEW_K) {
        typename El<E>::v8 x[FEW_AHEAD][FEW_K / 32], w[FEW_AHEAD][FEW_K / 32][FEW_N / 16];
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u)
#pragma unroll
            for (int s = 0; s < FEW_K / 32; ++s) {
                const int k = k0 + u * FEW_WAVES * FEW_K + 32 * s + 8 * g;
                const bool in = k < a.inner;  // eight at a time: the sum's length is a multiple of 8
                x[u][s] = load_chunk<E>(rx, in ? x_off + 2 * (uint32_t)k : DMA_OOB);
#pragma unroll
                for (int j = 0; j < FEW_N / 16; ++j)
                    w[u][s][j] = load_chunk<E>(rw, in ? w_off[j] + 2 * (uint32_t)k : DMA_OOB);
            }
        __builtin_amdgcn_sched_barrier(0);  // all of them in flight
#pragma unroll
        for (int u = 0; u < FEW_AHEAD; ++u)
#pragma unroll
            for (int s = 0; s < FEW_K / 32; ++s)
#pragma unroll
                for (int j = 0; j < FEW_N / 16; ++j)
                    acc[j] = El<E>::mfma(w[u][s][j], x[u][s], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < FEW_N / 16; ++j)
        sums[wave][j][lane] = acc[j];
    __syncthreads();
    // one element to a thread: row m, column n of the tile
    static_assert(FEW_M * FEW_N == 64 * FEW_WAVES, "a thread for each element");
    const int m = threadIdx.x / FEW_N, n = threadIdx.x % FEW_N, from = m + 16 * (n % 16 / 4);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < FEW_WAVES; ++v)
        sum += sums[v][n / 16][from][n % 4];
    if (m0 + m < t.rows && n0 + n < a.cols)
        d[(int64_t)(m0 + m) * a.ldd + n0 + n] = (E)sum;
}

// dW: tiles of one expert's weight, summed over its rows; PARTS: over a part of them,
// where there are too few tiles to fill the chip.
struct WeightArgs {
    const void *dy, *x;
    const int64_t *ends;
    void *dw;
    int64_t lddy, ldx, lddw, dw_stride;
    int M, E, N, K;
    bool vec, nt;
    int tiles_m, tiles_n;
    float *sums;  // PARTS
    int parts;
};
constexpr int DW_AHEAD = 3;  // K-tiles that are asked for ahead, at most
template <typename E, typename T, bool PARTS>
__global__ __launch_bounds__(T::THREADS) PT_WAVES_PER_SIMD(waves_of<T>()) void grouped_weight_kernel(
    WeightArgs a)
{
    static_assert(T::S <= DW_AHEAD, "the limit on rows counts them");
    __shared__ __attribute__((aligned(1024))) E smem[T::LDS_ELEMS];
    const int per = a.tiles_m * a.tiles_n, total = a.E * per;
    const int z = PARTS ? (int)blockIdx.x / total : 0;
    const int logical = xcd_chunks((int)blockIdx.x - z * total, total), e = logical / per;
    int tm, tn, lo, rows;
    grouped_tile<4>(logical - e * per, a.tiles_m, a.tiles_n, tm, tn);
    find_rows(a.ends, a.M, e, lo, rows);
    const int m0 = tm * T::BM, n0 = tn * T::BN;
    E *d = reinterpret_cast<E *>(a.dw) + (int64_t)e * a.dw_stride;
    if (rows == 0) {
        if (z == 0)
            zero_tile<E, T::BM, T::BN, T::THREADS>(d, a.lddw, m0, n0, a.N, a.K);
        return;
    }
    if constexpr (PARTS) {
        const int ktiles = (rows + BK - 1) / BK, k0 = (int)((int64_t)ktiles * z / a.parts) * BK;
        rows = imin((int)((int64_t)ktiles * (z + 1) / a.parts) * BK, rows) - k0;
        lo += k0;
    }
    f32x4 acc[T::TM][T::TN];
    T::clear(acc);
    const Operand dy = {reinterpret_cast<const E *>(a.dy) + (int64_t)lo * a.lddy, a.lddy, a.N};
    const Operand x = {reinterpret_cast<const E *>(a.x) + (int64_t)lo * a.ldx, a.ldx, a.K};
    T::run(smem, dy, x, m0, n0, rows, acc);
    if constexpr (PARTS)
        store_part<T>(acc, a.sums, (int64_t)z * total + logical);
    else
        store_tile<E, T>(smem, acc, d, a.lddw, m0, n0, a.N, a.K, a.vec, a.nt);
}
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) void grouped_weight_join_kernel(WeightArgs a)
{
    const int per = a.tiles_m * a.tiles_n, logical = (int)blockIdx.x / T::TM, e = logical / per;
    int tm, tn, lo, rows;
    grouped_tile<4>(logical - e * per, a.tiles_m, a.tiles_n, tm, tn);
    find_rows(a.ends, a.M, e, lo, rows);
    if (rows == 0)
        return;  // written as zeros
    join_parts<E, T>(a.sums, logical, (int64_t)a.E * per, a.parts, (int)blockIdx.x % T::TM,
                     reinterpret_cast<E *>(a.dw) + (int64_t)e * a.dw_stride, a.lddw, tm * T::BM, tn * T::BN, a.N, a.K, a.vec);
}

// ------------------------------------------------------------------- packing
// Rows of `cols` elements to 16-byte aligned rows of cols8, zeros behind (rows
// that the tile product cannot load as they lie).  `ends`: the rows are those of
// `per`-row weights, and weights of experts without rows are left out.
struct PackArgs {
    const uint16_t *src;
    uint16_t *dst;
    int64_t ld, stride, rows, per, cols, cols8;
    const int64_t *ends;
    int M, run;  // run: rows of a workgroup, of one weight
};
__global__ __launch_bounds__(256) void grouped_pack_kernel(PackArgs a)
{
    const int chunks = (int)(a.cols8 / 8);
    const int64_t runs = cdiv(a.per, a.run);
    for (int64_t b = blockIdx.x; b < (a.rows / a.per) * runs; b += gridDim.x) {
        const int64_t e = b / runs, r0 = (b - e * runs) * a.run;
        const int n = (int)(a.per - r0 < a.run ? a.per - r0 : a.run);
        if (a.ends) {
            int lo, rows;
            find_rows(a.ends, a.M, (int)e, lo, rows);
            if (rows == 0)
                continue;
        }
        const uint16_t *src = a.src + e * a.stride + r0 * a.ld;
        uint16_t *dst = a.dst + (e * a.per + r0) * a.cols8;
        // (fewer than 2^18 chunks a row, and more than one row only of up to 1024)
#pragma unroll 2
        for (int i = threadIdx.x; i < n * chunks; i += 256) {
            const int r = i / chunks, c = (i - r * chunks) * 8;
            *reinterpret_cast<uint4 *>(dst + r * a.cols8 + c) = load8(src + r * a.ld, c, a.cols, false);
        }
    }
}
__global__ __launch_bounds__(256) void grouped_zero_kernel(uint16_t *d, int64_t ld, int64_t stride, int64_t batch,
                                                           int64_t rows, int64_t cols)
{
    for (int64_t b = blockIdx.x; b < batch * rows; b += gridDim.x) {
        uint16_t *row = d + b / rows * stride + b % rows * ld;
        for (int64_t c = threadIdx.x; c < cols; c += 256)
            row[c] = 0;
    }
}

// ------------------------------------------------------------------- plans
enum Class { C256, C192, C128, C64, C64X128, ONE, CLASSES, FEW = CLASSES };
const char *const CLASS_NAME[] = {"256x256", "192x192", "128x128", "64x64", "64x128", "128x128x4", "16x32"};
// Tiles, workgroups per compute unit, and microseconds: per K-tile with all of them
// running and with one a unit, and per tile besides.  Here and below the numbers were
// fitted to the times of every class for 760 problems on one MI355X (1 to 16384 rows, 1
// to 128 experts, N and K from 64 to 14336, weights not in the caches): what is
// chosen takes 2.5% (Y), 1.5% (dX) and 1.5% (dW) more than the best of them in the geometric
// mean, at most 1.5 times as much.  A kernel that changes leaves its numbers stale: they choose
// a class, and no result depends on them beyond the order of its sums.
struct RowsModel {
    TileClass c[CLASSES];
    double more, tail;    // tile rows: how many more than of even shares, and of a share's last tile
    double rate, reread;  // of the weights: bytes a microsecond; what an expert's second and third tile row add
    double last, cut;     // what a last round takes beside the tiles in it, whole and in parts
    double split, base;   // microseconds: of the two launches more, of any
};
constexpr RowsModel Y_MODEL = {{{256, 256, 1, 1.08, 1.08, 16.4},
                                {192, 192, 1, 0.89, 0.84, 8.5},
                                {128, 128, 2, 1.50, 0.71, 5.5},
                                {64, 64, 2, 0.37, 0.28, 3.8},
                                {64, 128, 2, 0.77, 0.50, 4.8},
                                {128, 128, 4, 2.30, 1.05, 4.5}},
                               1.11, 0.35, 4.4e6, 0.50, 0.60, 0.38, 12.5, 3.1};
constexpr RowsModel DX_MODEL = {{{256, 256, 1, 1.52, 1.52, 15.1},
                                 {},
                                 {128, 128, 2, 0.92, 0.92, 8.4},
                                 {64, 64, 2, 0.45, 0.36, 4.9},
                                 {64, 128, 2, 0.81, 0.40, 5.0},
                                 {128, 128, 4, 2.06, 2.06, 5.7}},
                                1.53, 0.26, 5.8e6, 1.03, 0.36, 0.24, 8.6, 4.0};
// The 64×128 tiles of Y read W past the caches: its rate in whole 128-byte lines, and
// where rows end within a line, which is then read for both (76 experts of 1600×1464 and
// 2881 rows: 130 us, 108 with 64×64 tiles; 64 of 1024×2048 and 1100 rows: 47 and 67).
constexpr double STREAM_RATE = 7.3e6, STREAM_RATE_CUT = 3.6e6;
// of dW, and the rate in TB/s at which it writes
constexpr TileClass DW_CLASS[] = {{256, 256, 1, 1.26, 1.26, 16.4},
                                  {192, 192, 1, 1.38, 0.94, 9.0},
                                  {128, 128, 2, 0.95, 0.53, 5.9},
                                  {64, 64, 2, 0.62, 0.30, 4.0},
                                  {},
                                  {128, 128, 4, 1.76, 1.38, 5.0}};
constexpr double DW_RATE[] = {3.4, 2.6, 3.1, 1.5, 0.0, 5.9};
template <typename E, bool TA, bool TB, typename F>
bool with_tile(Class c, F f)
{
    constexpr bool MASK = !TA && TB, STREAM = !TA && !TB;
    switch (c) {
    case C256:
        return f(Tile<E, 256, 256, 2, 2, 2, TA, TB, false, MASK>{});
    case C192:
        if constexpr (TA == TB)
            return f(Tile<E, 192, 192, 2, 2, 2, TA, TB>{});
        [[fallthrough]];
    case C128:
        return f(Tile<E, 128, 128, 2, 2, 2, TA, TB, false, MASK>{});
    case ONE:
        return f(OneStage<E, TA, TB>{});
    case C64X128:
        if constexpr (!TA)
            return f(Tile<E, 64, 128, 1, 4, 3, TA, TB, STREAM, MASK>{});
        [[fallthrough]];
    default:
        return f(Tile<E, 64, 64, 2, 2, 3, TA, TB, false, MASK>{});
    }
}

struct Call {
    int product;
    const void *A, *B;
    int64_t M, E, N, K, lda, ldb, w_stride;
};
struct Plan {
    Class c;
    int64_t bm, bn, grid;
    bool pack_a, pack_b;
    int64_t a_cols, b_cols;  // of the operands' rows
    int64_t a_bytes, b_bytes;
    int slots;               // Y, dX with the last round in parts: the workgroups that run at once; 0 otherwise
    int parts;               // dW: into how many its sums are cut
    int64_t parts_bytes;
};
bool rows_ok(const void *p, int64_t ld, int64_t cols)
{
    return (uintptr_t)p % 16 == 0 && ld % 8 == 0 && cols % 8 == 0 && ld <= MAX_DMA_LD;
}
// Time in microseconds of `n` tiles with `ktiles` K-tiles each; how many there are is
// known to some 10% only, so that rounds are not counted whole.
double rounds_time(const TileClass &c, double n, double ktiles, double last)
{
    const double slots = (double)NUM_CU * c.per_cu;
    if (n > slots)
        return (n / slots + last) * (ktiles * c.ktile + c.fixed);
    return ktiles * (c.alone + (c.ktile - c.alone) * std::max(0.0, (n - NUM_CU) / std::max(1.0, slots - NUM_CU))) + c.fixed;
}
struct Estimate {
    double time;
    bool split;  // whether the last round, or the only one, is cut into parts
};
// A product over M rows of E experts.  Weights are read for each tile row, but
// mostly from a cache where they are shared; 64×128 tiles of Y stream them past the
// caches, which is faster for one tile row an expert and much slower for several.
// How many rows an expert has is known for one expert only.
// `stream`: that rate, or 0.
Estimate rows_time(const RowsModel &m, int cls, double stream, int64_t M, int64_t E, int64_t cols, int64_t inner)
{
    const TileClass &c = m.c[cls];
    const double hit = (double)std::min(M, E), each = (double)M / hit;
    const double tile_rows = E == 1 ? (double)cdiv(M, c.bm) : std::max(1.0, each / c.bm + m.tail);
    const double n = (E == 1 ? 1.0 : m.more) * hit * tile_rows * (double)cdiv(cols, c.bn);
    const double slots = (double)NUM_CU * c.per_cu, k = (double)cdiv(inner, BK);
    const double weights = 2.0 * hit * (double)cols * (double)inner, others = 2.0 * (double)M * (double)(cols + inner);
    const double again = stream > 0.0 ? 1.4 * (tile_rows - 1.0) * (tile_rows - 1.0) : m.reread * (std::min(tile_rows, 3.0) - 1.0);
    const double memory = weights * (1.0 + again) / (stream > 0.0 ? stream : m.rate) + others / 5e6 + m.base;
    const double whole = rounds_time(c, n, k, m.last);
    double cut = 1e30;
    if (n > slots) {
        if (n <= 12.0 * slots)
            cut = rounds_time(c, n, k, m.cut) + m.split;
    } else {
        const double parts = std::floor(std::min(std::min(slots / n, k / MIN_PART), (double)MAX_PARTS));
        if (parts >= 2.0)
            cut = k * c.ktile / parts + c.fixed + m.split;
    }
    const double a = std::max(whole, memory), b = std::max(cut, memory + 4.0);
    return {std::min(a, b), b < a};
}
double few_time(int64_t M, int64_t E, int64_t cols, int64_t inner)
{
    const double hit = (double)std::min(M, E), each = (double)M / hit;
    const double tile_rows = E == 1 ? (double)cdiv(M, FEW_M) : std::max(1.0, each / FEW_M + Y_MODEL.tail);
    const double n = hit * tile_rows * (double)cdiv(cols, FEW_N);
    return std::max(1.1 + 3.5 * (double)cdiv(inner, 2048) * std::max(1.0, n / 512.0),
                    2.0 * hit * (double)cols * (double)inner * tile_rows / 4.5e6 + Y_MODEL.base);
}
// dW, and into how many parts its sums are cut: 1, or as many as fill the chip.
struct WeightEstimate {
    double time;
    int parts;
};
WeightEstimate weight_time(int cls, const Call &q)
{
    const TileClass &c = DW_CLASS[cls];
    const int64_t n = q.E * cdiv(q.N, c.bm) * cdiv(q.K, c.bn), ktiles = cdiv(cdiv(q.M, q.E), BK);
    const double memory = 2.0 * (double)q.E * (double)q.N * (double)q.K / (DW_RATE[cls] * 1e6) + 4.0;
    const double whole = std::max(rounds_time(c, (double)n, (double)ktiles, 0.55), memory);
    const int64_t parts = std::min(std::min(NUM_CU * (int64_t)c.per_cu / n, ktiles / MIN_PART), (int64_t)MAX_PARTS);
    if (parts < 2)
        return {whole, 1};
    // the parts are written and read in fp32
    const double cut = std::max(rounds_time(c, (double)(n * parts), (double)cdiv(ktiles, parts), 0.55), memory) + 1.7 +
                       (double)(n * parts * c.bm * c.bn) * 8.0 / 4e6;
    return cut < whole ? WeightEstimate{cut, (int)parts} : WeightEstimate{whole, 1};
}
Plan make_plan(const Call &q)
{
    Plan p = {};
    const bool dw = q.product == TG_GROUPED_DW, dx = q.product == TG_GROUPED_DX;
    p.a_cols = q.product == TG_GROUPED_Y ? q.K : q.N;
    p.b_cols = q.K;
    p.pack_a = !rows_ok(q.A, q.M > 1 ? q.lda : round_up(q.lda, 8), p.a_cols);
    p.pack_b = !rows_ok(q.B, (dw ? q.M : q.N) > 1 ? q.ldb : round_up(q.ldb, 8), p.b_cols) ||
               (!dw && q.E > 1 && q.w_stride % 8 != 0);
    p.a_bytes = p.pack_a ? round_up(2 * q.M * round_up(p.a_cols, 8), 256) : 0;
    p.b_bytes = p.pack_b ? round_up(2 * (dw ? q.M : q.E * q.N) * round_up(p.b_cols, 8), 256) : 0;
    const int64_t out = dx ? q.K : q.N, inner = dx ? q.N : q.K;
    if (dw) {
        int c = 0;
        for (int i = 1; i < CLASSES; ++i)
            if (i != C64X128 && weight_time(i, q).time < weight_time(c, q).time)
                c = i;
        p.c = (Class)c, p.bm = DW_CLASS[c].bm, p.bn = DW_CLASS[c].bn;
        p.parts = weight_time(c, q).parts;
        p.grid = q.E * cdiv(q.N, p.bm) * cdiv(q.K, p.bn) * p.parts;
        p.parts_bytes = p.parts > 1 ? 4 * p.grid * p.bm * p.bn : 0;
        return p;
    }
    const int64_t row = p.pack_b ? round_up(q.K, 8) : q.ldb;
    const double stream = row % 64 == 0 ? STREAM_RATE : STREAM_RATE_CUT;
    const auto time = [&](int i) {
        return rows_time(dx ? DX_MODEL : Y_MODEL, i, !dx && i == C64X128 ? stream : 0.0, q.M, q.E, out, inner);
    };
    int c = 0;
    for (int i = 1; i < CLASSES; ++i)
        if (!(dx && i == C192) && time(i).time < time(c).time)
            c = i;
    const bool few = !dx && few_time(q.M, q.E, out, inner) < time(c).time, split = !few && time(c).split;
    p.c = few ? FEW : (Class)c;
    p.bm = few ? FEW_M : Y_MODEL.c[c].bm, p.bn = few ? FEW_N : Y_MODEL.c[c].bn;
    // each group adds at most bm - 1 rows to whole tiles
    p.grid = (q.M + std::min(q.E + 1, q.M) * (p.bm - 1)) / p.bm * cdiv(out, p.bn);
    if (split) {
        p.slots = NUM_CU * Y_MODEL.c[c].per_cu;
        p.parts_bytes = (int64_t)4 * p.slots * p.bm * p.bn;
    }
    return p;
}

// Results from this size on are written past the caches, which they would fill for
// nothing (dW of 8 experts of 14336×4096 from 128 rows 308 -> 237 us, of 64 of 1024×2048 from
// 16384 rows 163 -> 115; Y of 16384×14336 1522 -> 1505).
constexpr int64_t NT_BYTES = (int64_t)64 << 20;
constexpr int64_t LIM = (int64_t)1 << 31, LIM_STRIDE = (int64_t)1 << 42;
// Rows of dW's sums: their K-tiles, and the DW_AHEAD that are asked for past the last one,
// begin at rows of 31 bits.  (Y and dX sum over N and K, and have fewer rows: tiles of up to 256
// rows, fewer than MAX_GRID.)
constexpr int64_t LIM_ROWS = LIM - 256;
static_assert((cdiv(LIM_ROWS - 1, BK) + DW_AHEAD) * BK < LIM, "rows of 31 bits");
static_assert(MAX_GRID * 256 <= LIM, "rows of 31 bits");
// Whether anything is multiplied: otherwise the result is zeros, or nothing.
bool multiplies(const Call &q) { return q.M > 0 && q.E > 0 && q.N > 0 && q.K > 0; }
int validate(const Call &q)
{
    if (q.product < TG_GROUPED_Y || q.product > TG_GROUPED_DW || q.M < 0 || q.E < 0 || q.N < 0 || q.K < 0)
        return TG_ERR_INVALID_ARG;
    const bool dw = q.product == TG_GROUPED_DW;
    if (q.lda < (q.product == TG_GROUPED_Y ? q.K : q.N) || q.ldb < q.K || (!dw && q.E > 1 && q.w_stride < 0))
        return TG_ERR_INVALID_ARG;
    if (q.M >= (dw ? LIM_ROWS : LIM) || q.E >= 1 << 16 || q.N >= MAX_DMA_LD || q.K >= MAX_DMA_LD || q.lda >= LIM ||
        q.ldb >= LIM || (!dw && q.E > 1 && q.w_stride >= LIM_STRIDE))
        return TG_ERR_TOO_LARGE;
    if (!multiplies(q))
        return TG_OK;
    if (!q.A || !q.B || (uintptr_t)q.A % 2 || (uintptr_t)q.B % 2)
        return TG_ERR_INVALID_ARG;
    return make_plan(q).grid >= MAX_GRID ? TG_ERR_TOO_LARGE : TG_OK;
}
int64_t copy_grid(int64_t n) { return std::max((int64_t)1, std::min(n, (int64_t)16 * NUM_CU)); }

bool pack(const void *src, void *dst, int64_t ld, int64_t stride, int64_t batch, int64_t per, int64_t cols,
          const int64_t *ends, int64_t M, void *stream)
{
    PackArgs a = {reinterpret_cast<const uint16_t *>(src), reinterpret_cast<uint16_t *>(dst), ld, stride, batch * per,
                  per, cols, round_up(cols, 8), ends, (int)M, 0};
    // some 16 KB a workgroup
    a.run = (int)std::min(per, std::max((int64_t)1, 1024 / (a.cols8 / 8)));
    return launch(grouped_pack_kernel, copy_grid(batch * cdiv(per, a.run)), 256, stream, a);
}

// `ldd`, `d_stride`: of the result
template <typename E>
int product(const Call &q, const int64_t *ends, void *D, int64_t ldd, int64_t d_stride, void *ws, int64_t ws_bytes,
            void *stream)
{
    const int st = validate(q);
    const bool dw = q.product == TG_GROUPED_DW, y = q.product == TG_GROUPED_Y;
    const int64_t batch = dw ? q.E : 1, rows = dw ? q.N : q.M, cols = y ? q.N : q.K;
    if (st == TG_ERR_INVALID_ARG || ldd < cols || (dw && q.E > 1 && q.N > 0 && d_stride < (q.N - 1) * ldd + q.K))
        return TG_ERR_INVALID_ARG;
    if (st != TG_OK || ldd >= LIM || (dw && q.E > 1 && d_stride >= LIM_STRIDE))
        return TG_ERR_TOO_LARGE;
    if (batch == 0 || rows == 0 || cols == 0)
        return TG_OK;
    if (!D || (uintptr_t)D % 2)
        return TG_ERR_INVALID_ARG;
    if (!multiplies(q)) {
        if (gfx950_status() != 1)
            return TG_ERR_DEVICE;
        return launch(grouped_zero_kernel, copy_grid(batch * rows), 256, stream, (uint16_t *)D, ldd, d_stride, batch, rows,
                      cols)
                   ? TG_OK
                   : TG_ERR_LAUNCH;
    }
    const Plan p = make_plan(q);
    const int64_t need = p.a_bytes + p.b_bytes + p.parts_bytes;
    if (!ends || (uintptr_t)ends % 8 || (need > 0 && (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < need)))
        return TG_ERR_INVALID_ARG;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    const void *A = q.A, *B = q.B;
    int64_t lda = q.M > 1 ? q.lda : round_up(q.lda, 8), ldb = (dw ? q.M : q.N) > 1 ? q.ldb : round_up(q.ldb, 8);
    int64_t w_stride = q.E > 1 ? q.w_stride : 0;
    bool ok = true;
    if (p.pack_a) {
        ok = pack(A, ws, q.lda, 0, 1, q.M, p.a_cols, nullptr, q.M, stream);
        A = ws, lda = round_up(p.a_cols, 8);
    }
    if (p.pack_b) {
        void *to = reinterpret_cast<char *>(ws) + p.a_bytes;
        ok = ok && pack(B, to, q.ldb, w_stride, dw ? 1 : q.E, dw ? q.M : q.N, p.b_cols, dw ? nullptr : ends, q.M, stream);
        B = to, ldb = round_up(p.b_cols, 8), w_stride = q.N * ldb;
    }
    const bool vec = ldd % 8 == 0 && (uintptr_t)D % 16 == 0 && (!dw || q.E == 1 || d_stride % 8 == 0);
    const bool nt = 2 * batch * rows * cols >= NT_BYTES && ldd % 64 == 0 && (uintptr_t)D % 128 == 0;
    float *const sums = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + p.a_bytes + p.b_bytes);
    if (dw) {
        WeightArgs a = {};
        a.dy = A, a.x = B, a.ends = ends, a.dw = D;
        a.lddy = lda, a.ldx = ldb, a.lddw = ldd, a.dw_stride = q.E > 1 ? d_stride : 0;
        a.M = (int)q.M, a.E = (int)q.E, a.N = (int)q.N, a.K = (int)q.K;
        a.vec = vec, a.nt = nt;
        a.tiles_m = (int)cdiv(q.N, p.bm), a.tiles_n = (int)cdiv(q.K, p.bn);
        a.sums = sums, a.parts = p.parts;
        ok = ok && with_tile<E, true, true>(p.c, [&](auto t) {
            using T = decltype(t);
            if (p.parts == 1)
                return launch(grouped_weight_kernel<E, T, false>, p.grid, T::THREADS, stream, a);
            return launch(grouped_weight_kernel<E, T, true>, p.grid, T::THREADS, stream, a) &&
                   launch(grouped_weight_join_kernel<E, T>, p.grid / p.parts * T::TM, T::THREADS, stream, a);
        });
    } else {
        RowsArgs a = {};
        a.a = A, a.w = B, a.ends = ends, a.d = D;
        a.lda = lda, a.ldw = ldb, a.w_stride = w_stride, a.ldd = ldd;
        a.M = (int)q.M, a.E = (int)q.E;
        // over a packed row's zeros, but not over W's rows behind N
        a.inner = (int)(y ? (p.pack_a || p.pack_b ? round_up(q.K, 8) : q.K) : q.N);
        a.w_extent = (int)(y ? q.N : q.K), a.cols = (int)cols;
        a.vec = vec, a.nt = nt;
        a.tiles_n = (int)cdiv(cols, p.bn);
        a.parts = sums, a.slots = p.slots;
        const auto run = [&](auto t) {
            using T = decltype(t);
            if (p.slots == 0)
                return launch(grouped_rows_kernel<E, T, false>, p.grid, T::THREADS, stream, a);
            return launch(grouped_rows_kernel<E, T, true>, p.grid, T::THREADS, stream, a) &&
                   launch(grouped_parts_kernel<E, T>, p.slots, T::THREADS, stream, a) &&
                   launch(grouped_join_kernel<E, T>, (int64_t)p.slots / 2 * T::TM, T::THREADS, stream, a);
        };
        if (p.c == FEW)
            ok = ok && launch(grouped_few_kernel<E>, p.grid, 64 * FEW_WAVES, stream, a);
        else
            ok = ok && (y ? with_tile<E, false, false>(p.c, run) : with_tile<E, false, true>(p.c, run));
    }
    return ok ? TG_OK : TG_ERR_LAUNCH;
}
}  // namespace

extern "C" int64_t tg_grouped_workspace_bytes(int product, const void *A, const void *B, int64_t M, int64_t E,
                                              int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t w_stride)
{
    const Call q = {product, A, B, M, E, N, K, lda, ldb, w_stride};
    if (validate(q) != TG_OK)
        return -1;
    if (!multiplies(q))
        return 0;
    const Plan p = make_plan(q);
    return p.a_bytes + p.b_bytes + p.parts_bytes;
}

#define TG_GROUPED_ENTRIES(suffix, E)                                                                                 \
    extern "C" int tg_grouped_##suffix(const void *X, const void *W, const int64_t *ends, void *Y, int64_t M,         \
                                       int64_t experts, int64_t N, int64_t K, int64_t ldx, int64_t ldw,               \
                                       int64_t w_stride, int64_t ldy, void *workspace, int64_t workspace_bytes,       \
                                       void *stream)                                                                  \
    {                                                                                                                 \
        return product<E>({TG_GROUPED_Y, X, W, M, experts, N, K, ldx, ldw, w_stride}, ends, Y, ldy, 0, workspace,     \
                          workspace_bytes, stream);                                                                   \
    }                                                                                                                 \
    extern "C" int tg_grouped_dx_##suffix(const void *dY, const void *W, const int64_t *ends, void *dX, int64_t M,    \
                                          int64_t experts, int64_t N, int64_t K, int64_t lddy, int64_t ldw,           \
                                          int64_t w_stride, int64_t lddx, void *workspace, int64_t workspace_bytes,   \
                                          void *stream)                                                               \
    {                                                                                                                 \
        return product<E>({TG_GROUPED_DX, dY, W, M, experts, N, K, lddy, ldw, w_stride}, ends, dX, lddx, 0,           \
                          workspace, workspace_bytes, stream);                                                        \
    }                                                                                                                 \
    extern "C" int tg_grouped_dw_##suffix(const void *dY, const void *X, const int64_t *ends, void *dW, int64_t M,    \
                                          int64_t experts, int64_t N, int64_t K, int64_t lddy, int64_t ldx,           \
                                          int64_t lddw, int64_t dw_stride, void *workspace, int64_t workspace_bytes,  \
                                          void *stream)                                                               \
    {                                                                                                                 \
        return product<E>({TG_GROUPED_DW, dY, X, M, experts, N, K, lddy, ldx, 0}, ends, dW, lddw, dw_stride,          \
                          workspace, workspace_bytes, stream);                                                        \
    }
TG_GROUPED_ENTRIES(f16, _Float16)
TG_GROUPED_ENTRIES(bf16, __bf16)

extern "C" int tg_grouped_plan(int product, const void *A, const void *B, int64_t M, int64_t E, int64_t N, int64_t K,
                               int64_t lda, int64_t ldb, int64_t w_stride, char *name, int64_t name_len)
{
    if (name && name_len > 0)
        name[0] = 0;
    const Call q = {product, A, B, M, E, N, K, lda, ldb, w_stride};
    const int st = validate(q);
    if (st != TG_OK || !name || name_len <= 0)
        return st;
    if (!multiplies(q)) {
        const bool none = product == TG_GROUPED_DW ? E == 0 || N == 0 || K == 0 : M == 0 || (product == TG_GROUPED_Y ? N : K) == 0;
        snprintf(name, (size_t)name_len, "%s", none ? "" : "zero");
        return st;
    }
    const Plan p = make_plan(q);
    static const char *const WHAT[] = {"y", "dx", "dw"};
    snprintf(name, (size_t)name_len, "%s%s%s_%s%s", p.pack_a ? "pack_a " : "", p.pack_b ? "pack_b " : "", WHAT[product],
             CLASS_NAME[p.c], p.slots || p.parts > 1 ? "_split" : "");
    return st;
}
