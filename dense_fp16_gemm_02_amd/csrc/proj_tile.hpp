// proj_tile.hpp — the tile product behind the projection operators
// (tg_xent.hip, tg_ortho.hip, tg_grouped.hip): a BM×BN block of op(A)·op(B) accumulated in
// fp32 registers, with each operand either K-major (a row of K consecutive
// elements per output row, as tg_gemm takes them) or transposed (a row of
// consecutive output rows per K, as the gradient products need them), so that
// no operand is ever copied into another order.
//
//   product                 A            B
//   H·Wᵀ      (logits)      K-major      K-major
//   G·W       (dH, B·X)     K-major      transposed
//   Gᵀ·H      (dW, XᵀX)     transposed   transposed
//
// Operands move global → LDS with 16-byte direct-to-LDS buffer loads and are
// multiplied by v_mfma_f32_16x16x32.  The MFMA's first input is fed from B and
// its second from A, so that lane l of an accumulator holds row l % 16 and the
// four consecutive columns 4·(l/16) .. +3 of its 16×16 block.
//
// LDS images of one 64-K stage, both written by DMAs that fill 64 consecutive
// 16-byte slots per wave instruction, so every reordering is applied on the
// source side:
//   K-major    BX rows of 64 K (128 bytes); chunk c of row r at slot
//              c ^ ((r / 2) % 8), so that the sixteen rows a 128-bit fragment
//              read serves at once fall on sixteen different bank groups;
//   transposed 64 rows (K) of BX columns; a fragment (16 columns × 8 K per
//              lane) is read with two ds_read_b64_tr_b16, which transpose 4 K ×
//              16 columns inside each group of 16 lanes: lane s of a group
//              supplies row s / 4 and columns 4·(s % 4) .. +3, lane i receives
//              column i of the four rows.  The 32-byte column slots of row k
//              are XORed with k's bits 0, 1 and 3 (64 and 192 columns, whose
//              odd rows start half a bank line further: bits 1 and 3), so that
//              the eight rows a half wave reads fall on eight different 32-byte
//              bank groups (without it four rows share one).
//
// Rings: S + 1 stages of A and S of B, refilled S K-tiles ahead.  K-tile t is
// two 32-K steps: step 0 multiplies while step 1's fragments are read and
// A(t+S) is loaded into the stage drained at the barrier of t-1; then the wait
// for K-tile t+1 and one barrier; step 1 multiplies while the fragments of K-
// tile t+1 are read and B(t+S) is loaded into the stage just drained.
//
// K tails: the K-major × K-major product takes the partial K-tile first (its
// columns below 0 read as zero); a transposed operand takes it last (rows past
// K are past the end of the buffer range and read as zero), and a K-major
// operand beside it has to hold zeros up to a multiple of 64 or is masked (MASK).
// Rows (columns) past an operand's extent are clamped to its last one: they feed
// only outputs that are never stored.
#ifndef TG_PROJ_TILE_HPP
#define TG_PROJ_TILE_HPP

#include <hip/hip_runtime.h>

#include <atomic>
#include <tuple>
#include <type_traits>
#include <stdint.h>
#include <string.h>

#include "tile_layout.hpp"

namespace {
namespace pt {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void *lds_ptr;

template <typename E>
struct El;
template <>
struct El<_Float16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    typedef _Float16 v4 __attribute__((ext_vector_type(4)));
    __device__ static f32x4 mfma(v8 a, v8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct El<__bf16> {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    typedef __bf16 v4 __attribute__((ext_vector_type(4)));
    __device__ static f32x4 mfma(v8 a, v8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

__host__ __device__ constexpr int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ constexpr int imax(int a, int b) { return a > b ? a : b; }
__host__ __device__ constexpr int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ constexpr int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

constexpr int BK = 64;
constexpr int NUM_XCD = 8;
constexpr int NUM_CU = 256;
constexpr int DMA_RANGE = 0x7fffffff;
constexpr uint32_t DMA_OOB = 0x80000000u;
constexpr int BUFFER_WORD3 = 0x00020000;  // raw buffer, 32-bit data format
// leading dimensions whose 64-row (256-row) in-tile byte offsets fit the DMAs'
// 31-bit offsets; operands with larger ones are repacked first
constexpr int64_t MAX_DMA_LD = (int64_t)1 << 21;
static_assert(256 * MAX_DMA_LD * 2 + 512 <= (int64_t)DMA_RANGE, "in-tile offsets");

#if defined(__HIP_DEVICE_COMPILE__)
#define PT_WAVES_PER_SIMD(n) __attribute__((amdgpu_waves_per_eu(n, n)))
#else
#define PT_WAVES_PER_SIMD(n)
#endif

// 16 bytes per lane, buffer offset voff → LDS lds + 16·lane (lds wave-uniform).
// CPOL: the instruction's cache policy, 0 cached, 3 (sc0 | nt) for an operand
// that is read once and should not displace the other.
template <int CPOL = 0>
__device__ inline void dma16(__amdgpu_buffer_rsrc_t r, void *lds, uint32_t voff)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, voff, 0, 0, CPOL);
#else
    (void)r, (void)lds, (void)voff;
#endif
}
// 8 bytes per lane, transposed inside groups of 16 lanes.  `restrict` is there
// for the compiler's wait counts: it attaches alias information to the access,
// without which every such read waits for all LDS DMAs in flight (measured: the
// products with transposed operands ran at a third of their rate).  The
// waits that the data need are the explicit ones of the K loop.
#if defined(__HIP_DEVICE_COMPILE__)
typedef __attribute__((address_space(3))) s16x4 tr_word;
__device__ inline __attribute__((always_inline)) s16x4 lds_read_tr_(tr_word *__restrict__ p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}
#endif
__device__ inline __attribute__((always_inline)) s16x4 lds_read_tr(const void *p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    return lds_read_tr_((tr_word *)(lds_ptr)p);
#else
    (void)p;
    return s16x4{0, 0, 0, 0};
#endif
}
template <int N>
__device__ inline void wait_vmem()
{
    static_assert(N >= 0 && N <= 63, "vmcnt holds 6 bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// workgroup barrier that waits for this wave's LDS accesses, not for its DMAs
__device__ inline void barrier_lds()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ inline int lane_id()
{
    return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
}

__device__ inline void pin(f32x4 &v)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+a"(v));
#else
    (void)v;
#endif
}
// A value that is the same in every lane, in scalar registers: buffer
// descriptors built from values that the compiler takes for per-lane ones cost a
// loop over the lanes at every DMA.
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline const char *uniform(const char *p)
{
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
    return reinterpret_cast<const char *>((uint64_t)hi << 32 | lo);
}

// Workgroup id → tile.  Workgroup w runs on XCD w mod 8; each XCD takes a
// contiguous range of logical ids, which walk groups of GM tile rows column
// by column, so that the tiles resident on one XCD share operand bands in its
// L2.  Returns false for ids past the last tile.
__host__ __device__ constexpr int xcd_contiguous(int bid, int total)
{
    const int xcd = bid % NUM_XCD, local = bid / NUM_XCD;
    const int per = total / NUM_XCD, rem = total % NUM_XCD;
    return xcd * per + imin(xcd, rem) + local;
}
template <int GM>
__host__ __device__ constexpr void grouped_tile(int logical, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int group_size = GM * tiles_n;
    const int group = logical / group_size;
    const int first = group * GM;
    const int rows = imin(tiles_m - first, GM);
    const int in = logical - group * group_size;
    tm = first + in % rows;
    tn = in / rows;
}
constexpr bool order_is_bijective(int tiles_m, int tiles_n)
{
    bool seen[2048] = {};
    const int total = tiles_m * tiles_n;
    for (int b = 0; b < total; ++b) {
        int tm = -1, tn = -1;
        grouped_tile<4>(xcd_contiguous(b, total), tiles_m, tiles_n, tm, tn);
        if (tm < 0 || tm >= tiles_m || tn < 0 || tn >= tiles_n || seen[tm * tiles_n + tn])
            return false;
        seen[tm * tiles_n + tn] = true;
    }
    return true;
}
static_assert(order_is_bijective(32, 56) && order_is_bijective(1, 448) && order_is_bijective(7, 9) &&
                  order_is_bijective(1, 1) && order_is_bijective(13, 5) && order_is_bijective(3, 1),
              "workgroup → tile order must cover every tile once");
// Tile t of the lower triangle (tn <= tm) of a square tile grid, row by row.
__device__ inline void triangle_tile(int t, int &tm, int &tn)
{
    int r = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > t)
        --r;
    while ((r + 1) * (r + 2) / 2 <= t)
        ++r;
    tm = r;
    tn = t - r * (r + 1) / 2;
}

// ---------------------------------------------------------------- LDS images
__host__ __device__ constexpr int kmajor_swz(int r) { return (r >> 1) & 7; }
__host__ __device__ constexpr int kmajor_off(int r, int c) { return r * BK + ((c ^ kmajor_swz(r)) << 3); }
static_assert(tg::layout::check_swizzled_tile(tg::layout::swizzle_bank256_f16(256, 64), 256, 64, kmajor_off),
              "K-major LDS addressing disagrees with ComposeLayout(3, 3, 4)");
template <int BX>
__host__ __device__ constexpr int trans_swz(int k)
{
    return BX % 128 == 0 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
}
// element offset of column x (a multiple of 4) of K row k
template <int BX>
__host__ __device__ constexpr int trans_off(int k, int x)
{
    return k * BX + (((x >> 4) ^ trans_swz<BX>(k)) << 4) + (x & 15);
}
// The two 8-byte reads of fragment q by lane l touch each (k, column) once and
// a half wave's 32 lanes cover the 64 banks once.
template <int BX>
constexpr bool trans_reads_are_conflict_free()
{
    for (int half = 0; half < 2; ++half)
        for (int hw = 0; hw < 2; ++hw)
            for (int q = 0; q < BX / 16; ++q) {
                bool bank[64] = {};
                for (int i = 0; i < 32; ++i) {
                    const int l = hw * 32 + i;
                    const int k = 8 * (l >> 4) + ((l & 15) >> 2) + 4 * half;
                    const int b = trans_off<BX>(k, q * 16 + 4 * (l & 3)) * 2 / 4;
                    if (bank[b % 64] || bank[(b + 1) % 64])
                        return false;
                    bank[b % 64] = bank[(b + 1) % 64] = true;
                }
            }
    return true;
}
static_assert(trans_reads_are_conflict_free<256>() && trans_reads_are_conflict_free<192>() &&
                  trans_reads_are_conflict_free<128>() && trans_reads_are_conflict_free<64>(),
              "transposed fragment reads must spread over the banks");

// One operand of a tile product.
//   K-major:    row x of the operand at p + x·ld, K consecutive elements
//   transposed: row k of the operand at p + k·ld, `extent` consecutive columns
// p 16-byte aligned, ld a multiple of 8.  x runs over [0, extent).
struct Operand {
    const void *p;
    int64_t ld;
    int extent;
};

// STREAM: for a product bound by reading B (one tile row): B is loaded past the
// caches, and the workgroups of the eight XCDs start at K-tiles spread over K and
// wrap around, so that they read from different address ranges at any moment.
// MASK: for a K-major A beside a transposed B, whose rows do not hold zeros up to
// a multiple of 64: A's chunks past K, a multiple of 8, read as zero.
template <typename E, int BM_, int BN_, int WM_, int WN_, int S_, bool TA_, bool TB_, bool STREAM_ = false,
          bool MASK_ = false>
struct Tile {
    static constexpr bool STREAM = STREAM_, MASK = MASK_;
    static_assert(!STREAM_ || (!TA_ && !TB_), "rotation is for the K-major product");
    static_assert(!MASK_ || (!TA_ && TB_), "the other products need no mask");
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
    static constexpr bool TA = TA_, TB = TB_;
    using V8 = typename El<E>::v8;
    static constexpr int NW = WM * WN, THREADS = NW * 64;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int TM = WTM / 16, TN = WTN / 16;
    static constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW;  // DMAs per wave and stage
    static constexpr int STAGE_A = BM * BK, STAGE_B = BN * BK;
    static constexpr int LDS_ELEMS = (S + 1) * STAGE_A + S * STAGE_B;
    static constexpr bool FIRST = !TA && !TB;  // the partial K-tile comes first
    static_assert(WTM % 16 == 0 && WTN % 16 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && NW >= 2, "tile");
    static_assert(LDS_ELEMS * 2 <= 160 * 1024, "LDS budget");
    static_assert(S >= 2 && (S - 1) * (PA + PB) + PA <= 63, "vmcnt holds 6 bits");
    static_assert(BM * BN <= LDS_ELEMS, "the block's 16-bit image fits the stages");

    // per-lane byte offsets of this lane's DMAs of one stage, from the operand's
    // origin of the tile
    template <bool T, int BX, int P>
    __device__ static void dma_offsets(uint32_t (&off)[P], int64_t ld, int x0, int extent, int lane, int wave)
    {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if constexpr (!T) {
                const int t = 8 * (p * NW + wave) + (lane >> 3);
                const int kc = (lane & 7) ^ kmajor_swz(t);
                off[p] = (uint32_t)((int64_t)imin(t, extent - 1 - x0) * ld * 2 + 16 * kc);
            } else {
                constexpr int CPR = BX / 8;
                const int slot = (p * NW + wave) * 64 + lane;
                const int k = slot / CPR, cp = slot % CPR;
                const int x = ((((cp >> 1) ^ trans_swz<BX>(k)) << 1) | (cp & 1)) * 8;
                off[p] = (uint32_t)((int64_t)k * ld * 2 + 2 * imin(x, ((extent - 1 - x0) & ~7)));
            }
        }
    }

    // acc += the K range [0, K) of the product's block at rows x0a, columns x0b.
    // KT = cdiv(K, 64) K-tiles; K == 0 adds nothing.  Every wave's DMAs have
    // landed on return, but other waves may still read the stages: a caller
    // that reuses smem first passes a barrier.
    // `ahead` is called before the last K-tile's products (256×256) or after
    // them: a place for an epilogue's first loads.
    template <typename F>
    __device__ static __attribute__((always_inline)) void run(E *smem, const Operand &a, const Operand &b, int x0a,
                                                             int x0b, int K, f32x4 (&acc)[TM][TN], F ahead)
    {
        x0a = uniform(x0a), x0b = uniform(x0b), K = uniform(K);
        E *const a_ring = smem;
        E *const b_ring = smem + (S + 1) * STAGE_A;
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int KT = (K + BK - 1) / BK;
        const int k0 = FIRST ? K - BK * KT : 0;
        const int rot = STREAM ? (int)(blockIdx.x % NUM_XCD) * KT / NUM_XCD : 0;

        uint32_t a_off[PA], b_off[PB];
        dma_offsets<TA, BM>(a_off, a.ld, x0a, a.extent, lane, wave);
        dma_offsets<TB, BN>(b_off, b.ld, x0b, b.extent, lane, wave);
        const char *const a_base =
            uniform(reinterpret_cast<const char *>(a.p) + 2 * (TA ? (int64_t)x0a : (int64_t)x0a * a.ld + k0));
        const char *const b_base =
            uniform(reinterpret_cast<const char *>(b.p) + 2 * (TB ? (int64_t)x0b : (int64_t)x0b * b.ld + k0));
        const int64_t a_step = TA ? 2 * BK * a.ld : 2 * BK, b_step = TB ? 2 * BK * b.ld : 2 * BK;
        // K-tile t's buffer: empty past the end; a transposed operand's ends
        // with its last K row.  32-bit scalar arithmetic without branches: a
        // branch in the loop makes the register allocator move accumulators.  The
        // range is uniform in so many words: the compiler computes it in vector
        // registers and put a loop over the lanes around each of B's DMAs where A is
        // K-major (4096×4096 Newton–Schulz 1386 us with them, 1322 without).
        auto rsrc = [&](const char *base, int64_t step, int64_t ld, int x0, bool trans, int t) {
            int pt = t;  // K-tile in memory order
            if constexpr (STREAM) {
                pt += rot;
                pt -= pt >= KT ? KT : 0;
            }
            const int rows = imax(imin(K - t * BK, BK), 0);
            const int range = uniform(trans ? imax(rows * (2 * (int)ld) - 2 * x0, 0) : t < KT ? DMA_RANGE : 0);
            return __builtin_amdgcn_make_buffer_rsrc((void *)(base + step * pt), (short)0, range, BUFFER_WORD3);
        };
        auto rsrc_a = [&](int t) { return rsrc(a_base, a_step, a.ld, x0a, TA, t); };
        auto rsrc_b = [&](int t) { return rsrc(b_base, b_step, b.ld, x0b, TB, t); };
        // the first K-tile's columns below 0 read as zero; the passes' rows are
        // NW·8 apart, so a lane's chunk is the same in all of them
        const int kc = 8 * ((lane & 7) ^ kmajor_swz(8 * wave + (lane >> 3)));
        static_assert(NW % 2 == 0, "swizzle repeats per pass");
        auto below = [&](int t) {
            const int pt = STREAM ? (t + rot >= KT ? t + rot - KT : t + rot) : t;
            return FIRST && pt == 0 && k0 + kc < 0;
        };
        auto past = [&](int t) { return MASK && kc >= K - t * BK; };
        auto dma_a = [&](__amdgpu_buffer_rsrc_t r, int stage, int p, bool zero) {
            dma16(r, a_ring + stage * STAGE_A + (p * NW + wave) * 512, zero ? DMA_OOB : a_off[p]);
        };
        auto dma_b = [&](__amdgpu_buffer_rsrc_t r, int stage, int p, bool zero) {
            dma16<STREAM ? 3 : 0>(r, b_ring + stage * STAGE_B + (p * NW + wave) * 512, zero ? DMA_OOB : b_off[p]);
        };

        // fragment reads
        constexpr int NA = TA ? TM : 2, NB = TB ? TN : 2;
        int a_lane[NA], b_lane[NB];
        auto lane_offsets = [&](auto trans, auto bx, auto n, int w0, int *o) {
            constexpr bool T = decltype(trans)::value;
            constexpr int BX = decltype(bx)::value, N = decltype(n)::value;
#pragma unroll
            for (int q = 0; q < N; ++q) {
                if constexpr (T)
                    o[q] = trans_off<BX>(8 * (lane >> 4) + ((lane & 15) >> 2), w0 + q * 16 + 4 * (lane & 3));
                else
                    o[q] = kmajor_off(w0 + (lane & 15), q * 4 + (lane >> 4));
            }
        };
        lane_offsets(std::bool_constant<TA>{}, std::integral_constant<int, BM>{}, std::integral_constant<int, NA>{},
                     wm * WTM, a_lane);
        lane_offsets(std::bool_constant<TB>{}, std::integral_constant<int, BN>{}, std::integral_constant<int, NB>{},
                     wn * WTN, b_lane);
        auto read_one = [&](auto trans, auto bx, const E *st, const int *o, int kk, int q) {
            if constexpr (decltype(trans)::value) {
                constexpr int BX = decltype(bx)::value;
                union {
                    s16x4 h[2];
                    V8 v;
                } u;
                u.h[0] = lds_read_tr(st + o[q] + kk * 32 * BX);
                u.h[1] = lds_read_tr(st + o[q] + kk * 32 * BX + 4 * BX);
                return u.v;
            } else {
                return *reinterpret_cast<const V8 *>(st + o[kk] + q * 16 * BK);
            }
        };
        auto read_frag = [&](int sa, int sb, int kk, int q, V8 *fa, V8 *fb) {
            if (q < TM)
                fa[q] = read_one(std::bool_constant<TA>{}, std::integral_constant<int, BM>{},
                                 a_ring + sa * STAGE_A, a_lane, kk, q);
            else
                fb[q - TM] = read_one(std::bool_constant<TB>{}, std::integral_constant<int, BN>{},
                                      b_ring + sb * STAGE_B, b_lane, kk, q - TM);
        };

        constexpr int NFRAG = TM + TN, SLOTS = TM * TN;
        constexpr int RSTRIDE = SLOTS / NFRAG > 0 ? SLOTS / NFRAG : 1;
        auto frag_of_slot = [](int i) { return i == 0 ? 0 : i <= TN ? TM + i - 1 : i - TN; };
        // One 32-K step: an MFMA per slot; between them the next step's
        // fragment reads and the DMAs of operand `which` (1: A, 2: B), pinned
        // in program order so that they issue in the shadow of the MFMAs.
        auto step = [&](const V8 *fa, const V8 *fb, bool reads, int rsa, int rsb, int rkk, V8 *na, V8 *nb, int which,
                        __amdgpu_buffer_rsrc_t r, int stage, bool zero) {
            constexpr int EA = SLOTS / PA > 0 ? SLOTS / PA : 1, EB = SLOTS / PB > 0 ? SLOTS / PB : 1;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                acc[i / TN][i % TN] = El<E>::mfma(fb[i % TN], fa[i / TN], acc[i / TN][i % TN]);
                __builtin_amdgcn_sched_barrier(0);
                if (reads && i % RSTRIDE == 0 && i / RSTRIDE < NFRAG)
                    read_frag(rsa, rsb, rkk, frag_of_slot(i / RSTRIDE), na, nb);
                if (which == 1 && i % EA == EA / 4 && i / EA < PA)
                    dma_a(r, stage, i / EA, zero);
                if (which == 2 && i % EB == EB / 4 && i / EB < PB)
                    dma_b(r, stage, i / EB, zero);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int q = (SLOTS + RSTRIDE - 1) / RSTRIDE; q < NFRAG; ++q)
                if (reads)
                    read_frag(rsa, rsb, rkk, frag_of_slot(q), na, nb);
            if (which == 1)
#pragma unroll
                for (int p = (SLOTS + EA - 1) / EA; p < PA; ++p)
                    dma_a(r, stage, p, zero);
            if (which == 2)
#pragma unroll
                for (int p = (SLOTS + EB - 1) / EB; p < PB; ++p)
                    dma_b(r, stage, p, zero);
        };

        // prologue: K-tiles 0 .. S-1
#pragma unroll
        for (int t = 0; t < S; ++t) {
            const auto ra = rsrc_a(t), rb = rsrc_b(t);
            const bool zero = (STREAM || t == 0) && below(t);
#pragma unroll
            for (int p = 0; p < PA; ++p)
                dma_a(ra, t, p, zero || past(t));
#pragma unroll
            for (int p = 0; p < PB; ++p)
                dma_b(rb, t, p, zero);
        }
        wait_vmem<(S - 1) * (PA + PB)>();
        barrier_lds();
        V8 fa[2][TM], fb[2][TN];
#pragma unroll
        for (int q = 0; q < NFRAG; ++q)
            read_frag(0, 0, 0, q, fa[0], fb[0]);

        // Up to 192×192 the last K-tile is one like the others (its refills have
        // empty ranges, the fragments it reads ahead go unused; K == 0 runs
        // none): half the code, and a launch of few workgroups pays for its
        // instruction fetches.  At 256×256 it is peeled off (K == 0: on zeros):
        // there the allocator moves accumulators around the plain loop.
        constexpr bool PEEL = BM * BN >= 256 * 256;
        int sa = 0, sb = 0;       // stages of K-tile t
        int da = S % (S + 1);     // stage A(t+S) goes into
        for (int t = 0; t < (PEEL ? KT - 1 : KT); ++t) {
            step(fa[0], fb[0], true, sa, sb, 1, fa[1], fb[1], 1, rsrc_a(t + S), da,
                 (STREAM && below(t + S)) || past(t + S));
            wait_vmem<(S - 2) * (PA + PB) + PA>();  // K-tile t+1 has landed (this wave's part)
            barrier_lds();                          // ... for every wave; K-tile t's stages are drained
            const int sa1 = sa == S ? 0 : sa + 1, sb1 = sb == S - 1 ? 0 : sb + 1;
            step(fa[1], fb[1], true, sa1, sb1, 0, fa[0], fb[0], 2, rsrc_b(t + S), sb,
                 STREAM && below(t + S));
            da = da == S ? 0 : da + 1;
            sa = sa1;
            sb = sb1;
        }
        ahead();
        if constexpr (PEEL) {
            const auto none = __builtin_amdgcn_make_buffer_rsrc(nullptr, (short)0, 0, BUFFER_WORD3);
            step(fa[0], fb[0], true, sa, sb, 1, fa[1], fb[1], 0, none, 0, false);
            step(fa[1], fb[1], false, 0, 0, 0, fa[0], fb[0], 0, none, 0, false);
        }
        // (the accumulators stay where they are between the loop and the
        // epilogue: without this some instantiations spilled a few of them)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                pin(acc[i][j]);
        wait_vmem<0>();
    }

    __device__ static __attribute__((always_inline)) void run(E *smem, const Operand &a, const Operand &b, int x0a,
                                                             int x0b, int K, f32x4 (&acc)[TM][TN])
    {
        run(smem, a, b, x0a, x0b, K, acc, [] {});
    }

    __device__ static __attribute__((always_inline)) void clear(f32x4 (&acc)[TM][TN])
    {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
};

// Elements c .. c + 7 of a row of K 16-bit elements, zeros behind its end; vec:
// the row is 16-byte aligned and K a multiple of 8.
__device__ inline uint4 load8(const uint16_t *s, int64_t c, int64_t K, bool vec)
{
    if (vec)
        return *reinterpret_cast<const uint4 *>(s + c);
    union {
        uint4 u;
        uint16_t h[8];
    } w;
    if (c + 8 <= K) {
        // one load of 16 bytes at the alignment of an element
        __builtin_memcpy(&w, s + c, 16);
        return w.u;
    }
    w.u = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < K)
            w.h[e] = s[c + e];
    return w.u;
}

// ------------------------------------------------------- staged block stores
// A wave's R×C block of 16-bit values in LDS, row-major with the 16-byte
// chunk index of row r XORed with r mod the largest power of two in C/8.
template <int C>
__host__ __device__ constexpr int stage_off(int r, int c)
{
    constexpr int MASK = ((C / 8) & -(C / 8)) - 1;
    return r * C + (((c >> 3) ^ (r & MASK)) << 3) + (c & 7);
}
// Rows [0, R) of the staged block to D rows row0 + r (through `map` where it
// is given: D row map[row0 + r]), columns col0 .., inside rows × cols; `vec`:
// D's rows are 16-byte aligned.  WORKSPACE: they always are, and cols is a
// multiple of 8.  NT: past the caches.
template <typename E, int R, int C, bool WORKSPACE = false, bool NT = false>
__device__ inline void store_block(const E *stg, E *__restrict__ D, int64_t ld, int row0, int col0, int rows,
                                   int cols, bool vec, const int *__restrict__ map, int lane)
{
    using V8 = typename El<E>::v8;
    constexpr int CH = C / 8;
    static_assert(R * CH % 64 == 0, "whole passes");
    if (WORKSPACE || (vec && col0 + C <= cols)) {
#pragma unroll 4
        for (int p = 0; p < R * CH / 64; ++p) {
            const int at = p * 64 + lane, rc = at % CH, r = at / CH;
            const int row = row0 + r, col = col0 + 8 * rc;
            const V8 v = *reinterpret_cast<const V8 *>(stg + stage_off<C>(r, 8 * rc));
            if (row < rows && (!WORKSPACE || col < cols)) {
                V8 *const to = reinterpret_cast<V8 *>(D + (int64_t)(map ? map[row] : row) * ld + col);
                if constexpr (NT)
                    __builtin_nontemporal_store(v, to);
                else
                    *to = v;
            }
        }
    } else {
#pragma unroll 1
        for (int p = 0; p < R * CH / 64; ++p) {
            const int at = p * 64 + lane, rc = at % CH, r = at / CH;
            const int row = row0 + r, col = col0 + 8 * rc;
            const V8 v = *reinterpret_cast<const V8 *>(stg + stage_off<C>(r, 8 * rc));
            if (row < rows) {
                E *dst = D + (int64_t)(map ? map[row] : row) * ld + col;
                if (col + 8 <= cols) {
                    __builtin_memcpy(dst, &v, 16);  // at the alignment of an element
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < cols)
                            dst[e] = v[e];
                }
            }
        }
    }
}
// Zero what a staged R×C block holds from row `rows` or column `cols` on.
template <typename E, int R, int C>
__device__ inline void clear_outside(E *stg, int rows, int cols, int lane)
{
    using V8 = typename El<E>::v8;
#pragma unroll 1
    for (int p = 0; p < R * C / 8 / 64; ++p) {
        const int at = p * 64 + lane, c = at % (C / 8) * 8, r = at / (C / 8);
        V8 *q = reinterpret_cast<V8 *>(stg + stage_off<C>(r, c));
        V8 v = *q;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = r < rows && c + e < cols ? v[e] : (E)0.0f;
        *q = v;
    }
}

// The transpose of a staged R×C block: D rows row0 .. row0 + C - 1, columns
// col0 .. col0 + R - 1, inside rows × cols (cols a multiple of 8, D's rows
// 16-byte aligned).  Two transposing LDS reads give a lane 8 consecutive
// elements of one row of the transpose.
template <typename E, int R, int C>
__device__ inline void store_block_transposed(const E *stg, E *__restrict__ D, int64_t ld, int row0, int col0,
                                              int rows, int cols, int lane)
{
    static_assert(R % 32 == 0 && C % 16 == 0, "whole groups");
    const int s = lane & 15, g = lane >> 4;
#pragma unroll 2
    for (int q = 0; q < C / 16; ++q)
#pragma unroll
        for (int h = 0; h < R / 32; ++h) {
            const int r = 32 * h + 8 * g;
            union {
                s16x4 h4[2];
                uint4 v;
            } u;
            u.h4[0] = lds_read_tr(stg + stage_off<C>(r + (s >> 2), 16 * q + 4 * (s & 3)));
            u.h4[1] = lds_read_tr(stg + stage_off<C>(r + 4 + (s >> 2), 16 * q + 4 * (s & 3)));
            const int row = row0 + 16 * q + s, col = col0 + r;
            if (row < rows && col < cols)
                *reinterpret_cast<uint4 *>(D + (int64_t)row * ld + col) = u.v;
        }
}

// ------------------------------------------------------------------- host
// Time in microseconds of `n` tiles of class `c` with `ktiles` K-tiles each:
// whole rounds of the workgroups that run at once, each the K-tiles of its tiles
// and a fixed part (first loads, epilogue, instruction fetches).  The constants
// were measured on one MI355X with launches of 1, 4 and 16 rounds and 2 to 224
// K-tiles; the model is within some 15% of those times.
struct TileClass {
    int bm, bn;
    int per_cu;     // workgroups per compute unit
    double ktile;   // per K-tile with all of them running
    double alone;   // with one per unit
    double fixed;
};
inline double tile_time(const TileClass &c, int64_t n, int64_t ktiles)
{
    const int64_t slots = (int64_t)NUM_CU * c.per_cu, rounds = cdiv(n, slots), rest = n - (rounds - 1) * slots;
    const double k = (double)ktiles;
    return (double)(rounds - 1) * (k * c.ktile + c.fixed) + k * (rest > NUM_CU ? c.ktile : c.alone) + c.fixed;
}

// 1 yes, -1 no, 0 not yet asked, per device
inline int gfx950_status()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return -1;
    if (dev < 64) {
        const int s = known[dev].load(std::memory_order_relaxed);
        if (s != 0)
            return s;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return -1;
    const int s = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    if (dev < 64)
        known[dev].store(s, std::memory_order_relaxed);
    return s;
}

// A launch holds fewer than 2^32 threads; workgroups here have at most 512 where
// their number grows with the problem.
constexpr int64_t MAX_GRID = (int64_t)1 << 23;
template <typename... P, typename... A>
inline bool launch(void (*fn)(P...), int64_t grid, int threads, void *stream, A... args)
{
    std::tuple<P...> held(args...);
    void *argv[sizeof...(P)];
    std::apply([&](auto &...x) {
        int i = 0;
        ((argv[i++] = (void *)&x), ...);
    }, held);
    if (grid * threads >= (int64_t)1 << 32)
        return false;
    return hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3((unsigned)grid), dim3(threads), argv, 0,
                           (hipStream_t)stream) == hipSuccess;
}

}  // namespace pt
}  // namespace

#endif  // TG_PROJ_TILE_HPP
