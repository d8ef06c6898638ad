// tg_adamw.hip — AdamW over many tensors at once.  See include/tg_adamw.h for
// the contract.
//
// One pass: an element's p, g, m and v are read, and p, m, v (and the copy)
// written, 28 bytes in fp32 and 10 with 16-bit p and g and 8-bit moments; the
// arithmetic hides behind them.  The tensors' pointers travel in the kernel's
// arguments, so that a call needs no table in device memory that a captured
// graph would have to keep.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <math.h>
#include <new>
#include <stdint.h>
#include <string.h>
#include <vector>

#include "proj_tile.hpp"

#include "tg_adamw.h"
#include "tg_gemm.h"

namespace {
using namespace pt;

constexpr int BLOCK = TG_ADAMW_BLOCK;
constexpr int PER_LANE = 4;      // consecutive elements
static_assert(BLOCK == 64 * PER_LANE, "a wave holds a block");
constexpr int THREADS = 256, WAVES = THREADS / 64;
constexpr int STEPS = 4;         // blocks of a wave
constexpr int CHUNK = WAVES * STEPS * BLOCK;  // elements of a workgroup
constexpr int TABLE = 56;        // tensors of one launch: 4 KiB of kernel arguments
constexpr int64_t MOST = (int64_t)1 << 35;    // elements of a tensor: 2^23 workgroups
static_assert(MOST / CHUNK * THREADS < (int64_t)1 << 32, "threads of a launch");
constexpr float TOP = 448.0f;    // E4M3's largest value
constexpr float LEAST = 0x1p-9f; // its smallest above zero
constexpr float FLUSH = 0x1p-110f;
constexpr float ROOT_LEAST = 0x1p-74f;  // of a root: rounded to E4M3 and squared, still above zero in fp32

// What depends on the step alone, rounded once from 64 bits.
struct Factors {
    float b1, c1, b2, c2;   // β and 1 − β
    float keep, rate, root; // 1 − lr·wd, lr/(1 − β1^t), 1/√(1 − β2^t)
    float eps;
};
__host__ __device__ inline Factors factors(double lr, double b1, double b2, double eps, double wd, double t)
{
    Factors f;
    f.b1 = (float)b1, f.c1 = (float)(1.0 - b1);
    f.b2 = (float)b2, f.c2 = (float)(1.0 - b2);
    f.keep = (float)(1.0 - lr * wd);
    f.rate = (float)(lr / (1.0 - pow(b1, t)));
    f.root = (float)(1.0 / sqrt(1.0 - pow(b2, t)));
    f.eps = eps < 0x1p-126 ? 0.0f : (float)eps;  // a reciprocal takes no subnormal number
    return f;
}

struct Args {
    Factors f;
    double lr, b1, b2, eps, wd;  // for factors that are found on the device
    int64_t step;
    const float *lr_at;
    const int64_t *step_at;
    const float *g_scale;
    int count, copy_type;
    int first[TABLE];            // a tensor's first workgroup
    tg_adamw_tensor t[TABLE];
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

__device__ inline float to_f32(float x) { return x; }
__device__ inline float to_f32(_Float16 x) { return (float)x; }
__device__ inline float to_f32(__bf16 x) { return (float)x; }

// PER_LANE elements from i on, as they lie, `n` of them inside the tensor.  The
// elements' own alignment is all that is asked for: loads and stores of four elements
// may lie on any byte here, and are as fast as aligned ones.
template <typename T>
struct Raw {
    T e[PER_LANE];
};
template <bool WHOLE, typename T>
__device__ inline Raw<T> load(const T *p, int64_t i, int n)
{
    Raw<T> w;
    if (WHOLE || n >= PER_LANE) {
        __builtin_memcpy(&w, p + i, sizeof w);
    } else {
#pragma unroll
        for (int e = 0; e < PER_LANE; ++e)
            w.e[e] = e < n ? p[i + e] : (T)0;
    }
    return w;
}
template <bool WHOLE, typename T>
__device__ inline void store(const Raw<T> &w, T *p, int64_t i, int n)
{
    if (WHOLE || n >= PER_LANE) {
        __builtin_memcpy(p + i, &w, sizeof w);
    } else {
#pragma unroll
        for (int e = 0; e < PER_LANE; ++e)
            if (e < n)
                p[i + e] = w.e[e];
    }
}
template <bool WHOLE, typename T>
__device__ inline void store(const float (&x)[PER_LANE], T *p, int64_t i, int n)
{
    Raw<T> w;
#pragma unroll
    for (int e = 0; e < PER_LANE; ++e)
        w.e[e] = (T)x[e];
    store<WHOLE>(w, p, i, n);
}
__device__ inline void decode(float (&x)[PER_LANE], const Raw<uint8_t> &raw, float scale)
{
#if defined(__HIP_DEVICE_COMPILE__)
    int w;
    __builtin_memcpy(&w, &raw, 4);
    x[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * scale;
    x[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * scale;
    x[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * scale;
    x[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * scale;
#endif
}
// The block's E4M3 values of x, rounded to nearest even, and its scale.  The
// largest magnitude is found on the bit patterns, which order as the magnitudes
// do and put a NaN above an infinity, so that neither gets lost.
template <bool ROOT>
__device__ inline Raw<uint8_t> encode(const float (&x)[PER_LANE], float &scale)
{
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < PER_LANE; ++e)
        top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
    for (int o = 32; o; o >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, o));
    const float most = __uint_as_float(top);
    const bool held = !(most < FLUSH);
    const float per = held ? 1.0f / most * TOP : 0.0f;
    scale = held ? most * (1.0f / TOP) : 0.0f;
    // A root above zero is held as one whose square is above zero, so that v never reads as
    // zero where it is not: at least as the smallest value, and, in blocks whose largest is
    // below 2^-56, as 2^-74: an E4M3 value above 2^-9 is rounded down by less than a third, and
    // the square of 2/3·2^-74 is 0.9 of fp32's smallest number, to which it is rounded.
    const float least = ROOT ? fminf(fmaxf(ROOT_LEAST * per, LEAST), TOP) : 0.0f;
    float q[PER_LANE];
#pragma unroll
    for (int e = 0; e < PER_LANE; ++e) {
        q[e] = fminf(fmaxf(x[e] * per, -TOP), TOP);
        if (ROOT && q[e] > 0.0f)
            q[e] = fmaxf(q[e], least);
    }
    int w = 0;
#if defined(__HIP_DEVICE_COMPILE__)
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
#endif
    Raw<uint8_t> raw;
    __builtin_memcpy(&raw, &w, 4);
    return raw;
}

// A block on its way: what a lane holds of it.
template <typename P, typename G, int BITS>
struct Held {
    using M = std::conditional_t<BITS == 8, uint8_t, float>;
    Raw<P> p;
    Raw<G> g;
    Raw<M> m, v;
    float m_scale, v_scale;
};
template <typename P, typename G, int BITS, bool WHOLE>
__device__ inline void load_block(Held<P, G, BITS> &h, const tg_adamw_tensor &t, int64_t b, int lane)
{
    using M = typename Held<P, G, BITS>::M;
    const int64_t i = b + lane * PER_LANE;
    const int left = (int)(t.n - i < PER_LANE ? t.n - i : PER_LANE);  // <= 0 behind the end
    h.p = load<WHOLE>((const P *)t.p, i, left);
    h.g = load<WHOLE>((const G *)t.g, i, left);
    h.m = load<WHOLE>((const M *)t.m, i, left);
    h.v = load<WHOLE>((const M *)t.v, i, left);
    if constexpr (BITS == 8) {
        h.m_scale = t.m_scale[b / BLOCK];
        h.v_scale = t.v_scale[b / BLOCK];
    }
}
template <typename P, typename G, int BITS, bool WHOLE>
__device__ inline void step_block(const Held<P, G, BITS> &h, const tg_adamw_tensor &t, int64_t b, int lane,
                                  const Factors &f, float s, int copy_type)
{
#pragma clang fp contract(off)
    const int64_t i = b + lane * PER_LANE;
    const int left = (int)(t.n - i < PER_LANE ? t.n - i : PER_LANE);
    float p[PER_LANE], m[PER_LANE], v[PER_LANE], r[PER_LANE];
    if constexpr (BITS == 8) {
        decode(m, h.m, h.m_scale);
        decode(v, h.v, h.v_scale);
    }
#pragma unroll
    for (int e = 0; e < PER_LANE; ++e) {
        if constexpr (BITS == 32)
            m[e] = h.m.e[e], v[e] = h.v.e[e];
        else
            v[e] = v[e] * v[e];
        const float g = to_f32(h.g.e[e]) * s;
        m[e] = m[e] * f.b1 + g * f.c1;
        v[e] = v[e] * f.b2 + (g * g) * f.c2;
        r[e] = sqrtf(v[e]);
        // the quotient as a product with the hardware's reciprocal (1 ulp): a division
        // rounded to nearest takes ten instructions, and with 8-bit moments the
        // arithmetic shows (307M bf16 parameters 614 us, 652 with the division)
        p[e] = to_f32(h.p.e[e]) * f.keep - (m[e] * __builtin_amdgcn_rcpf(r[e] * f.root + f.eps)) * f.rate;
    }
    store<WHOLE>(p, (P *)t.p, i, left);
    if constexpr (std::is_same_v<P, float>) {
        if (t.copy) {
            if (copy_type == TG_ADAMW_BF16)
                store<WHOLE>(p, (__bf16 *)t.copy, i, left);
            else
                store<WHOLE>(p, (_Float16 *)t.copy, i, left);
        }
    }
    if constexpr (BITS == 32) {
        store<WHOLE>(m, (float *)t.m, i, left);
        store<WHOLE>(v, (float *)t.v, i, left);
    } else {
        if (!WHOLE)
#pragma unroll
            for (int e = 0; e < PER_LANE; ++e)  // a NaN gradients' scale makes them NaN
                if (e >= left)
                    m[e] = r[e] = 0.0f;
        float sm, sv;
        const Raw<uint8_t> wm = encode<false>(m, sm), wv = encode<true>(r, sv);
        store<WHOLE>(wm, (uint8_t *)t.m, i, left);
        store<WHOLE>(wv, (uint8_t *)t.v, i, left);
        if (lane == 0) {
            t.m_scale[b / BLOCK] = sm;
            t.v_scale[b / BLOCK] = sv;
        }
    }
}

// One workgroup takes CHUNK elements of one tensor, a wave STEPS blocks of them, all
// loaded before it works on the first (239M fp32 parameters with bf16 gradients and copies
// 1246 us, 1261 one block at a time: 5.4 TB/s, a large copy's rate; 307M bf16 ones with
// 8-bit moments 604 us, 5.1 TB/s).  READ: the rate or the step lies in device memory, and every
// lane finds the factors itself, in 64 bits (a kernel of its own: the powers take
// twice the registers).  Where the arithmetic shows this costs: the 307M with 8-bit moments 716 us
// instead of 593 in replayed graphs, the 239M in fp32 1258 instead of 1242, three small tensors 13.1 both.
template <typename P, typename G, int BITS, bool READ>
__global__ __launch_bounds__(THREADS) void adamw_kernel(Args a)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    // the last tensor that starts at or before this workgroup
    const int mine = lane < a.count ? a.first[lane] : 0x7fffffff;
    const int at = uniform(__popcll(__ballot(mine <= (int)blockIdx.x)) - 1);
    const tg_adamw_tensor t = a.t[at];
    const int64_t i0 = (int64_t)((int)blockIdx.x - a.first[at]) * CHUNK + (int64_t)wave * (STEPS * BLOCK);
    Factors f = a.f;
    if constexpr (READ) {
        const int64_t step = a.step_at ? *a.step_at : a.step;
        f = factors(a.lr_at ? (double)*a.lr_at : a.lr, a.b1, a.b2, a.eps, a.wd, (double)(step < 1 ? 1 : step));
    }
    const float s = a.g_scale ? *a.g_scale : 1.0f;
    if (i0 + STEPS * BLOCK <= t.n) {
        Held<P, G, BITS> h[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            load_block<P, G, BITS, true>(h[k], t, i0 + k * BLOCK, lane);
        __builtin_amdgcn_sched_barrier(0);  // the loads first
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            step_block<P, G, BITS, true>(h[k], t, i0 + k * BLOCK, lane, f, s, a.copy_type);
    } else {
        const int64_t end = t.n < i0 + STEPS * BLOCK ? t.n : i0 + STEPS * BLOCK;
#pragma unroll 1
        for (int64_t b = i0; b < end; b += BLOCK) {
            Held<P, G, BITS> h;
            load_block<P, G, BITS, false>(h, t, b, lane);
            step_block<P, G, BITS, false>(h, t, b, lane, f, s, a.copy_type);
        }
    }
}

// ------------------------------------------------------------------- host
int type_bytes(int type) { return type == TG_ADAMW_F32 ? 4 : 2; }
bool type_ok(int type) { return type == TG_ADAMW_F32 || type == TG_ADAMW_F16 || type == TG_ADAMW_BF16; }
bool range_ok(double x, double end) { return x >= 0.0 && x < end; }

struct Range {
    uintptr_t from, to;
    bool operator<(const Range &o) const { return from < o.from; }
};

int check(const tg_adamw_tensor *ts, int64_t count, const tg_adamw_config *c)
{
    if (count < 0 || !c || (count > 0 && !ts))
        return TG_ERR_INVALID_ARG;
    if (!type_ok(c->p_type) || !type_ok(c->g_type) || (c->g_type != c->p_type && c->p_type != TG_ADAMW_F32) ||
        (c->bits != 32 && c->bits != 8))
        return TG_ERR_INVALID_ARG;
    if (!range_ok(c->lr, INFINITY) || !range_ok(c->beta1, 1.0) || !range_ok(c->beta2, 1.0) ||
        !range_ok(c->eps, INFINITY) || !range_ok(c->weight_decay, INFINITY) || (!c->step_at && c->step < 1))
        return TG_ERR_INVALID_ARG;
    const uintptr_t pb = (uintptr_t)type_bytes(c->p_type), gb = (uintptr_t)type_bytes(c->g_type);
    std::vector<Range> written, read;
    written.reserve((size_t)count * 6), read.reserve((size_t)count + 3);
    bool ok = true, small = true;
    const auto add = [&](std::vector<Range> &to, const void *p, int64_t n, uintptr_t bytes) {
        const uintptr_t u = (uintptr_t)p;
        ok = ok && p && u % bytes == 0;
        to.push_back({u, u + (uintptr_t)n * bytes});
    };
    for (int64_t k = 0; k < count; ++k) {
        const tg_adamw_tensor &t = ts[k];
        ok = ok && t.n >= 0;
        small = small && t.n < MOST;
        if (t.n == 0 || !ok || !small)
            continue;
        const uintptr_t mb = c->bits == 32 ? 4 : 1;
        add(written, t.p, t.n, pb);
        add(read, t.g, t.n, gb);
        add(written, t.m, t.n, mb);
        add(written, t.v, t.n, mb);
        if (c->bits == 8) {
            add(written, t.m_scale, cdiv(t.n, BLOCK), 4);
            add(written, t.v_scale, cdiv(t.n, BLOCK), 4);
        }
        if (t.copy) {
            ok = ok && c->p_type == TG_ADAMW_F32 && (c->copy_type == TG_ADAMW_F16 || c->copy_type == TG_ADAMW_BF16);
            add(written, t.copy, t.n, 2);
        }
    }
    if (c->lr_at)
        add(read, c->lr_at, 1, 4);
    if (c->step_at)
        add(read, c->step_at, 1, 8);
    if (c->g_scale)
        add(read, c->g_scale, 1, 4);
    if (!ok)
        return TG_ERR_INVALID_ARG;
    if (!small)
        return TG_ERR_TOO_LARGE;
    std::sort(written.begin(), written.end());
    for (size_t k = 1; k < written.size(); ++k)
        if (written[k].from < written[k - 1].to)
            return TG_ERR_INVALID_ARG;
    for (const Range &r : read) {
        // the first that ends behind r's start
        const auto w = std::upper_bound(written.begin(), written.end(), r.from,
                                        [](uintptr_t x, const Range &y) { return x < y.to; });
        if (w != written.end() && w->from < r.to)
            return TG_ERR_INVALID_ARG;
    }
    return TG_OK;
}

template <typename P, typename G>
bool launch_typed(const Args &a, int64_t grid, int bits, void *stream)
{
    const bool read = a.lr_at || a.step_at;
    if (bits == 8)
        return read ? launch(adamw_kernel<P, G, 8, true>, grid, THREADS, stream, a)
                    : launch(adamw_kernel<P, G, 8, false>, grid, THREADS, stream, a);
    return read ? launch(adamw_kernel<P, G, 32, true>, grid, THREADS, stream, a)
                : launch(adamw_kernel<P, G, 32, false>, grid, THREADS, stream, a);
}

int step(const tg_adamw_tensor *ts, int64_t count, const tg_adamw_config *c, void *stream)
{
    const int st = check(ts, count, c);
    if (st != TG_OK)
        return st;
    if (std::all_of(ts, ts + count, [](const tg_adamw_tensor &t) { return t.n == 0; }))
        return TG_OK;
    if (gfx950_status() != 1)
        return TG_ERR_DEVICE;
    Args a;
    memset(&a, 0, sizeof a);
    a.lr = c->lr, a.b1 = c->beta1, a.b2 = c->beta2, a.eps = c->eps, a.wd = c->weight_decay, a.step = c->step;
    a.lr_at = c->lr_at, a.step_at = c->step_at, a.g_scale = c->g_scale;
    a.copy_type = c->copy_type;
    a.f = factors(a.lr, a.b1, a.b2, a.eps, a.wd, (double)std::max(c->step, (int64_t)1));
    int64_t grid = 0;
    const auto flush = [&] {
        if (a.count == 0)
            return true;
        bool ok;
        if (c->p_type == TG_ADAMW_F16)
            ok = launch_typed<_Float16, _Float16>(a, grid, c->bits, stream);
        else if (c->p_type == TG_ADAMW_BF16)
            ok = launch_typed<__bf16, __bf16>(a, grid, c->bits, stream);
        else if (c->g_type == TG_ADAMW_F16)
            ok = launch_typed<float, _Float16>(a, grid, c->bits, stream);
        else if (c->g_type == TG_ADAMW_BF16)
            ok = launch_typed<float, __bf16>(a, grid, c->bits, stream);
        else
            ok = launch_typed<float, float>(a, grid, c->bits, stream);
        a.count = 0, grid = 0;
        return ok;
    };
    for (int64_t k = 0; k < count; ++k) {
        if (ts[k].n == 0)
            continue;
        const int64_t need = cdiv(ts[k].n, CHUNK);
        if ((a.count == TABLE || grid + need > MOST / CHUNK) && !flush())
            return TG_ERR_LAUNCH;
        a.t[a.count] = ts[k];
        a.first[a.count++] = (int)grid;
        grid += need;
    }
    return flush() ? TG_OK : TG_ERR_LAUNCH;
}
}  // namespace

extern "C" int tg_adamw(const tg_adamw_tensor *tensors, int64_t count, const tg_adamw_config *config, void *stream)
{
    try {
        return step(tensors, count, config, stream);
    } catch (const std::bad_alloc &) {  // the host's list of ranges
        return TG_ERR_TOO_LARGE;
    } catch (...) {
        return TG_ERR_INVALID_ARG;
    }
}
