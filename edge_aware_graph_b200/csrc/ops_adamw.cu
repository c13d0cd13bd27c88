// One AdamW step over all tensors of a model (eaga_adamw_step), and the
// states in 32 bits (eaga_adamw_unpack).  Per element, with t the step being
// taken and every operation rounded to fp32 on its own (no contraction, so
// that a step is reproducible bit for bit, also by elementwise code):
//
//   g  = grad_scale * grad
//   m' = beta1 m + (1 - beta1) g        v' = beta2 v + (1 - beta2) (g g)
//   p' = (1 - lr wd) p - (lr / (1 - beta1^t)) (m' / (sqrt(v') / sqrt(1 - beta2^t) + eps))
//
// States in 8 bits hold m and r = sqrt(v) in blocks of 256 elements that
// share a scale (the block's largest magnitude over the largest code).  Codes
// are small floats: m a sign, 4 bits of exponent, 3 of fraction; r, never
// negative, 4 of exponent and 4 of fraction (the root halves the range that
// the exponent has to cover).  Both have gradual underflow, which here is the
// fp32 format's own: a value over its scale times 2^-112 has exactly the
// code in its upper bits, subnormal ones included, so a code is a shift away
// in both directions.  The bits below the code are rounded up or down at
// random (a hash of seed, step and element): at beta2 = 0.999 an average
// moves by less than half a code a step, and rounding to nearest would leave
// it where it is.  A positive r is never rounded to 0, where m / (0 + eps)
// would be a jump.  m' and v' enter the weight before they are rounded.
//
// Bound: HBM.  A bf16 weight with its fp32 master, an fp32 gradient and fp32
// states moves 30 bytes an element, with 8-bit states 18; the arithmetic (two
// divisions, a root, for 8 bits two hashes) hides behind it.  A warp takes
// 256 consecutive elements, 8 a lane: 16-byte accesses throughout, and the
// 8-bit scale is a warp maximum.  The tensors' table travels in the kernel's
// parameters: no device copy to keep, and a captured graph holds its own.
#include <math.h>
#include <stdlib.h>
#include <algorithm>
#include "common.cuh"
#include "ops.h"

namespace eaga {
namespace ops {

constexpr int AD_THR = 256, AD_WARP = 256, AD_TILE = 2048;   // threads; elements a warp / a CTA takes at once
constexpr int AD_BLOCK = 256;                                // elements that share a scale

struct AdEntry {
    void *p;
    float *master;
    const void *g;
    void *m, *v;
    float *ms, *vs;
    long long n;
    unsigned long long counter;
    float wd;
    unsigned first;      // the entry's first tile
};
struct AdScalars {
    double lr, beta1, beta2;
    float b1, omb1, b2, omb2, eps, gscale;
    const float *lr_dev;
    long long *state;    // [0] the step, [1] the CTAs done with it
    unsigned seed, tiles;
    int count, advance;
};
template <int CAP>
struct AdTable {
    AdScalars s;
    AdEntry e[CAP];
};
static_assert(sizeof(AdTable<384>) <= 32764, "kernel parameters");

// A 32-bit hash: xor-shift and odd multipliers, two rounds.
__host__ __device__ __forceinline__ unsigned mix32(unsigned x) {
    x = (x ^ (x >> 16)) * 0x6C8E9CF5u;
    x = (x ^ (x >> 15)) * 0x5B2D1A67u;
    return x ^ (x >> 16);
}

// base^t for t >= 0 in double, by repeated squaring.
__device__ __forceinline__ double ipow(double base, long long t) {
    double r = 1.0;
    for (; t > 0; t >>= 1, base *= base)
        if (t & 1) r *= base;
    return r;
}

__device__ __forceinline__ void ld8(const float *p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ld8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
    const unsigned w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ void st8(float *p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint4 o;
    __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    __stcs(reinterpret_cast<uint4 *>(p), o);
}
// 8 consecutive elements, the first `k` of them there (the last lanes of a tensor).
template <typename T>
__device__ __forceinline__ void load8(const T *p, int k, float (&v)[8]) {
    if (k == 8) {
        ld8(p, v);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = u < k ? ldf(p + u) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int k, const float (&v)[8]) {
    if (k == 8) {
        st8(p, v);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (u < k) stf(p + u, v[u]);
    }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int k) {
    if (k == 8) return __ldcs(reinterpret_cast<const uint2 *>(p));
    uint2 c = make_uint2(0, 0);
#pragma unroll
    for (int u = 0; u < 8; ++u)
        if (u < k) (u < 4 ? c.x : c.y) |= (unsigned)p[u] << (8 * (u & 3));
    return c;
}
__device__ __forceinline__ void store_codes(uint8_t *p, int k, uint2 c) {
    if (k == 8) {
        __stcs(reinterpret_cast<uint2 *>(p), c);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (u < k) p[u] = (uint8_t)((u < 4 ? c.x : c.y) >> (8 * (u & 3)));
    }
}
__device__ __forceinline__ unsigned code_at(uint2 c, int u) { return ((u < 4 ? c.x : c.y) >> (8 * (u & 3))) & 255u; }

constexpr float CODE_UP = 0x1p112f, CODE_DOWN = 0x1p-112f;   // between a code's bits and its value over the scale
constexpr float M_TOP = 1.875f, R_TOP = 1.9375f;             // the largest codes' values

__device__ __forceinline__ float decode_m(unsigned c, float scale) {
    const float a = __fmul_rn(__fmul_rn(__uint_as_float((c & 127u) << 20), CODE_UP), scale);
    return c & 128u ? -a : a;
}
__device__ __forceinline__ float decode_r(unsigned c, float scale) {
    return __fmul_rn(__fmul_rn(__uint_as_float(c << 19), CODE_UP), scale);
}
// The warp's largest magnitude; a NaN is larger than everything and stays.
__device__ __forceinline__ float warp_abs_max(const float (&v)[8]) {
    unsigned a = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) a = max(a, __float_as_uint(v[u]) & 0x7fffffffu);
    return __uint_as_float(__reduce_max_sync(0xffffffffu, a));
}
__device__ __forceinline__ unsigned scaled_bits(float a, float scale, bool zero) {
    return zero ? 0u : __float_as_uint(__fmul_rn(__fdiv_rn(a, scale), CODE_DOWN));
}

template <typename PT, typename GT, int BITS, bool MASTER, int CAP>
__global__ void __launch_bounds__(AD_THR)
k_adamw(const __grid_constant__ AdTable<CAP> tab) {
    after_previous();
    const AdScalars &s = tab.s;
    __shared__ float sh_size, sh_inv;
    __shared__ double sh_lr;
    __shared__ unsigned sh_key;
    if (threadIdx.x == 0) {
        const long long t = s.state[0] + 1;
        const double lr = s.lr_dev ? (double)*s.lr_dev : s.lr;
        sh_lr = lr;
        sh_size = (float)(lr / (1.0 - ipow(s.beta1, t)));
        sh_inv = (float)(1.0 / sqrt(1.0 - ipow(s.beta2, t)));
        sh_key = mix32((unsigned)t * 0x9E3779B9u + s.seed);
    }
    __syncthreads();
    const float size = sh_size, inv = sh_inv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (unsigned tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
        int lo = 0, hi = s.count;                    // the last entry whose first tile is at most `tile`
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tab.e[mid].first <= tile) lo = mid;
            else hi = mid;
        }
        const AdEntry &e = tab.e[lo];
        const long long w0 = (long long)(tile - e.first) * AD_TILE + warp * AD_WARP, i0 = w0 + 8 * lane;
        if (w0 >= e.n) continue;                      // whole warps only
        const int k = (int)max(0LL, min(8LL, e.n - i0));
        float g[8], p[8], m[8], v[8];
        load8(static_cast<const GT *>(e.g) + i0, k, g);
        if constexpr (MASTER) load8(e.master + i0, k, p);
        else load8(static_cast<const PT *>(e.p) + i0, k, p);
        const long long blk = w0 / AD_BLOCK;
        if constexpr (BITS == 32) {
            load8(static_cast<const float *>(e.m) + i0, k, m);
            load8(static_cast<const float *>(e.v) + i0, k, v);
        } else {
            const uint2 cm = load_codes(static_cast<const uint8_t *>(e.m) + i0, k);
            const uint2 cv = load_codes(static_cast<const uint8_t *>(e.v) + i0, k);
            const float sm = e.ms[blk], sv = e.vs[blk];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                m[u] = decode_m(code_at(cm, u), sm);
                const float r = decode_r(code_at(cv, u), sv);
                v[u] = __fmul_rn(r, r);
            }
        }
        const float keep = (float)__dsub_rn(1.0, __dmul_rn(sh_lr, (double)e.wd));
        float r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float gu = __fmul_rn(g[u], s.gscale);
            m[u] = __fadd_rn(__fmul_rn(m[u], s.b1), __fmul_rn(gu, s.omb1));
            v[u] = __fadd_rn(__fmul_rn(v[u], s.b2), __fmul_rn(__fmul_rn(gu, gu), s.omb2));
            r[u] = __fsqrt_rn(v[u]);
            const float d = __fadd_rn(__fmul_rn(r[u], inv), s.eps);
            p[u] = __fsub_rn(__fmul_rn(p[u], keep), __fmul_rn(__fdiv_rn(m[u], d), size));
        }
        if constexpr (MASTER) store8(e.master + i0, k, p);
        store8(static_cast<PT *>(e.p) + i0, k, p);
        if constexpr (BITS == 32) {
            store8(static_cast<float *>(e.m) + i0, k, m);
            store8(static_cast<float *>(e.v) + i0, k, v);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)               // past the tensor's end: nothing
                if (u >= k) m[u] = r[u] = 0.f;
            const float am = warp_abs_max(m), ar = warp_abs_max(r);
            const float sm = __fdiv_rn(am, M_TOP), sr = __fdiv_rn(ar, R_TOP);
            uint2 cm = make_uint2(0, 0), cr = make_uint2(0, 0);
            const unsigned long long c0 = e.counter + (unsigned long long)i0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const unsigned h = mix32((unsigned)(c0 + u) + sh_key);
                const unsigned h2 = h * 0x3C6EF35Fu;
                unsigned a = min(127u, (scaled_bits(fabsf(m[u]), sm, am == 0.f) + (h >> 12)) >> 20);
                if (m[u] < 0.f) a |= 128u;
                unsigned b = min(255u, (scaled_bits(r[u], sr, ar == 0.f) + (h2 >> 13)) >> 19);
                if (r[u] > 0.f) b = max(b, 1u);
                (u < 4 ? cm.x : cm.y) |= a << (8 * (u & 3));
                (u < 4 ? cr.x : cr.y) |= b << (8 * (u & 3));
            }
            store_codes(static_cast<uint8_t *>(e.m) + i0, k, cm);
            store_codes(static_cast<uint8_t *>(e.v) + i0, k, cr);
            if (lane == 0) {
                e.ms[blk] = sm;
                e.vs[blk] = sr;
            }
        }
    }
    before_next();
    // The last CTA of the call's last launch to have read the step advances it.
    if (s.advance && threadIdx.x == 0) {
        unsigned *done = reinterpret_cast<unsigned *>(s.state + 1);
        __threadfence();
        if (atomicInc(done, gridDim.x - 1) == gridDim.x - 1) s.state[0] += 1;
    }
}

// m and v = r^2 of 8-bit states as fp32: `p` the output for m, `master` that for v.
template <int CAP>
__global__ void __launch_bounds__(AD_THR)
k_adamw_unpack(const __grid_constant__ AdTable<CAP> tab) {
    after_previous();
    const AdScalars &s = tab.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (unsigned tile = blockIdx.x; tile < s.tiles; tile += gridDim.x) {
        int lo = 0, hi = s.count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tab.e[mid].first <= tile) lo = mid;
            else hi = mid;
        }
        const AdEntry &e = tab.e[lo];
        const long long w0 = (long long)(tile - e.first) * AD_TILE + warp * AD_WARP, i0 = w0 + 8 * lane;
        if (w0 >= e.n) continue;
        const int k = (int)max(0LL, min(8LL, e.n - i0));
        const uint2 cm = load_codes(static_cast<const uint8_t *>(e.m) + i0, k);
        const uint2 cv = load_codes(static_cast<const uint8_t *>(e.v) + i0, k);
        const float sm = e.ms[w0 / AD_BLOCK], sv = e.vs[w0 / AD_BLOCK];
        float m[8], v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            m[u] = decode_m(code_at(cm, u), sm);
            const float r = decode_r(code_at(cv, u), sv);
            v[u] = __fmul_rn(r, r);
        }
        if (e.p) store8(static_cast<float *>(e.p) + i0, k, m);
        if (e.master) store8(e.master + i0, k, v);
    }
}

// ------------------------------------------------------------------ host side

static int ad_grid(unsigned tiles) {
    // four CTAs an SM: 8 warps each with 64-128 bytes a lane in flight
    const unsigned most = 4u * (unsigned)sm_count();
    return (int)(tiles < 1 ? 1 : (tiles < most ? tiles : most));
}

template <typename PT, typename GT, int BITS, bool MASTER>
struct StepLaunch {
    template <int CAP>
    static cudaError_t go(const AdTable<CAP> &t, cudaStream_t st) {
        return launch_pdl(k_adamw<PT, GT, BITS, MASTER, CAP>, dim3(ad_grid(t.s.tiles)), dim3(AD_THR), 0, st, 1, t);
    }
};
struct UnpackLaunch {
    template <int CAP>
    static cudaError_t go(const AdTable<CAP> &t, cudaStream_t st) {
        return launch_pdl(k_adamw_unpack<CAP>, dim3(ad_grid(t.s.tiles)), dim3(AD_THR), 0, st, 1, t);
    }
};

// Entries lo .. hi-1 (no empty ones) in one launch.
template <typename LAUNCH, int CAP>
static cudaError_t launch_part(const AdScalars &s, const AdEntry *e, int count, bool last, cudaStream_t st) {
    AdTable<CAP> t;
    t.s = s;
    t.s.count = count;
    t.s.advance = last ? s.advance : 0;
    unsigned tiles = 0;
    for (int k = 0; k < count; ++k) {
        t.e[k] = e[k];
        t.e[k].first = tiles;
        tiles += (unsigned)((e[k].n + AD_TILE - 1) / AD_TILE);
    }
    t.s.tiles = tiles;
    return LAUNCH::go(t, st);
}

// A launch copies its whole table: up to 64 tensors (a block of the framework has 39) travel in a small one,
// more in launches of 384 (32 KB of parameters, the most a launch takes; 3 us more of the host's time).
template <typename LAUNCH>
static cudaError_t launch_all(const AdScalars &s, const AdEntry *e, int count, cudaStream_t st) {
    int at = 0;
    do {
        const int k = std::min(count - at, 384);
        const bool last = at + k == count;
        const cudaError_t err = k <= 64 ? launch_part<LAUNCH, 64>(s, e + at, k, last, st)
                                        : launch_part<LAUNCH, 384>(s, e + at, k, last, st);
        if (err != cudaSuccess) return err;
        at += k;
    } while (at < count);
    return cudaSuccess;
}

template <int BITS>
static cudaError_t launch_step(int pdt, int gdt, bool master, const AdScalars &s, const AdEntry *e, int count,
                               cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (pdt == EAGA_FP32)
        return gdt == EAGA_FP32 ? launch_all<StepLaunch<float, float, BITS, false>>(s, e, count, st)
                                : launch_all<StepLaunch<float, bf, BITS, false>>(s, e, count, st);
    if (master)
        return gdt == EAGA_FP32 ? launch_all<StepLaunch<bf, float, BITS, true>>(s, e, count, st)
                                : launch_all<StepLaunch<bf, bf, BITS, true>>(s, e, count, st);
    return gdt == EAGA_FP32 ? launch_all<StepLaunch<bf, float, BITS, false>>(s, e, count, st)
                            : launch_all<StepLaunch<bf, bf, BITS, false>>(s, e, count, st);
}

// A buffer of the call: its range, and whether it is written.
struct Range {
    uintptr_t lo, hi;
    bool out;
};

// EAGA_ERR_INVALID_ARG if a written range overlaps another one.  Lists whose
// buffers each lie in ascending order in a region of their own (parameters,
// gradients and states in flat buffers) are cleared in one pass; others are sorted.
static eaga_status check_ranges(Range *r, int n, int kinds) {
    bool plain = true;
    uintptr_t lo[8], hi[8];
    for (int k = 0; k < kinds && plain; ++k) {
        lo[k] = hi[k] = 0;
        for (int i = k; i < n; i += kinds) {
            if (r[i].lo == r[i].hi) continue;
            if (!hi[k]) lo[k] = r[i].lo;
            else if (r[i].lo < hi[k]) plain = false;
            hi[k] = r[i].hi;
        }
        for (int j = 0; j < k; ++j)
            if (hi[k] && hi[j] && lo[k] < hi[j] && lo[j] < hi[k]) plain = false;
    }
    if (plain) return EAGA_OK;
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t end = 0, end_out = 0;
    for (int i = 0; i < n; ++i) {
        if (r[i].lo == r[i].hi) continue;
        if (r[i].lo < end_out || (r[i].out && r[i].lo < end)) return EAGA_ERR_INVALID_ARG;
        end = std::max(end, r[i].hi);
        if (r[i].out) end_out = std::max(end_out, r[i].hi);
    }
    return EAGA_OK;
}



// Checks the tensors and lays out their entries (the empty ones left out) in `e`; `count` becomes their number.
static eaga_status gather(const eaga_adamw_tensor *t, int &count, int bits, int pbytes, int gbytes, AdEntry *e,
                          Range *ranges) {
    int kept = 0;
    long long tiles = 0;
    for (int i = 0; i < count; ++i) {
        const eaga_adamw_tensor &a = t[i];
        if (a.n < 0) return EAGA_ERR_INVALID_ARG;
        if (a.n == 0) continue;
        if (a.n > (1LL << 40)) return EAGA_ERR_UNSUPPORTED;
        if (!(a.weight_decay >= 0.f) || !std::isfinite(a.weight_decay)) return EAGA_ERR_INVALID_ARG;
        if (!a.m || !a.v || (bits == 8 && (!a.m_scale || !a.v_scale))) return EAGA_ERR_INVALID_ARG;
        if (pbytes && (!a.p || !a.g)) return EAGA_ERR_INVALID_ARG;
        for (const void *p : {(const void *)a.p, (const void *)a.master, a.g, (const void *)a.m, (const void *)a.v})
            if (bad_align16(p)) return EAGA_ERR_MISALIGNED;
        if ((reinterpret_cast<uintptr_t>(a.m_scale) | reinterpret_cast<uintptr_t>(a.v_scale)) & 3u)
            return EAGA_ERR_MISALIGNED;
        const long long blocks = bits == 8 ? (a.n + AD_BLOCK - 1) / AD_BLOCK * 4 : 0;
        const long long sb = bits == 8 ? a.n : 4 * a.n;
        auto range = [](const void *p, long long bytes, bool out) {
            const uintptr_t b = reinterpret_cast<uintptr_t>(p);
            return Range{b, p ? b + (uintptr_t)bytes : b, out};
        };
        Range *r = ranges + 7 * kept;
        const bool step = pbytes != 0;           // unpack writes its two fp32 outputs and reads the states
        r[0] = range(a.p, a.n * (step ? pbytes : 4), true);
        r[1] = range(a.master, a.n * 4, true);
        r[2] = range(a.g, a.n * gbytes, false);
        r[3] = range(a.m, sb, step);
        r[4] = range(a.v, sb, step);
        r[5] = range(bits == 8 ? a.m_scale : nullptr, blocks, step);
        r[6] = range(bits == 8 ? a.v_scale : nullptr, blocks, step);
        e[kept++] = {a.p, a.master, a.g, a.m, a.v, a.m_scale, a.v_scale, a.n, a.counter, a.weight_decay, 0};
        tiles += (a.n + AD_TILE - 1) / AD_TILE;
        if (tiles > 0x7fffffffLL) return EAGA_ERR_UNSUPPORTED;
    }
    count = kept;
    return check_ranges(ranges, 7 * kept, 7);
}

// Host memory of one call's table; freed on every way out.
struct HostTable {
    AdEntry *e;
    Range *r;
    explicit HostTable(int count)
        : e(static_cast<AdEntry *>(malloc(sizeof(AdEntry) * (size_t)(count + 1)))),
          r(static_cast<Range *>(malloc(sizeof(Range) * 7 * (size_t)(count + 1)))) {}
    ~HostTable() {
        free(e);
        free(r);
    }
    HostTable(const HostTable &) = delete;
};

}  // namespace ops
}  // namespace eaga

using namespace eaga;
using namespace eaga::ops;

extern "C" {

eaga_status eaga_adamw_step(const eaga_adamw_config *c, const eaga_adamw_tensor *t, int count, void *state,
                            const float *lr, void *stream) {
    if (!c || count < 0 || (count && !t) || !state) return EAGA_ERR_INVALID_ARG;
    if (count > (1 << 20)) return EAGA_ERR_UNSUPPORTED;
    if (bad_align16(state)) return EAGA_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(lr) & 3u) return EAGA_ERR_MISALIGNED;
    if (c->state_bits != 8 && c->state_bits != 32) return EAGA_ERR_INVALID_ARG;
    for (int dt : {c->param_dtype, c->grad_dtype})
        if (dt != EAGA_FP32 && dt != EAGA_BF16) return EAGA_ERR_INVALID_ARG;
    for (double x : {c->lr, c->beta1, c->beta2, c->eps, c->grad_scale})
        if (!std::isfinite(x)) return EAGA_ERR_INVALID_ARG;
    if (c->beta1 < 0 || c->beta1 >= 1 || c->beta2 < 0 || c->beta2 >= 1 || c->eps <= 0 || c->lr < 0)
        return EAGA_ERR_INVALID_ARG;
    // a master copy for every tensor or for none, and for bf16 weights only
    bool master = false, first = true;
    for (int i = 0; i < count; ++i) {
        if (t[i].n <= 0) continue;
        const bool has = t[i].master != nullptr;
        if ((first ? false : has != master) || (has && c->param_dtype == EAGA_FP32)) return EAGA_ERR_INVALID_ARG;
        master = has;
        first = false;
    }
    HostTable h(count);
    if (!h.e || !h.r) return EAGA_ERR_UNSUPPORTED;
    const int pb = c->param_dtype == EAGA_FP32 ? 4 : 2, gb = c->grad_dtype == EAGA_FP32 ? 4 : 2;
    if (eaga_status s = gather(t, count, c->state_bits, pb, gb, h.e, h.r); s != EAGA_OK) return s;
    AdScalars a = {};
    a.lr = c->lr; a.beta1 = c->beta1; a.beta2 = c->beta2;
    a.b1 = (float)c->beta1; a.omb1 = (float)(1.0 - c->beta1);
    a.b2 = (float)c->beta2; a.omb2 = (float)(1.0 - c->beta2);
    a.eps = (float)c->eps; a.gscale = (float)c->grad_scale;
    a.lr_dev = lr;
    a.state = static_cast<long long *>(state);
    a.seed = c->seed;
    a.advance = 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = c->state_bits == 8
                                ? launch_step<8>(c->param_dtype, c->grad_dtype, master, a, h.e, count, st)
                                : launch_step<32>(c->param_dtype, c->grad_dtype, master, a, h.e, count, st);
    return err == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

eaga_status eaga_adamw_unpack(const eaga_adamw_tensor *t, int count, void *stream) {
    if (count < 0 || (count && !t)) return EAGA_ERR_INVALID_ARG;
    if (count > (1 << 20)) return EAGA_ERR_UNSUPPORTED;
    HostTable h(count);
    if (!h.e || !h.r) return EAGA_ERR_UNSUPPORTED;
    if (eaga_status s = gather(t, count, 8, 0, 0, h.e, h.r); s != EAGA_OK) return s;
    if (!count) return EAGA_OK;
    AdScalars a = {};
    const cudaError_t err = launch_all<UnpackLaunch>(a, h.e, count, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

}  // extern "C"
