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
// Bound: HBM with 32-bit states, the instructions it issues with 8-bit ones.  A bf16 weight with its fp32 master, an fp32 gradient and fp32
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
    float b1, omb1, b2, omb2, eps, gscale, one;
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

// Codes' values, 8 at a time: the code's bits as a float, up, times the scale.
__device__ __forceinline__ void decode(uint2 c, float scale, int shift, unsigned mask, f2 (&v)[4]) {
    const f2 up = both(CODE_UP), sc = both(scale);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = pair(__uint_as_float((code_at(c, 2 * j) & mask) << shift), __uint_as_float((code_at(c, 2 * j + 1) & mask) << shift)) * up * sc;
}
__device__ __forceinline__ void decode_m(uint2 c, float scale, f2 (&v)[4]) {
    decode(c, scale, 20, 127u, v);
#pragma unroll
    for (int j = 0; j < 4; ++j)                      // the sign, bit 7 of the code
        v[j].b ^= ((unsigned long long)(code_at(c, 2 * j + 1) & 128u) << 56) | ((code_at(c, 2 * j) & 128u) << 24);
}
__device__ __forceinline__ void decode_v(uint2 c, float scale, f2 (&v)[4]) {
    decode(c, scale, 19, 255u, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * v[j];
}
// The warp's largest of values without a sign; a NaN is larger than everything and stays.
__device__ __forceinline__ float warp_max(const f2 (&v)[4]) {
    unsigned a = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) a = max(a, max(__float_as_uint(lo(v[j])) & 0x7fffffffu, __float_as_uint(hi(v[j])) & 0x7fffffffu));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, a));
}
// The quotients a / scale, rounded to nearest, times 2^-112: their bits.  A block has one divisor, so the division is a
// multiplication by its rounded reciprocal y and two corrections with the exact remainder, q + (a - scale q) y: the first makes q
// one of the two floats around the quotient, the second (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) the nearest.  The remainder is exact for a scale within 2^+-60 and an `a` above 2^-102, and a smaller `a` has
// code 0 for such a scale; other scales, NaN among them, are divided by in full.
__device__ __forceinline__ void scaled_bits(const f2 (&a)[4], float scale, float y, bool zero, unsigned (&bits)[8]) {
    const f2 down = both(CODE_DOWN);
    if (scale > 0x1p-60f && scale < 0x1p60f) {
        const f2 yy = both(y), ms = both(-scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f2 q = a[j] * yy;
            q = fma2(fma2(ms, q, a[j]), yy, q);
            q = fma2(fma2(ms, q, a[j]), yy, q) * down;
            bits[2 * j] = __float_as_uint(lo(q));
            bits[2 * j + 1] = __float_as_uint(hi(q));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bits[2 * j] = zero ? 0u : __float_as_uint(__fmul_rn(__fdiv_rn(lo(a[j]), scale), CODE_DOWN));
            bits[2 * j + 1] = zero ? 0u : __float_as_uint(__fmul_rn(__fdiv_rn(hi(a[j]), scale), CODE_DOWN));
        }
    }
}
__device__ __forceinline__ f2 abs2(f2 a) { return f2{a.b & 0x7fffffff7fffffffull}; }
__device__ __forceinline__ void pairs(const float (&v)[8], f2 (&o)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pair(v[2 * j], v[2 * j + 1]);
}
__device__ __forceinline__ void singles(const f2 (&v)[4], float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        o[2 * j] = lo(v[j]);
        o[2 * j + 1] = hi(v[j]);
    }
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
        int at = 0, past = s.count;                    // the last entry whose first tile is at most `tile`
        while (past - at > 1) {
            const int mid = (at + past) >> 1;
            if (tab.e[mid].first <= tile) at = mid;
            else past = mid;
        }
        const AdEntry &e = tab.e[at];
        const long long w0 = (long long)(tile - e.first) * AD_TILE + warp * AD_WARP, i0 = w0 + 8 * lane;
        if (w0 >= e.n) continue;                      // whole warps only
        const int k = (int)max(0LL, min(8LL, e.n - i0));
        float x[8];
        f2 g[4], p[4], m[4], v[4];
        load8(static_cast<const GT *>(e.g) + i0, k, x);
        pairs(x, g);
        if constexpr (MASTER) load8(e.master + i0, k, x);
        else load8(static_cast<const PT *>(e.p) + i0, k, x);
        pairs(x, p);
        const long long blk = w0 / AD_BLOCK;
        if constexpr (BITS == 32) {
            load8(static_cast<const float *>(e.m) + i0, k, x);
            pairs(x, m);
            load8(static_cast<const float *>(e.v) + i0, k, x);
            pairs(x, v);
        } else {
            const uint2 cm = load_codes(static_cast<const uint8_t *>(e.m) + i0, k);
            const uint2 cv = load_codes(static_cast<const uint8_t *>(e.v) + i0, k);
            decode_m(cm, e.ms[blk], m);
            decode_v(cv, e.vs[blk], v);
        }
        const f2 keep = both((float)__dsub_rn(1.0, __dmul_rn(sh_lr, (double)e.wd)));
        const f2 b1 = both(s.b1), omb1 = both(s.omb1), b2 = both(s.b2), omb2 = both(s.omb2), gs = both(s.gscale);
        // a sum behind a product: by a one that the compiler does not know, or it makes a fused one of the two
        const f2 one = both(s.one);
        const f2 iv = both(inv), ep = both(s.eps), msize = both(-size);
        f2 r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 gu = g[j] * gs;
            m[j] = fma2(m[j] * b1, one, gu * omb1);
            v[j] = fma2(v[j] * b2, one, (gu * gu) * omb2);
            r[j] = pair(__fsqrt_rn(lo(v[j])), __fsqrt_rn(hi(v[j])));
            const f2 d = fma2(r[j] * iv, one, ep);
            p[j] = fma2(p[j] * keep, one, pair(__fdiv_rn(lo(m[j]), lo(d)), __fdiv_rn(hi(m[j]), hi(d))) * msize);
        }
        singles(p, x);
        if constexpr (MASTER) store8(e.master + i0, k, x);
        store8(static_cast<PT *>(e.p) + i0, k, x);
        if constexpr (BITS == 32) {
            singles(m, x);
            store8(static_cast<float *>(e.m) + i0, k, x);
            singles(v, x);
            store8(static_cast<float *>(e.v) + i0, k, x);
        } else {
            if (k < 8) {                              // past the tensor's end: nothing
                float y[8];
                singles(m, x);
                singles(r, y);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (u >= k) x[u] = y[u] = 0.f;
                pairs(x, m);
                pairs(y, r);
            }
            f2 am[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) am[j] = abs2(m[j]);
            const float tm = warp_max(am), tr = warp_max(r);
            const float sm = __fdiv_rn(tm, M_TOP), sr = __fdiv_rn(tr, R_TOP);
            unsigned bm[8], br[8];
            scaled_bits(am, sm, __frcp_rn(sm), tm == 0.f, bm);
            scaled_bits(r, sr, __frcp_rn(sr), tr == 0.f, br);
            singles(m, x);
            uint2 cm = make_uint2(0, 0), cr = make_uint2(0, 0);
            const unsigned c0 = (unsigned)(e.counter + (unsigned long long)i0) + sh_key;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const unsigned h = mix32(c0 + u);
                const unsigned h2 = h * 0x3C6EF35Fu;
                unsigned a = min(127u, (bm[u] + (h >> 12)) >> 20);
                if (x[u] < 0.f) a |= 128u;
                unsigned b = min(255u, (br[u] + (h2 >> 13)) >> 19);
                if ((u & 1 ? hi(r[u / 2]) : lo(r[u / 2])) > 0.f) b = max(b, 1u);
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
        int at = 0, past = s.count;
        while (past - at > 1) {
            const int mid = (at + past) >> 1;
            if (tab.e[mid].first <= tile) at = mid;
            else past = mid;
        }
        const AdEntry &e = tab.e[at];
        const long long w0 = (long long)(tile - e.first) * AD_TILE + warp * AD_WARP, i0 = w0 + 8 * lane;
        if (w0 >= e.n) continue;
        const int k = (int)max(0LL, min(8LL, e.n - i0));
        const uint2 cm = load_codes(static_cast<const uint8_t *>(e.m) + i0, k);
        const uint2 cv = load_codes(static_cast<const uint8_t *>(e.v) + i0, k);
        f2 v[4];
        float x[8];
        if (e.p) {
            decode_m(cm, e.ms[w0 / AD_BLOCK], v);
            singles(v, x);
            store8(static_cast<float *>(e.p) + i0, k, x);
        }
        if (e.master) {
            decode_v(cv, e.vs[w0 / AD_BLOCK], v);
            singles(v, x);
            store8(e.master + i0, k, x);
        }
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
// `more`: two buffers beside the lists, for which `r` has room behind its n.
static eaga_status check_ranges(Range *r, int n, int kinds, const Range (&more)[2]) {
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
        for (const Range &m : more)
            if (hi[k] && lo[k] < m.hi && m.lo < hi[k]) plain = false;
    }
    if (more[0].lo < more[1].hi && more[1].lo < more[0].hi) return EAGA_ERR_INVALID_ARG;
    if (plain) return EAGA_OK;
    for (const Range &m : more) r[n++] = m;
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

static Range range_of(const void *p, long long bytes, bool out) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return Range{b, p ? b + (uintptr_t)bytes : b, out};
}

// Checks the tensors and lays out their entries (the empty ones left out) in `e`; `count` becomes their number.
// state, lr: a step's, else null.
static eaga_status gather(const eaga_adamw_tensor *t, int &count, int bits, int pbytes, int gbytes, const void *state, const void *lr,
                          AdEntry *e, Range *ranges) {
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
        Range *r = ranges + 7 * kept;
        const bool step = pbytes != 0;           // unpack writes its two fp32 outputs and reads the states
        r[0] = range_of(a.p, a.n * (step ? pbytes : 4), true);
        r[1] = range_of(a.master, a.n * 4, true);
        r[2] = range_of(a.g, a.n * gbytes, false);
        r[3] = range_of(a.m, sb, step);
        r[4] = range_of(a.v, sb, step);
        r[5] = range_of(bits == 8 ? a.m_scale : nullptr, blocks, step);
        r[6] = range_of(bits == 8 ? a.v_scale : nullptr, blocks, step);
        e[kept++] = {a.p, a.master, a.g, a.m, a.v, a.m_scale, a.v_scale, a.n, a.counter, a.weight_decay, 0};
        tiles += (a.n + AD_TILE - 1) / AD_TILE;
        if (tiles > 0x7fffffffLL) return EAGA_ERR_UNSUPPORTED;
    }
    count = kept;
    return check_ranges(ranges, 7 * kept, 7, {range_of(state, 16, true), range_of(lr, 4, false)});
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
    if (c->beta1 < 0 || c->beta1 >= 1 || c->beta2 < 0 || c->beta2 >= 1 || c->lr < 0) return EAGA_ERR_INVALID_ARG;
    // as the kernels use them: an eps that is 0 in fp32 would make 0 / 0 of an element without a gradient
    if (!((float)c->eps > 0.f) || !std::isfinite((float)c->eps) || !std::isfinite((float)c->grad_scale) || !std::isfinite((float)c->lr))
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
    if (eaga_status s = gather(t, count, c->state_bits, pb, gb, state, lr, h.e, h.r); s != EAGA_OK) return s;
    AdScalars a = {};
    a.lr = c->lr; a.beta1 = c->beta1; a.beta2 = c->beta2;
    a.b1 = (float)c->beta1; a.omb1 = (float)(1.0 - c->beta1);
    a.b2 = (float)c->beta2; a.omb2 = (float)(1.0 - c->beta2);
    a.one = 1.f;
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
    if (eaga_status s = gather(t, count, 8, 0, 0, nullptr, nullptr, h.e, h.r); s != EAGA_OK) return s;
    if (!count) return EAGA_OK;
    AdScalars a = {};
    const cudaError_t err = launch_all<UnpackLaunch>(a, h.e, count, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

}  // extern "C"
