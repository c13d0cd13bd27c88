// The linear operator (eaga_linear_forward / _backward):
//
//   Z = X W + b        Y = act(Z) + R
//   dZ = act'(Z) dY    dX = act_in'(Zin) (dZ W^T) + dR    dW = X^T dZ    db = sum of dZ's rows
//
// A few rows run in ops_linear_vec.cu, bound by the read of W; more on the
// tensor cores (ops_linear_tc.cu).  Those read bf16 operands by TMA, whose rows
// begin on 16 bytes (narrow fp32 products stay on the
// CUDA cores, ops_linear_f32.cu).  What is not so is prepared once in the workspace, by one
// kernel for all operands: rows of another length are copied into padded ones;
// fp32 values (operands in fp32, and dZ where act is not none) become three bf16
// parts that carry their 24 bits between them.  An fp32 result takes the products
// of all parts that count (six of nine), dX in bf16 the upper two parts of dZ (16
// bits: the rest is 2^-8 of the result's own rounding).
#include <algorithm>
#include <cstdio>
#include "ops_linear.h"

namespace eaga {
namespace ops {

// One operand to prepare: src [rows][n], times act'(z) where z is given, as `parts` bf16 parts [rows][ld]
// (zero past n).
struct PrepJob {
    const void *src, *z;
    void *dst[3];
    float *f32;                // or this: fp32 [rows][n]
    long long rows;
    int n, ld, act, parts;
};
struct PrepArgs {
    PrepJob job[3];
};

// A value's bf16 part number k (0, 1, 2, in turn), and what it leaves in v.  Of an infinity or a NaN nothing is left: the first part says
// it all.  A finite value above bf16's largest gives that, and where the first part is that one, the second is cut off, not rounded: no sum
// of parts is larger than the value, so the type's lowest value, with which masks are filled, times one stays finite.  (The third is exact.)
__device__ __forceinline__ float take_part(float &v, int k, float &first) {
    float hi = __bfloat162float(__float2bfloat16_rn(v));
    const float cut = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    if (k == 0) {
        if (isinf(hi)) hi = cut;
        v = isfinite(hi) ? v - hi : 0.f;
        first = fabsf(hi);
    } else {
        if (k == 1 && first == __uint_as_float(0x7f7f0000u)) hi = cut;
        v -= hi;
    }
    return hi;
}

// The 8 values from `at` on of a flat array of `total`, whatever their alignment: the two aligned 16 bytes (bf16; fp32 three)
// that hold them, shifted into place.  Near the array's end single loads.
template <typename T>
__device__ __forceinline__ void flat_ld8(const T *p, long long at, long long total, int have, float (&v)[8]) {
    constexpr int PER = 16 / sizeof(T), N = 8 / PER + 1;
    const int s = (int)(at % PER);
    const long long first = at / PER;
    const int need = s ? N : N - 1;
    if ((first + need) * PER > total) {
        lin_ld8(p + at, have, false, v);
        return;
    }
    unsigned w[4 * N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint4 a = n < need ? reinterpret_cast<const uint4 *>(p)[first + n] : make_uint4(0, 0, 0, 0);
        w[4 * n] = a.x; w[4 * n + 1] = a.y; w[4 * n + 2] = a.z; w[4 * n + 3] = a.w;
    }
    const int words = s * (int)sizeof(T) / 4;        // 0 .. 3
#pragma unroll
    for (int k = 0; k < 4 * N; ++k)
        if (words & 2) w[k] = k + 2 < 4 * N ? w[k + 2] : 0u;
#pragma unroll
    for (int k = 0; k < 4 * N; ++k)
        if (words & 1) w[k] = k + 1 < 4 * N ? w[k + 1] : 0u;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < have ? __uint_as_float(w[k]) : 0.f;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned x = s & 1 ? __funnelshift_r(w[k], w[k + 1], 16) : w[k];
            v[2 * k] = 2 * k < have ? __uint_as_float(x << 16) : 0.f;
            v[2 * k + 1] = 2 * k + 1 < have ? __uint_as_float(x & 0xffff0000u) : 0.f;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_lin_prep(const __grid_constant__ PrepArgs a) {
    after_previous();
    const PrepJob &j = a.job[blockIdx.y];
    const unsigned per = j.ld / 8;
    const T *src = static_cast<const T *>(j.src), *zs = static_cast<const T *>(j.z);
    const long long total = j.rows * per, step = (long long)gridDim.x * 256, all = j.rows * j.n;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += step) {
        const long long row = total <= 0xffffffffLL ? (unsigned)i / per : i / per;
        const int c = (int)(i - row * per) * 8, have = min(8, j.n - c);
        float v[8], z[8];
        flat_ld8(src, row * j.n + c, all, have, v);
        if (zs) {
            flat_ld8(zs, row * j.n + c, all, have, z);
            act_slope_mul<T>(v, z, j.act);
        }
        if (j.f32) lin_st8(j.f32 + row * j.n + c, have, j.n % 4 == 0, v);
        float first[8];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k >= j.parts) break;
            float o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = take_part(v[u], k, first[u]);
            lin_st8(static_cast<__nv_bfloat16 *>(j.dst[k]) + (size_t)row * j.ld + c, 8, true, o);
        }
    }
    before_next();
}

// The epilogue of a split forward or dX product, from the splits' sums in their order; VEC columns a thread.
template <typename T, int KIND, int VEC>
__global__ void __launch_bounds__(256) k_lin_join(const float *acc, int splits, long long M, int N, const LinEpi<T> e) {
    after_previous();
    const long long total = M * N, i = (blockIdx.x * 256LL + threadIdx.x) * VEC;
    if (i >= total) return;
    float y[8] = {}, o[8] = {};
    for (int s = 0; s < splits; ++s) {
        lin_ld8(acc + s * total + i, VEC, VEC > 1, o);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] += o[j];
    }
    if constexpr (KIND == LIN_FWD) {
        if (e.bias) {
            lin_ld8(e.bias + i % N, VEC, VEC > 1, o);
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] += o[j];
        }
        if (e.out2) lin_st8(e.out2 + i, VEC, VEC > 1, y);
        act_apply<T>(y, e.act);
    } else if (e.zin) {
        lin_ld8(e.zin + i, VEC, VEC > 1, o);
        act_slope_mul<T>(y, o, e.act);
    }
    if (e.add) {
        lin_ld8(e.add + i, VEC, VEC > 1, o);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] += o[j];
    }
    lin_st8(e.out + i, VEC, VEC > 1, y);
}

// dW and db from the splits' sums, in their order: a warp sums every eighth split of 32 VEC values, the CTA
// adds its eight warps' sums.
template <int VEC>
__global__ void __launch_bounds__(256)
k_lin_reduce(const float *acc, float *dW, long long n, int splits, const float *bacc, float *db, int out, int bparts, unsigned wblocks) {
    after_previous();
    __shared__ float sum[8][32 * VEC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool is_w = blockIdx.x < wblocks;
    const float *src = is_w ? acc : bacc;
    float *dst = is_w ? dW : db;
    const long long len = is_w ? n : out;
    const int parts = is_w ? splits : bparts;
    const long long i = ((is_w ? blockIdx.x : blockIdx.x - wblocks) * 32LL + lane) * VEC;
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k] = 0.f;
    if (i < len) {
#pragma unroll 8
        for (int r = warp; r < parts; r += 8) {
            if constexpr (VEC == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src + r * len + i);
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            } else {
                s[0] += src[r * len + i];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) sum[warp][lane * VEC + k] = s[k];
    __syncthreads();
    const int c = threadIdx.x;
    const long long o = (is_w ? blockIdx.x : blockIdx.x - wblocks) * 32LL * VEC + c;
    if (c < 32 * VEC && o < len) {
        float t = 0.f;
#pragma unroll
        for (int v = 0; v < 8; ++v) t += sum[v][c];
        dst[o] = t;
    }
}

// ------------------------------------------------------------------ host side

static int round8(int n) { return (n + 7) / 8 * 8; }

struct LinPlan {
    bool vec, cores;                   // few rows; fp32 on the CUDA cores
    int xparts, wparts, zparts;        // parts in the workspace; 0: the caller's tensor is read as it is
    int ldx, ldw, ldz;
    LinSplit fwd, dx, dw;
    int bparts;                        // of the bias gradient
    size_t X[3], W[3], dZ[3], dZ32, acc, bacc, total;      // workspace offsets
};

// The products of parts of an fp32 or a bf16 result: A's parts times B's, without those below 2^-24.
static int products(int aparts, int bparts, uint8_t (&seg)[6]) {
    int n = 0;
    for (int sum = 2; sum >= 0; --sum)               // the smallest first
        for (int a = 0; a < aparts; ++a)
            if (const int b = sum - a; b >= 0 && b < bparts) seg[n++] = (uint8_t)(a | b << 2);
    return n;
}

// Whether an fp32 call runs on the CUDA cores: by estimates of both, in us.  Those reach 22 TFLOP/s on wide
// results, 13 and 17 on tiles of 16 and 32 columns, 15 in narrow weight gradients (0.7 us for 16 steps of the reduction at the least); the tensor cores' operands are first copied into parts, 10 bytes an element.
// 1033088 x 8 -> 8 took 466 us on the tensor cores.
static double cores_us(long long M, int N, long long K) {
    if (lin_narrow(M, N, K))                         // by warps: 8 us for 2500 steps at the least
        return std::max(2.0 * M * ((N + 7) / 8 * 8) * (K + 80) / 17e6, K * 0.0035) + 4;
    const double n = N <= 16 ? 16 : (N + 31) / 32 * 32, flops = 2.0 * M * n * K, bytes = 4.0 * ((double)M * K + 2.0 * (double)M * N + (double)K * N);
    return std::max({flops / lin_tile_rate(N), bytes / 4.5e6, K / 16 * 0.7}) + 4;
}
static bool lin_cores(const eaga_linear_dims &d, bool back) {
    const double x = (double)d.rows * d.in, w = (double)d.in * d.out, z = (double)d.rows * d.out;
    double tc = 0, us = 0;
    if (!back) {
        lin_tc_split(d.rows, d.out, d.in, 6, true, &us);
        if (d.out <= 32) us *= 2;                    // lines of Y of 128 bytes or less: 200000 x 64 -> 24 91 us without the copies, 84 by warps
        return cores_us(d.rows, d.out, d.in) < us + 10 * (x + w) / 5e6 + 3;
    }
    lin_tc_split(d.rows, d.in, d.out, 6, true, &us);
    tc = us;
    lin_tc_split(d.in, d.out, d.rows, 6, false, &us);
    if (d.out <= 32) us *= 2.5;                      // rows of dZ of a few bytes load as slowly as long ones (300000 x 100 <- 8)
    tc += us + 10 * (x + w + z) / 5e6 + 3;
    // dW: splits of the rows, none shorter than 256
    const double dw = std::max(2.0 * d.rows * ((d.in + 31) / 32 * 32) * ((d.out + 31) / 32 * 32) / (d.in <= 32 || d.out <= 32 ? 15e6 : 22e6), 4 * (x + z) / 4.5e6) + 13;
    return cores_us(d.rows, d.in, d.out) + dw < tc;
}

static LinPlan lin_plan(const eaga_linear_dims &d, bool back) {
    LinPlan p = {};
    p.vec = lin_few_rows(d, back);
    size_t off = 256;                                // the status word
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    if (!p.vec && d.dtype == EAGA_FP32 && lin_cores(d, back)) {
        p.cores = true;
        if (back) {
            if (d.act != EAGA_ACT_NONE) p.dZ32 = take((size_t)d.rows * d.out * 4);
            p.dw = lin_f32_dw_split(d.rows, d.in, d.out);
            p.bparts = p.dw.splits;
            if (p.dw.splits > 1) {
                p.acc = take((size_t)p.dw.splits * d.in * d.out * 4);
                p.bacc = take((size_t)p.dw.splits * d.out * 4);
            }
        }
    } else if (!p.vec) {
        const size_t rows = (size_t)d.rows, in = d.in, out = d.out;
        const bool f32 = d.dtype == EAGA_FP32, dact = back && d.act != EAGA_ACT_NONE;
        p.ldx = round8(d.in);
        p.ldw = p.ldz = round8(d.out);
        p.xparts = f32 ? 3 : p.ldx != d.in ? 1 : 0;
        p.wparts = f32 ? 3 : p.ldw != d.out ? 1 : 0;
        p.zparts = !back ? 0 : f32 || dact ? 3 : p.ldz != d.out ? 1 : 0;
        for (int k = 0; k < p.xparts; ++k) p.X[k] = take(rows * p.ldx * 2);
        for (int k = 0; k < p.wparts; ++k) p.W[k] = take(in * p.ldw * 2);
        for (int k = 0; k < p.zparts; ++k) p.dZ[k] = take(rows * p.ldz * 2);
        uint8_t seg[6];
        size_t acc = 0;
        if (!back) {
            p.fwd = lin_tc_split(d.rows, d.out, d.in, f32 ? 6 : 1, f32);
            acc = p.fwd.splits > 1 ? p.fwd.splits * rows * out : 0;
        } else {
            const int z = std::max(1, p.zparts);
            p.dx = lin_tc_split(d.rows, d.in, d.out, f32 ? 6 : std::min(z, 2), f32);
            p.dw = lin_tc_split(d.in, d.out, d.rows, products(f32 ? 3 : 1, z, seg), false);
            acc = std::max(p.dx.splits > 1 ? p.dx.splits * rows * in : 0, p.dw.splits > 1 ? p.dw.splits * in * out : 0);
            p.bparts = lin_db_parts(p.dw, d.in);
        }
        if (acc) p.acc = take(acc * 4);
        if (p.bparts > 1) p.bacc = take(p.bparts * out * 4);
    }
    p.total = off;
    return p;
}

static eaga_status lin_check(const eaga_linear_dims *d) {
    if (!d || d->rows < 0 || d->in < 1 || d->out < 1) return EAGA_ERR_INVALID_ARG;
    if (d->dtype != EAGA_FP32 && d->dtype != EAGA_BF16) return EAGA_ERR_INVALID_ARG;
    if (d->act < EAGA_ACT_NONE || d->act > EAGA_ACT_SILU) return EAGA_ERR_INVALID_ARG;
    if (d->in > 65536 || d->out > 65536 || d->rows > 0x7fff0000LL) return EAGA_ERR_UNSUPPORTED;
    return EAGA_OK;
}

template <typename T>
static cudaError_t lin_prep(const PrepJob *jobs, int n, cudaStream_t st) {
    if (!n) return cudaSuccess;
    PrepArgs a = {};
    long long most = 0;
    for (int k = 0; k < n; ++k) {
        a.job[k] = jobs[k];
        most = std::max(most, (jobs[k].rows * (jobs[k].ld / 8) + 255) / 256);
    }
    const unsigned grid = (unsigned)std::max(1LL, std::min(most, 16LL * sm_count()));
    return launch_pdl(k_lin_prep<T>, dim3(grid, n), dim3(256), 0, st, 1, a);
}

// Whichever of the two sums is in more than one part.
static cudaError_t lin_reduce(long long n, int splits, const float *acc, float *dW, int out, int bparts, const float *bacc, float *db,
                              cudaStream_t st) {
    const bool v4 = n % 4 == 0 && out % 4 == 0;
    const long long per = v4 ? 128 : 32;
    const unsigned wb = splits > 1 ? (unsigned)((n + per - 1) / per) : 0, bb = db && bparts > 1 ? (unsigned)((out + per - 1) / per) : 0;
    if (!(wb + bb)) return cudaSuccess;
    return launch_pdl(v4 ? k_lin_reduce<4> : k_lin_reduce<1>, dim3(wb + bb), dim3(256), 0, st, 1, acc, dW, n, splits, bacc, db, out, bparts, wb);
}

static Span span(const void *q, size_t b) { return Span{q, q ? b : 0}; }

template <int KIND, typename T>
static cudaError_t lin_join(const LinSplit &s, const float *acc, long long M, int N, const LinEpi<T> &e, cudaStream_t st) {
    const bool v = N % 8 == 0;
    const long long blocks = (M * N + (v ? 2047 : 255)) / (v ? 2048 : 256);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(v ? k_lin_join<T, KIND, 8> : k_lin_join<T, KIND, 1>, dim3((unsigned)blocks), dim3(256), 0, st, 1, acc, s.splits, M, N, e);
}

struct LinBack {
    const void *X, *W, *Z, *dY;
    int act_in;
    const void *Zin, *dR;
    void *dX;
    float *dW, *db;
    char *ws;
};

// An operand's parts: the caller's tensor, or prepared ones (then with a job).
static void lin_operand(const __nv_bfloat16 *(&part)[3], const void *src, const void *z, int act, long long rows, int n, int ld, int parts,
                        const size_t (&at)[3], char *ws, PrepJob *jobs, int &count) {
    part[0] = static_cast<const __nv_bfloat16 *>(src);
    if (!parts) return;
    PrepJob j = {src, z, {}, nullptr, rows, n, ld, act, parts};
    for (int k = 0; k < parts; ++k) {
        j.dst[k] = ws + at[k];
        part[k] = reinterpret_cast<const __nv_bfloat16 *>(ws + at[k]);
    }
    jobs[count++] = j;
}

static LinTc lin_tc(const eaga_linear_dims &d, const LinPlan &p, char *ws) {
    LinTc q = {};
    q.rows = d.rows; q.in = d.in; q.out = d.out;
    q.ldx = p.ldx; q.ldw = p.ldw; q.ldz = p.ldz;
    q.status = reinterpret_cast<int *>(ws);
    q.clear = true;
    return q;
}

template <typename T>
static cudaError_t forward_tc(const eaga_linear_dims &d, const LinPlan &p, const void *X, const void *W, const LinEpi<T> &e, char *ws,
                              cudaStream_t st) {
    PrepJob jobs[2];
    int n = 0;
    LinTc q = lin_tc(d, p, ws);
    lin_operand(q.X, X, nullptr, 0, d.rows, d.in, p.ldx, p.xparts, p.X, ws, jobs, n);
    lin_operand(q.W, W, nullptr, 0, d.in, d.out, p.ldw, p.wparts, p.W, ws, jobs, n);
    if (cudaError_t err = lin_prep<T>(jobs, n, st); err != cudaSuccess) return err;
    const bool f32 = d.dtype == EAGA_FP32;
    q.nseg = products(f32 ? 3 : 1, f32 ? 3 : 1, q.seg);
    if (p.fwd.splits == 1) return lin_tc_forward<T>(q, p.fwd, e, st);
    LinEpi<float> sums = {};
    sums.out = reinterpret_cast<float *>(ws + p.acc);
    if (cudaError_t err = lin_tc_forward<float>(q, p.fwd, sums, st); err != cudaSuccess) return err;
    return lin_join<LIN_FWD, T>(p.fwd, sums.out, d.rows, d.out, e, st);
}

template <typename T>
static cudaError_t backward_tc(const eaga_linear_dims &d, const LinPlan &p, const LinBack &b, cudaStream_t st) {
    PrepJob jobs[3];
    int n = 0;
    LinTc q = lin_tc(d, p, b.ws);
    const bool f32 = d.dtype == EAGA_FP32;
    if (b.dW) lin_operand(q.X, b.X, nullptr, 0, d.rows, d.in, p.ldx, p.xparts, p.X, b.ws, jobs, n);
    if (b.dX) lin_operand(q.W, b.W, nullptr, 0, d.in, d.out, p.ldw, p.wparts, p.W, b.ws, jobs, n);
    const int zparts = f32 || b.dW ? p.zparts : std::min(p.zparts, 2);
    lin_operand(q.dZ, b.dY, b.Z, d.act, d.rows, d.out, p.ldz, zparts, p.dZ, b.ws, jobs, n);
    if (cudaError_t e = lin_prep<T>(jobs, n, st); e != cudaSuccess) return e;
    const int z = std::max(1, zparts);
    if (b.dX) {
        q.nseg = f32 ? products(3, 3, q.seg) : products(std::min(z, 2), 1, q.seg);
        const LinEpi<T> e = {nullptr, static_cast<const T *>(b.dR), static_cast<const T *>(b.Zin), static_cast<T *>(b.dX), nullptr, b.act_in};
        if (p.dx.splits == 1) {
            if (cudaError_t err = lin_tc_dx<T>(q, p.dx, e, st); err != cudaSuccess) return err;
        } else {
            LinEpi<float> sums = {};
            sums.out = reinterpret_cast<float *>(b.ws + p.acc);
            if (cudaError_t err = lin_tc_dx<float>(q, p.dx, sums, st); err != cudaSuccess) return err;
            if (cudaError_t err = lin_join<LIN_DX, T>(p.dx, sums.out, d.rows, d.in, e, st); err != cudaSuccess) return err;
        }
        q.clear = false;
    }
    if (b.dW) {
        q.nseg = products(f32 ? 3 : 1, z, q.seg);
        float *acc = p.dw.splits > 1 ? reinterpret_cast<float *>(b.ws + p.acc) : b.dW;
        float *bacc = !b.db ? nullptr : p.bparts > 1 ? reinterpret_cast<float *>(b.ws + p.bacc) : b.db;
        if (cudaError_t err = lin_tc_dw(q, p.dw, acc, bacc, st); err != cudaSuccess) return err;
        return lin_reduce((long long)d.in * d.out, p.dw.splits, acc, b.dW, d.out, p.bparts, bacc, b.db, st);
    }
    return cudaSuccess;
}

static cudaError_t forward_cores(const eaga_linear_dims &d, const void *X, const void *W, const LinEpi<float> &e, char *ws, cudaStream_t st) {
    const LinF32 q = {d.rows, d.in, d.out, static_cast<const float *>(X), static_cast<const float *>(W), nullptr, reinterpret_cast<int *>(ws)};
    return lin_f32_forward(q, e, st);
}
static cudaError_t backward_cores(const eaga_linear_dims &d, const LinPlan &p, const LinBack &b, cudaStream_t st) {
    LinF32 q = {d.rows, d.in, d.out, static_cast<const float *>(b.X), static_cast<const float *>(b.W), static_cast<const float *>(b.dY),
                reinterpret_cast<int *>(b.ws)};
    if (p.dZ32) {
        float *dz = reinterpret_cast<float *>(b.ws + p.dZ32);
        const PrepJob j = {b.dY, b.Z, {}, dz, d.rows, d.out, round8(d.out), d.act, 0};
        if (cudaError_t e = lin_prep<float>(&j, 1, st); e != cudaSuccess) return e;
        q.dZ = dz;
    }
    if (b.dX) {
        const LinEpi<float> e = {nullptr, static_cast<const float *>(b.dR), static_cast<const float *>(b.Zin), static_cast<float *>(b.dX), nullptr, b.act_in};
        if (cudaError_t err = lin_f32_dx(q, e, st); err != cudaSuccess) return err;
    }
    if (b.dW) {
        float *acc = p.dw.splits > 1 ? reinterpret_cast<float *>(b.ws + p.acc) : b.dW;
        float *bacc = !b.db ? nullptr : p.bparts > 1 ? reinterpret_cast<float *>(b.ws + p.bacc) : b.db;
        if (cudaError_t err = lin_f32_dw(q, p.dw, acc, bacc, st); err != cudaSuccess) return err;
        return lin_reduce((long long)d.in * d.out, p.dw.splits, acc, b.dW, d.out, p.bparts, bacc, b.db, st);
    }
    return cudaSuccess;
}

template <typename T>
static cudaError_t backward_vec(const eaga_linear_dims &d, const LinBack &b, cudaStream_t st) {
    const LinVec<T> q = {(int)d.rows, d.in, d.out, static_cast<const T *>(b.X), static_cast<const T *>(b.W), static_cast<const T *>(b.dY),
                         static_cast<const T *>(b.Z), d.act, static_cast<T *>(b.dX), b.dW, b.db, reinterpret_cast<int *>(b.ws)};
    const LinEpi<T> e = {nullptr, static_cast<const T *>(b.dR), static_cast<const T *>(b.Zin), nullptr, nullptr, b.act_in};
    return lin_vec_backward<T>(q, e, st);
}

template <typename T>
static LinEpi<T> forward_epi(const eaga_linear_dims &d, const void *b, const void *R, void *Y, void *Z) {
    return {static_cast<const T *>(b), static_cast<const T *>(R), nullptr, static_cast<T *>(Y), static_cast<T *>(Z), d.act};
}
template <typename T>
static cudaError_t forward_vec(const eaga_linear_dims &d, const void *X, const void *W, const LinEpi<T> &e, void *ws, cudaStream_t st) {
    LinVec<T> q = {};
    q.rows = (int)d.rows; q.in = d.in; q.out = d.out;
    q.X = static_cast<const T *>(X); q.W = static_cast<const T *>(W);
    q.status = static_cast<int *>(ws);
    return lin_vec_forward<T>(q, e, st);
}

// The forward's, dX's or dW's kernel by name.
static int lin_form(const eaga_linear_dims &d, int kind, char *to, size_t bytes) {
    const LinPlan p = lin_plan(d, kind != LIN_FWD);
    const bool f32 = d.dtype == EAGA_FP32;
    if (p.vec) return snprintf(to, bytes, "rows %d%s", lin_vec_rows((int)d.rows), lin_vec_wide(d.out, d.dtype) ? " wide" : "");
    const long long M = kind == LIN_DW ? d.in : d.rows, K = kind == LIN_FWD ? d.in : kind == LIN_DX ? d.out : d.rows;
    const int N = kind == LIN_DX ? d.in : d.out;
    if (p.cores) {
        static const char *const names[] = {"warps 4", "warps 2", "128x16", "128x32", "64x64", "32x32", "thin"};
        const int splits = kind == LIN_DW ? p.dw.splits : 1;
        return snprintf(to, bytes, "cores %s%s", names[lin_f32_form(kind, M, N, K, splits)], splits > 1 ? " split" : "");
    }
    const LinSplit &s = kind == LIN_FWD ? p.fwd : kind == LIN_DX ? p.dx : p.dw;
    uint8_t seg[6];
    const int z = std::max(1, p.zparts), nseg = f32 ? 6 : kind == LIN_FWD ? 1 : kind == LIN_DX ? std::min(z, 2) : products(1, z, seg);
    const LtForm t = lin_tc_form(kind, s, f32 || kind == LIN_DW || s.splits > 1, M, N, K, nseg);
    const char *tile = t.tile.pair ? "pair" : t.tile.bn == 128 ? "128" : t.two ? "64 two" : "64";
    return snprintf(to, bytes, "tc %s%s%s%s", tile, t.tma ? " tma" : "", t.promo ? " promoted" : "", s.splits > 1 ? " split" : "");
}

}  // namespace ops
}  // namespace eaga

using namespace eaga;
using namespace eaga::ops;

extern "C" {

size_t eaga_linear_workspace_size(const eaga_linear_dims *d, int for_backward) {
    if (lin_check(d) != EAGA_OK) return 0;
    return lin_plan(*d, for_backward != 0).total;
}

eaga_status eaga_linear_form(const eaga_linear_dims *d, int product, char *form, size_t bytes) {
    const eaga_status s = lin_check(d);
    if (s != EAGA_OK) return s;
    if (product < LIN_FWD || product > LIN_DW || !form) return EAGA_ERR_INVALID_ARG;
    const int n = d->rows ? lin_form(*d, product, form, bytes) : snprintf(form, bytes, "none");
    return n >= 0 && (size_t)n < bytes ? EAGA_OK : EAGA_ERR_WORKSPACE;
}

eaga_status eaga_linear_forward(const eaga_linear_dims *d, const void *X, const void *W, const void *b, const void *R,
                                void *Y, void *Z, void *workspace, size_t ws_bytes, void *stream) {
    eaga_status s = lin_check(d);
    if (s != EAGA_OK) return s;
    if (!workspace) return EAGA_ERR_INVALID_ARG;
    if (d->rows > 0 && (!X || !W || !Y)) return EAGA_ERR_INVALID_ARG;
    for (const void *q : {X, W, b, R, (const void *)Y, (const void *)Z, (const void *)workspace})
        if (bad_align16(q)) return EAGA_ERR_MISALIGNED;
    const LinPlan p = lin_plan(*d, false);
    const size_t es = d->dtype == EAGA_BF16 ? 2 : 4, nx = (size_t)d->rows * d->in * es, ny = (size_t)d->rows * d->out * es;
    const Span outs[3] = {span(Y, ny), span(Z, ny), span(workspace, p.total)};
    const Span ins[4] = {span(X, nx), span(W, (size_t)d->in * d->out * es), span(b, d->out * es), span(R, ny)};
    if ((s = check_no_alias(outs, 3, ins, 4)) != EAGA_OK) return s;
    if (ws_bytes < p.total) return EAGA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (d->rows == 0) return cudaMemsetAsync(workspace, 0, 4, st) == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    typedef __nv_bfloat16 bf;
    if (d->dtype == EAGA_BF16) {
        const LinEpi<bf> epi = forward_epi<bf>(*d, b, R, Y, Z);
        e = p.vec ? forward_vec(*d, X, W, epi, workspace, st) : forward_tc(*d, p, X, W, epi, ws, st);
    } else {
        const LinEpi<float> epi = forward_epi<float>(*d, b, R, Y, Z);
        e = p.vec ? forward_vec(*d, X, W, epi, workspace, st)
                  : p.cores ? forward_cores(*d, X, W, epi, ws, st) : forward_tc(*d, p, X, W, epi, ws, st);
    }
    return e == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

eaga_status eaga_linear_backward(const eaga_linear_dims *d, const void *X, const void *W, const void *Z, const void *dY,
                                 int act_in, const void *Zin, const void *dR, void *dX, float *dW, float *db,
                                 void *workspace, size_t ws_bytes, void *stream) {
    eaga_status s = lin_check(d);
    if (s != EAGA_OK) return s;
    if (!workspace || act_in < EAGA_ACT_NONE || act_in > EAGA_ACT_SILU) return EAGA_ERR_INVALID_ARG;
    if ((!dX && !dW) || (db && !dW) || (!dX && (Zin || dR))) return EAGA_ERR_INVALID_ARG;
    if (d->act == EAGA_ACT_NONE && Z) return EAGA_ERR_INVALID_ARG;
    if (act_in == EAGA_ACT_NONE && Zin) return EAGA_ERR_INVALID_ARG;
    if (d->rows > 0) {
        if (!dY || (dW && !X) || (dX && !W) || (d->act != EAGA_ACT_NONE && !Z) || (act_in != EAGA_ACT_NONE && dX && !Zin))
            return EAGA_ERR_INVALID_ARG;
    }
    for (const void *q : {X, W, Z, dY, Zin, dR, (const void *)dX, (const void *)dW, (const void *)db, (const void *)workspace})
        if (bad_align16(q)) return EAGA_ERR_MISALIGNED;
    const LinPlan p = lin_plan(*d, true);
    const size_t es = d->dtype == EAGA_BF16 ? 2 : 4, nx = (size_t)d->rows * d->in * es, ny = (size_t)d->rows * d->out * es;
    const size_t nw = (size_t)d->in * d->out;
    const Span outs[4] = {span(dX, nx), span(dW, nw * 4), span(db, (size_t)d->out * 4), span(workspace, p.total)};
    const Span ins[6] = {span(X, nx), span(W, nw * es), span(Z, ny), span(dY, ny), span(Zin, nx), span(dR, nx)};
    if ((s = check_no_alias(outs, 4, ins, 6)) != EAGA_OK) return s;
    if (ws_bytes < p.total) return EAGA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (d->rows == 0) {
        e = cudaMemsetAsync(workspace, 0, 4, st);
        if (e == cudaSuccess && dW) e = cudaMemsetAsync(dW, 0, nw * 4, st);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)d->out * 4, st);
        return e == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
    }
    const LinBack b = {X, W, Z, dY, act_in, Zin, dR, dX, dW, db, static_cast<char *>(workspace)};
    if (d->dtype == EAGA_BF16) e = p.vec ? backward_vec<__nv_bfloat16>(*d, b, st) : backward_tc<__nv_bfloat16>(*d, p, b, st);
    else e = p.vec ? backward_vec<float>(*d, b, st) : p.cores ? backward_cores(*d, p, b, st) : backward_tc<float>(*d, p, b, st);
    return e == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

}  // extern "C"
