// The linear operator's products: C = A B with a fused epilogue (ops_linear.cu, _tc.cu, _vec.cu, _f32.cu).
#pragma once
#include <cuda_runtime.h>
#include "ops.h"

namespace eaga {
namespace ops {

// Which product: forward Y = f(X W), input gradient dX = f(dZ W^T), weight gradient dW = X^T dZ.
enum LinKind { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

// Activations, for the epilogues: an exact division or erff an element costs more issue slots than a short
// product's whole tile (138936 x 64 -> 128: 13 us without, 45 us with silu by division, 36 us with gelu by erff).
// sigmoid(z) = 1 / (1 + 2^(-z log2 e)) from the hardware's reciprocal and power of two, each within 2 steps of fp32:
// z sigmoid(z) is off by less than 8 steps of |z| + |z sigmoid(z)|, as by division.
// Phi(z) = (1 + erf(z / sqrt 2)) / 2 from Abramowitz and Stegun 7.1.26: with t = 1 / (1 + 0.3275911 x), x = |z| / sqrt 2,
// erfc(x) = t (a1 + t (a2 + .. t a5)) e^(-x^2), within 1.5e-7, half of it here; the exponential is the slope's, too.
__device__ __forceinline__ float pow2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid(float z) { return rcp_approx(1.f + pow2_approx(z * -1.4426950408889634f)); }
// Phi of two values; e: e^(-z^2 / 2).
__device__ __forceinline__ void normal_cdf(float z0, float z1, float (&phi)[2], float (&e)[2]) {
    const f2 z = pair(z0, z1), x = pair(fabsf(z0), fabsf(z1));
    const f2 d = fma2(x, both(0.3275911f * 0.70710678118654752f), both(1.f));
    const f2 q = z * z * both(-0.5f * 1.4426950408889634f);
    const f2 t = pair(rcp_approx(lo(d)), rcp_approx(hi(d))), ex = pair(pow2_approx(lo(q)), pow2_approx(hi(q)));
    f2 p = fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
    p = fma2(t, p, both(0.5f * 1.421413741f));
    p = fma2(t, p, both(0.5f * -0.284496736f));
    p = fma2(t, p, both(0.5f * 0.254829592f));
    p = p * t * ex;                                  // half of erfc(|z| / sqrt 2)
    phi[0] = z0 < 0.f ? lo(p) : 1.f - lo(p);
    phi[1] = z1 < 0.f ? hi(p) : 1.f - hi(p);
    e[0] = lo(ex);
    e[1] = hi(ex);
}
// That is right to 1e-7 of |z|, far below a bf16 result's rounding, but would be an fp32 result's error, and in Phi's tail a large one.
// The same for fp32 results, right to 10 steps of 2^-23 of Phi itself: Phi(-x) e^(x^2 / 2) / t with t = 1 / (1 + 0.4 x) is smooth in t, and a
// polynomial of degree 9 in w, t from x = 13.4 .. 0 moved to -1 .. 1, fitted to it in its relative error, is within 2^-26; its terms' magnitudes add up to
// 2.7 times the least value.  The square is taken in two parts, or the exponent's rounding would be 40 steps at x = 9.  (CUDA's normcdff
// took 82 us for 138936 x 64 -> 128 where this takes 59 and the short form 57.)
__device__ __forceinline__ void normal_cdf_fp32(float z0, float z1, float (&phi)[2], float (&e)[2]) {
    const f2 x = pair(fminf(fabsf(z0), 14.f), fminf(fabsf(z1), 14.f));            // beyond, Phi(-x) is 0
    const f2 d = fma2(x, both(0.4f), both(1.f));
    const f2 t = pair(rcp_approx(lo(d)), rcp_approx(hi(d)));
    const f2 w = fma2(t, both(2.3731344f), both(-1.3731344f));
    f2 p = fma2(w, both(1.33773777e-05f), both(-8.94124969e-06f));
    p = fma2(p, w, both(-0.000112753536f));
    p = fma2(p, w, both(0.000230123333f));
    p = fma2(p, w, both(0.000607057475f));
    p = fma2(p, w, both(-0.00288472394f));
    p = fma2(p, w, both(-0.004540978f));
    p = fma2(p, w, both(0.0355934239f));
    p = fma2(p, w, both(0.159877628f));
    p = fma2(p, w, both(0.311225802f));
    const float c = -0.5f * 1.4426950408889634f;                  // e^(-x^2 / 2) = 2^(c x^2), and what c and x^2 lose in fp32
    const f2 sq = x * x, rest = fma2(x, x, both(-1.f) * sq), q = sq * both(c);
    const f2 small = fma2(rest, both(c), fma2(sq, both((float)(-0.5 * 1.4426950408889634 - c)), fma2(sq, both(c), both(-1.f) * q)));
    f2 ex = pair(pow2_approx(lo(q)), pow2_approx(hi(q)));
    ex = fma2(ex, small * both(0.69314718f), ex);
    p = p * t * ex;
    phi[0] = z0 < 0.f ? lo(p) : 1.f - lo(p);
    phi[1] = z1 < 0.f ? hi(p) : 1.f - hi(p);
    e[0] = lo(ex);
    e[1] = hi(ex);
}
template <typename T>
__device__ __forceinline__ void normal_cdf_of(float z0, float z1, float (&phi)[2], float (&e)[2]) {
    if constexpr (sizeof(T) == 4) normal_cdf_fp32(z0, z1, phi, e);
    else normal_cdf(z0, z1, phi, e);
}
// max(y, 0); a NaN stays one (fmaxf gives 0, which would hide it from the loss).
__device__ __forceinline__ float relu(float y) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(y));
    return r;
}
// y = act(y), and y *= act'(z), of results of type T, the kind chosen once for N values.
template <typename T, int N>
__device__ __forceinline__ void act_apply(float (&y)[N], int act) {
    if (act == EAGA_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = relu(y[j]);
    } else if (act == EAGA_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            float phi[2], e[2];
            normal_cdf_of<T>(y[j], j + 1 < N ? y[j + 1 < N ? j + 1 : j] : 0.f, phi, e);
            y[j] *= phi[0];
            if (j + 1 < N) y[j + 1 < N ? j + 1 : j] *= phi[1];
        }
    } else if (act == EAGA_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] *= sigmoid(y[j]);
    }
}
template <typename T, int N>
__device__ __forceinline__ void act_slope_mul(float (&y)[N], const float (&z)[N], int act) {
    if (act == EAGA_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = z[j] > 0.f ? y[j] : y[j] * (z[j] <= 0.f ? 0.f : z[j]);     // NaN where z is
    } else if (act == EAGA_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const int k = j + 1 < N ? j + 1 : j;
            float phi[2], e[2];
            normal_cdf_of<T>(z[j], z[k], phi, e);
            y[j] *= fmaf(z[j] * 0.39894228040143268f, e[0], phi[0]);
            if (k > j) y[k] *= fmaf(z[k] * 0.39894228040143268f, e[1], phi[1]);
        }
    } else if (act == EAGA_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float e = sigmoid(z[j]);
            y[j] *= e * fmaf(z[j], 1.f - e, 1.f);
        }
    }
}

// 8 consecutive values, the first `k` of them there; `vec`: p is on 16 bytes and k is 8, or (fp32) 4 or 8.
__device__ __forceinline__ void lin_ld8(const __nv_bfloat16 *p, int k, bool vec, float (&v)[8]) {
    if (vec) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const unsigned x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(x[j] << 16);
            v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < k ? __bfloat162float(p[j]) : 0.f;
    }
}
__device__ __forceinline__ void lin_ld8(const float *p, int k, bool vec, float (&v)[8]) {
    if (vec) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = k > 4 ? *reinterpret_cast<const float4 *>(p + 4) : make_float4(0, 0, 0, 0);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < k ? p[j] : 0.f;
    }
}
__device__ __forceinline__ void lin_st8(__nv_bfloat16 *p, int k, bool vec, const float (&v)[8]) {
    if (vec) {
        uint4 o;
        __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint4 *>(p) = o;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < k) p[j] = __float2bfloat16_rn(v[j]);
    }
}
__device__ __forceinline__ void lin_st8(float *p, int k, bool vec, const float (&v)[8]) {
    if (vec) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        if (k > 4) *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < k) p[j] = v[j];
    }
}

// A product's epilogue.  Forward: z = acc + bias, out2 = z, out = act(z) + add.
// Input gradient: out = acc * act'(zin) + add.
template <typename T>
struct LinEpi {
    const T *bias, *add, *zin;
    T *out, *out2;
    int act;
};

// Output tiles: 256 x 256 on a pair of CTAs, or 128 x bn on one.
struct LinTile {
    bool pair;
    int bn;
};
// Split of a product's reduction into parts of `chunk`, and its tiles.
struct LinSplit {
    int splits;
    long long chunk;
    LinTile tile;
};

// tcgen05 products of bf16 operands whose rows are ld elements long (a multiple of 8), zero past the true
// size.  An operand may come in parts that are added; seg: the products of parts to sum, A's part (of X, or of
// dZ in LIN_DX) in the low two bits, B's in the next two.
struct LinTc {
    long long rows;
    int in, out;
    const __nv_bfloat16 *X[3], *W[3], *dZ[3];
    int ldx, ldw, ldz;
    int nseg;
    uint8_t seg[6];
    int *status;
    bool clear;                // this launch clears the status word
};
// Of a product [M, K] x [K, N]; f32: of fp32 operands and tensors in the epilogue.  us: the estimated time, where not null.
LinSplit lin_tc_split(long long M, int N, long long K, int nseg, bool f32, double *us = nullptr);
// The kernel of such a product: its tile, whether outputs go by TMA (rows of whole 16 bytes), two CTAs an SM, sums that leave the
// accumulator on the way; and its units, tiles times splits.  kind: LinKind; f32: of an fp32 result (a split one is).
struct LtForm {
    LinTile tile;
    bool tma, two, promo;
    long long units;
};
LtForm lin_tc_form(int kind, const LinSplit &s, bool f32, long long M, int N, long long K, int nseg);
// With one split the finished outputs; with more e.out takes the splits' sums [splits][M][N] in fp32, and nothing else of e is there.
template <typename T>
cudaError_t lin_tc_forward(const LinTc &p, const LinSplit &s, const LinEpi<T> &e, cudaStream_t st);
template <typename T>
cudaError_t lin_tc_dx(const LinTc &p, const LinSplit &s, const LinEpi<T> &e, cudaStream_t st);
// dW likewise; and where db is not null the column sums in lin_db_parts() parts [parts][out].
inline int lin_db_parts(const LinSplit &s, int in) { return s.splits * (s.tile.pair ? (in + 255) / 256 : 1); }
cudaError_t lin_tc_dw(const LinTc &p, const LinSplit &s, float *dW, float *db, cudaStream_t st);

// CUDA-core products of fp32 operands of any size; partial sums [splits][in][out] (and [splits][out]) where splits > 1.
struct LinF32 {
    long long rows;
    int in, out;
    const float *X, *W, *dZ;
    int *status;               // cleared
};
// Whether an fp32 product of M x N over K runs by warps, which take columns in eights at 17 TFLOP/s and whose join is as long as
// 80 steps, or in tiles of 16 columns at 13 or of 32 at 17, which want four CTAs of 128 rows an SM (300000 x 100 -> 8 67 us
// against 82, 1000000 x 70 -> 9 343 against 196, 20000 x 128 -> 16 8.7 against 14.8).
inline double lin_tile_rate(int N) { return N <= 16 ? 13e6 : N <= 32 ? 17e6 : 22e6; }        // multiply-adds as two, a us
inline bool lin_narrow(long long M, int N, long long K) {
    if (N > 32 || K < 64) return false;
    return M < 512LL * sm_count() || (N + 7) / 8 * 8 * (K + 80) / 17e6 < (N <= 16 ? 16 : 32) * K / lin_tile_rate(N);
}
// The kernel of a product on the CUDA cores: by warps with four or two steps in flight, tiles, or rows in registers (narrow dW).
enum LfForm { LF_WARPS4, LF_WARPS2, LF_128x16, LF_128x32, LF_64x64, LF_32x32, LF_THIN };
LfForm lin_f32_form(int kind, long long M, int N, long long K, int splits);
cudaError_t lin_f32_forward(const LinF32 &p, const LinEpi<float> &e, cudaStream_t st);
cudaError_t lin_f32_dx(const LinF32 &p, const LinEpi<float> &e, cudaStream_t st);
LinSplit lin_f32_dw_split(long long rows, int in, int out);
cudaError_t lin_f32_dw(const LinF32 &p, const LinSplit &s, float *dW, float *db, cudaStream_t st);

// Few rows: the weights are read once, bound by memory (at most 8 rows in bf16, 16 in fp32).  Above four rows in bf16 the tensor
// cores' launch is the shorter one (8 x 4096 -> 4096: 12.6 us against 22.6 forward, 29 against 72 backward; at one row 13.4
// against 7.6 and 30 against 26), but for rows that they need copied (8 x 1000 -> 1001: 10.2 against 8.4 and 14 against 8.7) and
// gradients of small weights (8 x 512 -> 512: 9.7 against 5.8).  fp32 products take six of the tensor cores' and three copies
// (8 x 4096 -> 4096: 75 us against 29).
inline bool lin_few_rows(const eaga_linear_dims &d, bool back) {
    if (d.dtype == EAGA_FP32) return d.rows <= 16;
    if (d.rows <= 4) return true;
    return d.rows <= 8 && (d.in % 8 || d.out % 8 || (back && (long long)d.in * d.out <= 1 << 18));
}
template <typename T>
struct LinVec {
    int rows, in, out;
    const T *X, *W, *dY, *Z;
    int act;                   // backward: act of Z
    T *dX;
    float *dW, *db;
    int *status;               // cleared
};
// Rows such a kernel is made for, and whether it reads W 16 bytes at a time.
inline int lin_vec_rows(int rows) { return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }
inline bool lin_vec_wide(int out, int dtype) { return out % (dtype == EAGA_BF16 ? 8 : 4) == 0; }
template <typename T>
cudaError_t lin_vec_forward(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st);
template <typename T>
cudaError_t lin_vec_backward(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st);

}  // namespace ops
}  // namespace eaga
