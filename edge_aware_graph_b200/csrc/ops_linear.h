// The linear operator's products: C = A B with a fused epilogue (ops_linear.cu, _tc.cu, _vec.cu, _f32.cu).
#pragma once
#include <cuda_runtime.h>
#include "ops.h"

namespace eaga {
namespace ops {

// Which product: forward Y = f(X W), input gradient dX = f(dZ W^T), weight gradient dW = X^T dZ.
enum LinKind { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

__device__ __forceinline__ float gelu_value(float z) { return z * (0.5f + 0.5f * erff(z * 0.70710678118654752f)); }
__device__ __forceinline__ float gelu_slope(float z) {
    return 0.5f + 0.5f * erff(z * 0.70710678118654752f) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
}
__device__ __forceinline__ float silu_value(float z) { return z / (1.f + expf(-z)); }
__device__ __forceinline__ float silu_slope(float z) {
    const float e = 1.f / (1.f + expf(-z));
    return e * (1.f + z * (1.f - e));
}
// y = act(y), and y *= act'(z), the kind chosen once for N values.
template <int N>
__device__ __forceinline__ void act_apply(float (&y)[N], int act) {
    if (act == EAGA_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = fmaxf(y[j], 0.f);
    } else if (act == EAGA_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = gelu_value(y[j]);
    } else if (act == EAGA_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = silu_value(y[j]);
    }
}
template <int N>
__device__ __forceinline__ void act_slope_mul(float (&y)[N], const float (&z)[N], int act) {
    if (act == EAGA_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = z[j] > 0.f ? y[j] : y[j] * 0.f;
    } else if (act == EAGA_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] *= gelu_slope(z[j]);
    } else if (act == EAGA_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] *= silu_slope(z[j]);
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
// Of a product [M, K] x [K, N].
LinSplit lin_tc_split(long long M, int N, long long K, int nseg);
// With one split the finished outputs; with more e.out takes the splits' sums [splits][M][N] in fp32, and nothing else of e is there.
template <typename T>
cudaError_t lin_tc_forward(const LinTc &p, const LinSplit &s, const LinEpi<T> &e, cudaStream_t st);
template <typename T>
cudaError_t lin_tc_dx(const LinTc &p, const LinSplit &s, const LinEpi<T> &e, cudaStream_t st);
// dW likewise; and where db is not null the column sums in lin_db_parts() parts [parts][out].
inline int lin_db_parts(const LinSplit &s, int in) { return s.splits * (s.tile.pair ? (in + 255) / 256 : 1); }
cudaError_t lin_tc_dw(const LinTc &p, const LinSplit &s, float *dW, float *db, cudaStream_t st);

// Up to LIN_VEC_ROWS rows: the weights are read once, bound by memory.
constexpr int LIN_VEC_ROWS = 8;
template <typename T>
struct LinVec {
    int rows, in, out;
    const T *X, *W, *dY, *Z;
    int act;                   // backward: act of Z
    T *dX;
    float *dW, *db;
    int *status;               // cleared
};
template <typename T>
cudaError_t lin_vec_forward(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st);
template <typename T>
cudaError_t lin_vec_backward(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st);

}  // namespace ops
}  // namespace eaga
