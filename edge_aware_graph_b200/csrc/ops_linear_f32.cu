// The linear operator's products in fp32 on the CUDA cores, any size:
//
//   forward   Y  = f(X W)      dX  dX = f(dZ W^T)      dW  dW = X^T dZ
//
// A CTA of 256 threads takes a BT x BT tile (BT = 64, or 32 where that leaves
// SMs without one), 16 steps of the reduction at a time through two shared
// buffers, a thread (BT/16)^2 sums.  Bound: fp32 multiply-adds, at the sizes
// it is used for their latency.  The bias gradient is summed from the dZ tiles
// of the first row of dW's tiles.
#include <algorithm>
#include "ops_linear.h"

namespace eaga {
namespace ops {

constexpr int LF_BK = 16;

struct LfParams {
    const float *A, *B;
    LinEpi<float> e;
    float *acc, *db;
    int *status;
    int M, N;
    long long K, chunk;        // the reduction; a split's part of it
    long long lda, ldb;
};

template <int KIND, int BT>
__global__ void __launch_bounds__(256)
k_lin_f32(const LfParams p) {
    after_previous();
    constexpr int TM = BT / 16, PER = BT * LF_BK / 256;
    __shared__ float sa[2][LF_BK][BT + 4], sb[2][LF_BK][BT + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const unsigned tiles_n = (p.N + BT - 1) / BT;      // columns fastest
    const int n0 = blockIdx.x % tiles_n * BT, m0 = blockIdx.x / tiles_n * BT;
    const long long k0 = KIND == LIN_DW ? blockIdx.y * p.chunk : 0;
    const long long k1 = KIND == LIN_DW ? min(p.K, k0 + p.chunk) : p.K;
    // A(m, k): k contiguous, in dW m contiguous.  B(k, n): n contiguous, in dX k contiguous.
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.status = 0;
    float ra[PER], rb[PER];
    auto fetch = [&](long long k) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = tid + 256 * i;
            const int m = KIND == LIN_DW ? q % BT : q / LF_BK, ka = KIND == LIN_DW ? q / BT : q % LF_BK;
            ra[i] = m0 + m < p.M && k + ka < k1
                        ? p.A[KIND == LIN_DW ? (size_t)(k + ka) * p.lda + m0 + m : (size_t)(m0 + m) * p.lda + k + ka] : 0.f;
            const int n = KIND == LIN_DX ? q / LF_BK : q % BT, kb = KIND == LIN_DX ? q % LF_BK : q / BT;
            rb[i] = n0 + n < p.N && k + kb < k1
                        ? p.B[KIND == LIN_DX ? (size_t)(n0 + n) * p.ldb + k + kb : (size_t)(k + kb) * p.ldb + n0 + n] : 0.f;
        }
    };
    auto keep = [&](int b) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = tid + 256 * i;
            if (KIND == LIN_DW) sa[b][q / BT][q % BT] = ra[i];
            else sa[b][q % LF_BK][q / LF_BK] = ra[i];
            if (KIND == LIN_DX) sb[b][q % LF_BK][q / LF_BK] = rb[i];
            else sb[b][q / BT][q % BT] = rb[i];
        }
    };
    float acc[TM][TM], col = 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = 0.f;
    const bool sums = KIND == LIN_DW && p.db != nullptr && m0 == 0;
    int b = 0;
    fetch(k0);
    keep(0);
    __syncthreads();
    for (long long k = k0; k < k1; k += LF_BK, b ^= 1) {
        const bool more = k + LF_BK < k1;
        if (more) fetch(k + LF_BK);
#pragma unroll
        for (int kk = 0; kk < LF_BK; ++kk) {
            float x[TM], y[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) x[i] = sa[b][kk][ty * TM + i];
#pragma unroll
            for (int j = 0; j < TM; ++j) y[j] = sb[b][kk][tx * TM + j];
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) acc[i][j] += x[i] * y[j];
        }
        if (sums && tid < BT) {
#pragma unroll
            for (int kk = 0; kk < LF_BK; ++kk) col += sb[b][kk][tid];
        }
        if (more) keep(b ^ 1);
        __syncthreads();
    }
    before_next();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + ty * TM + i;
        if (m >= p.M) break;
        const int n = n0 + tx * TM;
        const size_t at = (size_t)m * p.N + n;
        if constexpr (KIND == LIN_DW) {
            float *o = p.acc + (size_t)blockIdx.y * p.M * p.N + at;
#pragma unroll
            for (int j = 0; j < TM; ++j)
                if (n + j < p.N) o[j] = acc[i][j];
        } else {
            float z[TM], y[TM];
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                y[j] = acc[i][j];
                if (KIND == LIN_FWD && p.e.bias && n + j < p.N) y[j] += p.e.bias[n + j];
                z[j] = KIND == LIN_DX && p.e.zin && n + j < p.N ? p.e.zin[at + j] : 0.f;
            }
            if constexpr (KIND == LIN_FWD) {
                if (p.e.out2) {
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        if (n + j < p.N) p.e.out2[at + j] = y[j];
                }
                act_apply(y, p.e.act);
            } else if (p.e.zin) {
                act_slope_mul(y, z, p.e.act);
            }
#pragma unroll
            for (int j = 0; j < TM; ++j)
                if (n + j < p.N) p.e.out[at + j] = p.e.add ? y[j] + p.e.add[at + j] : y[j];
        }
    }
    if (sums && tid < BT && n0 + tid < p.N) p.db[(size_t)blockIdx.y * p.N + n0 + tid] = col;
}

// ------------------------------------------------------------------ host side

template <int KIND>
static cudaError_t lf_launch(const LfParams &p, int splits, cudaStream_t st) {
    auto tiles = [&](int bt) { return ((long long)p.M + bt - 1) / bt * ((p.N + bt - 1) / bt); };
    const int bt = tiles(64) * splits >= sm_count() ? 64 : 32;
    if (tiles(bt) > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)tiles(bt), splits);
    return launch_pdl(bt == 64 ? k_lin_f32<KIND, 64> : k_lin_f32<KIND, 32>, grid, dim3(256), 0, st, 1, p);
}

cudaError_t lin_f32_forward(const LinF32 &q, const LinEpi<float> &e, cudaStream_t st) {
    LfParams p = {};
    p.status = q.status;
    p.A = q.X; p.B = q.W; p.e = e;
    p.M = (int)q.rows; p.N = q.out; p.K = q.in;
    p.lda = q.in; p.ldb = q.out;
    return lf_launch<LIN_FWD>(p, 1, st);
}
cudaError_t lin_f32_dx(const LinF32 &q, const LinEpi<float> &e, cudaStream_t st) {
    LfParams p = {};
    p.status = q.status;
    p.A = q.dZ; p.B = q.W; p.e = e;
    p.M = (int)q.rows; p.N = q.in; p.K = q.out;
    p.lda = q.out; p.ldb = q.out;
    return lf_launch<LIN_DX>(p, 1, st);
}
// Splits until there are about four CTAs an SM, of 256 rows or more.
LinSplit lin_f32_dw_split(long long rows, int in, int out) {
    const long long tiles = (long long)((in + 63) / 64) * ((out + 63) / 64);
    long long s = std::max(1LL, 4LL * sm_count() / tiles);
    s = std::max(1LL, std::min(s, rows / 256));
    const long long chunk = std::max(1LL, ((rows + s - 1) / s + LF_BK - 1) / LF_BK) * LF_BK;
    return {(int)std::max(1LL, (rows + chunk - 1) / chunk), chunk, {}};
}
cudaError_t lin_f32_dw(const LinF32 &q, const LinSplit &s, float *dW, float *db, cudaStream_t st) {
    LfParams p = {};
    p.status = q.status;
    p.A = q.X; p.B = q.dZ;
    p.acc = dW; p.db = db;
    p.M = q.in; p.N = q.out; p.K = q.rows; p.chunk = s.chunk;
    p.lda = q.in; p.ldb = q.out;
    return lf_launch<LIN_DW>(p, s.splits, st);
}

}  // namespace ops
}  // namespace eaga
