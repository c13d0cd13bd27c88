// The linear operator's products in fp32 on the CUDA cores, where reductions or results are so narrow that the tensor
// cores' copies and tiles cost more (lin_plan() estimates both):
//
//   forward   Y  = f(X W)      dX  dX = f(dZ W^T)      dW  dW = X^T dZ
//
// A CTA of 256 threads takes a BM x BN tile, 16 steps of the reduction at a time
// through two shared buffers, a thread BM/16 x BN/16 sums.  Bound: fp32 multiply-adds, at the sizes
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

template <int KIND, int BM, int BN>
__global__ void __launch_bounds__(256)
k_lin_f32(const LfParams p) {
    after_previous();
    constexpr int TM = BM / 16, TN = BN / 16, PA = BM * LF_BK / 256, PB = BN * LF_BK / 256;
    __shared__ float sa[2][LF_BK][BM + 4], sb[2][LF_BK][BN + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const unsigned tiles_n = (p.N + BN - 1) / BN;      // columns fastest
    const int n0 = blockIdx.x % tiles_n * BN, m0 = blockIdx.x / tiles_n * BM;
    const long long k0 = KIND == LIN_DW ? blockIdx.y * p.chunk : 0;
    const long long k1 = KIND == LIN_DW ? min(p.K, k0 + p.chunk) : p.K;
    // A(m, k): k contiguous, in dW m contiguous.  B(k, n): n contiguous, in dX k contiguous.
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.status = 0;
    float ra[PA], rb[PB];
    auto fetch = [&](long long k) {
#pragma unroll
        for (int i = 0; i < PA; ++i) {
            const int q = tid + 256 * i;
            const int m = KIND == LIN_DW ? q % BM : q / LF_BK, ka = KIND == LIN_DW ? q / BM : q % LF_BK;
            ra[i] = m0 + m < p.M && k + ka < k1
                        ? p.A[KIND == LIN_DW ? (size_t)(k + ka) * p.lda + m0 + m : (size_t)(m0 + m) * p.lda + k + ka] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int q = tid + 256 * i;
            const int n = KIND == LIN_DX ? q / LF_BK : q % BN, kb = KIND == LIN_DX ? q % LF_BK : q / BN;
            rb[i] = n0 + n < p.N && k + kb < k1
                        ? p.B[KIND == LIN_DX ? (size_t)(n0 + n) * p.ldb + k + kb : (size_t)(k + kb) * p.ldb + n0 + n] : 0.f;
        }
    };
    auto keep = [&](int b) {
#pragma unroll
        for (int i = 0; i < PA; ++i) {
            const int q = tid + 256 * i;
            if (KIND == LIN_DW) sa[b][q / BM][q % BM] = ra[i];
            else sa[b][q % LF_BK][q / LF_BK] = ra[i];
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int q = tid + 256 * i;
            if (KIND == LIN_DX) sb[b][q % LF_BK][q / LF_BK] = rb[i];
            else sb[b][q / BN][q % BN] = rb[i];
        }
    };
    float acc[TM][TN], col = 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
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
            float x[TM], y[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) x[i] = sa[b][kk][ty * TM + i];
#pragma unroll
            for (int j = 0; j < TN; ++j) y[j] = sb[b][kk][tx * TN + j];
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] += x[i] * y[j];
        }
        if (sums && tid < BN) {                      // 16 rows by themselves: a shorter chain of additions to a large sum
            float part = 0.f;
#pragma unroll
            for (int kk = 0; kk < LF_BK; ++kk) part += sb[b][kk][tid];
            col += part;
        }
        if (more) keep(b ^ 1);
        __syncthreads();
    }
    before_next();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + ty * TM + i;
        if (m >= p.M) break;
        const int n = n0 + tx * TN;
        const size_t at = (size_t)m * p.N + n;
        if constexpr (KIND == LIN_DW) {
            float *o = p.acc + (size_t)blockIdx.y * p.M * p.N + at;
#pragma unroll
            for (int j = 0; j < TN; ++j)
                if (n + j < p.N) o[j] = acc[i][j];
        } else {
            float z[TN], y[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                y[j] = acc[i][j];
                if (KIND == LIN_FWD && p.e.bias && n + j < p.N) y[j] += p.e.bias[n + j];
                z[j] = KIND == LIN_DX && p.e.zin && n + j < p.N ? p.e.zin[at + j] : 0.f;
            }
            if constexpr (KIND == LIN_FWD) {
                if (p.e.out2) {
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        if (n + j < p.N) p.e.out2[at + j] = y[j];
                }
                act_apply<float>(y, p.e.act);
            } else if (p.e.zin) {
                act_slope_mul<float>(y, z, p.e.act);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j)
                if (n + j < p.N) p.e.out[at + j] = p.e.add ? y[j] + p.e.add[at + j] : y[j];
        }
    }
    if (sums && tid < BN && n0 + tid < p.N) p.db[(size_t)blockIdx.y * p.N + n0 + tid] = col;
}

// ------------------------------------------------------------------ host side

// Narrow results (up to 32 columns) of long reductions: a warp takes four rows and eight columns, a lane every 32nd step of the
// reduction, so A is read in whole lines and a weight from shared memory serves four rows; the lanes' 32 sums are joined at
// the end, halving them with every exchange until a lane has one element.  (Tiles of 128 x 16 leave most threads' columns
// empty and take the reduction in one place.)  Weights of up to 1024 steps stay while a CTA goes through its rows.
// 60000 x 512 -> 8 33 us (3.7 TB/s; tensor cores, their copies included, 89), 6580 x 2576 -> 17 49 (86), 40000 x 1500 -> 10 125 (192):
// multiply-adds are at a fifth of their rate and DRAM at half, so the loads' latency bounds it, at 24 or 32 warps an SM.
constexpr int LN_K = 1024;     // steps whose weights are in shared memory at once
constexpr int LN_R = 4;        // rows of a warp
// U: steps whose loads are in flight.  Four leave registers for three CTAs an SM, two for four, which short reductions, of a
// few steps and the join, want: 300000 x 100 -> 8 67 us against 81, 60000 x 512 -> 8 37 against 33.5.
template <int KIND, int U>
__global__ void __launch_bounds__(256, U == 2 ? 4 : 3)
k_lin_narrow(const LfParams p) {
    after_previous();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    __shared__ __align__(16) float ws[LN_K][12];     // eight lanes' rows, read as two float4, lie in different banks
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned blocks = (p.N + 7) / 8;           // of columns, fastest
    const int n0 = blockIdx.x % blocks * 8, step = gridDim.x / blocks * 8 * LN_R;
    auto weights = [&](long long k0, int n) {
        if (KIND == LIN_DX) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c)              // a row of W at a time, as it lies in memory
                for (int k = threadIdx.x; k < n; k += 256)
                    ws[k][c] = n0 + c < p.N ? p.B[(size_t)(n0 + c) * p.ldb + k0 + k] : 0.f;
        } else {
#pragma unroll 4
            for (int q = threadIdx.x; q < n * 8; q += 256)
                ws[q / 8][q % 8] = n0 + q % 8 < p.N ? p.B[(size_t)(k0 + q / 8) * p.ldb + n0 + q % 8] : 0.f;
        }
    };
    const bool once = p.K <= LN_K;                   // the weights stay for all of the CTA's rows
    if (once) {
        weights(0, (int)p.K);
        __syncthreads();
    }
    for (long long row = (long long)(blockIdx.x / blocks) * (8 * LN_R); row < p.M; row += step) {
        const long long row0 = row + warp * LN_R;
        const float *A[LN_R];
#pragma unroll
        for (int r = 0; r < LN_R; ++r) A[r] = p.A + (size_t)(row0 + r < p.M ? row0 + r : 0) * p.lda;     // past the end row 0, not stored
        float a[8 * LN_R];
#pragma unroll
        for (int i = 0; i < 8 * LN_R; ++i) a[i] = 0.f;
        for (long long k0 = 0; k0 < p.K; k0 += LN_K) {
            const int n = (int)min((long long)LN_K, p.K - k0);
            if (!once) {
                __syncthreads();
                weights(k0, n);
                __syncthreads();
            }
            if (row0 >= p.M) continue;
#pragma unroll U
            for (int k = lane; k < n; k += 32) {
                float x[LN_R];
#pragma unroll
                for (int r = 0; r < LN_R; ++r) x[r] = A[r][k0 + k];
                const float4 u = *reinterpret_cast<const float4 *>(ws[k]), v = *reinterpret_cast<const float4 *>(ws[k] + 4);
                const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int r = 0; r < LN_R; ++r) a[8 * r + c] += x[r] * w[c];
            }
        }
        int at = 0;                                  // the element that this lane is left with
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const bool up = lane & o;
            at += up ? o : 0;
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const float send = up ? a[i] : a[i + o], kept = up ? a[i + o] : a[i];
                a[i] = kept + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
        const long long m = row0 + at / 8;
        const int n = n0 + at % 8;
        if (m >= p.M || n >= p.N) continue;
        const size_t to = (size_t)m * p.N + n;
        float y[2] = {a[0], 0.f}, z[2] = {0.f, 0.f};
        if (KIND == LIN_FWD && p.e.bias) y[0] += p.e.bias[n];
        if (KIND == LIN_DX && p.e.zin) z[0] = p.e.zin[to];
        if (KIND == LIN_FWD && p.e.out2) p.e.out2[to] = y[0];
        if (KIND == LIN_FWD) act_apply<float>(y, p.e.act);
        else if (p.e.zin) act_slope_mul<float>(y, z, p.e.act);
        p.e.out[to] = p.e.add ? y[0] + p.e.add[to] : y[0];
    }
    before_next();
}
static_assert(8 * LN_R == 32, "a sum for each lane");

// Weight gradients of narrow operands (in, out <= 32): a thread takes a row at a time and adds the outer product of 8 of its
// X and 8 of its dZ, read once, to sums in registers; the threads' sums are joined at the end.  (16 rows a step through
// shared memory, as above, took 283 us for a million rows of 8 -> 8.)
struct LtThin {
    const float *X, *Z;
    float *acc, *db;
    long long rows, chunk;
    int in, out;
    int *status;
};
__device__ __forceinline__ void thin_row(const float *p, long long row, int ld, int c0, bool vec, float (&v)[8]) {
    lin_ld8(p + row * ld + c0, min(8, ld - c0), vec, v);
}
__global__ void __launch_bounds__(256) k_lin_thin_dw(const LtThin p) {
    after_previous();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
    __shared__ float sum[8][72];
    const int tiles_n = (p.out + 7) / 8, i0 = blockIdx.y / tiles_n * 8, o0 = blockIdx.y % tiles_n * 8;
    const bool vx = p.in % 4 == 0, vz = p.out % 4 == 0;
    const long long r1 = min(p.rows, (blockIdx.x + 1) * p.chunk);
    float acc[8][8], col[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        col[i] = 0.f;
#pragma unroll
        for (int o = 0; o < 8; ++o) acc[i][o] = 0.f;
    }
#pragma unroll 2
    for (long long r = blockIdx.x * p.chunk + threadIdx.x; r < r1; r += 256) {
        float x[8], z[8];
        thin_row(p.X, r, p.in, i0, vx, x);
        thin_row(p.Z, r, p.out, o0, vz, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            col[i] += z[i];
#pragma unroll
            for (int o = 0; o < 8; ++o) acc[i][o] += x[i] * z[o];
        }
    }
    before_next();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = 0; o < 8; ++o) {
            const float t = warp_sum(acc[i][o]);
            if (lane == 0) sum[warp][i * 8 + o] = t;
        }
        const float t = warp_sum(col[i]);
        if (lane == 0) sum[warp][64 + i] = t;
    }
    __syncthreads();
    if (threadIdx.x < 72) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += sum[w][threadIdx.x];
        const int i = threadIdx.x / 8, o = o0 + threadIdx.x % 8;
        if (i < 8) {
            if (i0 + i < p.in && o < p.out) p.acc[((size_t)blockIdx.x * p.in + i0 + i) * p.out + o] = t;
        } else if (p.db && i0 == 0 && o < p.out) {
            p.db[(size_t)blockIdx.x * p.out + o] = t;
        }
    }
}
static bool lf_thin(int in, int out) { return in <= 32 && out <= 32 && ((in + 7) / 8) * ((out + 7) / 8) <= 8; }

// Narrow results by warps where lin_narrow() says so, else tiles: 64 x 64; narrow results of many rows 128 x 16 or 128 x 32; 32 x 32 where others leave SMs without one.
static long long lf_tiles(long long M, int N, int bm, int bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); }
LfForm lin_f32_form(int kind, long long M, int N, long long K, int splits) {
    if (kind == LIN_DW && lf_thin((int)M, N)) return LF_THIN;
    if (kind != LIN_DW) {
        if (lin_narrow(M, N, K)) return K < 256 ? LF_WARPS2 : LF_WARPS4;
        if (N <= 16 && lf_tiles(M, N, 128, 16) >= 2 * sm_count()) return LF_128x16;
        if (N <= 32 && lf_tiles(M, N, 128, 32) >= 2 * sm_count()) return LF_128x32;
    }
    return N > 32 && M > 32 && lf_tiles(M, N, 64, 64) * splits >= sm_count() ? LF_64x64 : LF_32x32;
}
template <int KIND>
static cudaError_t lf_launch(const LfParams &p, int splits, cudaStream_t st) {
    auto go = [&](auto kernel, int bm, int bn) {
        const long long n = lf_tiles(p.M, p.N, bm, bn);
        if (n > 0x7fffffffLL) return cudaErrorInvalidValue;
        return launch_pdl(kernel, dim3((unsigned)n, splits), dim3(256), 0, st, 1, p);
    };
    const LfForm form = lin_f32_form(KIND, p.M, p.N, p.K, splits);
    if constexpr (KIND != LIN_DW) {
        if (form == LF_WARPS2 || form == LF_WARPS4) {
            const bool brief = form == LF_WARPS2;
            const long long blocks = (p.N + 7) / 8, rows = ((long long)p.M + 8 * LN_R - 1) / (8 * LN_R);
            const dim3 grid((unsigned)(std::min(rows, std::max(1LL, (brief ? 4LL : 3LL) * sm_count() / blocks)) * blocks));
            return brief ? launch_pdl(k_lin_narrow<KIND, 2>, grid, dim3(256), 0, st, 1, p) : launch_pdl(k_lin_narrow<KIND, 4>, grid, dim3(256), 0, st, 1, p);
        }
        if (form == LF_128x16) return go(k_lin_f32<KIND, 128, 16>, 128, 16);
        if (form == LF_128x32) return go(k_lin_f32<KIND, 128, 32>, 128, 32);
    }
    return form == LF_64x64 ? go(k_lin_f32<KIND, 64, 64>, 64, 64) : go(k_lin_f32<KIND, 32, 32>, 32, 32);
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
    if (lf_thin(in, out)) {                          // one part for each CTA, of 1024 rows or more
        const long long tiles = ((in + 7) / 8) * ((out + 7) / 8), s = std::max(1LL, std::min(2LL * sm_count() / tiles, rows / 1024));
        const long long chunk = std::max(1LL, (rows + s - 1) / s);
        return {(int)std::max(1LL, (rows + chunk - 1) / chunk), chunk, {}};
    }
    const long long tiles = (long long)((in + 63) / 64) * ((out + 63) / 64);
    long long s = std::max(1LL, 4LL * sm_count() / tiles);
    s = std::max(1LL, std::min(s, rows / 256));
    const long long chunk = std::max(1LL, ((rows + s - 1) / s + LF_BK - 1) / LF_BK) * LF_BK;
    return {(int)std::max(1LL, (rows + chunk - 1) / chunk), chunk, {}};
}
cudaError_t lin_f32_dw(const LinF32 &q, const LinSplit &s, float *dW, float *db, cudaStream_t st) {
    if (lf_thin(q.in, q.out)) {
        const LtThin t = {q.X, q.dZ, dW, db, q.rows, s.chunk, q.in, q.out, q.status};
        return launch_pdl(k_lin_thin_dw, dim3(s.splits, (unsigned)(((q.in + 7) / 8) * ((q.out + 7) / 8))), dim3(256), 0, st, 1, t);
    }
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
