// The linear operator for a few rows (serving: one token, one graph's global
// features; lin_few_rows() says how many).  Bound: the read of W, and in the backward the write of dW;
// there is nothing for the tensor cores to do, so each weight goes from memory
// to registers once and is multiplied by all rows there.
//
// Forward: a CTA takes 128 bytes of columns of W and a part of its rows; the
// parts of one column tile are a cluster, whose first CTA adds the others'
// sums out of their shared memory (in order) and does the epilogue: one launch,
// no workspace.  Backward: a warp takes a row of W, the same row of dW and one
// column of dX, with dZ (all rows) in shared memory.
#include <algorithm>
#include <type_traits>
#include "ops_linear.h"
#include "sm100.cuh"

namespace eaga {
namespace ops {

using namespace sm100;

// VEC consecutive weights as they lie in memory, and their values.
template <typename T, int VEC>
struct VecIo {
    typedef typename std::conditional<VEC == 1, T, uint4>::type Raw;
    static __device__ __forceinline__ Raw fetch(const T *p) { return __ldg(reinterpret_cast<const Raw *>(p)); }
    static __device__ __forceinline__ void values(const Raw &a, float (&v)[VEC]) {
        if constexpr (VEC == 1) {
            v[0] = ldf(&a);
        } else {
            const unsigned x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (VEC == 4) {
                    v[j] = __uint_as_float(x[j]);
                } else {
                    v[2 * j] = __uint_as_float(x[j] << 16);
                    v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
                }
            }
        }
    }
};

template <int R> constexpr int lv_chunk() { return R > 8 ? 256 : 512; }      // rows of W whose X is in shared memory at once
constexpr int LV_BATCH = 8;        // loads a thread has in flight

// R: rows (the call's, rounded up).  part: rows of W a CTA takes.
template <typename T, int VEC, int R>
__global__ void __launch_bounds__(256)
k_lin_vec_fwd(const LinVec<T> p, const LinEpi<T> e, int part, int cluster) {
    after_previous();
    constexpr int LANES = VEC == 1 ? 32 : 8, C = LANES * VEC, KR = 256 / LANES;
    constexpr int LV_CHUNK = lv_chunk<R>();
    __shared__ float xs[R][LV_CHUNK];
    __shared__ float red[8][R][C];
    __shared__ float sum[R][C];
    const int tid = threadIdx.x, cl = tid % LANES, kr = tid / LANES, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % cluster, c0 = blockIdx.x / cluster * C;
    const int k0 = rank * part, k1 = min(p.in, k0 + part);
    const int col = c0 + cl * VEC;
    const bool on = col < p.out;
    if (blockIdx.x == 0 && tid == 0) *p.status = 0;
    float acc[R][VEC];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[r][j] = 0.f;
    typedef VecIo<T, VEC> IO;
    for (int kb = k0; kb < k1; kb += LV_CHUNK) {
        const int n = min(LV_CHUNK, k1 - kb);
        const T *w = p.W + (size_t)kb * p.out + col;
        typename IO::Raw raw[LV_BATCH];
        auto fetch = [&](int k) {                    // rows k, k + KR, ..
#pragma unroll
            for (int i = 0; i < LV_BATCH; ++i)
                if (on && k + i * KR < n) raw[i] = IO::fetch(w + (size_t)(k + i * KR) * p.out);
        };
        fetch(kr);                                   // on their way before X is there
        __syncthreads();
        for (int i = tid; i < R * LV_CHUNK; i += 256) {
            const int r = i / LV_CHUNK, k = i % LV_CHUNK;
            xs[r][k] = r < p.rows && k < n ? ldf(p.X + (size_t)r * p.in + kb + k) : 0.f;
        }
        __syncthreads();
        for (int k = kr; k < n; k += LV_BATCH * KR) {
            if (k != kr) fetch(k);
#pragma unroll
            for (int i = 0; i < LV_BATCH; ++i) {
                if (!on || k + i * KR >= n) break;
                float v[VEC];
                IO::values(raw[i], v);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float x = xs[r][k + i * KR];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[r][j] += x * v[j];
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float s = acc[r][j];
            if (LANES < 32) {
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
            }
            if (lane < LANES) red[warp][r][cl * VEC + j] = s;
        }
    before_next();
    __syncthreads();
    for (int i = tid; i < R * C; i += 256) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < 8; ++v) s += red[v][i / C][i % C];
        sum[i / C][i % C] = s;
    }
    __syncthreads();
    if (cluster > 1) cluster_sync_all();
    if (rank == 0) {
        for (int i = tid; i < p.rows * C; i += 256) {
            const int r = i / C, c = c0 + i % C;
            if (c >= p.out) continue;
            float z = sum[r][i % C];
            const uint32_t local = smem_u32(&sum[r][i % C]);
            for (int q = 1; q < cluster; ++q) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_map(local, q)) : "memory");
                z += v;
            }
            if (e.bias) z += ldf(e.bias + c);
            const size_t at = (size_t)r * p.out + c;
            if (e.out2) stf(e.out2 + at, z);
            float y[1] = {z};
            act_apply<T>(y, e.act);
            if (e.add) y[0] += ldf(e.add + at);
            stf(e.out + at, y[0]);
        }
    }
    __syncthreads();
    if (cluster > 1) cluster_sync_all();       // shared memory stays until the first CTA has read it
}

template <typename T, int VEC, int R>
__global__ void __launch_bounds__(256)
k_lin_vec_bwd(const LinVec<T> p, const LinEpi<T> e) {
    after_previous();
    constexpr int CC = 8192 / R;               // columns of dZ at once
    __shared__ __align__(16) float dz[R][CC];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i = blockIdx.x * 8 + warp;
    const bool on = i < p.in;
    if (blockIdx.x == 0 && tid == 0) *p.status = 0;
    float x[R], acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = on && p.dW && r < p.rows ? ldf(p.X + (size_t)r * p.in + i) : 0.f;
        acc[r] = 0.f;
    }
    for (int c0 = 0; c0 < p.out; c0 += CC) {
        const int n = min(CC, p.out - c0);
        __syncthreads();
        for (int c = tid; c < n; c += 256) {         // a column of all rows: their loads are on their way together
            float d[R], z[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const size_t at = (size_t)r * p.out + c0 + c;
                d[r] = r < p.rows ? ldf(p.dY + at) : 0.f;
                z[r] = p.Z && r < p.rows ? ldf(p.Z + at) : 0.f;
            }
            if (p.Z) act_slope_mul<T>(d, z, p.act);
#pragma unroll
            for (int r = 0; r < R; ++r) dz[r][c] = d[r];
        }
        __syncthreads();
        if (p.db && blockIdx.x == 0) {
            for (int c = tid; c < n; c += 256) {
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) s += dz[r][c];
                p.db[c0 + c] = s;
            }
        }
        if (on) {
            const T *w = p.W + (size_t)i * p.out + c0;
            float *o = p.dW ? p.dW + (size_t)i * p.out + c0 : nullptr;
#pragma unroll (VEC == 1 ? 8 : 4)
            for (int c = lane * VEC; c < n; c += 32 * VEC) {
                float v[VEC], s[VEC];
                if (p.dX) {
                    VecIo<T, VEC>::values(VecIo<T, VEC>::fetch(w + c), v);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) v[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[j] = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = dz[r][c + j];
                        acc[r] += v[j] * d;
                        s[j] += x[r] * d;
                    }
                if (o) {
                    if constexpr (VEC == 1) {
                        o[c] = s[0];
                    } else {
#pragma unroll
                        for (int j = 0; j < VEC; j += 4)
                            __stcs(reinterpret_cast<float4 *>(o + c + j), make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]));
                    }
                }
            }
        }
    }
    before_next();
    if (on && p.dX) {
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = warp_sum(acc[r]);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane == r && r < p.rows) {
                const size_t at = (size_t)r * p.in + i;
                float y[1] = {acc[r]};
                if (e.zin) {
                    const float z[1] = {ldf(e.zin + at)};
                    act_slope_mul<T>(y, z, e.act);
                }
                if (e.add) y[0] += ldf(e.add + at);
                stf(p.dX + at, y[0]);
            }
    }
}

// ------------------------------------------------------------------ host side

template <typename T, int VEC, int R>
static cudaError_t vec_fwd(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st) {
    constexpr int C = (VEC == 1 ? 32 : 8) * VEC;
    const int tiles = (p.out + C - 1) / C;
    // parts of 128 rows of W or more, up to eight, until there are about four CTAs an SM
    int cluster = 1;
    while (cluster < 8 && tiles * cluster < 4 * sm_count() && p.in >= 256 * cluster) cluster *= 2;
    const int part = (p.in + cluster - 1) / cluster;
    return launch_pdl(k_lin_vec_fwd<T, VEC, R>, dim3((unsigned)tiles * cluster), dim3(256), 0, st, cluster, p, e, part, cluster);
}
template <typename T, int VEC, int R>
static cudaError_t vec_bwd(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st) {
    return launch_pdl(k_lin_vec_bwd<T, VEC, R>, dim3((p.in + 7) / 8), dim3(256), 0, st, 1, p, e);
}

template <typename T, typename F>
static cudaError_t vec_pick(int rows, int out, F &&f) {
    auto go = [&](auto vec) {
        switch (lin_vec_rows(rows)) {
            case 1: return f(vec, std::integral_constant<int, 1>{});
            case 2: return f(vec, std::integral_constant<int, 2>{});
            case 4: return f(vec, std::integral_constant<int, 4>{});
            case 8: return f(vec, std::integral_constant<int, 8>{});
        }
        if constexpr (sizeof(T) == 4) return f(vec, std::integral_constant<int, 16>{});
        return cudaErrorInvalidValue;
    };
    return lin_vec_wide(out, sizeof(T) == 4 ? EAGA_FP32 : EAGA_BF16) ? go(std::integral_constant<int, 16 / sizeof(T)>{})
                                                                     : go(std::integral_constant<int, 1>{});
}

template <typename T>
cudaError_t lin_vec_forward(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st) {
    return vec_pick<T>(p.rows, p.out, [&](auto v, auto r) { return vec_fwd<T, decltype(v)::value, decltype(r)::value>(p, e, st); });
}
template <typename T>
cudaError_t lin_vec_backward(const LinVec<T> &p, const LinEpi<T> &e, cudaStream_t st) {
    return vec_pick<T>(p.rows, p.out, [&](auto v, auto r) { return vec_bwd<T, decltype(v)::value, decltype(r)::value>(p, e, st); });
}
template cudaError_t lin_vec_forward<float>(const LinVec<float> &, const LinEpi<float> &, cudaStream_t);
template cudaError_t lin_vec_forward<__nv_bfloat16>(const LinVec<__nv_bfloat16> &, const LinEpi<__nv_bfloat16> &, cudaStream_t);
template cudaError_t lin_vec_backward<float>(const LinVec<float> &, const LinEpi<float> &, cudaStream_t);
template cudaError_t lin_vec_backward<__nv_bfloat16>(const LinVec<__nv_bfloat16> &, const LinEpi<__nv_bfloat16> &, cudaStream_t);

}  // namespace ops
}  // namespace eaga
