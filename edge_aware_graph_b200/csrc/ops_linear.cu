// The linear operator (eaga_linear_forward / _backward):
//
//   Z = X W + b        Y = act(Z) + R
//   dZ = act'(Z) dY    dX = act_in'(Zin) (dZ W^T) + dR    dW = X^T dZ    db = sum of dZ's rows
//
// Which kernels run is a rule on rows, type and alignment:
//   up to 8 rows        ops_linear_vec.cu, bound by the read of W
//   bf16                ops_linear_tc.cu (tcgen05)
//   fp32                ops_linear_f32.cu (CUDA cores)
//
// The tensor-core kernels read their operands by TMA, whose rows begin on 16
// bytes: an operand with rows of another length is copied once into padded
// rows in the workspace.  dZ where act is not none is an fp32 value: it goes
// into the workspace as three bf16 parts that carry its 24 bits between them.
// dW, an fp32 result, takes all three; dX, rounded to bf16, the upper two (16
// bits: the rest is 2^-9 of the result's own rounding).
#include <algorithm>
#include "ops_linear.h"

namespace eaga {
namespace ops {

// One operand to prepare: src [rows][n], times act'(z) where z is given, as `parts` bf16 parts [rows][ld]
// (zero past n), or (f32) as fp32 [rows][n].
struct PrepJob {
    const void *src, *z;
    void *dst[3];
    float *f32;
    long long rows;
    int n, ld, act, parts;
};
struct PrepArgs {
    PrepJob job[3];
};

// A value's bf16 part and what it leaves.  Of an infinity or a NaN nothing is left: the first part says it all.
__device__ __forceinline__ float take_part(float &v) {
    const float hi = __bfloat162float(__float2bfloat16_rn(v));
    v = isfinite(hi) ? v - hi : 0.f;
    return hi;
}

template <typename T>
__global__ void __launch_bounds__(256) k_lin_prep(const __grid_constant__ PrepArgs a) {
    after_previous();
    const PrepJob &j = a.job[blockIdx.y];
    const int per = j.ld / 8;
    const bool vec = (long long)j.n * sizeof(T) % 16 == 0;
    const T *src = static_cast<const T *>(j.src), *zs = static_cast<const T *>(j.z);
    const long long total = j.rows * per, step = (long long)gridDim.x * 256;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += step) {
        const long long row = i / per;
        const int c = (int)(i % per) * 8, have = min(8, j.n - c);
        const size_t at = (size_t)row * j.n + c;
        float v[8], z[8];
        lin_ld8(src + at, have, vec, v);
        if (zs) {
            lin_ld8(zs + at, have, vec, z);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k >= have) z[k] = 0.f;
            act_slope_mul(v, z, j.act);
        }
        if (j.f32) {
            lin_st8(j.f32 + at, have, vec, v);
            continue;
        }
        for (int k = 0; k < j.parts; ++k) {
            float o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = take_part(v[u]);
            lin_st8(static_cast<__nv_bfloat16 *>(j.dst[k]) + (size_t)row * j.ld + c, 8, true, o);
        }
    }
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
    bool vec, tc;
    int ldx, ldw, ldz, zparts;
    LinSplit split;
    int bparts;                // of the bias gradient
    size_t X, W, dZ[3], dZ32, acc, bacc, total;      // workspace offsets; 0: not there
};

static LinPlan lin_plan(const eaga_linear_dims &d, bool back) {
    LinPlan p = {};
    p.vec = d.rows <= LIN_VEC_ROWS;
    p.tc = !p.vec && d.dtype == EAGA_BF16;
    p.split = {1, 0, {}};
    size_t off = 256;                                // the status word
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t rows = (size_t)d.rows, in = d.in, out = d.out;
    const bool dact = back && d.act != EAGA_ACT_NONE;
    if (p.tc) {
        p.ldx = round8(d.in);
        p.ldw = p.ldz = round8(d.out);
        if (p.ldx != d.in) p.X = take(rows * p.ldx * 2);
        if (p.ldw != d.out) p.W = take(in * p.ldw * 2);
        p.zparts = dact ? 3 : 1;
        if (back && (dact || p.ldz != d.out))
            for (int k = 0; k < p.zparts; ++k) p.dZ[k] = take(rows * p.ldz * 2);
        if (back) p.split = lin_tc_dw_split(d.rows, d.in, d.out, p.zparts);
    } else if (!p.vec && back) {
        if (dact) p.dZ32 = take(rows * out * 4);
        p.split = lin_f32_dw_split(d.rows, d.in, d.out);
    }
    if (p.split.splits > 1) p.acc = take(p.split.splits * in * out * 4);
    if (back && !p.vec) p.bparts = lin_db_parts(p.split, d.in);
    if (p.bparts > 1) p.bacc = take(p.bparts * out * 4);
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

struct LinBack {
    const void *X, *W, *Z, *dY;
    int act_in;
    const void *Zin, *dR;
    void *dX;
    float *dW, *db;
    char *ws;
};

static cudaError_t backward_tc(const eaga_linear_dims &d, const LinPlan &p, const LinBack &b, cudaStream_t st) {
    typedef __nv_bfloat16 bf;
    PrepJob jobs[3] = {};
    int n = 0;
    LinTc q = {};
    q.rows = d.rows; q.in = d.in; q.out = d.out;
    q.ldx = p.ldx; q.ldw = p.ldw; q.ldz = p.ldz;
    q.status = reinterpret_cast<int *>(b.ws);
    q.clear = true;
    auto at = [&](size_t off) { return reinterpret_cast<bf *>(b.ws + off); };
    q.X[0] = static_cast<const bf *>(b.X);
    q.W[0] = static_cast<const bf *>(b.W);
    q.dZ[0] = static_cast<const bf *>(b.dY);
    if (p.X && b.dW) {
        jobs[n++] = {b.X, nullptr, {at(p.X)}, nullptr, d.rows, d.in, p.ldx, 0, 1};
        q.X[0] = at(p.X);
    }
    if (p.W && b.dX) {
        jobs[n++] = {b.W, nullptr, {at(p.W)}, nullptr, d.in, d.out, p.ldw, 0, 1};
        q.W[0] = at(p.W);
    }
    const int zparts = b.dW ? p.zparts : std::min(p.zparts, 2);
    if (p.dZ[0]) {
        PrepJob j = {b.dY, b.Z, {}, nullptr, d.rows, d.out, p.ldz, d.act, zparts};
        for (int k = 0; k < zparts; ++k) {
            j.dst[k] = at(p.dZ[k]);
            q.dZ[k] = at(p.dZ[k]);
        }
        jobs[n++] = j;
    }
    if (cudaError_t e = lin_prep<bf>(jobs, n, st); e != cudaSuccess) return e;
    if (b.dX) {
        LinTc x = q;
        x.nseg = std::min(zparts, 2);
        for (int k = 0; k < x.nseg; ++k) x.seg[k] = (uint8_t)(x.nseg - 1 - k);              // A = dZ, W in one part
        const LinEpi<bf> e = {nullptr, static_cast<const bf *>(b.dR), static_cast<const bf *>(b.Zin), static_cast<bf *>(b.dX), nullptr, b.act_in};
        if (cudaError_t err = lin_tc_dx(x, e, st); err != cudaSuccess) return err;
        q.clear = false;
    }
    if (b.dW) {
        q.nseg = zparts;
        for (int k = 0; k < q.nseg; ++k) q.seg[k] = (uint8_t)((q.nseg - 1 - k) << 2);       // B = dZ, X in one part
        float *acc = p.split.splits > 1 ? reinterpret_cast<float *>(b.ws + p.acc) : b.dW;
        float *bacc = !b.db ? nullptr : p.bparts > 1 ? reinterpret_cast<float *>(b.ws + p.bacc) : b.db;
        if (cudaError_t err = lin_tc_dw(q, p.split, acc, bacc, st); err != cudaSuccess) return err;
        return lin_reduce((long long)d.in * d.out, p.split.splits, acc, b.dW, d.out, p.bparts, bacc, b.db, st);
    }
    return cudaSuccess;
}

static cudaError_t backward_f32(const eaga_linear_dims &d, const LinPlan &p, const LinBack &b, cudaStream_t st) {
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
        float *acc = p.split.splits > 1 ? reinterpret_cast<float *>(b.ws + p.acc) : b.dW;
        float *bacc = !b.db ? nullptr : p.bparts > 1 ? reinterpret_cast<float *>(b.ws + p.bacc) : b.db;
        if (cudaError_t err = lin_f32_dw(q, p.split, acc, bacc, st); err != cudaSuccess) return err;
        return lin_reduce((long long)d.in * d.out, p.split.splits, acc, b.dW, d.out, p.bparts, bacc, b.db, st);
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

}  // namespace ops
}  // namespace eaga

using namespace eaga;
using namespace eaga::ops;

extern "C" {

size_t eaga_linear_workspace_size(const eaga_linear_dims *d, int for_backward) {
    if (lin_check(d) != EAGA_OK) return 0;
    return lin_plan(*d, for_backward != 0).total;
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
    if (p.vec) {
        e = d->dtype == EAGA_BF16 ? forward_vec(*d, X, W, forward_epi<__nv_bfloat16>(*d, b, R, Y, Z), workspace, st)
                                  : forward_vec(*d, X, W, forward_epi<float>(*d, b, R, Y, Z), workspace, st);
    } else if (!p.tc) {
        const LinF32 q = {d->rows, d->in, d->out, static_cast<const float *>(X), static_cast<const float *>(W), nullptr, static_cast<int *>(workspace)};
        e = lin_f32_forward(q, forward_epi<float>(*d, b, R, Y, Z), st);
    } else {
        typedef __nv_bfloat16 bf;
        char *ws = static_cast<char *>(workspace);
        PrepJob jobs[2] = {};
        int n = 0;
        LinTc q = {};
        q.rows = d->rows; q.in = d->in; q.out = d->out;
        q.ldx = p.ldx; q.ldw = p.ldw; q.nseg = 1;
        q.X[0] = static_cast<const bf *>(X);
        q.W[0] = static_cast<const bf *>(W);
        q.status = static_cast<int *>(workspace);
        q.clear = true;
        if (p.X) {
            jobs[n++] = {X, nullptr, {ws + p.X}, nullptr, d->rows, d->in, p.ldx, 0, 1};
            q.X[0] = reinterpret_cast<const bf *>(ws + p.X);
        }
        if (p.W) {
            jobs[n++] = {W, nullptr, {ws + p.W}, nullptr, d->in, d->out, p.ldw, 0, 1};
            q.W[0] = reinterpret_cast<const bf *>(ws + p.W);
        }
        e = lin_prep<bf>(jobs, n, st);
        if (e == cudaSuccess) e = lin_tc_forward(q, forward_epi<bf>(*d, b, R, Y, Z), st);
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
    if (p.tc) e = backward_tc(*d, p, b, st);
    else if (!p.vec) e = backward_f32(*d, p, b, st);
    else e = d->dtype == EAGA_BF16 ? backward_vec<__nv_bfloat16>(*d, b, st) : backward_vec<float>(*d, b, st);
    return e == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

}  // extern "C"
