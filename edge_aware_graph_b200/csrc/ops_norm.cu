// The residual step between two sub-layers, with the norm after the one and
// before the other (eaga_residual_norm_forward / _backward).  Per row:
//
//   p = post(u)        r = alpha x + gate * p        h = pre(r)
//   norm(z) = gain * (z - mean z) / sqrt(var z + eps) + shift     (layer; rms: without the mean, no shift needed)
//
// and backward, with dr, dh given:
//   g  = dr + pre'(dh; r)           dx = alpha g          dp = gate * g
//   du = post'(dp; u)               dgate = sum over the group's rows of g * p
//   norm'(d; z) = (e - mean(e) - zh mean(e zh)) / sqrt(var z + eps),  e = gain * d, zh = the normalised z
//   dgain = sum over rows of d * zh,   dshift = sum over rows of d
//
// One pass: a team of threads holds a row in registers (8 or 16 elements a
// thread, in fp32), so every tensor is read once and written once, and a
// norm's mean and centred squares are two sums over registers (the centred
// form does not cancel).  Bound: HBM.  Teams of up to 32 threads share a warp
// with other rows and reduce by shuffles; wider rows take a CTA.  The
// normalisation of h reads r before r is rounded.
//
// The backward recomputes the statistics (the rows are there anyway) and
// keeps the sums over rows of the gains' and shifts' gradients in registers:
// a thread owns the same columns in every row.  Each CTA leaves one partial
// row per parameter and each run of a group's rows one of its gate, which
// k_rn_finish adds in a fixed order: no atomics, the same bits every time.
#include <algorithm>
#include <type_traits>
#include "common.cuh"
#include "ops.h"

namespace eaga {
namespace ops {

enum { RN_NONE = EAGA_NORM_NONE, RN_LAYER = EAGA_NORM_LAYER, RN_RMS = EAGA_NORM_RMS };

// The sums over partial rows that end a backward: the parameters' gradients (`parts`, a row a CTA and parameter), then
// the gate's groups (`gparts`, a row a run).
struct FinishArgs {
    const float *parts, *gparts;
    float *out[4], *all[4];    // those that are wanted; by parameter
    void *dgate;
    unsigned w, ctas, groups, runs_per_group, flat;
    int n_out, which[4], dtype;
};

struct RnArgs {
    const void *x, *u, *gate, *post_g, *post_s, *pre_g, *pre_s;
    const uint8_t *M;
    void *r, *h;
    // backward
    const void *rin, *dr, *dh;
    void *dx, *du, *dgate;
    float *parts, *gparts;     // [CTA][4][w] sums of the gains' and shifts' gradients, [run][w] of the gate's
    float alpha, eps, inv_w;
    unsigned rows, w, group, run, runs_per_group, runs;
    FinishArgs fin;
    int join;                  // the grid is one cluster (or CTA) and ends the backward itself
    int pre, post, team, crew; // threads that hold a row; threads that share a run (backward)
};

// ------------------------------------------------------------------ a row in registers
// E elements a thread.  VEC > 1: 16-byte vectors, thread k of a team holds
// vectors k, k + team, ..; VEC == 1: single elements, for rows whose length or
// start is not a multiple of 16 bytes.

template <typename T, int VEC, int E>
struct RowIo {
    static constexpr int NV = E / VEC;
    // A row's elements as they lie in memory: 16-byte vectors (fewer registers than the values), or elements.
    struct Raw {
        typename std::conditional<VEC == 1, T, uint4>::type v[NV];
    };
    // column of element q of this thread
    static __device__ __forceinline__ unsigned col(int q, unsigned k, unsigned team) {
        return (k + (q / VEC) * team) * VEC + q % VEC;
    }
    static __device__ __forceinline__ void fetch(const T *p, bool there, unsigned k, unsigned team, unsigned w, Raw &r) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const unsigned c = (k + n * team) * VEC;
            if constexpr (VEC == 1) {
                r.v[n] = there && c < w ? p[c] : T(0.f);
            } else {
                r.v[n] = there && c < w ? *reinterpret_cast<const uint4 *>(p + c) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    static __device__ __forceinline__ void values(const Raw &r, f2 (&v)[E / 2]) {
        if constexpr (VEC == 1) {
#pragma unroll
            for (int n = 0; n < E / 2; ++n) v[n] = pair(ldf(&r.v[2 * n]), ldf(&r.v[2 * n + 1]));
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const unsigned x[4] = {r.v[n].x, r.v[n].y, r.v[n].z, r.v[n].w};
                if constexpr (sizeof(T) == 4) {
                    v[2 * n] = pair(__uint_as_float(x[0]), __uint_as_float(x[1]));
                    v[2 * n + 1] = pair(__uint_as_float(x[2]), __uint_as_float(x[3]));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[4 * n + j] = pair(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u));
                }
            }
        }
    }
    static __device__ __forceinline__ void load(const T *p, unsigned k, unsigned team, unsigned w, f2 (&v)[E / 2]) {
        Raw r;
        fetch(p, true, k, team, w, r);
        values(r, v);
    }
    static __device__ __forceinline__ void store(T *p, unsigned k, unsigned team, unsigned w, const f2 (&v)[E / 2]) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const unsigned c = (k + n * team) * VEC;
            if (c >= w) continue;
            if constexpr (VEC == 1) {
                stf(p + c, n & 1 ? hi(v[n / 2]) : lo(v[n / 2]));
            } else if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4 *>(p + c) = make_float4(lo(v[2 * n]), hi(v[2 * n]), lo(v[2 * n + 1]), hi(v[2 * n + 1]));
            } else {
                uint4 o;
                __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = __floats2bfloat162_rn(lo(v[4 * n + j]), hi(v[4 * n + j]));
                *reinterpret_cast<uint4 *>(p + c) = o;
            }
        }
    }
    static __device__ __forceinline__ void store_zeros(T *p, unsigned k, unsigned team, unsigned w) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const unsigned c = (k + n * team) * VEC;
            if (c >= w) continue;
            if constexpr (VEC == 1) stf(p + c, 0.f);
            else *reinterpret_cast<uint4 *>(p + c) = make_uint4(0, 0, 0, 0);
        }
    }
    // v - m, nothing where the row has no element
    static __device__ __forceinline__ void centre(f2 (&v)[E / 2], float m, unsigned k, unsigned team, unsigned w) {
        if constexpr (VEC == 1) {
#pragma unroll
            for (int n = 0; n < E / 2; ++n)
                v[n] = v[n] + pair(col(2 * n, k, team) < w ? -m : 0.f, col(2 * n + 1, k, team) < w ? -m : 0.f);
        } else {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const f2 t = both(col(n * VEC, k, team) < w ? -m : 0.f);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) v[n * (VEC / 2) + j] = v[n * (VEC / 2) + j] + t;
            }
        }
    }
};

// Sums of N values over a row's team, the same in every thread of it.  Teams
// within a warp: shuffles.  A team that is a CTA (WIDE): shuffles, then the
// warps' sums in order from shared memory; two buffers in turn, so that one
// barrier a sum is enough (a buffer is written again only behind the next
// sum's barrier, which every thread reaches after it has read).
template <bool WIDE, int N>
__device__ __forceinline__ void team_sum(float (&a)[N], unsigned team, float (*buf)[4][32], unsigned &turn) {
#pragma unroll
    for (unsigned o = 16; o; o >>= 1)
        if (WIDE || o < team) {
#pragma unroll
            for (int n = 0; n < N; ++n) a[n] += __shfl_xor_sync(0xffffffffu, a[n], o);
        }
    if constexpr (WIDE) {
        float (*b)[32] = buf[turn & 1];
        ++turn;
        const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) b[n][warp] = a[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = lane < nw ? b[n][lane] : 0.f;
            for (unsigned o = nw >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            a[n] = __shfl_sync(0xffffffffu, s, 0);
        }
    }
}

// Rows' threads: the thread's team in the grid, its place in it.
struct Team {
    unsigned k, id, count;
};
template <bool WIDE>
__device__ __forceinline__ Team my_team(unsigned team) {
    if (WIDE) return {threadIdx.x, blockIdx.x, gridDim.x};
    const unsigned per = blockDim.x / team;
    return {threadIdx.x % team, blockIdx.x * per + threadIdx.x / team, gridDim.x * per};
}

constexpr int RN_ROUNDS = 16;     // runs a crew of the backward takes of a long input
constexpr int RN_DEPTH = 4;        // steps of the backward in shared memory, the one that is worked on among them

// What a thread of the forward keeps beside the row it works on.  AHEAD: the next row, as it
// lies in memory (4 registers a tensor for 8 bf16 elements, where there is room
// for them).  KEEP: the norms' gains and shifts; teams of a CTA's size read
// those from L1 again, and run two CTAs an SM instead.
template <int VEC, int E, bool WIDE>
struct RnKeep {
    static constexpr bool AHEAD = VEC == 8, KEEP = AHEAD && !WIDE;
};

template <typename T, int VEC, int E, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 && (E > 8 || !WIDE) ? 3 : E > 8 ? 1 : 1024 / MAXT)
k_rn_fwd(const RnArgs a) {
    after_previous();
    using IO = RowIo<T, VEC, E>;
    using Raw = typename IO::Raw;
    constexpr int H = E / 2;
    constexpr bool AHEAD = RnKeep<VEC, E, WIDE>::AHEAD, KEEP = RnKeep<VEC, E, WIDE>::KEEP;
    __shared__ float buf[2][4][32];
    unsigned turn = 0;
    const unsigned w = a.w, team = a.team;
    const Team tm = my_team<WIDE>(team);
    const T *x = static_cast<const T *>(a.x), *u = static_cast<const T *>(a.u), *gate = static_cast<const T *>(a.gate);
    T *r = static_cast<T *>(a.r), *h = static_cast<T *>(a.h);
    const unsigned last = WIDE ? a.rows : (a.rows + tm.count - 1) / tm.count * tm.count;   // warps stay whole
    // the next row's elements are on their way while this one is normalised; the mask a row further ahead
    Raw nu, nx, ng;
    auto alive = [&](unsigned row) { return row < a.rows && (!a.M || a.M[row]); };
    auto ask = [&](unsigned row, bool live) {
        const size_t at = (size_t)(live ? row : 0) * w;
        IO::fetch(u + at, live, tm.k, team, w, nu);
        IO::fetch(x + at, live && x, tm.k, team, w, nx);
        if (gate) IO::fetch(gate + (size_t)((live ? row : 0) / a.group) * w, live, tm.k, team, w, ng);
    };
    bool live = alive(tm.id), next = AHEAD && alive(tm.id + tm.count);
    if (AHEAD) ask(tm.id, live);
    Raw kept[4];                                     // the norms' parameters
    const T *const param[4] = {static_cast<const T *>(a.post_g), static_cast<const T *>(a.post_s), static_cast<const T *>(a.pre_g),
                               static_cast<const T *>(a.pre_s)};
    if (KEEP) {
#pragma unroll
        for (int n = 0; n < 4; ++n) IO::fetch(param[n], param[n], tm.k, team, w, kept[n]);
    }
    for (unsigned row = tm.id; row < last; row += tm.count) {
        const bool in = row < a.rows;
        const size_t at = (size_t)(in ? row : 0) * w;
        if (!AHEAD) {
            live = alive(row);
            ask(row, live);
        }
        const bool now = live;
        f2 p[H];
        IO::values(nu, p);
        const Raw rx = nx, rg = ng;
        if (AHEAD) {
            ask(row + tm.count, next);
            live = next;
            next = alive(row + 2 * tm.count);
        }
        if (WIDE && !now) {                         // the whole CTA holds this row
            if (r) IO::store_zeros(r + at, tm.k, team, w);
            if (h) IO::store_zeros(h + at, tm.k, team, w);
            continue;
        }
        auto values_of = [&](auto which, f2 (&c)[E / 2]) {
            constexpr int P = decltype(which)::value;
            if constexpr (KEEP) IO::values(kept[P], c);
            else IO::load(param[P], tm.k, team, w, c);
        };
        auto norm = [&](f2 (&v)[E / 2], int kind, auto first) {          // parameters `first` (gain) and the next (shift)
            if (kind == RN_NONE) return;
            constexpr int P = decltype(first)::value;
            float s[1];
            if (kind == RN_LAYER) {
                f2 t = v[0];
#pragma unroll
                for (int q = 1; q < H; ++q) t = t + v[q];
                s[0] = across(t);
                team_sum<WIDE, 1>(s, team, buf, turn);
                IO::centre(v, s[0] * a.inv_w, tm.k, team, w);
            }
            f2 t = v[0] * v[0];
#pragma unroll
            for (int q = 1; q < H; ++q) t = fma2(v[q], v[q], t);
            s[0] = across(t);
            team_sum<WIDE, 1>(s, team, buf, turn);
            const f2 rstd = both(rsqrtf(s[0] * a.inv_w + a.eps));
            f2 c[H];
            if (param[P]) {
                values_of(first, c);
#pragma unroll
                for (int q = 0; q < H; ++q) v[q] = v[q] * (rstd * c[q]);
            } else {
#pragma unroll
                for (int q = 0; q < H; ++q) v[q] = v[q] * rstd;
            }
            if (param[P + 1]) {
                values_of(std::integral_constant<int, P + 1>{}, c);
#pragma unroll
                for (int q = 0; q < H; ++q) v[q] = v[q] + c[q];
            }
        };
        norm(p, a.post, std::integral_constant<int, 0>{});
        if (gate) {
            f2 c[H];
            IO::values(rg, c);
#pragma unroll
            for (int q = 0; q < H; ++q) p[q] = p[q] * c[q];
        }
        if (x) {
            f2 t[H];
            IO::values(rx, t);
            const f2 al = both(a.alpha);
#pragma unroll
            for (int q = 0; q < H; ++q) p[q] = fma2(al, t[q], p[q]);
        }
        if (r && in) {
            if (now) IO::store(r + at, tm.k, team, w, p);
            else IO::store_zeros(r + at, tm.k, team, w);
        }
        if (!h) continue;
        norm(p, a.pre, std::integral_constant<int, 2>{});
        if (in) {
            if (now) IO::store(h + at, tm.k, team, w, p);
            else IO::store_zeros(h + at, tm.k, team, w);
        }
    }
    before_next();
}

// 16 bytes of global memory into shared memory, zeros where `there` is not set (the address is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// One output of the last sums.
struct FinishJob {
    bool param;
    unsigned job, rows;
    size_t stride;
    const float *src;
    __device__ __forceinline__ FinishJob(const FinishArgs &f, unsigned n) {
        param = n < (unsigned)f.n_out;
        job = param ? n : n - f.n_out;
        rows = param ? f.ctas : f.runs_per_group;
        stride = param ? (size_t)4 * f.w : f.w;
        src = param ? f.parts + (size_t)f.which[job] * f.w : f.gparts + (size_t)job * f.runs_per_group * f.w;
    }
    __device__ __forceinline__ void put(const FinishArgs &f, unsigned c, float s) const {
        if (param) f.out[job][c] = s;
        else if (f.dtype == EAGA_FP32) static_cast<float *>(f.dgate)[(size_t)job * f.w + c] = s;
        else static_cast<__nv_bfloat16 *>(f.dgate)[(size_t)job * f.w + c] = __float2bfloat16_rn(s);
    }
};

// Outputs from number `job0` on, a thread four columns of them at a time, each the sum of its rows one after another.
__device__ __forceinline__ void finish_flat(const FinishArgs &f, unsigned job0, unsigned long long first, unsigned long long step) {
    const unsigned long long n = (unsigned long long)(f.n_out + f.groups) * f.w;
    for (unsigned long long i = (unsigned long long)job0 * f.w + first; i < n; i += 4 * step) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const unsigned long long at = i + q * step;
            if (at >= n) break;
            const unsigned job = (unsigned)(at / f.w), c = (unsigned)(at - (unsigned long long)job * f.w);
            const FinishJob j(f, job);
#pragma unroll 4
            for (unsigned r = 0; r < j.rows; ++r) s[q] += j.src[r * j.stride + c];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const unsigned long long at = i + q * step;
            if (at >= n) break;
            const unsigned job = (unsigned)(at / f.w), c = (unsigned)(at - (unsigned long long)job * f.w);
            FinishJob(f, job).put(f, c, s[q]);
        }
    }
}

// A crew takes runs of consecutive rows of one group (a run is the whole group
// or a part of it).  A crew is a team, or a warp whose teams take a row each,
// where groups are long enough: one sum of the gate's gradient a run then, and
// 512 consecutive bytes a load.  Runs go to the crews of a CTA from far apart,
// since masked rows, which cost little, come in stretches.
//
// With 8 bf16 elements a thread (AHEAD) the rows of the next steps are on their
// way into shared memory, where each thread reads back what it copied itself.
//
// In a run the gate's row is the same, so the row sums that its gradient and
// those of the post norm's gain and shift need are two, A = sum of g zh and
// B = sum of g:  dgain += gate A, dshift += gate B, dgate = gain A + shift B.
template <typename T, int VEC, int E, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT)
k_rn_bwd(const RnArgs a) {
    after_previous();
    using IO = RowIo<T, VEC, E>;
    using Raw = typename IO::Raw;
    constexpr int H = E / 2;
    constexpr bool AHEAD = VEC == 8 && E == 8;
    __shared__ float buf[2][4][32];
    unsigned turn = 0;
    const unsigned w = a.w, team = a.team, lane = threadIdx.x & 31;
    const unsigned k = WIDE ? threadIdx.x : threadIdx.x % team;
    // rows a crew takes a step, this thread's among them; the crew's number among the grid's
    const unsigned abreast = WIDE ? 1 : a.crew / team, sub = WIDE ? 0 : threadIdx.x % a.crew / team;
    const unsigned count = WIDE ? gridDim.x : blockDim.x / a.crew * gridDim.x;
    const unsigned id = WIDE ? blockIdx.x : threadIdx.x / a.crew * gridDim.x + blockIdx.x;
    const T *u = static_cast<const T *>(a.u), *rin = static_cast<const T *>(a.rin), *dr = static_cast<const T *>(a.dr),
            *dh = static_cast<const T *>(a.dh), *gate = static_cast<const T *>(a.gate);
    T *dx = static_cast<T *>(a.dx), *du = static_cast<T *>(a.du);
    const bool need_u = gate != nullptr || a.post != RN_NONE, has_pre = a.pre != RN_NONE;
    // Sums of the gains' and shifts' gradients, post then pre: in registers, or, where a thread holds 16 columns
    // and they would not fit, in shared memory (each thread its own columns).
    constexpr bool IN_SMEM = E > 8;
    extern __shared__ __align__(16) float acc[];     // [4][w], of teams in a warp [warp][4][w]; before the end of the AHEAD form, the rows to come
    f2 sums[4][IN_SMEM ? 1 : H];
    if constexpr (IN_SMEM) {
        for (unsigned c = threadIdx.x; c < 4 * w; c += blockDim.x) acc[c] = 0.f;
        __syncthreads();
    } else {
#pragma unroll
        for (int q = 0; q < H; ++q) sums[0][q] = sums[1][q] = sums[2][q] = sums[3][q] = both(0.f);
    }
    // sums[P] += v * m
    auto add = [&](auto which, int q, f2 v, f2 m) {
        constexpr int P = decltype(which)::value;
        if constexpr (IN_SMEM) {
            const f2 t = v * m;
            if (IO::col(2 * q, k, team) < w) acc[P * w + IO::col(2 * q, k, team)] += lo(t);
            if (IO::col(2 * q + 1, k, team) < w) acc[P * w + IO::col(2 * q + 1, k, team)] += hi(t);
        } else {
            sums[P][q] = fma2(v, m, sums[P][q]);
        }
    };
    Raw pre_g, post_g;
    if (AHEAD) {
        IO::fetch(static_cast<const T *>(a.pre_g), a.pre_g, k, team, w, pre_g);
        IO::fetch(static_cast<const T *>(a.post_g), a.post_g, k, team, w, post_g);
    }
    auto gain_of = [&](const void *p, const Raw &kept, f2 (&c)[E / 2]) {
        if constexpr (AHEAD) IO::values(kept, c);
        else IO::load(static_cast<const T *>(p), k, team, w, c);
    };

    // A place in the crew's sequence of rows.
    struct Place {
        unsigned run, i, row0, n;                    // the run, the row in it (its crew's first), the run's first row and number of rows
    };
    auto enter = [&](Place &p) {                     // the run's rows
        p.row0 = p.n = 0;
        if (p.run < a.runs) {
            const unsigned grp = p.run / a.runs_per_group, part = p.run - grp * a.runs_per_group;
            p.row0 = grp * a.group + part * a.run;
            p.n = min(a.run, a.group - part * a.run);
        }
    };
    auto forward = [&](Place &p) {                   // true: into another run
        p.i += abreast;
        if (p.i < a.run) return false;
        p.i = 0;
        p.run = p.run < a.runs && a.runs - p.run > count ? p.run + count : a.runs;
        enter(p);
        return true;
    };
    auto inside = [&](const Place &p) { return p.i + sub < p.n; };
    auto alive = [&](const Place &p) { return inside(p) && (!a.M || a.M[p.row0 + p.i + sub]); };
    // the masks of a run's rows at once (up to 64), where all of the warp's lanes are in it
    const bool one_run = WIDE || a.crew == 32;
    auto masks = [&](const Place &p) {
        const bool m0 = lane < p.n && (!a.M || a.M[p.row0 + lane]), m1 = lane + 32 < p.n && (!a.M || a.M[p.row0 + lane + 32]);
        return (unsigned long long)__ballot_sync(0xffffffffu, m0) | (unsigned long long)__ballot_sync(0xffffffffu, m1) << 32;
    };
    // the crews of a warp take the same number of steps
    const unsigned rounds = one_run ? (id < a.runs ? (a.runs - id + count - 1) / count : 0) : (a.runs + count - 1) / count;
    const unsigned long long steps = (unsigned long long)rounds * ((a.run + abreast - 1) / abreast);

    Place cons = {id, 0, 0, 0};
    enter(cons);
    Place prod = cons;
    unsigned long long alive_run = AHEAD && one_run ? masks(prod) : 0;
    unsigned lives = 0;                              // of the steps asked for, the latest in bit 0
    const uint32_t slots = (uint32_t)__cvta_generic_to_shared(acc) + threadIdx.x * 16, slot = blockDim.x * 16, stage = 5 * slot;
    const uint4 *slots_p = reinterpret_cast<const uint4 *>(acc) + threadIdx.x;
    unsigned long long asked = 0;
    const bool in_row = k * VEC < w;
    auto ask = [&] {                                 // the next step's rows into its stage
        if (asked < steps) {
            const bool live = one_run ? (alive_run >> (prod.i + sub)) & 1 : alive(prod);
            const uint32_t to = slots + (unsigned)(asked % RN_DEPTH) * stage;
            const size_t at = (size_t)(prod.row0 + prod.i + sub) * w + k * VEC;
            const bool there = live && in_row;
            if (dr) copy16(to, dr + (there ? at : 0), there);
            if (has_pre) {
                copy16(to + slot, dh + (there ? at : 0), there);
                copy16(to + 2 * slot, rin + (there ? at : 0), there);
            }
            if (need_u) copy16(to + 3 * slot, u + (there ? at : 0), there);
            if (gate && prod.i == 0) {
                const bool has = prod.run < a.runs && in_row;
                copy16(to + 4 * slot, gate + (has ? (size_t)(prod.run / a.runs_per_group) * w + k * VEC : 0), has);
            }
            lives = lives << 1 | (live ? 1u : 0u);
            if (forward(prod) && one_run) alive_run = masks(prod);
        }
        ++asked;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (AHEAD) {
        for (int d = 0; d < RN_DEPTH - 1; ++d) ask();
    }
    Raw c_dr, c_dh, c_r, c_u, gt;
    auto fetch_all = [&](bool live) {
        const size_t at = (size_t)(live ? cons.row0 + cons.i + sub : 0) * w;
        IO::fetch(dr + at, live && dr, k, team, w, c_dr);
        IO::fetch(dh + at, live && has_pre, k, team, w, c_dh);
        IO::fetch(rin + at, live && has_pre, k, team, w, c_r);
        IO::fetch(u + at, live && need_u, k, team, w, c_u);
        if (cons.i == 0 && gate) IO::fetch(gate + (size_t)(cons.run < a.runs ? cons.run / a.runs_per_group : 0) * w, true, k, team, w, gt);
    };
    f2 sa[H], sb[H];                                 // the run's A and B
    for (unsigned long long step = 0; step < steps; ++step) {
        bool live;
        if constexpr (AHEAD) {
            asm volatile("cp.async.wait_group %0;" ::"n"(RN_DEPTH - 2) : "memory");
            const unsigned ahead = (unsigned)min((unsigned long long)(RN_DEPTH - 1), steps - step);
            live = (lives >> (ahead - 1)) & 1;
            const uint4 *from = slots_p + (unsigned)(step % RN_DEPTH) * 5 * blockDim.x;
            c_dr.v[0] = dr ? from[0] : make_uint4(0, 0, 0, 0);
            c_dh.v[0] = from[blockDim.x];
            c_r.v[0] = from[2 * blockDim.x];
            c_u.v[0] = from[3 * blockDim.x];
            if (cons.i == 0) gt.v[0] = from[4 * blockDim.x];
            ask();                                   // into the stage that the last step read
        } else {
            live = alive(cons);
            fetch_all(live);
        }
        const bool in = inside(cons);
        const size_t at = (size_t)(in ? cons.row0 + cons.i + sub : 0) * w;
        if (cons.i == 0) {
#pragma unroll
            for (int q = 0; q < H; ++q) sa[q] = sb[q] = both(0.f);
        }
        if (WIDE ? !live : !__any_sync(0xffffffffu, live)) {
            if (in && dx) IO::store_zeros(dx + at, k, team, w);
            if (in && du) IO::store_zeros(du + at, k, team, w);
        } else {
            // rows that are not live hold zeros, and add zeros to every sum
            f2 g[H], d[H], z[H];
            IO::values(c_dr, g);
            // d becomes norm'(d; z), z normalised; sum(q, d, zh) adds to the parameters' sums
            auto back = [&](f2 (&d)[E / 2], f2 (&z)[E / 2], int kind, const void *gain, const Raw &kept, auto &&sum) {
                if (kind == RN_LAYER) {
                    f2 t = z[0];
#pragma unroll
                    for (int q = 1; q < H; ++q) t = t + z[q];
                    float s[1] = {across(t)};
                    team_sum<WIDE, 1>(s, team, buf, turn);
                    IO::centre(z, s[0] * a.inv_w, k, team, w);
                }
                f2 e[H];
                if (gain) {
                    gain_of(gain, kept, e);
#pragma unroll
                    for (int q = 0; q < H; ++q) e[q] = e[q] * d[q];
                } else {
#pragma unroll
                    for (int q = 0; q < H; ++q) e[q] = d[q];
                }
                f2 zz = z[0] * z[0], ez = e[0] * z[0], es = e[0];
#pragma unroll
                for (int q = 1; q < H; ++q) {
                    zz = fma2(z[q], z[q], zz);
                    ez = fma2(e[q], z[q], ez);
                    es = es + e[q];
                }
                float s[3] = {across(zz), across(ez), across(es)};
                team_sum<WIDE, 3>(s, team, buf, turn);
                const float rstd = rsqrtf(s[0] * a.inv_w + a.eps);
                const f2 rs = both(rstd), c1 = both(-(s[1] * a.inv_w * rstd));
                const f2 c2 = both(kind == RN_LAYER ? -(s[2] * a.inv_w) : 0.f);
#pragma unroll
                for (int q = 0; q < H; ++q) {
                    z[q] = z[q] * rs;
                    sum(q, d[q], z[q]);
                    d[q] = (fma2(z[q], c1, e[q]) + c2) * rs;
                }
            };
            if (has_pre) {
                IO::values(c_dh, d);
                IO::values(c_r, z);
                back(d, z, a.pre, a.pre_g, pre_g, [&](int q, f2 dq, f2 zh) {
                    add(std::integral_constant<int, 2>{}, q, dq, zh);
                    add(std::integral_constant<int, 3>{}, q, dq, both(1.f));
                });
#pragma unroll
                for (int q = 0; q < H; ++q) g[q] = g[q] + d[q];
            }
            if (dx && in) {
                const f2 al = both(a.alpha);
#pragma unroll
                for (int q = 0; q < H; ++q) z[q] = al * g[q];
                if (live) IO::store(dx + at, k, team, w, z);
                else IO::store_zeros(dx + at, k, team, w);
            }
            if (gate) {
                IO::values(gt, d);
#pragma unroll
                for (int q = 0; q < H; ++q) d[q] = d[q] * g[q];
            } else {
#pragma unroll
                for (int q = 0; q < H; ++q) d[q] = g[q];
            }
            IO::values(c_u, z);
            if (a.post != RN_NONE) {
                back(d, z, a.post, a.post_g, post_g, [&](int q, f2, f2 zh) {
                    sa[q] = fma2(g[q], zh, sa[q]);
                    sb[q] = sb[q] + g[q];
                });
            } else if (gate) {
#pragma unroll
                for (int q = 0; q < H; ++q) sa[q] = fma2(g[q], z[q], sa[q]);
            }
            if (du && in) {
                if (live) IO::store(du + at, k, team, w, d);
                else IO::store_zeros(du + at, k, team, w);
            }
        }
        if (cons.i + abreast >= a.run) {             // the run's last step
            f2 c[H];
            if (gate) {
                IO::values(gt, c);
            } else {
#pragma unroll
                for (int q = 0; q < H; ++q) c[q] = both(1.f);
            }
            if (a.post != RN_NONE && (!gate || cons.run < a.runs)) {
#pragma unroll
                for (int q = 0; q < H; ++q) {
                    add(std::integral_constant<int, 0>{}, q, sa[q], c[q]);
                    add(std::integral_constant<int, 1>{}, q, sb[q], c[q]);
                }
            }
            if (a.dgate) {
                if (a.post != RN_NONE) {
                    if (a.post_g) {
                        gain_of(a.post_g, post_g, c);
#pragma unroll
                        for (int q = 0; q < H; ++q) sa[q] = sa[q] * c[q];
                    }
                    if (a.post_s) {
                        IO::load(static_cast<const T *>(a.post_s), k, team, w, c);
#pragma unroll
                        for (int q = 0; q < H; ++q) sa[q] = fma2(sb[q], c[q], sa[q]);
                    }
                }
                if (!WIDE && abreast > 1) {          // the crew's teams, in pairs
                    for (unsigned o = team; o < 32; o <<= 1)
#pragma unroll
                        for (int q = 0; q < H; ++q)
                            sa[q] = sa[q] + pair(__shfl_xor_sync(0xffffffffu, lo(sa[q]), o), __shfl_xor_sync(0xffffffffu, hi(sa[q]), o));
                }
                if (cons.run < a.runs && sub == 0) {
                    if (a.runs_per_group == 1) {
                        IO::store(static_cast<T *>(a.dgate) + (size_t)cons.run * w, k, team, w, sa);
                    } else {
                        float *o = a.gparts + (size_t)cons.run * w;
#pragma unroll
                        for (int q = 0; q < H; ++q) {
                            if (IO::col(2 * q, k, team) < w) o[IO::col(2 * q, k, team)] = lo(sa[q]);
                            if (IO::col(2 * q + 1, k, team) < w) o[IO::col(2 * q + 1, k, team)] = hi(sa[q]);
                        }
                    }
                }
            }
        }
        forward(cons);
    }
    before_next();
    if constexpr (AHEAD) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();                             // the sums take the rows' place
    }
    // The CTA's sums: its warps' teams by shuffles (same columns), the warps in order.
    // (One CTA alone writes the outputs.)
    const bool alone = a.join && gridDim.x == 1;
    float *const out = a.parts + (size_t)blockIdx.x * 4 * w;
    auto target = [&](int n) { return alone ? a.fin.all[n] : out + n * w; };
    if constexpr (WIDE && !IN_SMEM) {
#pragma unroll
        for (int q = 0; q < E; ++q)
            if (IO::col(q, k, team) < w) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (float *o = target(n)) o[IO::col(q, k, team)] = q & 1 ? hi(sums[n][q / 2]) : lo(sums[n][q / 2]);
            }
    } else if constexpr (!IN_SMEM) {
        const unsigned warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
        for (int q = 0; q < H; ++q)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                for (unsigned o = team; o < 32; o <<= 1)
                    sums[n][q] = sums[n][q] + pair(__shfl_xor_sync(0xffffffffu, lo(sums[n][q]), o), __shfl_xor_sync(0xffffffffu, hi(sums[n][q]), o));
        if (lane < team) {
#pragma unroll
            for (int q = 0; q < E; ++q)
                if (IO::col(q, k, team) < w) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) acc[(warp * 4 + n) * w + IO::col(q, k, team)] = q & 1 ? hi(sums[n][q / 2]) : lo(sums[n][q / 2]);
                }
        }
        __syncthreads();
        for (unsigned c = threadIdx.x; c < 4 * w; c += blockDim.x) {
            float s = 0.f;
            for (unsigned v = 0; v < nw; ++v) s += acc[v * 4 * w + c];
            const unsigned n = c / w;
            if (float *o = target(n)) o[c - n * w] = s;
        }
    }
    if constexpr (IN_SMEM) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 4; ++n)
            if (float *o = target(n))
                for (unsigned c = threadIdx.x; c < w; c += blockDim.x) o[c] = acc[n * w + c];
    }
    if (a.join) {                                    // few CTAs: no second launch
        __syncthreads();
        if (gridDim.x > 1) sm100::cluster_sync_all();       // what the others wrote is there
        finish_flat(a.fin, alone ? a.fin.n_out : 0, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
    }
}

// Many rows an output: a CTA takes 32 columns of it, its 32 warps sum every 32nd row each, then the 32 in a tree.  The
// gate's groups of up to 64 runs: a thread a column (`flat` CTAs, behind the others).
__global__ void __launch_bounds__(1024) k_rn_finish(const FinishArgs f) {
    after_previous();
    __shared__ float sum[32][33];
    const unsigned tree = gridDim.x - f.flat, jobs = f.n_out + (f.flat ? 0 : f.groups), blocks = (f.w + 31) / 32;
    if (blockIdx.x >= tree) {
        finish_flat(f, f.n_out, (blockIdx.x - tree) * 1024ull + threadIdx.x, f.flat * 1024ull);
        before_next();
        return;
    }
    const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (unsigned long long unit = blockIdx.x; unit < (unsigned long long)jobs * blocks; unit += tree) {
        const unsigned job = (unsigned)(unit / blocks), c0 = (unsigned)(unit - (unsigned long long)job * blocks) * 32, c = c0 + lane;
        const FinishJob j(f, job);
        float s = 0.f;
        if (c < f.w) {
#pragma unroll 8
            for (unsigned r = warp; r < j.rows; r += 32) s += j.src[r * j.stride + c];
        }
        sum[warp][lane] = s;
        __syncthreads();
        s = warp_sum(sum[lane][warp]);               // column `warp`
        if (lane == 0 && c0 + warp < f.w) j.put(f, c0 + warp, s);
        __syncthreads();
    }
    before_next();
}

// ------------------------------------------------------------------ host side

// Threads of a row and of a CTA.
struct RnShape {
    bool wide;
    int e, team, threads;
};
struct RnPlan {
    bool vec, join;
    RnShape fwd, bwd;
    int crew, ctas_fwd, ctas_bwd;
    unsigned run, runs_per_group, runs;
    size_t parts, gparts, total;      // workspace offsets
};

// e elements a thread; a team is the smallest power of two that holds a row.
static RnShape rn_shape(int w, int e) {
    RnShape p;
    p.e = e;
    const int slots = (w + e - 1) / e;
    p.team = 1;
    while (p.team < slots) p.team <<= 1;
    p.wide = p.team > 32;
    p.threads = p.wide ? p.team : 256;
    return p;
}

// Elements a thread: 8, so that up to 256 elements stay in a warp; 16 for rows beyond 4096 elements (a CTA of 512
// threads then has the registers for the backward), forward in bf16 beyond 2048 (three CTAs of 256 threads an SM hide
// each other's sums better than two of 512: 8192 x 4096 rms).
static RnPlan rn_plan(const eaga_residual_norm_dims &d) {
    RnPlan p;
    const int es = d.dtype == EAGA_BF16 ? 2 : 4;
    p.vec = (long long)d.w * es % 16 == 0;
    p.bwd = rn_shape(d.w, d.w > 4096 ? 16 : 8);
    p.fwd = rn_shape(d.w, d.w > (p.vec && es == 2 ? 2048 : 4096) ? 16 : 8);
    const long long rows = d.rows, sms = sm_count();
    const long long per_fwd = p.fwd.wide ? 1 : p.fwd.threads / p.fwd.team;
    const long long each = p.fwd.threads == 256 && (p.fwd.e > 8 || !p.fwd.wide) ? 3 : p.fwd.e > 8 ? 1 : 1024 / p.fwd.threads;    // CTAs an SM
    p.ctas_fwd = (int)std::max(1LL, std::min((rows + per_fwd - 1) / per_fwd, sms * each));
    // Backward.  A run costs a partial row of the gate's gradient, a CTA one of each parameter's: runs of two rows a team
    // (four a CTA) or more (up to 64 rows, whose masks a warp holds), long inputs RN_ROUNDS or more a crew.
    const RnShape &b = p.bwd;
    p.crew = b.wide ? b.team : d.rows_per_group >= 2 * 32 / b.team ? 32 : b.team;
    const long long abreast = p.crew / b.team, crews = b.threads / p.crew, room = sms * (512 / b.threads);    // 512 threads an SM
    long long want = std::max((b.wide ? 4 : 2) * abreast, (rows + room * crews - 1) / (room * crews));
    const long long most = b.wide ? 64 : std::max(abreast, std::min(64LL, 16 * abreast) / abreast * abreast);
    if (want > 4 * abreast) want = std::max(std::min(most, 4 * abreast), std::min(most, (rows + RN_ROUNDS * room * crews - 1) / (RN_ROUNDS * room * crews)));
    want = std::min(want, most);
    const long long parts = std::max(1LL, (d.rows_per_group + want - 1) / want);
    p.run = (unsigned)(((d.rows_per_group + parts - 1) / parts + abreast - 1) / abreast * abreast);
    p.runs_per_group = (unsigned)((d.rows_per_group + p.run - 1) / p.run);
    p.runs = (unsigned)(rows / d.rows_per_group * p.runs_per_group);
    p.ctas_bwd = (int)std::max(1LL, std::min((p.runs + crews - 1) / crews, room));
    p.join = p.ctas_bwd <= 8;                        // a cluster: 1, 2, 4 or 8 CTAs
    while (p.join && (p.ctas_bwd & (p.ctas_bwd - 1))) ++p.ctas_bwd;
    p.parts = 0;
    p.gparts = align256((size_t)p.ctas_bwd * 4 * d.w * 4);
    p.total = p.gparts + (p.runs_per_group > 1 ? align256((size_t)p.runs * d.w * 4) : 0);
    return p;
}

template <bool FWD, typename F>
static cudaError_t rn_dispatch(const eaga_residual_norm_dims &d, const RnPlan &p, F &&f) {
    using bf = __nv_bfloat16;
    const RnShape &sh = FWD ? p.fwd : p.bwd;
    auto pick = [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr int V = decltype(vec)::value;
        auto go = [&](auto e, auto wide, auto maxt) { return f(T{}, std::integral_constant<int, V>{}, e, wide, maxt); };
        constexpr std::integral_constant<int, 8> e8{};
        constexpr std::integral_constant<int, 16> e16{};
        constexpr std::integral_constant<int, 256> t256{};
        constexpr std::integral_constant<int, 512> t512{};
        if constexpr (FWD && V == 8) {
            if (sh.e == 16 && sh.threads <= 256) return go(e16, std::true_type{}, t256);
        }
        if (sh.e == 16) return go(e16, std::true_type{}, t512);
        if constexpr (!(FWD && V == 8)) {
            if (sh.threads > 256) return go(e8, std::true_type{}, t512);
        }
        return sh.wide ? go(e8, std::true_type{}, t256) : go(e8, std::false_type{}, t256);
    };
    if (d.dtype == EAGA_BF16)
        return p.vec ? pick(bf{}, std::integral_constant<int, 8>{}) : pick(bf{}, std::integral_constant<int, 1>{});
    return p.vec ? pick(float{}, std::integral_constant<int, 4>{}) : pick(float{}, std::integral_constant<int, 1>{});
}

static eaga_status rn_check(const eaga_residual_norm_dims *d) {
    if (!d || d->rows < 0 || d->w < 1 || d->rows_per_group < 1) return EAGA_ERR_INVALID_ARG;
    if (d->dtype != EAGA_FP32 && d->dtype != EAGA_BF16) return EAGA_ERR_INVALID_ARG;
    for (int k : {d->pre, d->post})
        if (k != RN_NONE && k != RN_LAYER && k != RN_RMS) return EAGA_ERR_INVALID_ARG;
    if (!(d->eps > 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->alpha)) return EAGA_ERR_INVALID_ARG;
    if (d->rows % d->rows_per_group) return EAGA_ERR_INVALID_ARG;
    if (d->w > 8192 || d->rows > 0x7fff0000LL || d->rows_per_group > 0x7fff0000LL) return EAGA_ERR_UNSUPPORTED;
    return EAGA_OK;
}

static RnArgs rn_args(const eaga_residual_norm_dims &d, const RnPlan &p, const RnShape &sh) {
    RnArgs a = {};
    a.alpha = d.alpha; a.eps = d.eps; a.inv_w = 1.f / (float)d.w;
    a.rows = (unsigned)d.rows; a.w = (unsigned)d.w; a.group = (unsigned)d.rows_per_group;
    a.run = p.run; a.runs_per_group = p.runs_per_group; a.runs = p.runs;
    a.pre = d.pre; a.post = d.post; a.team = sh.team; a.crew = p.crew;
    return a;
}

// A norm's gain or shift is given only where the norm is there.
static eaga_status rn_params(const eaga_residual_norm_dims &d, const void *post_g, const void *post_s,
                             const void *pre_g, const void *pre_s) {
    if ((d.post == RN_NONE && (post_g || post_s)) || (d.pre == RN_NONE && (pre_g || pre_s))) return EAGA_ERR_INVALID_ARG;
    return EAGA_OK;
}

}  // namespace ops
}  // namespace eaga

using namespace eaga;
using namespace eaga::ops;

extern "C" {

size_t eaga_residual_norm_workspace_size(const eaga_residual_norm_dims *d) {
    if (rn_check(d) != EAGA_OK) return 0;
    return std::max<size_t>(256, rn_plan(*d).total);
}

eaga_status eaga_residual_norm_forward(const eaga_residual_norm_dims *d, const void *x, const void *u,
                                       const uint8_t *M, const void *gate, const void *post_g, const void *post_s,
                                       const void *pre_g, const void *pre_s, void *r, void *h, void *stream) {
    eaga_status s = rn_check(d);
    if (s != EAGA_OK) return s;
    if ((s = rn_params(*d, post_g, post_s, pre_g, pre_s)) != EAGA_OK) return s;
    if (d->rows == 0) return EAGA_OK;       // tensors without rows have no address
    if ((d->pre == RN_NONE) != (h == nullptr) || (!r && !h) || !u) return EAGA_ERR_INVALID_ARG;
    for (const void *q : {x, u, gate, post_g, post_s, pre_g, pre_s, (const void *)r, (const void *)h, (const void *)M})
        if (bad_align16(q)) return EAGA_ERR_MISALIGNED;
    {
        const size_t es = d->dtype == EAGA_BF16 ? 2 : 4, n = (size_t)d->rows * d->w * es, w = (size_t)d->w * es;
        auto span = [](const void *q, size_t b) { return Span{q, q ? b : 0}; };
        const Span outs[2] = {span(r, n), span(h, n)};
        const Span ins[8] = {span(x, n), span(u, n), span(M, (size_t)d->rows), span(gate, n / d->rows_per_group),
                             span(post_g, w), span(post_s, w), span(pre_g, w), span(pre_s, w)};
        if ((s = check_no_alias(outs, 2, ins, 8)) != EAGA_OK) return s;
    }
    const RnPlan p = rn_plan(*d);
    RnArgs a = rn_args(*d, p, p.fwd);
    a.x = x; a.u = u; a.M = M; a.gate = gate;
    a.post_g = post_g; a.post_s = post_s; a.pre_g = pre_g; a.pre_s = pre_s;
    a.r = r; a.h = h;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = rn_dispatch<true>(*d, p, [&](auto t, auto vec, auto el, auto wide, auto maxt) {
        return launch_pdl(k_rn_fwd<decltype(t), decltype(vec)::value, decltype(el)::value, decltype(wide)::value, decltype(maxt)::value>,
                          dim3(p.ctas_fwd), dim3(p.fwd.threads), 0, st, 1, a);
    });
    return e == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

eaga_status eaga_residual_norm_backward(const eaga_residual_norm_dims *d, const void *r, const void *u,
                                        const uint8_t *M, const void *gate, const void *post_g, const void *post_s,
                                        const void *pre_g, const void *dr, const void *dh, void *dx, void *du,
                                        void *dgate, float *dpost_g, float *dpost_s, float *dpre_g, float *dpre_s,
                                        void *workspace, size_t ws_bytes, void *stream) {
    eaga_status s = rn_check(d);
    if (s != EAGA_OK) return s;
    if ((s = rn_params(*d, post_g, post_s, pre_g, nullptr)) != EAGA_OK) return s;
    const bool has_pre = d->pre != RN_NONE, has_post = d->post != RN_NONE;
    if (!workspace || (dh && !has_pre)) return EAGA_ERR_INVALID_ARG;
    if (((dpost_g || dpost_s) && !has_post) || ((dpre_g || dpre_s) && !has_pre)) return EAGA_ERR_INVALID_ARG;
    if (d->rows > 0) {
        if ((!dr && !dh) || (has_pre && (!dh || !r)) || (dgate && !gate) || ((has_post || gate) && !u))
            return EAGA_ERR_INVALID_ARG;
    }
    for (const void *q : {r, u, gate, post_g, post_s, pre_g, dr, dh, (const void *)dx, (const void *)du,
                          (const void *)dgate, (const void *)M, (const void *)dpost_g, (const void *)dpost_s,
                          (const void *)dpre_g, (const void *)dpre_s, (const void *)workspace})
        if (bad_align16(q)) return EAGA_ERR_MISALIGNED;
    const RnPlan p = rn_plan(*d);
    const size_t need = std::max<size_t>(256, p.total);
    {
        const size_t es = d->dtype == EAGA_BF16 ? 2 : 4, n = (size_t)d->rows * d->w * es, w = (size_t)d->w * es;
        const size_t ng = n / d->rows_per_group, wf = (size_t)d->w * 4;
        auto span = [](const void *q, size_t b) { return Span{q, q ? b : 0}; };
        const Span outs[8] = {span(dx, n), span(du, n), span(dgate, ng), span(dpost_g, wf), span(dpost_s, wf),
                              span(dpre_g, wf), span(dpre_s, wf), span(workspace, need)};
        const Span ins[9] = {span(r, n), span(u, n), span(M, (size_t)d->rows), span(gate, ng), span(post_g, w),
                             span(post_s, w), span(pre_g, w), span(dr, n), span(dh, n)};
        if ((s = check_no_alias(outs, 8, ins, 9)) != EAGA_OK) return s;
    }
    if (ws_bytes < need) return EAGA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    RnArgs a = rn_args(*d, p, p.bwd);
    a.u = u; a.M = M; a.gate = gate; a.post_g = post_g; a.post_s = post_s; a.pre_g = pre_g;
    a.rin = r; a.dr = dr; a.dh = dh; a.dx = dx; a.du = du; a.dgate = dgate;
    char *ws = static_cast<char *>(workspace);
    a.parts = reinterpret_cast<float *>(ws + p.parts);
    a.gparts = reinterpret_cast<float *>(ws + p.gparts);
    FinishArgs f = {};
    float *const out[4] = {dpost_g, dpost_s, dpre_g, dpre_s};
    for (int k = 0; k < 4; ++k)
        if (out[k]) {
            f.out[f.n_out] = out[k];
            f.which[f.n_out++] = k;
        }
    for (int k = 0; k < 4; ++k) f.all[k] = out[k];
    f.groups = dgate && p.runs_per_group > 1 ? (unsigned)(d->rows / d->rows_per_group) : 0;
    f.parts = a.parts; f.gparts = a.gparts; f.dgate = dgate;
    f.w = a.w; f.ctas = p.ctas_bwd; f.runs_per_group = p.runs_per_group; f.dtype = d->dtype;
    a.fin = f;
    a.join = p.join && f.n_out + f.groups > 0;
    cudaError_t e = rn_dispatch<false>(*d, p, [&](auto t, auto vec, auto el, auto wide, auto maxt) {
        constexpr int E = decltype(el)::value;
        constexpr bool AHEAD = decltype(vec)::value == 8 && E == 8;
        const size_t sums = decltype(wide)::value ? (E == 8 ? 0 : (size_t)4 * d->w * 4) : (size_t)p.bwd.threads / 32 * 4 * d->w * 4;
        const size_t smem = std::max(sums, AHEAD ? (size_t)RN_DEPTH * 5 * 16 * p.bwd.threads : 0);
        auto kernel = k_rn_bwd<decltype(t), decltype(vec)::value, E, decltype(wide)::value, decltype(maxt)::value>;
        if (E > 8 || AHEAD) {
            static std::atomic<uint32_t> attr_set{0};
            const int most = E > 8 ? 4 * 8192 * 4 : RN_DEPTH * 5 * 16 * decltype(maxt)::value;
            if (cudaError_t err = ensure_smem_attr(kernel, most, attr_set); err != cudaSuccess) return err;
        }
        return launch_pdl(kernel, dim3(p.ctas_bwd), dim3(p.bwd.threads), smem, st, a.join ? p.ctas_bwd : 1, a);
    });
    if (e != cudaSuccess) return EAGA_ERR_CUDA;
    if (a.join || f.n_out + f.groups == 0) return EAGA_OK;
    const unsigned long long cols = (a.w + 31) / 32, most = 2ull * sm_count();
    if (f.groups && f.runs_per_group <= 64) f.flat = (unsigned)std::min(most, ((unsigned long long)f.groups * f.w + 1023) / 1024);
    const unsigned long long units = (f.n_out + (f.flat ? 0ull : f.groups)) * cols;
    const unsigned grid = (unsigned)std::min(units, 1ull << 20) + f.flat;
    return launch_pdl(k_rn_finish, dim3(grid), dim3(1024), 0, st, 1, f) == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

}  // extern "C"
