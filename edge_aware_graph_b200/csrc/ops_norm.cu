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
    int pre, post, team;       // threads that hold a row
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
    static __device__ __forceinline__ void values(const Raw &r, float (&v)[E]) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if constexpr (VEC == 1) {
                v[n] = ldf(&r.v[n]);
            } else {
                const unsigned x[4] = {r.v[n].x, r.v[n].y, r.v[n].z, r.v[n].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(T) == 4) {
                        v[4 * n + j] = __uint_as_float(x[j]);
                    } else {
                        v[8 * n + 2 * j] = __uint_as_float(x[j] << 16);
                        v[8 * n + 2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
                    }
                }
            }
        }
    }
    static __device__ __forceinline__ void load(const T *p, unsigned k, unsigned team, unsigned w, float (&v)[E]) {
        Raw r;
        fetch(p, true, k, team, w, r);
        values(r, v);
    }
    static __device__ __forceinline__ void store(T *p, unsigned k, unsigned team, unsigned w, const float (&v)[E]) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const unsigned c = (k + n * team) * VEC;
            if (c >= w) continue;
            if constexpr (VEC == 1) {
                stf(p + c, v[n]);
            } else if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4 *>(p + c) = make_float4(v[4 * n], v[4 * n + 1], v[4 * n + 2], v[4 * n + 3]);
            } else {
                uint4 o;
                __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = __floats2bfloat162_rn(v[8 * n + 2 * j], v[8 * n + 2 * j + 1]);
                *reinterpret_cast<uint4 *>(p + c) = o;
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
    const unsigned span = WIDE ? 32u : team;
    for (unsigned o = span >> 1; o; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) a[n] += __shfl_xor_sync(0xffffffffu, a[n], o);
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
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            a[n] = s;
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

// What a thread keeps beside the row it works on.  AHEAD: the next row, as it
// lies in memory (4 registers a tensor for 8 bf16 elements, where there is room
// for them).  KEEP: the norms' gains and shifts; teams of a CTA's size read
// those from L1 again, and run two CTAs an SM instead.
template <int VEC, int E, bool WIDE>
struct RnKeep {
    static constexpr bool AHEAD = VEC == 8 && E == 8, KEEP = AHEAD && !WIDE;
};

template <typename T, int VEC, int E, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, E > 8 ? 1 : WIDE ? 1024 / MAXT : 3)
k_rn_fwd(const RnArgs a) {
    using IO = RowIo<T, VEC, E>;
    using Raw = typename IO::Raw;
    constexpr bool AHEAD = RnKeep<VEC, E, WIDE>::AHEAD, KEEP = RnKeep<VEC, E, WIDE>::KEEP;
    __shared__ float buf[2][4][32];
    unsigned turn = 0;
    const unsigned w = a.w, team = a.team;
    const Team tm = my_team<WIDE>(team);
    bool on_v[IO::NV];                               // a vector is in the row, or none of it
#pragma unroll
    for (int n = 0; n < IO::NV; ++n) on_v[n] = IO::col(n * VEC, tm.k, team) < w;
    auto on = [&](int q) { return on_v[q / VEC]; };
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
        IO::fetch(gate + (size_t)((live ? row : 0) / a.group) * w, live && gate, tm.k, team, w, ng);
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
        float p[E];
        IO::values(nu, p);
        const Raw rx = nx, rg = ng;
        if (AHEAD) {
            ask(row + tm.count, next);
            live = next;
            next = alive(row + 2 * tm.count);
        }
        if (WIDE && !now) {                         // the whole CTA holds this row
#pragma unroll
            for (int q = 0; q < E; ++q) p[q] = 0.f;
            if (r) IO::store(r + at, tm.k, team, w, p);
            if (h) IO::store(h + at, tm.k, team, w, p);
            continue;
        }
        auto values_of = [&](auto which, float (&c)[E]) {
            constexpr int P = decltype(which)::value;
            if constexpr (KEEP) IO::values(kept[P], c);
            else IO::load(param[P], tm.k, team, w, c);
        };
        auto norm = [&](float (&v)[E], int kind, auto first) {       // parameters `first` (gain) and the next (shift)
            if (kind == RN_NONE) return;
            constexpr int P = decltype(first)::value;
            float s[1];
            if (kind == RN_LAYER) {
                s[0] = 0.f;
#pragma unroll
                for (int q = 0; q < E; ++q) s[0] += v[q];
                team_sum<WIDE, 1>(s, team, buf, turn);
                const float mean = s[0] * a.inv_w;
#pragma unroll
                for (int q = 0; q < E; ++q) v[q] = on(q) ? v[q] - mean : 0.f;
            }
            s[0] = 0.f;
#pragma unroll
            for (int q = 0; q < E; ++q) s[0] += v[q] * v[q];
            team_sum<WIDE, 1>(s, team, buf, turn);
            const float rstd = rsqrtf(s[0] * a.inv_w + a.eps);
            float c[E];
            if (param[P]) {
                values_of(first, c);
#pragma unroll
                for (int q = 0; q < E; ++q) v[q] *= rstd * c[q];
            } else {
#pragma unroll
                for (int q = 0; q < E; ++q) v[q] *= rstd;
            }
            if (param[P + 1]) {
                values_of(std::integral_constant<int, P + 1>{}, c);
#pragma unroll
                for (int q = 0; q < E; ++q) v[q] += c[q];
            }
        };
        norm(p, a.post, std::integral_constant<int, 0>{});
        if (gate) {
            float c[E];
            IO::values(rg, c);
#pragma unroll
            for (int q = 0; q < E; ++q) p[q] *= c[q];
        }
        if (x) {
            float t[E];
            IO::values(rx, t);
#pragma unroll
            for (int q = 0; q < E; ++q) p[q] += a.alpha * t[q];
        }
        if (!now) {
#pragma unroll
            for (int q = 0; q < E; ++q) p[q] = 0.f;
        }
        if (r && in) IO::store(r + at, tm.k, team, w, p);
        if (!h) continue;
        norm(p, a.pre, std::integral_constant<int, 2>{});
        if (!now) {
#pragma unroll
            for (int q = 0; q < E; ++q) p[q] = 0.f;
        }
        if (in) IO::store(h + at, tm.k, team, w, p);
    }
}

// A team takes runs of consecutive rows of one group (a run is the whole group
// or a part of it), a row a step; every team of the launch takes the same number
// of steps.  While a row is worked on, the next one's elements are on their way
// into registers (as they lie in memory: 4 registers a tensor), and the mask of
// the row after that.
template <typename T, int VEC, int E, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT)
k_rn_bwd(const RnArgs a) {
    using IO = RowIo<T, VEC, E>;
    using Raw = typename IO::Raw;
    constexpr bool AHEAD = RnKeep<VEC, E, WIDE>::AHEAD, KEEP = RnKeep<VEC, E, WIDE>::KEEP;
    __shared__ float buf[2][4][32];
    unsigned turn = 0;
    const unsigned w = a.w, team = a.team;
    const Team tm = my_team<WIDE>(team);
    bool on_v[IO::NV];                               // a vector is in the row, or none of it
#pragma unroll
    for (int n = 0; n < IO::NV; ++n) on_v[n] = IO::col(n * VEC, tm.k, team) < w;
    auto on = [&](int q) { return on_v[q / VEC]; };
    const T *u = static_cast<const T *>(a.u), *rin = static_cast<const T *>(a.rin), *dr = static_cast<const T *>(a.dr),
            *dh = static_cast<const T *>(a.dh), *gate = static_cast<const T *>(a.gate);
    T *dx = static_cast<T *>(a.dx), *du = static_cast<T *>(a.du);
    const bool need_u = gate != nullptr || a.post != RN_NONE, has_pre = a.pre != RN_NONE;
    // Sums of the gains' and shifts' gradients, post then pre: in registers, or, where a thread holds 16 columns
    // and they would not fit, in shared memory (each thread its own columns).
    constexpr bool IN_SMEM = E > 8;
    extern __shared__ float acc[];                   // [4][w]
    float sums[4][IN_SMEM ? 1 : E];
    if constexpr (IN_SMEM) {
        for (unsigned c = threadIdx.x; c < 4 * w; c += blockDim.x) acc[c] = 0.f;
        __syncthreads();
    } else {
#pragma unroll
        for (int q = 0; q < E; ++q) sums[0][q] = sums[1][q] = sums[2][q] = sums[3][q] = 0.f;
    }
    auto add = [&](auto which, int q, float v) {
        constexpr int P = decltype(which)::value;
        if constexpr (IN_SMEM) {
            if (on(q)) acc[P * w + IO::col(q, tm.k, team)] += v;
        } else {
            sums[P][q] += v;
        }
    };
    Raw pre_g, post_g;
    if (KEEP) {
        IO::fetch(static_cast<const T *>(a.pre_g), a.pre_g, tm.k, team, w, pre_g);
        IO::fetch(static_cast<const T *>(a.post_g), a.post_g, tm.k, team, w, post_g);
    }
    auto gain_of = [&](const void *p, const Raw &kept, float (&c)[E]) {
        if constexpr (KEEP) IO::values(kept, c);
        else IO::load(static_cast<const T *>(p), tm.k, team, w, c);
    };

    // A place in the team's sequence of rows.
    struct Place {
        unsigned run, i, row0, n;                    // the run, the row in it, the run's first row and number of rows
        bool in;
    };
    auto enter = [&](Place &p) {                     // the run's rows
        if (p.run < a.runs) {
            const unsigned grp = p.run / a.runs_per_group, part = p.run - grp * a.runs_per_group;
            p.row0 = grp * a.group + part * a.run;
            p.n = min(a.run, a.group - part * a.run);
        } else {
            p.row0 = p.n = 0;
        }
    };
    auto forward = [&](Place &p) {
        if (++p.i == a.run) {
            p.i = 0;
            p.run = a.runs - p.run > tm.count && p.run < a.runs ? p.run + tm.count : a.runs;
            enter(p);
        }
        p.in = p.i < p.n;
    };
    auto alive = [&](const Place &p) { return p.in && (!a.M || a.M[p.row0 + p.i]); };
    Raw n_dr, n_dh, n_r, n_u, n_gate;
    auto ask = [&](const Place &p, bool live) {
        const size_t at = (size_t)(live ? p.row0 + p.i : 0) * w;
        IO::fetch(dr + at, live && dr, tm.k, team, w, n_dr);
        IO::fetch(dh + at, live && has_pre, tm.k, team, w, n_dh);
        IO::fetch(rin + at, live && has_pre, tm.k, team, w, n_r);
        IO::fetch(u + at, live && need_u, tm.k, team, w, n_u);
    };
    auto ask_gate = [&](const Place &p) {
        if (p.i == 0) IO::fetch(gate + (size_t)(p.run < a.runs ? p.run / a.runs_per_group : 0) * w, gate, tm.k, team, w, n_gate);
    };
    Place at0 = {tm.id, 0, 0, 0, false};
    enter(at0);
    at0.in = at0.n > 0;
    Place at1 = at0;
    if (AHEAD) forward(at1);
    bool live0 = alive(at0), live1 = AHEAD && alive(at1);
    if (AHEAD) ask(at0, live0);
    ask_gate(at0);
    Raw gt = n_gate;
    float s_gate[E];
    const unsigned steps = WIDE ? (tm.id < a.runs ? (a.runs - tm.id + tm.count - 1) / tm.count : 0)
                                : (a.runs + tm.count - 1) / tm.count;
    for (unsigned long long left = (unsigned long long)steps * a.run; left; --left) {
        const Place here = at0;
        if (!AHEAD) {
            live0 = alive(here);
            ask(here, live0);
            ask_gate(here);
        }
        const bool in = here.in, live = live0;
        const size_t at = (size_t)(in ? here.row0 + here.i : 0) * w;
        if (here.i == 0) {
            gt = n_gate;
#pragma unroll
            for (int q = 0; q < E; ++q) s_gate[q] = 0.f;
        }
        const Raw c_dr = n_dr, c_dh = n_dh, c_r = n_r, c_u = n_u;
        if (AHEAD) {
            ask(at1, live1);
            ask_gate(at1);
            at0 = at1;
            live0 = live1;
            forward(at1);
            live1 = alive(at1);
        } else {
            forward(at0);
        }
        if (WIDE ? !live : !__any_sync(0xffffffffu, live)) {
            float z[E];
#pragma unroll
            for (int q = 0; q < E; ++q) z[q] = 0.f;
            if (in && dx) IO::store(dx + at, tm.k, team, w, z);
            if (in && du) IO::store(du + at, tm.k, team, w, z);
        } else {
            float g[E], d[E], z[E];
            IO::values(c_dr, g);
            // d becomes norm'(d; z), z is centred; returns 1 / deviation
            auto back = [&](float (&d)[E], float (&z)[E], int kind, const void *gain, const Raw &kept, auto first) {
                constexpr int P = decltype(first)::value;
                if (kind == RN_LAYER) {
                    float s[1] = {0.f};
#pragma unroll
                    for (int q = 0; q < E; ++q) s[0] += z[q];
                    team_sum<WIDE, 1>(s, team, buf, turn);
                    const float mean = s[0] * a.inv_w;
#pragma unroll
                    for (int q = 0; q < E; ++q) z[q] = on(q) ? z[q] - mean : 0.f;
                }
                float e[E];
                if (gain) {
                    gain_of(gain, kept, e);
#pragma unroll
                    for (int q = 0; q < E; ++q) e[q] *= d[q];
                } else {
#pragma unroll
                    for (int q = 0; q < E; ++q) e[q] = d[q];
                }
                float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < E; ++q) {
                    s[0] += z[q] * z[q];
                    s[1] += e[q] * z[q];
                    s[2] += e[q];
                }
                team_sum<WIDE, 3>(s, team, buf, turn);
                const float rstd = rsqrtf(s[0] * a.inv_w + a.eps);
                const float c1 = s[1] * a.inv_w * rstd * rstd, c2 = kind == RN_LAYER ? s[2] * a.inv_w : 0.f;
#pragma unroll
                for (int q = 0; q < E; ++q) {
                    add(std::integral_constant<int, P>{}, q, d[q] * (z[q] * rstd));
                    add(std::integral_constant<int, P + 1>{}, q, d[q]);
                    d[q] = (e[q] - c2 - z[q] * c1) * rstd;
                }
                return rstd;
            };
            if (has_pre) {
                IO::values(c_dh, d);
                IO::values(c_r, z);
                back(d, z, a.pre, a.pre_g, pre_g, std::integral_constant<int, 2>{});
#pragma unroll
                for (int q = 0; q < E; ++q) g[q] = live ? g[q] + d[q] : 0.f;
            }
            if (dx && in) {
#pragma unroll
                for (int q = 0; q < E; ++q) z[q] = a.alpha * g[q];
                IO::store(dx + at, tm.k, team, w, z);
            }
            if (gate) {
                IO::values(gt, d);
#pragma unroll
                for (int q = 0; q < E; ++q) d[q] *= g[q];
            } else {
#pragma unroll
                for (int q = 0; q < E; ++q) d[q] = g[q];
            }
            IO::values(c_u, z);
            if (a.post != RN_NONE) {
                const float rstd = back(d, z, a.post, a.post_g, post_g, std::integral_constant<int, 0>{});
                if (gate) {                          // p = gain zh + shift; z is centred
                    float c[E];
                    if (a.post_g) {
                        gain_of(a.post_g, post_g, c);
#pragma unroll
                        for (int q = 0; q < E; ++q) z[q] *= rstd * c[q];
                    } else {
#pragma unroll
                        for (int q = 0; q < E; ++q) z[q] *= rstd;
                    }
                    if (a.post_s) {
                        IO::load(static_cast<const T *>(a.post_s), tm.k, team, w, c);
#pragma unroll
                        for (int q = 0; q < E; ++q) z[q] += c[q];
                    }
                }
            }
            if (gate) {
#pragma unroll
                for (int q = 0; q < E; ++q) s_gate[q] += g[q] * z[q];
            }
            if (du && in) {
                if (!live) {
#pragma unroll
                    for (int q = 0; q < E; ++q) d[q] = 0.f;
                }
                IO::store(du + at, tm.k, team, w, d);
            }
        }
        if (here.i == a.run - 1 && a.dgate && here.run < a.runs) {
            if (a.runs_per_group == 1) {
                IO::store(static_cast<T *>(a.dgate) + (size_t)here.run * w, tm.k, team, w, s_gate);
            } else {
                float *o = a.gparts + (size_t)here.run * w;
#pragma unroll
                for (int q = 0; q < E; ++q)
                    if (on(q)) o[IO::col(q, tm.k, team)] = s_gate[q];
            }
        }
    }
    // The CTA's sums: its warps' teams by shuffles (same columns), the warps one after another.
    float *out = a.parts + (size_t)blockIdx.x * 4 * w;
    if constexpr (WIDE && !IN_SMEM) {
#pragma unroll
        for (int q = 0; q < E; ++q)
            if (on(q)) {
#pragma unroll
                for (int n = 0; n < 4; ++n) out[n * w + IO::col(q, tm.k, team)] = sums[n][q];
            }
    } else if constexpr (!IN_SMEM) {
        const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
        for (int q = 0; q < E; ++q)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                for (unsigned o = team; o < 32; o <<= 1) sums[n][q] += __shfl_xor_sync(0xffffffffu, sums[n][q], o);
        for (unsigned v = 0; v < nw; ++v) {
            if (warp == v && lane < team) {
#pragma unroll
                for (int q = 0; q < E; ++q)
                    if (on(q)) {
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            float &o = acc[n * w + IO::col(q, tm.k, team)];
                            o = (v ? o : 0.f) + sums[n][q];
                        }
                    }
            }
            __syncthreads();
        }
    }
    if constexpr (!WIDE || IN_SMEM) {
        __syncthreads();
        for (unsigned c = threadIdx.x; c < 4 * w; c += blockDim.x) out[c] = acc[c];
    }
}

// The partial rows' sums, in a fixed order.  A CTA takes 32 columns of one
// output: its 32 warps sum every 32nd row each, then the 32 in order.
// Outputs: the four parameters' gradients (`parts` CTA rows each), then the gate's groups.
struct FinishArgs {
    const float *parts, *gparts;
    float *out[4];
    void *dgate;
    unsigned w, ctas, groups, runs_per_group;
    int n_out, which[4], dtype;
};
__global__ void __launch_bounds__(1024) k_rn_finish(const FinishArgs f) {
    __shared__ float sum[32][33];
    const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    for (unsigned job = blockIdx.y; job < f.n_out + f.groups; job += gridDim.y) {
        const bool param = job < (unsigned)f.n_out;
        const unsigned rows = param ? f.ctas : f.runs_per_group;
        const size_t stride = param ? (size_t)4 * f.w : f.w;
        const float *src = param ? f.parts + (size_t)f.which[job] * f.w
                                 : f.gparts + (size_t)(job - f.n_out) * f.runs_per_group * f.w;
        float s = 0.f;
        if (c < f.w) {
#pragma unroll 8
            for (unsigned r = warp; r < rows; r += 32) s += src[r * stride + c];
        }
        sum[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && c < f.w) {
            s = 0.f;
#pragma unroll
            for (int v = 0; v < 32; ++v) s += sum[v][lane];
            if (param) f.out[job][c] = s;
            else if (f.dtype == EAGA_FP32) static_cast<float *>(f.dgate)[(size_t)(job - f.n_out) * f.w + c] = s;
            else static_cast<__nv_bfloat16 *>(f.dgate)[(size_t)(job - f.n_out) * f.w + c] = __float2bfloat16_rn(s);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host side

struct RnPlan {
    bool vec, wide;
    int e, team, threads, ctas_fwd, ctas_bwd;
    unsigned run, runs_per_group, runs;
    size_t parts, gparts, total;      // workspace offsets
};

// Elements a thread: 8, so that up to 256 elements stay in a warp; 16 for rows
// beyond 4096 elements (a CTA of 512 threads then has the registers for the
// backward).  A team is the smallest power of two that holds a row.
static RnPlan rn_plan(const eaga_residual_norm_dims &d) {
    RnPlan p;
    const int es = d.dtype == EAGA_BF16 ? 2 : 4;
    p.vec = (long long)d.w * es % 16 == 0;
    p.e = d.w > 4096 ? 16 : 8;
    const int slots = (d.w + p.e - 1) / p.e;
    p.team = 1;
    while (p.team < slots) p.team <<= 1;
    p.wide = p.team > 32;
    p.threads = p.wide ? p.team : 256;
    const long long per = p.wide ? 1 : p.threads / p.team;
    const long long rows = d.rows, sms = sm_count();
    const long long room = sms * (512 / p.threads);        // the registers: 512 threads an SM, 768 or 1024 forward
    p.ctas_fwd = (int)std::max(1LL, std::min((rows + per - 1) / per, p.wide ? sms * (p.e > 8 ? 1 : 1024 / p.threads) : sms * 3));
    p.ctas_bwd = (int)std::max(1LL, std::min((rows + per - 1) / per, room));
    // runs: at least about four for each team, of 16 rows or more where groups are that long
    const long long groups = std::max(1LL, rows / d.rows_per_group), teams = p.ctas_bwd * per;
    long long per_group = std::max(1LL, (4 * teams + groups - 1) / groups);
    per_group = std::max(1LL, std::min(per_group, (d.rows_per_group + 15) / 16));
    p.run = (unsigned)((d.rows_per_group + per_group - 1) / per_group);
    p.runs_per_group = (unsigned)((d.rows_per_group + p.run - 1) / p.run);
    p.runs = (unsigned)(rows / d.rows_per_group * p.runs_per_group);
    p.parts = 0;
    p.gparts = align256((size_t)p.ctas_bwd * 4 * d.w * 4);
    p.total = p.gparts + (p.runs_per_group > 1 ? align256((size_t)p.runs * d.w * 4) : 0);
    return p;
}

template <typename F>
static cudaError_t rn_dispatch(const eaga_residual_norm_dims &d, const RnPlan &p, F &&f) {
    using bf = __nv_bfloat16;
    auto pick = [&](auto t, auto vec) {
        using T = decltype(t);
        constexpr int V = decltype(vec)::value;
        auto go = [&](auto e, auto wide, auto maxt) { return f(T{}, std::integral_constant<int, V>{}, e, wide, maxt); };
        constexpr std::integral_constant<int, 8> e8{};
        constexpr std::integral_constant<int, 16> e16{};
        constexpr std::integral_constant<int, 256> t256{};
        constexpr std::integral_constant<int, 512> t512{};
        if (p.e == 16) return go(e16, std::true_type{}, t512);
        if (p.threads > 256) return go(e8, std::true_type{}, t512);
        return p.wide ? go(e8, std::true_type{}, t256) : go(e8, std::false_type{}, t256);
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
    if (d->w > 8192 || d->rows > 0x7fff0000LL) return EAGA_ERR_UNSUPPORTED;
    return EAGA_OK;
}

static RnArgs rn_args(const eaga_residual_norm_dims &d, const RnPlan &p) {
    RnArgs a = {};
    a.alpha = d.alpha; a.eps = d.eps; a.inv_w = 1.f / (float)d.w;
    a.rows = (unsigned)d.rows; a.w = (unsigned)d.w; a.group = (unsigned)d.rows_per_group;
    a.run = p.run; a.runs_per_group = p.runs_per_group; a.runs = p.runs;
    a.pre = d.pre; a.post = d.post; a.team = p.team;
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
    RnArgs a = rn_args(*d, p);
    a.x = x; a.u = u; a.M = M; a.gate = gate;
    a.post_g = post_g; a.post_s = post_s; a.pre_g = pre_g; a.pre_s = pre_s;
    a.r = r; a.h = h;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = rn_dispatch(*d, p, [&](auto t, auto vec, auto el, auto wide, auto maxt) {
        k_rn_fwd<decltype(t), decltype(vec)::value, decltype(el)::value, decltype(wide)::value, decltype(maxt)::value>
            <<<p.ctas_fwd, p.threads, 0, st>>>(a);
        return cudaGetLastError();
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
    RnArgs a = rn_args(*d, p);
    a.u = u; a.M = M; a.gate = gate; a.post_g = post_g; a.post_s = post_s; a.pre_g = pre_g;
    a.rin = r; a.dr = dr; a.dh = dh; a.dx = dx; a.du = du; a.dgate = dgate;
    char *ws = static_cast<char *>(workspace);
    a.parts = reinterpret_cast<float *>(ws + p.parts);
    a.gparts = reinterpret_cast<float *>(ws + p.gparts);
    cudaError_t e = rn_dispatch(*d, p, [&](auto t, auto vec, auto el, auto wide, auto maxt) {
        constexpr int E = decltype(el)::value;
        const size_t smem = decltype(wide)::value && E == 8 ? 0 : (size_t)4 * d->w * 4;
        auto kernel = k_rn_bwd<decltype(t), decltype(vec)::value, E, decltype(wide)::value, decltype(maxt)::value>;
        if (E > 8) {
            static std::atomic<uint32_t> attr_set{0};
            if (cudaError_t err = ensure_smem_attr(kernel, 4 * 8192 * 4, attr_set); err != cudaSuccess) return err;
        }
        kernel<<<p.ctas_bwd, p.threads, smem, st>>>(a);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return EAGA_ERR_CUDA;
    FinishArgs f = {};
    float *const out[4] = {dpost_g, dpost_s, dpre_g, dpre_s};
    for (int k = 0; k < 4; ++k)
        if (out[k]) {
            f.out[f.n_out] = out[k];
            f.which[f.n_out++] = k;
        }
    f.groups = dgate && p.runs_per_group > 1 ? (unsigned)(d->rows / d->rows_per_group) : 0;
    if (f.n_out + f.groups == 0) return EAGA_OK;
    f.parts = a.parts; f.gparts = a.gparts; f.dgate = dgate;
    f.w = a.w; f.ctas = p.ctas_bwd; f.runs_per_group = p.runs_per_group; f.dtype = d->dtype;
    const dim3 grid((a.w + 31) / 32, std::min(f.n_out + f.groups, 65535u));
    k_rn_finish<<<grid, 1024, 0, st>>>(f);
    return cudaGetLastError() == cudaSuccess ? EAGA_OK : EAGA_ERR_CUDA;
}

}  // extern "C"
