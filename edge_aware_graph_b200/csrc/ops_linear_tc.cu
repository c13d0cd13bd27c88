// The linear operator's products on tcgen05 (bf16 operands, fp32 sums):
//
//   forward   Y  = f(X W)      A = X  [rows, in]  K-major    B = W  [in, out]   MN-major (as stored)
//   dX        dX = f(dZ W^T)   A = dZ [rows, out] K-major    B = W  [in, out]   K-major  (the reduction is out)
//   dW        dW = X^T dZ      A = X  [rows, in]  MN-major   B = dZ [rows, out] MN-major (the reduction is rows)
//
// so every operand is read as it lies in memory.  A persistent CTA takes 128 x
// BN output tiles: a TMA warp fills a ring of 64-deep operand tiles (128-byte
// swizzled), one thread of the next warp issues the MMAs into one of two fp32
// accumulators in TMEM, and eight warps drain the other one, so the epilogue
// of a tile hides behind the next tile's products.  The drain goes through a
// small staging tile per warp, in fp32, so that bias, activation, residual and
// the stores see rows in 16-byte pieces, and every output is rounded once.
//
// A weight gradient reduces over rows, of which there may be a million for a
// 64 x 128 result: its tiles are split over rows, the splits' sums are added
// in a fixed order by the caller's reduction.  The bias gradient, the column
// sums of dZ, comes from the dZ tiles in shared memory: two more warps multiply
// them with a matrix of ones (warp-level MMAs, joined in fp32 after every 64 rows),
// in the CTAs of the first row of tiles, so dZ is not read again.
//
// An operand in fp32 comes as bf16 parts (two carry 16 bits of it, three 24):
// the products of parts are segments of one longer reduction, the smallest first.
#include <algorithm>
#include "ops_linear.h"
#include "sm100.cuh"

namespace eaga {
namespace fast {
bool encode_2d(CUtensorMap *m, const void *base, int rows, int cols, int box_rows);
}
namespace ops {

using namespace sm100;
using fast::dev::cta_wait;
typedef __nv_bfloat16 bf16;

constexpr int LT_BM = 128, LT_BK = 64;
constexpr int LT_EPI = 8;                              // epilogue warps: two a TMEM quadrant
constexpr int LT_THR = 32 * (4 + LT_EPI);              // TMA, MMA, two column-sum warps, epilogue

template <int BN>
struct LtSmem {
    static constexpr uint32_t A_BYTES = LT_BM * LT_BK * 2, B_BYTES = BN * LT_BK * 2, STAGE = A_BYTES + B_BYTES;
    static constexpr int ST = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr uint32_t EPI = ST * STAGE;                      // staging, 4 KB a warp
    static constexpr uint32_t BAR = EPI + LT_EPI * 4096;             // full[ST], empty[ST], acc_full[2], acc_empty[2], drained
    static constexpr uint32_t TM = BAR + (2 * ST + 5) * 8;
    static constexpr uint32_t FAIL = TM + 4;
    static constexpr uint32_t BYTES = FAIL + 12 + 1024;
    static_assert(BYTES <= 232448, "shared memory");
};

// Maps of the operands' parts.
struct LtMaps {
    CUtensorMap a[3], b[3];
};

template <typename TO>
struct LtParams {
    LinEpi<TO> e;
    float *acc, *db;           // weight gradient: fp32 sums [split][M][N], [split][N]
    int *status;
    int M, N;                  // output
    int kts;                   // forward, dX: 64-deep steps a segment; weight gradient: those of all rows
    int nseg;
    uint32_t seg;              // four bits a segment: A's part, B's part
    int tiles_m, tiles_n, units;
    int per;                   // weight gradient: a split's steps
    int vec, clear;
};

template <int KIND, int BN, typename TO>
__global__ void __launch_bounds__(LT_THR, 1)
k_lin_tc(const __grid_constant__ LtMaps maps, const LtParams<TO> p) {
    using S = LtSmem<BN>;
    constexpr int ST = S::ST;
    constexpr bool A_MN = KIND == LIN_DW, B_MN = KIND != LIN_DX;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *sp = smem_raw + (sbase - smem_u32(smem_raw));
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    volatile int *fail = reinterpret_cast<volatile int *>(sp + S::FAIL);
    const uint32_t bar0 = sbase + S::BAR;
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (ST + s); };
    auto acc_full = [&](int b) { return bar0 + 8 * (2 * ST + b); };
    auto acc_empty = [&](int b) { return bar0 + 8 * (2 * ST + 2 + b); };
    const uint32_t drained = bar0 + 8 * (2 * ST + 4);

    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), KIND == LIN_DW ? 3 : 1);     // the MMAs; two column-sum warps
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), LT_EPI);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
        *fail = 0;
        if (p.clear && blockIdx.x == 0) *p.status = 0;       // a wait that gives up does so a second later
    }
    if (w == 1) {
        tmem_alloc(sbase + S::TM, 2 * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sp + S::TM);

    // unit -> output tile (columns fastest), split, its steps
    struct Unit {
        int m0, n0, split, k0, steps, tm;
    };
    auto unit_of = [&](int u) {
        Unit r;
        const int tiles = p.tiles_m * p.tiles_n;
        r.split = KIND == LIN_DW ? u / tiles : 0;
        const int t = KIND == LIN_DW ? u % tiles : u;
        r.tm = t / p.tiles_n;
        r.m0 = r.tm * LT_BM;
        r.n0 = (t % p.tiles_n) * BN;
        r.k0 = KIND == LIN_DW ? r.split * p.per : 0;
        r.steps = KIND == LIN_DW ? min(p.per, p.kts - r.k0) : p.kts;
        return r;
    };

    if (w == 0) {
        if (lane == 0) {
            int it = 0, issued = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit t = unit_of(u);
                for (int seg = 0; ok && seg < p.nseg; ++seg) {
                    const uint32_t parts = p.seg >> (4 * seg);
                    const CUtensorMap *am = &maps.a[parts & 3], *bm = &maps.b[(parts >> 2) & 3];
                    for (int k = 0; k < t.steps; ++k, ++it) {
                        const int s = it % ST, kk = (t.k0 + k) * LT_BK;
                        if (!cta_wait(empty(s), ((it / ST) & 1) ^ 1, fail, p.status)) { ok = false; break; }
                        const uint32_t st = sbase + s * S::STAGE;
                        mbar_expect_tx(full(s), S::STAGE);
                        if constexpr (A_MN) {
                            tma_load_2d(st, am, full(s), t.m0, kk);
                            tma_load_2d(st + 8192, am, full(s), t.m0 + 64, kk);
                        } else {
                            tma_load_2d(st, am, full(s), kk, t.m0);
                        }
                        if constexpr (B_MN) {
#pragma unroll
                            for (int h = 0; h < BN / 64; ++h)
                                tma_load_2d(st + S::A_BYTES + h * 8192, bm, full(s), t.n0 + 64 * h, kk);
                        } else {
                            tma_load_2d(st + S::A_BYTES, bm, full(s), kk, t.n0);
                        }
                        issued = it + 1;
                    }
                }
            }
            if (!ok)                                // what was issued lands before the CTA's memory is released
                for (int i = max(issued - ST, 0); i < issued; ++i) mbar_wait(full(i % ST), (i / ST) & 1);
        }
    } else if (w == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(LT_BM, BN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            int it = 0, n = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x, ++n) {
                const Unit t = unit_of(u);
                const int b = n & 1, nk = t.steps * p.nseg;
                if (!cta_wait(acc_empty(b), ((n >> 1) & 1) ^ 1, fail, p.status)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + b * BN;
                const bool sums = KIND == LIN_DW && p.db != nullptr && t.tm == 0;
                for (int k = 0; k < nk; ++k, ++it) {
                    const int s = it % ST;
                    if (!cta_wait(full(s), (it / ST) & 1, fail, p.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t st = sbase + s * S::STAGE;
#pragma unroll
                    for (int kk = 0; kk < LT_BK / 16; ++kk)
                        mma_bf16_ss(d,
                                    A_MN ? smem_desc(st + kk * 2048, 8192, 1024, LAYOUT_SW128)
                                         : smem_desc(st + kk * 32, 16, 1024, LAYOUT_SW128),
                                    B_MN ? smem_desc(st + S::A_BYTES + kk * 2048, 8192, 1024, LAYOUT_SW128)
                                         : smem_desc(st + S::A_BYTES + kk * 32, 16, 1024, LAYOUT_SW128),
                                    idesc, (k > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(empty(s));
                    if (KIND == LIN_DW && !sums) {  // no column sums: their two arrivals
                        mbar_arrive(empty(s));
                        mbar_arrive(empty(s));
                    }
                }
                if (ok) mma_commit(acc_full(b));
            }
            if (!ok) {                              // the products in flight end before TMEM is freed
                mma_commit(drained);
                mbar_wait(drained, 0);
            }
        }
    } else if (w < 4) {
        if constexpr (KIND == LIN_DW) {
            // column sums of the dZ tile: ones [16 x 16] times [16 rows x 8 columns] at a time
            constexpr int COLS = BN / 2, NT = COLS / 8;        // this warp's columns
            const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
            const int c0 = (w - 2) * COLS;
            int it = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const Unit t = unit_of(u);
                const int nk = t.steps * p.nseg;
                if (p.db == nullptr || t.tm != 0) {
                    it += nk;
                    continue;
                }
                float sum[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[j][0] = sum[j][1] = 0.f;
                for (int k = 0; k < nk; ++k, ++it) {
                    const int s = it % ST;
                    ok = __all_sync(0xffffffffu, cta_wait(full(s), (it / ST) & 1, fail, p.status));
                    if (!ok) break;
                    const uint32_t bt = sbase + s * S::STAGE + S::A_BYTES;
#pragma unroll
                    for (int j = 0; j < NT; j += 2) {
                        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int kk = 0; kk < LT_BK; kk += 16) {
                            // four 8 x 8 matrices: rows kk.., kk + 8.. of columns j, then of columns j + 1
                            const uint32_t row = kk + (lane & 7) + 8 * ((lane >> 3) & 1), col = c0 + 8 * (j + (lane >> 4));
                            uint32_t f[4];
                            ldsm_x4_t(bt + (col >> 6) * 8192 + fast::sw128(row, (col >> 3) & 7), f);
                            mma16816(d0, ones, f[0], f[1]);
                            mma16816(d1, ones, f[2], f[3]);
                        }
                        sum[j][0] += d0[0]; sum[j][1] += d0[1];
                        sum[j + 1][0] += d1[0]; sum[j + 1][1] += d1[1];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty(s));
                }
                if (ok && lane < 4) {               // row 0 of the product: columns 2 lane, 2 lane + 1 of each 8
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int c = t.n0 + c0 + 8 * j + 2 * lane;
                        float *o = p.db + (size_t)t.split * p.N + c;
                        if (c < p.N) o[0] = sum[j][0];
                        if (c + 1 < p.N) o[1] = sum[j][1];
                    }
                }
                __syncwarp();
            }
        }
    } else {
        const int q = w & 3, half = (w - 4) >> 2;   // TMEM quadrant: rows 32 q ..; columns: every other 32
        const uint32_t stg = sbase + S::EPI + (w - 4) * 4096;
        const uint8_t *stage = sp + S::EPI + (w - 4) * 4096;
        int n = 0;
        for (int u = blockIdx.x; u < p.units; u += gridDim.x, ++n) {
            const Unit t = unit_of(u);
            const int b = n & 1;
            const bool ok = __all_sync(0xffffffffu, cta_wait(acc_full(b), (n >> 1) & 1, fail, p.status));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 32 * half; c0 < BN; c0 += 64) {
                __syncwarp();                       // lanes without columns are back; the last chunk's reads are done
                float v[32];
                const uint32_t ta = tmem + b * BN + ((uint32_t)(32 * q) << 16) + c0;
                tmem_ld16(ta, *reinterpret_cast<float(*)[16]>(v));
                tmem_ld16(ta + 16, *reinterpret_cast<float(*)[16]>(v + 16));
                tmem_ld_wait();
                if (c0 + 64 >= BN) {                // the last read: the accumulator may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty(b));
                }
                const int n0 = t.n0 + c0;
                if (n0 >= p.N || t.m0 + 32 * q >= p.M) continue;
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    const uint32_t a = stg + fast::sw128(lane, ch);
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v[4 * ch]), "f"(v[4 * ch + 1]),
                                 "f"(v[4 * ch + 2]), "f"(v[4 * ch + 3])
                                 : "memory");
                }
                __syncwarp();
                // 4 lanes a row, 8 columns each; 8 rows at a time
                const int cl = lane & 3, col = n0 + 8 * cl, have = min(8, p.N - col);
                if (have <= 0) continue;
                const bool vec = p.vec && (have == 8 || KIND == LIN_DW || sizeof(TO) == 4);
                float bias[8];
                if constexpr (KIND == LIN_FWD) {
                    if (p.e.bias) {
                        lin_ld8(p.e.bias + col, have, vec, bias);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) bias[j] = 0.f;
                    }
                }
#pragma unroll
                for (int r8 = 0; r8 < 4; ++r8) {
                    const int rl = 8 * r8 + (lane >> 2), row = t.m0 + 32 * q + rl;
                    if (row >= p.M) break;
                    const float4 x0 = *reinterpret_cast<const float4 *>(stage + fast::sw128(rl, 2 * cl));
                    const float4 x1 = *reinterpret_cast<const float4 *>(stage + fast::sw128(rl, 2 * cl + 1));
                    float y[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    const size_t at = (size_t)row * p.N + col;
                    if constexpr (KIND == LIN_DW) {
                        lin_st8(p.acc + (size_t)t.split * p.M * p.N + at, have, vec, y);
                    } else {
                        float o[8];
                        if constexpr (KIND == LIN_FWD) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) y[j] += bias[j];
                            if (p.e.out2) lin_st8(p.e.out2 + at, have, vec, y);
                            act_apply(y, p.e.act);
                        } else if (p.e.zin) {
                            lin_ld8(p.e.zin + at, have, vec, o);
                            act_slope_mul(y, o, p.e.act);
                        }
                        if (p.e.add) {
                            lin_ld8(p.e.add + at, have, vec, o);
#pragma unroll
                            for (int j = 0; j < 8; ++j) y[j] += o[j];
                        }
                        lin_st8(p.e.out + at, have, vec, y);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (w == 1) tmem_dealloc(tmem, 2 * BN);
}

// ------------------------------------------------------------------ host side

template <int KIND, int BN, typename TO>
static cudaError_t lt_launch(const LtMaps &m, const LtParams<TO> &p, cudaStream_t st) {
    static std::atomic<uint32_t> attr_set{0};
    if (cudaError_t e = ensure_smem_attr(k_lin_tc<KIND, BN, TO>, LtSmem<BN>::BYTES, attr_set); e != cudaSuccess) return e;
    k_lin_tc<KIND, BN, TO><<<std::min(p.units, sm_count()), LT_THR, LtSmem<BN>::BYTES, st>>>(m, p);
    return cudaGetLastError();
}
template <int KIND, typename TO>
static cudaError_t lt_run(int bn, const LtMaps &m, const LtParams<TO> &p, cudaStream_t st) {
    if (bn == 256) return lt_launch<KIND, 256, TO>(m, p, st);
    if (bn == 128) return lt_launch<KIND, 128, TO>(m, p, st);
    return lt_launch<KIND, 64, TO>(m, p, st);
}

// The widest tile that leaves no SM without one; where none does, the narrowest.
static int lt_bn(long long tiles_m, int N) {
    const int sms = sm_count();
    for (int bn : {256, 128})
        if (N > bn / 2 && tiles_m * ((N + bn - 1) / bn) >= sms) return bn;
    return 64;
}

template <typename TO>
static LtParams<TO> lt_params(const LinTc &q, long long M, int N, int bn) {
    LtParams<TO> p = {};
    p.status = q.status;
    p.clear = q.clear;
    p.M = (int)M;
    p.N = N;
    p.nseg = q.nseg;
    for (int s = 0; s < q.nseg; ++s) p.seg |= (uint32_t)q.seg[s] << (4 * s);
    p.tiles_m = (p.M + LT_BM - 1) / LT_BM;
    p.tiles_n = (N + bn - 1) / bn;
    return p;
}
// The maps of the parts that are there.
static bool lt_encode(CUtensorMap (&m)[3], const bf16 *const (&base)[3], long long rows, int ld, int box) {
    for (int k = 0; k < 3 && base[k]; ++k)
        if (!fast::encode_2d(&m[k], base[k], (int)rows, ld, box)) return false;
    return true;
}

template <typename T>
cudaError_t lin_tc_forward(const LinTc &q, const LinEpi<T> &e, cudaStream_t st) {
    const int bn = lt_bn((q.rows + LT_BM - 1) / LT_BM, q.out);
    LtParams<T> p = lt_params<T>(q, q.rows, q.out, bn);
    if ((long long)p.tiles_m * p.tiles_n > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.units = p.tiles_m * p.tiles_n;
    p.e = e;
    p.kts = (q.in + LT_BK - 1) / LT_BK;
    p.vec = (long long)q.out * sizeof(T) % 16 == 0;
    LtMaps m;
    if (!lt_encode(m.a, q.X, q.rows, q.ldx, LT_BM) || !lt_encode(m.b, q.W, q.in, q.ldw, 64)) return cudaErrorInvalidValue;
    return lt_run<LIN_FWD, T>(bn, m, p, st);
}

template <typename T>
cudaError_t lin_tc_dx(const LinTc &q, const LinEpi<T> &e, cudaStream_t st) {
    const int bn = lt_bn((q.rows + LT_BM - 1) / LT_BM, q.in);
    LtParams<T> p = lt_params<T>(q, q.rows, q.in, bn);
    if ((long long)p.tiles_m * p.tiles_n > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.units = p.tiles_m * p.tiles_n;
    p.e = e;
    p.kts = (q.out + LT_BK - 1) / LT_BK;
    p.vec = (long long)q.in * sizeof(T) % 16 == 0;
    LtMaps m;
    if (!lt_encode(m.a, q.dZ, q.rows, q.ldz, LT_BM) || !lt_encode(m.b, q.W, q.in, q.ldw, bn)) return cudaErrorInvalidValue;
    return lt_run<LIN_DX, T>(bn, m, p, st);
}

template cudaError_t lin_tc_forward<bf16>(const LinTc &, const LinEpi<bf16> &, cudaStream_t);
template cudaError_t lin_tc_dx<bf16>(const LinTc &, const LinEpi<bf16> &, cudaStream_t);

static int lt_dw_bn(int out) { return out > 128 ? 256 : out > 64 ? 128 : 64; }

// Splits so that the units fill the SMs about twice, each with eight steps of 64 rows or more.
LinSplit lin_tc_dw_split(long long rows, int in, int out) {
    const int bn = lt_dw_bn(out);
    const long long tiles = (long long)((in + LT_BM - 1) / LT_BM) * ((out + bn - 1) / bn);
    const long long steps = std::max(1LL, (rows + LT_BK - 1) / LT_BK);
    long long s = std::max(1LL, 2 * sm_count() / tiles);
    s = std::max(1LL, std::min(s, steps / 8));
    const long long per = (steps + s - 1) / s;
    return {(int)((steps + per - 1) / per), per * LT_BK};
}

cudaError_t lin_tc_dw(const LinTc &q, const LinSplit &s, float *dW, float *db, cudaStream_t st) {
    const int bn = lt_dw_bn(q.out);
    LtParams<bf16> p = lt_params<bf16>(q, q.in, q.out, bn);
    const long long units = (long long)p.tiles_m * p.tiles_n * s.splits;
    if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.units = (int)units;
    p.acc = dW; p.db = db;
    p.per = (int)(s.chunk / LT_BK);
    p.kts = (int)((q.rows + LT_BK - 1) / LT_BK);
    p.vec = q.out % 4 == 0;
    LtMaps m;
    if (!lt_encode(m.a, q.X, q.rows, q.ldx, 64) || !lt_encode(m.b, q.dZ, q.rows, q.ldz, 64)) return cudaErrorInvalidValue;
    return lt_run<LIN_DW, bf16>(bn, m, p, st);
}

}  // namespace ops
}  // namespace eaga
