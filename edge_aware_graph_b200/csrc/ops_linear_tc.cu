// The linear operator's products on tcgen05 (bf16 operands, fp32 sums):
//
//   forward   Y  = f(X W)      A = X  [rows, in]  K-major    B = W  [in, out]   MN-major (as stored)
//   dX        dX = f(dZ W^T)   A = dZ [rows, out] K-major    B = W  [in, out]   K-major  (the reduction is out)
//   dW        dW = X^T dZ      A = X  [rows, in]  MN-major   B = dZ [rows, out] MN-major (the reduction is rows)
//
// so every operand is read as it lies in memory.  Persistent CTAs take output
// tiles: a TMA warp fills a ring of 64-deep operand tiles (128-byte swizzled),
// one thread of the next warp issues the MMAs into one of two fp32 accumulators
// in TMEM, and 8 or 16 warps drain the other one, so the epilogue of a tile hides
// behind the next tile's products.
//
// Large products (CG = 2) run on pairs of CTAs: a 256 x 256 tile, of which each
// CTA keeps 128 rows of A and 128 columns of B in its shared memory and 128 rows
// of sums in its TMEM.  A pair loads 64 KB for 2 x 256 x 256 x 64 operations, half
// of what two 128 x 256 tiles would: what bounds the single form is the
// shared memory's and L2's traffic, not the tensor cores.  Small ones (CG = 1)
// take 128 x 128 or 128 x 64 tiles.
//
// Epilogue: a lane holds a row; bias, activation, slope and residual work on
// registers; residual and Zin come, and the outputs go, by TMA through one small
// swizzled tile a warp and tensor, so global memory sees whole rows of 64
// bytes.  Every output is rounded once.  Outputs whose rows do not begin on 16
// bytes (VEC = false) take a plain path.
//
// The tensor cores add with truncation: a chain of n products of 16 is off by up
// to n steps of fp32, all in one direction (measured 1e-6 relative after 1024
// rows, 1.9e-5 after 16384, 3.4e-4 after 65536).  The sums therefore leave the accumulator
// (PROMO) for sums in registers, rounded to nearest: of fp32 results every 512 steps of
// the reduction, of bf16 ones every 1024, a drift of 2^-17 at the most and 8e-7 as measured, 2000 times below
// the result's own rounding.  Bf16 results of 8192 x 4096 -> 4096 with gelu, R and Z take 256 us with it, 251 without
// (265 every 512 steps: a pair's epilogue is then longer than the two accumulators' next products).
// Reductions of one such stretch go to the epilogue as they are.
//
// A weight gradient reduces over rows, of which there may be a million for a
// 64 x 128 result, and a few rows' products over thousands of features: where
// tiles are few, the reduction is split, and the splits' fp32 sums are added in a
// fixed order by a kernel that has the epilogue then.  The bias gradient, the column
// sums of dZ, comes from two more warps: on single tiles in those of the first
// row, from the dZ tiles in shared memory times a matrix of ones (warp-level MMAs,
// joined in fp32 after every 64 rows); on pairs, where the barriers are the first
// CTA's, from dZ itself, which the tiles' loads have brought into L2, a share of
// the rows in every row of tiles.
//
// An operand in fp32 comes as bf16 parts (two carry 16 bits of it, three 24),
// and a step of the reduction is one for each product of parts that counts: fp32
// products take six, all but those below 2^-24, at a sixth of the bf16 rate, which is
// 2.5 times what the CUDA cores could reach.
#include <algorithm>
#include <type_traits>
#include "ops_linear.h"
#include "sm100.cuh"

namespace eaga {
namespace fast {
bool encode_2d(CUtensorMap *m, const void *base, int rows, int cols, int box_rows);
bool encode_blocks(CUtensorMap *m, const void *base, int rows, int cols, int blocks);
bool encode_3d(CUtensorMap *m, const void *base, bool f32, long long planes, long long rows, long long cols, int box_rows);
}
namespace ops {

using namespace sm100;
typedef __nv_bfloat16 bf16;

constexpr int LT_BM = 128, LT_BK = 64;
// 64-deep steps an accumulator takes before its sums move on to registers, of an fp32 and of a bf16 result.
template <typename TO> constexpr int lt_promo() { return sizeof(TO) == 4 ? 8 : 16; }

// PER: CTAs an SM.  Two where reductions are short and tiles narrow and many: each waits for its loads and accumulators most of
// the time (1M x 34 -> 48).
template <int KIND, int BN, int CG, typename TO, bool VEC, int PER>
struct Lt {
    static constexpr int BM = LT_BM * CG, PB = BN / CG;              // the tile's rows; B columns a CTA holds
    // Epilogue warps: two or four a TMEM quadrant (32 rows), each with its part of the columns.  A short reduction's tile is
    // bound by them: with 8 warps on 128 columns 34355 x 16 -> 1320 with silu and Z took 60 us.
    static constexpr int EPI = BN == 64 ? 8 : 16, THR = 32 * (4 + EPI);      // TMA, MMA, two column-sum warps, epilogue
    static constexpr int COLS = BN / (EPI / 4);                      // columns of an epilogue warp
    static constexpr int PC = VEC ? 64 / (int)sizeof(TO) : 32;       // a piece's columns: rows of 64 bytes in a slot
    static constexpr int PIECES = COLS / PC;
    static constexpr uint32_t A_BYTES = LT_BM * LT_BK * 2, B_BYTES = PB * LT_BK * 2, STAGE = A_BYTES + B_BYTES;
    static constexpr uint32_t SLOT = VEC ? 2048 : 4096;
    // Slots of a warp: the output's (in it the residual), two in turn where the epilogue is not hidden behind long
    // products anyway; one for Z or Zin.
    static constexpr int NIO = !VEC || (CG == 2 && KIND != LIN_DW) ? 1 : 2, SLOTS = !VEC || KIND == LIN_DW ? NIO : NIO + 1;
    static constexpr uint32_t MOST = PER == 2 ? 115712 : 232448, RING = MOST - 1024 - 1024 - EPI * SLOTS * SLOT;
    static constexpr int ST = RING / STAGE < 8 ? RING / STAGE : 8;
    static constexpr uint32_t EPI_AT = ST * STAGE;
    static constexpr uint32_t BAR = EPI_AT + EPI * SLOTS * SLOT;     // full[ST], empty[ST], acc_full[2], acc_empty[2], drained, slots' [EPI][3]
    static constexpr uint32_t TM = BAR + (2 * ST + 5 + 3 * EPI) * 8;
    static constexpr uint32_t FAIL = TM + 4;
    static constexpr uint32_t BYTES = FAIL + 4 + 1024;
    static_assert(ST >= (PER == 2 ? 2 : 3) && BYTES <= MOST && COLS % 32 == 0, "shared memory");
};

// A bounded wait that looks at the CTA's failure flag only where the barrier is not there yet.
__device__ __forceinline__ bool lt_wait(uint32_t bar, uint32_t parity, volatile int *fail, int *status) {
    if (mbar_try_wait(bar, parity)) return true;
    return fast::dev::cta_wait(bar, parity, fail, status);
}

// Maps of the operands' parts, the outputs and the epilogue's inputs.
struct LtMaps {
    CUtensorMap a[3], b[3];
    CUtensorMap out, out2, add, zin;
};

template <typename TO>
struct LtParams {
    LinEpi<TO> e;              // out: [split][M][N]
    float *db;                 // weight gradient: [split][N], on pairs [split][row of tiles][N]
    const bf16 *dz[3];         // on pairs, for db: dZ's parts, their row length
    int ldz, rows;
    int *status;
    int M, N;                  // output
    int kts, per;              // 64-deep steps of the reduction, of a split
    int nseg;
    uint32_t seg;              // products of parts, four bits each: A's part, B's part
    int tiles_m, tiles_n, units;
    int clear;
    int ablocks, bblocks;      // an MN-major operand's map has blocks of 64 columns: one load a step
};

template <int KIND, int BN, int CG, typename TO, bool VEC, int PER, bool PROMO>
__global__ void __launch_bounds__(Lt<KIND, BN, CG, TO, VEC, PER>::THR, PER)
k_lin_tc(const __grid_constant__ LtMaps maps, const __grid_constant__ LtParams<TO> p) {
    using S = Lt<KIND, BN, CG, TO, VEC, PER>;
    constexpr int ST = S::ST, PC = S::PC, PIECES = S::PIECES;
    constexpr bool A_MN = KIND == LIN_DW, B_MN = KIND != LIN_DX, PAIR = CG == 2;
    constexpr bool SMEM_SUMS = KIND == LIN_DW && !PAIR;
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
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;

    if (tid == 32) {
        prefetch_map(&maps.a[0]);
        prefetch_map(&maps.b[0]);
        if (VEC) prefetch_map(&maps.out);
    }
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), SMEM_SUMS && p.db ? 3 : 1);  // the MMAs; two column-sum warps
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), S::EPI * CG);
        }
        mbar_init(drained, 1);
        for (int k = 0; k < 3 * S::EPI; ++k) mbar_init(drained + 8 + 8 * k, 1);
        fence_mbar_init();
        *fail = 0;
    }
    if (w == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(sbase + S::TM, 2 * BN);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(sbase + S::TM, 2 * BN);
            tmem_relinquish();
        }
    }
    after_previous();
    if (p.clear && blockIdx.x == 0 && tid == 0) *p.status = 0;     // a wait that gives up does so a second later
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();                  // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sp + S::TM);
    // unit -> output tile (columns fastest), split, its steps
    struct Unit {
        int m0, n0, split, k0, steps, tm;
    };
    auto unit_of = [&](int u) {
        Unit r;
        const int tiles = p.tiles_m * p.tiles_n;
        r.split = tiles == p.units ? 0 : u / tiles;
        const int t = u - r.split * tiles;
        r.tm = t / p.tiles_n;
        r.m0 = r.tm * S::BM + rank * LT_BM;                  // this CTA's rows
        r.n0 = (t - r.tm * p.tiles_n) * BN;
        r.k0 = r.split * p.per;
        r.steps = min(p.per, p.kts - r.k0);
        return r;
    };

    if (w < 4) {
        if (w == 0) {
            if (lane == 0) {
                int s = 0, issued = 0;                       // the stage; stages filled
                uint32_t ph = 1;
                bool ok = true;
                const CUtensorMap *am = &maps.a[p.seg & 3], *bm = &maps.b[(p.seg >> 2) & 3];
                const uint32_t full0 = PAIR ? cluster_map(full(0), 0) : full(0);     // the first CTA's barriers
                // One 64-deep step of a unit.  This thread, like the MMAs', has 512 clocks for it on pairs: the fewer
                // instructions and loads, the better (an MN-major operand is one load where its rows are blocks of 64 columns).
                auto step = [&](const CUtensorMap *am, const CUtensorMap *bm, int kk, int m0, int nb) {
                    if (!lt_wait(empty(s), ph, fail, p.status)) return false;
                    const uint32_t st = sbase + s * S::STAGE, bar = full0 + 8 * s;
                    if (rank == 0) mbar_expect_tx(full(s), S::STAGE * CG);
                    auto load = [&](uint32_t dst, const CUtensorMap *m, int c0, int c1) {
                        if constexpr (PAIR) tma_load_2d_pair(dst, m, bar, c0, c1);
                        else tma_load_2d(dst, m, bar, c0, c1);
                    };
                    auto load_blocks = [&](uint32_t dst, const CUtensorMap *m, int row, int block) {
                        if constexpr (PAIR) tma_load_3d_pair(dst, m, bar, 0, row, block);
                        else tma_load_3d(dst, m, bar, 0, row, block);
                    };
                    if constexpr (!A_MN) {
                        load(st, am, kk, m0);
                    } else if (p.ablocks) {
                        load_blocks(st, am, kk, m0 >> 6);
                    } else {
                        load(st, am, m0, kk);
                        load(st + 8192, am, m0 + 64, kk);
                    }
                    if constexpr (!B_MN) {
                        load(st + S::A_BYTES, bm, kk, nb);
                    } else if (p.bblocks) {
                        load_blocks(st + S::A_BYTES, bm, kk, nb >> 6);
                    } else {
#pragma unroll
                        for (int h = 0; h < S::PB / 64; ++h) load(st + S::A_BYTES + h * 8192, bm, nb + 64 * h, kk);
                    }
                    ++issued;
                    if (++s == ST) {
                        s = 0;
                        ph ^= 1;
                    }
                    return true;
                };
                for (int u = first; ok && u < p.units; u += stride) {
                    const Unit t = unit_of(u);
                    const int nb = t.n0 + rank * S::PB;      // this CTA's columns of B
                    int kk = t.k0 * LT_BK;
                    if (p.nseg == 1) {
                        for (int k = t.steps; ok && k > 0; --k, kk += LT_BK) ok = step(am, bm, kk, t.m0, nb);
                    } else {
                        for (int k = t.steps; ok && k > 0; --k, kk += LT_BK) {
                            uint32_t parts = p.seg;
                            for (int seg = p.nseg; ok && seg > 0; --seg, parts >>= 4)
                                ok = step(&maps.a[parts & 3], &maps.b[(parts >> 2) & 3], kk, t.m0, nb);
                        }
                    }
                }
                // After a wait that gave up: what was issued lands before the CTA's memory is released.  (Of a pair the first
                // CTA's barriers count both CTAs' loads, and the two leave together.)
                if (!ok && rank == 0)
                    for (int i = max(issued - ST, 0); i < issued; ++i) mbar_wait(full(i % ST), (i / ST) & 1);
            }
        } else if (w == 1) {
            if (lane == 0 && rank == 0) {
                constexpr uint32_t idesc = idesc_bf16_f32(S::BM, BN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
                // One thread feeds the tensor cores: between two stages it has 512 clocks (a pair's, 256 or 128 a single
                // tile's), so descriptors are one addition away, and a wait looks at the failure flag only when it has to.
                const uint64_t ad0 = A_MN ? smem_desc(sbase, 8192, 1024, LAYOUT_SW128) : smem_desc(sbase, 16, 1024, LAYOUT_SW128);
                const uint64_t bd0 = B_MN ? smem_desc(sbase + S::A_BYTES, 8192, 1024, LAYOUT_SW128)
                                          : smem_desc(sbase + S::A_BYTES, 16, 1024, LAYOUT_SW128);
                constexpr uint32_t AK = (A_MN ? 2048 : 32) >> 4, BK = (B_MN ? 2048 : 32) >> 4;     // 16 steps on
                int s = 0, n = 0;                                // the stage; accumulators
                uint32_t ph = 0;
                bool ok = true;
                for (int u = first; ok && u < p.units; u += stride) {
                    const Unit t = unit_of(u);
                    const int nk = t.steps * p.nseg;
                    for (int k0 = 0; ok && k0 < nk; ++n) {
                        const int b = n & 1, k1 = PROMO ? min(k0 + lt_promo<TO>(), nk) : nk;
                        if (!lt_wait(acc_empty(b), ((n >> 1) & 1) ^ 1, fail, p.status)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t d = tmem + b * BN;
                        for (int k = k0; k < k1; ++k) {
                            if (!lt_wait(full(s), ph, fail, p.status)) { ok = false; break; }
                            tc_fence_after();
                            const uint64_t ad = ad0 + (uint32_t)(s * (S::STAGE >> 4)), bd = bd0 + (uint32_t)(s * (S::STAGE >> 4));
#pragma unroll
                            for (int kk = 0; kk < LT_BK / 16; ++kk) {
                                const uint32_t more = k > k0 || kk > 0 ? 1u : 0u;
                                if constexpr (PAIR) mma_bf16_ss_pair(d, ad + kk * AK, bd + kk * BK, idesc, more);
                                else mma_bf16_ss(d, ad + kk * AK, bd + kk * BK, idesc, more);
                            }
                            if constexpr (PAIR) mma_commit_pair(empty(s), 3);
                            else mma_commit(empty(s));
                            if (++s == ST) {
                                s = 0;
                                ph ^= 1;
                            }
                        }
                        if (ok) {
                            if constexpr (PAIR) mma_commit_pair(acc_full(b), 3);
                            else mma_commit(acc_full(b));
                        }
                        k0 = k1;
                    }
                }
                if (!ok) {                                       // the products in flight end before TMEM is freed
                    if constexpr (PAIR) mma_commit_pair(drained, 1);
                    else mma_commit(drained);
                    mbar_wait(drained, 0);
                }
            }
        } else if (w < 4) {
            if constexpr (SMEM_SUMS) {
                // column sums of the dZ tile: ones [16 x 16] times [16 rows x 8 columns] at a time
                constexpr int COLS = BN / 2, NT = COLS / 8;        // this warp's columns
                const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
                const int c0 = (w - 2) * COLS;
                int it = 0;
                bool ok = true;
                // every step of every unit, the unsummed ones too: a wait by parity knows a phase from its neighbours only
                for (int u = first; p.db != nullptr && ok && u < p.units; u += stride) {
                    const Unit t = unit_of(u);
                    const int nk = t.steps * p.nseg;
                    float sum[NT][2];
#pragma unroll
                    for (int j = 0; j < NT; ++j) sum[j][0] = sum[j][1] = 0.f;
                    for (int k = 0, seg = 0; k < nk; ++k, ++it, seg = seg + 1 < p.nseg ? seg + 1 : 0) {
                        const int s = it % ST;
                        ok = __all_sync(0xffffffffu, lt_wait(full(s), (it / ST) & 1, fail, p.status));
                        if (!ok) break;
                        if (t.tm != 0 || ((p.seg >> (4 * seg)) & 3)) {     // each part of dZ once: beside X's first
                            if (lane == 0) mbar_arrive(empty(s));
                            continue;
                        }
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
                    if (ok && t.tm == 0 && lane < 4) {  // row 0 of the product: columns 2 lane, 2 lane + 1 of each 8
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
            } else if constexpr (KIND == LIN_DW) {
                // column sums of dZ from memory, each row of tiles its share of the unit's rows: a warp 64 columns, 8 a
                // lane, four rows at a time
                for (int u = first; p.db != nullptr && u < p.units; u += stride) {
                    const Unit t = unit_of(u);
                    const int c = t.n0 + rank * S::PB + (w - 2) * 64 + 8 * (lane & 7);
                    const long long all = min((long long)p.rows - (long long)t.k0 * LT_BK, (long long)t.steps * LT_BK);
                    const long long part = (all + p.tiles_m - 1) / p.tiles_m, base = (long long)t.k0 * LT_BK;
                    const long long r0 = base + min(all, part * t.tm), r1 = base + min(all, part * (t.tm + 1));
                    float sum[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
                    if (c < p.ldz) {
                        for (int seg = 0; seg < p.nseg; ++seg) {
                            if ((p.seg >> (4 * seg)) & 3) continue;
                            const bf16 *z = p.dz[(p.seg >> (4 * seg + 2)) & 3] + c;
#pragma unroll 8
                            for (long long r = r0 + (lane >> 3); r < r1; r += 4) {
                                float v[8];
                                lin_ld8(z + r * p.ldz, 8, true, v);
#pragma unroll
                                for (int j = 0; j < 8; ++j) sum[j] += v[j];
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
                        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
                    }
                    if (lane < 8) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < p.N) p.db[((size_t)t.split * p.tiles_m + t.tm) * p.N + c + j] = sum[j];
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        const int q = w & 3, ew = w - 4, first_col = (ew >> 2) * S::COLS;   // TMEM quadrant: rows 32 q ..; its columns of the tile
        const uint32_t slots = sbase + S::EPI_AT + ew * S::SLOTS * S::SLOT;
        const uint8_t *slots_p = sp + S::EPI_AT + ew * S::SLOTS * S::SLOT;
        const uint32_t slot_bar = drained + 8 + 24 * ew;
        const bool has_add = VEC && KIND != LIN_DW && p.e.add != nullptr, has_zin = VEC && KIND == LIN_DX && p.e.zin != nullptr;
        const bool has_z = VEC && KIND == LIN_FWD && p.e.out2 != nullptr;
        const bool two = has_add && has_zin;        // Zin goes to the third slot where the residual has the output's
        // the pieces with something in them, in order
        auto some = [&](const Unit &t, int c) { return t.m0 + 32 * q < p.M && t.n0 + first_col + c * PC < p.N; };
        struct Place {
            int u, c;
        };
        auto seek = [&](Place x) {                  // the first such piece from x on
            while (x.u < p.units) {
                const Unit t = unit_of(x.u);
                if (some(t, x.c)) break;
                x = {x.u + stride, 0};
            }
            return x;
        };
        auto after = [&](Place x) { return seek(x.c + 1 < PIECES ? Place{x.u, x.c + 1} : Place{x.u + stride, 0}); };
        // ask for the inputs of a piece, the k-th of this warp (lane 0; the slot's last store has been read)
        auto ask = [&](Place x, int k, bool side) {
            if (x.u >= p.units) return;
            const Unit t = unit_of(x.u);
            const int col = t.n0 + first_col + x.c * PC, row = t.m0 + 32 * q;
            const int s = side ? S::NIO : k % S::NIO;
            mbar_expect_tx(slot_bar + 8 * s, S::SLOT);
            tma_load_3d(slots + s * S::SLOT, side || !has_add ? &maps.zin : &maps.add, slot_bar + 8 * s, col, row, 0);
        };
        int k = 0;                                  // pieces of this warp so far
        if constexpr (VEC && KIND != LIN_DW) {
            if (lane == 0 && (has_add || has_zin)) {
                const Place x = seek({first, 0});
                ask(x, 0, false);
                if (two) ask(x, 0, true);
            }
            __syncwarp();
        }
        int n = 0;
        bool ok = true;
        for (int u = first; ok && u < p.units; u += stride) {
            const Unit t = unit_of(u);
            const int nk = t.steps * p.nseg, chunks = PROMO ? (nk + lt_promo<TO>() - 1) / lt_promo<TO>() : 1;
            float acc[PROMO ? S::COLS : 1] = {};
            auto released = [&](int b) {            // the accumulator may be written again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(cluster_map(acc_empty(b), 0));
                    else mbar_arrive(acc_empty(b));
                }
            };
            for (int ch = 0; ch < chunks; ++ch, ++n) {
                const int b = n & 1;
                ok = __all_sync(0xffffffffu, lt_wait(acc_full(b), (n >> 1) & 1, fail, p.status));
                if (!ok) break;
                tc_fence_after();
                if constexpr (PROMO) {
                    const uint32_t ta = tmem + b * BN + ((uint32_t)(32 * q) << 16) + first_col;
#pragma unroll
                    for (int c = 0; c < S::COLS; c += 16) {
                        float v[16];
                        tmem_ld16(ta + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
                    }
                    released(b);
                }
            }
            if (!ok) break;
            const int b = (n - 1) & 1;
            const int row0 = t.m0 + 32 * q;
            auto piece = [&](int c, float (&v)[PC]) {
                const int col = t.n0 + first_col + c * PC;
                if (row0 >= p.M || col >= p.N) return;
                if constexpr (VEC) {
                    const int s = k % S::NIO;
                    if constexpr (KIND != LIN_DW) {
                        if (has_add || has_zin) {
                            // the next piece's inputs, into the other slot: its store (the last piece's) has been read by now
                            if (lane == 0) {
                                tma_store_wait_read0();
                                if (S::NIO == 2) ask(after({u, c}), k + 1, false);
                            }
                            __syncwarp();
                            ok = __all_sync(0xffffffffu, lt_wait(slot_bar + 8 * s, (k / S::NIO) & 1, fail, p.status));
                            if (two) ok = ok && __all_sync(0xffffffffu, lt_wait(slot_bar + 8 * S::NIO, k & 1, fail, p.status));
                            if (!ok) return;
                        }
                    }
                    if (!(has_add || has_zin)) {
                        // a slot is free when all stores but the last piece's have been read; Z's slot when that one has, too
                        if (lane == 0) {
                            if (has_z || S::NIO == 1) tma_store_wait_read0();
                            else tma_store_wait_read1();
                        }
                        __syncwarp();
                    }
                    const uint32_t io = slots + s * S::SLOT, side = slots + S::NIO * S::SLOT;
                    const uint8_t *iop = slots_p + s * S::SLOT, *sidep = slots_p + (two ? S::NIO : s) * S::SLOT;
                    constexpr int PER = 16 / sizeof(TO);        // columns of a 16-byte chunk
                    auto put = [&](uint32_t base) {
#pragma unroll
                        for (int x = 0; x < PC / PER; ++x) {
                            uint32_t o[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if constexpr (sizeof(TO) == 2) o[j] = pack_bf16(v[x * 8 + 2 * j], v[x * 8 + 2 * j + 1]);
                                else o[j] = __float_as_uint(v[x * 4 + j]);
                            }
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + fast::sw64(lane, x)), "r"(o[0]), "r"(o[1]),
                                         "r"(o[2]), "r"(o[3])
                                         : "memory");
                        }
                    };
                    auto get = [&](const uint8_t *base, int x, float (&f)[PER]) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(base + fast::sw64(lane, x));
                        const uint32_t y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (sizeof(TO) == 2) {
                                f[2 * j] = __uint_as_float(y[j] << 16);
                                f[2 * j + 1] = __uint_as_float(y[j] & 0xffff0000u);
                            } else {
                                f[j] = __uint_as_float(y[j]);
                            }
                        }
                    };
                    if constexpr (KIND == LIN_FWD) {
                        if (p.e.bias) {
#pragma unroll
                            for (int x = 0; x < PC / 8; ++x) {
                                float f[8];
                                const int have = min(8, p.N - col - 8 * x);        // 8, or 4 of an fp32 row, or none
                                if (have > 0) {
                                    lin_ld8(p.e.bias + col + 8 * x, have, true, f);
#pragma unroll
                                    for (int j = 0; j < 8; ++j) v[8 * x + j] += f[j];
                                }
                            }
                        }
                        if (has_z) put(side);
                        act_apply<TO>(v, p.e.act);
                    } else if constexpr (KIND == LIN_DX) {
                        if (has_zin) {
#pragma unroll
                            for (int x = 0; x < PC / PER; ++x) {
                                float f[PER], y[PER];
                                get(sidep, x, f);
#pragma unroll
                                for (int j = 0; j < PER; ++j) y[j] = v[x * PER + j];
                                act_slope_mul<TO>(y, f, p.e.act);
#pragma unroll
                                for (int j = 0; j < PER; ++j) v[x * PER + j] = y[j];
                            }
                        }
                    }
                    if (has_add) {
#pragma unroll
                        for (int x = 0; x < PC / PER; ++x) {
                            float f[PER];
                            get(iop, x, f);
#pragma unroll
                            for (int j = 0; j < PER; ++j) v[x * PER + j] += f[j];
                        }
                    }
                    put(io);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&maps.out, io, col, row0, t.split);
                        if (has_z) tma_store_3d(&maps.out2, side, col, row0, 0);
                        tma_store_commit();
                        if (S::NIO == 1 && (has_add || has_zin)) {
                            tma_store_wait_read0();
                            ask(after({u, c}), k + 1, false);
                        }
                        if (two) ask(after({u, c}), k + 1, true);      // Zin of the next piece: this one's has been read
                    }
                    __syncwarp();
                    ++k;
                } else {
                    // rows that do not begin on 16 bytes: a lane a column, 16 rows' loads in flight
                    __syncwarp();                   // the last piece's reads are done
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(slots + fast::sw128(lane, x)), "f"(v[4 * x]),
                                     "f"(v[4 * x + 1]), "f"(v[4 * x + 2]), "f"(v[4 * x + 3])
                                     : "memory");
                    __syncwarp();
                    const int cc = col + lane;
                    if (cc < p.N) {
                        const float bias = KIND == LIN_FWD && p.e.bias ? ldf(p.e.bias + cc) : 0.f;
#pragma unroll 1
                        for (int r0 = 0; r0 < 32 && row0 + r0 < p.M; r0 += 16) {
                            const size_t at = (size_t)(row0 + r0) * p.N + cc;
                            TO zi[16], ad[16];
                            if (KIND == LIN_DX && p.e.zin) {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (row0 + r0 + j < p.M) zi[j] = p.e.zin[at + (size_t)j * p.N];
                            }
                            if (KIND != LIN_DW && p.e.add) {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (row0 + r0 + j < p.M) ad[j] = p.e.add[at + (size_t)j * p.N];
                            }
                            TO *o = p.e.out + (size_t)t.split * p.M * p.N + at;
                            float y[16];            // the rows of one column: the activation's code once for all
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                y[j] = *reinterpret_cast<const float *>(slots_p + fast::sw128(r0 + j, lane >> 2) + 4 * (lane & 3)) + bias;
                            if constexpr (KIND == LIN_FWD) {
                                if (p.e.out2) {
#pragma unroll
                                    for (int j = 0; j < 16; ++j)
                                        if (row0 + r0 + j < p.M) stf(p.e.out2 + at + (size_t)j * p.N, y[j]);
                                }
                                act_apply<TO>(y, p.e.act);
                            } else if constexpr (KIND == LIN_DX) {
                                if (p.e.zin) {
                                    float z[16];
#pragma unroll
                                    for (int j = 0; j < 16; ++j) z[j] = row0 + r0 + j < p.M ? ldf(&zi[j]) : 0.f;
                                    act_slope_mul<TO>(y, z, p.e.act);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                if (row0 + r0 + j >= p.M) break;
                                if (KIND != LIN_DW && p.e.add) y[j] += ldf(&ad[j]);
                                stf(o + (size_t)j * p.N, y[j]);
                            }
                        }
                    }
                    __syncwarp();
                }
            };
            if constexpr (PROMO) {
#pragma unroll
                for (int c = 0; c < PIECES; ++c) {
                    float v[PC];
#pragma unroll
                    for (int j = 0; j < PC; ++j) v[j] = acc[c * PC + j];
                    piece(c, v);
                    if (!ok) break;
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < PIECES; ++c) {
                    float v[PC];
                    const uint32_t ta = tmem + b * BN + ((uint32_t)(32 * q) << 16) + first_col + c * PC;
#pragma unroll
                    for (int j = 0; j < PC; j += 32) tmem_ld32(ta + j, *reinterpret_cast<float(*)[32]>(v + j));
                    tmem_ld_wait();
                    if (c == PIECES - 1) released(b);
                    piece(c, v);
                    if (!ok) break;
                }
            }
        }
        if constexpr (VEC) {
            if (lane == 0) {
                tma_store_wait_all();
                // after a wait that gave up: inputs asked for land before the CTA's memory is released
                if (!ok && (has_add || has_zin)) {
                    for (int x = k; x < k + S::NIO; ++x) mbar_wait(slot_bar + 8 * (x % S::NIO), (x / S::NIO) & 1);
                    if (two) mbar_wait(slot_bar + 8 * S::NIO, k & 1);
                }
            }
            __syncwarp();
        }
    }
    before_next();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    if (w == 1) {
        if constexpr (PAIR) tmem_dealloc_pair(tmem, 2 * BN);
        else tmem_dealloc(tmem, 2 * BN);
    }
}

// ------------------------------------------------------------------ host side

template <int KIND, int BN, int CG, typename TO, bool VEC, int PER, bool PROMO>
static cudaError_t lt_launch(const LtMaps &m, const LtParams<TO> &p, cudaStream_t st) {
    using S = Lt<KIND, BN, CG, TO, VEC, PER>;
    auto kernel = k_lin_tc<KIND, BN, CG, TO, VEC, PER, PROMO>;
    static std::atomic<uint32_t> attr_set{0};
    if (cudaError_t e = ensure_smem_attr(kernel, S::BYTES, attr_set); e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)(std::min(p.units, PER * sm_count() / CG) * CG)), dim3(S::THR), S::BYTES, st, CG, m, p);
}
template <int KIND, typename TO, bool VEC, bool PROMO>
static cudaError_t lt_tiles(const LinTile &t, const LtMaps &m, const LtParams<TO> &p, cudaStream_t st) {
    if (t.pair) return lt_launch<KIND, 256, 2, TO, VEC, 1, true>(m, p, st);
    return t.bn == 128 ? lt_launch<KIND, 128, 1, TO, VEC, 1, PROMO>(m, p, st) : lt_launch<KIND, 64, 1, TO, VEC, 1, PROMO>(m, p, st);
}
template <int KIND, typename TO, bool VEC>
static cudaError_t lt_run(const LtForm &f, const LtMaps &m, const LtParams<TO> &p, cudaStream_t st) {
    if constexpr (KIND != LIN_DW && sizeof(TO) == 2) {
        if constexpr (VEC) {
            if (f.two) return lt_launch<KIND, 64, 1, TO, VEC, 2, false>(m, p, st);
        }
        if (!f.promo) return lt_tiles<KIND, TO, VEC, false>(f.tile, m, p, st);
    }
    return lt_tiles<KIND, TO, VEC, true>(f.tile, m, p, st);
}
// (An fp32 result has six products a step, or splits of more steps than `two` is for; pairs are chosen for longer reductions
// than one stretch: their epilogue is as long as 40 steps.)
LtForm lin_tc_form(int kind, const LinSplit &s, bool f32, long long M, int N, long long K, int nseg) {
    const int bm = s.tile.pair ? 2 * LT_BM : LT_BM;
    LtForm f = {s.tile, (long long)N * (f32 ? 4 : 2) % 16 == 0, false, true, (M + bm - 1) / bm * ((N + s.tile.bn - 1) / s.tile.bn) * s.splits};
    const long long steps = std::min(s.chunk / LT_BK, (K + LT_BK - 1) / LT_BK) * nseg;     // of a unit, the longest
    if (kind != LIN_DW && !f32) {
        f.two = f.tma && !s.tile.pair && s.tile.bn == 64 && f.units >= 4 * sm_count() && steps <= 4;
        f.promo = s.tile.pair || steps > lt_promo<bf16>();
    }
    return f;
}

// Tiles and splits: the least of an estimate of each form's time.  The unit is a 64-deep step of a pair's tile,
// 0.28 us.  A step of the single tiles takes as long (128 columns) or 0.75 of it (64) for a half and a quarter of
// a CTA's work: 32 and 24 KB from L2 bound them (measured 1.0e15 op/s, pairs 1.4e15).  A tile's epilogue runs
// beside the next one's steps and bounds short reductions: 1.5 us and 1.3 us of a single tile, 11 us of a pair's, which
// has one slot a warp and waits for each store (138936 x 24 -> 136 with two outputs: 98 us on pairs).  fp32 tensors take 4 us of a
// 128-wide tile, 7 us where their rows are not 16 bytes (94180 x 31 -> 520, 102998 x 431 <- 32).  Splits cost the
// write and read of their sums and, of products that need no second kernel otherwise, its launch.
static double lt_cost(const LinTile &t, long long M, int N, long long steps, int splits, bool f32) {
    const int bm = t.pair ? 256 : 128, sms = sm_count();
    const double units = (double)((M + bm - 1) / bm) * ((N + t.bn - 1) / t.bn) * splits;
    const double step = t.bn == 64 ? 0.75 : 1.0, wide = !f32 ? 1 : N % 4 ? 4.5 : 2.7;
    const double epilogue = t.pair ? 40 : wide * (t.bn == 128 ? 5.5 : 4.8);
    const double waves = std::ceil(units / (t.pair ? sms / 2 : sms));
    const double per = (double)((steps + splits - 1) / splits) * step;
    double c = (waves - 1) * std::max(per, epilogue) + per + epilogue + 4;
    if (splits > 1) c += 8 + (double)splits * M * N * 8 / 6.5e6 / 0.28;             // bytes / (bytes a us) / (us a step)
    return c;
}

LinSplit lin_tc_split(long long M, int N, long long K, int nseg, bool f32, double *us) {
    static const LinTile tiles[3] = {{true, 256}, {false, 128}, {false, 64}};
    const long long steps = std::max(1LL, (K + LT_BK - 1) / LT_BK);
    LinSplit best = {1, steps * LT_BK, tiles[2]};
    double least = 1e300;
    for (const LinTile &t : tiles) {
        if (t.pair ? M <= 128 || N <= 128 : t.bn == 128 && N <= 64) continue;
        // splits of four steps or more, while they are not more than four units an SM; of the many, every eighth or so
        // (this runs on the host in every call)
        const int bm = t.pair ? 256 : 128;
        const long long units = (M + bm - 1) / bm * ((N + t.bn - 1) / t.bn);
        const int most = (int)std::max(1LL, std::min(steps * nseg / 4, std::min(steps, 4LL * sm_count() / units)));
        for (int s = 1; s <= most; s += s < 8 ? 1 : s / 8) {
            const long long per = (steps + s - 1) / s;
            const int real = (int)((steps + per - 1) / per);
            const double c = lt_cost(t, M, N, steps * nseg, real, f32);
            if (c < least) {
                least = c;
                best = {real, per * LT_BK, t};
            }
        }
    }
    if (us) *us = 0.28 * least;
    return best;
}

// The maps of the parts that are there: boxes of 64 columns and `box` rows, or of 64 rows and `blocks` blocks of columns.
static bool lt_encode(CUtensorMap (&m)[3], const bf16 *const (&base)[3], long long rows, int ld, int box, int blocks = 0) {
    for (int k = 0; k < 3 && base[k]; ++k)
        if (!(blocks ? fast::encode_blocks(&m[k], base[k], (int)rows, ld, blocks) : fast::encode_2d(&m[k], base[k], (int)rows, ld, box)))
            return false;
    return true;
}
// The maps of the outputs and the epilogue's inputs, a warp's piece at a time.
template <typename TO>
static bool lt_encode_out(LtMaps &m, const LinEpi<TO> &e, long long planes, long long M, int N) {
    auto enc = [&](CUtensorMap *x, const void *base) { return !base || fast::encode_3d(x, base, sizeof(TO) == 4, planes, M, N, 32); };
    return enc(&m.out, e.out) && enc(&m.out2, e.out2) && enc(&m.add, e.add) && enc(&m.zin, e.zin);
}

template <int KIND, typename T>
static cudaError_t lt_product(const LinTc &q, const LinSplit &sp, const LinEpi<T> &e, float *db, long long M, int N, long long K,
                              cudaStream_t st) {
    LtParams<T> p = {};
    p.status = q.status;
    p.clear = q.clear;
    p.M = (int)M;
    p.N = N;
    p.nseg = q.nseg;
    for (int s = 0; s < q.nseg; ++s) p.seg |= (uint32_t)q.seg[s] << (4 * s);
    const int bm = sp.tile.pair ? 2 * LT_BM : LT_BM;
    p.tiles_m = (int)((M + bm - 1) / bm);
    p.tiles_n = (N + sp.tile.bn - 1) / sp.tile.bn;
    const LtForm form = lin_tc_form(KIND, sp, sizeof(T) == 4, M, N, K, q.nseg);
    if (form.units > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.units = (int)form.units;
    p.kts = (int)((K + LT_BK - 1) / LT_BK);
    p.per = (int)(sp.chunk / LT_BK);
    p.e = e;
    p.db = db;
    for (int k = 0; k < 3; ++k) p.dz[k] = q.dZ[k];
    p.ldz = q.ldz;
    p.rows = (int)q.rows;
    LtMaps m;
    bool ok;
    const int nb = sp.tile.pair ? 2 : sp.tile.bn / 64;       // blocks of B a CTA loads
    if (KIND != LIN_DX) p.bblocks = (KIND == LIN_FWD ? q.ldw : q.ldz) % 64 == 0 ? nb : 0;
    if (KIND == LIN_DW) p.ablocks = q.ldx % 64 == 0 ? 2 : 0;
    if (KIND == LIN_FWD) ok = lt_encode(m.a, q.X, q.rows, q.ldx, LT_BM) && lt_encode(m.b, q.W, q.in, q.ldw, 64, p.bblocks);
    else if (KIND == LIN_DX) ok = lt_encode(m.a, q.dZ, q.rows, q.ldz, LT_BM) && lt_encode(m.b, q.W, q.in, q.ldw, sp.tile.pair ? 128 : sp.tile.bn);
    else ok = lt_encode(m.a, q.X, q.rows, q.ldx, 64, p.ablocks) && lt_encode(m.b, q.dZ, q.rows, q.ldz, 64, p.bblocks);
    if (!ok) return cudaErrorInvalidValue;
    if (!form.tma) return lt_run<KIND, T, false>(form, m, p, st);
    if (!lt_encode_out<T>(m, e, sp.splits, M, N)) return cudaErrorInvalidValue;
    return lt_run<KIND, T, true>(form, m, p, st);
}
template <typename T>
cudaError_t lin_tc_forward(const LinTc &q, const LinSplit &s, const LinEpi<T> &e, cudaStream_t st) {
    return lt_product<LIN_FWD, T>(q, s, e, nullptr, q.rows, q.out, q.in, st);
}
template <typename T>
cudaError_t lin_tc_dx(const LinTc &q, const LinSplit &s, const LinEpi<T> &e, cudaStream_t st) {
    return lt_product<LIN_DX, T>(q, s, e, nullptr, q.rows, q.in, q.out, st);
}
cudaError_t lin_tc_dw(const LinTc &q, const LinSplit &s, float *dW, float *db, cudaStream_t st) {
    LinEpi<float> e = {};
    e.out = dW;
    return lt_product<LIN_DW, float>(q, s, e, db, q.in, q.out, q.rows, st);
}
template cudaError_t lin_tc_forward<bf16>(const LinTc &, const LinSplit &, const LinEpi<bf16> &, cudaStream_t);
template cudaError_t lin_tc_forward<float>(const LinTc &, const LinSplit &, const LinEpi<float> &, cudaStream_t);
template cudaError_t lin_tc_dx<bf16>(const LinTc &, const LinSplit &, const LinEpi<bf16> &, cudaStream_t);
template cudaError_t lin_tc_dx<float>(const LinTc &, const LinSplit &, const LinEpi<float> &, cudaStream_t);

}  // namespace ops
}  // namespace eaga
