// linear_pair.cu -- the dense product of linear.cu on CTA pairs (tcgen05 cta_group::2), for
// batches with enough rows to be bound by the tensor cores.
//
// A persistent cluster of two CTAs takes 256-row x NB-column tiles (NB 256, or 128 where
// that leaves too many SMs idle): each CTA holds the 128 x rows whose products it keeps
// and half of the NB w rows (gated: NB / 2 w rows in CTA 0, the w_up rows of the same columns
// in CTA 1), and one M = 256, N = NB MMA reads both.  Per CTA a 128-column stage of
// NB = 256 moves 64 KB for 256 x 256 x 128 products of the pair, half of what a lone CTA
// would move for the same work.  Two TMEM accumulators of NB columns let the epilogue of one
// tile run under the next one's products.
//
// Warp 0 streams x and w (TMA), warp 1 of CTA 0 issues the MMAs, warps 2-9 finish tiles:
// each takes its 32 accumulator rows, a lane each, and half the columns in boxes of 32, applies
// bias, activation and gate in registers, and stores a box from shared memory by
// tensor map; the residual's box arrives at the same place before.  (Rows turned in shared
// memory and stored four columns a lane took 3700 cycles a box's worth, whose latency a tile
// that is a CTA's last does not hide: 512 x 2048 x 2048 11.6 us.)  Where rows of out or
// residual are not 16-byte aligned a box is written row by row, a column a lane, and so is the last
// box of aligned rows whose N ends inside of a 16-byte piece.  Tiles are
// dealt out statically, bands of 8 row tiles walked column by column, so that the
// tiles in flight share x and w rows in L2.  Every wait is bounded.
#include <mutex>

#include "linear.cuh"
#include "moe_internal.h"
#include "pair_ptx.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int P_SUB = 128 * 128;        // 128 x rows x 64 columns
constexpr int P_EPI_WARPS = 8;
constexpr int P_THREADS = 64 + 32 * P_EPI_WARPS;
constexpr int P_BAND = 8;               // row tiles of a band
constexpr int P_BOX = 4096;             // bytes of a warp's boxes: 32 x 32 fp32, or two of bf16 in turn
constexpr int PST_MAX = 4;

// Tiles of 256 rows x NB accumulator columns; a CTA's stage: 128 x rows, NB / 2 w rows, 128
// columns of K each.
template <int NB>
struct PairShape {
    static constexpr int W_SUB = NB / 2 * 128;  // NB / 2 w rows x 64 columns
    static constexpr int STAGE = 2 * (P_SUB + W_SUB);
    static constexpr int ST = NB == 256 ? 3 : 4;
};

struct PairCtrl {
    uint64_t full[PST_MAX];   // leader: both CTAs' bytes of stage s landed (2 arrivals + tx)
    uint64_t empty[PST_MAX];  // each: the MMAs reading stage s finished
    uint64_t accf[2];     // each: accumulator a holds a finished tile
    uint64_t acce[2];     // leader: every epilogue warp of the pair drained accumulator a
    uint64_t fin;         // each: every MMA of the pair completed
    uint64_t res[2 * P_EPI_WARPS];  // the residual's box of an epilogue warp is here
    uint64_t never;       // nothing ever arrives here (timeout test)
    uint32_t tmem_base;
};

template <int NB>
constexpr size_t kPairSmem =
    1024 + (size_t)PairShape<NB>::ST * PairShape<NB>::STAGE + P_EPI_WARPS * P_BOX + sizeof(PairCtrl);
static_assert(kPairSmem<256> <= 227 * 1024 && kPairSmem<128> <= 227 * 1024, "one CTA's shared memory");

struct PairTile {
    int mt, nt;
};
// Tile i in bands of P_BAND row tiles, column tile by column tile inside a band.
__device__ __forceinline__ PairTile pair_tile(int i, int mtiles, int ntiles)
{
    const int band = i / (P_BAND * ntiles), at = i - band * P_BAND * ntiles;
    const int h = min(P_BAND, mtiles - band * P_BAND);
    return {band * P_BAND + at % h, at / h};
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *tm, const void *src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(tm)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
// At most N of this thread's stores still read shared memory.
template <int N>
__device__ __forceinline__ void stores_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Box (row, col) row by row, a column a lane, with plain accesses: fp32 in `from`, 16-byte
// piece p of row r at p ^ (r % 8).  FULL: all 32 rows are there, none needs a test.
template <typename T, bool FULL>
__device__ __forceinline__ void store_rows(const LinArgs &g, const uint8_t *from, int row, int rows, int c, int lane)
{
    T *out = static_cast<T *>(g.out) + (int64_t)row * g.ldo + c;
    const T *res = static_cast<const T *>(g.res) + (int64_t)row * g.ldr + c;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 16) {
        T r[16];
        if (g.res)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (FULL || r0 + i < rows) r[i] = res[(r0 + i) * g.ldr];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float o = *reinterpret_cast<const float *>(from + (r0 + i) * 128 + ((lane / 4) ^ (i & 7)) * 16 + lane % 4 * 4);
            if (g.res) o += static_cast<float>(r[i]);
            if (FULL || r0 + i < rows) out[(r0 + i) * g.ldo] = static_cast<T>(o);
        }
    }
}

// The box of finished values at `from`, laid out as its tensor map has it, row by row, a column a lane:
// those inside out only.
template <typename T>
__device__ __forceinline__ void store_box_rows(const LinArgs &g, const uint8_t *from, int row, int col, int lane)
{
    constexpr int EACH = 16 / (int)sizeof(T);  // columns of a 16-byte piece
    const int rows = min(32, g.M - row);
    if (col + lane >= g.N) return;
    T *out = static_cast<T *>(g.out) + (int64_t)row * g.ldo + col + lane;
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        const int swizzle = sizeof(T) == 4 ? r & 7 : r >> 1 & 3;
        out[r * g.ldo] = *reinterpret_cast<const T *>(from + r * 32 * (int)sizeof(T) + ((lane / EACH) ^ swizzle) * 16 +
                                                      lane % EACH * (int)sizeof(T));
    }
}

// An epilogue warp's part of the tiles: rows 32 (ew % 4) .. of the CTA's 128, columns ew / 4 of
// two halves.
template <int NB, bool GATED, bool PROMOTE>
__device__ __forceinline__ void pair_epilogue(const LinMaps &maps, const LinArgs &g, PairCtrl *S, uint8_t *box,
                                              uint32_t tmem, int ew, int lane, uint32_t rank, int part)
{
    constexpr int BNO = GATED ? NB / 2 : NB, BOXES = BNO / 2 / 32;
    const int warp = ew + 2, q = warp & 3, half = ew / 4;  // a warp reads the TMEM lanes of its quarter
    const int mtiles = (g.M + 255) / 256, ntiles = (g.N + BNO - 1) / BNO;
    const int tiles = mtiles * ntiles, step = gridDim.x / 2, first = blockIdx.x / 2;
    const int kstages = (g.K + 127) / 128;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * (BNO / 2);
    const bool as_f32 = g.out_f32 || !g.maps_out;  // a box's type
    const int row_bytes = as_f32 ? 128 : 64, turns = as_f32 ? 1 : 2;
    const int swizzle = as_f32 ? lane & 7 : lane >> 1 & 3;
    uint64_t *rbar = &S->res[2 * ew];
    const bool res_maps = g.res && g.maps_out;

    auto origin = [&](const PairTile &t, int &row, int &col) {
        row = t.mt * 256 + (int)rank * 128 + q * 32;
        col = t.nt * BNO + half * (BNO / 2);
    };
    auto boxes_of = [&](int row, int col) {  // how many boxes of a tile lie in out, from the first on
        return row < g.M && col < g.N ? min(BOXES, (g.N - col + 31) / 32) : 0;
    };
    int bx = 0, loads = 0;  // boxes begun, residual boxes asked for
    // the residual's box into place `slot`, once what was stored from there has been read
    auto load_residual = [&](int slot, int row, int col) {
        if (lane == 0) {
            stores_read<0>();
            mbar_arrive_expect_tx(rbar + slot, 32 * row_bytes);
            tma_load_2d(box + slot * 2048, &maps.res, rbar + slot, col, row);
        }
        ++loads;
        __syncwarp();
    };
    // the residual of the next box after box j of `count` of tile i
    auto load_next = [&](int i, int j, int count, int row, int col) {
        if (j + 1 < count) {
            load_residual(bx & (turns - 1), row, col + (j + 1) * 32);
            return;
        }
        for (i += step; i < tiles; i += step) {
            origin(pair_tile(i, mtiles, ntiles), row, col);
            if (boxes_of(row, col)) {
                load_residual(bx & (turns - 1), row, col);
                return;
            }
        }
    };
    auto drained = [&](int a) {  // the accumulator is free for the part after next
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (rank == 0)
                mbar_arrive(&S->acce[a]);
            else
                arrive_remote(peer_addr(&S->acce[a], 0));
        }
    };
    // 16 columns, the part h of a box at `to`: v the products with w, u those with w_up
    auto finish = [&](float (&v)[4][4], const float (&u)[4][4], uint8_t *to, int h, float bias,
                      float bias_up) __attribute__((always_inline)) {
        if (g.bias)
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i / 4][i % 4] += __shfl_sync(0xffffffffu, bias, h * 16 + i);
        lin_act_all(g.act, v);
        if (GATED)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i / 4][i % 4] *= u[i / 4][i % 4] + __shfl_sync(0xffffffffu, bias_up, h * 16 + i);
        uint8_t *mine = to + lane * row_bytes;
        if (as_f32) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float4 *at = reinterpret_cast<float4 *>(mine + ((h * 4 + p) ^ swizzle) * 16);
                if (res_maps) {
                    const float4 r = *at;
                    v[p][0] += r.x, v[p][1] += r.y, v[p][2] += r.z, v[p][3] += r.w;
                }
                *at = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
            }
        } else {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint4 *at = reinterpret_cast<uint4 *>(mine + ((h * 2 + p) ^ swizzle) * 16);
                uint32_t w[4];
                if (res_maps) {
                    const uint4 r = *at;
                    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a = v[2 * p + i / 2][i % 2 * 2], b = v[2 * p + i / 2][i % 2 * 2 + 1];
                    if (res_maps) {
                        a += __uint_as_float(w[i] << 16);
                        b += __uint_as_float(w[i] & 0xffff0000u);
                    }
                    const __nv_bfloat162 o = __floats2bfloat162_rn(a, b);
                    w[i] = *reinterpret_cast<const uint32_t *>(&o);
                }
                *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };

    if (res_maps) load_next(first - step, 0, 0, 0, 0);
    int n = 0;  // accumulators read
    for (int i = first; i < tiles; i += step) {
        int row, col;
        origin(pair_tile(i, mtiles, ntiles), row, col);
        const int count = boxes_of(row, col);
        float bias[BOXES], bias_up[BOXES];  // a column a lane
#pragma unroll
        for (int j = 0; j < BOXES; ++j) {
            const int c = col + j * 32 + lane;
            bias[j] = g.bias && c < g.N ? g.bias[c] : 0.0f;
            bias_up[j] = GATED && g.bias_up && c < g.N ? g.bias_up[c] : 0.0f;
        }
        float sum[PROMOTE ? NB / 2 : 1];
        uint32_t acc = lanes;
        if constexpr (PROMOTE) {
#pragma unroll
            for (int j = 0; j < NB / 2; ++j) sum[j] = 0.0f;
        }
        const int parts = PROMOTE ? (kstages + part - 1) / part : 1;
        for (int k = 0; k < parts; ++k) {
            if (!wait2(&S->accf[n & 1], n / 2 & 1, g.wait_ns)) {
                lin_record(g.status);
                stores_done();  // never leave with copies still landing
                if (loads > bx && !mbar_wait(rbar + (bx & (turns - 1)), bx / turns & 1)) lin_record(g.status);
                __syncwarp();
                return;
            }
            __syncwarp();
            tc_fence_after();
            acc = lanes + (n & 1) * NB;
            if constexpr (PROMOTE) {
#pragma unroll
                for (int c = 0; c < NB / 32; ++c) {
                    uint32_t r[16];
                    tmem_ld16_sync(acc + (GATED && c >= NB / 64 ? NB / 2 + (c - NB / 64) * 16 : c * 16), r);
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[c * 16 + j] += __uint_as_float(r[j]);
                }
                drained(n & 1);
            } else if (count == 0) {
                drained(n & 1);
            }
            ++n;
        }
#pragma unroll(PROMOTE ? BOXES : 1)
        for (int j = 0; j < BOXES; ++j) {
            if (j >= count) continue;
            const int slot = bx & (turns - 1);
            uint8_t *to = box + slot * 2048;
            float b = bias[0], bu = bias_up[0];
#pragma unroll
            for (int k = 1; k < BOXES; ++k)
                if (j == k) b = bias[k], bu = bias_up[k];
            if (res_maps) {
                if (!mbar_wait(rbar + slot, bx / turns & 1, g.wait_ns)) lin_record(g.status);
            } else if (g.maps_out && lane == 0) {
                if (turns == 2)
                    stores_read<1>();
                else
                    stores_read<0>();
            }
            __syncwarp();
            ++bx;
            if (res_maps && turns == 2) load_next(i, j, count, row, col);
#pragma unroll(PROMOTE ? 2 : 1)
            for (int h = 0; h < 2; ++h) {
                float v[4][4], u[4][4];
                if constexpr (PROMOTE) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        v[e / 4][e % 4] = sum[(2 * j + h) * 16 + e];
                        if (GATED) u[e / 4][e % 4] = sum[NB / 4 + (2 * j + h) * 16 + e];
                    }
                } else {
                    uint32_t lo[16], hi[16];
                    const uint32_t at = acc + (2 * j + h) * 16;
                    if (GATED)
                        tmem_ld16x2_sync(at, at + NB / 2, lo, hi);
                    else
                        tmem_ld16_sync(at, lo);
                    if (h == 1 && j == count - 1) drained((n - 1) & 1);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        v[e / 4][e % 4] = __uint_as_float(lo[e]);
                        if (GATED) u[e / 4][e % 4] = __uint_as_float(hi[e]);
                    }
                }
                finish(v, u, to, h, b, bu);
            }
            if (g.maps_out) {
                // A tensor-map store writes 16-byte pieces whole, those that the last column lies in too: up
                // to 14 bytes behind a row of N columns.  The last box of such rows goes by plain stores.
                const bool plain = col + j * 32 + 31 >= g.N && g.N % (g.out_f32 ? 4 : 8) != 0;
                if (plain) {
                    __syncwarp();
                    if (g.out_f32)
                        store_box_rows<float>(g, to, row, col + j * 32, lane);
                    else
                        store_box_rows<__nv_bfloat16>(g, to, row, col + j * 32, lane);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && !plain) tma_store_2d(&maps.out, to, col + j * 32, row);
                if (res_maps && turns == 1) load_next(i, j, count, row, col);
            } else {
                __syncwarp();
                const int c = col + j * 32 + lane, rows = min(32, g.M - row);
                if (c < g.N) {
                    if (g.out_f32) {
                        rows == 32 ? store_rows<float, true>(g, to, row, rows, c, lane)
                                   : store_rows<float, false>(g, to, row, rows, c, lane);
                    } else {
                        rows == 32 ? store_rows<__nv_bfloat16, true>(g, to, row, rows, c, lane)
                                   : store_rows<__nv_bfloat16, false>(g, to, row, rows, c, lane);
                    }
                }
            }
            __syncwarp();
        }
    }
    stores_done();
}

// PROMOTE: after every 512 columns of K the accumulator is added to fp32 registers of the
// epilogue warps (see kPromote).
template <int NB, bool GATED, bool PROMOTE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
    linear_pair_kernel(const __grid_constant__ LinMaps maps, const LinArgs g)
{
    constexpr int BNO = GATED ? NB / 2 : NB;  // output columns of a tile
    constexpr int PST = PairShape<NB>::ST, P_STAGE = PairShape<NB>::STAGE, W_SUB = PairShape<NB>::W_SUB;
    extern __shared__ uint8_t pair_smem[];
    const uint32_t pad = (1024u - (smem_u32(pair_smem) & 1023u)) & 1023u;
    uint8_t *buf = pair_smem + pad;  // stages: x chunks, w chunks
    uint8_t *boxes = buf + PST * P_STAGE;
    PairCtrl *S = reinterpret_cast<PairCtrl *>(boxes + P_EPI_WARPS * P_BOX);
    const int warp = uniform_warp(), lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int mtiles = (g.M + 255) / 256, ntiles = (g.N + BNO - 1) / BNO;
    const int tiles = mtiles * ntiles, step = gridDim.x / 2, first = blockIdx.x / 2;
    const int kstages = (g.K + 127) / 128;
    const int part = PROMOTE ? kPromote / 128 : kstages;  // K stages of an accumulator

    if (threadIdx.x == 0) {
        for (int s = 0; s < PST; ++s) {
            mbar_init(&S->full[s], 2);
            mbar_init(&S->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&S->accf[a], 1);
            mbar_init(&S->acce[a], 2 * P_EPI_WARPS);
        }
        mbar_init(&S->fin, 1);
        for (int i = 0; i < 2 * P_EPI_WARPS; ++i) mbar_init(&S->res[i], 1);
        mbar_init(&S->never, 1);
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(GATED && rank == 1 ? &maps.w_up : &maps.w);
        if (g.maps_out) tma_prefetch_desc(&maps.out);
        if (g.maps_out && g.res) tma_prefetch_desc(&maps.res);
    }
    if (warp == 1) tmem_alloc_pair(&S->tmem_base, 2 * NB);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, S->tmem_base, 0);
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        const CUtensorMap *wm = GATED && rank == 1 ? &maps.w_up : &maps.w;
        int s = 0, issued = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int i = first; ok && i < tiles; i += step) {
            const PairTile t = pair_tile(i, mtiles, ntiles);
            const int xr = t.mt * 256 + (int)rank * 128;
            const int wr = t.nt * BNO + (GATED ? 0 : (int)rank * (NB / 2));
            for (int k = 0; k < kstages; ++k, ++issued) {
                if (!warp_wait2(&S->empty[s], ph, g.wait_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = peer_addr(&S->full[s], 0);
                uint8_t *d = buf + s * P_STAGE;
                if (elect_one()) {
                    if (rank == 0)
                        mbar_arrive_expect_tx(&S->full[s], P_STAGE);
                    else
                        arrive_expect_tx_remote(fb, P_STAGE);
                    if (g.chunked) {
                        tma_load_3d_pair(d, &maps.x, fb, 0, xr, 2 * k);
                        tma_load_3d_pair(d + 2 * P_SUB, wm, fb, 0, wr, 2 * k);
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            tma_load_2d_pair(d + c * P_SUB, &maps.x, fb, k * 128 + c * 64, xr);
                            tma_load_2d_pair(d + 2 * P_SUB + c * W_SUB, wm, fb, k * 128 + c * 64, wr);
                        }
                    }
                }
                __syncwarp();
                if (++s == PST) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) {
            if (!ok) lin_record(g.status);
            if (rank == 0)  // never leave with either CTA's copies still landing
                for (int j = max(0, issued - PST); j < issued; ++j)
                    if (!wait2(&S->full[j % PST], j / PST & 1)) lin_record(g.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t IDESC = idesc_bf16_f32(256, NB);
            const uint32_t buf0 = smem_u32(buf);
            int s = 0, n = 0;
            uint32_t ph = 0;
            bool ok = !(g.stall_test && !warp_wait2(&S->never, 0, g.wait_ns));
            for (int i = first; ok && i < tiles; i += step)
                for (int k0 = 0; ok && k0 < kstages; k0 += part, ++n) {
                    const int a = n & 1;
                    if (!warp_wait2(&S->acce[a], (n / 2 & 1) ^ 1, g.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int k1 = min(kstages, k0 + part);
                    for (int k = k0; k < k1; ++k) {
                        if (!warp_wait2(&S->full[s], ph, g.wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t x0 = buf0 + s * P_STAGE, w0 = x0 + 2 * P_SUB;
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                mma_bf16_pair(tmem + a * NB, sw128_kmajor_desc(x0 + (j >> 2) * P_SUB + (j & 3) * 32),
                                              sw128_kmajor_desc(w0 + (j >> 2) * W_SUB + (j & 3) * 32), IDESC,
                                              (k - k0 | j) != 0);
                            mma_commit_pair(&S->empty[s]);
                            if (k == k1 - 1) mma_commit_pair(&S->accf[a]);
                        }
                        __syncwarp();
                        if (++s == PST) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                }
            if (!ok && lane == 0) lin_record(g.status);
            if (elect_one()) mma_commit_pair(&S->fin);  // once every MMA issued here has completed
        }
        __syncwarp();
    } else {
        pair_epilogue<NB, GATED, PROMOTE>(maps, g, S, boxes + (warp - 2) * P_BOX, tmem, warp - 2, lane, rank, part);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        // every MMA of the pair (which reads this CTA's shared memory and writes its
        // TMEM) has completed before TMEM is freed and the CTA may leave
        if (lane == 0 && !wait2(&S->fin, 0)) lin_record(g.status);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * NB);
    }
    // leave only after the other CTA is done with this one (nothing is published: relaxed)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int NB, bool GATED, bool PROMOTE>
cudaError_t launch_pair(const LinMaps &maps, const LinArgs &g, cudaStream_t st)
{
    static std::mutex mu;
    static uint64_t done = 0;  // per device: the kernel's shared memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    auto kern = linear_pair_kernel<NB, GATED, PROMOTE>;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!(done >> dev & 1ull)) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem<NB>);
            if (e != cudaSuccess) return e;
            done |= 1ull << dev;
        }
    }
    const int bno = GATED ? NB / 2 : NB;
    const long long tiles = (long long)((g.M + 255) / 256) * ((g.N + bno - 1) / bno);
    const int clusters = num_sms() / 2 < tiles ? num_sms() / 2 : (int)tiles;
    return launch_pdl(kern, dim3(2 * clusters), dim3(P_THREADS), kPairSmem<NB>, st, maps, g);
}


}  // namespace

cudaError_t launch_linear_pair(const LinMaps &maps, const LinArgs &g, bool gated, int nb, cudaStream_t st)
{
    if (g.promote) {  // the sums of a 256-column tile would not fit the epilogue's registers
        if (nb != 128) return cudaErrorInvalidValue;
        return gated ? launch_pair<128, true, true>(maps, g, st) : launch_pair<128, false, true>(maps, g, st);
    }
    if (nb == 256) return gated ? launch_pair<256, true, false>(maps, g, st) : launch_pair<256, false, false>(maps, g, st);
    return gated ? launch_pair<128, true, false>(maps, g, st) : launch_pair<128, false, false>(maps, g, st);
}

}  // namespace moe
