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
// each reads its 32 accumulator rows 32 columns at a time, turns them in shared memory so
// that a row's columns lie in neighbouring lanes, and finishes four columns a lane (one
// contiguous run of residual and out a row, whatever the rows' alignment).  Tiles are
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
constexpr int P_TURN = 32 * 32;         // floats of a warp's turning buffer
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
    uint64_t bye;         // each: the other CTA is done touching this one
    uint64_t never;       // nothing ever arrives here (timeout test)
    uint32_t tmem_base;
};

template <int NB>
constexpr size_t kPairSmem =
    1024 + (size_t)PairShape<NB>::ST * PairShape<NB>::STAGE + P_EPI_WARPS * P_TURN * 4 + sizeof(PairCtrl);
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
    float *turn = reinterpret_cast<float *>(buf + PST * P_STAGE);
    PairCtrl *S = reinterpret_cast<PairCtrl *>(turn + P_EPI_WARPS * P_TURN);
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
        mbar_init(&S->bye, 1);
        mbar_init(&S->never, 1);
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(GATED && rank == 1 ? &maps.w_up : &maps.w);
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
        const int q = warp & 3, half = (warp - 2) / 4;
        float *my = turn + (warp - 2) * P_TURN;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        // chunk c of this warp's NB / 2 accumulator columns: 32 of them (gated: 16 of w, 16 of w_up)
        auto load = [&](int a, int c, uint32_t (&r)[32]) {
            const uint32_t tb = lanes + a * NB;
            if (GATED) {
                uint32_t lo[16], hi[16];
                tmem_ld16x2_sync(tb + half * (NB / 4) + c * 16, tb + NB / 2 + half * (NB / 4) + c * 16, lo, hi);
#pragma unroll
                for (int j = 0; j < 16; ++j) r[j] = lo[j], r[16 + j] = hi[j];
            } else {
                tmem_ld32_sync(tb + half * (NB / 2) + c * 32, r);
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
        // turns the chunk and finishes it, the 16-byte pieces of row r at p ^ (r % 8) so that
        // neither side meets a bank twice
        auto finish = [&](const PairTile &t, int c, const uint32_t (&r)[32]) {
            const int row0 = t.mt * 256 + (int)rank * 128 + q * 32;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                *reinterpret_cast<uint4 *>(my + lane * 32 + ((p ^ (lane & 7)) * 4)) =
                    make_uint4(r[4 * p], r[4 * p + 1], r[4 * p + 2], r[4 * p + 3]);
            __syncwarp();
            // lane l: four columns of row r0 + it * RW; the residual of four rows at a time is in flight
            constexpr int RW = GATED ? 8 : 4;
            const int p = GATED ? lane & 3 : lane & 7;
            const int r0 = GATED ? lane / 8 + (lane >> 2 & 1) * 4 : lane / 8;
            const LinCols cols(g, t.nt * BNO + half * (BNO / 2) + c * (GATED ? 16 : 32) + p * 4);
#pragma unroll 1
            for (int it = 0; it < 32 / RW; it += 4) {
                float v[4][4], u[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = r0 + (it + j) * RW;
                    const float4 a = *reinterpret_cast<const float4 *>(my + rr * 32 + ((p ^ (rr & 7)) * 4));
                    v[j][0] = a.x, v[j][1] = a.y, v[j][2] = a.z, v[j][3] = a.w;
                    if (GATED) {
                        const float4 b = *reinterpret_cast<const float4 *>(my + rr * 32 + (((p + 4) ^ (rr & 7)) * 4));
                        u[j][0] = b.x, u[j][1] = b.y, u[j][2] = b.z, u[j][3] = b.w;
                    }
                }
                lin_finish<GATED>(g, cols, row0 + r0 + it * RW, RW, g.M, v, u);
            }
            __syncwarp();
        };
        int n = 0;
        bool ok = true;
        for (int i = first; ok && i < tiles; i += step) {
            const PairTile t = pair_tile(i, mtiles, ntiles);
            if (!PROMOTE) {
                const int a = n & 1;
                if (!wait2(&S->accf[a], n / 2 & 1, g.wait_ns)) {
                    ok = false;
                    break;
                }
                ++n;
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < NB / 64; ++c) {
                    uint32_t r[32];
                    load(a, c, r);
                    if (c == NB / 64 - 1) drained(a);
                    finish(t, c, r);
                }
                continue;
            }
            float sum[NB / 2];
#pragma unroll
            for (int j = 0; j < NB / 2; ++j) sum[j] = 0.0f;
            for (int k0 = 0; k0 < kstages; k0 += part, ++n) {
                const int a = n & 1;
                if (!wait2(&S->accf[a], n / 2 & 1, g.wait_ns)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < NB / 64; ++c) {
                    uint32_t r[32];
                    load(a, c, r);
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c * 32 + j] += __uint_as_float(r[j]);
                }
                drained(a);
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < NB / 64; ++c) {
                uint32_t r[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(sum[c * 32 + j]);
                finish(t, c, r);
            }
        }
        if (!ok) lin_record(g.status);
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
    __syncthreads();
    if (threadIdx.x == 0) {  // leave only after the other CTA is done with this one
        arrive_remote(peer_addr(&S->bye, rank ^ 1u));
        if (!wait2(&S->bye, 0)) lin_record(g.status);
    }
    __syncthreads();
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

template <int NB>
cudaError_t launch_pair_nb(const LinMaps &maps, const LinArgs &g, bool gated, cudaStream_t st)
{
    if (g.promote)
        return gated ? launch_pair<NB, true, true>(maps, g, st) : launch_pair<NB, false, true>(maps, g, st);
    return gated ? launch_pair<NB, true, false>(maps, g, st) : launch_pair<NB, false, false>(maps, g, st);
}

}  // namespace

cudaError_t launch_linear_pair(const LinMaps &maps, const LinArgs &g, bool gated, int nb, cudaStream_t st)
{
    return nb == 256 ? launch_pair_nb<256>(maps, g, gated, st) : launch_pair_nb<128>(maps, g, gated, st);
}

}  // namespace moe
