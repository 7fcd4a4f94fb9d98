// linear_pair.cu -- the dense product of linear.cu on CTA pairs (tcgen05 cta_group::2), for
// batches with enough rows to be bound by the tensor cores.
//
// A persistent cluster of two CTAs takes 256-row x 256-column tiles: each CTA holds the
// 128 x rows whose products it keeps and half of the 256 w rows (gated: the 128 w rows in
// CTA 0, the 128 w_up rows of the same columns in CTA 1), and one M = 256, N = 256 MMA
// reads both.  Per CTA a 128-column stage moves 64 KB for 256 x 256 x 128 products of the
// pair, half of what a lone CTA would move for the same work.  Two TMEM accumulators of 256
// columns let the epilogue of one tile run under the next one's products.
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

constexpr int PST = 3;                  // stages of 128 K columns
constexpr int P_SUB = 128 * 128;        // 128 rows x 64 columns
constexpr int P_OPER = 2 * P_SUB;       // one operand's stage
constexpr int P_STAGE = 2 * P_OPER;
constexpr int P_EPI_WARPS = 8;
constexpr int P_THREADS = 64 + 32 * P_EPI_WARPS;
constexpr int P_BAND = 8;               // row tiles of a band
constexpr int P_TURN = 32 * 32;         // floats of a warp's turning buffer

struct PairCtrl {
    uint64_t full[PST];   // leader: both CTAs' bytes of stage s landed (2 arrivals + tx)
    uint64_t empty[PST];  // each: the MMAs reading stage s finished
    uint64_t accf[2];     // each: accumulator a holds a finished tile
    uint64_t acce[2];     // leader: every epilogue warp of the pair drained accumulator a
    uint64_t fin;         // each: every MMA of the pair completed
    uint64_t bye;         // each: the other CTA is done touching this one
    uint64_t never;       // nothing ever arrives here (timeout test)
    uint32_t tmem_base;
};

constexpr size_t P_SMEM = 1024 + (size_t)PST * P_STAGE + P_EPI_WARPS * P_TURN * 4 + sizeof(PairCtrl);
static_assert(P_SMEM <= 227 * 1024, "one CTA's shared memory");

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

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
    linear_pair_kernel(const __grid_constant__ LinMaps maps, const LinArgs g)
{
    constexpr int BNO = GATED ? 128 : 256;  // output columns of a tile
    extern __shared__ uint8_t pair_smem[];
    const uint32_t pad = (1024u - (smem_u32(pair_smem) & 1023u)) & 1023u;
    uint8_t *buf = pair_smem + pad;  // stages: x chunks, w chunks
    float *turn = reinterpret_cast<float *>(buf + PST * P_STAGE);
    PairCtrl *S = reinterpret_cast<PairCtrl *>(turn + P_EPI_WARPS * P_TURN);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int mtiles = (g.M + 255) / 256, ntiles = (g.N + BNO - 1) / BNO;
    const int tiles = mtiles * ntiles, step = gridDim.x / 2, first = blockIdx.x / 2;
    const int kstages = (g.K + 127) / 128;

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
    if (warp == 1) tmem_alloc_pair(&S->tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = S->tmem_base;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            const CUtensorMap *wm = GATED && rank == 1 ? &maps.w_up : &maps.w;
            int issued = 0;
            bool ok = true;
            for (int i = first; ok && i < tiles; i += step) {
                const PairTile t = pair_tile(i, mtiles, ntiles);
                const int xr = t.mt * 256 + (int)rank * 128;
                const int wr = t.nt * BNO + (GATED ? 0 : (int)rank * 128);
                for (int k = 0; k < kstages; ++k, ++issued) {
                    const int s = issued % PST;
                    if (!wait2(&S->empty[s], (issued / PST & 1) ^ 1, g.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = peer_addr(&S->full[s], 0);
                    uint8_t *d = buf + s * P_STAGE;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&S->full[s], P_STAGE);
                    else
                        arrive_expect_tx_remote(fb, P_STAGE);
                    if (g.chunked) {
                        tma_load_3d_pair(d, &maps.x, fb, 0, xr, 2 * k);
                        tma_load_3d_pair(d + P_OPER, wm, fb, 0, wr, 2 * k);
                    } else {
                        for (int c = 0; c < 2; ++c) {
                            tma_load_2d_pair(d + c * P_SUB, &maps.x, fb, k * 128 + c * 64, xr);
                            tma_load_2d_pair(d + P_OPER + c * P_SUB, wm, fb, k * 128 + c * 64, wr);
                        }
                    }
                }
            }
            if (!ok) lin_record(g.status);
            if (rank == 0)  // never leave with either CTA's copies still landing
                for (int j = max(0, issued - PST); j < issued; ++j)
                    if (!wait2(&S->full[j % PST], j / PST & 1)) lin_record(g.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t IDESC = idesc_bf16_f32(256, 256);
            int used = 0, n = 0;
            bool ok = !(g.stall_test && !wait2(&S->never, 0, g.wait_ns));
            for (int i = first; ok && i < tiles; i += step, ++n) {
                const int a = n & 1;
                if (!wait2(&S->acce[a], (n / 2 & 1) ^ 1, g.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int k = 0; k < kstages; ++k, ++used) {
                    const int s = used % PST;
                    if (!wait2(&S->full[s], used / PST & 1, g.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t x0 = smem_u32(buf + s * P_STAGE), w0 = x0 + P_OPER;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t off = (j >> 2) * P_SUB + (j & 3) * 32;
                        mma_bf16_pair(tmem + a * 256, sw128_kmajor_desc(x0 + off), sw128_kmajor_desc(w0 + off), IDESC,
                                      (k | j) != 0);
                    }
                    mma_commit_pair(&S->empty[s]);
                }
                if (ok) mma_commit_pair(&S->accf[a]);
            }
            if (!ok) lin_record(g.status);
            mma_commit_pair(&S->fin);  // once every MMA issued here has completed
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) / 4;
        float *my = turn + (warp - 2) * P_TURN;
        int n = 0;
        for (int i = first; i < tiles; i += step, ++n) {
            const int a = n & 1;
            if (!wait2(&S->accf[a], n / 2 & 1, g.wait_ns)) {
                lin_record(g.status);
                break;
            }
            __syncwarp();
            tc_fence_after();
            const PairTile t = pair_tile(i, mtiles, ntiles);
            const int row0 = t.mt * 256 + (int)rank * 128 + q * 32;
            const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + a * 256;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                // 32 accumulator columns of this lane's row (gated: 16 of w, 16 of w_up), its
                // 16-byte pieces at p ^ (row % 8) so that neither side meets a bank twice
                uint32_t r[32];
                if (GATED) {
                    uint32_t lo[16], hi[16];
                    tmem_ld16x2_sync(tb + half * 64 + c * 16, tb + 128 + half * 64 + c * 16, lo, hi);
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = lo[j], r[16 + j] = hi[j];
                } else {
                    tmem_ld32_sync(tb + half * 128 + c * 32, r);
                }
                if (c == 3) {  // the accumulator is free for the tile after next
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(&S->acce[a]);
                        else
                            arrive_remote(peer_addr(&S->acce[a], 0));
                    }
                }
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    *reinterpret_cast<uint4 *>(my + lane * 32 + ((p ^ (lane & 7)) * 4)) =
                        make_uint4(r[4 * p], r[4 * p + 1], r[4 * p + 2], r[4 * p + 3]);
                __syncwarp();
                if (GATED) {
                    const LinCols cols(g, t.nt * BNO + half * 64 + c * 16 + (lane & 3) * 4);
#pragma unroll 1
                    for (int it = 0; it < 4; ++it) {
                        const int rr = it * 8 + lane / 8 + (lane >> 2 & 1) * 4, p = lane & 3;
                        const float4 v = *reinterpret_cast<const float4 *>(my + rr * 32 + ((p ^ (rr & 7)) * 4));
                        const float4 u = *reinterpret_cast<const float4 *>(my + rr * 32 + (((p + 4) ^ (rr & 7)) * 4));
                        float o[4] = {v.x, v.y, v.z, v.w};
                        const float up[4] = {u.x, u.y, u.z, u.w};
                        if (row0 + rr < g.M) lin_finish4<true>(g, cols, row0 + rr, o, up);
                    }
                } else {
                    const LinCols cols(g, t.nt * BNO + half * 128 + c * 32 + (lane & 7) * 4);
#pragma unroll 1
                    for (int it = 0; it < 8; ++it) {
                        const int rr = it * 4 + lane / 8, p = lane & 7;
                        const float4 v = *reinterpret_cast<const float4 *>(my + rr * 32 + ((p ^ (rr & 7)) * 4));
                        float o[4] = {v.x, v.y, v.z, v.w};
                        const float up[4] = {0.f, 0.f, 0.f, 0.f};
                        if (row0 + rr < g.M) lin_finish4<false>(g, cols, row0 + rr, o, up);
                    }
                }
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        // every MMA of the pair (which reads this CTA's shared memory and writes its
        // TMEM) has completed before TMEM is freed and the CTA may leave
        if (lane == 0 && !wait2(&S->fin, 0)) lin_record(g.status);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    __syncthreads();
    if (threadIdx.x == 0) {  // leave only after the other CTA is done with this one
        arrive_remote(peer_addr(&S->bye, rank ^ 1u));
        if (!wait2(&S->bye, 0)) lin_record(g.status);
    }
    __syncthreads();
}

template <bool GATED>
cudaError_t launch_pair(const LinMaps &maps, const LinArgs &g, cudaStream_t st)
{
    static std::mutex mu;
    static uint64_t done = 0;  // per device: the kernel's shared memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!(done >> dev & 1ull)) {
            e = cudaFuncSetAttribute(linear_pair_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)P_SMEM);
            if (e != cudaSuccess) return e;
            done |= 1ull << dev;
        }
    }
    const int bno = GATED ? 128 : 256;
    const long long tiles = (long long)((g.M + 255) / 256) * ((g.N + bno - 1) / bno);
    const int clusters = num_sms() / 2 < tiles ? num_sms() / 2 : (int)tiles;
    return launch_pdl(linear_pair_kernel<GATED>, dim3(2 * clusters), dim3(P_THREADS), P_SMEM, st, maps, g);
}

}  // namespace

cudaError_t launch_linear_pair(const LinMaps &maps, const LinArgs &g, bool gated, cudaStream_t st)
{
    return gated ? launch_pair<true>(maps, g, st) : launch_pair<false>(maps, g, st);
}

}  // namespace moe
