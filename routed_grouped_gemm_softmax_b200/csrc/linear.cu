// linear.cu -- dense products with the layer's elementwise work in their epilogue:
//
//   out = act(x w^T + bias) [* (x w_up^T + bias_up)] [+ residual]
//
// x [M, K], w and w_up [N, K] bf16, products accumulated in fp32 on the tensor cores,
// bias in fp32, one rounding to the output's type at the end.
//
// linear_kernel: 128 rows of w (gated: 64 of w over 64 of w_up) on the MMA's M side and BN
// rows of x on its N side, so that the tensor work of a short batch follows its rows.  A
// tile's K range is split over the S CTAs of a cluster; each leaves its fp32 partial tile in
// its own shared memory, and every CTA then sums its share of the tile's rows over the S
// partials (in rank order, through distributed shared memory) and finishes them.
// With at most half an SM's shared memory a CTA, two are resident per SM: 33 clusters of 8
// fit on the GPU, where one CTA an SM leaves room for 15 (the GPCs' SMs do not divide by
// 8) and 16 x (2 x 2048) x 7168 ran in two waves, 22.9 us.
// linear_pair.cu takes the batches with enough rows to be bound by the tensor cores.
#include <mutex>

#include "linear.cuh"
#include "moe_internal.h"
#include "pdl.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int LBM = 128;             // w rows per tile
constexpr int LSTAGES_MAX = 8;
constexpr int LW_BYTES = LBM * 128;  // one 64-column chunk of 128 w rows
constexpr int LTHREADS = 192;        // warps 0-3: accumulators; 4: TMA; 5: MMA; all: epilogue
constexpr int L_HALF_SM = 113 * 1024;  // shared memory of a CTA of which an SM holds two

struct LinCtrl {
    uint64_t full[LSTAGES_MAX];
    uint64_t empty[LSTAGES_MAX];
    uint64_t accf[2];  // accumulator a holds a finished part
    uint64_t acce[2];  // its four warps have read it
    uint64_t fin;      // every MMA of this CTA is done
    uint64_t never;    // nothing ever arrives here (timeout test)
    uint32_t tmem_base;
};

__device__ __forceinline__ void lin_cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void lin_cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(r)
                 : "memory");
    return v;
}

// Rows rank, rank + S, ... of the tile, each the sum over the cluster's partials.
template <int BN, bool GATED>
__device__ __forceinline__ void finish_rows(const LinArgs &g, const float *tile_f, int nt, int mt, int rank)
{
    constexpr int COLS = GATED ? LBM / 2 : LBM, LANES = COLS / 4, RW = 32 / LANES;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, at = (lane % LANES) * 4;
    const LinCols cols(g, nt * COLS + at);
    const int rows = min(BN, g.M - mt * BN);
    const uint32_t base = smem_u32(tile_f);
    for (int t = rank + g.split * (warp * RW + lane / LANES); t < rows; t += g.split * (LTHREADS / 32) * RW) {
        float v[4], u[4] = {0.f, 0.f, 0.f, 0.f};
        if (g.split == 1) {
            const float4 a = *reinterpret_cast<const float4 *>(tile_f + t * LBM + at);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            if (GATED) {
                const float4 b = *reinterpret_cast<const float4 *>(tile_f + t * LBM + COLS + at);
                u[0] = b.x, u[1] = b.y, u[2] = b.z, u[3] = b.w;
            }
        } else {
            float4 a[8], b[8];  // every rank's loads in flight before the first sum
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < g.split) {
                    a[q] = ld_cluster4(base + (t * LBM + at) * 4, q);
                    if (GATED) b[q] = ld_cluster4(base + (t * LBM + COLS + at) * 4, q);
                }
            v[0] = a[0].x, v[1] = a[0].y, v[2] = a[0].z, v[3] = a[0].w;
            if (GATED) u[0] = b[0].x, u[1] = b[0].y, u[2] = b[0].z, u[3] = b[0].w;
#pragma unroll
            for (int q = 1; q < 8; ++q)
                if (q < g.split) {
                    v[0] += a[q].x, v[1] += a[q].y, v[2] += a[q].z, v[3] += a[q].w;
                    if (GATED) u[0] += b[q].x, u[1] += b[q].y, u[2] += b[q].z, u[3] += b[q].w;
                }
        }
        lin_finish4<GATED>(g, cols, (int64_t)mt * BN + t, v, u);
    }
}

template <int BN>
__global__ void __launch_bounds__(LTHREADS)
linear_kernel(const __grid_constant__ LinMaps maps, const LinArgs g)
{
    constexpr uint32_t ACC = BN < 32 ? 32 : BN;  // TMEM columns of an accumulator
    extern __shared__ uint8_t lin_smem[];
    const uint32_t pad = (1024u - (smem_u32(lin_smem) & 1023u)) & 1023u;
    uint8_t *buf = lin_smem + pad;  // stages: w chunks, x chunks
    const int stage_bytes = g.kc * (LW_BYTES + BN * 128), kstep = g.kc * 64;
    LinCtrl *S = reinterpret_cast<LinCtrl *>(buf + (size_t)g.stages * stage_bytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
    const int nt = tile / g.mtiles, mt = tile - nt * g.mtiles;
    const int cols_tile = g.gated ? LBM / 2 : LBM;
    // this CTA's K stages, and those of one accumulator
    const int total = (g.K + kstep - 1) / kstep;
    const int k0 = (int)((int64_t)total * rank / g.split), k1 = (int)((int64_t)total * (rank + 1) / g.split);
    const int part = g.promote ? kPromote / kstep : total;

    if (threadIdx.x == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&S->full[s], 1);
            mbar_init(&S->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&S->accf[a], 1);
            mbar_init(&S->acce[a], 4);
        }
        mbar_init(&S->fin, 1);
        mbar_init(&S->never, 1);
        fence_mbar_init();
        tma_prefetch_desc(&maps.w);
        if (g.gated) tma_prefetch_desc(&maps.w_up);
        tma_prefetch_desc(&maps.x);
    }
    if (warp == 5) tmem_alloc(&S->tmem_base, 2 * ACC);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S->tmem_base;
    pdl_wait();
    pdl_trigger();

    float sum[BN];  // warps 0-3: lane (of the tile's 128 w rows) x BN rows of x
#pragma unroll
    for (int j = 0; j < BN; ++j) sum[j] = 0.0f;
    if (warp < 4) {
        for (int i = k0, n = 0; i < k1; i += part, ++n) {
            if (!mbar_wait(&S->accf[n & 1], n / 2 & 1, g.wait_ns)) {
                lin_record(g.status);
                break;
            }
            __syncwarp();
            tc_fence_after();
            const uint32_t tb = tmem + (static_cast<uint32_t>(warp * 32) << 16) + (n & 1) * ACC;
#pragma unroll
            for (int c = 0; c < BN; c += 16) {
                uint32_t r[16];
                tmem_ld16_sync(tb + c, r);
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(r[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S->acce[n & 1]);
        }
    } else if (warp == 4) {
        if (lane == 0) {
            int i = 0;
            for (; i < k1 - k0; ++i) {
                const int s = i % g.stages;
                if (!mbar_wait(&S->empty[s], (i / g.stages & 1) ^ 1, g.wait_ns)) {
                    lin_record(g.status);
                    break;
                }
                uint64_t *bar = &S->full[s];
                uint8_t *d = buf + (size_t)s * stage_bytes, *dx = d + g.kc * LW_BYTES;
                const int k = k0 + i;
                mbar_arrive_expect_tx(bar, stage_bytes);
                if (g.chunked) {
                    if (!g.gated) {
                        tma_load_3d(d, &maps.w, bar, 0, nt * LBM, k * g.kc);
                    } else {
                        for (int c = 0; c < g.kc; ++c) {
                            tma_load_3d(d + c * LW_BYTES, &maps.w, bar, 0, nt * (LBM / 2), k * g.kc + c);
                            tma_load_3d(d + c * LW_BYTES + LW_BYTES / 2, &maps.w_up, bar, 0, nt * (LBM / 2),
                                        k * g.kc + c);
                        }
                    }
                    tma_load_3d(dx, &maps.x, bar, 0, mt * BN, k * g.kc);
                } else {
                    for (int c = 0; c < g.kc; ++c) {
                        const int x = k * kstep + c * 64;
                        tma_load_2d(d + c * LW_BYTES, &maps.w, bar, x, nt * cols_tile);
                        if (g.gated)
                            tma_load_2d(d + c * LW_BYTES + LW_BYTES / 2, &maps.w_up, bar, x, nt * cols_tile);
                        tma_load_2d(dx + c * BN * 128, &maps.x, bar, x, mt * BN);
                    }
                }
            }
            // never go on with TMA copies still landing in shared memory
            for (int j = max(0, i - g.stages); j < i; ++j)
                if (!mbar_wait(&S->full[j % g.stages], j / g.stages & 1)) lin_record(g.status);
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            constexpr uint32_t IDESC = idesc_bf16_f32(LBM, BN);
            bool ok = !(g.stall_test && !mbar_wait(&S->never, 0, g.wait_ns));
            for (int i = 0; ok && i < k1 - k0; ++i) {
                const int s = i % g.stages, n = i / part, in = i % part;
                if ((in == 0 && !mbar_wait(&S->acce[n & 1], (n / 2 & 1) ^ 1, g.wait_ns)) ||
                    !mbar_wait(&S->full[s], i / g.stages & 1, g.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t w0 = smem_u32(buf + (size_t)s * stage_bytes), x0 = w0 + g.kc * LW_BYTES;
                for (int c = 0; c < g.kc; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + (n & 1) * ACC, sw128_kmajor_desc(w0 + c * LW_BYTES + k * 32),
                                 sw128_kmajor_desc(x0 + c * BN * 128 + k * 32), IDESC, (in | c | k) != 0);
                mma_commit(&S->empty[s]);
                if (in == part - 1 || i == k1 - k0 - 1) mma_commit(&S->accf[n & 1]);
            }
            if (!ok) lin_record(g.status);
            mma_commit(&S->fin);
            if (!mbar_wait(&S->fin, 0)) lin_record(g.status);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();  // the stages' shared memory is free
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * ACC);
    }

    // the fp32 tile, [BN rows of x][128 rows of w], in the stages' place
    float *tile_f = reinterpret_cast<float *>(buf);
    if (warp < 4) {
#pragma unroll
        for (int j = 0; j < BN; ++j) tile_f[j * LBM + threadIdx.x] = sum[j];
    }
    if (g.split > 1) {
        lin_cluster_arrive();
        lin_cluster_wait();
    } else {
        __syncthreads();
    }

    // four columns a lane; a warp takes one row of 128 columns, or two of 64
    if (g.gated)
        finish_rows<BN, true>(g, tile_f, nt, mt, rank);
    else
        finish_rows<BN, false>(g, tile_f, nt, mt, rank);
    if (g.split > 1) {  // leave only when no CTA reads this one's partials any more
        lin_cluster_arrive();
        lin_cluster_wait();
    }
}

// The kernel's limits on the current device: its shared memory limit is raised, and how
// many clusters of s CTAs of half an SM's shared memory are resident (index s).
template <int BN>
cudaError_t linear_ready(int (&resident)[9])
{
    static std::mutex mu;
    static uint64_t done = 0;
    static int known[64][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (!(done >> dev & 1ull)) {
        e = cudaFuncSetAttribute(linear_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        for (int s = 1; e == cudaSuccess && s <= 8; ++s) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = s;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(s);
            cfg.blockDim = dim3(LTHREADS);
            cfg.dynamicSmemBytes = L_HALF_SM;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&known[dev][s], linear_kernel<BN>, &cfg);
        }
        if (e != cudaSuccess) return e;
        done |= 1ull << dev;
    }
    for (int s = 1; s <= 8; ++s) resident[s] = known[dev][s];
    return cudaSuccess;
}

// Tensor map of a bf16 matrix [rows, cols] with rows ld apart: boxes of box_rows rows x
// `chunks` chunks of 64 columns (cols a multiple of 64), else of 64 columns; what lies outside
// reads as zero.
bool encode_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows,
                 uint32_t chunks)
{
    if (rows == 1) ld = (cols + 7) / 8 * 8;
    if (cols % 64 == 0) {
        const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)cols / 64}, strides[2] = {(uint64_t)ld * 2, 128};
        const uint32_t box[3] = {64, box_rows, chunks};
        return encode_sw128_bf16(m, base, 3, dims, strides, box);
    }
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64, box_rows};
    return encode_sw128_bf16(m, base, 2, dims, strides, box);
}

bool encode_operands(LinMaps *maps, const moe_linear_t &d, const void *x, const void *w, const void *w_up,
                     uint32_t x_rows, uint32_t w_rows, uint32_t x_chunks, uint32_t w_chunks)
{
    return encode_rows(&maps->x, x, d.M, d.K, d.ldx, x_rows, x_chunks) &&
           encode_rows(&maps->w, w, d.N, d.K, d.ldw, w_rows, w_chunks) &&
           (!w_up || encode_rows(&maps->w_up, w_up, d.N, d.K, d.ldw, w_rows, w_chunks));
}

template <int BN>
cudaError_t launch_split(const moe_linear_t &d, const void *x, const void *w, const void *w_up, LinArgs g,
                         cudaStream_t st)
{
    int resident[9];
    cudaError_t e = linear_ready<BN>(resident);
    if (e != cudaSuccess) return e;
    g.kc = BN <= 64 ? 2 : 1;
    LinMaps maps{};
    // gated stages interleave the chunks of w and w_up, so their boxes hold one chunk
    if (!encode_operands(&maps, d, x, w, w_up, BN, g.gated ? LBM / 2 : LBM, g.kc, g.gated ? 1 : g.kc))
        return cudaErrorInvalidValue;
    const int stage = g.kc * (LW_BYTES + BN * 128), cols = g.gated ? LBM / 2 : LBM;
    g.mtiles = (g.M + BN - 1) / BN;
    const long long tiles = (long long)((g.N + cols - 1) / cols) * g.mtiles;
    const int total = (g.K + g.kc * 64 - 1) / (g.kc * 64);
    // as many CTAs as are resident at once, each with a K stage at least
    g.split = 1;
    for (int s = 2; s <= 8 && s <= total; ++s)
        if (tiles <= resident[s]) g.split = s;
    const int own = (total + g.split - 1) / g.split;
    const int room = g.split <= 2 && tiles * g.split <= num_sms() ? 227 * 1024 : L_HALF_SM;
    const int need = (BN * LBM * 4 + stage - 1) / stage;  // stages that hold the fp32 tile
    g.stages = (room - 1024 - (int)sizeof(LinCtrl)) / stage;
    if (g.stages > own) g.stages = own;
    if (g.stages > LSTAGES_MAX) g.stages = LSTAGES_MAX;
    if (g.stages < need) g.stages = need;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = g.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * g.split));
    cfg.blockDim = dim3(LTHREADS);
    cfg.dynamicSmemBytes = 1024 + (size_t)g.stages * stage + sizeof(LinCtrl);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = g.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<BN>, maps, g);
}

cudaError_t launch_pairs(const moe_linear_t &d, const void *x, const void *w, const void *w_up, const LinArgs &g,
                         int nb, cudaStream_t st)
{
    LinMaps maps{};
    if (!encode_operands(&maps, d, x, w, w_up, 128, nb / 2, 2, 2)) return cudaErrorInvalidValue;
    return launch_linear_pair(maps, g, g.gated, nb, st);
}

// The kernel and tile of a call.  Up to 128 rows the narrowest tile that holds them (4096 x 4096
// in us: 16 rows 10.7 on tiles of 16, 11.1 of 32, 13.9 of 128; 64 rows 12.6 of 64, 16.8 of 32, 15.1 of
// 128).  Above, CTA pairs once their 256 x 128 tiles occupy 64 SMs (4096 x 256 x 2048: 15.0 on 32 of
// them, 16.2 to 17.8 on linear_kernel's; 300 x 1000 x 1000, 16 tiles: 12.0 against 8.1).  A stage of a
// 256 x 256 tile takes half as long again as one of a 256 x 128 tile, and the tiles run in waves of
// all pairs: 512 x 4096 x 4096 22.4 on 64 tiles of 128, 30.6 on 32 of 256; 1024 rows 37.5 and 31.4.
cudaError_t launch_linear(const moe_linear_t &d, const void *x, const void *w, const void *w_up, const LinArgs &g,
                          cudaStream_t st)
{
    const int pairs = num_sms() / 2;
    auto tiles = [&](int nb) {
        const int cols = g.gated ? nb / 2 : nb;
        return ((d.M + 255ll) / 256) * (((long long)d.N + cols - 1) / cols);
    };
    if (d.M > 128 && tiles(128) >= 32) {
        const long long w128 = (tiles(128) + pairs - 1) / pairs, w256 = (tiles(256) + pairs - 1) / pairs;
        return launch_pairs(d, x, w, w_up, g, 3 * w256 <= 2 * w128 ? 256 : 128, st);
    }
    if (d.M <= 16) return launch_split<16>(d, x, w, w_up, g, st);
    if (d.M <= 32) return launch_split<32>(d, x, w, w_up, g, st);
    if (d.M <= 64) return launch_split<64>(d, x, w, w_up, g, st);
    return launch_split<128>(d, x, w, w_up, g, st);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_linear_workspace_size(void) { return 256; }

moe_status_t moe_linear(const moe_linear_t *d, const void *x, const void *w, const void *w_up, const float *bias,
                        const float *bias_up, const void *residual, void *out, void *ws, size_t ws_bytes, void *stream)
{
    if (!d || d->M < 0 || d->N <= 0 || d->K <= 0) return MOE_ERR_INVALID_ARG;
    if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SILU) return MOE_ERR_INVALID_ARG;
    if (d->out_dtype != MOE_OUT_BF16 && d->out_dtype != MOE_OUT_F32) return MOE_ERR_INVALID_ARG;
    if (d->M > 1 && (d->ldx < d->K || d->ldx % 8 || d->ldo < d->N || (residual && d->ldr < d->N)))
        return MOE_ERR_INVALID_ARG;
    if (d->N > 1 && (d->ldw < d->K || d->ldw % 8)) return MOE_ERR_INVALID_ARG;
    if (bias_up && !w_up) return MOE_ERR_INVALID_ARG;
    const int64_t far = (int64_t)1 << 38;  // a tensor map's stride is below 2^40 bytes
    if (d->ldx >= far || d->ldw >= far) return MOE_ERR_UNSUPPORTED;
    if (((int64_t)d->M + 15) / 16 * (((int64_t)d->N + 127) / 128) > INT32_MAX / 8) return MOE_ERR_UNSUPPORTED;
    if (d->M == 0) return MOE_OK;
    if (!x || !w || !out) return MOE_ERR_INVALID_ARG;
    auto off = [](const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
    const uintptr_t size = d->out_dtype == MOE_OUT_BF16 ? 2 : 4;
    if (off(x, 16) || off(w, 16) || off(w_up, 16) || off(bias, 4) || off(bias_up, 4) || off(residual, size) ||
        off(out, size))
        return MOE_ERR_INVALID_ARG;
    if (!ws || off(ws, 256) || ws_bytes < moe_linear_workspace_size()) return MOE_ERR_WORKSPACE;
    moe::LinArgs g{};
    g.M = d->M;
    g.N = d->N;
    g.K = d->K;
    g.act = d->act;
    g.out_f32 = d->out_dtype == MOE_OUT_F32;
    g.bias = bias;
    g.bias_up = bias_up;
    g.res = residual;
    g.out = out;
    g.ldr = d->M > 1 ? d->ldr : 0;
    g.ldo = d->M > 1 ? d->ldo : 0;
    // four columns of a row at once where every row of out (and residual) allows it
    g.vec = !off(out, 4 * size) && !off(residual, 4 * size) && g.ldo % 4 == 0 && (!residual || g.ldr % 4 == 0);
    g.chunked = d->K % 64 == 0;
    g.gated = w_up != nullptr;
    g.promote = g.out_f32 && d->K > moe::kPromote;
    g.status = static_cast<int32_t *>(ws);
    moe::wait_settings(&g.wait_ns, &g.stall_test);
    return moe::launch_linear(*d, x, w, w_up, g, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                 : MOE_ERR_CUDA;
}

}  // extern "C"
