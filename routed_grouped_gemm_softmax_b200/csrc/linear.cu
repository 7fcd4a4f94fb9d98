// linear.cu -- dense products with the layer's elementwise work in their epilogue:
//
//   out = act(x w^T + bias) [* (x w_up^T + bias_up)] [+ residual]
//
// x [M, K], w and w_up [N, K] bf16, products accumulated in fp32 on the tensor cores,
// bias in fp32, one rounding to the output's type at the end.
//
// linear_kernel: 128 rows of w on the MMA's M side and BN rows of x on its N side, so
// that the tensor work of a short batch follows its rows.  A tile's K range is split
// over the S CTAs of a cluster; each leaves its fp32 partial tile in its own shared
// memory, and every CTA then sums its share of the tile's rows over the S partials (in
// rank order, through distributed shared memory) and finishes them.
// Stages hold 128 columns of K: 256 contiguous bytes a row, which DRAM streams about a
// third faster than 128-byte row pieces.
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
constexpr int LTHREADS = 128;

struct LinCtrl {
    uint64_t full[LSTAGES_MAX];
    uint64_t empty[LSTAGES_MAX];
    uint64_t accf;   // every MMA of this CTA is done
    uint64_t never;  // nothing ever arrives here (timeout test)
    uint32_t tmem_base;
};

template <int BN, bool GATED>
constexpr int kLinStage = 2 * LW_BYTES * (GATED ? 2 : 1) + 2 * BN * 128;

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

template <int BN, bool GATED>
__global__ void __launch_bounds__(LTHREADS)
linear_kernel(const __grid_constant__ LinMaps maps, const LinArgs g)
{
    constexpr int NW = GATED ? 2 : 1;
    constexpr int STAGE = kLinStage<BN, GATED>;
    constexpr uint32_t TMEM_COLS = BN * NW < 32 ? 32 : BN * NW;
    extern __shared__ uint8_t lin_smem[];
    const uint32_t pad = (1024u - (smem_u32(lin_smem) & 1023u)) & 1023u;
    uint8_t *buf = lin_smem + pad;  // stages: w chunks, w_up chunks, x chunks
    LinCtrl *S = reinterpret_cast<LinCtrl *>(buf + (size_t)g.stages * STAGE);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
    const int nt = tile / g.mtiles, mt = tile - nt * g.mtiles;
    // this CTA's K stages
    const int total = (g.K + 127) / 128;
    const int k0 = (int)((int64_t)total * rank / g.split), k1 = (int)((int64_t)total * (rank + 1) / g.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&S->full[s], 1);
            mbar_init(&S->empty[s], 1);
        }
        mbar_init(&S->accf, 1);
        mbar_init(&S->never, 1);
        fence_mbar_init();
        tma_prefetch_desc(&maps.w);
        if (GATED) tma_prefetch_desc(&maps.w_up);
        tma_prefetch_desc(&maps.x);
    }
    if (warp == 1) tmem_alloc(&S->tmem_base, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S->tmem_base;
    pdl_wait();
    pdl_trigger();

    if (threadIdx.x == 0) {
        int i = 0;
        for (; i < k1 - k0; ++i) {
            const int s = i % g.stages;
            if (!mbar_wait(&S->empty[s], (i / g.stages & 1) ^ 1, g.wait_ns)) {
                lin_record(g.status);
                break;
            }
            uint64_t *bar = &S->full[s];
            uint8_t *d = buf + (size_t)s * STAGE;
            mbar_arrive_expect_tx(bar, STAGE);
            if (g.chunked) {
                const int z = (k0 + i) * 2;
                tma_load_3d(d, &maps.w, bar, 0, nt * LBM, z);
                if (GATED) tma_load_3d(d + 2 * LW_BYTES, &maps.w_up, bar, 0, nt * LBM, z);
                tma_load_3d(d + 2 * LW_BYTES * NW, &maps.x, bar, 0, mt * BN, z);
            } else {
                for (int c = 0; c < 2; ++c) {
                    const int k = (k0 + i) * 128 + c * 64;
                    tma_load_2d(d + c * LW_BYTES, &maps.w, bar, k, nt * LBM);
                    if (GATED) tma_load_2d(d + (2 + c) * LW_BYTES, &maps.w_up, bar, k, nt * LBM);
                    tma_load_2d(d + 2 * LW_BYTES * NW + c * BN * 128, &maps.x, bar, k, mt * BN);
                }
            }
        }
        // never go on with TMA copies still landing in shared memory
        for (int j = max(0, i - g.stages); j < i; ++j)
            if (!mbar_wait(&S->full[j % g.stages], j / g.stages & 1)) lin_record(g.status);
    } else if (threadIdx.x == 32) {
        constexpr uint32_t IDESC = idesc_bf16_f32(LBM, BN);
        bool ok = !(g.stall_test && !mbar_wait(&S->never, 0, g.wait_ns));
        for (int i = 0; ok && i < k1 - k0; ++i) {
            const int s = i % g.stages;
            if (!mbar_wait(&S->full[s], i / g.stages & 1, g.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t w0 = smem_u32(buf + (size_t)s * STAGE), x0 = w0 + 2 * LW_BYTES * NW;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t off = (k & 3) * 32;
                const uint64_t xd = sw128_kmajor_desc(x0 + (k >> 2) * BN * 128 + off);
                mma_bf16(tmem, sw128_kmajor_desc(w0 + (k >> 2) * LW_BYTES + off), xd, IDESC, (i | k) != 0);
                if (GATED)
                    mma_bf16(tmem + BN, sw128_kmajor_desc(w0 + (2 + (k >> 2)) * LW_BYTES + off), xd, IDESC,
                             (i | k) != 0);
            }
            mma_commit(&S->empty[s]);
        }
        if (!ok) lin_record(g.status);
        mma_commit(&S->accf);
    }
    __syncthreads();
    if (!mbar_wait(&S->accf, 0)) lin_record(g.status);
    tc_fence_after();

    // the fp32 tile, [BN rows of x][128 rows of w], in the stages' place
    float *part = reinterpret_cast<float *>(buf);
#pragma unroll 1
    for (int c = 0; c < BN * NW; c += 16) {
        uint32_t r[16];
        tmem_ld16_sync(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * LBM + threadIdx.x] = __uint_as_float(r[j]);
    }
    tc_fence_before();
    if (g.split > 1) {
        lin_cluster_arrive();
        lin_cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }

    // four columns a lane, a warp per row
    const int n = nt * LBM + lane * 4;
    const LinCols cols(g, n);
    const int rows = min(BN, g.M - mt * BN);
    const uint32_t p0 = smem_u32(part) + lane * 16;
    for (int t = rank + g.split * warp; t < rows; t += g.split * (LTHREADS / 32)) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), u = v;
        if (g.split == 1) {
            v = *reinterpret_cast<const float4 *>(part + t * LBM + lane * 4);
            if (GATED) u = *reinterpret_cast<const float4 *>(part + (BN + t) * LBM + lane * 4);
        } else {
            for (int q = 0; q < g.split; ++q) {
                const float4 a = ld_cluster4(p0 + t * LBM * 4, q);
                v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
                if (GATED) {
                    const float4 b = ld_cluster4(p0 + (BN + t) * LBM * 4, q);
                    u.x += b.x, u.y += b.y, u.z += b.z, u.w += b.w;
                }
            }
        }
        float o[4] = {v.x, v.y, v.z, v.w};
        const float up[4] = {u.x, u.y, u.z, u.w};
        lin_finish4<GATED>(g, cols, (int64_t)mt * BN + t, o, up);
    }
    if (g.split > 1) {  // leave only when no CTA reads this one's partials any more
        lin_cluster_arrive();
        lin_cluster_wait();
    }
}

template <int BN, bool GATED>
cudaError_t launch_linear(const LinMaps &maps, LinArgs g, cudaStream_t st)
{
    constexpr int STAGE = kLinStage<BN, GATED>;
    static std::mutex mu;
    static uint64_t done = 0;  // per device: the kernel's shared memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!(done >> dev & 1ull)) {
            e = cudaFuncSetAttribute(linear_kernel<BN, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
            if (e != cudaSuccess) return e;
            done |= 1ull << dev;
        }
    }
    const long long tiles = (long long)((g.N + LBM - 1) / LBM) * g.mtiles;
    const int total = (g.K + 127) / 128, own = (total + g.split - 1) / g.split;
    g.stages = (227 * 1024 - 1024 - (int)sizeof(LinCtrl)) / STAGE;
    if (g.stages > own) g.stages = own;
    if (g.stages > LSTAGES_MAX) g.stages = LSTAGES_MAX;
    const int part = (BN * LBM * 4 * (GATED ? 2 : 1) + STAGE - 1) / STAGE;  // stages that hold the fp32 tile
    if (g.stages < part) g.stages = part;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = g.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * g.split));
    cfg.blockDim = dim3(LTHREADS);
    cfg.dynamicSmemBytes = 1024 + (size_t)g.stages * STAGE + sizeof(LinCtrl);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = g.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<BN, GATED>, maps, g);
}

// Tensor map of a bf16 matrix [rows, cols] with rows ld apart: boxes of box_rows rows x
// 128 columns as two 64-column chunks (cols a multiple of 64), else of 64 columns;
// what lies outside reads as zero.
bool encode_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows)
{
    if (rows == 1) ld = (cols + 7) / 8 * 8;
    if (cols % 64 == 0) {
        const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)cols / 64}, strides[2] = {(uint64_t)ld * 2, 128};
        const uint32_t box[3] = {64, box_rows, 2};
        return encode_sw128_bf16(m, base, 3, dims, strides, box);
    }
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64, box_rows};
    return encode_sw128_bf16(m, base, 2, dims, strides, box);
}

template <int BN>
cudaError_t launch_tile(const moe_linear_t &d, const void *x, const void *w, const void *w_up, LinArgs g,
                        cudaStream_t st)
{
    LinMaps maps{};
    if (!encode_rows(&maps.w, w, d.N, d.K, d.ldw, LBM) || (w_up && !encode_rows(&maps.w_up, w_up, d.N, d.K, d.ldw, LBM)) ||
        !encode_rows(&maps.x, x, d.M, d.K, d.ldx, BN))
        return cudaErrorInvalidValue;
    g.mtiles = (d.M + BN - 1) / BN;
    const long long tiles = (long long)((d.N + LBM - 1) / LBM) * g.mtiles;
    const int total = (d.K + 127) / 128;
    g.split = 1;
    while (g.split < 8 && tiles * g.split * 2 <= num_sms() && g.split * 2 <= total) g.split *= 2;
    return w_up ? launch_linear<BN, true>(maps, g, st) : launch_linear<BN, false>(maps, g, st);
}

cudaError_t launch_pairs(const moe_linear_t &d, const void *x, const void *w, const void *w_up, const LinArgs &g,
                         cudaStream_t st)
{
    LinMaps maps{};
    if (!encode_rows(&maps.w, w, d.N, d.K, d.ldw, 128) || (w_up && !encode_rows(&maps.w_up, w_up, d.N, d.K, d.ldw, 128)) ||
        !encode_rows(&maps.x, x, d.M, d.K, d.ldx, 128))
        return cudaErrorInvalidValue;
    return launch_linear_pair(maps, g, w_up != nullptr, st);
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
    g.status = static_cast<int32_t *>(ws);
    moe::wait_settings(&g.wait_ns, &g.stall_test);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const long long pairs = (long long)((d->M + 255) / 256) * ((d->N + (w_up ? 127 : 255)) / (w_up ? 128 : 256));
    if (d->M > 128 && pairs * 2 >= moe::num_sms() && (!g.out_f32 || d->K <= 512))
        e = moe::launch_pairs(*d, x, w, w_up, g, st);
    else if (d->M <= 16)
        e = moe::launch_tile<16>(*d, x, w, w_up, g, st);
    else if (d->M <= 32)
        e = moe::launch_tile<32>(*d, x, w, w_up, g, st);
    else if (d->M <= 64)
        e = moe::launch_tile<64>(*d, x, w, w_up, g, st);
    else
        e = moe::launch_tile<128>(*d, x, w, w_up, g, st);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
