// linear.cu -- dense products with the layer's elementwise work in their epilogue:
//
//   out = act(x w^T + bias) [* (x w_up^T + bias_up)] [+ residual]
//
// x [M, K], w and w_up [N, K] bf16, products accumulated in fp32 on the tensor cores,
// bias in fp32, one rounding to the output's type at the end.
//
// linear_kernel: 128 rows of w (gated: 64 of w over 64 of w_up) on the MMA's M side and BN
// rows of x on its N side, so that the tensor work of a short batch follows its rows.  A
// tile's K range is split over the S CTAs of a cluster; each copies to every CTA the rows of
// its fp32 partial tile that this one finishes, which sums them in rank order.
// Bound by latency, not by the weight stream, while that is short: of the 3.6 us of
// 1 x 2048 x 2048 (1.3 at the memory's rate) 0.5 are the first load, 0.5 to 1 the tensor core's
// results, 1 the exchange and the epilogue, the rest the launch.  16 x 4096 x 4096 8.9 us (5.2).
// linear_pair.cu takes the batches with enough rows to be bound by the tensor cores.
#include <mutex>

#include "linear.cuh"
#include "moe_internal.h"
#include "pair_ptx.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int LBM = 128;             // w rows per tile
constexpr int LSTAGES_MAX = 8;
constexpr int LW_BYTES = LBM * 128;  // one 64-column chunk of 128 w rows
constexpr int LTHREADS = 192;        // warps 0-3: accumulators; 4: TMA; 5: MMA; all: epilogue
constexpr int L_SMEM = 227 * 1024;   // a CTA's shared memory at most

constexpr int LKC = 2;  // 64-column chunks of a stage: 256 contiguous bytes a row

// A CTA may wait in tcgen05.alloc for what others hold, while those wait for their clusters: no such
// ring closes as long as all that fit an SM at once have their columns. Registers admit 7 CTAs
// of 64 columns (48 registers a thread, tiles of 16), 5 of 64 or 3 of 128 (102), below 512 in all.  The
// kernels of 256 or 512 columns leave no shared memory for a CTA of this one beside them, but for the MX
// GEMM, whose CTAs wait for no other block.

// Rows of a tile that each of `split` CTAs finishes.
__host__ __device__ __forceinline__ int lin_own(int bn, int split) { return (bn + split - 1) / split; }
// Floats of a CTA's buffer for the cluster's partials of its rows.
__host__ __device__ __forceinline__ int lin_recv(int bn, int split)
{
    return split > 1 ? split * lin_own(bn, split) * LBM : 0;
}

struct LinCtrl {
    uint64_t full[LSTAGES_MAX];
    uint64_t empty[LSTAGES_MAX];
    uint64_t accf[2];  // accumulator a holds a finished part
    uint64_t acce[2];  // its four warps have read it
    uint64_t fin;      // every MMA of this CTA is done
    uint64_t red;      // the other CTAs' partials of this one's rows are here
    uint64_t never;    // nothing ever arrives here (timeout test)
    uint32_t tmem_base;
};

// Relaxed: neither use publishes data (barriers are initialised behind a fence of their own),
// and a release at cluster scope waits for the thread's earlier memory operations.
__device__ __forceinline__ void lin_cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void lin_cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Copies bytes (a multiple of 16) to the same shared-memory address as dst in CTA `rank` of the
// cluster, completing on its barrier.
__device__ __forceinline__ void push_cluster(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 d, b;\n\tmapa.shared::cluster.u32 d, %0, %4;\n\tmapa.shared::cluster.u32 b, %3, %4;\n\t"
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [d], [%1], %2, [b];\n\t}" ::"r"(
            smem_u32(dst)),
        "r"(smem_u32(src)), "r"(bytes), "r"(smem_u32(bar)), "r"(rank)
        : "memory");
}

// Finishes rows lo .. hi of the tile: four columns a lane, a warp takes one row of 128 columns
// or two of 64, U times over.  Each is the sum, in rank order, over the cluster's partials:
// `from` holds `stride` rows of each, from row lo on, once `red` completes.  A short
// batch's epilogue is one pass through this code, most of it latency: the residual and
// the biases are loaded before the wait, and U is no more than such a batch fills.
template <int BN, bool GATED>
__device__ __forceinline__ void finish_rows(const LinArgs &g, const float *from, int stride, uint64_t *red, int nt,
                                            int mt, int lo, int hi)
{
    constexpr int COLS = GATED ? LBM / 2 : LBM, LANES = COLS / 4, RW = 32 / LANES, U = BN / 16;
    constexpr int STEP = LTHREADS / 32 * RW;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, at = (lane % LANES) * 4;
    const LinCols cols(g, nt * COLS + at);
    const int64_t m0 = (int64_t)mt * BN;
    int t0 = lo + warp * RW + lane / LANES;
    float r[U][4];
    lin_residual<U, STEP>(g, cols, m0 + t0, hi - t0, r);
    if (g.split > 1) {
        if (!wait2(red, 0, g.wait_ns)) lin_record(g.status);
        __syncwarp();
        lin_cluster_arrive();  // this CTA has what it waits for
    }
#pragma unroll 1
    while (t0 < hi) {
        float v[U][4], u[U][4];
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = u[j][i] = 0.0f;
        const float *row[U];
#pragma unroll
        for (int j = 0; j < U; ++j) row[j] = from + (min(t0 + j * STEP, hi - 1) - lo) * LBM + at;
#pragma unroll 2
        for (int q = 0; q < g.split; ++q)
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const float *p = row[j] + q * stride * LBM;
                const float4 a = *reinterpret_cast<const float4 *>(p);
                v[j][0] += a.x, v[j][1] += a.y, v[j][2] += a.z, v[j][3] += a.w;
                if (GATED) {
                    const float4 b = *reinterpret_cast<const float4 *>(p + COLS);
                    u[j][0] += b.x, u[j][1] += b.y, u[j][2] += b.z, u[j][3] += b.w;
                }
            }
        lin_finish<GATED, U, STEP>(g, cols, m0 + t0, hi - t0, v, u, r);
        t0 += U * STEP;
        if (t0 < hi) lin_residual<U, STEP>(g, cols, m0 + t0, hi - t0, r);
    }
}

template <int BN>
__global__ void __launch_bounds__(LTHREADS)
linear_kernel(const __grid_constant__ LinMaps maps, const LinArgs g)
{
    constexpr uint32_t ACC = BN < 32 ? 32 : BN;  // TMEM columns of an accumulator
    constexpr int KC = LKC, STAGE = KC * (LW_BYTES + BN * 128), KSTEP = KC * 64;
    extern __shared__ uint8_t lin_smem[];
    const uint32_t pad = (1024u - (smem_u32(lin_smem) & 1023u)) & 1023u;
    uint8_t *buf = lin_smem + pad;  // stages: w chunks, x chunks
    float *recv = reinterpret_cast<float *>(buf + (size_t)g.stages * STAGE);  // every CTA's partials of this one's rows
    LinCtrl *S = reinterpret_cast<LinCtrl *>(recv + lin_recv(BN, g.split));
    const int warp = uniform_warp(), lane = threadIdx.x % 32;
    const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
    const int nt = tile / g.mtiles, mt = tile - nt * g.mtiles;
    const int cols_tile = g.gated ? LBM / 2 : LBM;
    // this CTA's K stages, and those of one accumulator
    const int total = (g.K + KSTEP - 1) / KSTEP;
    const int k0 = (int)((int64_t)total * rank / g.split), k1 = (int)((int64_t)total * (rank + 1) / g.split);
    const int part = g.promote ? kPromote / KSTEP : total;
    // CTA q finishes the rows q * own .. of the tile
    const int rows = min(BN, g.M - mt * BN), own = lin_own(BN, g.split);
    const int lo = min(rows, rank * own), hi = min(rows, lo + own);

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
        mbar_init(&S->red, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&S->red, g.split > 1 ? g.split * (hi - lo) * LBM * 4 : 0);
        tma_prefetch_desc(&maps.w);
        if (g.gated) tma_prefetch_desc(&maps.w_up);
        tma_prefetch_desc(&maps.x);
    }
    if (warp == 5) tmem_alloc(&S->tmem_base, 2 * ACC);
    tc_fence_before();
    __syncthreads();
    if (g.split > 1) {  // every CTA's barriers exist before a copy may complete on them
        lin_cluster_arrive();
        lin_cluster_wait();
    }
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, S->tmem_base, 0);
    pdl_wait();
    pdl_trigger();

    float *tile_f = reinterpret_cast<float *>(buf);  // the fp32 tile, [BN rows of x][128 rows of w], in the stages' place
    if (warp < 4) {
        float sum[BN];  // lane (of the tile's 128 w rows) x BN rows of x
#pragma unroll
        for (int j = 0; j < BN; ++j) sum[j] = 0.0f;
        bool ok = true;
        for (int i = k0, n = 0; i < k1; i += part, ++n) {
            if (!mbar_wait(&S->accf[n & 1], n / 2 & 1, g.wait_ns)) {
                lin_record(g.status);
                ok = false;
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
        if (ok) {  // every stage was read by an MMA that has completed: its place is free
#pragma unroll
            for (int j = 0; j < BN; ++j) tile_f[j * LBM + threadIdx.x] = sum[j];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    } else if (warp == 4) {
        int s = 0, loaded = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int k = k0; k < k1; ++k, ++loaded) {
            if (!warp_wait(&S->empty[s], ph, g.wait_ns)) {
                ok = false;
                break;
            }
            uint64_t *bar = &S->full[s];
            uint8_t *d = buf + s * STAGE, *dx = d + KC * LW_BYTES;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, STAGE);
                if (g.chunked) {
                    if (!g.gated) {
                        tma_load_3d(d, &maps.w, bar, 0, nt * LBM, k * KC);
                    } else {
#pragma unroll
                        for (int c = 0; c < KC; ++c) {
                            tma_load_3d(d + c * LW_BYTES, &maps.w, bar, 0, nt * (LBM / 2), k * KC + c);
                            tma_load_3d(d + c * LW_BYTES + LW_BYTES / 2, &maps.w_up, bar, 0, nt * (LBM / 2), k * KC + c);
                        }
                    }
                    tma_load_3d(dx, &maps.x, bar, 0, mt * BN, k * KC);
                } else {
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const int x = k * KSTEP + c * 64;
                        tma_load_2d(d + c * LW_BYTES, &maps.w, bar, x, nt * cols_tile);
                        if (g.gated) tma_load_2d(d + c * LW_BYTES + LW_BYTES / 2, &maps.w_up, bar, x, nt * cols_tile);
                        tma_load_2d(dx + c * BN * 128, &maps.x, bar, x, mt * BN);
                    }
                }
            }
            __syncwarp();
            if (++s == g.stages) {
                s = 0;
                ph ^= 1;
            }
        }
        if (lane == 0) {
            if (!ok) lin_record(g.status);
            // never go on with TMA copies still landing in shared memory
            for (int j = max(0, loaded - g.stages); j < loaded; ++j)
                if (!mbar_wait(&S->full[j % g.stages], j / g.stages & 1)) lin_record(g.status);
        }
        __syncwarp();
    } else {
        constexpr uint32_t IDESC = idesc_bf16_f32(LBM, BN);
        const uint32_t buf0 = smem_u32(buf);
        bool ok = !(g.stall_test && !warp_wait(&S->never, 0, g.wait_ns));
        int s = 0, in = 0, n = 0;  // stage, K stage of the accumulator, accumulators begun
        uint32_t ph = 0;
        for (int k = k0; ok && k < k1; ++k) {
            if ((in == 0 && !warp_wait(&S->acce[n & 1], (n / 2 & 1) ^ 1, g.wait_ns)) ||
                !warp_wait(&S->full[s], ph, g.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t w0 = buf0 + s * STAGE, x0 = w0 + KC * LW_BYTES, acc = tmem + (n & 1) * ACC;
            const bool last = in + 1 == part || k == k1 - 1;
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16(acc, sw128_kmajor_desc(w0 + c * LW_BYTES + j * 32),
                                 sw128_kmajor_desc(x0 + c * BN * 128 + j * 32), IDESC, (in | c | j) != 0);
                mma_commit(&S->empty[s]);
                if (last) mma_commit(&S->accf[n & 1]);
            }
            __syncwarp();
            if (++s == g.stages) {
                s = 0;
                ph ^= 1;
            }
            ++in;
            if (last) {
                in = 0;
                ++n;
            }
        }
        if (elect_one()) mma_commit(&S->fin);
        __syncwarp();
        if (!warp_wait(&S->fin, 0)) ok = false;
        if (!ok && lane == 0) lin_record(g.status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * ACC);
    }
    if (threadIdx.x < g.split && g.split > 1) {  // thread q: CTA q's rows of this partial tile
        const int q = threadIdx.x, qlo = min(rows, q * own), n = min(rows, qlo + own) - qlo;
        if (n > 0) push_cluster(recv + rank * own * LBM, tile_f + qlo * LBM, n * LBM * 4, &S->red, q);
    }
    __syncwarp();
    const float *from = g.split > 1 ? recv : tile_f;
    if (g.gated)
        finish_rows<BN, true>(g, from, own, &S->red, nt, mt, lo, hi);
    else
        finish_rows<BN, false>(g, from, own, &S->red, nt, mt, lo, hi);
    if (g.split > 1) lin_cluster_wait();  // leave only when no CTA reads this one's tile any more
}

// The kernel's limits on the current device: its shared memory limit is raised, and how
// many clusters of s CTAs, one an SM, are resident (index s).
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
        e = cudaFuncSetAttribute(linear_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, L_SMEM);
        for (int s = 1; e == cudaSuccess && s <= 8; ++s) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = s;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(s);
            cfg.blockDim = dim3(LTHREADS);
            cfg.dynamicSmemBytes = L_SMEM;
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
    constexpr int KC = LKC, stage = KC * (LW_BYTES + BN * 128);
    LinMaps maps{};
    // gated stages interleave the chunks of w and w_up, so their boxes hold one chunk
    if (!encode_operands(&maps, d, x, w, w_up, BN, g.gated ? LBM / 2 : LBM, KC, g.gated ? 1 : KC))
        return cudaErrorInvalidValue;
    const int cols = g.gated ? LBM / 2 : LBM;
    g.mtiles = (g.M + BN - 1) / BN;
    const long long tiles = (long long)((g.N + cols - 1) / cols) * g.mtiles;
    const int total = (g.K + KC * 64 - 1) / (KC * 64);
    // as many CTAs as are resident at once, each with a K stage at least
    g.split = 1;
    for (int s = 2; s <= 8 && s <= total; ++s)
        if (tiles <= resident[s]) g.split = s;
    const int own = (total + g.split - 1) / g.split;
    const int recv = lin_recv(BN, g.split) * 4;
    const int need = (BN * LBM * 4 + stage - 1) / stage;  // stages that hold the fp32 tile
    g.stages = (L_SMEM - 1024 - (int)sizeof(LinCtrl) - recv) / stage;
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
    cfg.dynamicSmemBytes = 1024 + (size_t)g.stages * stage + recv + sizeof(LinCtrl);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = g.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<BN>, maps, g);
}

cudaError_t launch_pairs(const moe_linear_t &d, const void *x, const void *w, const void *w_up, LinArgs g, int nb,
                         cudaStream_t st)
{
    LinMaps maps{};
    if (!encode_operands(&maps, d, x, w, w_up, 128, nb / 2, 2, 2)) return cudaErrorInvalidValue;
    const int size = g.out_f32 ? 4 : 2;
    auto mapped = [&](const void *p, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && ld < (int64_t)1 << 37;
    };
    g.maps_out = mapped(g.out, g.ldo) && (!g.res || mapped(g.res, g.ldr));
    if (g.maps_out && (!encode_rows_32(&maps.out, g.out, g.out_f32, d.M, d.N, g.ldo) ||
                       (g.res && !encode_rows_32(&maps.res, g.res, g.out_f32, d.M, d.N, g.ldr))))
        return cudaErrorInvalidValue;
    return launch_linear_pair(maps, g, g.gated, nb, st);
}

// The kernel and tile of a call.  The narrowest tile that holds the rows, of 16, 32 or 64 (x 4096 x
// 4096, us: 16 rows 8.9 on tiles of 16, 8.9 of 32, 9.3 of 64; 64 rows 14.3, 10.3, 10.1).  Above 128
// rows CTA pairs once their 256 x 128 tiles occupy 64 SMs (600 x 2048 x 512, 48 tiles: 6.4 on
// them, 10.4 on linear_kernel's; 512 x 2048 x 2048, 32 tiles: 10.8 and 10.5; 300 x 1000 x 1000, 16
// tiles: 9.2 and 6.2).  A stage of a 256 x 256 tile takes half as long again as one of a 256 x
// 128 tile, and the tiles run in waves of all pairs: 512 x 4096 x 4096 17.8 on 64 tiles of 128, 25.7
// on 32 of 256; 1024 rows 30.0 and 27.4; 1500 x 4104 x 1408, 3 waves and 2, 18.1 and 20.5.  The rule
// counts stages alone.  Where rows of out are not 16-byte aligned the epilogue is the longer part, and
// the two are close: gelu with residual, 128 and 256 columns, 1001 x 4099 x 1416 25.4 and 26.4, 2001 rows
// 45.9 and 46.5, 1024 x 4098 x 512 17.5 and 18.1.
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
        return launch_pairs(d, x, w, w_up, g, !g.promote && 3 * w256 < 2 * w128 ? 256 : 128, st);
    }
    if (d.M <= 16) return launch_split<16>(d, x, w, w_up, g, st);
    if (d.M <= 32) return launch_split<32>(d, x, w, w_up, g, st);
    return launch_split<64>(d, x, w, w_up, g, st);
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
    // sizes are rounded up to whole tiles (of up to 256 rows, 128 of K) in 32 bits
    const int32_t most = INT32_MAX - 255;
    if (d->M > most || d->N > most || d->K > most) return MOE_ERR_UNSUPPORTED;
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
