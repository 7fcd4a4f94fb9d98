// combine.cu -- the gate-weighted combine as its own kernel, for batches whose
// combine would lengthen the down GEMM's epilogue more than it saves: a CTA per
// token, eight columns per thread, the arithmetic of combine.cuh.
#include "combine.cuh"
#include "moe_internal.h"
#include "pdl.cuh"

namespace moe {
namespace {

// A CTA per token; thread c covers columns 8c .. 8c+7 (and c + 256, ...).
__global__ void __launch_bounds__(256) combine_kernel(const __nv_bfloat16 *__restrict__ y,
                                                      const float *__restrict__ gate, int T, int H, int k,
                                                      __nv_bfloat16 *__restrict__ out, int sh_count, int sh_rows0)
{
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    for (int c0 = 0; c0 < H; c0 += 256 * 8)
        combine_cols<false>(y, gate, out, t, k, H, c0 + threadIdx.x * 8, sh_count, T, sh_rows0);
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(q[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// out[t] = bf16(sum of w[t,j] y[t*k + j] over the slots j with an expert), fp32 fma in
// ascending j.  A slot without an expert has no y row: its memory is not read.  Bound by the
// rows' latency where they are loaded one by one (2048 tokens, k 6, H 2048: 18.4 us, 88 MB).
// PARTS: a row's second part lies `parts` rows further on.
template <typename TY, bool PARTS>
__global__ void __launch_bounds__(256) combine_given_kernel(const TY *y, int parts, const int32_t *idx, const float *w, int H, int E,
                                                            int k, __nv_bfloat16 *out)
{
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const size_t t = blockIdx.x;
    for (int c = threadIdx.x * 8; c < H; c += 256 * 8) {
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < k; j0 += U) {  // U rows are under way at once
            float v[U][8], v2[U][8], g[U];
            bool any[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                any[j] = j0 + j < k && (unsigned)idx[t * k + min(j0 + j, k - 1)] < (unsigned)E;
                g[j] = any[j] ? w[t * k + j0 + j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (any[j]) {
                    load8(y + (t * k + j0 + j) * H + c, v[j]);
                    if constexpr (PARTS) load8(y + (t * k + j0 + j + parts) * H + c, v2[j]);
                }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (any[j])
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[j], PARTS ? v[j][i] + v2[j][i] : v[j][i], acc[i]);
        }
        uint4 o;
        __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
        *reinterpret_cast<uint4 *>(out + t * H + c) = o;
    }
}

}  // namespace

cudaError_t launch_combine_given(const void *y, bool y_f32, int parts, const int32_t *idx, const float *w, int T, int H, int E,
                                 int top_k, __nv_bfloat16 *out, cudaStream_t st)
{
    const dim3 grid(T), block(256);
    const auto *yf = static_cast<const float *>(y);
    if (!y_f32)
        return launch_pdl(combine_given_kernel<__nv_bfloat16, false>, grid, block, 0, st,
                          static_cast<const __nv_bfloat16 *>(y), 0, idx, w, H, E, top_k, out);
    return parts ? launch_pdl(combine_given_kernel<float, true>, grid, block, 0, st, yf, parts, idx, w, H, E, top_k, out)
                 : launch_pdl(combine_given_kernel<float, false>, grid, block, 0, st, yf, 0, idx, w, H, E, top_k, out);
}

cudaError_t launch_combine(const __nv_bfloat16 *y, const float *gate, int T, int H, int top_k,
                           __nv_bfloat16 *out, cudaStream_t st, int sh_count, int sh_rows0)
{
    return launch_pdl(combine_kernel, dim3(T), dim3(256), 0, st, y, gate, T, H, top_k, out, sh_count, sh_rows0);
}

}  // namespace moe
