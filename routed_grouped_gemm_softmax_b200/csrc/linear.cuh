// linear.cuh -- arguments and epilogue arithmetic of the dense products (linear.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "../../include/moe.h"

namespace moe {

struct LinMaps {
    CUtensorMap w, w_up, x;
};

struct LinArgs {
    int M, N, K;
    int act;
    bool out_f32, vec, chunked;
    const float *bias, *bias_up;  // or null
    const void *res;              // or null; the output's type
    void *out;
    int64_t ldr, ldo;
    int32_t *status;
    uint64_t wait_ns;
    int stall_test;
    bool promote;  // see kPromote
    // linear_kernel: tiles of x rows, CTAs of a cluster, stages and their 64-column chunks
    bool gated;
    int mtiles, split, stages, kc;
};

// The tensor cores truncate as they accumulate, an error that grows with the depth of the
// sum: against 64 bits an fp32 result was off by a relative 7e-7 after 1024 columns of K
// (standard normal operands), where an fp32 chain of rounded sums is at 3e-7.  For fp32 outputs the
// accumulators are therefore added up outside, with rounding, after every kPromote
// columns; a bf16 output's own rounding is a thousand times that error.
constexpr int kPromote = 512;

// linear_pair.cu: 256 x nb tiles (nb 128 or 256) on CTA pairs; maps with boxes of 128 x
// rows and nb / 2 w rows, two chunks each.
cudaError_t launch_linear_pair(const LinMaps &maps, const LinArgs &g, bool gated, int nb, cudaStream_t st);

__device__ __forceinline__ void lin_record(int32_t *status) { atomicCAS(status, 0, MOE_ERR_TIMEOUT); }

// act(v).  The forms keep their relative accuracy where v is far below zero: gelu by
// erfc, and its tanh form as v * sigmoid(2 u), since (1 + tanh u) / 2 = sigmoid(2 u).
template <int ACT>
__device__ __forceinline__ float lin_act(float v)
{
    if (ACT == MOE_ACT_RELU) return v < 0.0f ? 0.0f : v;  // a NaN stays
    if (ACT == MOE_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
    if (ACT == MOE_ACT_GELU_TANH) {
        const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);  // sqrt(2 / pi) (...)
        return v / (1.0f + expf(-2.0f * u));
    }
    if (ACT == MOE_ACT_SILU) return v / (1.0f + expf(-v));
    return v;
}

// act of n values; the activation is the same for the whole launch, so the branch is uniform.
template <int N>
__device__ __forceinline__ void lin_act_n(int act, float (&v)[N])
{
    switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lin_act<MOE_ACT_RELU>(v[i]);
        break;
    case MOE_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lin_act<MOE_ACT_GELU>(v[i]);
        break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lin_act<MOE_ACT_GELU_TANH>(v[i]);
        break;
    case MOE_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lin_act<MOE_ACT_SILU>(v[i]);
        break;
    default: break;
    }
}

// The four output columns n .. n+3 of a thread: which exist, and their biases.
struct LinCols {
    int n, count;  // columns inside N
    float b[4], bu[4];
    __device__ __forceinline__ LinCols(const LinArgs &g, int n0) : n(n0), count(min(4, g.N - n0))
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = g.bias && i < count ? g.bias[n + i] : 0.0f;
            bu[i] = g.bias_up && i < count ? g.bias_up[n + i] : 0.0f;
        }
    }
};

// Finishes and stores the four columns of row m: v the products with w, u those with w_up.
template <bool GATED>
__device__ __forceinline__ void lin_finish4(const LinArgs &g, const LinCols &c, int64_t m, float (&v)[4],
                                            const float (&u)[4])
{
    if (c.count <= 0) return;
    const int64_t ro = m * g.ldr + c.n, oo = m * g.ldo + c.n;
    const bool vec = g.vec && c.count == 4;
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    if (g.res) {
        if (g.out_f32) {
            const float *p = static_cast<const float *>(g.res) + ro;
            if (vec) {
                const float4 q = *reinterpret_cast<const float4 *>(p);
                r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < c.count) r[i] = p[i];
            }
        } else {
            const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(g.res) + ro;
            if (vec) {
                const uint2 q = *reinterpret_cast<const uint2 *>(p);
                const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&q.x));
                const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&q.y));
                r[0] = a.x, r[1] = a.y, r[2] = b.x, r[3] = b.y;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < c.count) r[i] = __bfloat162float(p[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += c.b[i];
    lin_act_n(g.act, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (GATED) v[i] *= u[i] + c.bu[i];
        if (g.res) v[i] += r[i];
    }
    if (g.out_f32) {
        float *p = static_cast<float *>(g.out) + oo;
        if (vec) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < c.count) p[i] = v[i];
        }
    } else {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(g.out) + oo;
        if (vec) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2 *>(p) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < c.count) p[i] = __float2bfloat16_rn(v[i]);
        }
    }
}

}  // namespace moe
