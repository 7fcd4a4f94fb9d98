// linear.cuh -- arguments and epilogue arithmetic of the dense products (linear.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "../../include/moe.h"

namespace moe {

struct LinMaps {
    CUtensorMap w, w_up, x;
    CUtensorMap out, res;  // linear_pair.cu with LinArgs::maps_out: 32 x 32 boxes
};

struct LinArgs {
    int M, N, K;
    int act;
    bool out_f32, vec, chunked;
    bool maps_out;  // out (and the residual) have tensor maps
    const float *bias, *bias_up;  // or null
    const void *res;              // or null; the output's type
    void *out;
    int64_t ldr, ldo;
    int32_t *status;
    uint64_t wait_ns;
    int stall_test;
    bool promote;  // see kPromote
    // linear_kernel: tiles of x rows, CTAs of a cluster, stages
    bool gated;
    int mtiles, split, stages;
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

// 1 / x by the approximate reciprocal: 1 unit in the last place, and no special cases and so no
// branch, for x >= 1 (0 for an infinite x).
__device__ __forceinline__ float lin_recip(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + exp(-x)) from exp(-|x|), which is at most 1.
__device__ __forceinline__ float lin_sigmoid(float x)
{
    const float e = expf(-fabsf(x)), r = lin_recip(1.0f + e);
    return x < 0.0f ? e * r : r;
}

// v times the normal distribution function of v, whose lower tail is exp(-v^2 / 2) t p / 2 with
// t = 1 / (1 + 0.4 |v| / sqrt 2): t p is exp(z^2) erfc(z), z = |v| / sqrt 2, smooth in t over
// all of (0, 1], and p a degree-10 fit of least largest relative error in x = 2 t - 1, computed for
// this: 6e-9, and 4.4e-8 with every constant rounded to fp32.  No branch; erfcf took 75 issue
// slots a value, 4800 cycles a 32 x 32 box.
__device__ __forceinline__ float lin_gelu(float v)
{
    const float t = lin_recip(fmaf(0.282842712f, fabsf(v), 1.0f)), x = fmaf(2.0f, t, -1.0f);
    float p = -2.85304377e-05f;
    p = fmaf(p, x, -1.09938819e-05f);
    p = fmaf(p, x, 2.64894246e-04f);
    p = fmaf(p, x, 1.65984980e-04f);
    p = fmaf(p, x, -1.91998319e-03f);
    p = fmaf(p, x, -3.35355173e-03f);
    p = fmaf(p, x, 1.13430424e-02f);
    p = fmaf(p, x, 6.84998706e-02f);
    p = fmaf(p, x, 1.81565762e-01f);
    p = fmaf(p, x, 3.21860760e-01f);
    p = fmaf(p, x, 4.21612740e-01f);
    const float h = 0.5f * expf(-0.5f * v * v) * (p * t);
    return v * (v < 0.0f ? h : 1.0f - h);
}

// act(v).  The forms keep their relative accuracy where v is far below zero; gelu's tanh form
// is v * sigmoid(2 u), since (1 + tanh u) / 2 = sigmoid(2 u).
template <int ACT>
__device__ __forceinline__ float lin_act(float v)
{
    if (ACT == MOE_ACT_RELU) return v < 0.0f ? 0.0f : v;  // a NaN stays
    if (ACT == MOE_ACT_GELU) return lin_gelu(v);
    if (ACT == MOE_ACT_GELU_TANH)
        return v * lin_sigmoid(1.59576912160573072f * (v + 0.044715f * v * v * v));  // 2 sqrt(2 / pi) (...)
    if (ACT == MOE_ACT_SILU) return v * lin_sigmoid(v);
    return v;
}

// act of U x 4 values; the activation is the same for the whole launch, so the branch is uniform.
template <int ACT, int U>
__device__ __forceinline__ void lin_act_each(float (&v)[U][4])
{
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = lin_act<ACT>(v[j][i]);
}
template <int U>
__device__ __forceinline__ void lin_act_all(int act, float (&v)[U][4])
{
    switch (act) {
    case MOE_ACT_RELU: lin_act_each<MOE_ACT_RELU>(v); break;
    case MOE_ACT_GELU: lin_act_each<MOE_ACT_GELU>(v); break;
    case MOE_ACT_GELU_TANH: lin_act_each<MOE_ACT_GELU_TANH>(v); break;
    case MOE_ACT_SILU: lin_act_each<MOE_ACT_SILU>(v); break;
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

// The residual's four columns of the rows m + j * DM, j * DM < left, all loads under way at once.
template <int U, int DM>
__device__ __forceinline__ void lin_residual(const LinArgs &g, const LinCols &c, int64_t m, int left, float (&r)[U][4])
{
    if (!g.res || c.count <= 0) return;
    const bool vec = g.vec && c.count == 4;
    const int64_t at = m * g.ldr + c.n, step = DM * g.ldr;
    if (g.out_f32) {
        const float *p = static_cast<const float *>(g.res) + at;
        if (vec) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (j * DM < left) {
                    const float4 q = *reinterpret_cast<const float4 *>(p + j * step);
                    r[j][0] = q.x, r[j][1] = q.y, r[j][2] = q.z, r[j][3] = q.w;
                }
        } else {
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < c.count && j * DM < left) r[j][i] = p[j * step + i];
        }
    } else {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(g.res) + at;
        if (vec) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (j * DM < left) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(p + j * step);
                    r[j][0] = __uint_as_float(q.x << 16), r[j][1] = __uint_as_float(q.x & 0xffff0000u);
                    r[j][2] = __uint_as_float(q.y << 16), r[j][3] = __uint_as_float(q.y & 0xffff0000u);
                }
        } else {
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < c.count && j * DM < left) r[j][i] = __bfloat162float(p[j * step + i]);
        }
    }
}

// Finishes and stores the four columns of those rows: v the products with w, u those with w_up,
// r the residual.
template <bool GATED, int U, int DM>
__device__ __forceinline__ void lin_finish(const LinArgs &g, const LinCols &c, int64_t m, int left, float (&v)[U][4],
                                           const float (&u)[U][4], const float (&r)[U][4])
{
    if (c.count <= 0) return;
    const bool vec = g.vec && c.count == 4;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] += c.b[i];
    lin_act_all(g.act, v);
    if (GATED)
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] *= u[j][i] + c.bu[i];
    if (g.res)
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] += r[j][i];
    const int64_t at = m * g.ldo + c.n, step = DM * g.ldo;
    if (g.out_f32) {
        float *p = static_cast<float *>(g.out) + at;
        if (vec) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (j * DM < left)
                    *reinterpret_cast<float4 *>(p + j * step) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
        } else {
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < c.count && j * DM < left) p[j * step + i] = v[j][i];
        }
    } else {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(g.out) + at;
        if (vec) {
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (j * DM < left) {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v[j][0], v[j][1]);
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[j][2], v[j][3]);
                    *reinterpret_cast<uint2 *>(p + j * step) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
                }
        } else {
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < c.count && j * DM < left) p[j * step + i] = __float2bfloat16_rn(v[j][i]);
        }
    }
}

}  // namespace moe
