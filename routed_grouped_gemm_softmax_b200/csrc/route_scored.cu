// route_scored.cu -- scored routing: top-k experts of given router logits.
//
// For each token t with logits l[t, 0..E):
//   p_e = 1 / (1 + exp(-l_e))                      (sigmoid)   or
//   p_e = exp(l_e - max l) / sum_e' exp(l_e' - max l)  (softmax over the available experts)
//   c_e = p_e + bias_e, or l_e without a bias      (l and p order experts alike)
// With groups > 1 the experts come in `groups` runs of E / groups; a group's value is the
// largest c of its experts, or the sum of its two largest (of p without a bias), and
// only the experts of the topk_groups best groups are candidates.  The k candidates of
// largest c are chosen in descending order; equal values go to the lower index, for
// groups too.  The weight of choice j is p of its expert, divided by the sum over the
// choices if `renormalize`, times `scale`.
// An expert is available to a token if its logit and its bias are neither NaN nor
// -inf; +inf logits count as the largest finite float.  Slots left without a candidate
// get index -1 and weight 0.
#include <cfloat>
#include <climits>

#include "moe_internal.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;  // tokens per CTA
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

struct Best {
    double c;
    int e;  // expert, or INT_MAX: none
};

// The largest (c, lowest e) over the warp, on every lane.
__device__ __forceinline__ Best warp_best(Best b)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double oc = __shfl_xor_sync(kFull, b.c, o);
        const int oe = __shfl_xor_sync(kFull, b.e, o);
        if (oe != INT_MAX && (b.e == INT_MAX || oc > b.c || (oc == b.c && oe < b.e))) {
            b.c = oc;
            b.e = oe;
        }
    }
    return b;
}

// One token by one warp, every comparison between 64-bit values; lane holds the
// experts lane, lane + 32, ... (V of them).
template <int V, typename TL>
__device__ void route_token_exact(const ScoredArgs &a, const TL *row, int t, int lane)
{
    float l[V];
    double p[V], c[V];
    unsigned alive = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.E ? load_logit(row + e) : -INFINITY;
        const float b = a.bias && e < a.E ? a.bias[e] : 0.0f;
        if (l[i] > -INFINITY && b > -INFINITY) alive |= 1u << i;  // false for NaN
        l[i] = fminf(l[i], FLT_MAX);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (alive >> i & 1u) m = fmaxf(m, l[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = alive >> i & 1u ? exp((double)l[i] - (double)m) : 0.0;
            s += p[i];
        }
        s = warp_sum(s);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = s > 0.0 ? p[i] / s : 0.0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        c[i] = a.bias && e < a.E ? p[i] + (double)a.bias[e] : (double)l[i];
    }

    if (a.groups > 1) {
        // lane g keeps group g's value
        const int size = a.E / a.groups;
        const bool by_p = a.top2 && !a.bias;
        Best mine{0.0, INT_MAX};
        for (int g = 0; g < a.groups; ++g) {
            Best b{0.0, INT_MAX}, b2{0.0, INT_MAX};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                const double v = by_p ? p[i] : c[i];
                if ((alive >> i & 1u) && e >= g * size && e < (g + 1) * size && (b.e == INT_MAX || v > b.c)) b = {v, e};
            }
            b = warp_best(b);
            if (a.top2) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 32 * i;
                    const double v = by_p ? p[i] : c[i];
                    if ((alive >> i & 1u) && e >= g * size && e < (g + 1) * size && e != b.e &&
                        (b2.e == INT_MAX || v > b2.c))
                        b2 = {v, e};
                }
                b2 = warp_best(b2);
            }
            if (lane == g && b.e != INT_MAX) mine = {b2.e != INT_MAX ? b.c + b2.c : b.c, g};
        }
        unsigned keep = 0;
        for (int j = 0; j < a.topk_groups; ++j) {
            const Best b = warp_best(mine);
            if (b.e == INT_MAX) break;
            keep |= 1u << b.e;
            if (lane == b.e) mine.e = INT_MAX;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((alive >> i & 1u) && !(keep >> ((lane + 32 * i) / size) & 1u)) alive &= ~(1u << i);
    }

    // lane j % 32 keeps p of choice j until the sum is known
    int32_t *idx = a.idx + (size_t)t * a.k;
    double sum = 0.0, kept[V];
    for (int j = 0; j < a.k; ++j) {
        Best b{0.0, INT_MAX};
        double bp = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((alive >> i & 1u) && (b.e == INT_MAX || c[i] > b.c)) {
                b = {c[i], lane + 32 * i};
                bp = p[i];
            }
        b = warp_best(b);
        const bool any = b.e != INT_MAX;
        const double pj = any ? __shfl_sync(kFull, bp, b.e & 31) : 0.0;
        if (any && lane == (b.e & 31)) alive &= ~(1u << (b.e >> 5));
        sum += pj;
        if (lane == (j & 31)) {
            idx[j] = any ? b.e : -1;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == j >> 5) kept[i] = pj;
        }
    }
    if (!a.renormalize) sum = 1.0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.k)
            a.w[(size_t)t * a.k + lane + 32 * i] = sum > 0.0 ? (float)(kept[i] / sum * (double)a.scale) : 0.0f;
}

template <int V, typename TL>
__global__ void __launch_bounds__(kWarps * 32) route_scored_kernel(const ScoredArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.T) return;
    route_token_exact<V, TL>(a, static_cast<const TL *>(a.logits) + (size_t)t * a.ld, t, threadIdx.x % 32);
}

template <typename TL>
cudaError_t launch(const ScoredArgs &a, cudaStream_t st)
{
    const dim3 grid((a.T + kWarps - 1) / kWarps), block(kWarps * 32);
    if (a.E <= 64) return launch_pdl(route_scored_kernel<2, TL>, grid, block, 0, st, a);
    if (a.E <= 256) return launch_pdl(route_scored_kernel<8, TL>, grid, block, 0, st, a);
    return launch_pdl(route_scored_kernel<32, TL>, grid, block, 0, st, a);
}

}  // namespace

cudaError_t launch_route_scored(const ScoredArgs &a, bool bf16, cudaStream_t st)
{
    return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace moe

extern "C" moe_status_t moe_route_scored(const moe_scored_t *o, const void *logits, const float *bias,
                                         int32_t *topk_idx, float *topk_w, void *stream)
{
    if (!o || o->T < 0 || o->E <= 0 || o->top_k < 1 || o->top_k > o->E) return MOE_ERR_INVALID_ARG;
    if (o->scoring != MOE_SCORE_SOFTMAX && o->scoring != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (o->group_score != MOE_GROUP_MAX && o->group_score != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
    if (o->logits_dtype != MOE_LOGITS_F32 && o->logits_dtype != MOE_LOGITS_BF16) return MOE_ERR_INVALID_ARG;
    if (o->n_groups < 1 || o->E % o->n_groups != 0) return MOE_ERR_INVALID_ARG;
    if (o->topk_groups < 1 || o->topk_groups > o->n_groups) return MOE_ERR_INVALID_ARG;
    if (o->top_k > o->topk_groups * (o->E / o->n_groups)) return MOE_ERR_INVALID_ARG;
    if (o->ld < o->E) return MOE_ERR_INVALID_ARG;
    if (o->E > moe::kMaxExperts || o->n_groups > 32) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)o->T * o->top_k > (int64_t)INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if (o->T == 0) return MOE_OK;
    if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
    const uintptr_t align = o->logits_dtype == MOE_LOGITS_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % align || reinterpret_cast<uintptr_t>(bias) % 4 ||
        reinterpret_cast<uintptr_t>(topk_idx) % 4 || reinterpret_cast<uintptr_t>(topk_w) % 4)
        return MOE_ERR_INVALID_ARG;
    const moe::ScoredArgs a{logits, o->ld, bias, o->T, o->E, o->top_k, o->scoring == MOE_SCORE_SIGMOID, o->n_groups,
                            o->topk_groups, o->group_score == MOE_GROUP_TOP2, o->renormalize != 0, o->scale,
                            topk_idx, topk_w};
    return moe::launch_route_scored(a, o->logits_dtype == MOE_LOGITS_BF16, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
