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
//
// Choices are those of 64-bit scores, taken in fp32 wherever that is provably the same.
// Without a bias experts are ordered by the logits themselves, exactly.  Else fp32 scores
// carry a bound of their error, and a token is settled by them if every decision of its
// (each choice against the next, the last one against all that remain, each group
// kept or dropped) is clear of twice the bound, or is between experts of equal logit
// and bias, whose scores are equal in any precision.  The few tokens left, and those whose
// weights leave fp32's range, are done again in 64 bits by one warp each.
// (16 tokens of 256 experts, sigmoid, bias, groups: 17 us all in 64 bits.)
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
__device__ __noinline__ void route_token_exact(const ScoredArgs &a, const TL *row, int t, int lane)
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

// Every token in 64 bits: the layouts that route_scored_kernel does not take.
template <int V, typename TL>
__global__ void __launch_bounds__(kWarps * 32) route_exact_kernel(const ScoredArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.T) return;
    route_token_exact<V, TL>(a, static_cast<const TL *>(a.logits) + (size_t)t * a.ld, t, threadIdx.x % 32);
}

// Floats other than NaN in the order of these keys; 0 is below all of them.
__device__ __forceinline__ uint32_t key_of(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 and 0 are equal
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

// The largest value over the G lanes of a token, on each of them.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (G == 32) {
        return __reduce_max_sync(kFull, v);
    } else {
#pragma unroll
        for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
}
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// V consecutive logits by 16-byte loads.
template <int V>
__device__ __forceinline__ void load_vec(const float *p, float (&l)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(p + i);
        l[i] = q.x, l[i + 1] = q.y, l[i + 2] = q.z, l[i + 3] = q.w;
    }
}
template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float (&l)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += 8) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            l[i + 2 * j] = __uint_as_float(w[j] << 16);
            l[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

// A token by G lanes, lane s of them the experts s v .. s v + v - 1 (v <= V): a group of experts
// is a whole number of lanes, equal scores go to the lowest lane.  VE: the experts a lane
// of route_token_exact holds.
template <int G, int V, int VE, typename TL>
__global__ void __launch_bounds__(kWarps * 32) route_scored_kernel(const ScoredArgs a, const int v, const bool vec)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % 32, sub = lane % G, seg = lane / G;
    const int t0 = (blockIdx.x * kWarps + threadIdx.x / 32) * (32 / G);
    if (t0 >= a.T) return;
    const bool live = t0 + seg < a.T;
    const int t = live ? t0 + seg : t0;
    const TL *row = static_cast<const TL *>(a.logits) + (size_t)t * a.ld;
    const bool sigmoid = a.sigmoid, biased = a.bias != nullptr;
    const int e0 = sub * v;

    float l[V], b[V], c[V];
    if (vec) {
        if (e0 < a.E)
            load_vec<V>(row + e0, l);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = i < v && e0 + i < a.E ? load_logit(row + e0 + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = biased && i < v && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
    unsigned alive = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (l[i] > -INFINITY && b[i] > -INFINITY) alive |= 1u << i;  // false for NaN
        l[i] = fminf(l[i], FLT_MAX);
    }

    float m = 0.0f, inv = 1.0f;
    if (!sigmoid) {
        uint32_t mk = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (alive >> i & 1u) mk = max(mk, key_of(l[i]));
        mk = group_max<G>(mk);
        m = mk ? of_key(mk) : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (alive >> i & 1u) s += c[i] = expf(l[i] - m);
        s = group_sum<G>(s);
        inv = mk ? 1.0f / s : 0.0f;
    }
    auto score = [&](float x) { return sigmoid ? __frcp_rn(1.0f + expf(-x)) : expf(x - m) * inv; };
    // Two scores are in their 64-bit order if they are apart by more than near: each is off by
    // at most 2^-18 of the largest p (softmax: exp 4 steps of 2^-24 and its argument's
    // rounding, a sum of V + 5 terms of such, under 64 in all) or by 6 steps of 2^-24 (sigmoid:
    // exp 4, one sum, one reciprocal); the sum with the bias is rounded once.
    const float base = (sigmoid ? 0x1p-20f : 0x1p-17f * inv) + 0x1p-120f;
    bool sure = true;
    const bool by_p = a.groups > 1 && a.top2 && !biased;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[i] = l[i];
        if (biased || by_p) {
            const float p = sigmoid ? score(l[i]) : expf(l[i] - m) * inv;
            c[i] = biased ? p + b[i] : p;
        }
    }

    if (a.groups > 1) {
        const int span = a.E / a.groups / v;  // lanes of a group
        const int g = sub / span, in = sub - g * span;
        float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (alive >> i & 1u) {
                t2 = fmaxf(t2, fminf(t1, c[i]));
                t1 = fmaxf(t1, c[i]);
            }
        for (int o = 1; o < span; o <<= 1) {  // a group's first lane gathers it
            const float o1 = __shfl_down_sync(kFull, t1, o, G), o2 = __shfl_down_sync(kFull, t2, o, G);
            if (in + o < span) {
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
        }
        const bool two = a.top2 && t2 > -INFINITY;
        float value = two ? t1 + t2 : t1, mag = two ? fabsf(t1) + fabsf(t2) : fabsf(t1);
        const int from = sub < a.groups ? sub * span : 0;  // lane h takes group h
        value = __shfl_sync(kFull, value, from, G);
        mag = __shfl_sync(kFull, mag, from, G);
        if (sub >= a.groups) value = -INFINITY;
        const bool exact = !biased && !a.top2;  // the values are logits
        int above = 0, clear = 0, close = 0;
        for (int h = 0; h < a.groups; ++h) {
            const float other = __shfl_sync(kFull, value, h, G);
            const float near = 2.0f * base + 0x1p-22f * (mag + __shfl_sync(kFull, mag, h, G));
            above += other > value || (other == value && h < sub);
            clear += other > value + near;                            // above it in any case
            close += h != sub && other > -INFINITY && !(other < value - near);  // perhaps
        }
        const bool keep = value > -INFINITY && above < a.topk_groups;
        if (!exact && value > -INFINITY) sure = close < a.topk_groups || clear >= a.topk_groups;
        const unsigned kept = __ballot_sync(kFull, keep) >> (seg * G);
        if (g >= a.groups || !(kept >> g & 1u)) alive = 0;
    }

    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = alive >> i & 1u ? key_of(biased ? c[i] : l[i]) : 0;

    // lane j keeps choice j
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, key[i]);
        const uint32_t top = group_max<G>(best);
        const unsigned has = (__ballot_sync(kFull, best == top) >> (seg * G)) & (G == 32 ? kFull : (1u << (G % 32)) - 1u);
        const int win = __ffs(has) - 1;
        bool take = sub == win && top != 0;
        int e = -1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool hit = take && key[i] == top;
            if (hit) {
                e = e0 + i;
                key[i] = 0;
                take = false;
            }
        }
        e = __shfl_sync(kFull, e, win, G);
        if (sub == j) mine = e;
    }

    const bool any = mine >= 0;
    const float lj = any ? fminf(load_logit(row + mine), FLT_MAX) : 0.0f;
    const float bj = any && biased ? a.bias[mine] : 0.0f;
    const float pj = any ? score(lj) : 0.0f;
    // below fp32's range, but not below that of 64 bits
    if (any && pj < 1e-30f && lj - m > -750.0f) sure = false;
    if (biased) {
        const float cj = pj + bj;
        const float cn = __shfl_down_sync(kFull, cj, 1, G), ln = __shfl_down_sync(kFull, lj, 1, G);
        const float bn = __shfl_down_sync(kFull, bj, 1, G);
        const int next = __shfl_down_sync(kFull, mine, 1, G);
        if (sub < a.k - 1 && next >= 0 && !(cj - cn > base + 0x1p-22f * fabsf(cj)) && !(lj == ln && bj == bn)) sure = false;
        const float ck = __shfl_sync(kFull, cj, a.k - 1, G), lk = __shfl_sync(kFull, lj, a.k - 1, G);
        const float bk = __shfl_sync(kFull, bj, a.k - 1, G);
        const float floor_k = ck - (base + 0x1p-22f * fabsf(ck));
#pragma unroll
        for (int i = 0; i < V; ++i)  // a key is left only where every choice is made
            if (key[i] && !(of_key(key[i]) < floor_k) && !(l[i] == lk && b[i] == bk)) sure = false;
    }
    unsigned open = __ballot_sync(kFull, live && !sure);
    const float sum = group_sum<G>(pj);
    const unsigned of_seg = G == 32 ? kFull : ((1u << (G % 32)) - 1u) << (seg * G % 32);
    if (live && sub < a.k && !(open & of_seg)) {
        a.idx[(size_t)t * a.k + sub] = mine;
        const float w = a.renormalize ? (sum > 0.0f ? pj / sum : 0.0f) : pj;
        a.w[(size_t)t * a.k + sub] = w * a.scale;
    }
    for (int q = 0; open && q < 32 / G; ++q) {
        const unsigned of_q = G == 32 ? kFull : ((1u << (G % 32)) - 1u) << (q * G % 32);
        if (open & of_q)
            route_token_exact<VE, TL>(a, static_cast<const TL *>(a.logits) + (size_t)(t0 + q) * a.ld, t0 + q, lane);
    }
}

// Experts a lane holds when a token has `lanes` of them, V at most: whole lanes a group (0: none).
int experts_per_lane(const ScoredArgs &a, int lanes, int V)
{
    const int size = a.E / a.groups;
    if (a.k > lanes) return 0;
    for (int v = (a.E + lanes - 1) / lanes; v <= V; ++v)
        if (a.groups == 1 || (size % v == 0 && a.groups * (size / v) <= lanes)) return v;
    return 0;
}

template <int G, int V, int VE, typename TL>
cudaError_t launch_lanes(const ScoredArgs &a, int v, cudaStream_t st)
{
    const int tokens = kWarps * (32 / G), each = 16 / (int)sizeof(TL);
    const bool vec = v == V && a.E % V == 0 && a.ld % each == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    return launch_pdl(route_scored_kernel<G, V, VE, TL>, dim3((a.T + tokens - 1) / tokens), dim3(kWarps * 32), 0, st, a,
                      v, vec);
}

// The fewest lanes a token that hold its experts, eight a lane where that is enough, and its
// choices: the work of a choice's round is a warp's, so tokens that share a warp share it.
template <typename TL>
cudaError_t launch(const ScoredArgs &a, cudaStream_t st)
{
    if (int v = experts_per_lane(a, 8, 8)) return launch_lanes<8, 8, 2, TL>(a, v, st);
    if (int v = experts_per_lane(a, 16, 8)) return launch_lanes<16, 8, 4, TL>(a, v, st);
    if (int v = experts_per_lane(a, 32, 8)) return launch_lanes<32, 8, 8, TL>(a, v, st);
    if (int v = experts_per_lane(a, 32, 16)) return launch_lanes<32, 16, 16, TL>(a, v, st);
    if (int v = experts_per_lane(a, 32, 32)) return launch_lanes<32, 32, 32, TL>(a, v, st);
    const dim3 grid((a.T + kWarps - 1) / kWarps), block(kWarps * 32);
    if (a.E <= 256) return launch_pdl(route_exact_kernel<8, TL>, grid, block, 0, st, a);
    return launch_pdl(route_exact_kernel<32, TL>, grid, block, 0, st, a);
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
