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
// Without a bias experts are ordered by the logits themselves.  Else fp32 scores carry a
// bound of their error, and a choice stands if it is clear of the next one (the last of all that
// remain) by twice the bound, or equal to it in logit and bias and so in any precision.  Where
// not, the experts in question take the place of their 64-bit scores, one a lane; a
// token whose groups are in question, or whose weights leave fp32's range, is done again with
// 64-bit scores throughout, and so is a softmax with a bias, for its 64-bit sum.
// Bound by instructions: about 1100 a warp with bias and groups (256 experts, k 8), 650 a warp of
// four tokens without (64, k 6).  16 x 256 in 64 bits throughout 17.0 us, so 3.4; 4096 x 256
// (sigmoid, bias, groups) 31.8 and 8.7; 65536 x 64 bf16 softmax 71.4 and 13.9.
#include <cfloat>
#include <climits>

#include "moe_internal.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;  // warps per CTA: a token each, or 32 / G where one has G lanes
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

// Numbers other than NaN in the order of their keys; 0 is below all of them.
template <typename S>
struct Keys;
template <>
struct Keys<float> {
    using T = uint32_t;
    static __device__ __forceinline__ T of(float f)
    {
        const T u = __float_as_uint(f + 0.0f);  // -0 and 0 are equal
        return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
    }
    static __device__ __forceinline__ float value(T k)
    {
        return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
    }
};
template <>
struct Keys<double> {
    using T = unsigned long long;
    static __device__ __forceinline__ T of(double f)
    {
        const T u = static_cast<T>(__double_as_longlong(f + 0.0));
        return u ^ (u >> 63 ? ~0ull : 1ull << 63);
    }
};

// The largest key over the G lanes of a token, on each of them.
template <int G, typename K>
__device__ __forceinline__ K group_max(K v)
{
    if constexpr (G == 32 && sizeof(K) == 4) {
        return __reduce_max_sync(kFull, v);
    } else if constexpr (G == 32) {
        const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(v >> 32));
        const uint32_t lo = __reduce_max_sync(kFull, v >> 32 == hi ? static_cast<uint32_t>(v) : 0u);
        return static_cast<K>(hi) << 32 | lo;
    } else {
#pragma unroll
        for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
}
template <int G, typename S>
__device__ __forceinline__ S group_sum(S v)
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

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

// Sorts V (a power of two) numbers, the largest first: Batcher's odd-even merges.
template <int V, typename T>
__device__ __forceinline__ void sort_down(T (&x)[V])
{
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int d = p; d >= 1; d /= 2)
#pragma unroll
            for (int j = d % p; j + d < V; j += 2 * d)
#pragma unroll
                for (int i = j; i < j + d && i + d < V; ++i)
                    if (i / (2 * p) == (i + d) / (2 * p)) {
                        const T hi = max(x[i], x[i + d]), lo = min(x[i], x[i + d]);
                        x[i] = hi, x[i + d] = lo;
                    }
}

// How a token's experts lie over its lanes: lane s has the experts s v .. s v + v - 1, so
// that a group of experts is `span` whole lanes and equal scores go to the lowest lane.
struct Lanes {
    int v, span;
    unsigned per_span;  // lane / span = lane * per_span >> 16
    bool vec;           // V logits of a lane by 16-byte loads
};

// Routes a warp's 32 / G tokens from t0 on with scores of type S, those in `wanted` (a
// mask of their lanes) only.  Writes the tokens whose choices are those of 64 bits and returns
// a mask of the lanes that found another one (none for S = double).
template <typename S, int G, int V, typename TL>
__device__ __forceinline__ unsigned route_tokens(const ScoredArgs &a, const Lanes &at, int t0, unsigned wanted)
{
    using K = Keys<S>;
    constexpr bool kBound = sizeof(S) == 4;  // scores are off by a bounded error
    // 64 bits: loops rather than straight code, which would be fetched for a token in hundreds
    constexpr int kUnroll = kBound ? V : 1;
    const int lane = threadIdx.x % 32, sub = lane % G, seg = lane / G;
    const bool live = wanted >> lane & 1u;
    const int t = t0 + seg < a.T ? t0 + seg : t0;
    const TL *row = static_cast<const TL *>(a.logits) + (size_t)t * a.ld;
    const bool sigmoid = a.sigmoid, biased = a.bias != nullptr;
    const int e0 = sub * at.v;

    float l[V], b[V];  // l = -inf: no such expert, or not available
    if (at.vec) {
        if (e0 < a.E)
            load_vec<V>(row + e0, l);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = i < at.v && e0 + i < a.E ? load_logit(row + e0 + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = l[i] > -INFINITY ? fminf(l[i], FLT_MAX) : -INFINITY;  // NaN too
    if (biased)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b[i] = i < at.v && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
            l[i] = b[i] > -INFINITY ? l[i] : -INFINITY;
        }

    S m = 0, total = 1, inv = 1;
    if (!sigmoid) {
        float most = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) most = fmaxf(most, l[i]);
        most = Keys<float>::value(group_max<G>(Keys<float>::of(most)));
        const bool some = most > -INFINITY;
        m = some ? most : 0.0f;
        S s = 0;
#pragma unroll kUnroll
        for (int i = 0; i < V; ++i) s += exp_of(static_cast<S>(l[i]) - m);
        s = group_sum<G>(s);
        if (some) total = s;
        inv = 1 / total;
    }
    // 64 bits: the quotient itself, since sums of scores and biases can tie but for a rounding
    auto score = [&](float x) {
        if (sigmoid) return inverse(1 + exp_of(-static_cast<S>(x)));
        const S e = exp_of(static_cast<S>(x) - m);
        return kBound ? e * inv : e / total;
    };
    // Two fp32 scores are in their 64-bit order if they are apart by more than base: each is off
    // by at most 2^-18 of the largest p (softmax: exp 4 steps of 2^-24 and its argument's
    // rounding, a sum of V + 5 terms of such, under 64 in all) or by 7 steps of 2^-24 (sigmoid:
    // exp 4, one sum, reciprocal 2); and the sum with the bias is rounded once (rel).  Logits
    // are compared as they are.
    const float base = static_cast<float>(sigmoid ? 0x1p-20f : 0x1p-17f * inv) + 0x1p-120f;
    bool sure = true;
    S c[V];  // what orders the experts
    if (biased) {
#pragma unroll kUnroll
        for (int i = 0; i < V; ++i) c[i] = l[i] > -INFINITY ? score(l[i]) + b[i] : -INFINITY;
    } else {
#pragma unroll kUnroll
        for (int i = 0; i < V; ++i) c[i] = l[i];
    }

    bool dropped = false;
    if (a.groups > 1) {
        const int g = sub * at.per_span >> 16, in = sub - g * at.span;
        S t1 = -INFINITY, t2 = -INFINITY;
        if (a.top2 && !biased) {
#pragma unroll kUnroll
            for (int i = 0; i < V; ++i) {
                const S p = l[i] > -INFINITY ? score(l[i]) : -INFINITY;
                t2 = max(t2, min(t1, p));
                t1 = max(t1, p);
            }
        } else {
#pragma unroll kUnroll
            for (int i = 0; i < V; ++i) {
                t2 = max(t2, min(t1, c[i]));
                t1 = max(t1, c[i]);
            }
        }
        for (int o = 1; o < at.span; o <<= 1) {  // a group's first lane gathers it
            const S o1 = __shfl_down_sync(kFull, t1, o, G), o2 = __shfl_down_sync(kFull, t2, o, G);
            if (in + o < at.span) {
                t2 = max(min(t1, o1), max(t2, o2));
                t1 = max(t1, o1);
            }
        }
        const bool two = a.top2 && t2 > -INFINITY;
        const int from = sub < a.groups ? sub * at.span : 0;  // lane h takes group h
        S value = __shfl_sync(kFull, two ? t1 + t2 : t1, from, G);
        if (sub >= a.groups) value = -INFINITY;
        const bool bound = kBound && (biased || a.top2);  // else the values are logits
        float mag = 0.0f;
        if (bound) mag = __shfl_sync(kFull, static_cast<float>(two ? fabs(t1) + fabs(t2) : fabs(t1)), from, G);
        int above = 0, clear = 0, close = 0;
        for (int h = 0; h < a.groups; ++h) {
            const S other = __shfl_sync(kFull, value, h, G);
            above += other > value || (other == value && h < sub);
            if (bound) {
                const float near = 2.0f * base + 0x1p-22f * (mag + __shfl_sync(kFull, mag, h, G));
                clear += other > value + near;                                               // above in any case
                close += h != sub && other > -INFINITY && !(other < value - near);  // perhaps
            }
        }
        const bool keep = value > -INFINITY && above < a.topk_groups;
        if (bound && value > -INFINITY) sure = close < a.topk_groups || clear >= a.topk_groups;
        const unsigned kept = __ballot_sync(kFull, keep) >> (seg * G);
        dropped = g >= a.groups || !(kept >> g & 1u);
    }

    // Choices: lane j keeps choice j.  A key at or below that of -inf is none.
    const typename K::T none = K::of(-INFINITY) | (V - 1);
    // fp32: the low bits of a key give way to the expert's place in its lane, the lower place
    // the larger key, so that a lane's keys can be sorted as they are.  Numbers that differ in
    // those bits alone may come out of order, which the checks below find.
    typename K::T key[V];
#pragma unroll kUnroll
    for (int i = 0; i < V; ++i) {
        key[i] = dropped ? 0 : K::of(c[i]);
        if (kBound && !dropped) key[i] = (key[i] & ~static_cast<typename K::T>(V - 1)) | (V - 1 - i);
    }
    int mine = -1;
    // fp32: the best expert left becomes lane j's if its key is at least `from`; a round compares the
    // lanes' first keys and the winner moves up
    auto pick = [&](int j, typename K::T from) {
        const typename K::T first = key[0] & ~static_cast<typename K::T>(V - 1);  // equal ones: the lowest lane's
        const typename K::T top = group_max<G>(first);
        unsigned has = __ballot_sync(kFull, first == top);
        if (G < 32) has = has >> (seg * G) & ((1u << (G % 32)) - 1u);
        const int win = __ffs(has) - 1;
        const int e = __shfl_sync(kFull, e0 + V - 1 - static_cast<int>(key[0] & (V - 1)), win, G);
        const bool ok = (top | (V - 1)) >= from;
        if (sub == win && ok) {
#pragma unroll
            for (int i = 0; i < V - 1; ++i) key[i] = key[i + 1];
            key[V - 1] = 0;
        }
        if (sub == j && ok) mine = e;
        return ok;
    };
    if constexpr (kBound) {
        sort_down(key);
        for (int j = 0; j < a.k; ++j) pick(j, none + 1);
    } else {
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            typename K::T best = 0;
            int place = 0;
#pragma unroll 1
            for (int i = 0; i < V; ++i)
                if (key[i] > best) {
                    best = key[i];
                    place = i;
                }
            const typename K::T top = group_max<G>(best);
            unsigned has = __ballot_sync(kFull, best == top);
            if (G < 32) has = has >> (seg * G) & ((1u << (G % 32)) - 1u);
            const int win = __ffs(has) - 1;
            if (sub == win) key[place] = 0;
            const int e = __shfl_sync(kFull, e0 + place, win, G);
            if (sub == j && top > none) mine = e;
        }
    }

    float lj = mine >= 0 ? fminf(load_logit(row + mine), FLT_MAX) : 0.0f;
    float bj = mine >= 0 && biased ? a.bias[mine] : 0.0f;
    S pj = mine >= 0 ? score(lj) : static_cast<S>(0);
    int place = sub;  // this lane's choice among the token's
    const bool whole_keys = sizeof(TL) == 2 && !biased;  // of bf16 logits: what gave way was zero
    if (kBound && !whole_keys) {
        // each choice is clear of the next, or equal to it
        const float cj = biased ? pj + bj : lj, step = biased ? base + 0x1p-22f * fabsf(cj) : 0.0f;
        const float cn = __shfl_down_sync(kFull, cj, 1, G), ln = __shfl_down_sync(kFull, lj, 1, G);
        const float bn = __shfl_down_sync(kFull, bj, 1, G);
        const int next = __shfl_down_sync(kFull, mine, 1, G);
        bool settled = !(sub < a.k - 1 && next >= 0 && !(cj - cn > step) && !(lj == ln && bj == bn));
        // and the experts that are not clearly below the last choice, nor equal to it, are choices
        const float lk = __shfl_sync(kFull, lj, a.k - 1, G), bk = __shfl_sync(kFull, bj, a.k - 1, G);
        const float least = __shfl_sync(kFull, cj - step, a.k - 1, G);
        const bool full = __shfl_sync(kFull, mine, a.k - 1, G) >= 0;
        int more = mine >= 0 && !(cj < least) && !(lj == lk && bj == bk) ? -1 : 0;
        if (!dropped)
#pragma unroll
            for (int i = 0; i < V; ++i)
                more += l[i] > -INFINITY && !(c[i] < least) && !(l[i] == lk && (!biased || b[i] == bk));
#pragma unroll
        for (int o = G / 2; o; o >>= 1) more += __shfl_xor_sync(kFull, more, o);
        if (full && more) settled = false;
        const unsigned doubt = __ballot_sync(kFull, live && !settled);
        if (doubt) {
            // All experts that may belong to the choices become candidates, one a lane, and take
            // the place of their 64-bit score.  A softmax's takes a 64-bit sum: done again below.
            const unsigned of_seg = G == 32 ? kFull : ((1u << (G % 32)) - 1u) << (seg * G % 32);
            const bool here = doubt & of_seg;
            float low = mine >= 0 ? cj - step : INFINITY;
            const unsigned odd = __ballot_sync(kFull, mine >= 0 && !isfinite(low)) & of_seg;
#pragma unroll
            for (int o = G / 2; o; o >>= 1) low = fminf(low, __shfl_xor_sync(kFull, low, o));
            if (here && (odd || (biased && !sigmoid))) sure = false;
            bool open = here && full && sure;
            int n = a.k;
            while (__any_sync(kFull, open)) {
                if (n == G) {
                    if (open) sure = false;
                    break;
                }
                open = pick(n, open ? K::of(low) : 0xffffffffu) && open;
                ++n;
            }
            if (mine >= 0) {
                lj = fminf(load_logit(row + mine), FLT_MAX);
                bj = biased ? a.bias[mine] : 0.0f;
                pj = score(lj);
            }
            const double mj = !biased ? lj : 1.0 / (1.0 + exp(-static_cast<double>(lj))) + bj;
            int before = 0;
            for (int h = 0; h < n; ++h) {
                const double mh = __shfl_sync(kFull, mj, h, G);
                const int eh = __shfl_sync(kFull, mine, h, G);
                before += eh >= 0 && (mh > mj || (mh == mj && eh < mine));
            }
            if (here && mine >= 0) place = before;
            if (place >= a.k || mine < 0) {
                pj = 0.0f;
                if (here && mine >= 0) mine = -2;  // a candidate that is not chosen
            }
        }
    }
    // below fp32's range, but not below that of 64 bits
    if (kBound && mine >= 0 && pj < 1e-30f && lj - m > -750.0f) sure = false;
    const unsigned open = __ballot_sync(kFull, live && !sure);
    const unsigned of_seg = G == 32 ? kFull : ((1u << (G % 32)) - 1u) << (seg * G % 32);
    const S sum = group_sum<G>(pj);
    if (live && place < a.k && mine > -2 && !(open & of_seg)) {
        a.idx[(size_t)t * a.k + place] = mine;
        const S w = a.renormalize ? (sum > 0 ? pj / sum : static_cast<S>(0)) : pj;
        a.w[(size_t)t * a.k + place] = static_cast<float>(w * a.scale);
    }
    unsigned again = 0;
    if (kBound && open)
        for (int q = 0; q < 32 / G; ++q) {
            const unsigned of_q = G == 32 ? kFull : ((1u << (G % 32)) - 1u) << (q * G % 32);
            if (open & of_q) again |= of_q;
        }
    return again;
}

template <int G, int V, typename TL>
__device__ __noinline__ void route_tokens_64(const ScoredArgs &a, const Lanes &at, int t0, unsigned wanted)
{
    route_tokens<double, G, V, TL>(a, at, t0, wanted);
}

template <int G, int V, typename TL>
__global__ void __launch_bounds__(kWarps * 32) route_scored_kernel(const ScoredArgs a, const Lanes at)
{
    pdl_wait();
    pdl_trigger();
    const int t0 = (blockIdx.x * kWarps + threadIdx.x / 32) * (32 / G);
    if (t0 >= a.T) return;
    const unsigned here = __ballot_sync(kFull, t0 + (int)(threadIdx.x % 32) / G < a.T);
    const unsigned again = route_tokens<float, G, V, TL>(a, at, t0, here);
    if (again) route_tokens_64<G, V, TL>(a, at, t0, again);
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

template <int G, int V, typename TL>
cudaError_t launch_lanes(const ScoredArgs &a, int v, cudaStream_t st)
{
    const int tokens = kWarps * (32 / G), each = 16 / (int)sizeof(TL);
    const bool vec = v == V && a.E % V == 0 && a.ld % each == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    const int span = a.groups > 1 ? a.E / a.groups / v : 32;
    const Lanes at{v, span, 65536u / span + 1u, vec};
    return launch_pdl(route_scored_kernel<G, V, TL>, dim3((a.T + tokens - 1) / tokens), dim3(kWarps * 32), 0, st, a, at);
}

// The fewest lanes a token that hold its experts, eight a lane where that is enough, and its
// choices: the work of a choice's round is a warp's, so tokens that share a warp share it.
template <typename TL>
cudaError_t launch(const ScoredArgs &a, cudaStream_t st)
{
    if (int v = experts_per_lane(a, 8, 8)) return launch_lanes<8, 8, TL>(a, v, st);
    if (int v = experts_per_lane(a, 16, 8)) return launch_lanes<16, 8, TL>(a, v, st);
    if (int v = experts_per_lane(a, 32, 8)) return launch_lanes<32, 8, TL>(a, v, st);
    if (int v = experts_per_lane(a, 32, 16)) return launch_lanes<32, 16, TL>(a, v, st);
    if (int v = experts_per_lane(a, 32, 32)) return launch_lanes<32, 32, TL>(a, v, st);
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
