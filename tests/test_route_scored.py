"""moe_route_scored: refusals on the host, and the GPU kernel against a 64-bit NumPy form of the
same definition (choices equal, weights within the rounding of their fp32 evaluation)."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

from routed_grouped_gemm_softmax_b200 import api, build

F32_MAX = float(np.finfo(np.float32).max)


def scored(T=4, E=8, k=2, scoring=0, groups=1, topk_groups=1, group_score=0, renorm=1, scale=1.0, dtype=0, ld=None):
    return api.Scored(T, E, k, scoring, groups, topk_groups, group_score, renorm, scale, dtype, E if ld is None else ld)


def test_host_refusals():
    build.build()
    L = api.lib()
    buf = ctypes.create_string_buffer(4096)
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def call(o, logits=p, bias=None, idx=p, w=p):
        return L.moe_route_scored(None if o is None else ctypes.byref(o), logits, bias, idx, w, None)

    assert call(None) == 1
    assert call(scored(T=-1)) == 1
    assert call(scored(E=0, k=1)) == 1
    assert call(scored(k=0)) == 1 and call(scored(k=9)) == 1
    assert call(scored(scoring=2)) == 1 and call(scored(scoring=-1)) == 1
    assert call(scored(group_score=2)) == 1 and call(scored(dtype=2)) == 1
    assert call(scored(groups=3)) == 1 and call(scored(groups=0)) == 1   # 8 experts in 3 groups
    assert call(scored(groups=4, topk_groups=5)) == 1 and call(scored(groups=4, topk_groups=0)) == 1
    assert call(scored(groups=4, topk_groups=1, k=3)) == 1               # one group has 2 experts
    assert call(scored(ld=7)) == 1
    assert call(scored(E=1025)) == 2 and call(scored(E=66, groups=33)) == 2
    assert call(scored(T=(1 << 30), k=2)) == 2
    assert call(scored(T=0), None, None, None, None) == 0
    assert call(scored(), None) == 1 and call(scored(), idx=None) == 1 and call(scored(), w=None) == 1
    assert call(scored(), p + 2) == 1 and call(scored(dtype=1), p + 1) == 1
    assert call(scored(), bias=p + 2) == 1 and call(scored(), idx=p + 2) == 1 and call(scored(), w=p + 2) == 1


def test_python_refusals_need_no_gpu():
    with pytest.raises(ValueError):
        api.moe_route_scored(torch.zeros(4, 8), 2)          # not on a GPU
    with pytest.raises(ValueError):
        api.moe_route_scored(torch.zeros(8), 2)


# ------------------------------------------------------------------ the 64-bit form

def oracle(logits, k, scoring, bias, groups, topk_groups, group_score, renorm, scale):
    x = logits.astype(np.float64)
    T, E = x.shape
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        l = np.minimum(x[t], F32_MAX)
        b = np.zeros(E) if bias is None else bias.astype(np.float64)
        ok = [e for e in range(E) if l[e] > -math.inf and b[e] > -math.inf]
        if not ok:
            continue
        p = np.zeros(E)
        with np.errstate(over="ignore"):
            if scoring == "sigmoid":
                p[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
            else:
                m = max(l[e] for e in ok)
                p[ok] = np.exp(l[ok] - m)
                p /= p.sum()
        c = l if bias is None else p + b
        if groups > 1:
            n = E // groups
            value = {}
            for g in range(groups):
                v = p if group_score == "top2" and bias is None else c
                v = sorted((v[e] for e in ok if e // n == g), reverse=True)
                if v:
                    value[g] = sum(v[:2]) if group_score == "top2" else v[0]
            best = sorted(value, key=lambda g: (-value[g], g))[:topk_groups]
            ok = [e for e in ok if e // n in best]
        chosen = sorted(ok, key=lambda e: (-c[e], e))[:k]
        idx[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = p[chosen]
        if renorm:
            s = w[t].sum()
            w[t] = w[t] / s if s > 0 else 0.0
    return idx, w * scale


def check(logits, k, scoring="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renorm=True, scale=1.0):
    idx, w = api.moe_route_scored(logits, k, scoring, bias, groups, topk_groups, group_score, renorm, scale)
    torch.cuda.synchronize()
    x = logits.float().cpu().numpy()
    ri, rw = oracle(x, k, scoring, None if bias is None else bias.cpu().numpy(), groups, topk_groups, group_score,
                    renorm, scale)
    gi = idx.cpu().numpy()
    assert np.array_equal(gi, ri), f"rows {np.unique(np.argwhere(gi != ri)[:, 0])[:5]}"
    # fp32 evaluation of a weight: the exponent's argument is rounded once (relative error
    # |l - max l| / 2^24), exp is within 2 units in the last place, the sum over the experts
    # takes at most 32 + 5 roundings, the renormalising sum k, the rest under 8
    fin = np.where(np.isfinite(x), x, 0.0)
    depth = np.minimum((fin.max(1) - fin.min(1)), 104.0)[:, None] if scoring == "softmax" else 0.0
    rtol = (depth + 4 + 37 + k + 8) * 2.0 ** -24
    gw = w.cpu().double().numpy()
    # below the normal range a float keeps an absolute spacing of 2^-149, and exp may flush to 0 there
    assert np.all(np.abs(gw - rw) <= rtol * np.abs(rw) + 2.0 ** -125 * max(1.0, scale)), np.max(np.abs(gw - rw))


def rows(T, E, pad=0, dtype=torch.float32, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E + pad, generator=g) * std).to(dtype).cuda()[:, :E]


def a_bias(E, seed=1):
    return (0.05 * torch.randn(E, generator=torch.Generator().manual_seed(seed))).cuda()


SHAPES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (5, 8, 8, 4, 4), (33, 60, 4, 4, 2), (64, 64, 6, 8, 3), (7, 160, 6, 8, 3),
          (129, 256, 8, 8, 4), (3, 257, 7, 1, 1), (9, 384, 9, 1, 1), (17, 512, 8, 16, 4), (4, 1000, 40, 1, 1),
          (3, 1024, 64, 32, 5), (2, 1024, 1024, 1, 1), (2, 96, 33, 2, 2), (31, 32, 3, 32, 7)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,groups,topk_groups", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_64_bits(T, E, k, groups, topk_groups, dtype):
    for n, (scoring, bias, group_score, renorm, scale, pad) in enumerate([
            ("softmax", None, "max", True, 1.0, 0), ("sigmoid", None, "top2", True, 2.5, 3),
            ("sigmoid", a_bias(E), "top2", True, 2.5, 0), ("softmax", a_bias(E), "max", False, 16.0, 8),
            ("softmax", None, "top2", False, 1.0, 1), ("sigmoid", a_bias(E), "max", False, 1.0, 5)]):
        check(rows(T, E, pad, dtype, seed=n), k, scoring, bias, groups, topk_groups, group_score, renorm, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(64, 1, 1, 6), (64, 8, 3, 6), (256, 8, 4, 8), (160, 8, 2, 10)])
def test_masked_experts_and_empty_rows(scoring, dtype, E, groups, topk_groups, k):
    low = torch.finfo(dtype).min
    x = rows(12, E, 2, dtype, seed=3).clone()
    x[0] = -math.inf                       # nothing available
    x[1] = math.nan
    x[2] = low                             # available, all equal
    x[3, 3:] = -math.inf                   # fewer than k
    x[4, 1:] = low
    x[5, ::2] = math.nan
    x[6, 5] = math.inf                     # the largest finite value
    x[7, :] = math.inf
    x[8, E // 2:] = -math.inf              # whole groups
    x[9, torch.arange(E) % (E // groups) != 0] = -math.inf  # one expert a group
    x[10] = 0.0                            # ties: the lowest indices
    x[11, 1:] = x[11, 0]
    bias = a_bias(E)
    gone = bias.clone()
    gone[1::3] = -math.inf
    gone[2] = math.nan
    for b in (None, bias, gone):
        for group_score in ("max", "top2"):
            for renorm in (True, False):
                check(x, k, scoring, b, groups, topk_groups, group_score, renorm, 2.0)


@pytest.mark.gpu
def test_near_ties_are_decided_in_64_bits():
    # scores that differ by less than an fp32 step of the value they are compared at
    E, k = 64, 8
    T = 200
    g = torch.Generator().manual_seed(5)
    x = 3.0 + 1e-6 * torch.randn(T, E, generator=g)
    bias = (1e-7 * torch.randn(E, generator=g)).cuda()
    for scoring in ("softmax", "sigmoid"):
        check(x.cuda(), k, scoring, bias)
        check(x.cuda(), k, scoring, None, 8, 2, "top2")
        check(x.cuda(), k, scoring, bias, 8, 2, "top2")
        check((x * 1e4).cuda(), k, scoring, None)        # saturated sigmoids keep the logits' order
    check((-x * 60).cuda(), k, "sigmoid", None)          # scores below fp32's normal range


@pytest.mark.gpu
def test_extreme_ranges():
    x = rows(16, 256, 0, torch.float32, 7, std=50.0)
    check(x, 8, "softmax")
    check(x, 8, "sigmoid", a_bias(256), 8, 4, "top2", True, 2.5)
    check(x * 1e30, 8, "softmax", None, 8, 4, "max", False)
    b = a_bias(256) * 1e30
    check(x, 8, "sigmoid", b, 8, 4, "top2")
    inf = a_bias(256)
    inf[[3, 77]] = math.inf
    check(x, 8, "sigmoid", inf, 8, 4, "max")


def batch64(x, k, scoring, bias, groups, topk_groups, group_score):
    """The choices and scores of many rows of finite logits, in 64 bits: stable sorts, ties to the lower index."""
    T, E = x.shape
    x = x.double()
    p = torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, 1)
    c = x if bias is None else p + bias.double()
    # A group's sum (p1 + b1) + (p2 + b2) takes three roundings of up to 2^-53 a unit (values here are below 4, so 2^-52
    # apart at most 3 * 2^-52 each); where two groups have the same p's and the same sum of biases in another order (biases
    # that are multiples of 1/64), the sums are equal in exact arithmetic and those roundings alone order
    # them: 2^-49 > 2 * 3 * 2^-52 apart or less, the choice of group is not a matter of 64-bit scores.
    open_ = torch.zeros(T, dtype=torch.bool, device=x.device)
    if groups > 1:
        v = (p if bias is None and group_score == "top2" else c).view(T, groups, E // groups)
        v = v.sort(dim=2, descending=True).values[:, :, :2 if group_score == "top2" else 1].sum(2)
        if bias is not None and group_score == "top2" and bool((bias != bias[0]).any()):
            s = v.sort(dim=1, descending=True).values
            open_ = s[:, topk_groups - 1] - s[:, topk_groups] < 2.0 ** -49
        best = v.sort(dim=1, descending=True, stable=True).indices[:, :topk_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        c = c.masked_fill(~keep.repeat_interleave(E // groups, 1), -math.inf)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    return idx, p.gather(1, idx), open_


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(8, 1, 1, 2), (64, 1, 1, 6), (64, 8, 3, 8), (96, 1, 1, 10), (120, 4, 2, 16),
                                                    (148, 4, 2, 6), (160, 8, 3, 6), (256, 8, 4, 8), (256, 1, 1, 32), (384, 1, 1, 8), (512, 16, 4, 8),
                                                    (1000, 1, 1, 8), (1024, 32, 4, 30)])
def test_every_choice_of_many_rows(scoring, E, groups, topk_groups, k):
    T = 6001
    g = torch.Generator().manual_seed(E + k)
    base = torch.randn(T, E, generator=g)
    coarse = (torch.randn(E, generator=g) * 4).round() / 64  # biases that repeat
    for logits in (base, base.bfloat16(), (base * 2).round() / 2, 12 + 3 * base.bfloat16().float(), -9 + 1e-4 * base):
        x = logits.cuda()
        for bias in (None, a_bias(E), coarse.cuda(), torch.zeros(E, device="cuda")):
            for group_score in ("max", "top2") if groups > 1 else ("max",):
                idx, w = api.moe_route_scored(x, k, scoring, bias, groups, topk_groups, group_score, False)
                ri, rp, open_ = batch64(x.float(), k, scoring, bias, groups, topk_groups, group_score)
                assert int(open_.sum()) < T // 10
                rp = torch.where(open_[:, None], w.double(), rp)
                wrong = (idx != ri).any(1) & ~open_
                assert not bool(wrong.any()), (int(wrong.sum()), int(wrong.nonzero()[0]))
                # exp 4 steps of 2^-24 and its argument's rounding (up to 60 below the maximum here), a sum of at most 37 terms
                # of such, a quotient and a product
                assert bool(((w.double() - rp).abs() <= 2.0 ** -24 * (60 + 4 + 60 + 4 + 37 + 4) * rp).all())


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,topk_groups,k", [(8, 1, 1, 8), (64, 1, 1, 6), (64, 8, 3, 6), (1000, 1, 1, 32), (256, 8, 4, 8)])
def test_bf16_logits_of_few_values(E, groups, topk_groups, k):
    # many equal logits, zeros of both signs, the largest finite values beside infinities
    g = torch.Generator().manual_seed(E)
    top = torch.finfo(torch.bfloat16).max
    pool = torch.tensor([0.0, -0.0, 1.0, 1.0078125, -3.0, top, -top, math.inf, -math.inf, 2.0 ** -130, -2.0 ** -130, math.nan])
    for n in (len(pool), 7, 3):
        x = pool[torch.randint(0, n, (60, E), generator=g)].bfloat16().cuda()
        for group_score in ("max", "top2"):
            check(x, k, "softmax", None, groups, topk_groups, group_score)
            check(x, k, "sigmoid", None, groups, topk_groups, group_score, True, 2.5)
            check(x, k, "sigmoid", a_bias(E), groups, topk_groups, group_score)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    T, E, ld = 70000, 64, 31000
    assert (T - 1) * ld > 2 ** 31
    x = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, E), (ld, 1))
    x.copy_(torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
    for bias in (None, a_bias(E)):
        a, b = (api.moe_route_scored(v, 6, "sigmoid", bias) for v in (x, x.contiguous()))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ri, _, _ = batch64(x.float(), 6, "sigmoid", bias, 1, 1, "max")
        assert torch.equal(a[0], ri.int())


@pytest.mark.gpu
def test_given_outputs_streams_and_replay():
    x = rows(300, 256, 4, torch.float32, 11)
    b = a_bias(256)
    args = dict(scoring="sigmoid", bias=b, n_groups=8, topk_groups=4, group_score="top2", scale=2.5)
    ri, rw = api.moe_route_scored(x, 8, **args)
    # rows past the batch stay as they were
    idx = torch.full((302, 8), 77, dtype=torch.int32, device="cuda")
    w = torch.full((302, 8), -5.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    api.moe_route_scored(x, 8, topk_idx=idx[:300], topk_w=w[:300], stream=s, **args)
    i2, w2 = api.moe_route_scored(x, 8, stream=s, **args)
    s.synchronize()
    assert torch.equal(idx[:300], ri) and torch.equal(w[:300], rw) and torch.equal(i2, ri) and torch.equal(w2, rw)
    assert bool((idx[300:] == 77).all()) and bool((w[300:] == -5.0).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gi, gw = api.moe_route_scored(x, 8, **args)
    x.copy_(rows(300, 256, 0, torch.float32, 12))
    graph.replay()
    torch.cuda.synchronize()
    ni, nw = api.moe_route_scored(x, 8, **args)
    assert torch.equal(gi, ni) and torch.equal(gw, nw) and not torch.equal(ni, ri)


@pytest.mark.gpu
def test_python_refusals():
    x = rows(4, 16)
    for bad in (lambda: api.moe_route_scored(x.t(), 2), lambda: api.moe_route_scored(x.half(), 2),
                lambda: api.moe_route_scored(x, 2, scoring="relu"),
                lambda: api.moe_route_scored(x, 2, bias=torch.zeros(16, device="cuda", dtype=torch.bfloat16)),
                lambda: api.moe_route_scored(x, 2, bias=torch.zeros(16)),
                lambda: api.moe_route_scored(x, 2, topk_idx=torch.zeros(4, 2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: api.moe_route_scored(x, 17), lambda: api.moe_route_scored(x, 2, n_groups=3),
                lambda: api.moe_route_scored(x, 5, n_groups=4, topk_groups=1),
                lambda: api.moe_route_scored(x[:1].expand(4, 16), 2)):
        with pytest.raises(api.MoEError):
            bad()
    i, w = api.moe_route_scored(x[:0], 2)
    assert i.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused():
    # 2^32 + 4 rows are not 4
    x, big = rows(4, 16), torch.empty(2 ** 32 + 4, 1, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: api.moe_route_scored(big, 1), lambda: api.moe_route_scored(x, 2, n_groups=2 ** 32 + 1),
                lambda: api.moe_route_scored(x, 2, n_groups=4, topk_groups=2 ** 32 + 2)):
        with pytest.raises(api.MoEError) as e:
            bad()
        assert e.value.code == 2


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,k", [(64, 8, 3, 8), (120, 4, 2, 16), (160, 8, 3, 6), (256, 8, 4, 8), (512, 16, 4, 8),
                                                    (1024, 32, 4, 30)])
def test_rows_whose_groups_tie_but_for_64_bit_roundings(scoring, E, groups, topk_groups, k):
    """The rows that batch64 leaves open: the choice is that of some set of groups that takes every
    group clearly above the cut and fills up with those at it, and exact within that set."""
    T, n = 20000, E // groups
    g = torch.Generator().manual_seed(E + k)
    bias = ((torch.randn(E, generator=g) * 4).round() / 64).cuda()
    seen = 0
    for logits in ((torch.randn(T, E, generator=g) * 2).round() / 2, torch.randint(0, 2, (T, E), generator=g).float()):
        x = logits.cuda()
        idx, w = api.moe_route_scored(x, k, scoring, bias, groups, topk_groups, "top2", False)
        _, _, open_ = batch64(x, k, scoring, bias, groups, topk_groups, "top2")
        rows_ = open_.nonzero()[:300, 0]
        seen += rows_.numel()
        z = x[rows_].double()
        p = torch.sigmoid(z) if scoring == "sigmoid" else torch.softmax(z, 1)
        c = p + bias.double()
        v = c.view(-1, groups, n).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        for p_, c_, v_, i_, w_ in zip(*(t.cpu().numpy() for t in (p, c, v, idx[rows_], w[rows_].double()))):
            cut = np.sort(v_)[-topk_groups]
            above = [h for h in range(groups) if v_[h] > cut + 2.0 ** -49]
            at = [h for h in range(groups) if abs(v_[h] - cut) <= 2.0 ** -49]
            assert len(above) < topk_groups <= len(above) + len(at)
            found = False
            for more in itertools.combinations(at, topk_groups - len(above)):
                kept = np.isin(np.arange(E) // n, above + list(more))
                want = np.argsort(-np.where(kept, c_, -np.inf), kind="stable")[:k]
                found = found or np.array_equal(want, i_)
            assert found, (i_, v_)
            # as in the test of every choice
            assert np.all(np.abs(w_ - p_[i_]) <= 2.0 ** -24 * (60 + 4 + 60 + 4 + 37 + 4) * p_[i_])
    assert seen > 0
