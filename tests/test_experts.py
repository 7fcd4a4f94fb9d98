"""moe_experts (and its fp8 and MX forms): the experts' products on a given routing, against the
formula in 64 bits and against the routed forwards; and the scored router, the dense product and
the experts together, as one layer."""
import ctypes

import numpy as np
import pytest
import torch

from routed_grouped_gemm_softmax_b200 import api, build


def test_host_refusals():
    build.build()
    L = api.lib()
    buf = ctypes.create_string_buffer(8192)
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    d = api.dims(4, 512, 512, 8, 2)
    b = ctypes.byref
    for dtype in (0, 1, 2):
        n = L.moe_experts_workspace_size(b(d), dtype)
        assert 0 < n and n % 1024 == 0
    assert L.moe_experts_workspace_size(b(d), 3) == 0
    assert L.moe_experts_workspace_size(b(api.dims(4, 512, 512, 8, 9)), 0) == 0
    assert L.moe_experts_workspace_size(b(api.dims(4, 256, 512, 8, 2)), 2) == 0
    forms = [(L.moe_experts, 3), (L.moe_experts_fp8, 6), (L.moe_experts_mx, 6)]
    for fn, nw in forms:
        big = 1 << 40
        good = [b(d), p, p, p] + [p] * nw + [p, p, 1024, None]
        assert fn(*good) == 3                                   # a workspace that is too small
        assert fn(*(good[:-3] + [p + 16, big, None])) == 3      # ... or misaligned
        assert fn(*(good[:-3] + [None, big, None])) == 3
        for i in range(1, 5 + nw):                              # every pointer is needed
            assert fn(*(good[:i] + [None] + good[i + 1:])) == 1, i
        assert fn(*(good[:1] + [p + 8] + good[2:])) == 1
        assert fn(*(good[:2] + [p + 2] + good[3:])) == 1 and fn(*(good[:3] + [p + 2] + good[4:])) == 1
        assert fn(*([None] + good[1:])) == 1
        assert fn(*([b(api.dims(4, 512, 512, 8, 0))] + good[1:])) == 1
        assert fn(*([b(api.dims(0, 512, 512, 8, 2))] + [None] * (len(good) - 3) + [0, None])) == 0


def test_sizes_past_32_bits_are_refused():
    build.build()
    for at in range(5):
        sizes = [4, 512, 512, 8, 2]
        sizes[at] += 1 << 32  # 4 tokens, 8 experts and so on, were they wrapped
        for call in (lambda: api.dims(*sizes), lambda: api.experts_workspace(*sizes, device="cpu")):
            with pytest.raises(api.MoEError) as e:
                call()
            assert e.value.code == 2


def test_a_workspace_is_contiguous_memory_of_the_device():
    cpu = torch.device("cpu")
    api._need_ws(torch.zeros(64, dtype=torch.uint8), cpu)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(64), torch.zeros(8, dtype=torch.uint8).expand(8, 8),
               torch.zeros(128, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            api._need_ws(ws, cpu)
    with pytest.raises(ValueError):
        api._need_ws(torch.zeros(64, dtype=torch.uint8, device="meta"), cpu)


def rnd(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def weights(E, H, I):
    return rnd((E, I, H), 2, H ** -0.5), rnd((E, I, H), 3, H ** -0.5), rnd((E, H, I), 4, I ** -0.5)


def routing(T, E, k, seed=5, empty=0.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)  # an expert may come twice
    idx[torch.rand(T, k, generator=g) < empty] = -1
    return idx.cuda(), torch.randn(T, k, generator=g).cuda()


def check(out, x, idx, w, w_gate, w_up, w_down, eps_h=2.0 ** -8):
    H, E, I = x.shape[1], w_gate.shape[0], w_gate.shape[1]
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(y)
    eps = 2.0 ** -8  # one rounding to bf16
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        X = x[t].double()
        a, u = X @ w_gate[e].double().T, X @ w_up[e].double().T
        # fp32 sums of H exact products in any order, truncated: at most H steps of 2^-23 of the magnitudes
        da = H * 2.0 ** -23 * (X.abs() @ w_gate[e].double().abs().T)
        du = H * 2.0 ** -23 * (X.abs() @ w_up[e].double().abs().T)
        s = a / (1 + torch.exp(-a))
        # silu: slope at most 1.1, __expf within 2 + 1.17 |a| units in the last place, a division
        ds = 1.1 * da + (8 + 2 * a.abs()) * 2.0 ** -23 * s.abs()
        h = s * u
        dh = ds * u.abs() + s.abs() * du + ds * du + 2.0 ** -24 * h.abs()
        dh = dh + eps_h * (h.abs() + dh)
        D = w_down[e].double().T
        g = w[t, j].double()[:, None]
        y.index_add_(0, t, g * (h @ D))
        err.index_add_(0, t, g.abs() * (dh @ D.abs() + I * 2.0 ** -23 * ((h.abs() + dh) @ D.abs())))
        err.index_add_(0, t, (idx.shape[1] + 1) * 2.0 ** -24 * (g * (h @ D)).abs())
    tol = err * (1 + eps) + eps * y.abs()
    d = (out.double() - y).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


SHAPES = [(1, 64, 64, 1, 1), (1, 256, 128, 8, 2), (3, 128, 192, 5, 5), (16, 512, 256, 64, 8), (33, 192, 64, 60, 4),
          (64, 256, 512, 8, 2), (300, 320, 128, 16, 3), (640, 256, 128, 4, 2), (2100, 128, 128, 2, 2), (40, 64, 64, 300, 12)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
@pytest.mark.parametrize("empty", [0.0, 0.4, 1.0])
def test_against_64_bits(T, H, I, E, k, empty):
    x, W = rnd((T, H), 1), weights(E, H, I)
    idx, w = routing(T, E, k, empty=empty)
    w[idx < 0] = float("nan")  # an empty slot's weight is not read into the sum
    # whatever the workspace held before
    ws = api.experts_workspace(T, H, I, E, k, "cuda").fill_(0xFF)
    out = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        api.moe_experts(x, idx, w, *W, out=out[:T], ws=ws)
        assert api.moe_get_device_status(ws) == api.MOE_OK
        check(out[:T], x, idx, w, *W)
        assert bool((out[T] == 7.0).all())
    gone = (idx < 0).all(1)
    assert bool((out[:T][gone] == 0).all())


# lists on both sides of what one block groups (4096 entries, 376 experts), tiles whose last rows fill part of a warp, and
# groups of hundreds of rows
MORE = [(512, 128, 64, 16, 8), (513, 128, 64, 16, 8), (300, 64, 64, 376, 3), (300, 64, 64, 377, 3), (400, 192, 320, 4, 4),
        (700, 256, 64, 3, 3), (1, 2048, 512, 64, 6), (1, 64, 64, 8, 1), (4, 192, 320, 8, 2), (30, 448, 192, 16, 2), (200, 320, 1024, 2, 1),
        (1200, 64, 1024, 48, 8), (2000, 192, 640, 30, 10), (1000, 320, 1088, 31, 8), (95, 64, 64, 1, 1), (3100, 64, 192, 4, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", MORE)
@pytest.mark.parametrize("skew", [False, True])
def test_groups_of_any_size(T, H, I, E, k, skew):
    x, W = rnd((T, H), 1), weights(E, H, I)
    idx, w = routing(T, E, k, empty=0.1)
    if skew:  # most rows with one expert
        hot = torch.rand(T, k, generator=torch.Generator().manual_seed(8)).cuda() < 0.8
        idx[hot & (idx >= 0)] = E // 2
    ws = api.experts_workspace(T, H, I, E, k, "cuda").fill_(0x7F)
    out = api.moe_experts(x, idx, w, *W, ws=ws)
    assert api.moe_get_device_status(ws) == api.MOE_OK
    check(out, x, idx, w, *W)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 17, 130, 600])
def test_a_chain_of_launches_sees_what_the_last_one_wrote(T):
    """Routing and experts on one workspace, one after the other with nothing between: each call's
    experts take the routing of the call just before."""
    H, I, E, k, n = 256, 128, 32, 4, 6
    W = weights(E, H, I)
    xs, logits = [rnd((T, H), 30 + i) for i in range(n)], [rnd((T, E), 40 + i, 2.0, torch.float32) for i in range(n)]
    ws = api.experts_workspace(T, H, I, E, k, "cuda")
    idx, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")

    def chain():
        outs = []
        for x, l in zip(xs, logits):
            api.moe_route_scored(l, k, topk_idx=idx, topk_w=w)
            outs.append(api.moe_experts(x, idx, w, *W, ws=ws))
        return outs

    want = []
    for x, l in zip(xs, logits):
        i, v = api.moe_route_scored(l, k)
        torch.cuda.synchronize()
        want.append(api.moe_experts(x, i, v, *W))
        torch.cuda.synchronize()
        check(want[-1], x, i, v, *W)
    for _ in range(3):
        for a, b in zip(chain(), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 400])
def test_kernel_choices_agree(T):
    x, W = rnd((T, 256), 1), weights(8, 256, 128)
    idx, w = routing(T, 8, 4, empty=0.2)
    ref = api.moe_experts(x, idx, w, *W)
    check(ref, x, idx, w, *W)
    try:
        for name, modes in (("set_layer_gemm", ("always", "never")), ("set_direct_a", ("always", "never")),
                            ("set_fused_combine", ("always",)), ("set_pair_mma", ("always",))):
            for m in modes:
                getattr(api, name)(m)
                check(api.moe_experts(x, idx, w, *W), x, idx, w, *W)
                getattr(api, name)("auto")
    finally:
        for name in ("set_layer_gemm", "set_direct_a", "set_fused_combine", "set_pair_mma"):
            getattr(api, name)("auto")



# up to 64 assignments h is two bf16 parts: its own rounding leaves at most 2^-8 of it, and the
# rounding of that 2^-8 of the rest
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 8), (64, 128, 64, 3, 1), (16, 320, 192, 8, 4), (8, 64, 1088, 60, 8),
                                       (63, 192, 2048, 1, 1), (32, 2048, 64, 16, 2), (2, 64, 4096, 64, 32)])
@pytest.mark.parametrize("one", [False, True])
def test_h_of_few_rows_in_two_parts(T, H, I, E, k, one):
    x, W = rnd((T, H), 1), weights(E, H, I)
    idx, w = routing(T, E, k, empty=0.1)
    if one:  # a tile of all the rows
        idx.fill_(E - 1)
    ws = api.experts_workspace(T, H, I, E, k, "cuda").fill_(0xFF)
    try:
        for layer in ("auto", "always"):
            for direct in ("auto", "always", "never"):
                api.set_layer_gemm(layer)
                api.set_direct_a(direct)
                out = api.moe_experts(x, idx, w, *W, ws=ws)
                assert api.moe_get_device_status(ws) == api.MOE_OK
                check(out, x, idx, w, *W, eps_h=2.0 ** -16)
    finally:
        api.set_layer_gemm("auto")
        api.set_direct_a("auto")


@pytest.mark.parametrize("H,I,E,k", [(256, 128, 8, 1), (128, 4096, 300, 1), (2048, 512, 64, 3)])
def test_a_batch_s_workspace_serves_smaller_ones(H, I, E, k):
    build.build()
    sizes = [api.lib().moe_experts_workspace_size(ctypes.byref(api.dims(T, H, I, E, k)), 0) for T in range(1, 300)]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 65])
def test_infinite_h_stays_infinite(T):
    H = I = 64
    x = torch.full((T, H), 1e20, dtype=torch.bfloat16, device="cuda")
    x[1] = float("nan")
    ones = torch.ones(1, 64, 64, dtype=torch.bfloat16, device="cuda")
    idx, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    out = api.moe_experts(x, idx, w, ones, ones, ones)
    assert bool(out[1].isnan().all()) and bool((out[0] == float("inf")).all()) and bool((out[2:] == float("inf")).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 400])
def test_indices_outside_are_flagged_and_skipped(T):
    x, W = rnd((T, 256), 1), weights(8, 256, 128)
    idx, w = routing(T, 8, 4, empty=0.1)
    bad = idx.clone()
    bad[3, 1], bad[7, 0], bad[T - 1, 3] = 8, -2, 2 ** 31 - 1
    ws = api.experts_workspace(T, 256, 128, 8, 4, "cuda")
    out = api.moe_experts(x, bad, w, *W, ws=ws)
    assert api.moe_get_device_status(ws) == 6
    check(out, x, torch.where((bad < 0) | (bad >= 8), -1, bad), w, *W)
    api.moe_experts(x, idx, w, *W, ws=ws)
    assert api.moe_get_device_status(ws) == api.MOE_OK


@pytest.mark.gpu
def test_indices_outside_of_a_long_list():
    T = 1500  # more entries than one block groups
    x, W = rnd((T, 256), 1), weights(8, 256, 128)
    idx, w = routing(T, 8, 4, empty=0.1)
    bad = idx.clone()
    bad[3, 1], bad[1207, 0], bad[T - 1, 3] = 8, -2, 2 ** 31 - 1
    ws = api.experts_workspace(T, 256, 128, 8, 4, "cuda").fill_(0xFF)
    for _ in range(2):
        out = api.moe_experts(x, bad, w, *W, ws=ws)
        assert api.moe_get_device_status(ws) == 6
        check(out, x, torch.where((bad < 0) | (bad >= 8), -1, bad), w, *W)
        out = api.moe_experts(x, idx, w, *W, ws=ws)
        assert api.moe_get_device_status(ws) == api.MOE_OK
        check(out, x, idx, w, *W)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 9, 120, 1500])
def test_any_number_of_blocks_gives_the_same(T):
    x, W = rnd((T, 256), 1), weights(8, 256, 192)
    idx, w = routing(T, 8, 4, empty=0.1)
    ref = api.moe_experts(x, idx, w, *W)
    check(ref, x, idx, w, *W)
    try:
        for n in (1, 3, 40):
            api.set_gemm_ctas(n)
            assert torch.equal(ref, api.moe_experts(x, idx, w, *W))
    finally:
        api.set_gemm_ctas(0)


@pytest.mark.gpu
def test_streams_and_replay():
    T, H, I, E, k = 100, 256, 128, 16, 4
    x, W = rnd((T, H), 1), weights(E, H, I)
    idx, w = routing(T, E, k, empty=0.2)
    ref = api.moe_experts(x, idx, w, *W)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [api.moe_experts(x, idx, w, *W, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(ref, o) for o in outs)
    ws = api.experts_workspace(T, H, I, E, k, "cuda")
    out = torch.empty_like(ref)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            api.moe_experts(x, idx, w, *W, out=out, ws=ws)
    idx.copy_(routing(T, E, k, seed=9, empty=0.5)[0])
    for g in graphs:
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        check(out, x, idx, w, *W)


def quantised(kind, E, H, I):
    g = torch.Generator(device="cuda").manual_seed(8)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
    if kind == "fp8":
        codes = lambda *s: torch.where((byte(*s) & 0x7F) == 0x7F, 0, byte(*s) & 0xBF)  # |value| < 2, never NaN
        scale = lambda *s: torch.rand(*s, generator=g, device="cuda") * 0.02 + 0.01
        return (codes(E, I, H), scale(E, I // 128, H // 128), codes(E, I, H), scale(E, I // 128, H // 128),
                codes(E, H, I), scale(E, H // 128, I // 128))
    x8 = lambda *s: torch.full(s, 127 - 6, dtype=torch.uint8, device="cuda")
    return (byte(E, I, H // 2), x8(E, I, H // 32), byte(E, I, H // 2), x8(E, I, H // 32), byte(E, H, I // 2), x8(E, H, I // 32))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp8", "mx"])
@pytest.mark.parametrize("T", [1, 24, 70, 500])
def test_quantised_forms_follow_the_routed_forwards(kind, T):
    H, I, E, k = 512, 512, 8, 2
    x, W = rnd((T, H), 1), quantised(kind, E, H, I)
    rw = rnd((H, E), 7, 0.05)
    idx, w = api.moe_route(x, rw, None, k)
    ref = getattr(api, f"moe_forward_{kind}")(x, rw, None, *W, k)
    fn = getattr(api, f"moe_experts_{kind}")
    out = fn(x, idx, w, *W)
    assert bool(torch.isfinite(ref.float()).all()) and float(ref.float().abs().max()) > 0
    assert torch.equal(out, ref)  # the same kernels and sums on the same routing
    # a slot without an expert is a slot of weight 0
    gone = torch.rand(T, k, generator=torch.Generator().manual_seed(3)).cuda() < 0.4
    ws = api.experts_workspace(T, H, I, E, k, "cuda", {"fp8": 1, "mx": 2}[kind]).fill_(0xFF)
    some = fn(x, torch.where(gone, -1, idx), torch.where(gone, float("nan"), w), *W, ws=ws)
    assert api.moe_get_device_status(ws) == api.MOE_OK
    assert torch.equal(some, fn(x, idx, torch.where(gone, 0.0, w), *W))
    none = fn(x, torch.full_like(idx, -1), w, *W, ws=ws)
    assert bool((none == 0).all())


@pytest.mark.gpu
def test_python_refusals():
    x, W = rnd((4, 64), 1), weights(4, 64, 64)
    idx, w = routing(4, 4, 2)
    for bad in (lambda: api.moe_experts(x.float(), idx, w, *W), lambda: api.moe_experts(x, idx.long(), w, *W),
                lambda: api.moe_experts(x, idx, w.bfloat16(), *W), lambda: api.moe_experts(x, idx[:3], w, *W),
                lambda: api.moe_experts(x, idx, w[:, :1], *W), lambda: api.moe_experts(x, idx, w, W[0], W[1], W[0][:, :32]),
                lambda: api.moe_experts(x.cpu(), idx, w, *W), lambda: api.moe_experts(x, idx.cpu(), w, *W),
                lambda: api.moe_experts(x[:, ::2], idx, w, *W)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(api.MoEError):
        api.moe_experts(x, idx, w, *W, ws=torch.zeros(1024, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 333])
def test_a_layer_of_scored_router_experts_and_shared_dense(T):
    """Router logits, group-limited sigmoid routing, the experts, and a dense gated half added to
    them, captured as one graph: every stage against 64 bits on the inputs that it had."""
    from test_linear import check as check_linear
    from test_route_scored import oracle as route_oracle
    H, I, E, k, S = 256, 128, 32, 4, 200
    x, W = rnd((T, H), 1), weights(E, H, I)
    rw = rnd((E, H), 11, H ** -0.5)
    bias = rnd((E,), 12, 0.05, torch.float32)
    sg, su, sd = rnd((S, H), 13, H ** -0.5), rnd((S, H), 14, H ** -0.5), rnd((H, S), 15, S ** -0.5)
    lws, ews = api.linear_workspace("cuda"), api.experts_workspace(T, H, I, E, k, "cuda")

    def layer():
        logits = api.moe_linear(x, rw, out_dtype=torch.float32, ws=lws)
        idx, w = api.moe_route_scored(logits, k, "sigmoid", bias, 8, 3, "top2", True, 2.5)
        routed = api.moe_experts(x, idx, w, *W, ws=ews)
        h = api.moe_linear(x, sg, act="silu", w_up=su, ws=lws)
        return logits, idx, w, routed, h, api.moe_linear(h, sd, residual=routed, ws=lws)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    x.copy_(rnd((T, H), 21))
    graph.replay()
    torch.cuda.synchronize()
    logits, idx, w, routed, h, out = got
    assert torch.equal(logits, check_linear(x, rw, out_dtype=torch.float32))
    ri, rwt = route_oracle(logits.cpu().numpy(), k, "sigmoid", bias.cpu().numpy(), 8, 3, "top2", True, 2.5)
    assert np.array_equal(idx.cpu().numpy(), ri) and np.allclose(w.cpu().numpy(), rwt, rtol=1e-5, atol=0)
    check(routed, x, idx, w, *W)
    assert torch.equal(h, check_linear(x, sg, act="silu", w_up=su))
    assert torch.equal(out, check_linear(h, sd, residual=routed))
    assert api.moe_get_device_status(ews) == api.MOE_OK and api.moe_get_device_status(lws) == api.MOE_OK
    for a, b in zip(layer(), got):
        assert torch.equal(a, b)


# each form of the experts' GEMM: rows of gate and of up an item, K chunks a stage, parts of h
FORMS = {"32 rows, h in two parts": (1, 2048, 512, 64, 6), "64 rows, two parts": (8, 256, 512, 64, 8),
         "128 rows, two parts": (16, 256, 1024, 64, 4), "32 rows": (9, 256, 128, 8, 8), "64 rows": (40, 256, 512, 64, 8),
         "128 rows, rows gathered from x": (80, 256, 1024, 64, 8), "128 rows, two chunks": (160, 256, 1024, 64, 8),
         "128 rows, one chunk": (1024, 256, 1024, 64, 4), "pairs": (1600, 256, 128, 2, 1)}


@pytest.mark.gpu
@pytest.mark.parametrize("form", list(FORMS))
def test_down_items_read_the_h_of_their_own_call(form):
    """Calls of different inputs on one workspace, nothing between them: a down item that read h
    before it saw the other blocks' stores would find the rows of the call before."""
    T, H, I, E, k = FORMS[form]
    W = weights(E, H, I)
    idx, w = routing(T, E, k, empty=0.1)
    xs = [rnd((T, H), 60 + i) for i in range(3)]
    want = []
    for x in xs:
        want.append(api.moe_experts(x, idx, w, *W))
        torch.cuda.synchronize()
        check(want[-1], x, idx, w, *W)
    ws = api.experts_workspace(T, H, I, E, k, "cuda")
    outs = [api.moe_experts(xs[i % 3], idx, w, *W, ws=ws) for i in range(60)]
    assert api.moe_get_device_status(ws) == api.MOE_OK
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 3]), i


@pytest.mark.gpu
def test_workspaces_that_repeat_memory_are_refused():
    from test_linear import operands
    x, W = rnd((4, 64), 1), weights(4, 64, 64)
    idx, w = routing(4, 4, 2)
    ws = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 24)
    y, v, _ = operands(4, 16, 32)
    for bad in (lambda: api.moe_experts(x, idx, w, *W, ws=ws), lambda: api.moe_experts(x, idx, w, *W, ws=ws[:1].cpu()),
                lambda: api.moe_linear(y, v, ws=ws), lambda: api.moe_linear(y, v, ws=ws[:1].cpu())):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.gpu
@pytest.mark.parametrize("form", [f for f in FORMS if f != "pairs"])  # their MMA warp has no stall hook
def test_a_wait_that_runs_out_is_reported_and_recoverable(form):
    # the MMA warps wait 20 ms for what never comes: every role unwinds behind its own copies, and the
    # next call on the same workspace has the result of an undisturbed one
    T, H, I, E, k = FORMS[form]
    x, W = rnd((T, H), 1), weights(E, H, I)
    idx, w = routing(T, E, k, empty=0.1)
    ws = api.experts_workspace(T, H, I, E, k, "cuda")
    ref = api.moe_experts(x, idx, w, *W, ws=ws)
    assert api.moe_get_device_status(ws) == api.MOE_OK
    check(ref, x, idx, w, *W)
    api.set_wait_limit_us(20000, stall_test=True)
    try:
        api.moe_experts(x, idx, w, *W, ws=ws)
        assert api.moe_get_device_status(ws) == 5
    finally:
        api.set_wait_limit_us(0)
    assert torch.equal(ref, api.moe_experts(x, idx, w, *W, ws=ws))
    assert api.moe_get_device_status(ws) == api.MOE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 8), (16, 320, 192, 8, 4), (8, 64, 1088, 60, 8), (64, 128, 64, 3, 1)])
def test_few_rows_by_the_other_kernels_round_h_once(T, H, I, E, k):
    x, W = rnd((T, H), 1), weights(E, H, I)
    idx, w = routing(T, E, k, empty=0.1)
    ws = api.experts_workspace(T, H, I, E, k, "cuda").fill_(0xFF)
    for name, mode in (("set_layer_gemm", "never"), ("set_pair_mma", "always")):
        for direct in ("always", "never"):
            try:
                getattr(api, name)(mode)
                api.set_direct_a(direct)
                out = api.moe_experts(x, idx, w, *W, ws=ws)
                assert api.moe_get_device_status(ws) == api.MOE_OK
                check(out, x, idx, w, *W)  # eps_h: one rounding
            finally:
                getattr(api, name)("auto")
                api.set_direct_a("auto")


@pytest.mark.gpu
@pytest.mark.parametrize("H,I,E,k", [(320, 192, 16, 8), (512, 1024, 64, 8)])
def test_a_token_s_bits_depend_on_its_company_only_through_h(H, I, E, k):
    # batches of up to 64 assignments agree among themselves and larger ones do, whatever kernels their sizes choose
    n = 900 * E // k  # pair tiles at the end
    x, W = rnd((n, H), 1), weights(E, H, I)
    g = torch.Generator().manual_seed(5)
    idx = torch.rand(n, E, generator=g).argsort(1)[:, :k].int().cuda()
    w = torch.randn(n, k, generator=g).cuda()
    few = 64 // k
    small = api.moe_experts(x[:few], idx[:few], w[:few], *W)
    for T in range(1, few):
        assert torch.equal(api.moe_experts(x[:T], idx[:T], w[:T], *W), small[:T]), T
    large = api.moe_experts(x, idx, w, *W)
    for T in (few + 1, 2 * few, 5 * few, 20 * few, 100 * few, n // 10, n // 3):
        assert torch.equal(api.moe_experts(x[:T], idx[:T], w[:T], *W), large[:T]), T


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(270000, 2048, 64, 4, 4), (270000, 64, 2048, 4, 4)])
@pytest.mark.parametrize("pair", ["auto", "never"])
def test_offsets_past_32_bits(T, H, I, E, k, pair):
    # y or h of more than 2^31 elements
    assert T * k * max(H, I) > 2 ** 31
    x, W = rnd((T, H), 1), weights(E, H, I)
    g = torch.Generator().manual_seed(5)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].int()
    idx[torch.rand(T, k, generator=g) < 0.01] = -1
    idx, w = idx.cuda(), torch.randn(T, k, generator=g).cuda()
    ws = api.experts_workspace(T, H, I, E, k, "cuda")
    try:
        api.set_pair_mma(pair)
        out = api.moe_experts(x, idx, w, *W, ws=ws)
    finally:
        api.set_pair_mma("auto")
    assert api.moe_get_device_status(ws) == api.MOE_OK
    del ws
    some = torch.cat([torch.arange(300), T - 1 - torch.arange(300), torch.randint(0, T, (2000,), generator=g)]).cuda()
    check(out[some], x[some], idx[some], w[some], *W)


# lists that one block groups and longer ones, experts on both sides of what it takes, several sizes
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp8", "mx"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 1024, 512, 16, 8), (33, 512, 1024, 60, 5), (1200, 1024, 512, 8, 4), (4100, 512, 512, 3, 1),
                                       (300, 512, 512, 376, 2), (300, 512, 512, 400, 2)])
def test_quantised_forms_at_other_sizes(kind, T, H, I, E, k):
    x, W = rnd((T, H), 1), quantised(kind, E, H, I)
    rw = rnd((H, E), 7, 0.05)
    idx, w = api.moe_route(x, rw, None, k)
    ref = getattr(api, f"moe_forward_{kind}")(x, rw, None, *W, k)
    fn = getattr(api, f"moe_experts_{kind}")
    ws = api.experts_workspace(T, H, I, E, k, "cuda", {"fp8": 1, "mx": 2}[kind]).fill_(0xFF)
    assert torch.equal(fn(x, idx, w, *W, ws=ws), ref) and bool((ref != 0).any())
    g = torch.Generator().manual_seed(3)
    gone = torch.rand(T, k, generator=g).cuda() < 0.4
    want = fn(x, idx, torch.where(gone, 0.0, w), *W)
    for bad in (-1, E):
        some = fn(x, torch.where(gone, bad, idx), torch.where(gone, float("nan"), w), *W, ws=ws)
        assert api.moe_get_device_status(ws) == (6 if bad == E and bool(gone.any()) else api.MOE_OK)
        assert torch.equal(some, want)


@pytest.mark.gpu
def test_calls_from_two_threads():
    # each thread with a stream, inputs and workspaces of its own; the library's own state is shared
    import threading
    from test_linear import operands
    from test_route_scored import rows
    cases = []
    for n, (T, H, I, E, k) in enumerate([(5, 256, 128, 16, 4), (200, 320, 192, 8, 2), (1000, 256, 128, 32, 4)]):
        W = weights(E, H, I)
        idx, w = routing(T, E, k, seed=n, empty=0.1)
        cases.append((rows(T, E, 0, torch.float32, n), rnd((T, H), n), idx, w, W, k, operands(T, 300 + 1000 * n, 256)))

    def run(c, stream=None, ews=None, lws=None):
        logits, x, idx, w, W, k, (a, b, u) = c
        return (*api.moe_route_scored(logits, k, "sigmoid", stream=stream), api.moe_experts(x, idx, w, *W, ws=ews, stream=stream),
                api.moe_linear(a, b, act="silu", w_up=u, ws=lws, stream=stream))

    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(order):
        try:
            s = torch.cuda.Stream()
            lws = api.linear_workspace("cuda", s)
            ews = [api.experts_workspace(c[1].shape[0], c[1].shape[1], c[4][0].shape[1], c[4][0].shape[0], c[5], "cuda", stream=s)
                   for c in cases]
            got = []
            for _ in range(30):
                got += [(i, run(cases[i], s, ews[i], lws)) for i in order]
            s.synchronize()
            assert api.moe_get_device_status(lws, s) == api.MOE_OK
            for i, outs in got:
                assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), i
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(o,)) for o in ((0, 1, 2), (2, 1, 0), (1, 2, 0))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


FIRST_CALL = """
import sys, torch
from routed_grouped_gemm_softmax_b200 import api
which, T = sys.argv[1], int(sys.argv[2])
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda")
logits, x = r(T, 16), r(T, 256).bfloat16()
W = [(r(*s) / 16).bfloat16() for s in ((16, 128, 256), (16, 128, 256), (16, 256, 128))]
idx, w, a, b = torch.randint(0, 16, (T, 4), generator=g, device="cuda").int(), r(T, 4), r(T, 256).bfloat16(), r(2100, 256).bfloat16()
call = {"route": lambda: api.moe_route_scored(logits, 4, "sigmoid"), "experts": lambda: (api.moe_experts(x, idx, w, *W),),
        "linear": lambda: (api.moe_linear(a, b, act="gelu"),), "linear gated": lambda: (api.moe_linear(a, b, w_up=b),)}[which]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
for o in got:
    o.zero_()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(o, v) and bool((o != 0).any()) for o, v in zip(got, call()))
print("the same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["route", "experts", "linear", "linear gated"])
def test_the_first_call_of_a_process_may_be_captured(which):
    import subprocess
    import sys
    from conftest import ROOT
    for T in (3, 700):
        p = subprocess.run([sys.executable, "-c", FIRST_CALL, which, str(T)], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert p.returncode == 0 and "the same" in p.stdout, p.stderr[-2000:]


@pytest.mark.gpu
def test_an_empty_batch():
    x, W = rnd((4, 64), 1), weights(4, 64, 64)
    idx, w = routing(4, 4, 2)
    assert api.moe_experts(x[:0], idx[:0], w[:0], *W).shape == (0, 64)
