"""Calls in front of the layer as programs make them: several at once on streams of their own, captured and replayed,
two graphs on one workspace, very many rows, buffers in the wrong place (needs an MI355X)."""
import numpy as np
import pytest
import torch

import front_reference as ref
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def linear_weights(N, K, fmt="mxfp4"):
    codes, scales, zeros, ts, _ = ref.weights(fmt, N, K, np.random.default_rng(N + K))
    return moe.LinearWeights(dev(codes), dev(scales), fmt, dev(zeros), dev(ts))


def calls(T):
    """name -> (call, inputs): call(*inputs) enqueues one operator and returns its outputs."""
    norm = moe.RmsNorm((1 + 0.1 * rand(1056)).to(DEV))
    rule = moe.RouteRule(4, "sigmoid", (0.1 * rand(96)).to(DEV), 8, 3, n_shared=1)
    router = (0.05 * rand(96, 512)).to(DEV)
    W = {f: linear_weights(384, 2048, f) for f in ("mxfp4", "int4g32", "nvfp4")}
    x = lambda w, s: rand(T, w, seed=s).bfloat16().to(DEV)
    r = {"norm": (lambda a, b: moe.moe_add_rms_norm(a, norm, b, mx="fp8"), (x(1056, 1), x(1056, 2))),
         "select": (lambda a: moe.moe_select_experts(a, rule, want_scores=True), (x(96, 3),)),
         "route": (lambda a: moe.moe_route_grouped(a, router, rule, want_scores=True), (x(512, 4),))}
    for f, w in W.items():
        r["linear " + f] = (lambda a, w=w: (moe.moe_linear(a, w),), (x(2048, 5),))
    return r


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # (bits: a random scale may overflow)


@pytest.mark.parametrize("T", [1, 3, 24, 200])
def test_at_once_on_streams_of_their_own(T):
    """Every operator eight times on each of three streams together, on the same inputs and weights."""
    c = calls(T)
    want = {k: f(*a) for k, (f, a) in c.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                got += [(k, f(*a)) for k, (f, a) in c.items()]
    torch.cuda.synchronize()
    for k, g in got:
        same(g, want[k])


@pytest.mark.parametrize("T", [1, 4, 24, 48, 200])
def test_each_call_in_a_graph(T):
    """One call captured, replayed on new inputs with eager work and synchronisations between the replays."""
    for k, (f, a) in calls(T).items():
        note(f"graph of {k} T={T}")
        f(*a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f(*a)
        torch.cuda.synchronize()
        for i in range(4):
            for j, v in enumerate(a):
                v.copy_(rand(*v.shape, seed=10 * i + j).bfloat16())
            g.replay()
            want = f(*a)
            torch.cuda.synchronize()
            same(out, want)


def test_two_graphs_on_one_workspace():
    """Products that share K over workgroups, captured twice with one workspace and replayed in turn."""
    T, W = 150, linear_weights(384, 16384)
    ws = torch.empty(moe.moe_linear_workspace_bytes(T, W), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    xs = [rand(T, 16384, seed=s).bfloat16().to(DEV) for s in (1, 2)]
    outs = [torch.zeros(T, 384, device=DEV) for _ in xs]
    moe.moe_linear(xs[0], W, out=outs[0], workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for x, y in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_linear(x, W, out=y, workspace=ws)
        graphs.append(g)
    want = [moe.moe_linear(x, W) for x in xs]
    for _ in range(3):
        for y in outs:
            y.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        same(outs, want)


def test_one_tensor_as_both_terms():
    X = rand(5, 1000).to(DEV)
    norm = moe.RmsNorm(torch.ones(1000, device=DEV))
    a = moe.moe_add_rms_norm(X, norm, X)
    b = moe.moe_add_rms_norm(X, norm, X.clone())
    same(a[:2], b[:2])


@pytest.mark.parametrize("H,in_place", [(32, False), (32, True), (9, True)])
def test_more_rows_than_a_launch(H, in_place):
    T = (1 << 20) + 3
    note(f"norm T={T} H={H}")
    X = torch.randn(T, H, device=DEV).bfloat16()
    R = torch.randn(T, H, device=DEV).bfloat16()
    wt = torch.rand(H, device=DEV) + 0.5
    s = X.double() + R.double()
    want = s * wt.double() / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6)
    mx = "fp8" if H % 32 == 0 else None
    Y = torch.empty(T, H, device=DEV)
    codes = torch.empty(T, H, dtype=torch.uint8, device=DEV) if mx else None
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV) if mx else None
    RO = R if in_place else torch.empty_like(R)
    moe.moe_add_rms_norm(X, moe.RmsNorm(wt), R, mx=mx, out=(Y, RO, codes, scales))
    # fp32 throughout: at most 9 additions one after another and 6 of a tree, each term off by 3 * 2^-24; the root
    # halves them; division, root and two products 5 more
    assert bool(((Y.double() - want).abs() <= want.abs() * 40 * 2.0 ** -24).all())
    assert bool(((RO.double() - s).abs() <= s.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    if mx:
        tail = slice(T - 5, T)
        ref.check_mx(want[tail].cpu().numpy(), codes[tail].cpu().numpy(), scales[tail].cpu().numpy(), mx, 40 * 2.0 ** -24)


def test_buffers_in_the_wrong_place_are_refused():
    """An output or workspace in host memory, which the library could not tell from its pointer."""
    T = 200
    X = rand(T, 64).bfloat16().to(DEV)
    norm = moe.RmsNorm(torch.ones(64, device=DEV))
    y, u8 = torch.empty(T, 64), lambda *s: torch.empty(*s, dtype=torch.uint8)
    g = torch.empty(T, 64, device=DEV)
    for bad in (dict(norm=moe.RmsNorm(torch.ones(64))), dict(norm=norm, residual=X.cpu()),
                dict(norm=norm, out=(y, None, None, None)),
                dict(norm=norm, residual=X, out=(g, X.cpu(), None, None)),
                dict(norm=norm, mx="fp8", out=(g, None, u8(T, 64), u8(T, 2).to(DEV))),
                dict(norm=norm, mx="fp8", out=(g, None, u8(T, 64).to(DEV), u8(T, 2)))):
        with pytest.raises(ValueError):
            moe.moe_add_rms_norm(X, **bad)
    rule, w = moe.RouteRule(2), torch.zeros(16, 64, device=DEV)
    ids, wt = torch.empty(T, 2, dtype=torch.int32), torch.empty(T, 2)
    for out in ((ids, wt.to(DEV), None), (ids.to(DEV), wt, None), (ids.to(DEV), wt.to(DEV), torch.empty(T, 64))):
        with pytest.raises(ValueError):
            moe.moe_select_experts(X, rule, out=out)
        with pytest.raises(ValueError):
            moe.moe_route_grouped(X, w, rule, out=out)
    with pytest.raises(ValueError):
        moe.moe_select_experts(X, moe.RouteRule(2, selection_bias=torch.zeros(64)))
    with pytest.raises(ValueError):
        moe.moe_route_grouped(X, w.cpu(), rule)
    with pytest.raises(ValueError):
        moe.moe_route_grouped(X, w, rule, workspace=u8(1 << 20))
    W = linear_weights(32, 64)
    codes, scales = W.tensors[:2]
    for bad in (dict(W=moe.LinearWeights(codes.cpu(), scales.cpu())), dict(W=W, bias=torch.zeros(32)),
                dict(W=W, out=torch.empty(T, 32)), dict(W=W, workspace=u8(1 << 20)),
                dict(W=W, workspace=torch.empty(1 << 18, device=DEV))):
        with pytest.raises(ValueError):
            moe.moe_linear(X, **bad)
    with pytest.raises(ValueError):
        moe.LinearWeights(codes, scales.cpu())


@pytest.mark.parametrize("T", [1, 20, 100])
def test_weights_past_32_bits(T):
    """More than 2^31 bytes of codes: the last rows."""
    N, K = (1 << 18) + 21, 16384
    note(f"linear T={T} N={N} K={K}")
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((N, K // 32), 120, dtype=torch.uint8, device=DEV)
    codes.zero_()
    codes[-24:] = torch.randint(0, 256, (24, K // 2), dtype=torch.uint8, generator=torch.Generator().manual_seed(2)).to(DEV)
    x = rand(T, K, seed=3).bfloat16()
    y = moe.moe_linear(x.to(DEV), moe.LinearWeights(codes, scales))
    c = codes[-24:].cpu().numpy()
    w = ref.E2M1[np.stack([c & 15, c >> 4], 2).reshape(24, K)] * 2.0 ** -7
    x = x.double().numpy()
    want = x @ w.T
    assert np.all(np.abs(y[:, -24:].double().cpu().numpy() - want) <= ref.linear_tolerance(x, w, K, want, "fp32"))
    assert not bool(y[:, :-24].any())


def test_rows_past_32_bits():
    """Rows whose offsets pass 2^32 values: a product's x and y, logits, and a norm's x, residual and outputs."""
    T, far = 1040, (1 << 22) + 8
    buf = torch.empty(T * far, dtype=torch.bfloat16, device=DEV).view(T, far)
    x = rand(T, 512, seed=1).bfloat16().to(DEV)
    wide = buf[:, :512].copy_(x)
    W = linear_weights(96, 512)
    out = buf[:, 1024:1120]
    for t in (T, 48, 1):
        same((moe.moe_linear(wide[T - t:], W, out=out[T - t:]).contiguous(),),
             (moe.moe_linear(x[T - t:], W, dtype=torch.bfloat16),))
    rule = moe.RouteRule(8, "sigmoid", n_groups=8, topk_groups=4)
    same(moe.moe_select_experts(wide, rule, want_scores=True), moe.moe_select_experts(x, rule, want_scores=True))
    norm = moe.RmsNorm(torch.rand(512, device=DEV))
    a = moe.moe_add_rms_norm(wide, norm, wide, out=(torch.empty_like(x), buf[:, 2048:2560], None, None))
    same([v.contiguous() for v in a[:2]], moe.moe_add_rms_norm(x, norm, x)[:2])
