"""The calls in front of the layer on the host: every documented refusal, with fake device pointers that validation
never dereferences, and the binding's own checks (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import front_reference as ref
import mxfp4_routed_expert_router_amd as m

OK, NULL, SHAPE, BLOCK, ALIGN, DTYPE, TOPK, WORKSPACE = 0, 1, 2, 3, 4, 5, 6, 7
P = 0x7F0000000000


def fake(off=0):
    return ctypes.c_void_p(P + off)


def rule(**k):
    d = dict(score=0, top_k=2, n_shared=0, n_groups=1, topk_groups=1, group_score=0, renormalise=1, routed_scale=1.0,
             shared_weight=1.0, selection_bias=None)
    d.update(k)
    return m.moe_route_rule(*(d[f] for f, _ in m.moe_route_rule._fields_))


def test_select_refusals():
    L = m.lib()
    keys = ("logits", "dt", "stride", "T", "E", "ids", "w", "sc")

    def s(**k):
        a = dict(logits=fake(), dt=2, stride=64, T=4, E=64, ids=fake(64), w=fake(128), sc=None)
        a.update({x: k.pop(x) for x in keys if x in k})
        r = ctypes.byref(rule(**k)) if k.pop("rule", 1) is not None else None
        return L.moe_select_experts(a["logits"], a["dt"], a["stride"], a["T"], a["E"], r, a["ids"], a["w"], a["sc"], None)

    assert L.moe_select_experts(None, 9, 0, 0, 0, None, None, None, None, None) == OK  # T = 0
    assert L.moe_select_experts(fake(), 2, 64, 4, 64, None, fake(), fake(), None, None) == NULL
    for name in ("logits", "ids", "w"):
        assert s(**{name: None}) == NULL
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, stride=1025), dict(n_shared=-1), dict(stride=63), dict(n_groups=0),
                dict(n_groups=65, E=65, stride=65), dict(n_groups=5), dict(n_groups=8, topk_groups=0),
                dict(n_groups=8, topk_groups=9), dict(routed_scale=float("nan")), dict(shared_weight=float("inf")),
                dict(stride=1 << 62), dict(T=(1 << 25) + 1, E=8, stride=8)):
        assert s(**bad) == SHAPE, bad
    for bad in (dict(top_k=0), dict(top_k=65), dict(n_groups=8, topk_groups=2, top_k=17), dict(top_k=60, n_shared=200),
                dict(n_shared=2 ** 31 - 1)):
        assert s(**bad) == TOPK, bad
    for bad in (dict(dt=3), dict(dt=-1), dict(score=2), dict(group_score=2)):
        assert s(**bad) == DTYPE, bad
    for bad in (dict(logits=fake(2)), dict(dt=0, logits=fake(1)), dict(ids=fake(2)), dict(w=fake(1)), dict(sc=fake(3)),
                dict(selection_bias=P + 2)):
        assert s(**bad) == ALIGN, bad


def test_route_grouped_refusals():
    L = m.lib()
    need = L.moe_route_workspace_bytes(4, 64, 64)

    def r(x=fake(), xdt=0, T=4, H=64, w=fake(256), E=64, ids=fake(64), wt=fake(128), ws=fake(1024), wsb=need, **k):
        return L.moe_route_grouped(x, xdt, T, H, w, E, ctypes.byref(rule(**k)), ids, wt, None, ws, wsb, None)

    assert L.moe_route_grouped(None, 0, 0, 0, None, 0, None, None, None, None, None, 0, None) == OK
    assert r(x=None) == NULL and r(w=None) == NULL and r(ids=None) == NULL and r(wt=None) == NULL
    assert L.moe_route_grouped(fake(), 0, 4, 64, fake(), 64, None, fake(), fake(), None, fake(), need, None) == NULL
    assert r(H=0) == SHAPE and r(T=-2) == SHAPE and r(n_groups=7) == SHAPE
    assert r(xdt=2) == DTYPE and r(top_k=0) == TOPK
    assert r(x=fake(8)) == ALIGN and r(w=fake(2)) == ALIGN and r(ws=fake(8)) == ALIGN
    assert r(ws=None) == WORKSPACE and r(wsb=need - 1) == WORKSPACE


def test_norm_refusals():
    L = m.lib()

    def n(w=P, wdt=2, H=64, eps=1e-6, x=fake(), xdt=0, xs=64, res=fake(256), rdt=0, rs=64, T=4, ro=fake(512), ros=64,
          y=fake(1024), ydt=0, fmt=0, codes=None, scales=None, norm=True):
        c = m.moe_norm(w, wdt, H, eps)
        return L.moe_add_rms_norm(ctypes.byref(c) if norm else None, x, xdt, xs, res, rdt, rs, T, ro, ros, y, ydt, fmt,
                                  codes, scales, None)

    mx = dict(fmt=1, codes=fake(2048), scales=fake(4096))
    assert L.moe_add_rms_norm(None, None, 0, 0, None, 0, 0, 0, None, 0, None, 0, 0, None, None, None) == OK
    for bad in (dict(norm=False), dict(w=None), dict(x=None), dict(res=None), dict(y=None),
                dict(mx, codes=None), dict(mx, scales=None), dict(codes=fake(2048)), dict(scales=fake(2048))):
        assert n(**bad) == NULL, bad
    for bad in (dict(T=-1), dict(H=0), dict(xs=63), dict(rs=63), dict(ros=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(xs=1 << 62), dict(ro=fake(256), ros=72)):
        assert n(**bad) == SHAPE, bad
    assert n(**dict(mx, H=48, xs=48, rs=48, ros=48)) == BLOCK
    for bad in (dict(xdt=3), dict(rdt=3), dict(ydt=-1), dict(wdt=7), dict(mx, fmt=4), dict(mx, fmt=-1)):
        assert n(**bad) == DTYPE, bad
    for bad in (dict(x=fake(1)), dict(xdt=2, x=fake(2)), dict(res=fake(1)), dict(ro=fake(1)), dict(y=fake(1)),
                dict(ydt=2, y=fake(2)), dict(w=P + 2), dict(mx, codes=fake(8))):
        assert n(**bad) == ALIGN, bad


def linear_desc(fmt=m.MOE_W_MXFP4, N=32, K=64, **over):
    d = m.moe_linear_weights()
    d.fmt, d.n_out, d.k_in = fmt, N, K
    d.w.w, d.w.w_row_stride = P, K // 2
    d.w.scales = P + 0x1000
    d.w.s_row_stride = K // 32 if fmt == m.MOE_W_MXFP4 else K // 16
    if fmt == m.MOE_W_INT4_G32:
        d.w.zeros, d.w.z_row_stride = P + 0x2000, (K // 32 + 1) // 2
    if fmt == m.MOE_W_NVFP4:
        d.w.tensor_scale = P + 0x3000
    for k, v in over.items():
        setattr(d.w if k not in ("fmt", "n_out", "k_in") else d, k, v)
    return d


@pytest.mark.parametrize("fmt", [m.MOE_W_MXFP4, m.MOE_W_INT4_G32, m.MOE_W_NVFP4])
def test_linear_refusals(fmt):
    L = m.lib()

    def f(d=None, x=fake(), xdt=0, xs=64, T=4, bias=None, y=fake(0x5000), ydt=2, ys=32, ws=fake(0x8000), wsb=None):
        d = linear_desc(fmt) if d is None else d
        need = L.moe_linear_workspace_bytes(T, ctypes.byref(d))
        return L.moe_linear(x, xdt, xs, T, ctypes.byref(d), bias, y, ydt, ys, ws, need if wsb is None else wsb, None)

    D = lambda **k: linear_desc(**{"fmt": fmt, **k})
    assert L.moe_linear(None, 0, 0, 0, None, None, None, 0, 0, None, 0, None) == OK
    assert L.moe_linear(fake(), 0, 64, 4, None, None, fake(), 2, 32, None, 0, None) == NULL
    assert f(x=None) == NULL and f(y=None) == NULL and f(D(w=None)) == NULL and f(D(scales=None)) == NULL
    for bad in (dict(T=-1), dict(xs=56), dict(ys=31), dict(xs=1 << 62), dict(xs=1 << 23), dict(ys=1 << 62),
                dict(d=D(s_row_stride=1 << 24)), dict(d=D(n_out=0)), dict(d=D(k_in=0)),
                dict(d=D(n_out=(1 << 26) + 1), ys=1 << 27), dict(T=(1 << 30) + 1), dict(T=(1 << 31) - 1),
                dict(d=D(w_row_stride=16)), dict(d=D(s_row_stride=1)), dict(d=D(w_row_stride=1 << 24))):
        assert f(**bad) == SHAPE, bad
    assert f(D(k_in=48)) == BLOCK and f(D(w=P + 8)) == BLOCK and f(D(w_row_stride=40)) == BLOCK
    assert f(xdt=1) == DTYPE and f(ydt=3) == DTYPE and f(D(fmt=m.MOE_W_FP16)) == DTYPE and f(D(fmt=9)) == DTYPE
    assert f(x=fake(8)) == ALIGN and f(xs=68) == ALIGN and f(y=fake(0x5002)) == ALIGN and f(bias=fake(2)) == ALIGN
    if fmt == m.MOE_W_INT4_G32:
        assert f(D(zeros=None)) == NULL and f(D(z_row_stride=0)) == SHAPE
    if fmt == m.MOE_W_NVFP4:
        assert f(D(tensor_scale=None)) == NULL and f(D(tensor_scale=P + 2)) == ALIGN
    assert L.moe_linear_workspace_bytes(4, ctypes.byref(D())) == 0
    # K = 16384 is shared over workgroups, which takes a workspace
    wide = D(k_in=16384, w_row_stride=8192, s_row_stride=1024,
             **({"z_row_stride": 256} if fmt == m.MOE_W_INT4_G32 else {}))
    need = L.moe_linear_workspace_bytes(200, ctypes.byref(wide))
    assert need >= 4 * 200 * 32
    assert f(wide, T=200, xs=16384, ws=None) == WORKSPACE and f(wide, T=200, xs=16384, wsb=need - 1) == WORKSPACE
    assert f(wide, T=200, xs=16384, ws=fake(0x8008)) == ALIGN
    assert L.moe_linear_workspace_bytes(4, None) == 0 and L.moe_linear_workspace_bytes(0, ctypes.byref(D())) == 0


def test_ffn_mx_codes_refusals():
    L = m.lib()
    W = m.moe_expert_weights()
    W.fmt, W.n_experts, W.hidden, W.inter = m.MOE_W_MXFP4, 4, 256, 512
    for name, (N, K) in (("gate", (512, 256)), ("up", (512, 256)), ("down", (256, 512))):
        p = getattr(W, name)
        p.w, p.scales = P + 0x10000, P + 0x20000
        p.w_row_stride, p.w_expert_stride = K // 2, N * K // 2
        p.s_row_stride, p.s_expert_stride = K // 32, N * K // 32
    need = L.moe_expert_ffn_mx_workspace_bytes(4, 2, ctypes.byref(W), 1)

    def f(xc=fake(), xs=fake(256), T=4, kt=2, fmt=1, off=fake(512), y=fake(1024), ws=fake(4096), wsb=need):
        return L.moe_expert_ffn_mx_codes(xc, xs, T, kt, ctypes.byref(W), fmt, off, fake(768), y, ws, wsb, None)

    assert L.moe_expert_ffn_mx_codes(None, None, 0, 2, None, 1, None, None, None, None, 0, None) == OK
    assert f(xc=None) == NULL and f(xs=None) == NULL and f(off=None) == NULL and f(y=None) == NULL
    assert f(T=-1) == SHAPE and f(kt=0) == SHAPE and f(fmt=0) == DTYPE
    assert f(xc=fake(8)) == ALIGN and f(xs=fake(2)) == ALIGN and f(ws=fake(8)) == ALIGN
    assert f(ws=None) == WORKSPACE and f(wsb=need - 1) == WORKSPACE


def test_binding_refuses_what_it_can_see():
    """Shapes, types and devices that the C call could not tell from its pointers."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    norm = m.RmsNorm(torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        m.moe_add_rms_norm(x, norm)
    for bad in (dict(x=x[:, :32], norm=norm), dict(x=x.t().contiguous().t(), norm=norm),
                dict(x=x, norm=norm, residual=x[:3]), dict(x=x, norm=norm, residual=x[:, :32]),
                dict(x=x, norm=norm, out=(x, x, None, None)), dict(x=x, norm=norm, out=(x[:2], None, None, None)),
                dict(x=x, norm=norm, residual=x, out=(x, x.float(), None, None)),
                dict(x=x, norm=norm, mx="fp8", out=(x, None, torch.zeros(4, 32, dtype=torch.uint8), None))):
        with pytest.raises((ValueError, AttributeError)):
            m.moe_add_rms_norm(**bad)
    with pytest.raises(TypeError):
        m.RmsNorm(torch.ones(64, dtype=torch.float64))
    with pytest.raises(KeyError):
        m.RouteRule(2, "tanh")
    with pytest.raises(ValueError):
        m.RouteRule(2, selection_bias=torch.zeros(8, dtype=torch.float64))
    r = m.RouteRule(2, selection_bias=torch.zeros(8))
    lg = torch.zeros(4, 16)
    for bad in (dict(logits=lg, rule=r), dict(logits=lg.t(), rule=m.RouteRule(2)),
                dict(logits=lg, rule=m.RouteRule(2), out=(torch.zeros(4, 2), torch.zeros(4, 2), None)),
                dict(logits=lg, rule=m.RouteRule(2))):
        with pytest.raises(ValueError):
            m.moe_select_experts(**bad)
    codes, scales, _, _, _ = ref.weights("mxfp4", 8, 64, np.random.default_rng(0))
    codes, scales = torch.from_numpy(codes), torch.from_numpy(scales)
    W = m.LinearWeights(codes, scales)
    assert (W.n_out, W.k_in) == (8, 64)
    for bad in (dict(scales=scales[:4]), dict(scales=scales, fmt="nvfp4"), dict(scales=scales, fmt="int4g32"),
                dict(scales=scales.int())):
        with pytest.raises(ValueError):
            m.LinearWeights(codes, **bad)
    for bad in (dict(x=x[:, :32]), dict(x=x, bias=torch.zeros(7)), dict(x=x, out=torch.zeros(4, 9)),
                dict(x=x, out=torch.zeros(3, 8)), dict(x=x)):
        with pytest.raises(ValueError):
            m.moe_linear(W=W, **bad)
    with pytest.raises(ValueError):
        m.moe_expert_ffn_mx_codes(codes, scales, type("W", (), {"hidden": 256})(), "fp8", None, None, 2)


def test_reference_forms():
    """The tests' own references: element tables against torch's types, code packing round trips, and a check that
    a planted mistake fails."""
    v = ref.element_values("fp8")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v[np.isfinite(v)], t[np.isfinite(t)]) and np.isnan(t[np.isnan(v)]).all()
    assert ref.element_values("fp6").max() == 7.5 and np.array_equal(np.sort(ref.element_values("fp4")), np.sort(ref.E2M1))
    rng = np.random.default_rng(0)
    y = rng.standard_normal((3, 64))
    sc = np.floor(np.log2(np.abs(y).reshape(3, 2, 32).max(2))).astype(int) - 8 + 127
    q = y / np.repeat(2.0 ** (sc - 127.0), 32, 1)
    codes = torch.from_numpy(np.clip(q, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ref.check_mx(y, codes, sc.astype(np.uint8), "fp8", 1e-6)
    wrong = codes.copy()
    wrong[1, 5] ^= 1
    with pytest.raises(AssertionError):
        ref.check_mx(y, wrong, sc.astype(np.uint8), "fp8", 1e-6)
    ids, w, s = ref.select(np.array([[0.0, 2.0, 1.0, 3.0]]), 2, "softmax", np.array([0, 0, 0, -np.inf], np.float32))
    assert ids.tolist() == [[1, 2]] and abs(w.sum() - 1) < 1e-12 and abs(s.sum() - 1) < 1e-12
