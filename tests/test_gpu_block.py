"""The MoE half of a decoder block run as a user runs it (MoEBlock: projection, residual addition + norm, routing by
a rule, bucketing, expert FFN, combine), step by step against 64 bits and the oracle, in the exact and the MX
mode, eager and from captured graphs (needs an MI355X).  Every step is checked on the inputs that the GPU's
previous step gave it, with that step's own tolerance."""
import numpy as np
import pytest
import torch

import front_reference as ref
import oracle
import synth
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, EXACT_TOL, expert_weights, note, require_gpu, rms_ratio

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def make(T, mx=None, fmt_o="mxfp4", K_o=512, bias=None, seed=21):
    H, E, k, S, I = 512, 32, 4, 1, 256
    wl = synth.custom(hidden=H, n_routed=E, top_k=k, n_shared=S, inter=I, router_std=0.05)
    L = synth.make_layer(wl, T, seed=seed)
    t = synth.to_torch(L, DEV)
    rng = np.random.default_rng(seed)
    codes, scales, zeros, ts, w_o = ref.weights(fmt_o, H, K_o, rng)
    if fmt_o == "mxfp4":
        scales = rng.integers(118, 122, scales.shape).astype(np.uint8)
        c = np.stack([codes & 15, codes >> 4], 2).reshape(H, K_o)
        w_o = ref.E2M1[c] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
    W_o = moe.LinearWeights(dev(codes), dev(scales), fmt_o, dev(zeros), dev(ts))
    b = bias if bias is not None else (0.02 * rng.standard_normal(E)).astype(np.float32)
    args = dict(score="sigmoid", n_groups=4, topk_groups=2, group_score="top2", renormalise=True, routed_scale=2.5,
                n_shared=S)
    rule = moe.RouteRule(k, selection_bias=dev(b), **args)
    wn = (1 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    block = moe.MoEBlock(expert_weights(t), T, rule, t["router"], moe.RmsNorm(dev(wn)), W_o, mx)
    attn = torch.from_numpy(rng.standard_normal((T, K_o))).bfloat16().to(DEV)
    res = torch.from_numpy(rng.standard_normal((T, H))).bfloat16().to(DEV)
    return L, block, attn, res, w_o, wn, b, args


def check_steps(L, block, attn, res, w_o, wn, b, args, y, r):
    f = lambda v: v.detach().double().cpu().numpy()
    T, H = L.T, L.wl.hidden
    a = f(block.a)
    want = f(attn) @ w_o.T
    assert np.all(np.abs(a - want) <= ref.linear_tolerance(f(attn), w_o, w_o.shape[1], want, "fp32"))
    s, x = ref.add_rms_norm(a, f(res), wn, 1e-6)
    rel = (H / 256 + 80) * 2.0 ** -24
    assert np.all(np.abs(f(r) - s) <= np.abs(s) * (2.0 ** -8 + 2.0 ** -23))
    assert np.all(np.abs(f(block.x) - x) <= np.abs(x) * (2.0 ** -8 + 2 * rel))
    if block.mx is not None:
        ref.check_mx(x, block.codes.cpu().numpy(), block.scales.cpu().numpy(),
                     {v: k for k, v in moe.MX_FORMATS.items()}[block.mx], rel)
    logits = f(block.x) @ L.router.astype(np.float64).T
    ids, w, sc = ref.select(logits, block.rule.top_k, bias=b, **args)
    got = block.ids.cpu().numpy()
    per = logits.shape[1] // args["n_groups"]
    key = sc + b
    flagged = 0
    for t in range(T):  # a choice that differs has to lie within the logits' fp32 rounding (1e-5 of a key)
        if not np.array_equal(got[t], ids[t]):
            flagged += 1
            d = np.abs(np.sort(key[t, got[t, :4]]) - np.sort(key[t, ids[t, :4]]))
            part = np.sort(key[t].reshape(-1, per), 1)
            rank = np.sort(part[:, -1] + part[:, -2])
            assert d.max() <= 1e-5 or rank[-2] - rank[-3] <= 1e-5
    assert flagged <= max(1, T // 50)
    same = np.all(got == ids, 1)
    assert np.max(np.abs(f(block.weights)[same] - w[same])) <= 2.5e-5
    if block.mx is None:
        orc = oracle.load()
        E2, kt = L.wl.n_experts, block.k_total
        bk = orc.bucket(got.astype(np.int32), E2)
        xb = block.x.view(torch.int16).cpu().numpy().view(np.uint16)
        ys = orc.expert_ffn(xb, oracle.X_BF16, kt, oracle.ExpertWeights.from_layer(L), bk["offsets"], bk["sorted_slot"])
        err = rms_ratio(f(y), orc.combine(ys, f(block.weights).astype(np.float32)))
        note(f"  block output: max-abs / rms = {err:.2e}")
        assert err <= EXACT_TOL


@pytest.mark.parametrize("T", [1, 7, 40, 130])
@pytest.mark.parametrize("fmt_o", ["mxfp4", "int4g32", "nvfp4"])
def test_block(T, fmt_o):
    note(f"block T={T} {fmt_o}")
    m = make(T, None, fmt_o)
    block, attn, res = m[1:4]
    if fmt_o == "nvfp4":
        attn *= 2.0 ** -10  # its random scales are large
    y, r = block.forward(attn, res)
    torch.cuda.synchronize()
    check_steps(*m, y, r)


@pytest.mark.parametrize("T", [1, 40, 130])
@pytest.mark.parametrize("mx", ["fp8", "fp6", "fp4"])
def test_block_mx(T, mx):
    """The norm's codes feed the MX expert FFN; the FFN on codes equals its own quantisation bit for bit."""
    note(f"block T={T} mx={mx}")
    m = make(T, mx)
    L, block, attn, res = m[:4]
    y, r = block.forward(attn, res)
    torch.cuda.synchronize()
    check_steps(*m, y, r)
    off, ss, kt = block.buckets.offsets, block.buckets.sorted_slot, block.k_total
    direct = moe.moe_expert_ffn_mx(block.x, block.W, mx, off, ss, kt)
    codes, scales = moe.moe_mx_quantize(block.x, mx)
    given = moe.moe_expert_ffn_mx_codes(codes, scales, block.W, mx, off, ss, kt)
    assert torch.equal(direct, given)
    ys = moe.moe_expert_ffn_mx_codes(block.codes, block.scales, block.W, mx, off, ss, kt)
    assert torch.equal(moe.moe_combine(ys, block.weights), y)
    rel = float((y - moe.moe_combine(direct, block.weights)).norm() / y.norm())
    # two roundings to the element type of the same values, at most half a step each and both of the block's x and
    # h: the outputs differ by less than the coarsest format's quantisation itself
    assert rel <= {"fp8": 2.0 ** -4, "fp6": 2.0 ** -4, "fp4": 2.0 ** -2}[mx]


@pytest.mark.parametrize("mx", [None, "fp8"])
@pytest.mark.parametrize("T", [1, 40, 150])
def test_block_in_a_graph(T, mx):
    """One captured pass replayed with new inputs, with eager work of another block and synchronisations between
    the replays: every replay equals the eager pass bit for bit."""
    L, block, attn, res, *_ = make(T, mx)
    other = make(T, mx, seed=5)
    r = torch.empty_like(res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(attn, res, r)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _ = block.forward(attn, res, r)
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(1)
    for _ in range(4):
        attn.copy_(torch.randn(attn.shape, generator=gen).bfloat16())
        res.copy_(torch.randn(res.shape, generator=gen).bfloat16())
        g.replay()
        other[1].forward(other[2], other[3])
        torch.cuda.synchronize()
        got = [v.clone() for v in (y, r, block.x, block.ids, block.weights)]
        y2, r2 = block.forward(attn, res)
        torch.cuda.synchronize()
        for u, v in zip(got, (y2, r2, block.x, block.ids, block.weights)):
            assert torch.equal(u, v)


def test_two_blocks_in_turn():
    """A block's fp32 output joins the residual stream in the next block's norm, in place."""
    a, b = make(9), make(9, seed=5)
    y1, r = a[1].forward(a[2], a[3], a[3])
    assert r is a[3]
    b[1].W_o = None  # y1 goes to the norm directly
    y2, r2 = b[1].forward(y1, r, r)
    torch.cuda.synchronize()
    assert r2 is r and bool(torch.isfinite(y2).all())
    s, x = ref.add_rms_norm(y1.double().cpu().numpy(), np.zeros((9, 512)), b[5], 1e-6)
    assert x.shape == (9, 512)


def test_masked_experts_leave_slots_empty():
    """A bias of -inf leaves fewer experts than slots: the empty slots add nothing, also after passes that left
    NaN in their rows."""
    E = 32
    bias = np.full(E, -np.inf, np.float32)
    bias[[2, 9, 30]] = 0.1
    L, block, attn, res, *_ = make(6, bias=bias)
    assert block.clear
    block.y_slots.fill_(float("nan"))
    y, _ = block.forward(attn, res)
    torch.cuda.synchronize()
    ids = block.ids.cpu().numpy()
    assert set(np.unique(ids[:, :4])) <= {-1, 2, 9, 30} and np.all((ids[:, :4] == -1).sum(1) >= 1)
    assert np.all(block.weights.cpu().numpy()[ids == -1] == 0) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("mx", [None, "fp8"])
def test_slots_that_logits_leave_empty(mx):
    """Logits of -inf leave a token with fewer experts than slots, or none: choice, buckets, FFN and combine give
    what its experts alone give, whatever the slots' rows hold."""
    T, kt = 9, 4
    L, block, *_ = make(T, mx)
    W, x = block.W, torch.randn(T, 512, device=DEV).bfloat16()
    logits = torch.randn(T, 32, device=DEV)
    logits[1, 3:] = -float("inf")
    logits[4] = -float("inf")
    logits[7, 1:] = float("nan")
    ids, w, _ = moe.moe_select_experts(logits, moe.RouteRule(kt, "sigmoid"))
    b = moe.moe_bucket(ids, W.n_experts)

    def ffn(fill):
        ys = torch.full((T * kt, 512), fill, device=DEV)
        if mx:
            moe.moe_expert_ffn_mx(x, W, mx, b.offsets, b.sorted_slot, kt, out=ys)
        else:
            moe.moe_expert_ffn(x, W, b.offsets, b.sorted_slot, kt, out=ys)
        return ys

    want = moe.moe_combine(ffn(0.0), w)
    assert (ids == -1).sum(1).tolist() == [0, 1, 0, 0, 4, 0, 0, 3, 0] and not bool(want[4].any())
    assert bool(torch.isfinite(want).all()) and bool(want[[1, 7]].any(1).all())
    for fill in (float("nan"), float("inf"), -3.0):
        assert torch.equal(moe.moe_combine(ffn(fill), w), want)


def test_empty_slots_in_restored_sums():
    """moe_combine_restore, likewise: a slot of weight 0 adds nothing, whatever its row holds."""
    T, kt, H = 3, 4, 64
    g = torch.Generator().manual_seed(3)
    ys = torch.randn(T * kt, H, generator=g).half().to(DEV)
    w = torch.rand(T, kt, generator=g).to(DEV)
    w[0, 2] = w[1, :] = 0.0
    rows = torch.tensor([2, 4, 5, 6, 7], device=DEV)
    ys[rows] = 0.0
    want = moe.moe_combine_restore(ys, w, 2)
    for fill in (float("nan"), float("inf")):
        ys[rows] = fill
        assert torch.equal(moe.moe_combine_restore(ys, w, 2), want)


def test_a_token_that_is_not_finite_depends_on_no_earlier_pass():
    """A token of NaN has no expert to go to: its output is the same after any earlier pass, and no other token's
    output changes."""
    T = 6
    L, block, attn, res, *_ = make(T)
    y0, _ = block.forward(attn, res)
    y0 = y0.clone()
    bad = res.clone()
    bad[2, 5] = float("nan")
    seen = []
    for fill in (0.0, float("nan"), 7.0):
        block.y_slots.fill_(fill)
        y, r = block.forward(attn, bad)
        assert (block.ids[2, :4] == -1).all() and bool(torch.isnan(r[2, 5]))
        seen.append(y.clone())
    keep = [0, 1, 3, 4, 5]
    for y in seen:
        assert torch.equal(y[keep], y0[keep])
        assert torch.equal(y[2].view(torch.int32), seen[0][2].view(torch.int32))


def test_the_next_block_adds_the_output():
    """Two blocks in turn, in place: the second block's residual is the first one's plus its output, and what it
    routes is the norm of that sum."""
    a, b = make(9), make(9, seed=5)
    y1, r = a[1].forward(a[2], a[3], a[3])
    before, y1 = r.clone(), y1.clone()
    b[1].W_o = None
    y2, r2 = b[1].forward(y1, r, r)
    torch.cuda.synchronize()
    f = lambda v: v.double().cpu().numpy()
    s, x = ref.add_rms_norm(f(y1), f(before), b[5], 1e-6)
    rel = (512 / 256 + 80) * 2.0 ** -24  # as derived for the norm: its fp32 steps
    assert np.all(np.abs(f(r2) - s) <= np.abs(s) * (2.0 ** -8 + 2.0 ** -23))
    assert np.all(np.abs(f(b[1].x) - x) <= np.abs(x) * (2.0 ** -8 + 2 * rel))
    orc, block = oracle.load(), b[1]
    bk = orc.bucket(block.ids.cpu().numpy(), b[0].wl.n_experts)
    xb = block.x.view(torch.int16).cpu().numpy().view(np.uint16)
    ys = orc.expert_ffn(xb, oracle.X_BF16, block.k_total, oracle.ExpertWeights.from_layer(b[0]), bk["offsets"],
                        bk["sorted_slot"])
    assert rms_ratio(f(y2), orc.combine(ys, block.weights.cpu().numpy())) <= EXACT_TOL


@pytest.mark.parametrize("mx", [None, "fp8"])
@pytest.mark.parametrize("T", [1, 40])
def test_no_token_has_an_expert(T, mx):
    """Every slot empty: the FFN has no row to compute, and the combine gives zeros."""
    W = make(1, mx)[1].W
    x = torch.randn(T, 512, device=DEV).bfloat16()
    ids, w, _ = moe.moe_select_experts(torch.full((T, 32), -float("inf"), device=DEV), moe.RouteRule(4))
    b = moe.moe_bucket(ids, W.n_experts)
    ys = torch.full((T * 4, 512), float("nan"), device=DEV)
    if mx:
        moe.moe_expert_ffn_mx(x, W, mx, b.offsets, b.sorted_slot, 4, out=ys)
    else:
        moe.moe_expert_ffn(x, W, b.offsets, b.sorted_slot, 4, out=ys)
    y = moe.moe_combine(ys, w)
    assert bool((ids == -1).all()) and not bool(y.any())
