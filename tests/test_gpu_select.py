"""Routing by a rule (moe_select_experts, moe_route_grouped) on the GPU against extended precision (needs an
MI355X).  ids have to be equal: the choice is that of the exact keys.

Tolerances.  A score is off by at most (16 + VPL + |d|) * 2^-24 relative with VPL <= 32 experts per lane and
exponents |d| <= 104 (beyond it fp32 holds nothing), a renormalised weight by twice that and the sum's log2(256)
additions and two more operations: below 400 * 2^-24 = 2.4e-5 relative; scores below 2^-120 lose bits as
subnormals (absolute 2^-140)."""
import numpy as np
import pytest
import torch

import front_reference as ref
import mxfp4_routed_expert_router_amd as moe
import synth
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RTOL = 400 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def close(got, want):
    assert np.all(np.abs(got - want) <= RTOL * np.abs(want) + 2.0 ** -140), np.max(np.abs(got - want))


def check(L, **rule):
    """L: a CPU tensor of logits, maybe strided."""
    bias = rule.pop("bias", None)
    k = rule.pop("top_k")
    close_ranks = rule.pop("close_ranks", False)
    note(f"select {tuple(L.shape)} {L.dtype} k={k} bias={bias is not None} {rule}")
    ids, w, sc = ref.select(L.double().numpy(), k, bias=None if bias is None else bias.numpy(), **rule)
    r = moe.RouteRule(k, selection_bias=None if bias is None else bias.to(DEV), **rule)
    D = torch.empty_strided(L.shape, L.stride(), dtype=L.dtype, device=DEV).copy_(L)
    gi, gw, gs = moe.moe_select_experts(D, r, want_scores=True)
    gi2, gw2, none = moe.moe_select_experts(D, r)
    torch.cuda.synchronize()
    assert none is None and torch.equal(gi, gi2) and torch.equal(gw, gw2)
    same = np.all(gi.cpu().numpy() == ids, 1)
    if close_ranks and not same.all():
        # Ranks of logits that are neighbours in fp32 differ by as little as s'' d^2 with d near 1e-8, about 1e-17:
        # less than 64 bits hold.  There a score is off by at most 3 * 2^-53, a key (below 2) by another 2^-53, the
        # sum of two (below 4) by 2^-52, so two ranks by at most 2 (2 * 4 + 2) 2^-53 < 2^-48 together.
        gap = ref.rank_gap(L.double().numpy(), rule["score"], None if bias is None else bias.numpy(), rule["n_groups"],
                           rule["topk_groups"])
        note(f"  {int((~same).sum())} rows with ranks closer than 64 bits")
        # (0 where several groups of equal members share the boundary with one that is that close to them)
        assert np.all(gap[~same] <= 2.0 ** -48), gap[~same]
        gi, gw, gs, ids, w, sc = gi[same], gw[same], gs[same], ids[same], w[same], sc[same]
    assert np.array_equal(gi.cpu().numpy(), ids), np.argwhere(gi.cpu().numpy() != ids)[:5]
    close(gw.cpu().numpy().astype(np.float64), w)
    close(gs.cpu().numpy().astype(np.float64), sc)


def logits(T, E, dtype="fp32", seed=0, std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(T, E + pad, generator=g)).to(TYPES[dtype])[:, :E]


def bias_of(E, std=0.02, seed=9):
    return std * torch.randn(E, generator=torch.Generator().manual_seed(seed))


SHAPES = [  # T, E, top_k, n_groups, topk_groups
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 8, 2, 1, 1), (9, 64, 8, 8, 3), (17, 256, 8, 8, 4), (4, 160, 6, 8, 3),
    (6, 100, 5, 4, 2), (3, 512, 10, 16, 4), (2, 1024, 16, 1, 1), (2, 1023, 9, 33, 5), (2, 1024, 12, 64, 9),
    (3, 256, 16, 64, 4), (4, 60, 7, 3, 2), (2, 300, 200, 1, 1), (3, 384, 8, 1, 1), (5, 96, 48, 2, 1), (2, 256, 250, 1, 1)]


@pytest.mark.parametrize("T,E,k,G,keep", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_shapes(T, E, k, G, keep, score, biased):
    for by in ("top2", "max"):
        check(logits(T, E, seed=E), top_k=k, score=score, bias=bias_of(E) if biased else None, n_groups=G,
              topk_groups=keep, group_score=by, renormalise=by == "top2", routed_scale=2.5, n_shared=2 if k < 250 else 0,
              shared_weight=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_types_and_strides(dtype, pad):
    """16-bit logits have many exact ties: the lowest index wins."""
    L = logits(33, 128, dtype, seed=pad, std=0.02 if dtype != "fp32" else 1.0, pad=pad)
    check(L, top_k=8)
    check(L, top_k=8, score="sigmoid", bias=bias_of(128), n_groups=4, topk_groups=2)
    check(L, top_k=8, n_groups=8, topk_groups=3, group_score="max")
    check(L, top_k=8, n_groups=8, topk_groups=3)


def test_exact_ties():
    """Equal keys, equal ranks, zeros of both signs: the lowest index."""
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(64)):
            check(torch.zeros(2, 64), top_k=6, score=score, bias=bias, n_groups=8, topk_groups=4)
            L = torch.zeros(3, 64)
            L[:, ::3] = -0.0
            check(L, top_k=40, score=score, bias=bias)
            L = torch.full((2, 64), -1.0)
            L[:, 5::8] = 1.5
            check(L, top_k=5, score=score, bias=bias, n_groups=8, topk_groups=3, group_score="max")


def test_keys_closer_than_fp32():
    """Keys and ranks that round to the same fp32 value, or in the wrong order, are told apart."""
    g = torch.Generator().manual_seed(4)
    for T in (1, 40):
        base = torch.randn(T, 1, generator=g)
        L = base + torch.randint(-3, 4, (T, 64), generator=g) * 2.0 ** -23 * base.abs()  # neighbours in fp32
        for score in ("softmax", "sigmoid"):
            check(L, top_k=8, score=score, bias=bias_of(64, 1e-9))
            check(L, top_k=8, score=score, bias=torch.full((64,), 0.75), n_groups=8, topk_groups=4, close_ranks=True)
            check(L, top_k=8, score=score, n_groups=8, topk_groups=4, close_ranks=True)
            check(L, top_k=8, score=score)
    L = torch.linspace(17.0, 30.0, 64).repeat(2, 1)  # sigmoid rounds to 1 in fp32 from about 17
    check(L, top_k=12, score="sigmoid")
    check(L, top_k=12, score="sigmoid", bias=torch.zeros(64))


def test_many_close_keys():
    """More close keys than lanes of a wave, around the last slot and among many slots."""
    for dtype in ("bf16", "fp32"):
        L = logits(3, 512, dtype, seed=6, std=0.01 if dtype == "bf16" else 1.0)
        if dtype == "fp32":
            L = L.mul(2.0 ** -22).add(0.75)  # a few hundred neighbours
        for score in ("softmax", "sigmoid"):
            for k in (4, 62, 63, 64, 130):
                check(L, top_k=k, score=score, bias=torch.zeros(512))
            check(L, top_k=9, score=score, bias=torch.full((512,), -0.5), n_groups=4, topk_groups=2, group_score="max")
    same = torch.zeros(2, 256)
    for k in (1, 8, 63, 64, 200):
        check(same, top_k=k, score="sigmoid", bias=torch.full((256,), 0.25))
    check(logits(5, 700, seed=3), top_k=120, score="sigmoid", bias=bias_of(700))
    check(logits(5, 700, seed=3), top_k=120, bias=bias_of(700, 1e-3), n_groups=7, topk_groups=3)


def test_wide_logits():
    """Scores over the whole range of fp32, and keys under a large bias."""
    for std in (5.0, 40.0):
        check(logits(8, 96, seed=2, std=std), top_k=8, renormalise=False)
        check(logits(8, 96, seed=2, std=std).clamp(-80, 80), top_k=8, score="sigmoid", bias=bias_of(96, 10.0), n_groups=6,
              topk_groups=2)
    check(logits(8, 96, seed=2, std=5.0), top_k=8, bias=bias_of(96, 1e4), n_groups=6, topk_groups=2)


def test_masked_experts():
    """Logits that are not finite and a bias of -inf mask experts; slots that stay empty get id -1, weight 0."""
    inf, nan = float("inf"), float("nan")
    L = logits(10, 48, seed=8)
    L[0, 5:] = -inf              # five left
    L[1, :] = -inf               # none left
    L[2, 1:] = -inf              # one left
    L[3, ::2] = nan
    L[4, 0] = inf
    L[5, :24] = -inf             # whole groups masked
    L[6, 8:] = -inf
    L[7, :] = torch.finfo(torch.float32).min  # a mask of the type's lowest value keeps the experts available
    L[8, 4:] = torch.finfo(torch.float32).min
    low = bias_of(48)
    low[::3] = -inf
    for score in ("softmax", "sigmoid"):
        for bias in (None, bias_of(48), low, torch.full((48,), -inf)):
            if score == "sigmoid":
                L2 = L.clone()
                L2[7:9] = L2[7:9].clamp(min=-80.0)  # (e^-L of the lowest value has no place in 64 bits)
            else:
                L2 = L
            check(L2, top_k=8, score=score, bias=bias, n_shared=1)
            for by in ("top2", "max"):
                check(L2, top_k=8, score=score, bias=bias, n_groups=6, topk_groups=2, group_score=by)


def test_lowest_value_sigmoid():
    """Sigmoid of the type's lowest value: score 0, still available, chosen last; weights 0 where all are 0."""
    low = torch.finfo(torch.float32).min
    L = torch.full((2, 16), low)
    L[0, 3] = 1.0
    ids, w, s = moe.moe_select_experts(L.to(DEV), moe.RouteRule(4, "sigmoid"), want_scores=True)
    assert ids.cpu().tolist() == [[3, 0, 1, 2], [0, 1, 2, 3]]
    assert w.cpu().tolist() == [[1.0, 0.0, 0.0, 0.0], [0.0] * 4] and int(torch.count_nonzero(s)) == 1


def test_large_batch_and_nothing_else_written():
    T, E = 3001, 256
    L = logits(T, E, seed=1)
    b = bias_of(E)
    rule = moe.RouteRule(8, "sigmoid", b.to(DEV), 8, 4, "top2", True, 2.5, 1)
    ids = torch.full((T + 2, 9), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T + 2, 9), 77.0, device=DEV)
    sc = torch.full((T + 2, E), 77.0, device=DEV)
    moe.moe_select_experts(L.to(DEV), rule, out=(ids[1:-1], w[1:-1], sc[1:-1]))
    for buf in (ids, w, sc):
        assert bool((buf[0] == 77).all() & (buf[-1] == 77).all())
    some = np.linspace(0, T - 1, 150).astype(int)
    wi, ww, _ = ref.select(L.double().numpy()[some], 8, "sigmoid", b.numpy(), 8, 4, "top2", True, 2.5, 1)
    assert np.array_equal(ids[1:-1].cpu().numpy()[some], wi)
    close(w[1:-1].cpu().numpy()[some].astype(np.float64), ww)
    kept = np.array([len(set(r // 32)) for r in ids[1:-1, :8].cpu().numpy()])
    assert kept.max() <= 4


ROUTES = [(1, 7168, 256, "bf16"), (13, 4096, 128, "bf16"), (176, 7168, 256, "bf16"), (33, 96, 100, "fp16"), (300, 512, 64, "fp16")]


@pytest.mark.parametrize("T,H,E,dt", ROUTES)
def test_route_grouped(T, H, E, dt):
    """From x: the ids of the rule on the 64-bit logits wherever no two compared keys lie within the fp32 logits'
    own rounding, and weights within the routers' 1e-5."""
    wl = synth.custom(hidden=H, n_routed=E, top_k=4, router_std=1.0 / np.sqrt(H), act_dtype=dt,
                      weight_format="mxfp4" if dt == "bf16" else "fp16")
    x = synth.make_x(wl, T, seed=3)
    router, _ = synth.make_router(wl, seed=3)
    xt = torch.from_numpy(x).view(torch.bfloat16 if dt == "bf16" else torch.float16)
    L = xt.double().numpy() @ router.astype(np.float64).T
    b = bias_of(E)
    G = 4
    args = ("sigmoid", b.numpy(), G, 2, "top2", True, 2.5, 1)
    ids, w, sc = ref.select(L, 4, *args)
    rule = moe.RouteRule(4, "sigmoid", b.to(DEV), G, 2, "top2", True, 2.5, 1)
    gi, gw, gs = moe.moe_route_grouped(xt.to(DEV), torch.from_numpy(router).to(DEV), rule, want_scores=True)
    gi, gw, gs = gi.cpu().numpy(), gw.cpu().numpy(), gs.cpu().numpy()
    assert np.max(np.abs(gs - sc)) <= 1e-5
    key = sc + b.numpy()
    part = np.sort(key.reshape(T, G, E // G), 2)
    rank = np.sort(part[:, :, -1] + part[:, :, -2], 1)
    top = np.sort(np.take_along_axis(key, ids[:, :4], 1), 1)
    # the fifth key among the kept groups
    fifth = np.empty(T)
    for t in range(T):
        per = E // G
        order = sorted(range(G), key=lambda g: -(part[t, g, -1] + part[t, g, -2]))[:2]
        fifth[t] = np.sort(np.concatenate([key[t, g * per:(g + 1) * per] for g in order]))[-5]
    gap = np.minimum(np.diff(np.concatenate([fifth[:, None], top], 1), axis=1).min(1), rank[:, -2] - rank[:, -3])
    ok = gap > 1e-5
    assert ok.mean() > 0.8
    assert np.array_equal(gi[ok], ids[ok])
    assert np.max(np.abs(gw[ok] - w[ok])) <= 2.5e-5


def test_matches_the_plain_routers():
    """Without groups the rule chooses what moe_route and moe_route_sigmoid choose (from the same logits)."""
    T, H, E, k = 64, 512, 96, 6
    x = torch.randn(T, H, device=DEV).bfloat16()
    w = torch.randn(E, H, device=DEV) / H ** 0.5
    b = bias_of(E).to(DEV)
    i1, w1, _ = moe.moe_route(x, w, k, None, 2)
    i2, w2, _ = moe.moe_route_grouped(x, w, moe.RouteRule(k, n_shared=2))
    assert torch.equal(i1, i2) and float((w1 - w2).abs().max()) <= 1e-6
    i1, w1, _ = moe.moe_route_sigmoid(x, w, k, b, 1, 2.5, 0.5)
    i2, w2, _ = moe.moe_route_grouped(x, w, moe.RouteRule(k, "sigmoid", b, routed_scale=2.5, n_shared=1, shared_weight=0.5))
    assert float((i1 == i2).float().mean()) > 0.99 and float((w1 - w2).abs().max()) <= 1e-5


def test_empty_batch():
    ids, w, s = moe.moe_select_experts(torch.empty(0, 16, device=DEV), moe.RouteRule(2), want_scores=True)
    assert ids.shape == (0, 2) and s.shape == (0, 16)


def test_ranks_past_fp32():
    """Finite biases near the end of fp32: two of them overflow as a group's rank, which stays a rank (a group with
    available experts comes before one without, and a larger sum before a smaller)."""
    low = float(torch.finfo(torch.float32).min)
    E = 32
    groups = [  # a bias per group of eight
        (-float("inf"), -2e38, -3e38, 0.1), (-float("inf"), low, low, 0.1), (-float("inf"), low, -float("inf"), low),
        (-3e38, -2e38, -float("inf"), low), (1.9e38, 2e38, -low, 0.0), (2e38, 2e38, 1.9e38, -low), (-low, -low, -low, 1.0),
        (1e38, -float("inf"), low, -2e38)]
    for score in ("softmax", "sigmoid"):
        for per_group in groups:
            bias = torch.tensor(per_group).repeat_interleave(8)
            for keep in (1, 2, 3):
                for by in ("top2", "max"):
                    check(logits(3, E, seed=7), top_k=6, score=score, bias=bias, n_groups=4, topk_groups=keep,
                          group_score=by)
        mixed = torch.tensor([2e38, -2e38] + [low] * 6).repeat(4)  # the sum of a group's two is small
        mixed[8] = 2.1e38
        check(logits(3, E, seed=7), top_k=6, score=score, bias=mixed, n_groups=4, topk_groups=2)


def test_scores_that_64_bits_cannot_tell_apart():
    """Sigmoid scores of logits beyond 37 are all 1 in 64 bits, softmax scores 745 below the largest all 0.  Without
    a bias the logits order such experts; keys with a bias tie, so the lowest index comes first."""
    L = torch.linspace(40.0, 60.0, 64).repeat(2, 1)
    zero = torch.zeros(64, device=DEV)
    ids = lambda X, **k: moe.moe_select_experts(X.to(DEV), moe.RouteRule(6, **k))[0].cpu().tolist()[0]
    assert ids(L, score="sigmoid") == [63, 62, 61, 60, 59, 58]
    assert ids(L, score="sigmoid", selection_bias=zero) == [0, 1, 2, 3, 4, 5]
    grouped = dict(score="sigmoid", n_groups=4, topk_groups=1)
    assert ids(L, group_score="max", **grouped) == [63, 62, 61, 60, 59, 58]
    assert ids(L, group_score="top2", **grouped) == [15, 14, 13, 12, 11, 10]  # (ranks are sums of scores: they tie)
    assert ids(L, group_score="max", selection_bias=zero, **grouped) == [0, 1, 2, 3, 4, 5]
    L = torch.linspace(-900.0, -800.0, 64).repeat(2, 1)
    L[:, 20] = 0.0
    assert ids(L) == [20, 63, 62, 61, 60, 59]
    assert ids(L, selection_bias=zero) == [20, 0, 1, 2, 3, 4]
