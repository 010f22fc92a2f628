"""The attention half of a decoder block as a user runs it (AttentionBlock: residual addition + norm, the product for q, k
and v, rotary positions and the cache write, attention), alone and in front of MoEBlock, prompts first and then tokens one
at a time over the cache that they filled, eager and from captured graphs (needs an MI355X).  Every step is checked on the
inputs that the GPU's previous step gave it, with that step's own tolerance."""
import numpy as np
import pytest
import torch

import attention_reference as aref
import front_reference as ref
import synth
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, expert_weights, note, require_gpu
from test_gpu_rope import tolerance as rope_tolerance

pytestmark = pytest.mark.gpu
H, HQ, HKV, D, PAGE, N = 512, 8, 2, 64, 16, 400


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(T, fmt="bf16", window=0, pairs="halves", seed=5):
    rng = np.random.default_rng(seed)
    n_out = (HQ + 2 * HKV) * D
    codes, _, _, _, _ = ref.weights("mxfp4", n_out, H, rng)
    scales = rng.integers(119, 123, (n_out, H // 32)).astype(np.uint8)
    c = np.stack([codes & 15, codes >> 4], 2).reshape(n_out, H)
    w = ref.E2M1[c] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
    wn = (1 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    cos, sin = aref.angles(N, D // 2 if pairs == "neighbours" else D)
    cache = moe.KvCache.empty(80, PAGE, HKV, D, fmt, device=DEV)
    for t in cache.tensors:
        if t is not None:
            t.zero_()
    block = moe.AttentionBlock(moe.LinearWeights(dev(codes), dev(scales)), T, moe.RmsNorm(dev(wn)), HQ, cache,
                               moe.Rope(cos.to(DEV), sin.to(DEV), pairs), window)
    return block, w, wn, cos, sin, pairs


def inputs(T, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(DEV), torch.randn(T, H, generator=g).bfloat16().to(DEV)


def check_front(m, x, res, r, t, positions):
    """Norm, product and rotation of the block's last pass; -> q as the attention saw it."""
    block, w, wn, cos, sin, pairs = m
    f = lambda v: v.detach().double().cpu().numpy()
    s, y = ref.add_rms_norm(f(x), f(res), wn, 1e-6)
    rel = (H / 256 + 80) * 2.0 ** -24
    assert np.all(np.abs(f(r) - s) <= np.abs(s) * (2.0 ** -8 + 2.0 ** -23))
    assert np.all(np.abs(f(block.x[:t]) - y) <= np.abs(y) * (2.0 ** -8 + 2 * rel))
    xb = f(block.x[:t])
    want = xb @ w.T
    assert np.all(np.abs(f(block.qkv[:t]) - want) <= ref.linear_tolerance(xb, w, H, want, "fp32"))
    q = block.qkv[:t].cpu().double().view(t, -1, D)[:, :HQ]
    turned = aref.rope(q, cos, sin, positions, pairs)
    aref.check(block.q[:t], turned, rope_tolerance(q, turned, cos, sin, positions, pairs, "bf16"), "q")


def layout(lens, extra, seed=1):
    """Shuffled pages for sequences that will hold lens + extra tokens: table, and slots of token j of sequence b."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(80, generator=g).int()
    pages = [(n + extra + PAGE - 1) // PAGE for n in lens]
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    return table, lambda b, j: int(table[b, j // PAGE]) * PAGE + j % PAGE


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("window,pairs", [(0, "halves"), (50, "neighbours")])
def test_prompts_then_tokens(fmt, window, pairs):
    lens = [70, 1, 133]
    note(f"attention block {fmt} window={window} {pairs}")
    m = make(256, fmt, window, pairs)
    block = m[0]
    table, slot = layout(lens, 4)
    cu = np.cumsum([0] + lens).tolist()
    positions = torch.tensor([j for n in lens for j in range(n)], dtype=torch.int32)
    slots = ints([slot(b, j) for b, n in enumerate(lens) for j in range(n)])
    T = cu[-1]
    x, res = inputs(T)
    attn, r = block.prompt(x, res, positions.to(DEV), slots, ints(cu))
    torch.cuda.synchronize()
    assert attn.shape == (T, HQ * D)
    check_front(m, x, res, r, T, positions)
    y, _, tol, _ = aref.prompt(block.q[:T], block.k[:T], block.v[:T], cu, cu, D ** -0.5, True, window)
    aref.check(attn.view(T, HQ, D), y, tol, "prompt attention")
    if fmt == "bf16":  # the cache holds the rows that the prompt attended to
        k, v, _ = aref.cache_rows(block.cache, table[2], lens[2])
        assert torch.equal(k, block.k[cu[2]:cu[3]].double().cpu()) and torch.equal(v, block.v[cu[2]:cu[3]].double().cpu())
    for step in range(3):
        B = len(lens)
        now = [n + step for n in lens]
        x, res = inputs(B, 10 + step)
        attn, r = block.decode(x, res, ints(now), ints([slot(b, n) for b, n in enumerate(now)]), table.to(DEV),
                               ints([n + 1 for n in now]))
        torch.cuda.synchronize()
        check_front(m, x, res, r, B, torch.tensor(now, dtype=torch.int32))
        y, _, tol, _ = aref.decode(block.q[:B], block.cache, table, [n + 1 for n in now], D ** -0.5, window)
        aref.check(attn.view(B, HQ, D), y, tol, "decode attention")
        assert float(y.abs().max()) > 0.05


def test_prompt_and_decode_agree():
    """A sequence's last token by a prompt and by decoding over a bf16 cache: the same attention but for the rounding of
    the prompt's exponentials (2^-8 of each, at most) and of both outputs (2^-8 each)."""
    n = 150
    m = make(256)
    block = m[0]
    table, slot = layout([n], 0)
    x, res = inputs(n, 3)
    pos, slots = ints(list(range(n))), ints([slot(0, j) for j in range(n)])
    attn, r = block.prompt(x, res, pos, slots, ints([0, n]))
    last = attn[-1].double().cpu()
    vmax = float(block.v[:n].abs().max())
    a2, _ = block.decode(x[-1:], res[-1:], ints([n - 1]), ints([slot(0, n - 1)]), table.to(DEV), ints([n]))
    torch.cuda.synchronize()
    assert float((a2[0].double().cpu() - last).abs().max()) <= vmax * 4 * 2.0 ** -8


@pytest.mark.parametrize("mx", [None, "fp8"])
def test_decoder_block(mx):
    """Both halves in turn, twice, as two layers of a decoder: attention's output and residual into MoEBlock, its output and
    residual into the next attention; eager and from a graph replayed on changed inputs."""
    import test_gpu_block as front
    B, lens = 7, [40, 3, 99, 17, 64, 1, 30]
    note(f"decoder block mx={mx}")
    table, slot = layout([n + 1 for n in lens], 0)
    table = table.to(DEV)
    layers = []
    for i in range(2):
        a = make(B, "bf16", seed=5 + i)[0]
        for t in a.cache.tensors[:2]:
            t.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
        _, b, _, _, _, _, _, _ = front.make(B, mx, K_o=HQ * D, seed=21 + i)
        layers.append((a, b))
    x, res = inputs(B, 4)
    pos, slots, ln = ints(lens), ints([slot(b, n) for b, n in enumerate(lens)]), ints([n + 1 for n in lens])
    mid = [torch.empty_like(res) for _ in range(4)]

    def run():
        h, r = x, res
        for i, (a, b) in enumerate(layers):
            attn, r = a.decode(h, r, pos, slots, table, ln, max_len=100, residual_out=mid[2 * i])
            h, r = b.forward(attn, r, residual_out=mid[2 * i + 1])
        return h, r

    for _ in range(2):  # two passes give the same: the second writes the same rows into the cache
        y, r = run()
        torch.cuda.synchronize()
        first = (y.clone(), r.clone()) if _ == 0 else first
    assert torch.equal(first[0], y) and torch.equal(first[1], r) and bool(torch.isfinite(y).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for k in range(3):
        x2, r2 = inputs(B, 30 + k)
        x.copy_(x2)
        res.copy_(r2)
        y, r = run()
        want = (y.clone(), r.clone())
        out[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_no_tokens():
    block = make(4)[0]
    x, res = inputs(0)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    attn, r = block.prompt(x, res, none, none, ints([0, 0]))
    assert attn.shape == (0, HQ * D) and r.shape == (0, H)
    attn, r = block.decode(x, res, none, none, torch.zeros(0, 3, dtype=torch.int32, device=DEV), none)
    assert attn.shape == (0, HQ * D)


def test_refusals():
    block = make(4)[0]
    x, res = inputs(5)
    with pytest.raises(ValueError, match="built for 4"):
        block.decode(x, res, ints([0] * 5), ints([0] * 5), ints([[0]] * 5), ints([1] * 5))
    half = moe.KvCache.empty(4, 16, HKV, D, "fp16", device=DEV)
    with pytest.raises(ValueError, match="bf16"):
        moe.AttentionBlock(block.W_qkv, 4, block.norm, HQ, half)
    with pytest.raises(ValueError, match="do not fit"):
        moe.AttentionBlock(block.W_qkv, 4, block.norm, HQ + 1, block.cache)
    q = torch.zeros(2, HQ, D, device=DEV)
    with pytest.raises(moe.MoEError):  # fp32 q
        moe.moe_attention_decode(q, block.cache, ints([[0], [0]]), ints([1, 1]))
    with pytest.raises(ValueError):
        moe.moe_attention_decode(q.bfloat16(), block.cache, ints([[0], [0]]).cpu(), ints([1, 1]))
    with pytest.raises(ValueError):
        moe.moe_attention_decode(q.bfloat16(), block.cache, ints([[0], [0]]), ints([1, 1]).cpu())
    with pytest.raises(ValueError):
        moe.moe_attention_decode(q.bfloat16(), block.cache, ints([[0], [0]]), ints([1, 1]).long())
    with pytest.raises(moe.MoEError):
        moe.moe_attention_decode(q.bfloat16(), block.cache, ints([[0], [0]]), ints([1, 1]), max_len=17)
    with pytest.raises(moe.MoEError):
        moe.moe_attention_prompt(q.bfloat16(), q.bfloat16()[:, :2].contiguous(), q.bfloat16()[:, :2].contiguous(), ints([0, 2]),
                                 causal=False, window=3)
