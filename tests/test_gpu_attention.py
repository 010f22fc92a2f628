"""moe_attention_prompt and moe_attention_decode on the GPU against 64 bits (needs an MI355X).  The tolerances are
derived in attention_reference.attend."""
import math

import pytest
import torch

import attention_reference as ref
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# ---------------------------------------------------------------------------------------------------- prompts
def strided(t, layout):
    """The same values, tokens or heads of a larger buffer."""
    if layout == "tokens":  # [tokens][heads][D] inside rows of more heads
        big = torch.full((t.shape[0], t.shape[1] + 3, t.shape[2]), math.nan, dtype=t.dtype, device=t.device)
        big[:, 1:1 + t.shape[1]] = t
        return big[:, 1:1 + t.shape[1]]
    if layout == "heads":  # [heads][tokens][D]
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    return t


def prompt_inputs(nq, nk, Hq, Hkv, D, dt, seed=0, layout="plain", spread=2.0, tail=3):
    g = torch.Generator().manual_seed(seed)
    cu_q, cu_k = [0], [0]
    for a, b in zip(nq, nk):
        cu_q.append(cu_q[-1] + a)
        cu_k.append(cu_k[-1] + b)
    t = TYPES[dt]
    q = (spread * torch.randn(cu_q[-1] + tail, Hq, D, generator=g)).to(t)
    k = torch.randn(cu_k[-1] + tail, Hkv, D, generator=g).to(t)
    v = torch.randn(cu_k[-1] + tail, Hkv, D, generator=g).to(t)
    for x, n in ((q, cu_q[-1]), (k, cu_k[-1]), (v, cu_k[-1])):
        x[n:] = math.nan  # behind the last sequence
    return (*(strided(x.to(DEV), layout) for x in (q, k, v)), cu_q, cu_k)


def run_prompt(q, k, v, cu_q, cu_k, causal=True, window=0, scale=None, what=""):
    D = q.shape[2]
    s = D ** -0.5 if scale is None else scale
    c = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    moe.moe_attention_prompt(q, k, v, c(cu_q), c(cu_k), scale=scale, causal=causal, window=window, out=(y, lse))
    torch.cuda.synchronize()
    wy, wl, ty, tl = ref.prompt(q, k, v, cu_q, cu_k, s, causal, window)
    outside = torch.isnan(wl)
    assert bool((y.cpu()[outside] == 7.0).all()) and bool((lse.cpu()[outside] == 7.0).all()), "rows outside the sequences"
    r = ref.check(y.cpu()[~outside], wy[~outside], ty[~outside], what + " y")
    rl = ref.check(lse.cpu()[~outside], wl[~outside], tl[~outside], what + " lse")
    note(f"  {what}: {r:.2f} of the tolerance, lse {rl:.2f}")
    return y, lse


def prompt(nq, nk, Hq, Hkv, D, dt="bf16", causal=True, window=0, layout="plain", seed=0, scale=None, spread=2.0):
    what = f"prompt nq={nq} nk={nk} heads={Hq}/{Hkv} D={D} {dt} causal={causal} window={window} {layout}"
    note(what)
    return run_prompt(*prompt_inputs(nq, nk, Hq, Hkv, D, dt, seed, layout, spread), causal, window, scale, what)


@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257, 400])
def test_prompt_lengths(n):
    prompt([n], [n], 4, 2, 64, seed=n)


@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 80, 96, 128, 160, 192, 200, 256])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_prompt_head_sizes(D, dt):
    prompt([150, 3], [150, 3], 4, 2, D, dt, seed=D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (5, 1), (14, 2), (24, 8), (16, 16), (64, 8), (40, 1), (200, 1)])
def test_prompt_head_groups(Hq, Hkv):
    prompt([70, 1, 33], [70, 1, 33], Hq, Hkv, 64, seed=Hq)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [([5, 0, 64, 1], [5, 0, 64, 1]), ([1, 7, 100], [300, 7, 131]), ([40, 130], [20, 3]),
                                   ([0, 0], [5, 0]), ([3, 4], [0, 70]), ([300], [64])])
def test_prompt_ragged(nq, nk, causal):
    """Empty sequences, more keys than queries (earlier ones), fewer (rows that see nothing), no keys at all."""
    prompt(nq, nk, 4, 2, 64, causal=causal, seed=len(nq))


@pytest.mark.parametrize("n", [63, 64, 65, 129, 400, 5000])
def test_prompt_many_sequences(n):
    """Sequences of 0 to 4 tokens, some with more keys: their places are searched for, 64 at a step."""
    nq = [(7 * i) % 5 for i in range(n)]
    prompt(nq, [x + (i % 3) for i, x in enumerate(nq)], 3, 1, 16, seed=n)
    if n == 400:
        nq[200], nq[399] = 300, 150
        prompt(nq, nq, 5, 1, 64, seed=n)


@pytest.mark.parametrize("cu", [[0, 300, 100, 40, 400, 200, 350], [-7, 50, 20, 2 ** 31 - 1, 10, 300, 400], [400, 0, 400], [400, 100]])
@pytest.mark.parametrize("Tk", [400, 9000])
def test_prompt_sequences_out_of_order(cu, Tk):
    """Offsets that descend or leave the rows have no defined result, but nothing outside q's rows is written."""
    n, guard = 400, 64
    q, k, v, _, _ = prompt_inputs([n], [Tk], 4, 2, 64, "bf16", 5, tail=0)
    y = torch.full((n + 2 * guard, 4, 64), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((n + 2 * guard, 4), 7.0, device=DEV)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    moe.moe_attention_prompt(q, k, v, c, out=(y[guard:-guard], lse[guard:-guard]))
    torch.cuda.synchronize()
    for t in (y, lse):
        assert bool((t[:guard] == 7.0).all()) and bool((t[-guard:] == 7.0).all())


@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 1000])
@pytest.mark.parametrize("G", [1, 4])
def test_prompt_windows(window, G):
    prompt([330, 50], [330, 90], 4, 4 // G, 64, "fp16", window=window, seed=window)


@pytest.mark.parametrize("window", [200, 2 ** 30, 2 ** 31 - 1])
def test_prompt_windows_past_the_keys(window):
    """Also for queries in front of the first key, whose positions are negative."""
    prompt([10, 150, 64], [5, 20, 200], 4, 2, 64, window=window, seed=8)
    prompt([3], [5000], 4, 2, 64, window=window + (0 if window > 200 else 4800), seed=8)


@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_prompt_strides(layout, D):
    prompt([129, 40], [140, 40], 6, 3, D, "fp16", layout=layout, seed=D)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_prompt_many_keys(D):
    prompt([1500, 10], [1500, 1300], 4, 2, D, seed=D)


@pytest.mark.parametrize("nq,nk,Hq,Hkv", [(1, 5000, 4, 2), (16, 9001, 8, 1), (100, 3100, 8, 2), (3, 70, 2, 2)])
@pytest.mark.parametrize("window", [0, 1500])
def test_prompt_pieces(nq, nk, Hq, Hkv, window):
    """The last rows of long contexts, whose keys several workgroups share."""
    prompt([nq], [nk], Hq, Hkv, 128, seed=nq, window=window)
    prompt([nq, 2], [nk, 2], Hq, Hkv, 64, "fp16", seed=nq, window=window)


@pytest.mark.parametrize("scale,spread", [(1.0, 3.0), (0.01, 1.0), (1e-6, 1.0), (4.0, 2.0)])
def test_prompt_scales(scale, spread):
    """Nearly uniform weights and ones where a few keys take all."""
    prompt([200], [200], 4, 2, 64, scale=scale, spread=spread, seed=5)


def test_prompt_rising_scores():
    """Every key beats all before it by far, so that the reference rises with every tile; and the other way round."""
    for sign in (1.0, -1.0):
        q, k, v, cu_q, cu_k = prompt_inputs([300], [300], 2, 1, 64, "bf16", 1)
        q[:300, :, 0] = 16.0
        k[:300, 0, 0] = sign * torch.arange(300, device=DEV).to(k.dtype)
        run_prompt(q, k, v, cu_q, cu_k, scale=0.25, what=f"rising {sign}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("fp16", 128), ("bf16", 96)])
def test_prompt_values_of_masked_keys(bad, dt, D):
    """A value that is not finite reaches the rows that see its key and no other; nor does a key behind a row.  What it
    does not reach is held against the 64-bit form of the finite inputs, not bit for bit: a masked tile with such a value
    adds its keys one at a time, the same terms in another order, for which the tolerance's (3 n + 64) 2^-24 holds alike."""
    note(f"masked {bad} {dt} {D}")
    q, k, v, cu_q, cu_k = prompt_inputs([150], [150], 4, 2, D, dt, 3)
    c = torch.tensor(cu_q, dtype=torch.int32, device=DEV)
    for window in (0, 40):
        clean, lse = moe.moe_attention_prompt(q, k, v, c, window=window, want_lse=True)
        want, _, tol, _ = (x[:150] for x in ref.prompt(q, k, v, cu_q, cu_k, D ** -0.5, True, window))
        for at in (0, 31, 70, 149):
            v2, k2 = v.clone(), k.clone()
            v2[at, 1, 5] = bad
            y, l2 = moe.moe_attention_prompt(q, k, v2, c, window=window, want_lse=True)
            torch.cuda.synchronize()
            rows = torch.arange(150)
            sees = (rows >= at) & ((rows < at + window) if window else (rows >= 0))
            same = torch.ones(150, 4, D, dtype=torch.bool)
            same[sees, 2:, 5] = False
            y, ref_y = y[:150].float().cpu(), clean[:150].float().cpu()
            ref.check(y[same], want[same], tol[same], f"key {at} window {window}")
            assert torch.equal(l2[:150], lse[:150])
            hit = y[sees][:, 2:, 5]
            assert bool((torch.isnan(hit) if math.isnan(bad) else hit == bad).all())
            k2[at, 1] = bad
            y, _ = moe.moe_attention_prompt(q, k2, v, c, window=window)
            y = y[:150].float().cpu()
            same = torch.ones(150, 4, D, dtype=torch.bool)
            same[sees, 2:] = False
            assert torch.equal(y[same], ref_y[same])


def test_prompt_edges_of_the_mask():
    """Keys just outside the mask with huge values and scores, keys just inside that take all the weight."""
    n, D, w = 193, 64, 65
    q, k, v, cu_q, cu_k = prompt_inputs([n], [n], 2, 2, D, "bf16", 9)
    k[:n] = 0.0
    q[:n] = 0.0
    v[:n] = torch.arange(n, device=DEV)[:, None, None].to(v.dtype)  # whole numbers up to 192 are exact in bf16
    c = torch.tensor(cu_q, dtype=torch.int32, device=DEV)
    y, lse = moe.moe_attention_prompt(q, k, v, c, window=w, want_lse=True)
    torch.cuda.synchronize()
    i = torch.arange(n, dtype=torch.float64)
    first = (i - w + 1).clamp(min=0)
    # equal scores: the mean of the visible whole numbers, ln of how many; P = 1 is exact
    mean = (first + i) / 2
    ref.check(y[:n, 0, 0], mean, mean * 2.0 ** -8 + 1e-30, "mean")
    ref.check(lse[:n, 0], torch.log(i - first + 1), torch.full((n,), 1e-6, dtype=torch.float64), "count")


@pytest.mark.parametrize("D,window", [(64, 0), (128, 100), (256, 40)])
def test_prompt_waves_without_a_share(D, window):
    """One query head per key-value head: a workgroup's waves stand at different tokens, so some have no part in a tile
    that they load for the others.  The same bits every time, and the right ones."""
    q, k, v, cu_q, cu_k = prompt_inputs([700, 129], [700, 129], 8, 8, D, "bf16", 6)
    first, _ = run_prompt(q, k, v, cu_q, cu_k, True, window, what=f"waves D={D} window={window}")
    c = torch.tensor(cu_q, dtype=torch.int32, device=DEV)
    for _ in range(20):
        y, _ = moe.moe_attention_prompt(q, k, v, c, window=window)
        assert torch.equal(y[:cu_q[-1]], first[:cu_q[-1]])


def test_prompt_same_bits_again_and_on_other_streams():
    q, k, v, cu_q, cu_k = prompt_inputs([1000, 77], [1000, 400], 8, 2, 128, "bf16", 4)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu_q, cu_k))
    first, l1 = moe.moe_attention_prompt(q, k, v, cq, ck, want_lse=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2):
        with torch.cuda.stream(s):
            outs.append(moe.moe_attention_prompt(q, k, v, cq, ck, want_lse=True))
    torch.cuda.synchronize()
    n = cu_q[-1]
    for y, l2 in outs:
        assert torch.equal(y[:n], first[:n]) and torch.equal(l1[:n], l2[:n])


# ---------------------------------------------------------------------------------------------------- decoding
def make_cache(lens, page, Hkv, D, fmt, seed=0, order="head", extra=2):
    """A cache whose sequences lie on shuffled pages; what no token is on holds NaN (codes: NaN)."""
    g = torch.Generator().manual_seed(seed)
    pages = [(n + page - 1) // page for n in lens]
    n_pages = sum(pages) + extra
    perm = torch.randperm(n_pages, generator=g).int()
    width = max(pages + [1])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    used = torch.zeros(n_pages, page, dtype=torch.bool)
    at = 0
    for b, (n, m) in enumerate(zip(lens, pages)):
        table[b, :m] = perm[at:at + m]
        for i in range(m):
            used[perm[at + i], :min(page, n - i * page)] = True
        at += m
    shape = (n_pages, Hkv, page, D)
    keep = used[:, None, :, None]

    def place(t):  # another order of pages, heads and tokens in memory
        if order == "token":
            t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        elif order == "head first":
            t = t.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
        elif order == "padded":
            big = torch.zeros(t.shape[0], t.shape[1] + 1, t.shape[2] + 2, t.shape[3], dtype=t.dtype)
            big[:, :-1, 1:-1] = t
            return big.to(DEV)[:, :-1, 1:-1]
        return t.to(DEV)

    if fmt == "mxfp8":
        mk = lambda: torch.where(keep, torch.randint(0, 0x7F, shape, generator=g) + 128 * torch.randint(0, 2, shape, generator=g),
                                 torch.tensor(0x7F)).to(torch.uint8)
        sc = lambda: torch.randint(117, 121, shape[:3] + (D // 32,), generator=g).to(torch.uint8)
        k, v, ks, vs = mk(), mk(), sc(), sc()
        return moe.KvCache(place(k), place(v), place(ks), place(vs)), table
    t = TYPES[fmt]
    mk = lambda: torch.where(keep, torch.randn(shape, generator=g), torch.tensor(math.nan)).to(t)
    return moe.KvCache(place(mk()), place(mk())), table


def decode(lens, page, Hq, Hkv, D, fmt="bf16", window=0, seed=0, order="head", max_len=None, scale=None, spread=2.0):
    what = f"decode lens={lens[:6]} page={page} heads={Hq}/{Hkv} D={D} {fmt} window={window} {order}"
    note(what)
    cache, table = make_cache(lens, page, Hkv, D, fmt, seed, order)
    g = torch.Generator().manual_seed(seed + 1)
    q = (spread * torch.randn(len(lens), Hq, D, generator=g)).to(cache.act).to(DEV)
    return run_decode(q, cache, table, lens, window, max_len, scale, what)


def run_decode(q, cache, table, lens, window=0, max_len=None, scale=None, what=""):
    s = q.shape[2] ** -0.5 if scale is None else scale
    y, lse = moe.moe_attention_decode(q, cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                      max_len=max_len, window=window, scale=scale, want_lse=True)
    torch.cuda.synchronize()
    if max_len is None:
        max_len = table.shape[1] * cache.page_size
    wy, wl, ty, tl = ref.decode(q, cache, table, lens, s, window, max_len)
    r = ref.check(y, wy, ty, what + " y")
    rl = ref.check(lse, wl, tl, what + " lse")
    note(f"  {what}: {r:.2f} of the tolerance, lse {rl:.2f}")
    return y, lse


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 100])
def test_decode_pages(fmt, page):
    decode([1, 2, 31, 0, 33, 64, 127, 128, 129, 200, 300], page, 4, 2, 64, fmt, seed=page)


@pytest.mark.parametrize("D", [8, 24, 64, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
def test_decode_head_sizes(D, fmt):
    if fmt == "mxfp8" and D % 32:
        D = (D + 31) // 32 * 32
    decode([150, 3, 77], 16, 4, 2, D, fmt, seed=D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (8, 1), (7, 1), (16, 1), (17, 1), (40, 1), (64, 8), (33, 1), (6, 3)])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_decode_head_groups(Hq, Hkv, fmt):
    decode([90, 1, 257], 32, Hq, Hkv, 64, fmt, seed=Hq)


@pytest.mark.parametrize("n", [1000, 4097, 20011])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
@pytest.mark.parametrize("B", [1, 3])
def test_decode_long(n, fmt, B):
    """Split over the cache's length and joined."""
    decode([n] + [n // 3, 5][:B - 1], 64, 8, 2, 128, fmt, seed=n)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 999, 5000])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_decode_windows(window, fmt):
    decode([3, 64, 65, 1000, 2500], 48, 4, 2, 64, fmt, window=window, seed=window)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_decode_windows_past_the_keys(fmt):
    decode([1, 0, 700, 64], 16, 8, 2, 64, fmt, window=2 ** 31 - 1)


@pytest.mark.parametrize("order", ["token", "head first", "padded"])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
def test_decode_orders(order, fmt):
    decode([130, 40, 7], 16, 6, 3, 96, fmt, order=order, seed=2)


def test_decode_many_rows():
    decode([(37 * i) % 300 for i in range(400)], 16, 8, 4, 64, seed=3)


def test_decode_max_len():
    """Lengths beyond max_len, and negative ones, are clamped."""
    decode([100, 250, 77], 16, 4, 2, 64, max_len=90, seed=4)
    cache, table = make_cache([100, 50], 16, 2, 64, "bf16", 5)
    q = torch.randn(2, 4, 64).bfloat16().to(DEV)
    run_decode(q, cache, table, [-5, 1 << 30], max_len=50, what="clamped")
    y, lse = moe.moe_attention_decode(q, cache, table.to(DEV), torch.tensor([3, 4], dtype=torch.int32, device=DEV),
                                      max_len=0, want_lse=True)
    assert not bool(y.any()) and bool((lse == -math.inf).all())


def test_decode_pages_that_are_none():
    """Tokens on page numbers outside the cache are left out."""
    lens = [200, 100, 64]
    cache, table = make_cache(lens, 16, 2, 64, "bf16", 6)
    table[0, 3], table[0, 12], table[1, 0], table[1, 6] = -1, cache.n_pages, 1 << 30, -(1 << 31)
    table[2, :] = -7  # none at all
    q = torch.randn(3, 4, 64).bfloat16().to(DEV)
    run_decode(q, cache, table, lens, what="missing pages")
    run_decode(q, cache, table, lens, window=50, what="missing pages, window")


def test_decode_shared_rows():
    """Several newest tokens of one sequence: rows with the same pages and rising lengths."""
    cache, table = make_cache([300], 16, 2, 64, "mxfp8", 7)
    q = torch.randn(4, 4, 64).bfloat16().to(DEV)
    run_decode(q, cache, table.expand(4, -1).contiguous(), [297, 298, 299, 300], what="four newest tokens")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("fmt", ["bf16", "fp16"])
def test_decode_values_outside_the_range(bad, fmt):
    """What lies in front of the window or on another page changes nothing; an infinite value that is seen shows, as an
    infinity or a NaN: a weight is multiplied in two parts, of which the low one may be zero or negative, and 0 * inf and
    inf - inf are NaN."""
    lens = [100, 70]
    cache, table = make_cache(lens, 16, 2, 64, fmt, 8)
    q = torch.randn(2, 4, 64).to(cache.act).to(DEV)
    k, v = cache.tensors[:2]
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean, _ = moe.moe_attention_decode(q, cache, table.to(DEV), ln, window=40)
    p, o = int(table[0, 59 // 16]), 59 % 16  # key 59 of sequence 0, just in front of its window
    k[p, :, o], v[p, :, o] = bad, bad
    y, _ = moe.moe_attention_decode(q, cache, table.to(DEV), ln, window=40)
    assert torch.equal(y, clean)
    v[p, :, o + 1, 3] = math.inf
    y, _ = moe.moe_attention_decode(q, cache, table.to(DEV), ln, window=40)
    assert not bool(torch.isfinite(y[0, :, 3]).any()) and torch.equal(y[0, :, 4:], clean[0, :, 4:]) and torch.equal(y[1], clean[1])


@pytest.mark.parametrize("scale,spread", [(1.0, 3.0), (1e-6, 1.0), (4.0, 2.0)])
def test_decode_scales(scale, spread):
    decode([300, 1, 2000], 16, 4, 2, 64, scale=scale, spread=spread, seed=9)


def test_decode_far_offsets():
    """A cache beyond 2^31 values: pages at its far end."""
    page, Hkv, D = 64, 8, 256
    n_pages = (1 << 31) // (page * Hkv * D) + 40  # 4.3 GB each for K and V
    cache = moe.KvCache.empty(n_pages, page, Hkv, D)
    k, v = cache.tensors[:2]
    k[-8:].normal_()
    v[-8:].normal_()
    table = torch.arange(n_pages - 8, n_pages, dtype=torch.int32).flip(0)[None]
    q = torch.randn(1, Hkv * 2, D).bfloat16().to(DEV)
    lens = torch.tensor([500], dtype=torch.int32, device=DEV)
    y, lse = moe.moe_attention_decode(q, cache, table.to(DEV), lens, want_lse=True)
    near = moe.KvCache(k[-8:].clone(), v[-8:].clone())
    y2, lse2 = moe.moe_attention_decode(q, near, (table - (n_pages - 8)).to(DEV), lens, want_lse=True)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)
    run_decode(q, near, table - (n_pages - 8), [500], what="far pages")


def test_attention_in_graphs():
    """Captured once, replayed on changed inputs with eager work between, each replay against the eager call; two graphs
    with a workspace each."""
    cache, table = make_cache([3000, 1500], 64, 2, 128, "bf16", 10)
    table = table.to(DEV)
    lens = torch.tensor([3000, 1500], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 8, 128).bfloat16().to(DEV)
    pq, pk, pv, cu, _ = prompt_inputs([20, 100], [20, 100], 8, 2, 128, "bf16", 11)
    cu_k = torch.tensor([0, 20, 120], dtype=torch.int32, device=DEV)

    def both(out):
        moe.moe_attention_decode(q, cache, table, lens, out=out[:2])
        moe.moe_attention_prompt(pq, pk, pv, cu_k, out=out[2:])

    def buffers():
        return (torch.zeros_like(q), torch.zeros(2, 8, device=DEV), torch.zeros_like(pq),
                torch.zeros(pq.shape[:2], device=DEV))

    a, b, eager = buffers(), buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(a)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for out in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(out)
        graphs.append(g)
    for i in range(4):
        q.copy_(torch.randn(2, 8, 128).bfloat16())
        lens.copy_(torch.tensor([3000 - 700 * i, 1500 - 499 * i], dtype=torch.int32))
        pv[:120].copy_(torch.randn(120, 2, 128).bfloat16())
        both(eager)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, y, z in zip(a, b, eager):
            assert torch.equal(x, y) and torch.equal(x, z)
