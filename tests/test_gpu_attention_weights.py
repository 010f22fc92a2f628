"""Softmax weights far below a row's largest (needs an MI355X).

What the kernels promise of a weight w of a row, in the 16-bit type of the rows: bf16 has fp32's exponents, so a weight is off
by one rounding (2^-8 w) in prompts and by 2^-16 w in decoding, which multiplies two parts.  fp16 ends at 2^-24 and loses its bits
below 2^-14: the reference of a tile's exponentials puts the largest of the tile between 2^0 and 2^15.5, and the row's largest at
2^7 at least.  So a weight is off by 2^-11 w (2^-22 w in decoding), or, where it or its low part is subnormal, by half of 2^-24:
2^-25 of its tile's largest weight, and 2^-32 in the tile of the row's largest.  A prompt's weight is subnormal below 2^-14 of its
tile's largest (2^-21 there).  A reference falls no further than 40 bits below where it last rose, with the row's largest at
2^47 then, which leaves 2^-72 of that.  A tile is 64 keys of a prompt and 32 of a cache."""
import math

import pytest
import torch

import attention_reference as ref
import mxfp4_routed_expert_router_amd as moe
from front_reference import half_step
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES
LN2 = math.log(2.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def expected(bits, v, seen, t, tile, decoding):
    """Rows of exponents `bits` [rows][keys] (base 2) over values v [keys][D] -> y and its tolerance, in 64 bits.  Scores are
    exact here (one product each): the fma and the reference add 2 roundings of at most 2^-24 max |bits|, the exponential
    2^-22; sums in fp32 as in attention_reference.attend."""
    bits, v = bits.double(), v.double()
    n = bits.shape[1]
    s = torch.where(seen, bits, torch.tensor(-math.inf, dtype=torch.float64))
    w = torch.exp2(s - s.max(1, keepdim=True).values)
    total = w.sum(1, keepdim=True)
    y = w @ v / total
    e = 4 * 2.0 ** -24 * bits.abs().max() * LN2 + 2.0 ** -22
    step = half_step(t) ** (2 if decoding else 1)
    tol = (w / total) @ v.abs() * (step + 2 * e + (3 * n + 64) * 2.0 ** -24) + y.abs() * half_step(t) * 1.001
    if t == "fp16":
        pad = -n % tile
        wt = torch.nn.functional.pad(w / total, (0, pad)).view(len(w), -1, tile)
        vt = torch.nn.functional.pad(v.abs(), (0, 0, 0, pad)).view(-1, tile, v.shape[1])
        top = wt.max(2, keepdim=True).values
        far = torch.where(top == top.max(1, keepdim=True).values, 2.0 ** 7, 1.0)
        lost = torch.where((wt < top * 2.0 ** -14 / far) | decoding, top * 2.0 ** -25 / far, 0.0)
        tol = tol + lost.flatten(1) @ vt.flatten(0, 1) + 2.0 ** -72 * v.abs().sum(0) + 2.0 ** -25
    else:
        tol = tol + 2.0 ** -134
    return y, tol


def sink_inputs(n, at, gap, D, t, seed=0):
    """One key `gap` bits above all others, whose value is zero: y is made of the small weights alone."""
    g = torch.Generator().manual_seed(seed)
    k = torch.zeros(n, 1, D)
    k[:, 0, 0] = -torch.rand(n, generator=g) * 2  # the others' scores, within 2 bits
    k[at, 0, 0] = gap
    v = 0.5 + torch.rand(n, 1, D, generator=g)
    v[:, :, ::2] = 1.0
    v[at] = 0.0
    return k.to(TYPES[t]), v.to(TYPES[t])


@pytest.mark.parametrize("gap", [8, 14, 17.25, 20.5, 24, 30, 38, 60])
@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("n,at", [(50, 0), (64, 63), (1000, 0), (1000, 500), (1000, 999), (5000, 70)])
def test_prompt_weights_beside_a_large_one(n, at, gap, t):
    """A key that takes the weight and adds nothing."""
    D, rows = 64, 40
    k, v = sink_inputs(n, at, gap, D, t, n)
    q = torch.zeros(rows, 2, D, dtype=TYPES[t])
    q[:, :, 0] = 1.0
    c = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for causal in (True, False):
        y, _ = moe.moe_attention_prompt(q.to(DEV), k.to(DEV), v.to(DEV), c(0, rows), c(0, n), scale=LN2, causal=causal)
        torch.cuda.synchronize()
        i = torch.arange(rows)[:, None] + n - rows
        seen = torch.arange(n) <= i if causal else torch.ones(rows, n, dtype=torch.bool)
        want, tol = expected(k[:, 0, 0].double().expand(rows, n), v[:, 0], seen, t, 64, False)
        for h in range(2):
            r = ref.check(y[:, h], want, tol, f"prompt {t} n={n} at={at} gap={gap} causal={causal}")
        note(f"prompt {t} n={n} at={at} gap={gap} causal={causal}: {r:.2f} of the tolerance")


@pytest.mark.parametrize("gap", [14, 20.5, 24, 38])
@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n,at,B", [(20, 3, 1), (32, 31, 1), (1000, 0, 1), (1000, 999, 130), (1000, 97, 130), (5000, 70, 130)])
def test_decode_weights_beside_a_large_one(n, at, B, page, gap, t):
    """The same over a cache.  130 rows of eight key-value heads take their keys in one part, so that a wave that meets the
    large key walks over many others."""
    D, Hkv = 64, 8
    k, v = sink_inputs(n, at, gap, D, t, n)
    pages = (n + page - 1) // page
    pad = lambda x: torch.nn.functional.pad(x[:, 0], (0, 0, 0, pages * page - n)).view(pages, 1, page, D).expand(-1, Hkv, -1, -1)
    cache = moe.KvCache(pad(k).contiguous().to(DEV), pad(v).contiguous().to(DEV))
    table = torch.arange(pages, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    q = torch.zeros(B, 2 * Hkv, D, dtype=TYPES[t])
    q[:, :, 0] = 1.0
    y, _ = moe.moe_attention_decode(q.to(DEV), cache, table, torch.full((B,), n, dtype=torch.int32, device=DEV), scale=LN2)
    torch.cuda.synchronize()
    want, tol = expected(k[:, 0, 0].double()[None], v[:, 0], torch.ones(1, n, dtype=torch.bool), t, 32, True)
    r = max(ref.check(y[:, h], want.expand(B, -1), tol.expand(B, -1), f"decode {t} n={n} at={at} gap={gap}")
            for h in range(2 * Hkv))
    note(f"decode {t} n={n} at={at} gap={gap} page={page} B={B}: {r:.2f} of the tolerance")


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_references_that_rise_and_fall(D, t):
    """Keys whose scores go up and down by tens of bits from tile to tile, each tile's largest with the value zero."""
    n, rows = 1000, 70
    g = torch.Generator().manual_seed(D)
    level = torch.tensor([0.0, 12, -9, 25, 3, 3, -20, 30, 8, 18, -12, 31, 29, 5, 0, -31])
    k = torch.zeros(n, 1, D)
    k[:, 0, 0] = level[torch.arange(n) // 64] - 4 * torch.rand(n, generator=g)
    k[::32, 0, 0] += 9
    v = 0.5 + torch.rand(n, 1, D, generator=g)
    v[::32] = 0.0
    k, v = k.to(TYPES[t]), v.to(TYPES[t])
    q = torch.zeros(rows, 4, D, dtype=TYPES[t])
    q[:, :, 0] = 1.0
    c = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for a, b in ((0, n), (0, 300), (100, 1000)):  # the first rows of a context, the last ones, a shorter one
        kk, vv = k[a:b], v[a:b]
        m = b - a
        y, lse = moe.moe_attention_prompt(q.to(DEV), kk.to(DEV), vv.to(DEV), c(0, rows), c(0, m), scale=LN2, want_lse=True)
        torch.cuda.synchronize()
        seen = torch.arange(m) <= torch.arange(rows)[:, None] + m - rows
        bits = kk[:, 0, 0].double().expand(rows, m)
        want, tol = expected(bits, vv[:, 0], seen, t, 64, False)
        r = max(ref.check(y[:, h], want, tol, f"rise and fall D={D} {t} {a}..{b}") for h in range(4))
        wl = torch.logsumexp(torch.where(seen, bits * LN2, torch.tensor(-math.inf, dtype=torch.float64)), 1)
        ref.check(lse[:, 1], wl, (m + 64) * 2.0 ** -24 + 2.0 ** -20 * (1 + wl.abs()), "lse")
        note(f"rise and fall D={D} {t} {a}..{b}: {r:.2f} of the tolerance")
