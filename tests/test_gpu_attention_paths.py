"""moe_attention_decode on every head size, type and kind of page, over several tiles of a wave, and MXFP8 scales at both ends
(needs an MI355X).  Tolerances: attention_reference.attend."""
import math

import pytest
import torch

import attention_reference as ref
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, note, require_gpu
from test_gpu_attention import make_cache, run_decode

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES
SIZES = [(t, D) for t in ("bf16", "fp16", "mxfp8") for D in (24, 32, 64, 80, 96, 128, 136, 160, 192, 200, 224, 256)
         if t != "mxfp8" or D % 32 == 0]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def queries(rows, heads, D, act, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(rows, heads, D, generator=g)).to(act).to(DEV)


@pytest.mark.parametrize("fmt,D", SIZES)
@pytest.mark.parametrize("page", [32, 64, 128])
def test_decode_aligned_pages(page, fmt, D):
    """Pages of whole tiles: all keys, windows that start inside a tile, page numbers outside the cache."""
    lens = [150, 3, 77, 0, 300, 32]
    for order in ("head", "token"):
        what = f"aligned page={page} D={D} {fmt} {order}"
        note(what)
        cache, table = make_cache(lens, page, 2, D, fmt, D, order)
        q = queries(len(lens), 6, D, cache.act, D + 1)
        for window in (0, 45):
            run_decode(q, cache, table, lens, window, what=f"{what} window={window}")
        table[0, 0], table[2, table.shape[1] - 1], table[4, 1], table[4, 2] = -1, 1 << 30, cache.n_pages, -(1 << 31)
        run_decode(q, cache, table, lens, what=what + " missing pages")
        run_decode(q, cache, table, lens, 130, what=what + " missing pages, window")


def ramp(cache, up):
    """Scores that rise (or fall) with the tokens, by more than 2^8 again and again: value 0 of a head's keys."""
    k, _, ks, _ = cache.tensors
    n = cache.n_pages * cache.page_size
    j = torch.arange(n, device=DEV).view(cache.n_pages, 1, cache.page_size)
    j = j if up else n - 1 - j
    if ks is None:
        k[..., 0] = (j / 16).to(k.dtype).expand(k.shape[:3])
    else:
        k[..., :32] = 0
        k[..., 0] = 0x38  # 1
        ks[..., 0] = (112 + 15 * j // n).to(torch.uint8).expand(k.shape[:3])


@pytest.mark.parametrize("fmt,D", SIZES)
@pytest.mark.parametrize("page", [64, 16])
def test_decode_many_tiles(page, fmt, D):
    """A wave that walks over eight tiles: 130 rows of eight key-value heads are enough workgroups without parts."""
    B, n, Hkv, rows = 130, 1000, 8, torch.tensor([0, 1, 56, 63, 128, 129])
    what = f"many tiles page={page} D={D} {fmt}"
    note(what)
    pages = (n + page - 1) // page
    cache, _ = make_cache([pages * page], page, Hkv, D, fmt, D, extra=0)
    lens = [1 + (611 * i) % n for i in range(B)]
    lens[56], lens[128], lens[129] = n, n - 500, n - 33
    assert moe.moe_attention_decode_workspace_bytes(B, Hkv, cache, n) == 0  # one part
    g = torch.Generator().manual_seed(D)
    table = torch.stack([torch.arange(pages)] + [torch.randperm(pages, generator=g) for _ in range(3)])
    table = table[torch.arange(B) % 4].int().contiguous()
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for kind in ("random", "up", "down"):
        if kind != "random":
            ramp(cache, kind == "up")
        q = queries(B, 2 * Hkv, D, cache.act, D + 1)
        q[..., 0] = 8.0
        for window in (0, 333):
            y, lse = moe.moe_attention_decode(q, cache, table.to(DEV), ln, window=window, want_lse=True, max_len=n)
            torch.cuda.synchronize()
            wy, wl, ty, tl = ref.decode(q[rows], cache, table[rows], [lens[i] for i in rows], D ** -0.5, window, n)
            r = ref.check(y[rows], wy, ty, f"{what} {kind} window={window} y")
            rl = ref.check(lse[rows], wl, tl, f"{what} {kind} window={window} lse")
            note(f"  {kind} window={window}: {r:.2f} of the tolerance, lse {rl:.2f}")


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
@pytest.mark.parametrize("page", [32, 48])
@pytest.mark.parametrize("D", [64, 192])
def test_decode_page_numbers_reloaded(D, page, fmt):
    """More than 64 tiles of one wave, which holds the page numbers of 64 at a time."""
    B, n, Hkv, rows = 128, 9500, 8, torch.tensor([3, 127])
    what = f"reloaded page={page} D={D} {fmt}"
    note(what)
    pages = (n + page - 1) // page
    cache, _ = make_cache([pages * page], page, Hkv, D, fmt, 1, extra=0)
    assert moe.moe_attention_decode_workspace_bytes(B, Hkv, cache, n) == 0
    g = torch.Generator().manual_seed(2)
    table = torch.randperm(pages, generator=g).int().expand(B, -1).contiguous()
    table[127, 5], table[127, -1] = -1, cache.n_pages
    lens = [n if i == 3 else (n - 77 if i == 127 else 1 + i) for i in range(B)]
    q = queries(B, Hkv, D, cache.act, 3)
    y, lse = moe.moe_attention_decode(q, cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), max_len=n,
                                      want_lse=True)
    torch.cuda.synchronize()
    wy, wl, ty, tl = ref.decode(q[rows], cache, table[rows], [lens[i] for i in rows], D ** -0.5, 0, n)
    r = ref.check(y[rows], wy, ty, what + " y")
    ref.check(lse[rows], wl, tl, what + " lse")
    note(f"  {what}: {r:.2f} of the tolerance")


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("D", [64, 128, 160, 256])
def test_decode_scale_codes(D, page):
    """Every E8M0 scale with every E4M3 code: one token of weight 1, whose value comes back.  Values are exact in bf16 down to
    its smallest subnormal, 2^-133: below that they are rounded to a multiple of it, twice at most.  From 2^128 on they are no
    bf16 values (an infinity, or a NaN by the weight's low part)."""
    note(f"scale codes D={D} page={page}")
    rounds = 256 // D + (256 % D > 0)
    codes = torch.arange(256)
    codes[0x7F], codes[0xFF] = 0, 0
    codes = torch.cat([codes, torch.zeros(rounds * D - 256, dtype=torch.long)]).view(rounds, D).to(torch.uint8)
    B = 255 * rounds
    k = torch.zeros(B, 1, page, D, dtype=torch.uint8)
    v = k.clone()
    v[:, 0, 0] = codes.repeat(255, 1)
    ks = torch.full((B, 1, page, D // 32), 127, dtype=torch.uint8)
    vs = ks.clone()
    vs[:, 0, 0] = torch.arange(255).repeat_interleave(rounds)[:, None].to(torch.uint8)
    cache = moe.KvCache(*(t.to(DEV) for t in (k, v, ks, vs)))
    table = torch.arange(B, dtype=torch.int32)[:, None]
    q = torch.ones(B, 1, D, dtype=torch.bfloat16, device=DEV)
    y, lse = moe.moe_attention_decode(q, cache, table.to(DEV), torch.ones(B, dtype=torch.int32, device=DEV), want_lse=True)
    torch.cuda.synchronize()
    want = ref.dequant(v[:, 0, 0], vs[:, 0, 0])
    y = y[:, 0].double().cpu()
    large = want.abs() >= 2.0 ** 128
    assert not bool(torch.isfinite(y[large]).any())
    # (a NaN or an infinity stays in its own value)
    small = ~large
    tol = torch.where(want.abs() < 2.0 ** -125, torch.tensor(2.0 ** -133, dtype=torch.float64), torch.tensor(0.0, dtype=torch.float64))
    ref.check(y[small], want[small], tol[small], "values")
    assert not bool(lse.any())


@pytest.mark.parametrize("code", [0, 1, 60, 180, 200])
def test_decode_key_scale_codes(code):
    """Keys of scales far from 127: one key of that scale among others whose scores are zero."""
    D, page, n = 128, 32, 70
    cache, table = make_cache([n], page, 2, D, "mxfp8", code)
    k, _, ks, _ = cache.tensors
    k.fill_(0)
    ks.fill_(code)
    at = (int(table[0, 1]), 5)
    k[at[0], :, at[1], 3] = 0x44  # 3
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 3] = 2.0 ** max(-120, min(120, 128 - code))
    run_decode(q, cache, table, [n], scale=0.25, what=f"key scale {code}")


def test_numbers_beyond_32_bits():
    """The C calls take 32-bit numbers: a larger one is refused, not taken without its upper half (2^32 + 5 as 5)."""
    cache, table = make_cache([40], 16, 2, 64, "bf16", 1)
    q = queries(1, 4, 64, torch.bfloat16, 2)
    t, n = table.to(DEV), torch.tensor([40], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    k = queries(1, 2, 64, torch.bfloat16, 3)
    for large in (1 << 31, 1 << 32, (1 << 32) + 5, 1 << 40):
        for call in (lambda: moe.moe_attention_decode(q, cache, t, n, max_len=large),
                     lambda: moe.moe_attention_decode(q, cache, t, n, window=large),
                     lambda: moe.moe_attention_prompt(q, k, k, cu, window=large)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
    wide = torch.zeros(1, 1 << 24, dtype=torch.int32, device=DEV)  # 2^24 pages of 256 tokens: max_len would be 0
    big = moe.KvCache.empty(1, 256, 2, 64)
    with pytest.raises(ValueError, match="32 bits"):
        moe.moe_attention_decode(q, big, wide, n)
    few = torch.zeros(1, 1, 8, dtype=torch.bfloat16, device=DEV)
    many = few.expand((1 << 32) + 1, 1, 8)
    with pytest.raises(ValueError, match="32 bits"):
        moe.moe_rope_cache(many, None, None, out=(many, None, None))
    with pytest.raises(ValueError, match="32 bits"):
        moe.moe_attention_prompt(few, many, many, cu)
    for bad in (dict(window=-1), dict(max_len=-1)):
        with pytest.raises(moe.MoEError):
            moe.moe_attention_decode(q, cache, t, n, **bad)
