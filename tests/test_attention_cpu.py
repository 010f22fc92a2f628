"""Rotary positions, cache write and attention on the host: every documented refusal, with fake device pointers that
validation never dereferences, the binding's own checks, and the tests' reference forms (no GPU)."""
import ctypes
import math

import pytest
import torch

import attention_reference as ref
import mxfp4_routed_expert_router_amd as m

OK, NULL, SHAPE, BLOCK, ALIGN, DTYPE, TOPK, WORKSPACE = 0, 1, 2, 3, 4, 5, 6, 7
P = 0x7F0000000000
BF16, FP16, FP32 = 0, 1, 2


def heads(p=P, dt=BF16, ts=1024, hs=64):
    return m.moe_heads(p, dt, ts, hs)


def cache_desc(fmt=m.MOE_KV_BF16, **over):
    c = m.moe_kv_cache(fmt, 10, 16, 2, 64, P, P + (1 << 20), 2048, 1024, 64)
    if fmt == m.MOE_KV_MXFP8:
        c.k_scales, c.v_scales = P + (2 << 20), P + (3 << 20)
        c.s_page_stride, c.s_head_stride, c.s_token_stride = 64, 32, 2
    for k, v in over.items():
        setattr(c, k, v)
    return c


ref_ = lambda s: None if s is None else ctypes.byref(s)
CACHES = [dict(fmt=m.MOE_KV_BF16), dict(fmt=m.MOE_KV_FP16), dict(fmt=m.MOE_KV_MXFP8)]
BAD_CACHES = [(NULL, dict(k=None)), (NULL, dict(v=None)), (SHAPE, dict(n_pages=0)), (SHAPE, dict(page_size=0)),
              (SHAPE, dict(n_pages=1 << 27)), (SHAPE, dict(page_stride=-8)), (SHAPE, dict(token_stride=1 << 41)),
              (ALIGN, dict(k=P + 8)), (ALIGN, dict(v=P + 2)), (ALIGN, dict(page_stride=2044)), (ALIGN, dict(head_stride=4)),
              (ALIGN, dict(token_stride=68)), (DTYPE, dict(fmt=3)), (DTYPE, dict(fmt=-1))]


@pytest.mark.parametrize("fmt", [c["fmt"] for c in CACHES])
def test_rope_refusals(fmt):
    L = m.lib()

    def f(rope=m.moe_rope(P, P + 4096, 100, 64, 0), pos=P, T=4, nq=4, nkv=2, D=64, q=heads(), k=heads(), v=heads(),
          qo=heads(P + 0x10000), ko=None, vo=None, cache=cache_desc(fmt), slots=P):
        return L.moe_rope_cache(ref_(rope), pos, T, nq, nkv, D, ref_(q), ref_(k), ref_(v), ref_(qo), ref_(ko), ref_(vo),
                                ref_(cache), slots, None)

    assert f(T=0, q=None, k=None, rope=None, pos=None, cache=None) == OK
    R = lambda **k: m.moe_rope(*{**dict(cos=P, sin=P + 4096, n=100, r=64, pairs=0), **k}.values())
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(q=heads(None)), dict(k=heads(None)),
                dict(vo=heads(), v=None), dict(cache=None), dict(slots=None), dict(cache=None, slots=None),
                dict(pos=None), dict(rope=None), dict(rope=R(cos=None)), dict(rope=R(sin=None)), dict(ko=heads(None))):
        assert f(**bad) == NULL, bad
    for bad in (dict(T=-1), dict(nq=-1), dict(nkv=-1), dict(nq=0, nkv=0), dict(nq=1025), dict(D=0), dict(D=60), dict(D=264),
                dict(T=1 << 25), dict(rope=R(n=0)), dict(rope=R(r=0)), dict(rope=R(r=3)), dict(rope=R(r=66)),
                dict(q=heads(ts=-1)), dict(k=heads(hs=-1)), dict(v=heads(ts=1 << 41)), dict(nkv=1), dict(D=32),
                dict(q=heads(P), qo=heads(P, ts=2048)), dict(q=heads(P), qo=heads(P, dt=FP16))):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(q=heads(dt=3)), dict(qo=heads(P + 64, dt=-1)), dict(k=heads(dt=FP32)), dict(rope=R(pairs=2))):
        assert f(**bad) == DTYPE, bad
    for bad in (dict(q=heads(P + 1)), dict(qo=heads(P + 2, dt=FP32)), dict(pos=P + 2), dict(slots=P + 1),
                dict(rope=R(cos=P + 2)), dict(rope=R(sin=P + 1))):
        assert f(**bad) == ALIGN, bad
    for want, over in BAD_CACHES:
        assert f(cache=cache_desc(**{"fmt": fmt, **over})) == want, over
    if fmt == m.MOE_KV_MXFP8:
        assert f(cache=cache_desc(fmt, k_scales=None)) == NULL and f(cache=cache_desc(fmt, v_scales=None)) == NULL
        assert f(cache=cache_desc(fmt, head_dim=40), D=40, rope=R(r=40)) == BLOCK
        assert f(cache=cache_desc(fmt, s_page_stride=-1)) == SHAPE
        assert f(cache=cache_desc(fmt, token_stride=72)) == ALIGN
    else:
        assert f(cache=cache_desc(fmt, k_scales=P)) == DTYPE


def test_prompt_refusals():
    L = m.lib()

    def f(q=heads(), k=heads(), v=heads(), cq=P, ck=P, n=2, Tq=8, Tk=8, nq=4, nkv=2, D=64, scale=0.125, causal=1, window=0,
          y=heads(P + 0x10000), lse=None, ws=P, wsb=None):
        need = L.moe_attention_prompt_workspace_bytes(Tq, Tk, n, nq, nkv, D)
        return L.moe_attention_prompt(ref_(q), ref_(k), ref_(v), cq, ck, n, Tq, Tk, nq, nkv, D, scale, causal, window,
                                      ref_(y), lse, ws, need if wsb is None else wsb, None)

    assert f(Tq=0, q=None) == OK and f(n=0, q=None) == OK
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(y=None), dict(cq=None), dict(ck=None), dict(q=heads(None)),
                dict(k=heads(None)), dict(v=heads(None)), dict(y=heads(None))):
        assert f(**bad) == NULL, bad
    for bad in (dict(Tq=-1), dict(Tk=-1), dict(n=-1), dict(n=(1 << 20) + 1), dict(nq=0), dict(nkv=0), dict(nq=3),
                dict(nq=1026, nkv=2), dict(D=4), dict(D=65), dict(D=264), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38), dict(window=-1), dict(window=5, causal=0),
                dict(Tq=1 << 30), dict(Tq=1 << 24, Tk=(1 << 31) - 5, nq=4), dict(q=heads(ts=-8)), dict(v=heads(hs=1 << 41)),
                dict(Tq=1 << 21, nq=256, nkv=1), dict(Tq=8, Tk=(1 << 30) - 7)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(q=heads(dt=FP32)), dict(k=heads(dt=FP16)), dict(y=heads(dt=FP16)), dict(v=heads(dt=7)),
                dict(**{x: heads(dt=FP32) for x in "qkvy"})):
        assert f(**bad) == DTYPE, bad
    for bad in (dict(q=heads(P + 8)), dict(k=heads(ts=1028)), dict(v=heads(hs=68)), dict(y=heads(P + 2)), dict(cq=P + 2),
                dict(ck=P + 1), dict(lse=P + 2)):
        assert f(**bad) == ALIGN, bad
    need = L.moe_attention_prompt_workspace_bytes(1, 50000, 1, 4, 2, 64)
    assert need >= 4 * 66 * 4  # one row over many keys: several workgroups share them
    one = dict(Tq=1, Tk=50000, n=1)
    assert f(**one, ws=None) == WORKSPACE and f(**one, wsb=need - 1) == WORKSPACE and f(**one, ws=P + 8) == ALIGN
    for bad in ((0, 8, 1, 4, 2, 64), (8, -1, 1, 4, 2, 64), (8, 8, 0, 4, 2, 64), (8, 8, 1, 3, 2, 64), (8, 8, 1, 4, 2, 60)):
        assert L.moe_attention_prompt_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("fmt", [c["fmt"] for c in CACHES])
def test_decode_refusals(fmt):
    L = m.lib()
    dt = FP16 if fmt == m.MOE_KV_FP16 else BF16

    def f(q=heads(dt=dt), B=3, nq=4, cache=cache_desc(fmt), table=P, ts=10, width=10, lens=P, max_len=160, scale=0.125,
          window=0, y=heads(P + 0x10000, dt=dt), lse=None, ws=P, wsb=None):
        c = cache if cache is not None else cache_desc(fmt)
        need = L.moe_attention_decode_workspace_bytes(B, nq, c.n_kv_heads, c.head_dim, max_len)
        return L.moe_attention_decode(ref_(q), B, nq, ref_(cache), table, ts, width, lens, max_len, scale, window, ref_(y),
                                      lse, ws, need if wsb is None else wsb, None)

    assert f(B=0, q=None, cache=None) == OK
    for bad in (dict(q=None), dict(y=None), dict(cache=None), dict(q=heads(None, dt)), dict(y=heads(None, dt)),
                dict(table=None), dict(lens=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(B=-1), dict(nq=0), dict(nq=3), dict(nq=1026), dict(ts=-1), dict(ts=1 << 41), dict(width=-1),
                dict(max_len=161), dict(max_len=-1), dict(max_len=(1 << 30) + 1, width=1 << 28), dict(scale=0.0), dict(scale=math.nan), dict(window=-1),
                dict(B=1 << 22, nq=4), dict(q=heads(dt=dt, ts=-8)), dict(y=heads(dt=dt, hs=-8))):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(q=heads(dt=FP32)), dict(y=heads(dt=FP32)), dict(q=heads(dt=1 - dt)), dict(y=heads(dt=1 - dt))):
        assert f(**bad) == DTYPE, bad
    for bad in (dict(q=heads(P + 8, dt)), dict(q=heads(dt=dt, ts=1028)), dict(y=heads(P + 2, dt)), dict(table=P + 2),
                dict(lens=P + 1), dict(lse=P + 2)):
        assert f(**bad) == ALIGN, bad
    for want, over in BAD_CACHES:
        assert f(cache=cache_desc(**{"fmt": fmt, **over})) == want, over
    assert f(cache=cache_desc(fmt, head_dim=264)) == SHAPE and f(cache=cache_desc(fmt, n_kv_heads=0)) == SHAPE
    need = L.moe_attention_decode_workspace_bytes(1, 4, 2, 64, 5000)
    long = dict(B=1, width=400, max_len=5000)
    assert need > 0 and f(**long, ws=None) == WORKSPACE and f(**long, wsb=need - 1) == WORKSPACE
    assert f(**long, ws=P + 8) == ALIGN
    for bad in ((0, 4, 2, 64, 5000), (1, 3, 2, 64, 5000), (1, 4, 2, 64, 0), (1, 4, 2, 63, 5000)):
        assert L.moe_attention_decode_workspace_bytes(*bad) == 0


def test_outputs_that_overlap():
    """Rows of one output over each other (a broadcast one) would be written by several workgroups at once."""
    L = m.lib()
    out = P + 0x10000
    for ts, hs in ((0, 64), (256, 0), (32, 128), (256, 56)):
        y = heads(out, ts=ts, hs=hs)
        assert L.moe_attention_prompt(ref_(heads()), ref_(heads()), ref_(heads()), P, P, 2, 8, 8, 4, 2, 64, 0.125, 1, 0,
                                      ref_(y), None, None, 0, None) == SHAPE
        assert L.moe_attention_decode(ref_(heads()), 3, 4, ref_(cache_desc(m.MOE_KV_BF16)), P, 10, 10, P, 16, 0.125, 0,
                                      ref_(y), None, None, 0, None) == SHAPE
        for at in range(3):
            outs = [ref_(y if i == at else heads(out + 4096 * i)) for i in range(3)]
            assert L.moe_rope_cache(None, None, 4, 4, 2, 64, ref_(heads()), ref_(heads()), ref_(heads()), *outs, None, None,
                                    None) == SHAPE
    for fmt in (m.MOE_KV_BF16, m.MOE_KV_FP16, m.MOE_KV_MXFP8):
        names = ["page_stride", "head_stride", "token_stride"]
        for name in names + ["s_" + n for n in names] * (fmt == m.MOE_KV_MXFP8):
            assert L.moe_rope_cache(None, None, 4, 0, 2, 64, None, ref_(heads()), ref_(heads()), None, None, None,
                                    ref_(cache_desc(fmt, **{name: 0})), P, None) == SHAPE


def test_workspaces_stay_small():
    """The parts of a row are few where rows are many: a workspace never passes the 16-bit rows it serves by far."""
    L = m.lib()
    for B in (1, 7, 64, 300, 5000):
        for n in (1, 100, 4096, 131072, 1 << 22):
            need = L.moe_attention_decode_workspace_bytes(B, 64, 8, 128, n)
            assert need <= (64 << 20) + B * 64 * 130 * 4 * 16, (B, n, need)
    for Tq in (1, 100, 5000, 100000):
        for Tk in (1, 5000, 1 << 20):
            assert L.moe_attention_prompt_workspace_bytes(Tq, Tk, 4, 64, 8, 128) <= 512 << 20


def test_binding_refuses_what_it_can_see():
    """Shapes, types and devices that the C call could not tell from its pointers."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache = m.KvCache(bf(4, 2, 16, 64), bf(4, 2, 16, 64))
    assert (cache.n_pages, cache.n_kv_heads, cache.page_size, cache.head_dim, cache.fmt) == (4, 2, 16, 64, m.MOE_KV_BF16)
    mx = m.KvCache.empty(4, 16, 2, 64, "mxfp8", device="cpu")
    assert mx.fmt == m.MOE_KV_MXFP8 and mx.tensors[2].shape == (4, 2, 16, 2) and mx.act is torch.bfloat16
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    for bad in ((bf(4, 2, 16, 64), bf(4, 2, 16, 32)), (bf(4, 2, 64), bf(4, 2, 64)),
                (bf(4, 2, 16, 64), bf(4, 16, 2, 64).transpose(1, 2)), (bf(4, 2, 64, 16).transpose(2, 3),) * 2,
                (u8(4, 2, 16, 64), u8(4, 2, 16, 64)), (u8(4, 2, 16, 64), u8(4, 2, 16, 64), u8(4, 2, 16, 2), u8(4, 2, 16, 1)),
                (bf(4, 2, 16, 64), bf(4, 2, 16, 64), u8(4, 2, 16, 2), u8(4, 2, 16, 2))):
        with pytest.raises(ValueError):
            m.KvCache(*bad)
    for bad in ((bf(4, 2, 16, 64).float(),) * 2, (bf(4, 2, 16, 64), bf(4, 2, 16, 64).half())):
        with pytest.raises(TypeError):
            m.KvCache(*bad)
    with pytest.raises(KeyError):
        m.KvCache.empty(4, 16, 2, 64, "fp4", device="cpu")
    t = torch.zeros(10, 32)
    rope = m.Rope(t, t)
    assert rope.rotary_dim == 64
    for bad in ((t, t[:5]), (t, t.double()), (t[:, ::2], t[:, ::2]), (t[0], t[0])):
        with pytest.raises(ValueError):
            m.Rope(*bad)
    with pytest.raises(KeyError):
        m.Rope(t, t, "pairs")
    q, k = bf(3, 4, 64), bf(3, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        m.moe_rope_cache(q, k, k, rope, i32(3), cache, i32(3))
    with pytest.raises(ValueError):
        m.moe_rope_cache(None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        m.moe_attention_prompt(q, k, k, i32(2))
    with pytest.raises(ValueError, match="GPU"):
        m.moe_attention_decode(q, cache, i32(3, 2), i32(3))


def test_reference_forms():
    """The tests' own references on cases whose answers are known, and planted mistakes that they have to see."""
    cos, sin = ref.angles(50, 8)
    x = torch.randn(3, 2, 12, dtype=torch.float64)
    pos = torch.tensor([0, 7, 49], dtype=torch.int32)
    for pairs in ("halves", "neighbours"):
        y = ref.rope(x, cos, sin, pos, pairs)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 8:], x[..., 8:])
        assert torch.allclose(y[..., :8].norm(dim=2), x[..., :8].norm(dim=2), rtol=1e-6)
    assert not torch.allclose(ref.rope(x, cos, sin, pos, "halves"), ref.rope(x, cos, sin, pos, "neighbours"))
    assert float(ref.dequant(torch.full((1, 32), 0x38, dtype=torch.uint8), torch.full((1, 1), 128, dtype=torch.uint8))[0, 0]) == 2.0
    # equal scores: the mean of what is seen; no key: zeros and -inf
    q, k = torch.zeros(4, 2, 8).bfloat16(), torch.zeros(4, 1, 8).bfloat16()
    v = torch.arange(4.0)[:, None, None].expand(4, 1, 8).bfloat16()
    y, lse, ty, tl = ref.prompt(q, k, v, [0, 4], [0, 4], 1.0, True, 2)
    assert torch.equal(y[:, 0, 0], torch.tensor([0.0, 0.5, 1.5, 2.5], dtype=torch.float64))
    assert torch.allclose(lse[:, 1], torch.log(torch.tensor([1.0, 2, 2, 2], dtype=torch.float64)))
    y, lse, _, _ = ref.prompt(q, k, v, [0, 3], [0, 2], 1.0, True, 0)
    assert not bool(y[0].any()) and bool((lse[0] == -math.inf).all()) and bool(torch.isnan(y[3]).all())
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(20, h, 16, generator=g).bfloat16() for h in (2, 1, 1))
    y, lse, ty, tl = ref.prompt(q, k, v, [0, 20], [0, 20], 0.25, True, 0)
    wrong, wl, _, _ = ref.prompt(q, k, v, [0, 20], [0, 20], 0.25, True, 19)  # one key of the last row left out
    ref.check(y, y, ty, "same")
    with pytest.raises(AssertionError):
        ref.check(wl, lse, tl, "planted")
    pages = torch.tensor([[2, 0, 7]])
    c = m.KvCache(torch.randn(3, 1, 4, 8).bfloat16(), torch.randn(3, 1, 4, 8).bfloat16())
    kk, vv, there = ref.cache_rows(c, pages[0], 9)
    assert torch.equal(kk[5], c.tensors[0][0, :, 1].double()) and there.tolist() == [True] * 8 + [False]


def test_outputs_whose_strides_do_not_nest():
    """Each stride alone steps over a row, but two of them together come back to the same memory: (t, h + 1) is (t + 1, h)."""
    L = m.lib()
    out = P + 0x10000

    def rows_refused(ts, hs, T=8, n=4):
        y, x = heads(out, ts=ts, hs=hs), heads(ts=4096)
        got = {L.moe_attention_prompt(ref_(x), ref_(x), ref_(x), P, P, 2, T, 8, n, 2, 64, 0.125, 1, 0, ref_(y), None, None, 0,
                                      None),
               L.moe_attention_decode(ref_(x), T, n, ref_(cache_desc(m.MOE_KV_BF16)), P, 10, 10, P, 16, 0.125, 0, ref_(y), None,
                                      None, 0, None)}
        for at in range(3):
            outs = [ref_(y if i == at else heads(out + (1 << 20) * (i + 1), ts=4096)) for i in range(3)]
            got.add(L.moe_rope_cache(None, None, T, n, n, 64, ref_(x), ref_(x), ref_(x), *outs, None, None, None))
        return got == {SHAPE}

    for ts, hs in ((64, 64), (192, 64), (64, 448), (128, 128), (248, 64), (72, 64), (64, 504)):
        assert rows_refused(ts, hs), (ts, hs)

    def cache_refused(fmt, **over):
        k = heads(ts=4096)
        return L.moe_rope_cache(None, None, 4, 0, 2, 64, None, ref_(k), ref_(k), None, None, None, ref_(cache_desc(fmt, **over)),
                                P, None) == SHAPE

    for fmt in (m.MOE_KV_BF16, m.MOE_KV_FP16, m.MOE_KV_MXFP8):
        # ten pages of 16 tokens and 2 heads of 64
        for over in (dict(page_stride=1024), dict(page_stride=2032), dict(head_stride=64), dict(head_stride=1008),
                     dict(token_stride=128), dict(token_stride=1024), dict(page_stride=64), dict(token_stride=2048, head_stride=64),
                     dict(page_stride=1 << 40, head_stride=1 << 40), dict(head_stride=1 << 40, token_stride=1 << 40)):
            assert cache_refused(fmt, **over), over
    for over in (dict(s_page_stride=32), dict(s_page_stride=62), dict(s_head_stride=2), dict(s_token_stride=4),
                 dict(s_head_stride=2, s_token_stride=2)):
        assert cache_refused(m.MOE_KV_MXFP8, **over), over


def test_nesting_against_all_rows():
    """What passes the check lies apart by the list of all rows.  (Passing calls end at their missing workspace.)"""
    L = m.lib()
    Tq, Tk, n, D = 3, 50000, 4, 8
    assert L.moe_attention_prompt_workspace_bytes(Tq, Tk, 1, n, 2, D) > 0
    x = heads(ts=64, hs=8)
    some = 0
    for ts in range(0, 121, 8):
        for hs in range(0, 121, 8):
            st = L.moe_attention_prompt(ref_(x), ref_(x), ref_(x), P, P, 1, Tq, Tk, n, 2, D, 0.125, 1, 0,
                                        ref_(heads(P + 0x100000, ts=ts, hs=hs)), None, None, 0, None)
            nested = (ts >= (n - 1) * hs + D and hs >= D) or (hs >= (Tq - 1) * ts + D and ts >= D)
            assert st == (WORKSPACE if nested else SHAPE), (ts, hs, st)
            at = sorted(i * ts + j * hs for i in range(Tq) for j in range(n))
            assert not nested or all(b - a >= D for a, b in zip(at, at[1:])), (ts, hs)
            some += nested
    assert some > 50


def test_workspace_queries_are_not_kept_without_end():
    """A server that passes each step's longest length asks for a new size every step."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    cache = m.KvCache(bf(4, 2, 16, 64), bf(4, 2, 16, 64))
    L = m.lib()
    sizes = set()
    for n in list(range(1, 5000)) + [7, 4999]:
        got = m.moe_attention_decode_workspace_bytes(3, 4, cache, n)
        assert got == L.moe_attention_decode_workspace_bytes(3, 4, 2, 64, n)
        sizes.add(got)
    assert len(sizes) > 10
    held = sum(len(v) for v in vars(cache).values() if isinstance(v, (dict, list, set)))
    assert held <= 64, held


def test_rope_without_key_value_heads_uses_none_of_their_pointers():
    """n_kv_heads 0: k, v and their outputs do not count, whatever they are.  (The calls end at the misaligned table.)"""
    L = m.lib()
    bad = m.moe_rope(P + 2, P + 4096, 100, 64, 0)
    for k, v, ko, vo in ((None, None, None, heads()), (None, None, heads(), heads()), (heads(None), None, None, heads(None)),
                         (None, heads(dt=7), None, None)):
        assert L.moe_rope_cache(ref_(bad), P, 4, 4, 0, 64, ref_(heads()), ref_(k), ref_(v), ref_(heads(P + 0x10000)), ref_(ko),
                                ref_(vo), None, None, None) == ALIGN
