"""moe_rope_cache on the GPU against 64 bits (needs an MI355X).

Tolerances.  A turned value is two fp32 products and their sum, 2^-24 of each product and of the sum: at most 2^-23
(|a c| + |b s|) in all; values that do not turn are exact in fp32.  One rounding to the output's type follows."""
import numpy as np
import pytest
import torch

import attention_reference as ref
import front_reference as front
import mxfp4_routed_expert_router_amd as moe
from gpu_support import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES
N = 5000


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(T, Hq, Hkv, D, R, x, fmt, pairs="halves", page=16, order="head", seed=0, fused=True, positions=None):
    g = torch.Generator().manual_seed(seed)
    if fused:  # parts of one product's output
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).mul(3.0).to(TYPES[x]).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (torch.randn(T, h, D, generator=g).to(TYPES[x]).to(DEV) for h in (Hq, Hkv, Hkv))
    cos, sin = ref.angles(N, R)
    rope = moe.Rope(cos.to(DEV), sin.to(DEV), pairs)
    pos = torch.randint(0, N, (T,), generator=g, dtype=torch.int32) if positions is None else positions
    n_pages = (T + page - 1) // page + 2
    slots = torch.randperm(n_pages * page, generator=g)[:T].int()
    shape = (n_pages, Hkv, page, D)
    like = lambda s, t: torch.full(s, 3, dtype=t, device=DEV)
    if order == "token":
        like = lambda s, t: torch.full((s[0], s[2], s[1], s[3]), 3, dtype=t, device=DEV).permute(0, 2, 1, 3)
    if fmt == "mxfp8":
        sc = shape[:3] + (D // 32,)
        cache = moe.KvCache(like(shape, torch.uint8), like(shape, torch.uint8), like(sc, torch.uint8),
                            like(sc, torch.uint8))
    else:
        cache = moe.KvCache(like(shape, TYPES[fmt]), like(shape, TYPES[fmt]))
    return q, k, v, rope, cos, sin, pos, cache, slots


def tolerance(x, y, cos, sin, pos, pairs, t, turn=True):
    """Of the turned rows y of x in type t."""
    tol = torch.zeros_like(y)
    if turn:
        size = ref.rope(x.abs(), cos.abs(), -sin.abs(), pos, pairs).abs()  # |a c| + |b s| for the first of a pair
        size = torch.maximum(size, ref.rope(x.abs(), cos.abs(), sin.abs(), pos, pairs).abs())  # and for the second
        tol = size * 2.0 ** -23
    return tol + y.abs() * front.half_step(t) * (1 + 2.0 ** -20) + (2.0 ** -25 if t == "fp16" else 0.0)


def check(T, Hq, Hkv, D, R, x="fp32", fmt="bf16", pairs="halves", page=16, order="head", seed=0, fused=True):
    what = f"rope T={T} heads={Hq}/{Hkv} D={D} R={R} {x} -> {fmt} {pairs} page={page} {order}"
    note(what)
    q, k, v, rope, cos, sin, pos, cache, slots = make(T, Hq, Hkv, D, R, x, fmt, pairs, page, order, seed, fused)
    out = moe.moe_rope_cache(q, k, v, rope, pos.to(DEV), cache, slots.to(DEV))
    torch.cuda.synchronize()
    t = ref.NAMES[cache.act]
    rows = {}
    for name, got, x0, turn in zip("qkv", out, (q, k, v), (True, True, False)):
        x0 = x0.cpu().double()
        want = ref.rope(x0, cos, sin, pos, pairs) if turn else x0
        assert got.dtype == cache.act
        ref.check(got, want, tolerance(x0, want, cos, sin, pos, pairs, t, turn), f"{what} {name}")
        rows[name] = (want, x0)
    page_of, off = slots.long() // page, slots.long() % page
    for name, got, sc in zip("kv", cache.tensors[:2], cache.tensors[2:]):
        got = got.cpu()
        want, x0 = rows[name]
        held = got[page_of, :, off]
        if fmt == "mxfp8":
            s = sc.cpu()
            # relative to a block's largest magnitude the fp32 error is at most 2^-22 (a turned value may cancel)
            a = held.reshape(T * Hkv, D).numpy()
            front.check_mx(want.reshape(T * Hkv, D).numpy(), a, s[page_of, :, off].reshape(T * Hkv, -1).numpy(), "fp8",
                           2.0 ** -16)
            s[page_of, :, off] = 3
            assert bool((s == 3).all())
        else:
            ref.check(held, want, tolerance(x0, want, cos, sin, pos, pairs, fmt, name == "k"), f"{what} cache {name}")
            assert torch.equal(held, out[1 if name == "k" else 2].cpu())
        got[page_of, :, off] = 3  # nothing else was written
        assert bool((got == 3).all())


@pytest.mark.parametrize("T", [1, 2, 5, 64, 177])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
def test_tokens(T, fmt):
    check(T, 8, 2, 128, 128, fmt=fmt, seed=T)


@pytest.mark.parametrize("D,R", [(8, 8), (8, 2), (16, 16), (24, 24), (64, 64), (64, 48), (72, 36), (80, 80), (96, 96), (96, 32),
                                 (128, 64), (128, 10), (200, 200), (256, 256), (256, 128), (192, 64)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_head_sizes(D, R, pairs):
    check(7, 5, 3, D, R, pairs=pairs, seed=D)
    if D % 32 == 0:
        check(7, 5, 3, D, R, pairs=pairs, seed=D, fmt="mxfp8", x="bf16")


@pytest.mark.parametrize("x", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", ["bf16", "fp16", "mxfp8"])
@pytest.mark.parametrize("order", ["head", "token"])
def test_types_and_orders(x, fmt, order):
    check(20, 6, 3, 64, 64, x, fmt, order=order, fused=False)
    check(20, 6, 3, 64, 32, x, fmt, "neighbours", page=5, order=order)


@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 1), (64, 8, 64), (16, 16, 48), (40, 1, 100)])
def test_heads_and_pages(Hq, Hkv, page):
    check(33, Hq, Hkv, 64, 64, "bf16", "mxfp8", page=page)


@pytest.mark.parametrize("D,R", [(64, 64), (96, 96), (96, 20), (128, 64), (256, 256), (200, 200), (24, 10)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_in_place(D, R, pairs, x):
    """q, k and v turned where they are: the same bits as into other buffers."""
    q, k, v, rope, cos, sin, pos, cache, slots = make(50, 6, 2, D, R, x, "bf16", pairs)
    other = tuple(torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in (q, k, v))
    moe.moe_rope_cache(q, k, v, rope, pos.to(DEV), out=other)
    want = [t.clone() for t in other]
    moe.moe_rope_cache(q, k, v, rope, pos.to(DEV), out=(q, k, v))
    torch.cuda.synchronize()
    for a, b in zip((q, k, v), want):
        assert torch.equal(a, b)


def test_far_positions_and_padding():
    """Positions outside the table are padding: no output of theirs is written.  Slots outside the cache likewise."""
    T = 9
    pos = torch.tensor([0, N - 1, N, -1, 17, 1 << 30, -(1 << 31), 3, 4], dtype=torch.int32)
    q, k, v, rope, cos, sin, _, cache, slots = make(T, 4, 2, 64, 64, "fp32", "bf16", positions=pos)
    slots[7], slots[8] = -1, cache.n_pages * cache.page_size
    out = tuple(torch.full(t.shape, 5.0, dtype=torch.bfloat16, device=DEV) for t in (q, k, v))
    moe.moe_rope_cache(q, k, v, rope, pos.to(DEV), cache, slots.to(DEV), out=out)
    torch.cuda.synchronize()
    good = (pos >= 0) & (pos < N)
    for got, x0, turn in zip(out, (q, k, v), (True, True, False)):
        assert bool((got[~good.to(DEV)] == 5.0).all())
        x0 = x0.cpu().double()[good]
        want = ref.rope(x0, cos, sin, pos[good], "halves") if turn else x0
        ref.check(got.cpu()[good], want, tolerance(x0, want, cos, sin, pos[good], "halves", "bf16", turn), "padding")
    written = torch.zeros(cache.n_pages * cache.page_size, dtype=torch.bool)
    written[slots[:7][good[:7]].long()] = True
    held = cache.tensors[0].cpu().transpose(1, 2).flatten(0, 1)
    assert bool((held[~written] == 3).all()) and bool((held[written] != 3).any(2).any(1).all())


def test_parts_alone():
    """q alone, k and v alone, a write without turning, some outputs left out."""
    q, k, v, rope, cos, sin, pos, cache, slots = make(30, 4, 2, 64, 64, "bf16", "bf16")
    p, s = pos.to(DEV), slots.to(DEV)
    both = moe.moe_rope_cache(q, k, v, rope, p, cache, s)
    held = [t.clone() for t in cache.tensors[:2]]
    assert torch.equal(moe.moe_rope_cache(q, None, None, rope, p)[0], both[0])
    kv = moe.moe_rope_cache(None, k, v, rope, p)
    assert kv[0] is None and torch.equal(kv[1], both[1]) and torch.equal(kv[2], both[2])
    assert torch.equal(moe.moe_rope_cache(None, k, None, rope, p)[1], both[1])
    for t in cache.tensors[:2]:
        t.fill_(3)
    moe.moe_rope_cache(None, k, v, rope, p, cache, s, out=(None, None, None))
    assert torch.equal(cache.tensors[0], held[0]) and torch.equal(cache.tensors[1], held[1])
    moe.moe_rope_cache(None, k, v, None, None, cache, s, out=(None, None, None))
    pg, of = slots.long() // 16, slots.long() % 16
    assert torch.equal(cache.tensors[0].cpu()[pg, :, of], k.cpu()) and torch.equal(cache.tensors[1].cpu()[pg, :, of], v.cpu())


def test_far_cache():
    """Slots beyond 2^31 values."""
    page, Hkv, D = 64, 8, 256
    n_pages = (1 << 31) // (page * Hkv * D) + 40
    cache = moe.KvCache.empty(n_pages, page, Hkv, D)
    k = torch.randn(70, Hkv, D, device=DEV).bfloat16()
    v = torch.randn(70, Hkv, D, device=DEV).bfloat16()
    slots = torch.arange(n_pages * page - 70, n_pages * page, dtype=torch.int32, device=DEV)
    moe.moe_rope_cache(None, k, v, cache=cache, slots=slots, out=(None, None, None))
    last = cache.tensors[0][-2:].transpose(1, 2).flatten(0, 1)[-70:]
    assert torch.equal(last, k) and torch.equal(cache.tensors[1][-2:].transpose(1, 2).flatten(0, 1)[-70:], v)


def test_zero_values():
    """Blocks of zeros: codes 0 with scale code 0."""
    q, k, v, rope, cos, sin, pos, cache, slots = make(3, 2, 2, 64, 64, "fp32", "mxfp8")
    k = torch.zeros_like(k)
    moe.moe_rope_cache(None, k, k, rope, pos.to(DEV), cache, slots.to(DEV))
    pg, of = slots.long() // 16, slots.long() % 16
    for t in cache.tensors:
        got = t.cpu()[pg, :, of]
        assert bool(((got == 0) | (got == 128)).all() if t.shape[3] == 64 else (got == 0).all())


def test_more_tokens_than_a_launch():
    """Two launches: tokens around the seam and at the end."""
    T = (1 << 24) + 37
    k = torch.randn(T, 1, 8, device=DEV).bfloat16()
    cos, sin = ref.angles(N, 8)
    rope = moe.Rope(cos.to(DEV), sin.to(DEV))
    pos = (torch.arange(T, device=DEV) % N).int()
    _, got, _ = moe.moe_rope_cache(None, k, None, rope, pos)
    for at in (slice(0, 50), slice((1 << 24) - 50, (1 << 24) + 37)):
        _, want, _ = moe.moe_rope_cache(None, k[at].clone(), None, rope, pos[at].clone())
        assert torch.equal(got[at], want)
