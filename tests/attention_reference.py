"""Plain 64-bit forms of rotary positions, of the 8-bit cache and of attention, on the CPU, for their tests, with the
tolerances of the attention kernels.  They share no code with the library."""
import math

import torch

import front_reference as ref

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NAMES = {v: k for k, v in TYPES.items()}
E4M3 = torch.from_numpy(ref.element_values("fp8"))


def angles(n, R, seed=0, base=10000.0):
    """fp32 tables of positions 0 .. n-1."""
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cos(a).float(), torch.sin(a).float()


def rope(x, cos, sin, positions, pairs):
    """x [T][heads][D] turned, in 64 bits."""
    x = x.double()
    R = 2 * cos.shape[1]
    c, s = (t.double()[positions.long()][:, None, :] for t in (cos, sin))
    at = torch.arange(R // 2)
    low, high = (at, at + R // 2) if pairs == "halves" else (2 * at, 2 * at + 1)
    y = x.clone()
    y[..., low] = x[..., low] * c - x[..., high] * s
    y[..., high] = x[..., high] * c + x[..., low] * s
    return y


def dequant(codes, scales):
    """E4M3 codes [..., D] and E8M0 scales [..., D/32] -> 64-bit values."""
    return E4M3[codes.long()] * torch.exp2(scales.double() - 127.0).repeat_interleave(32, -1)


def cache_rows(cache, pages, n):
    """K and V [n][heads][D] in 64 bits of the first n tokens on `pages`, and whether each one's page exists."""
    k, v, ks, vs = (None if t is None else t.cpu() for t in cache.tensors)
    j = torch.arange(n)
    page = pages.cpu().long()[j // cache.page_size]
    there = (page >= 0) & (page < cache.n_pages)
    page = page.clamp(0, cache.n_pages - 1)
    off = j % cache.page_size
    k, v = k[page, :, off], v[page, :, off]
    if ks is None:
        return k.double(), v.double(), there
    return dequant(k, ks[page, :, off]), dequant(v, vs[page, :, off]), there


def attend(q, k, v, seen, scale, t, p_step):
    """Queries q [i][Hq][D] over keys k, v [j][Hkv][D] where seen [i][j] -> (y, lse, tolerance of y, tolerance of lse) in
    64 bits.

    Tolerances, for 16-bit type t.  A score's fp32 sum of D products is off by at most (D + 2) 2^-24 sum |q k| scale.  Its
    exponent (base 2) adds the rounding of the reference and of the fma, 2^-24 (|s| + |m|) each over ln 2, and the
    exponential at most 2^-22; so a weight's relative error is e = 2 (...) once numerator and sum are divided.  The
    exponentials are rounded by p_step (relative), or by half the smallest fp16 subnormal.  Sums of n terms in fp32, with
    factors from a reference that rises at most n/32 times and from joining, add (3 n + 64) 2^-24 of the sum of magnitudes.
    y is rounded once."""
    q, k, v = q.double(), k.double(), v.double()
    nq, Hq, D = q.shape
    G = Hq // k.shape[1]
    n = max(1, k.shape[0])
    y, tol = torch.zeros(nq, Hq, D, dtype=torch.float64), torch.zeros(nq, Hq, D, dtype=torch.float64)
    lse, ltol = torch.full((nq, Hq), -math.inf, dtype=torch.float64), torch.zeros(nq, Hq, dtype=torch.float64)
    some = seen.any(1)
    h = ref.half_step(t)
    for x in range(Hq):
        kk, vv = k[:, x // G], v[:, x // G]
        s = (q[:, x] @ kk.T) * scale
        s = torch.where(seen, s, torch.tensor(-math.inf, dtype=torch.float64))
        if not bool(some.any()):
            continue
        top = s.max(1).values
        w = torch.softmax(s[some], 1)
        clean = torch.where(w > 0, torch.ones_like(w), torch.zeros_like(w))
        # a key of weight zero adds nothing, whatever its value
        vals = torch.where(seen[some].any(0)[:, None], vv, torch.zeros_like(vv))
        y[some, x] = w @ vals
        lse[:, x] = torch.where(some, torch.logsumexp(s, 1), torch.tensor(-math.inf, dtype=torch.float64))
        mag = scale * (q[:, x].abs() @ kk.abs().T)
        mag = torch.where(seen, mag, torch.zeros_like(mag))[some].max(1).values
        span = torch.where(seen, s.abs(), torch.zeros_like(s))[some].max(1).values
        e = (D + 2) * 2.0 ** -24 * mag + 4 * 2.0 ** -24 * span + 2.0 ** -22
        A = w @ vals.abs()
        big = (clean @ vals.abs())
        tol[some, x] = A * (p_step + 2 * e[:, None] + (3 * n + 64) * 2.0 ** -24) + y[some, x].abs() * h * 1.001 \
            + (big * 2.0 ** -25 + 2.0 ** -25 if t == "fp16" else 0.0)
        ltol[some, x] = e + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * lse[some, x].abs() + 2.0 ** -22
    return y, lse, tol, ltol


def prompt(q, k, v, cu_q, cu_k, scale, causal, window):
    """All sequences -> (y, lse, tolerances) on all rows; rows outside are NaN."""
    t = NAMES[q.dtype]
    q, k, v = q.cpu(), k.cpu(), v.cpu()
    out = [torch.full(s, math.nan, dtype=torch.float64) for s in (q.shape, q.shape[:2], q.shape, q.shape[:2])]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        p = torch.arange(q1 - q0)[:, None] + (k1 - k0) - (q1 - q0)
        j = torch.arange(k1 - k0)
        seen = j <= p if causal else (j >= 0).expand(q1 - q0, -1)
        if window:
            seen = seen & (j > p - window)
        if q1 > q0:
            r = attend(q[q0:q1], k[k0:k1], v[k0:k1], seen, scale, t, ref.half_step(t))
            for o, x in zip(out, r):
                o[q0:q1] = x
    return out


def decode(q, cache, table, lens, scale, window, max_len=None):
    t = NAMES[q.dtype]
    q, table = q.cpu(), table.cpu()
    out = [torch.zeros(s, dtype=torch.float64) for s in (q.shape, q.shape[:2], q.shape, q.shape[:2])]
    for b, n in enumerate(lens):
        n = max(0, n if max_len is None else min(n, max_len))
        k, v, seen = cache_rows(cache, table[b], n)
        if window:
            seen = seen & (torch.arange(n) >= n - window)
        v = torch.where(seen[:, None, None], v, torch.zeros_like(v))
        k = torch.where(seen[:, None, None], k, torch.zeros_like(k))
        # exponentials in two 16-bit parts: each rounding leaves half a step of what is left
        r = attend(q[b:b + 1], k, v, seen[None], scale, t, ref.half_step(t) ** 2)
        for o, x in zip(out, r):
            o[b:b + 1] = x
    return out


def check(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])
    live = tol > 0
    return float(((got - want).abs()[live] / tol[live]).max()) if bool(live.any()) else 0.0
