"""Plain 64-bit forms of the calls in front of the layer (residual addition + RMS norm, routing by a rule, 4-bit
products), on the CPU, for their tests.  They share no code with the library."""
import math

import numpy as np



def half_step(dtype: str) -> float:
    """Largest relative error of one rounding to the type."""
    return {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}[dtype]


# ---------------------------------------------------------------------------------------------------- norm
def add_rms_norm(x, residual, w, eps):
    s = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * w.astype(np.float64)
    return s, y


def element_values(fmt: str) -> np.ndarray:
    """Value of every code of an MX element format (NaN codes as NaN)."""
    bits, mb, bias = {"fp8": (8, 3, 7), "fp6": (6, 3, 1), "fp4": (4, 1, 1)}[fmt]
    v = np.empty(1 << bits)
    for c in range(1 << bits):
        m, e = c & ((1 << mb) - 1), (c >> mb) & ((1 << (bits - 1 - mb)) - 1)
        mag = m * 2.0 ** (1 - bias - mb) if e == 0 else (1 + m / 2.0 ** mb) * 2.0 ** (e - bias)
        if fmt == "fp8" and (c & 0x7F) == 0x7F:
            mag = math.nan
        v[c] = -mag if c >> (bits - 1) else mag
    return v


def unpack_codes(codes: np.ndarray, fmt: str, K: int) -> np.ndarray:
    """[T][row bytes] packed rows -> integer codes [T][K]."""
    if fmt == "fp8":
        return codes.astype(np.int64)
    if fmt == "fp4":
        return np.stack([codes & 15, codes >> 4], 2).reshape(len(codes), K).astype(np.int64)
    bits = np.unpackbits(codes.reshape(len(codes), K // 32, 24), axis=2, bitorder="little").reshape(-1, K, 6)
    return (bits.astype(np.int64) << np.arange(6)).sum(2)


def check_mx(y, codes, scales, fmt, rel):
    """Codes and scales are those of y (64 bits, off by at most `rel` relative): the scale code is
    floor(log2 amax) - emax of an amax within rel, each element a nearest value of y / X within rel |y / X|."""
    T, K = y.shape
    emax = {"fp8": 8, "fp6": 2, "fp4": 2}[fmt]
    amax = np.abs(y).reshape(T, K // 32, 32).max(2)
    lo = np.where(amax > 0, np.floor(np.log2(np.maximum(amax * (1 - rel), 1e-300))) - emax + 127, 0)
    hi = np.where(amax > 0, np.floor(np.log2(np.maximum(amax * (1 + rel), 1e-300))) - emax + 127, 0)
    sc = scales.astype(np.int64)
    assert np.all((sc >= np.clip(lo, 0, 254)) & (sc <= np.clip(hi, 0, 254)))
    q = y / np.repeat(2.0 ** (sc - 127.0), 32, axis=1)
    c = unpack_codes(codes, fmt, K)
    table = element_values(fmt)
    values = np.unique(table[np.isfinite(table)])
    got = table[c]
    assert np.all(np.isfinite(got))
    at = np.clip(np.searchsorted(values, q), 1, len(values) - 1)
    nearest = np.minimum(np.abs(q - values[at - 1]), np.abs(q - values[at]))
    assert np.all(np.abs(got - q) <= nearest + 2 * rel * np.abs(q) + 1e-300)
    assert np.array_equal(np.signbit(got)[y != 0], np.signbit(y)[y != 0])


# ---------------------------------------------------------------------------------------------------- routing
def select(L, top_k, score="softmax", bias=None, n_groups=1, topk_groups=1, group_score="top2", renormalise=True,
           routed_scale=1.0, n_shared=0, shared_weight=1.0):
    """ids, weights, scores of the rule, expert by expert in extended precision."""
    L = L.astype(np.longdouble)
    T, E = L.shape
    per = E // n_groups
    b = np.zeros(E, np.longdouble) if bias is None else bias.astype(np.longdouble)
    ids = np.full((T, top_k + n_shared), -1, np.int64)
    wts = np.zeros((T, top_k + n_shared), np.float64)
    scores = np.zeros((T, E), np.float64)
    for t in range(T):
        fin = np.isfinite(L[t])
        s = np.zeros(E, np.longdouble)
        if score == "sigmoid":
            s[fin] = 1 / (1 + np.exp(-L[t][fin]))
        elif fin.any():
            e = np.exp(L[t][fin] - L[t][fin].max())
            s[fin] = e / e.sum()
        scores[t] = s
        with np.errstate(invalid="ignore"):
            order = L[t] if bias is None else s + b  # without a bias the logits order the experts
        avail = [i for i in range(E) if fin[i] and np.isfinite(b[i])]
        if topk_groups < n_groups:
            rank = []
            for g in range(n_groups):
                mine = [i for i in avail if i // per == g]
                if group_score == "max" and bias is None:
                    k = sorted((L[t][i] for i in mine), reverse=True)[:1]
                else:
                    k = sorted((s[i] + b[i] for i in mine), reverse=True)[:1 if group_score == "max" else 2]
                rank.append(sum(k) if k else -np.inf)
            kept = sorted(range(n_groups), key=lambda g: (-rank[g], g))[:topk_groups]
            avail = [i for i in avail if i // per in kept]
        pick = sorted(avail, key=lambda i: (-order[i], i))[:top_k]
        ids[t, :len(pick)] = pick
        den = sum(s[i] for i in pick) if renormalise else np.longdouble(1)
        for j, i in enumerate(pick):
            wts[t, j] = routed_scale * (s[i] / den) if den > 0 else 0.0
        ids[t, top_k:] = np.arange(E, E + n_shared)
        wts[t, top_k:] = shared_weight
    return ids, wts, scores


def rank_gap(L, score, bias, n_groups, topk_groups):
    """Distance between the last kept and the first dropped group's TOP2 rank, in extended precision (finite L)."""
    L = L.astype(np.longdouble)
    s = 1 / (1 + np.exp(-L)) if score == "sigmoid" else np.exp(L - L.max(1, keepdims=True))
    if score == "softmax":
        s = s / s.sum(1, keepdims=True)
    key = s if bias is None else s + bias.astype(np.longdouble)
    part = np.sort(key.reshape(len(L), n_groups, -1), 2)
    rank = np.sort(part[:, :, -1] + part[:, :, -2], 1)
    return (rank[:, -topk_groups] - rank[:, -topk_groups - 1]).astype(np.float64)


# ---------------------------------------------------------------------------------------------------- 4-bit weights
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def weights(fmt, N, K, rng):
    """Random codes, scales, zeros, tensor scale (as stored) and the decoded matrix in 64 bits."""
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    c = np.stack([codes & 15, codes >> 4], 2).reshape(N, K)
    zeros = ts = None
    if fmt == "mxfp4":
        scales = rng.integers(110, 130, (N, K // 32)).astype(np.uint8)
        w = E2M1[c] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, 1)
    elif fmt == "int4g32":
        h = (rng.standard_normal((N, K // 32)) * 0.02).astype(np.float16)
        scales = h.view(np.uint8).reshape(N, K // 16)
        zeros = rng.integers(0, 256, (N, (K // 32 + 1) // 2), dtype=np.uint8)
        z = np.stack([zeros & 15, zeros >> 4], 2).reshape(N, -1)[:, :K // 32]
        w = (c.astype(np.float64) - np.repeat(z, 32, 1)) * np.repeat(h.astype(np.float64), 32, 1)
    else:
        scales = rng.integers(0, 256, (N, K // 16), dtype=np.uint8)
        scales[(scales & 0x7F) == 0x7F] = 0x38
        ts = np.array([rng.uniform(0.5, 2.0)], np.float32)
        w = E2M1[c] * np.repeat(element_values("fp8")[scales], 16, 1) * np.float64(ts[0])
    return codes, scales, zeros, ts, w


def linear_tolerance(x, w, K, ref, dtype):
    """Sums of K exact products in fp32: at most one rounding for each of the K/32 matrix instructions of a chain
    and their 32-wide inner sums (counted as two), plus 32 for the joins, each below 2^-23 of the sum of
    magnitudes; then one multiplication, one addition and the output's rounding."""
    mag = np.abs(x) @ np.abs(w).T
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    return (K / 16 + 32) * 2.0 ** -23 * mag + np.abs(ref) * (half_step(dtype) + 2.0 ** -22) + tiny
