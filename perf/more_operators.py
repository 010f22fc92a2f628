"""The attention half of a routed-MoE block, measured: rotary positions with the write into a paged key-value cache
(`moe_rope_cache`), attention of one new token per sequence over that cache (`moe_attention_decode`), and attention
over whole prompts, packed one after another (`moe_attention_prompt`).

`own` chooses between the plain forms (elementary torch operations) and the library's kernels.  `listed()` and
`draw()` give cases, `prepare()` makes a case's inputs from a seed, `run()` is one call, `work()` the bytes and
operations that one call cannot do without, `exact()` the outputs in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------------------------------------------
# cases
def _rope(T, Hq, Hkv, D, R, x, fmt, page, pairs="halves", packed=False):
    """x: type of q, k and v; fmt: of the cache; packed: the rotated k and the v are wanted as 16-bit rows too."""
    return {"op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "x": x, "fmt": fmt, "page": page,
            "pairs": pairs, "packed": packed}


def _decode(B, n, Hq, Hkv, D, fmt, page, window=0, lse=False, idle=False):
    """B sequences of 1 .. n cached tokens (the longest n; with idle every fifth one has none)."""
    return {"op": "decode", "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "fmt": fmt, "page": page, "window": window,
            "lse": lse, "idle": idle}


def _prompt(B, n, past, Hq, Hkv, D, dt, causal=True, window=0, lse=False):
    """B prompts of 1 .. n tokens (the longest n), each behind `past` earlier keys."""
    return {"op": "prompt", "B": B, "n": n, "past": past, "Hq": Hq, "Hkv": Hkv, "D": D, "dt": dt, "causal": causal,
            "window": window, "lse": lse}


def listed():
    return [
        # one decoded token: the fp32 output of its projection, rotated, into a bf16 cache
        dict(_rope(1, 64, 8, 128, 128, "fp32", "bf16", 64), name="rope T1 bf16"),
        # a decode batch into an 8-bit cache, half of each head rotated in neighbouring pairs
        dict(_rope(176, 64, 8, 128, 64, "bf16", "mxfp8", 64, "neighbours"), name="rope T176 mxfp8"),
        # a prompt, whose attention also reads the 16-bit rows
        dict(_rope(8192, 64, 8, 128, 128, "bf16", "bf16", 64, packed=True), name="rope T8192 bf16"),
        # one user's next token, a short context
        dict(_decode(1, 777, 64, 8, 128, "bf16", 64), name="decode B1 n777 bf16"),
        # the decode sweep's batch, contexts of up to 4096 tokens
        dict(_decode(176, 4096, 64, 8, 128, "bf16", 64, idle=True), name="decode B176 n4096 bf16"),
        # three long contexts in an 8-bit cache, statistics kept for joining with another device's share
        dict(_decode(3, 131072, 64, 8, 128, "mxfp8", 128, lse=True), name="decode B3 n131072 mxfp8"),
        # one key-value head per query head, heads of 96, a sliding window, pages of 48
        dict(_decode(33, 5001, 24, 24, 96, "fp16", 48, window=1000), name="decode B33 n5001 D96 fp16"),
        # one short prompt
        dict(_prompt(1, 301, 0, 64, 8, 128, "bf16"), name="prompt B1 n301"),
        # prompts of 1 to 4096 tokens, packed
        dict(_prompt(8, 4096, 0, 64, 8, 128, "bf16", lse=True), name="prompt B8 n4096"),
        # one long prompt
        dict(_prompt(1, 16384, 0, 64, 8, 128, "bf16"), name="prompt B1 n16384"),
        # a small model: one key-value head per query head, heads of 64, a sliding window
        dict(_prompt(5, 2500, 0, 16, 16, 64, "fp16", window=512), name="prompt B5 n2500 D64 fp16"),
        # the last piece of a prompt that is taken in pieces
        dict(_prompt(1, 128, 16000, 64, 8, 128, "bf16"), name="prompt B1 n128 past16000"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _draw(rng)
    most = [work(x) for x in listed() if x["op"] == c["op"]]
    while any(work(c)[u] > max(w[u] for w in most) for u in ("bytes", "flops")):  # no more than the largest listed one
        size = "T" if c["op"] == "rope" else "n"
        c[size] = max(1, c[size] * 4 // 5)
        if c.get("past"):
            c["past"] = c["past"] * 4 // 5
        if c.get("window"):
            c["window"] = max(1, c["window"] * 4 // 5)
    return c


def _draw(rng):
    op = rng.choice(["rope", "decode", "prompt"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
    while Hkv * G > 64:
        G = rng.choice([1, 2, 4])
    Hq = Hkv * G
    D = rng.choice([64, 96, 128, 128, 128, 192, 256])
    if op == "rope":
        fmt = rng.choice(["bf16", "fp16", "mxfp8"])
        x = rng.choice([fmt, "fp32"]) if fmt != "mxfp8" else rng.choice(["bf16", "fp32"])
        T = _log(rng, 1, min(8192, 8192 * 80 * 128 // ((Hq + 2 * Hkv) * D * (BYTES[x] // 2))))
        return _rope(T, Hq, Hkv, D, rng.choice([D, D // 2]), x, fmt, rng.choice([16, 48, 64, 128]),
                     rng.choice(["halves", "neighbours"]), rng.random() < 0.5)
    if op == "decode":
        fmt = rng.choice(["bf16", "fp16", "mxfp8"])
        B = _log(rng, 1, 256)
        n = _log(rng, 1, min(131072, 176 * 4096 * 8 * 128 // (B * Hkv * D), 176 * 4096 * 64 * 128 // (B * Hq * D)))
        lse = rng.random() < 0.3
        return _decode(B, n, Hq, Hkv, D, fmt, rng.choice([16, 48, 64, 128]),
                       max(1, n // 3) if rng.random() < 0.3 else 0, lse, not lse and rng.random() < 0.5)
    causal = rng.random() < 0.75
    B = _log(rng, 1, 32)
    most = 16384 ** 2 * 64 * 128 // (B * Hq * D * (1 if causal else 2))
    n = _log(rng, 1, min(16384, math.isqrt(most)))
    past = _log(rng, 1, 16384) if rng.random() < 0.3 else 0
    while past and 2 * n * (n + past) > most:
        past //= 2
    return _prompt(B, n, past, Hq, Hkv, D, rng.choice(["bf16", "fp16"]), causal,
                   max(1, (n + past) // 4) if causal and rng.random() < 0.3 else 0, rng.random() < 0.3)


def _lengths(B, n, idle=False):
    """Lengths of B sequences, spread over 1 .. n; the middle one has n."""
    r = [1 + int((n - 1) * ((i + 1) * GOLDEN % 1.0)) for i in range(B)]
    if idle:
        r = [0 if i % 5 == 4 else v for i, v in enumerate(r)]
    r[B // 2] = n
    return r


# ---------------------------------------------------------------------------------------------------------------
# inputs
def _pool(c, g, n_pages, fill):
    """Pages of a cache, [n_pages][Hkv][page][D], and the scales of an 8-bit one.  Values as a norm and a rotation
    leave them, or zeros."""
    shape = (n_pages, c["Hkv"], c["page"], c["D"])
    if c["fmt"] != "mxfp8":
        if not fill:
            return torch.zeros(shape, dtype=DTYPES[c["fmt"]], device=DEV), None
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[c["fmt"]]), None
    scales = torch.zeros(shape[:3] + (c["D"] // 32,), dtype=torch.uint8, device=DEV)
    codes = torch.zeros(shape, dtype=torch.uint8, device=DEV)
    if fill:  # blocks whose largest magnitude is between 1 and 4
        scales = torch.randint(119, 121, scales.shape, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        for p in range(0, n_pages, 4096):  # (in parts: random numbers are made in 32 bits)
            part = torch.randn((min(4096, n_pages - p),) + shape[1:], generator=g, device=DEV, dtype=torch.float32)
            codes[p:p + 4096] = (128.0 * part).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)

    if own:
        import mxfp4_routed_expert_router_amd as moe
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    s = {"case": dict(c)}
    if c["op"] == "rope":
        T, R, page = c["T"], c["R"], c["page"]
        act = torch.float16 if c["fmt"] == "fp16" else torch.bfloat16
        # one product's output holds q, k and v of a token
        qkv = normal(T, Hq + 2 * Hkv, D).to(DTYPES[c["x"]])
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        n_positions = 32768
        freq = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        angle = torch.arange(n_positions, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
        # a prompt's positions follow one another; those of a batch of single tokens do not
        first = int(torch.randint(0, n_positions - T, (1,), generator=g, device=DEV))
        s["positions"] = torch.arange(first, first + T, dtype=torch.int32, device=DEV)
        if T <= 256:
            s["positions"] = torch.randint(0, n_positions, (T,), generator=g, device=DEV, dtype=torch.int32)
        n_pages = (T + page - 1) // page + 3
        order = torch.randperm(n_pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + page // 2
        s["slots"] = (order[at // page] * page + at % page).int()
        s["kc"], s["ks"] = _pool(c, g, n_pages, False)
        s["vc"], s["vs"] = _pool(c, g, n_pages, False)
        s["out"] = tuple(torch.empty(T, h, D, dtype=act, device=DEV) if want else None
                         for h, want in ((Hq, True), (Hkv, c["packed"]), (Hkv, c["packed"])))
        if own:
            s["rope"] = moe.Rope(s["cos"], s["sin"], c["pairs"])
            s["cache"] = moe.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
    elif c["op"] == "decode":
        B, page = c["B"], c["page"]
        act = torch.float16 if c["fmt"] == "fp16" else torch.bfloat16
        lens = _lengths(B, c["n"], c["idle"])
        width = (c["n"] + page - 1) // page
        pages = [(n + page - 1) // page for n in lens]
        n_pages = sum(pages) + 2
        order = torch.randperm(n_pages, generator=g, device=DEV).int()
        s["table"] = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, m in enumerate(pages):
            s["table"][b, :m] = order[at:at + m]
            at += m
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = 2.0 * normal(B, Hq, D)
        s["q"] = s["q"].to(act)
        s["kc"], s["ks"] = _pool(c, g, n_pages, True)
        s["vc"], s["vs"] = _pool(c, g, n_pages, True)
        s["out"] = (torch.empty(B, Hq, D, dtype=act, device=DEV),
                    torch.empty(B, Hq, dtype=torch.float32, device=DEV) if c["lse"] else None)
        if own:
            s["cache"] = moe.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
            need = moe.moe_attention_decode_workspace_bytes(B, Hq, s["cache"], c["n"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    else:
        B, dt = c["B"], DTYPES[c["dt"]]
        s["nq"] = _lengths(B, c["n"])
        s["nk"] = [n + c["past"] for n in s["nq"]]
        cu = lambda lens: torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(device=DEV, dtype=torch.int32)
        s["cu_q"], s["cu_k"] = cu(s["nq"]), cu(s["nk"])
        Tq, Tk = sum(s["nq"]), sum(s["nk"])
        s["q"] = (2.0 * normal(Tq, Hq, D)).to(dt)
        s["k"], s["v"] = normal(Tk, Hkv, D).to(dt), normal(Tk, Hkv, D).to(dt)
        s["out"] = (torch.empty(Tq, Hq, D, dtype=dt, device=DEV),
                    torch.empty(Tq, Hq, dtype=torch.float32, device=DEV) if c["lse"] else None)
        if own:
            need = moe.moe_attention_prompt_workspace_bytes(Tq, Tk, B, Hq, Hkv, D)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
def _cache_outputs(s):
    if s["ks"] is None:
        return {"k_cache": s["kc"], "v_cache": s["vc"]}
    return {"k_cache": s["kc"].view(torch.float8_e4m3fn), "v_cache": s["vc"].view(torch.float8_e4m3fn),
            "k_scales": s["ks"].view(torch.float8_e8m0fnu), "v_scales": s["vs"].view(torch.float8_e8m0fnu)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "decode": _plain_decode, "prompt": _plain_prompt}[c["op"]](s)
    import mxfp4_routed_expert_router_amd as moe
    if c["op"] == "rope":
        q, k, v = moe.moe_rope_cache(s["q"], s["k"], s["v"], s["rope"], s["positions"], s["cache"], s["slots"],
                                     out=s["out"])
        return {"q": q, "k": k, "v": v, **_cache_outputs(s)}
    if c["op"] == "decode":
        y, lse = moe.moe_attention_decode(s["q"], s["cache"], s["table"], s["lens"], max_len=c["n"],
                                          window=c["window"], out=s["out"], workspace=s["workspace"])
    else:
        y, lse = moe.moe_attention_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"],
                                          window=c["window"], out=s["out"], workspace=s["workspace"])
    return {"y": y, "lse": lse}


def _plain_rope(s):
    c = s["case"]
    R, page = c["R"], c["page"]
    act = torch.float16 if c["fmt"] == "fp16" else torch.bfloat16
    cos, sin = (t[s["positions"].long()][:, None, :] for t in (s["cos"], s["sin"]))

    def rotate(x):
        x = x.float()
        r = x.clone()
        if c["pairs"] == "halves":
            a, b = x[..., :R // 2], x[..., R // 2:R]
            r[..., :R // 2], r[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            r[..., 0:R:2], r[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
        return r

    q, k, v = rotate(s["q"]), rotate(s["k"]), s["v"].float()
    at = (s["slots"] // page).long(), slice(None), (s["slots"] % page).long()
    for x, cache, scales in ((k, s["kc"], s["ks"]), (v, s["vc"], s["vs"])):
        if scales is None:
            cache[at] = x.to(act)
            continue
        b = x.reshape(x.shape[0], x.shape[1], -1, 32)
        # floor(log2 amax) is the binary32 exponent field (0 for zero and subnormals, below every scale used here)
        code = ((b.abs().amax(3).view(torch.int32) >> 23) - 127 - 8 + 127).clamp(0, 254)
        w = b * torch.exp2((127 - code).float())[..., None]
        cache[at] = w.clamp(-448.0, 448.0).view(x.shape).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[at] = code.to(torch.uint8)
    return {"q": q.to(act), "k": k.to(act) if c["packed"] else None, "v": v.to(act) if c["packed"] else None,
            **_cache_outputs(s)}


def _softmax_product(score, mask, v):
    """(sum_j p_j v_j, log sum exp) along the last dimension of `score`, over the keys that `mask` leaves."""
    score = score.masked_fill(~mask, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p, v) / torch.where(total == 0.0, torch.ones_like(total), total)
    return y, (torch.log(total) + top)[..., 0]


def _values(cache, scales, pages):
    """fp32 values of the tokens in `pages` ([b][w] page numbers): [b][Hkv][tokens][D]."""
    x = cache[pages]  # [b][w][Hkv][page][D]
    if scales is None:
        x = x.float()
    else:
        e = torch.exp2(scales[pages].float() - 127.0)
        x = x.view(torch.float8_e4m3fn).float().view(*e.shape, 32) * e[..., None]
    b, w, h, p = x.shape[:4]
    return x.reshape(b, w, h, p, -1).transpose(1, 2).reshape(b, h, w * p, -1)


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    y, lse = s["out"][0], torch.empty(B, Hq, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 28) // (c["n"] * Hkv * D))
    pos = torch.arange(s["table"].shape[1] * c["page"], device=DEV)
    for b in range(0, B, step):
        pages = s["table"][b:b + step].long().clamp(min=0)
        n = s["lens"][b:b + step, None, None, None]
        k, v = _values(s["kc"], s["ks"], pages), _values(s["vc"], s["vs"], pages)
        q = s["q"][b:b + step].float().view(-1, Hkv, Hq // Hkv, D)
        score = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
        mask = (pos < n) & (pos >= n - c["window"] if c["window"] else pos < n)
        r, t = _softmax_product(score, mask, v)
        y[b:b + step], lse[b:b + step] = r.reshape(-1, Hq, D), t.reshape(-1, Hq)
    return {"y": y, "lse": lse if c["lse"] else None}


def _plain_prompt(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    y, lse = s["out"][0], torch.empty(sum(s["nq"]), Hq, dtype=torch.float32, device=DEV)
    q0 = k0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        k = s["k"][k0:k0 + nk].float().permute(1, 2, 0)[:, None]
        v = s["v"][k0:k0 + nk].float().transpose(0, 1)[:, None].contiguous()
        step = max(1, (1 << 29) // (nk * Hq))
        for i in range(0, nq, step):
            rows = slice(q0 + i, q0 + min(nq, i + step))
            q = s["q"][rows].float().view(-1, Hkv, G, D).permute(1, 2, 0, 3)
            score = torch.matmul(q, k) * D ** -0.5
            far = torch.arange(i, min(nq, i + step), device=DEV)[:, None] + (nk - nq)
            key = torch.arange(nk, device=DEV)
            mask = key <= far if c["causal"] else key < nk
            if c["window"]:
                mask = mask & (key > far - c["window"])
            r, t = _softmax_product(score, mask, v)
            y[rows], lse[rows] = r.permute(2, 0, 1, 3).reshape(-1, Hq, D), t.permute(2, 0, 1).reshape(-1, Hq)
        q0, k0 = q0 + nq, k0 + nk
    return {"y": y, "lse": lse if c["lse"] else None}


# ---------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        T = c["T"]
        row = D + D // 32 if c["fmt"] == "mxfp8" else 2 * D
        b = (Hq + 2 * Hkv) * D * BYTES[c["x"]] + Hq * D * 2 + 2 * Hkv * row + (4 * Hkv * D if c["packed"] else 0)
        return {"bytes": T * (b + 4 * c["R"] + 8),
                "flops": T * (3 * (Hq + Hkv) * c["R"] + (6 * Hkv * D if c["fmt"] == "mxfp8" else 0))}
    if c["op"] == "decode":
        lens = _lengths(c["B"], c["n"], c["idle"])
        keys = sum(min(n, c["window"]) if c["window"] else n for n in lens)
        row = D + D // 32 if c["fmt"] == "mxfp8" else 2 * D
        return {"bytes": 2 * keys * Hkv * row + 4 * c["B"] * Hq * D + (4 * c["B"] * Hq if c["lse"] else 0),
                "flops": 4 * keys * Hq * D}
    pairs = tq = tk = 0
    for n in _lengths(c["B"], c["n"]):
        nk = n + c["past"]
        tq, tk = tq + n, tk + nk
        if not c["causal"]:
            pairs += n * nk
        else:
            w = c["window"] or nk
            # query i sees min(w, i + 1 + past) keys
            m = min(n, max(0, w - c["past"]))
            pairs += m * c["past"] + m * (m + 1) // 2 + (n - m) * w
    return {"bytes": 4 * tq * Hq * D + 4 * tk * Hkv * D + (4 * tq * Hq if c["lse"] else 0), "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    """The definitions in 64 bits, by other steps than the plain forms."""
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    if c["op"] == "rope":
        R = c["R"]
        p = s["positions"].to(torch.int64)
        turn = torch.complex(s["cos"].to(f64)[p], s["sin"].to(f64)[p])[:, None]

        def rotate(x):
            x = x.to(f64)
            z = x[..., :R]
            z = z.unflatten(2, (2, R // 2)).transpose(2, 3) if c["pairs"] == "halves" else z.unflatten(2, (R // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.transpose(2, 3) if c["pairs"] == "halves" else z
            return torch.cat([z.flatten(2), x[..., R:]], 2)

        q, k, v = rotate(s["q"]), rotate(s["k"]), s["v"].to(f64)
        r = {"q": q, "k": k if c["packed"] else None, "v": v if c["packed"] else None}
        slot = s["slots"].to(torch.int64)
        for name, x in (("k", k), ("v", v)):
            # slots of a page are rows of [n_pages][page][Hkv] here
            held = torch.zeros(s["kc"].shape[0] * c["page"], Hkv, D, dtype=f64, device=DEV)
            if c["fmt"] != "mxfp8":
                held[slot] = x
            else:
                b = x.reshape(-1, 32)
                _, e = torch.frexp(b.abs().max(1).values)  # amax = m 2^e, m in [1/2, 1)
                X = torch.ldexp(torch.ones_like(b[:, 0]), (e - 9).clamp(-127, 127))
                a = (b / X[:, None]).abs()
                _, ea = torch.frexp(a)
                step = torch.ldexp(torch.ones_like(a), ea.clamp(-5, 9) - 4)  # 3 fraction bits, subnormals below 2^-6
                held[slot] = torch.copysign((torch.round(a / step) * step).clamp(max=448.0), b).view(x.shape)
                scale = torch.full((held.shape[0], Hkv, D // 32), 2.0 ** -127, dtype=f64, device=DEV)
                scale[slot] = X.view(-1, Hkv, D // 32)
                r[name + "_scales"] = scale.view(-1, c["page"], Hkv, D // 32).transpose(1, 2)
            r[name + "_cache"] = held.view(-1, c["page"], Hkv, D).transpose(1, 2)
        names = ("q", "k", "v", "k_cache", "v_cache", "k_scales", "v_scales")
        return {n: r[n] for n in names if n in r}

    def attend(q, k, v, lo, hi):
        """Queries q [i][Hq][D] over keys lo[i] <= j < hi[i] of k, v [j][Hkv][D]."""
        key = torch.arange(k.shape[0], device=DEV)
        seen = (key >= lo[:, None]) & (key < hi[:, None])
        y = torch.zeros(q.shape, dtype=f64, device=DEV)
        lse = torch.full(q.shape[:2], -math.inf, dtype=f64, device=DEV)
        some = hi > lo
        for h in range(Hq):
            z = (q[:, h] @ k[:, h // G].T) / math.sqrt(D)
            z = torch.where(seen, z, -math.inf)
            lse[:, h] = torch.logsumexp(z, 1)
            y[:, h] = torch.where(some[:, None], torch.softmax(z, 1) @ v[:, h // G], 0.0)
        return y, lse

    ys, ls = [], []
    if c["op"] == "decode":
        def rows(cache, scales, pages, n):
            x = cache.transpose(1, 2)[pages].flatten(0, 1)[:n]  # [n][Hkv][D]
            if scales is None:
                return x.to(f64)
            e = scales.transpose(1, 2)[pages].flatten(0, 1)[:n].to(f64)
            b = x.to(torch.int32)  # E4M3: three fraction bits, bias 7
            f, g = (b % 8).to(f64), (b // 8) % 16
            w = torch.where(g == 0, f / 8.0 * 2.0 ** -6, (1.0 + f / 8.0) * torch.exp2((g - 7).to(f64)))
            return torch.where(b >= 128, -w, w) * torch.exp2(e - 127.0).repeat_interleave(32, 2)

        for b, n in enumerate(_lengths(c["B"], c["n"], c["idle"])):
            pages = s["table"][b, :(n + c["page"] - 1) // c["page"]].long()
            k, v = rows(s["kc"], s["ks"], pages, n), rows(s["vc"], s["vs"], pages, n)
            hi = torch.tensor([n], device=DEV)
            lo = (hi - c["window"]).clamp(min=0) if c["window"] else hi * 0
            y, lse = attend(s["q"][b:b + 1].to(f64), k, v, lo, hi)
            ys.append(y)
            ls.append(lse)
    else:
        if 4.0 * c["Hq"] * D * sum(a * b for a, b in zip(s["nq"], s["nk"])) > 2e13:
            return None
        for b in range(c["B"]):
            k, v = (s[x][int(s["cu_k"][b]):int(s["cu_k"][b + 1])].to(f64) for x in ("k", "v"))
            first = int(s["cu_q"][b])
            for i in range(0, s["nq"][b], 2048):
                m = min(2048, s["nq"][b] - i)
                p = torch.arange(i, i + m, device=DEV) + s["nk"][b] - s["nq"][b]
                hi = p + 1 if c["causal"] else torch.full_like(p, s["nk"][b])
                lo = (p + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(p)
                y, lse = attend(s["q"][first + i:first + i + m].to(f64), k, v, lo, hi)
                ys.append(y)
                ls.append(lse)
    return {"y": torch.cat(ys), "lse": torch.cat(ls) if c["lse"] else None}
