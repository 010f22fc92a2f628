"""The dense front of a routed-MoE block, measured: the residual addition with the RMS norm and its 8-bit output
(`moe_add_rms_norm`), the choice of experts from router logits (`moe_select_experts`), and products with 4-bit
weights (`moe_linear`).

`own` chooses between the plain forms (elementary torch operations) and the library's kernels.  `listed()` and
`draw()` give cases, `prepare()` makes a case's inputs from a seed, `run()` is one call, `work()` the bytes and
operations that one call cannot do without, `exact()` the outputs in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------------------------------------------
# cases
def _norm(T, H, x, residual, y, mx, w="bf16"):
    return {"op": "norm", "T": T, "H": H, "x": x, "residual": residual, "y": y, "mx": mx, "w": w}


def _select(T, E, k, score, groups, keep, by, bias, logits="fp32", renorm=True, scale=1.0, shared=0, scores=False):
    return {"op": "select", "T": T, "E": E, "k": k, "score": score, "groups": groups, "keep": keep, "by": by,
            "bias": bias, "logits": logits, "renorm": renorm, "scale": scale, "shared": shared, "scores": scores}


def _linear(T, N, K, fmt, y, bias=False):
    return {"op": "linear", "T": T, "N": N, "K": K, "fmt": fmt, "y": y, "bias": bias}


def listed():
    return [
        # one decoded token: the fp32 output of the previous layer's combine joins the bf16 residual stream
        dict(_norm(1, 7168, "fp32", "bf16", "bf16", False), name="norm T1 H7168"),
        # the decode sweep's batch, with the FP8 codes that the MX expert FFN reads
        dict(_norm(176, 7168, "fp32", "bf16", "bf16", True), name="norm T176 H7168 fp8"),
        # a prompt: 16-bit attention output, norm and codes
        dict(_norm(8192, 7168, "bf16", "bf16", "bf16", True), name="norm T8192 H7168 fp8"),
        # rows of an odd length in binary16 (no 16-byte vectors)
        dict(_norm(333, 4097, "fp16", "fp16", "fp16", False, "fp32"), name="norm T333 H4097 fp16"),
        # one decoded token, group-limited sigmoid routing with a balance bias
        dict(_select(1, 256, 8, "sigmoid", 8, 4, "top2", True, scale=2.5), name="select T1 E256 g8"),
        # a decode batch, plain softmax top-8 of 128 experts from 16-bit logits
        dict(_select(64, 128, 8, "softmax", 1, 1, "max", False, logits="bf16"), name="select T64 E128 softmax"),
        # a prompt, group-limited sigmoid routing, the scores kept for load statistics
        dict(_select(8192, 256, 8, "sigmoid", 8, 4, "top2", True, scale=2.5, scores=True), name="select T8192 E256 g8"),
        # groups of 20 ranked by their best expert, weights not renormalised, two shared experts
        dict(_select(1001, 160, 6, "softmax", 8, 3, "max", False, renorm=False, scale=16.0, shared=2),
             name="select T1001 E160 g8"),
        # one decoded token through an attention output projection
        dict(_linear(1, 7168, 7168, "mxfp4", "fp32"), name="linear T1 7168x7168 mxfp4"),
        # a few tokens of speculative decoding, a small ragged projection with a bias
        dict(_linear(3, 1000, 2080, "int4g32", "bf16", True), name="linear T3 1000x2080 int4"),
        # a decode batch through the dense FFN's gate projection
        dict(_linear(32, 16384, 4096, "nvfp4", "bf16"), name="linear T32 16384x4096 nvfp4"),
        # a prompt chunk
        dict(_linear(2048, 4096, 7168, "mxfp4", "fp32"), name="linear T2048 4096x7168 mxfp4"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "select", "linear"])
    if op == "norm":
        mx = rng.random() < 0.5
        H = _log(rng, 64, 16384)
        H = max(32, H // 32 * 32) if mx else (H | 1 if rng.random() < 0.3 else max(8, H // 8 * 8))
        T = _log(rng, 1, max(1, min(8192, 8192 * 7168 // H)))
        x = rng.choice(["bf16", "fp16", "fp32"])
        if T * H * BYTES[x] > 8192 * 7168 * 2:
            x = "bf16"
        act = rng.choice(["bf16", "fp16"])
        return _norm(T, H, x, act, act, mx, rng.choice(["bf16", "fp32"]))
    if op == "select":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = min(512, groups * max(2, _log(rng, 16, 512) // groups))
        E = E // groups * groups
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        T = _log(rng, 1, 8192 * 256 // E)
        score = rng.choice(["softmax", "sigmoid"])
        return _select(min(T, 8192), E, k, score, groups, keep, rng.choice(["top2", "max"]), rng.random() < 0.6,
                       rng.choice(["fp32", "bf16", "fp16"]), rng.random() < 0.7, rng.choice([1.0, 2.5]),
                       rng.randint(0, 2), rng.random() < 0.3)
    N = _log(rng, 64, 16384)
    K = max(32, _log(rng, 256, 16384) // 32 * 32)
    while N * K > 7168 * 16384:
        K = max(32, K // 64 * 32)
    T = _log(rng, 1, max(1, min(4096, 2048 * 4096 * 7168 // (N * K), (1 << 25) // N, (1 << 25) // K)))
    return _linear(T, N, K, rng.choice(["mxfp4", "int4g32", "nvfp4"]), rng.choice(["fp32", "bf16", "fp16"]),
                   rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------------------------
# inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)

    if own:
        import mxfp4_routed_expert_router_amd as moe
    s = {"case": dict(case)}
    c = case
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s["x"] = normal(T, H).to(DTYPES[c["x"]])
        s["residual"] = (4.0 * normal(T, H)).to(DTYPES[c["residual"]])
        s["weight"] = (1.0 + 0.1 * normal(H)).to(DTYPES[c["w"]])
        s["out"] = (torch.empty(T, H, dtype=DTYPES[c["y"]], device=DEV),
                    torch.empty(T, H, dtype=DTYPES[c["residual"]], device=DEV),
                    torch.empty(T, H, dtype=torch.uint8, device=DEV) if c["mx"] else None,
                    torch.empty(T, H // 32, dtype=torch.uint8, device=DEV) if c["mx"] else None)
        if own:
            s["norm"] = moe.RmsNorm(s["weight"], EPS)
    elif c["op"] == "select":
        T, E, kt = c["T"], c["E"], c["k"] + c["shared"]
        s["logits"] = normal(T, E).to(DTYPES[c["logits"]])
        s["bias"] = 0.02 * normal(E) if c["bias"] else None
        s["out"] = (torch.empty(T, kt, dtype=torch.int32, device=DEV),
                    torch.empty(T, kt, dtype=torch.float32, device=DEV),
                    torch.empty(T, E, dtype=torch.float32, device=DEV) if c["scores"] else None)
        if own:
            s["rule"] = moe.RouteRule(c["k"], c["score"], s["bias"], c["groups"], c["keep"], c["by"], c["renorm"],
                                      c["scale"], c["shared"])
    else:
        T, N, K, fmt = c["T"], c["N"], c["K"], c["fmt"]
        s["x"] = normal(T, K).to(torch.bfloat16)
        s["codes"] = ints(0, 256, N, K // 2).to(torch.uint8)
        s["zeros"] = s["tensor_scale"] = None
        if fmt == "mxfp4":      # E8M0 codes of weights around a few hundredths
            s["scales"] = ints(118, 124, N, K // 32).to(torch.uint8)
        elif fmt == "int4g32":  # binary16 scales around 0.01, zero points around the middle
            s["scales"] = (0.005 + 0.01 * torch.rand(N, K // 32, generator=g, device=DEV)).half().view(torch.uint8)
            s["zeros"] = (ints(4, 12, N, (K // 32 + 1) // 2) + 16 * ints(4, 12, N, (K // 32 + 1) // 2)).to(torch.uint8)
        else:                   # E4M3 block scales of 2^-3 .. 448 under one tensor scale
            s["scales"] = ints(0x20, 0x7F, N, K // 16).to(torch.uint8)
            s["tensor_scale"] = torch.full((1,), 2.0 ** -12, device=DEV)
        s["bias"] = normal(N) if c["bias"] else None
        s["out"] = torch.empty(T, N, dtype=DTYPES[c["y"]], device=DEV)
        if own:
            s["W"] = moe.LinearWeights(s["codes"], s["scales"], fmt, zeros=s["zeros"], tensor_scale=s["tensor_scale"])
            need = moe.moe_linear_workspace_bytes(T, s["W"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
def run(state):
    if own:
        import mxfp4_routed_expert_router_amd as moe
        op = state["case"]["op"]
        if op == "norm":
            y, residual, codes, scales = moe.moe_add_rms_norm(
                state["x"], state["norm"], state["residual"], mx="fp8" if state["case"]["mx"] else None,
                out=state["out"])
            if codes is None:
                return {"y": y, "residual": residual}
            return {"y": y, "residual": residual, "codes": codes.view(torch.float8_e4m3fn),
                    "scales": scales.view(torch.float8_e8m0fnu)}
        if op == "select":
            ids, weights, scores = moe.moe_select_experts(state["logits"], state["rule"], out=state["out"])
            return {"ids": ids, "weights": weights, "scores": scores}
        return {"y": moe.moe_linear(state["x"], state["W"], state["bias"], out=state["out"],
                                    workspace=state["workspace"])}
    return {"norm": _plain_norm, "select": _plain_select, "linear": _plain_linear}[state["case"]["op"]](state)


def _plain_norm(s):
    c = s["case"]
    v = s["x"].float() + s["residual"].float()
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["weight"].float()
    r = {"y": y.to(DTYPES[c["y"]]), "residual": v.to(DTYPES[c["residual"]])}
    if c["mx"]:
        b = y.view(c["T"], -1, 32)
        amax = b.abs().amax(2)
        # floor(log2 amax) is the binary32 exponent field (0 for zero and subnormals, below every scale used here)
        code = ((amax.view(torch.int32) >> 23) - 127 - 8 + 127).clamp(0, 254)
        q = b * torch.exp2((127 - code).float())[:, :, None]
        r["codes"] = q.clamp(-448.0, 448.0).view(c["T"], -1).to(torch.float8_e4m3fn)
        r["scales"] = code.to(torch.uint8).view(torch.float8_e8m0fnu)
    return r


def _plain_select(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    L = s["logits"].double()  # 64 bits: keys of two experts, or sums of two groups, may lie next to each other
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-L))
    else:
        e = torch.exp(L - L.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["keep"] < G:
        of = key.view(T, G, E // G)
        best = of.sort(dim=2, descending=True).values
        rank = best[:, :, 0] + best[:, :, 1] if c["by"] == "top2" else best[:, :, 0]
        keep = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter(1, keep, False)
        key = of.masked_fill(mask[:, :, None], -math.inf).view(T, E)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    shared = torch.arange(E, E + c["shared"], device=DEV).expand(T, -1)
    return {"ids": torch.cat([ids, shared], 1).int(),
            "weights": torch.cat([w, torch.ones_like(shared, dtype=torch.float64)], 1).float(),
            "scores": score.float() if c["scores"] else None}


def _plain_linear(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2)  # even k in the low nibble
    if c["fmt"] == "int4g32":
        z = torch.stack([s["zeros"] & 15, s["zeros"] >> 4], 2).view(N, -1)[:, :K // 32]
        w = (code.view(N, -1, 32).float() - z[:, :, None].float()) * s["scales"].view(torch.float16).float()[:, :, None]
    else:
        v = torch.tensor(E2M1, device=DEV)[code.int()]
        if c["fmt"] == "mxfp4":
            w = v.view(N, -1, 32) * torch.exp2(s["scales"].float() - 127.0)[:, :, None]
        else:
            w = v.view(N, -1, 16) * s["scales"].view(torch.float8_e4m3fn).float()[:, :, None] * s["tensor_scale"]
    y = s["x"].float() @ w.view(N, K).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(DTYPES[c["y"]])}


# ---------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        b = n * (BYTES[c["x"]] + 2 * BYTES[c["residual"]] + BYTES[c["y"]]) + c["H"] * BYTES[c["w"]]
        return {"bytes": b + (n + n // 32 if c["mx"] else 0), "flops": n * (9 if c["mx"] else 5)}
    if c["op"] == "select":
        n = c["T"] * c["E"]
        b = n * (BYTES[c["logits"]] + (4 if c["scores"] else 0)) + 8 * c["T"] * (c["k"] + c["shared"])
        return {"bytes": b + (4 * c["E"] if c["bias"] else 0), "flops": 6 * n}
    T, N, K = c["T"], c["N"], c["K"]
    scale = {"mxfp4": K // 32, "int4g32": K // 16 + (K // 32 + 1) // 2, "nvfp4": K // 16}[c["fmt"]]
    return {"bytes": N * (K // 2 + scale) + 2 * T * K + T * N * BYTES[c["y"]] + (4 * N if c["bias"] else 0),
            "flops": 2 * T * N * K}


# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    """The definitions in 64 bits, by other steps than the plain forms."""
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "norm":
        v = s["x"].to(f64) + s["residual"].to(f64)
        y = v / torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / c["H"] + EPS) * s["weight"].to(f64)
        r = {"y": y, "residual": v}
        if c["mx"]:
            b = y.reshape(-1, 32)
            _, e = torch.frexp(b.abs().max(1).values)  # amax = m 2^e, m in [1/2, 1)
            X = torch.ldexp(torch.ones_like(b[:, 0]), (e - 9).clamp(-127, 127))
            a = (b / X[:, None]).abs()
            _, ea = torch.frexp(a)
            step = torch.ldexp(torch.ones_like(a), ea.clamp(-5, 9) - 4)  # 3 fraction bits, subnormals below 2^-6
            q = (torch.round(a / step) * step).clamp(max=448.0)
            r["codes"] = torch.copysign(q, b).view(c["T"], c["H"])
            r["scales"] = X.view(c["T"], -1)
        return r
    if c["op"] == "select":
        T, E, G, per = c["T"], c["E"], c["groups"], c["E"] // c["groups"]
        L = s["logits"].to(f64)
        score = torch.special.expit(L) if c["score"] == "sigmoid" else torch.exp(L - torch.logsumexp(L, 1, keepdim=True))
        key = score + (s["bias"].to(f64) if s["bias"] is not None else 0.0)
        chosen = torch.zeros(T, E, dtype=torch.bool, device=DEV)
        allowed = torch.ones(T, E, dtype=torch.bool, device=DEV)
        row = torch.arange(T, device=DEV)
        if c["keep"] < G:
            two = key.view(T, G, per).topk(min(2, per), 2).values
            rank = two.sum(2) if c["by"] == "top2" else two[:, :, 0]
            allowed.zero_()
            for _ in range(c["keep"]):
                at = rank.argmax(1)
                allowed.view(T, G, per)[row, at] = True
                rank[row, at] = -math.inf
        w = torch.empty(T, c["k"], dtype=f64, device=DEV)
        for j in range(c["k"]):
            at = key.masked_fill(chosen | ~allowed, -math.inf).argmax(1)
            chosen[row, at] = True
            w[:, j] = score[row, at]
        w = c["scale"] * (w / w.sum(1, keepdim=True) if c["renorm"] else w)
        w = torch.cat([w, torch.ones(T, c["shared"], dtype=f64, device=DEV)], 1)
        return {"ids": None, "weights": w, "scores": score if c["scores"] else None}
    N, K = c["N"], c["K"]
    byte = s["codes"].to(torch.int32)
    code = torch.zeros(N, K, dtype=torch.int32, device=DEV)
    code[:, 0::2] = byte % 16
    code[:, 1::2] = byte // 16
    if c["fmt"] == "int4g32":
        zb = s["zeros"].to(torch.int32)
        z = torch.zeros(N, 2 * zb.shape[1], dtype=torch.int32, device=DEV)
        z[:, 0::2] = zb % 16
        z[:, 1::2] = zb // 16
        w = (code.to(f64) - z[:, :K // 32].repeat_interleave(32, 1).to(f64))
        w *= s["scales"].view(torch.float16).to(f64).repeat_interleave(32, 1)
    else:
        m, e = (code % 2).to(f64), (code // 2) % 4  # E2M1: one fraction bit, bias 1
        w = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).to(f64)))
        w = torch.where(code >= 8, -w, w)
        if c["fmt"] == "mxfp4":
            w *= torch.exp2(s["scales"].to(f64) - 127.0).repeat_interleave(32, 1)
        else:  # E4M3 scales: three fraction bits, bias 7
            sc = s["scales"].to(torch.int32)
            f, e = (sc % 8).to(f64), (sc // 8) % 16
            v = torch.where(e == 0, f / 8.0 * 2.0 ** -6, (1.0 + f / 8.0) * torch.exp2((e - 7).to(f64)))
            w *= torch.where(sc >= 128, -v, v).repeat_interleave(16, 1) * s["tensor_scale"].to(f64)
    y = torch.matmul(s["x"].to(f64), w.T)
    return {"y": y if s["bias"] is None else y + s["bias"].to(f64)}
