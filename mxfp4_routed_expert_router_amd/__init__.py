"""Routed Mixture-of-Experts FFN layer for AMD Instinct MI355X (gfx950).

Thin Python binding of the C ABI in include/moe.h (libmoe.so, built from csrc/ by _build.py).  The
functions keep the C names and only marshal arguments: torch tensors provide device memory and the
current HIP stream; every step of the layer runs in the library's HIP kernels.  There is no CPU
fallback -- importing works anywhere, but any call raises when libmoe.so is missing or no GPU is
present.

    ids, w, probs = moe_route(x, w_router, top_k, bias, n_shared)     # router
    b = moe_bucket(ids, n_experts)                                     # group slots by expert
    y_slots = moe_expert_ffn(x, W, b.offsets, b.sorted_slot, k_total)  # SwiGLU experts
    y = moe_combine(y_slots, w)                                        # weighted combine, fp32

In front of the layer stand the projection of the attention output, the residual addition with its norm, and
group-limited routing (MoEBlock runs them all):

    a = moe_linear(attn, W_o)                                          # 4-bit weights, fp32 out
    x, r, _, _ = moe_add_rms_norm(a, norm, residual)                   # residual stream and the layer's input
    ids, w, _ = moe_route_grouped(x, w_router, rule)                   # scores, bias, groups, top-k

The attention that gives `attn` (AttentionBlock runs it with its norm and projection):

    q, k, v = moe_rope_cache(q, k, v, rope, positions, cache, slots)   # rotary positions, write into the paged cache
    attn, _ = moe_attention_prompt(q, k, v, cu)                        # whole prompts, packed
    attn, _ = moe_attention_decode(q, cache, page_table, lens)         # one new token per sequence
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libmoe.so")
ROOT = os.path.dirname(PKG)
HEADER = os.path.join(ROOT, "include", "moe.h")

MOE_ACT_BF16, MOE_ACT_FP16 = 0, 1
MOE_W_MXFP4, MOE_W_FP16, MOE_W_INT4_G32, MOE_W_NVFP4 = 0, 1, 2, 3
W_FORMATS = {"mxfp4": MOE_W_MXFP4, "fp16": MOE_W_FP16, "int4g32": MOE_W_INT4_G32, "nvfp4": MOE_W_NVFP4}
MOE_MX_FP8_E4M3, MOE_MX_FP4_E2M1, MOE_MX_FP6_E2M3 = 1, 2, 3
MX_FORMATS = {"fp8": MOE_MX_FP8_E4M3, "fp4": MOE_MX_FP4_E2M1, "fp6": MOE_MX_FP6_E2M3}
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # moe_dtype
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"top2": 0, "max": 1}
MOE_MAX_GROUPS = 64
MOE_KV_BF16, MOE_KV_FP16, MOE_KV_MXFP8 = 0, 1, 2
KV_FORMATS = {"bf16": MOE_KV_BF16, "fp16": MOE_KV_FP16, "mxfp8": MOE_KV_MXFP8}
KV_TYPES = {MOE_KV_BF16: torch.bfloat16, MOE_KV_FP16: torch.float16, MOE_KV_MXFP8: torch.uint8}
ROPE_PAIRS = {"halves": 0, "neighbours": 1}
MOE_MAX_HEADS, MOE_MAX_HEAD_DIM = 1024, 256

STATUS = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_BLOCK", 4: "MOE_ERR_ALIGN",
          5: "MOE_ERR_DTYPE", 6: "MOE_ERR_TOPK", 7: "MOE_ERR_WORKSPACE", 8: "MOE_ERR_HIP"}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, text: str):
        super().__init__(f"{where}: {STATUS.get(status, status)} ({text})")
        self.status = status


class moe_proj(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("w_expert_stride", ctypes.c_int64), ("w_row_stride", ctypes.c_int64),
                ("s_expert_stride", ctypes.c_int64), ("s_row_stride", ctypes.c_int64),
                ("zeros", ctypes.c_void_p), ("z_expert_stride", ctypes.c_int64), ("z_row_stride", ctypes.c_int64),
                ("tensor_scale", ctypes.c_void_p)]


class moe_expert_weights(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("n_experts", ctypes.c_int), ("hidden", ctypes.c_int),
                ("inter", ctypes.c_int), ("gate", moe_proj), ("up", moe_proj), ("down", moe_proj)]


class moe_route_rule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("top_k", ctypes.c_int), ("n_shared", ctypes.c_int),
                ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int), ("group_score", ctypes.c_int),
                ("renormalise", ctypes.c_int), ("routed_scale", ctypes.c_float), ("shared_weight", ctypes.c_float),
                ("selection_bias", ctypes.c_void_p)]


class moe_norm(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int), ("hidden", ctypes.c_int),
                ("eps", ctypes.c_float)]


class moe_linear_weights(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("n_out", ctypes.c_int), ("k_in", ctypes.c_int), ("w", moe_proj)]


class moe_heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("dtype", ctypes.c_int), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("s_page_stride", ctypes.c_int64),
                ("s_head_stride", ctypes.c_int64), ("s_token_stride", ctypes.c_int64)]


class moe_rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("n_positions", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("pairs", ctypes.c_int)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError(f"{LIBRARY} is missing: build it with `python -m mxfp4_routed_expert_router_amd._build` "
                               "(or __graft_entry__.build()); there is no fallback implementation")
        L = ctypes.CDLL(LIBRARY)
        vp, i, st, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        L.moe_status_str.restype = ctypes.c_char_p; L.moe_status_str.argtypes = [i]
        L.moe_abi_version.restype = i; L.moe_abi_version.argtypes = []
        L.moe_route_workspace_bytes.restype = st; L.moe_route_workspace_bytes.argtypes = [i, i, i]
        L.moe_route.restype = i
        L.moe_route.argtypes = [vp, i, i, i, vp, vp, i, i, i, vp, vp, vp, vp, st, vp]
        L.moe_route_bucket_workspace_bytes.restype = st
        L.moe_route_bucket_workspace_bytes.argtypes = [i, i, i, i, i]
        L.moe_route_bucket.restype = i
        L.moe_route_bucket.argtypes = [vp, i, i, i, vp, vp, i, i, i, vp, vp, vp, vp, vp, vp, vp,
                                       ctypes.POINTER(moe_expert_weights), vp, st, vp, st, vp]
        L.moe_route_sigmoid.restype = i
        L.moe_route_sigmoid.argtypes = [vp, i, i, i, vp, vp, i, i, i, ctypes.c_float, ctypes.c_float, vp, vp, vp,
                                        vp, st, vp]
        L.moe_row_shape.restype = i; L.moe_row_shape.argtypes = [i, ctypes.POINTER(ctypes.c_int), i]
        L.moe_pad_rows.restype = i; L.moe_pad_rows.argtypes = [vp, i, i, vp, vp, vp]
        L.moe_bucket_workspace_bytes.restype = st; L.moe_bucket_workspace_bytes.argtypes = [i, i]
        L.moe_bucket.restype = i
        L.moe_bucket.argtypes = [vp, i, i, vp, vp, vp, vp, vp, st, vp]
        L.moe_expert_ffn_workspace_bytes.restype = st
        L.moe_expert_ffn_workspace_bytes.argtypes = [i, i, ctypes.POINTER(moe_expert_weights)]
        L.moe_expert_ffn.restype = i
        L.moe_expert_ffn.argtypes = [vp, i, i, i, ctypes.POINTER(moe_expert_weights), vp, vp, vp, vp, st, vp]
        L.moe_expert_ffn_static.restype = i
        L.moe_expert_ffn_static.argtypes = [vp, i, i, i, ctypes.POINTER(moe_expert_weights), vp, vp, vp, vp]
        L.moe_expert_ffn_f16_workspace_bytes.restype = st
        L.moe_expert_ffn_f16_workspace_bytes.argtypes = [i, i, ctypes.POINTER(moe_expert_weights)]
        L.moe_expert_ffn_f16.restype = i
        L.moe_expert_ffn_f16.argtypes = [vp, i, i, i, ctypes.POINTER(moe_expert_weights), i, vp, vp, vp, vp, st, vp]
        L.moe_combine_restore.restype = i
        L.moe_combine_restore.argtypes = [vp, vp, i, i, i, i, vp, vp]
        L.moe_expert_ffn_plan.restype = i
        L.moe_expert_ffn_plan.argtypes = [i, i, i, ctypes.POINTER(moe_expert_weights), vp, vp, st, vp]
        L.moe_expert_ffn_gateup.restype = i
        L.moe_expert_ffn_gateup.argtypes = [vp, i, i, i, ctypes.POINTER(moe_expert_weights), vp, vp, vp, st, vp]
        L.moe_expert_ffn_down.restype = i
        L.moe_expert_ffn_down.argtypes = [i, i, i, ctypes.POINTER(moe_expert_weights), vp, vp, vp, vp, st, vp]
        L.moe_combine.restype = i
        L.moe_combine.argtypes = [vp, vp, i, i, i, vp, vp]
        L.moe_mxfp4_dequant.restype = i
        L.moe_mxfp4_dequant.argtypes = [vp, vp, i, i, i64, i64, vp, vp]
        L.moe_mx_row_bytes.restype = st; L.moe_mx_row_bytes.argtypes = [i, i]
        L.moe_mx_quantize.restype = i
        L.moe_mx_quantize.argtypes = [vp, i, i, i, i, vp, vp, vp]
        L.moe_expert_ffn_mx_workspace_bytes.restype = st
        L.moe_expert_ffn_mx_workspace_bytes.argtypes = [i, i, ctypes.POINTER(moe_expert_weights), i]
        L.moe_expert_ffn_mx_workspace_layout.restype = i
        L.moe_expert_ffn_mx_workspace_layout.argtypes = [i, i, ctypes.POINTER(moe_expert_weights), i,
                                                         ctypes.POINTER(ctypes.c_size_t)]
        L.moe_expert_ffn_mx.restype = i
        L.moe_expert_ffn_mx.argtypes = [vp, i, i, i, ctypes.POINTER(moe_expert_weights), i, vp, vp, vp, vp, st, vp]
        L.moe_expert_ffn_mx_codes.restype = i
        L.moe_expert_ffn_mx_codes.argtypes = [vp, vp, i, i, ctypes.POINTER(moe_expert_weights), i, vp, vp, vp, vp, st,
                                              vp]
        L.moe_select_experts.restype = i
        L.moe_select_experts.argtypes = [vp, i, i64, i, i, vp, vp, vp, vp, vp]
        L.moe_route_grouped.restype = i
        L.moe_route_grouped.argtypes = [vp, i, i, i, vp, i, vp, vp, vp, vp, vp, st, vp]
        L.moe_add_rms_norm.restype = i
        L.moe_add_rms_norm.argtypes = [vp, vp, i, i64, vp, i, i64, i, vp, i64, vp, i, i, vp, vp, vp]
        L.moe_linear_workspace_bytes.restype = st; L.moe_linear_workspace_bytes.argtypes = [i, vp]
        L.moe_linear.restype = i
        L.moe_linear.argtypes = [vp, i, i64, i, vp, vp, vp, i, i64, vp, st, vp]
        L.moe_rope_cache.restype = i
        L.moe_rope_cache.argtypes = [vp, vp, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_attention_prompt_workspace_bytes.restype = st
        L.moe_attention_prompt_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.moe_attention_prompt.restype = i
        L.moe_attention_prompt.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float, i, i, vp, vp, vp, st, vp]
        L.moe_attention_decode_workspace_bytes.restype = st
        L.moe_attention_decode_workspace_bytes.argtypes = [i, i, i, i, i]
        L.moe_attention_decode.restype = i
        L.moe_attention_decode.argtypes = [vp, i, i, vp, vp, i64, i, vp, i, ctypes.c_float, i, vp, vp, vp, st, vp]
        L.moe_stream_read.restype = i
        L.moe_stream_read.argtypes = [vp, st, vp, vp]
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise MoEError(status, where, lib().moe_status_str(status).decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _act_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return MOE_ACT_BF16
    if x.dtype == torch.float16:
        return MOE_ACT_FP16
    raise TypeError(f"activations must be bfloat16 or float16, got {x.dtype}")


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None


class ExpertWeights:
    """Device weights of all experts of a layer, described for moe_expert_ffn.

    MXFP4: gate/up codes uint8 [E'][I][H/2], scales uint8 [E'][I][H/32]; down codes [E'][H][I/2],
    scales [E'][H][I/32].  FP16: gate/up float16 [E'][I][H], down [E'][H][I], scales None.
    INT4_G32 (fmt="int4g32"): codes as MXFP4, scales [E'][N][K/32] binary16 bits as uint8 pairs
    ([E'][N][K/16] uint8), extras {"gate"/"up"/"down": zero points uint8 [E'][N][ceil(K/64)]}.
    NVFP4 (fmt="nvfp4"): codes as MXFP4, scales uint8 E4M3 [E'][N][K/16], extras {matrix: fp32
    tensor scales [E']}.
    Any strided view whose last dimension is contiguous is accepted (slices of a larger matrix)."""

    def __init__(self, gate, gate_scales, up, up_scales, down, down_scales, fmt=None, extras=None):
        if fmt is None:
            fmt = MOE_W_FP16 if gate.dtype == torch.float16 else MOE_W_MXFP4
        elif isinstance(fmt, str):
            fmt = W_FORMATS[fmt]
        extras = dict(extras or {})
        self.extras = extras
        self.tensors = (gate, gate_scales, up, up_scales, down, down_scales)
        E2, I = gate.shape[0], gate.shape[1]
        H = down.shape[1]
        self.fmt, self.n_experts, self.hidden, self.inter = fmt, E2, H, I

        def proj(c, s, ex):
            p = moe_proj()
            p.w = c.data_ptr()
            es = c.element_size()
            p.w_expert_stride, p.w_row_stride = c.stride(0) * es, c.stride(1) * es
            if c.stride(2) != 1:
                raise ValueError("weight rows must be contiguous")
            if s is not None:
                p.scales = s.data_ptr()
                ss = s.element_size()
                p.s_expert_stride, p.s_row_stride = s.stride(0) * ss, s.stride(1) * ss
            if ex is not None and fmt == MOE_W_INT4_G32:
                p.zeros = ex.data_ptr()
                p.z_expert_stride, p.z_row_stride = ex.stride(0), ex.stride(1)
            if ex is not None and fmt == MOE_W_NVFP4:
                if ex.dtype != torch.float32 or not ex.is_contiguous():
                    raise ValueError("NVFP4 tensor scales must be a contiguous float32 tensor")
                p.tensor_scale = ex.data_ptr()
            return p

        self.c = moe_expert_weights(fmt, E2, H, I, proj(gate, gate_scales, extras.get("gate")),
                                    proj(up, up_scales, extras.get("up")), proj(down, down_scales, extras.get("down")))

    @property
    def device(self):
        return self.tensors[0].device

    def weight_bytes(self, experts=None) -> int:
        """Logical bytes (codes + scales) of the given experts (all when None)."""
        per = 0
        for t in self.tensors:
            if t is not None:
                per += t[0].numel() * t.element_size()
        n = self.n_experts if experts is None else len(experts)
        return per * n


# ----------------------------------------------------------------------------------------------------
def moe_route_workspace_bytes(T: int, H: int, E: int) -> int:
    return lib().moe_route_workspace_bytes(T, H, E)


def moe_route(x: torch.Tensor, w_router: torch.Tensor, top_k: int, logit_bias: Optional[torch.Tensor] = None,
              n_shared: int = 0, want_probs: bool = False, out=None, workspace=None):
    """-> (ids int32 [T][k'], weights fp32 [T][k'], probs fp32 [T][E] or None)."""
    T, H = x.shape
    E = w_router.shape[0]
    kt = top_k + n_shared
    dev = x.device
    if out is None:
        ids = torch.empty((T, kt), dtype=torch.int32, device=dev)
        w = torch.empty((T, kt), dtype=torch.float32, device=dev)
        probs = torch.empty((T, E), dtype=torch.float32, device=dev) if want_probs else None
    else:
        ids, w, probs = out
    need = moe_route_workspace_bytes(T, H, E)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(lib().moe_route(_ptr(x), _act_dtype(x), T, H, _ptr(w_router), _ptr(logit_bias), E, top_k, n_shared,
                           _ptr(ids), _ptr(w), _ptr(probs), _ptr(ws), 0 if ws is None else ws.numel(),
                           _stream(dev)), "moe_route")
    return ids, w, probs


def moe_route_bucket_workspace_bytes(T: int, H: int, E: int, top_k: int, n_shared: int = 0) -> int:
    return lib().moe_route_bucket_workspace_bytes(T, H, E, top_k, n_shared)


def moe_route_bucket(x: torch.Tensor, w_router: torch.Tensor, top_k: int, logit_bias: Optional[torch.Tensor],
                     n_shared: int, ids: torch.Tensor, weights: torch.Tensor, buckets: "Buckets",
                     W: Optional[ExpertWeights] = None, ffn_workspace: Optional[torch.Tensor] = None,
                     probs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> None:
    """moe_route + moe_bucket (+ moe_expert_ffn_plan into ffn_workspace when W is given) in one call,
    into the caller's buffers."""
    T, H = x.shape
    E = w_router.shape[0]
    need = moe_route_bucket_workspace_bytes(T, H, E, top_k, n_shared)
    ws = workspace if workspace is not None else _workspace(need, x.device)
    _check(lib().moe_route_bucket(_ptr(x), _act_dtype(x), T, H, _ptr(w_router), _ptr(logit_bias), E, top_k, n_shared,
                                  _ptr(ids), _ptr(weights), _ptr(probs), _ptr(buckets.counts), _ptr(buckets.offsets),
                                  _ptr(buckets.sorted_slot), _ptr(buckets.slot_pos),
                                  None if W is None else ctypes.byref(W.c), _ptr(ffn_workspace),
                                  0 if ffn_workspace is None else ffn_workspace.numel(), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream(x.device)), "moe_route_bucket")


def moe_route_sigmoid(x: torch.Tensor, w_router: torch.Tensor, top_k: int,
                      selection_bias: Optional[torch.Tensor] = None, n_shared: int = 0, routed_scale: float = 1.0,
                      shared_weight: float = 1.0, want_scores: bool = False, out=None, workspace=None):
    """Cascadia's sigmoid router -> (ids int32 [T][k'], weights fp32 [T][k'], scores fp32 [T][E] or None)."""
    T, H = x.shape
    E = w_router.shape[0]
    kt = top_k + n_shared
    dev = x.device
    if out is None:
        ids = torch.empty((T, kt), dtype=torch.int32, device=dev)
        w = torch.empty((T, kt), dtype=torch.float32, device=dev)
        scores = torch.empty((T, E), dtype=torch.float32, device=dev) if want_scores else None
    else:
        ids, w, scores = out
    need = moe_route_workspace_bytes(T, H, E)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(lib().moe_route_sigmoid(_ptr(x), _act_dtype(x), T, H, _ptr(w_router), _ptr(selection_bias), E, top_k,
                                   n_shared, routed_scale, shared_weight, _ptr(ids), _ptr(w), _ptr(scores), _ptr(ws),
                                   0 if ws is None else ws.numel(), _stream(dev)), "moe_route_sigmoid")
    return ids, w, scores


def moe_row_shape(T: int, shapes) -> int:
    """Smallest supported row shape >= T (-1 if none)."""
    arr = (ctypes.c_int * len(shapes))(*shapes)
    return lib().moe_row_shape(T, arr, len(shapes))


def moe_pad_rows(n_rows: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor) -> None:
    """Rows >= n_rows[0] (a device int32 scalar) get zero weights and id -1, in place."""
    T, kt = ids.shape
    _check(lib().moe_pad_rows(_ptr(n_rows), T, kt, _ptr(ids), _ptr(weights), _stream(ids.device)), "moe_pad_rows")


@dataclass
class Buckets:
    counts: torch.Tensor
    offsets: torch.Tensor
    sorted_slot: torch.Tensor
    slot_pos: Optional[torch.Tensor]


def moe_bucket_workspace_bytes(n_slots: int, n_buckets: int) -> int:
    return lib().moe_bucket_workspace_bytes(n_slots, n_buckets)


def moe_bucket(ids: torch.Tensor, n_buckets: int, out: Optional[Buckets] = None, workspace=None) -> Buckets:
    n = ids.numel()
    dev = ids.device
    if out is None:
        out = Buckets(torch.empty(n_buckets, dtype=torch.int32, device=dev),
                      torch.empty(n_buckets + 1, dtype=torch.int32, device=dev),
                      torch.empty(n, dtype=torch.int32, device=dev),
                      torch.empty(n, dtype=torch.int32, device=dev))
    need = moe_bucket_workspace_bytes(n, n_buckets)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(lib().moe_bucket(_ptr(ids), n, n_buckets, _ptr(out.counts), _ptr(out.offsets), _ptr(out.sorted_slot),
                            _ptr(out.slot_pos), _ptr(ws), 0 if ws is None else ws.numel(), _stream(dev)),
           "moe_bucket")
    return out


def moe_expert_ffn_workspace_bytes(T: int, k_total: int, W: ExpertWeights) -> int:
    return lib().moe_expert_ffn_workspace_bytes(T, k_total, ctypes.byref(W.c))


def moe_expert_ffn(x: torch.Tensor, W: ExpertWeights, offsets: torch.Tensor, sorted_slot: torch.Tensor,
                   k_total: int, out: Optional[torch.Tensor] = None, workspace=None) -> torch.Tensor:
    """-> y_slots fp32 [T*k_total][hidden] (rows of dropped slots are left as allocated)."""
    T = x.shape[0]
    dev = x.device
    y = out if out is not None else torch.empty((T * k_total, W.hidden), dtype=torch.float32, device=dev)
    need = moe_expert_ffn_workspace_bytes(T, k_total, W)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(lib().moe_expert_ffn(_ptr(x), _act_dtype(x), T, k_total, ctypes.byref(W.c), _ptr(offsets),
                                _ptr(sorted_slot), _ptr(y), _ptr(ws), 0 if ws is None else ws.numel(),
                                _stream(dev)), "moe_expert_ffn")
    return y


MOE_FFN_STATIC_SCRATCH_BYTES = 16 << 20


def moe_expert_ffn_static(x: torch.Tensor, W: ExpertWeights, offsets: torch.Tensor, sorted_slot: torch.Tensor,
                          k_total: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_expert_ffn with the library's fixed device scratch array as its workspace (no workspace
    argument; calls needing more than MOE_FFN_STATIC_SCRATCH_BYTES are refused).  Only `out` may be
    allocated here, and only when the caller passes none."""
    T = x.shape[0]
    dev = x.device
    y = out if out is not None else torch.empty((T * k_total, W.hidden), dtype=torch.float32, device=dev)
    _check(lib().moe_expert_ffn_static(_ptr(x), _act_dtype(x), T, k_total, ctypes.byref(W.c), _ptr(offsets),
                                       _ptr(sorted_slot), _ptr(y), _stream(dev)), "moe_expert_ffn_static")
    return y


def moe_expert_ffn_plan(T: int, W: ExpertWeights, offsets: torch.Tensor, k_total: int,
                        workspace: torch.Tensor) -> None:
    """Step 1 of moe_expert_ffn: the tile schedule (from offsets) into `workspace`
    (moe_expert_ffn_workspace_bytes bytes), read by the two phases below."""
    xdt = MOE_ACT_FP16 if W.fmt == MOE_W_FP16 else MOE_ACT_BF16
    _check(lib().moe_expert_ffn_plan(xdt, T, k_total, ctypes.byref(W.c), _ptr(offsets), _ptr(workspace),
                                     workspace.numel(), _stream(offsets.device)),
           "moe_expert_ffn_plan")


def moe_expert_ffn_gateup(x: torch.Tensor, W: ExpertWeights, offsets: torch.Tensor, sorted_slot: torch.Tensor,
                          k_total: int, workspace: torch.Tensor) -> None:
    """Phase 1 of moe_expert_ffn: h into `workspace`, after moe_expert_ffn_plan on it."""
    T = x.shape[0]
    _check(lib().moe_expert_ffn_gateup(_ptr(x), _act_dtype(x), T, k_total, ctypes.byref(W.c), _ptr(offsets),
                                       _ptr(sorted_slot), _ptr(workspace), workspace.numel(), _stream(x.device)),
           "moe_expert_ffn_gateup")


def moe_expert_ffn_down(T: int, W: ExpertWeights, offsets: torch.Tensor, sorted_slot: torch.Tensor, k_total: int,
                        workspace: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """Phase 2 of moe_expert_ffn: y_slots from the h left in `workspace` by the gate/up phase."""
    xdt = MOE_ACT_FP16 if W.fmt == MOE_W_FP16 else MOE_ACT_BF16
    _check(lib().moe_expert_ffn_down(xdt, T, k_total, ctypes.byref(W.c), _ptr(offsets), _ptr(sorted_slot),
                                     _ptr(out), _ptr(workspace), workspace.numel(), _stream(out.device)),
           "moe_expert_ffn_down")
    return out


def moe_expert_ffn_f16_workspace_bytes(T: int, k_total: int, W: ExpertWeights) -> int:
    return lib().moe_expert_ffn_f16_workspace_bytes(T, k_total, ctypes.byref(W.c))


def moe_expert_ffn_f16(x: torch.Tensor, W: ExpertWeights, attenuation_log2: int, offsets: torch.Tensor,
                       sorted_slot: torch.Tensor, k_total: int, out: Optional[torch.Tensor] = None,
                       workspace=None) -> torch.Tensor:
    """Range-managed expert FFN (Cascadia Eq. 1): -> binary16 y_slots [T*k_total][hidden] holding
    E(x) / 2^attenuation_log2 (float16 tensor)."""
    T = x.shape[0]
    dev = x.device
    y = out if out is not None else torch.empty((T * k_total, W.hidden), dtype=torch.float16, device=dev)
    need = moe_expert_ffn_f16_workspace_bytes(T, k_total, W)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(lib().moe_expert_ffn_f16(_ptr(x), _act_dtype(x), T, k_total, ctypes.byref(W.c), attenuation_log2,
                                    _ptr(offsets), _ptr(sorted_slot), _ptr(y), _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(dev)), "moe_expert_ffn_f16")
    return y


def moe_combine_restore(y_slots: torch.Tensor, weights: torch.Tensor, attenuation_log2: int,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Eq. 1 combination of binary16 attenuated slots with row factors, restored to fp32 y [T][H]."""
    T, kt = weights.shape
    H = y_slots.shape[-1]
    y = out if out is not None else torch.empty((T, H), dtype=torch.float32, device=y_slots.device)
    _check(lib().moe_combine_restore(_ptr(y_slots), _ptr(weights), T, kt, H, attenuation_log2, _ptr(y),
                                     _stream(y_slots.device)), "moe_combine_restore")
    return y


def moe_combine(y_slots: torch.Tensor, weights: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    T, kt = weights.shape
    H = y_slots.shape[-1]
    y = out if out is not None else torch.empty((T, H), dtype=torch.float32, device=y_slots.device)
    _check(lib().moe_combine(_ptr(y_slots), _ptr(weights), T, kt, H, _ptr(y), _stream(y_slots.device)),
           "moe_combine")
    return y


def moe_mxfp4_dequant(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """[N][K/2] codes + [N][K/32] scales -> [N][K] bfloat16 (the FFN's decode primitive)."""
    N, K = codes.shape[0], codes.shape[1] * 2
    out = torch.empty((N, K), dtype=torch.bfloat16, device=codes.device)
    _check(lib().moe_mxfp4_dequant(_ptr(codes), _ptr(scales), N, K, codes.stride(0), scales.stride(0), _ptr(out),
                                   _stream(codes.device)), "moe_mxfp4_dequant")
    return out


def moe_stream_read(buf: torch.Tensor, sink: torch.Tensor) -> None:
    """Read every byte of the contiguous device tensor `buf` once with whole-line nontemporal loads
    (a measurement utility: timing it over a buffer far larger than the caches gives the practical
    HBM read rate).  `sink` is a one-element int32 device tensor whose contents are meaningless."""
    if not buf.is_contiguous() or sink.numel() < 1 or sink.dtype != torch.int32:
        raise ValueError("moe_stream_read: needs a contiguous buffer and an int32 sink")
    _check(lib().moe_stream_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), _stream(buf.device)),
           "moe_stream_read")


def _mx_fmt(fmt) -> int:
    return MX_FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def moe_mx_row_bytes(fmt, K: int) -> int:
    return lib().moe_mx_row_bytes(_mx_fmt(fmt), K)


def moe_mx_quantize(x: torch.Tensor, fmt) -> tuple:
    """[n][K] bf16/fp16 -> (packed codes uint8 [n][row bytes], E8M0 scales uint8 [n][K/32])."""
    n, K = x.shape
    f = _mx_fmt(fmt)
    codes = torch.empty((n, max(moe_mx_row_bytes(f, K), 1)), dtype=torch.uint8, device=x.device)
    scales = torch.empty((n, max(K // 32, 1)), dtype=torch.uint8, device=x.device)
    _check(lib().moe_mx_quantize(_ptr(x), _act_dtype(x), n, K, f, _ptr(codes), _ptr(scales), _stream(x.device)),
           "moe_mx_quantize")
    return codes, scales


def moe_expert_ffn_mx_workspace_bytes(T: int, k_total: int, W: ExpertWeights, fmt) -> int:
    return lib().moe_expert_ffn_mx_workspace_bytes(T, k_total, ctypes.byref(W.c), _mx_fmt(fmt))


def moe_expert_ffn_mx_workspace_layout(T: int, k_total: int, W: ExpertWeights, fmt) -> dict:
    """Byte offsets of the quantised x and h that moe_expert_ffn_mx leaves in its workspace."""
    offs = (ctypes.c_size_t * 4)()
    _check(lib().moe_expert_ffn_mx_workspace_layout(T, k_total, ctypes.byref(W.c), _mx_fmt(fmt), offs),
           "moe_expert_ffn_mx_workspace_layout")
    return dict(x_codes=offs[0], x_scales=offs[1], h_codes=offs[2], h_scales=offs[3])


def moe_expert_ffn_mx(x: torch.Tensor, W: ExpertWeights, fmt, offsets: torch.Tensor, sorted_slot: torch.Tensor,
                      k_total: int, out: Optional[torch.Tensor] = None, workspace=None) -> torch.Tensor:
    """MX mode of moe_expert_ffn (x and h quantised to the MX format `fmt`): -> y_slots fp32."""
    T = x.shape[0]
    dev = x.device
    f = _mx_fmt(fmt)
    y = out if out is not None else torch.empty((T * k_total, W.hidden), dtype=torch.float32, device=dev)
    need = moe_expert_ffn_mx_workspace_bytes(T, k_total, W, f)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(lib().moe_expert_ffn_mx(_ptr(x), _act_dtype(x), T, k_total, ctypes.byref(W.c), f, _ptr(offsets),
                                   _ptr(sorted_slot), _ptr(y), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream(dev)), "moe_expert_ffn_mx")
    return y


def moe_expert_ffn_mx_codes(x_codes: torch.Tensor, x_scales: torch.Tensor, W: ExpertWeights, fmt,
                            offsets: torch.Tensor, sorted_slot: torch.Tensor, k_total: int,
                            out: Optional[torch.Tensor] = None, workspace=None) -> torch.Tensor:
    """moe_expert_ffn_mx on an x given as MX codes [T][row bytes] and E8M0 scales [T][hidden/32] (uint8, as
    moe_mx_quantize and moe_add_rms_norm write them): -> y_slots fp32."""
    T = x_codes.shape[0]
    dev = x_codes.device
    f = _mx_fmt(fmt)
    _dense("moe_expert_ffn_mx_codes: x_codes", x_codes, torch.uint8, (T, moe_mx_row_bytes(f, W.hidden)))
    _dense("moe_expert_ffn_mx_codes: x_scales", x_scales, torch.uint8, (T, W.hidden // 32), x_codes.get_device())
    y = out if out is not None else torch.empty((T * k_total, W.hidden), dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else _workspace(moe_expert_ffn_mx_workspace_bytes(T, k_total, W, f), dev)
    _check(lib().moe_expert_ffn_mx_codes(_ptr(x_codes), _ptr(x_scales), T, k_total, ctypes.byref(W.c), f,
                                         _ptr(offsets), _ptr(sorted_slot), _ptr(y), _ptr(ws),
                                         0 if ws is None else ws.numel(), _stream(dev)), "moe_expert_ffn_mx_codes")
    return y


# ----------------------------------------------------------------------------------------------------
# In front of the layer.  These calls take few microseconds of GPU time at small T: descriptions are built once, a
# call checks what its pointers cannot tell and passes plain integers.
def _dense(what: str, t: torch.Tensor, dtype, shape, index: Optional[int] = None) -> None:
    """Contiguous, of this type and shape, and on GPU `index` (None: anywhere)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{what} must be on GPU {index}, got {t.device}")


def _rows(what: str, t: torch.Tensor, shape, index: int) -> int:
    """Row stride (in values) of a tensor of shape (rows, width) with contiguous rows on GPU `index` (-1: the CPU)."""
    if t.shape == shape and t.get_device() == index:
        far, near = t.stride()
        if near == 1 or shape[1] <= 1:
            return far if shape[0] > 1 else shape[1]
    raise ValueError(f"{what} must be [{shape[0]}][{shape[1]}] with contiguous rows on GPU {index}, got "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _on_gpu(what: str, ws: torch.Tensor, index: int) -> None:
    if ws.get_device() != index or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"{what} must be contiguous uint8 on GPU {index}, got {ws.dtype} on {ws.device}")


def _dtype(what: str, t: torch.Tensor) -> int:
    d = DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    return d


def _gpu(t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"needs a GPU tensor, got one on {t.device}")
    return index


def _enqueue(name: str, index: int, *args) -> None:
    """Calls the library on GPU `index` and its current stream (the last argument)."""
    fn = getattr(lib(), name)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status, name)


class RouteRule:
    """How experts are chosen from logits (moe_route_rule): score "softmax" or "sigmoid"; an optional fp32
    selection_bias [E] that moves the choice only; n_groups groups of which the topk_groups best stay, ranked by
    their two best keys ("top2") or their best ("max"); top_k experts, whose weights are renormalised or not and
    scaled; n_shared experts after them with a fixed weight."""

    def __init__(self, top_k: int, score: str = "softmax", selection_bias: Optional[torch.Tensor] = None,
                 n_groups: int = 1, topk_groups: int = 1, group_score: str = "top2", renormalise: bool = True,
                 routed_scale: float = 1.0, n_shared: int = 0, shared_weight: float = 1.0):
        if selection_bias is not None:
            _dense("RouteRule: selection_bias", selection_bias, torch.float32, (selection_bias.numel(),))
        self.selection_bias, self.top_k, self.n_shared, self.k_total = selection_bias, top_k, n_shared, top_k + n_shared
        self.c = moe_route_rule(SCORES[score], top_k, n_shared, n_groups, topk_groups, GROUP_SCORES[group_score],
                                int(bool(renormalise)), routed_scale, shared_weight,
                                None if selection_bias is None else selection_bias.data_ptr())
        self.at = ctypes.addressof(self.c)


def _route_out(rule: RouteRule, T: int, E: int, like: torch.Tensor, gpu: int, want_scores: bool, out):
    b = rule.selection_bias
    if b is not None and (b.numel() != E or b.get_device() != gpu):
        raise ValueError(f"the selection bias has {b.numel()} values on {b.device}, expected {E} on GPU {gpu}")
    shape = (T, rule.k_total)
    if out is None:
        dev = like.device
        return (torch.empty(shape, dtype=torch.int32, device=dev), torch.empty(shape, dtype=torch.float32, device=dev),
                torch.empty((T, E), dtype=torch.float32, device=dev) if want_scores else None)
    ids, w, scores = out
    _dense("ids", ids, torch.int32, shape, gpu)
    _dense("weights", w, torch.float32, shape, gpu)
    if scores is not None:
        _dense("scores", scores, torch.float32, (T, E), gpu)
    return out


def moe_select_experts(logits: torch.Tensor, rule: RouteRule, want_scores: bool = False, out=None):
    """The rule on router logits [T][E] (bf16, fp16 or fp32, contiguous rows)
    -> (ids int32 [T][k'], weights fp32 [T][k'], scores fp32 [T][E] or None)."""
    T, E = shape = logits.shape
    gpu = _gpu(logits)
    stride = _rows("moe_select_experts: logits", logits, shape, gpu)
    ids, w, scores = _route_out(rule, T, E, logits, gpu, want_scores, out)
    _enqueue("moe_select_experts", gpu, logits.data_ptr(), _dtype("logits", logits), stride, T, E, rule.at,
             ids.data_ptr(), w.data_ptr(), None if scores is None else scores.data_ptr())
    return ids, w, scores


def moe_route_grouped(x: torch.Tensor, w_router: torch.Tensor, rule: RouteRule, want_scores: bool = False, out=None,
                      workspace=None):
    """The rule on the logits x w_router^T -> (ids, weights, scores) as moe_select_experts."""
    T, H = x.shape
    E = w_router.shape[0]
    gpu = _gpu(x)
    _dense("moe_route_grouped: x", x, x.dtype, (T, H))
    _dense("moe_route_grouped: w_router", w_router, torch.float32, (E, H), gpu)
    ids, w, scores = _route_out(rule, T, E, x, gpu, want_scores, out)
    ws = workspace
    if ws is None:
        ws = _workspace(moe_route_workspace_bytes(T, H, E), x.device)
    else:
        _on_gpu("moe_route_grouped: workspace", ws, gpu)
    _enqueue("moe_route_grouped", gpu, x.data_ptr(), _act_dtype(x), T, H, w_router.data_ptr(), E, rule.at,
             ids.data_ptr(), w.data_ptr(), None if scores is None else scores.data_ptr(),
             None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return ids, w, scores


class RmsNorm:
    """Weight [hidden] (bf16, fp16 or fp32) and eps of a root-mean-square norm (moe_norm)."""

    def __init__(self, weight: torch.Tensor, eps: float = 1e-6):
        _dense("RmsNorm: weight", weight, weight.dtype, (weight.numel(),))
        self.weight, self.hidden = weight, weight.numel()
        self.c = moe_norm(weight.data_ptr(), _dtype("RmsNorm: weight", weight), self.hidden, eps)
        self.at = ctypes.addressof(self.c)


def moe_add_rms_norm(x: torch.Tensor, norm: RmsNorm, residual: Optional[torch.Tensor] = None, mx=None,
                     dtype: torch.dtype = torch.bfloat16, out=None):
    """s = x + residual, y = s * weight / sqrt(mean(s^2) + eps), rows of `norm.hidden` values
    -> (y, residual_out, codes, scales): y [T][hidden] in `dtype`; residual_out = s in the residual's type (None
    without a residual); for mx "fp8", "fp6" or "fp4" the MX codes and scales of y as moe_mx_quantize lays them
    out (None without).  `out` gives the four buffers; a None for y or residual_out there leaves that output
    out, and residual_out may be residual itself."""
    T, H = shape = x.shape
    gpu = _gpu(x)
    f = 0 if mx is None else _mx_fmt(mx)
    if norm.hidden != H or norm.weight.get_device() != gpu:
        raise ValueError(f"moe_add_rms_norm: rows of {H} values on GPU {gpu}, the weight has {norm.hidden} on "
                         f"{norm.weight.device}")
    xs = _rows("moe_add_rms_norm: x", x, shape, gpu)
    rp = rop = cp = sp = None
    rs = ros = rdt = 0
    if residual is not None:
        rs, rdt, rp = (_rows("moe_add_rms_norm: residual", residual, shape, gpu), _dtype("residual", residual),
                       residual.data_ptr())
    if out is None:
        dev = x.device
        y = torch.empty((T, H), dtype=dtype, device=dev)
        ro = None if residual is None else torch.empty((T, H), dtype=residual.dtype, device=dev)
        codes = scales = None
        if f:
            codes = torch.empty((T, moe_mx_row_bytes(f, H)), dtype=torch.uint8, device=dev)
            scales = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
    else:
        y, ro, codes, scales = out
        if y is not None:
            _dense("moe_add_rms_norm: y", y, y.dtype, shape, gpu)
        if f:
            if codes is None or scales is None:
                raise ValueError("moe_add_rms_norm: mx needs codes and scales")
            _dense("moe_add_rms_norm: codes", codes, torch.uint8,
                   (T, H if f == MOE_MX_FP8_E4M3 else moe_mx_row_bytes(f, H)), gpu)
            _dense("moe_add_rms_norm: scales", scales, torch.uint8, (T, H // 32), gpu)
        if ro is not None and (residual is None or ro.dtype is not residual.dtype):
            raise ValueError("moe_add_rms_norm: residual_out needs a residual of its type")
    if ro is not None:
        ros, rop = _rows("moe_add_rms_norm: residual_out", ro, shape, gpu), ro.data_ptr()
    if f:
        cp, sp = codes.data_ptr(), scales.data_ptr()
    _enqueue("moe_add_rms_norm", gpu, norm.at, x.data_ptr(), _dtype("x", x), xs, rp, rdt, rs, T, rop, ros,
             None if y is None else y.data_ptr(), 0 if y is None else _dtype("y", y), f, cp, sp)
    return y, ro, codes, scales


class LinearWeights:
    """One 4-bit weight matrix [n_out][k_in] for moe_linear, stored as one matrix of ExpertWeights: codes uint8
    [N][K/2]; scales uint8 [N][K/32] (mxfp4), binary16 bits as uint8 pairs [N][K/16] (int4g32) or E4M3 [N][K/16]
    (nvfp4); zeros uint8 [N][ceil(K/64)] (int4g32); tensor_scale fp32 [1] (nvfp4).  Rows may be strided."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, fmt: str = "mxfp4",
                 zeros: Optional[torch.Tensor] = None, tensor_scale: Optional[torch.Tensor] = None):
        self.fmt, self.n_out, self.k_in = W_FORMATS[fmt], codes.shape[0], 2 * codes.shape[1]
        self.device, self.index = codes.device, codes.get_device()
        K = self.k_in
        p = moe_proj()

        def rows(what, t, width):
            if t is None or t.dtype != torch.uint8 or t.shape[0] != self.n_out or t.device != codes.device:
                raise ValueError(f"LinearWeights: {what} must be uint8 [{self.n_out}][{width}] on {codes.device}")
            return t.data_ptr(), _rows(f"LinearWeights: {what}", t, (self.n_out, width), self.index)

        p.w, p.w_row_stride = rows("codes", codes, K // 2)
        p.scales, p.s_row_stride = rows("scales", scales, K // 32 if self.fmt == MOE_W_MXFP4 else K // 16)
        if self.fmt == MOE_W_INT4_G32:
            p.zeros, p.z_row_stride = rows("zeros", zeros, (K // 32 + 1) // 2)
        elif self.fmt == MOE_W_NVFP4:
            if tensor_scale is None or tensor_scale.device != codes.device:
                raise ValueError(f"LinearWeights: nvfp4 needs a tensor_scale on {codes.device}")
            _dense("LinearWeights: tensor_scale", tensor_scale, torch.float32, (1,))
            p.tensor_scale = tensor_scale.data_ptr()
        self.tensors = (codes, scales, zeros, tensor_scale)
        self._need = {}  # workspace bytes by T
        self.c = moe_linear_weights(self.fmt, self.n_out, K, p)
        self.at = ctypes.addressof(self.c)


def moe_linear_workspace_bytes(T: int, W: LinearWeights) -> int:
    need = W._need.get(T)
    if need is None:
        need = W._need[T] = lib().moe_linear_workspace_bytes(T, W.at)
    return need


def moe_linear(x: torch.Tensor, W: LinearWeights, bias: Optional[torch.Tensor] = None,
               dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None, workspace=None) -> torch.Tensor:
    """x [T][k_in] bf16 (rows contiguous) times W^T, plus an fp32 bias [n_out] -> y [T][n_out] in `dtype` (or in
    `out`'s type, whose rows may be strided)."""
    T = x.shape[0]
    gpu = _gpu(x)
    if W.index != gpu:
        raise ValueError(f"moe_linear: x is on GPU {gpu}, the weights on {W.device}")
    xs = _rows("moe_linear: x", x, (T, W.k_in), gpu)
    if bias is not None:
        _dense("moe_linear: bias", bias, torch.float32, (W.n_out,), gpu)
    if out is None:
        out = torch.empty((T, W.n_out), dtype=dtype, device=x.device)
    ys = _rows("moe_linear: out", out, (T, W.n_out), gpu)
    ws = workspace
    if ws is None:
        need = moe_linear_workspace_bytes(T, W)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _on_gpu("moe_linear: workspace", ws, gpu)
    _enqueue("moe_linear", gpu, x.data_ptr(), _act_dtype(x), xs, T, W.at, None if bias is None else bias.data_ptr(),
             out.data_ptr(), _dtype("out", out), ys, None if ws is None else ws.data_ptr(),
             0 if ws is None else ws.numel())
    return out


# ----------------------------------------------------------------------------------------------------
# Attention
def _heads(what: str, t: torch.Tensor, shape, index: int) -> tuple:
    """Fields of a moe_heads: a tensor [tokens][heads][head_dim] with contiguous heads on GPU `index` (-1: the CPU)."""
    if t.shape == shape and t.get_device() == index:
        ts, hs, ds = t.stride()
        if ds == 1 or shape[2] <= 1:
            dt = DTYPES.get(t.dtype)
            if dt is None:
                raise TypeError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
            return (t.data_ptr(), dt, ts if shape[0] > 1 else shape[1] * shape[2], hs if shape[1] > 1 else shape[2])
    raise ValueError(f"{what} must be {tuple(shape)} with contiguous heads on GPU {index}, got {tuple(t.shape)} with strides "
                     f"{t.stride()} on {t.device}")


_HEADS_BYTES = ctypes.sizeof(moe_heads)
_HEADS_PACKED = {n: (struct.Struct("@" + "Pi4xqq" * n), ctypes.c_char * (n * _HEADS_BYTES)) for n in (2, 4, 6)}
_NO_HEADS = (0, 0, 0, 0)


def _packed(fields: tuple, n: int):
    """n moe_heads behind one another, from their fields: one object instead of n (which a call of few microseconds
    would feel).  The caller keeps it until its call is made."""
    pack, kind = _HEADS_PACKED[n]
    return kind.from_buffer_copy(pack.pack(*fields))


def _ints(what: str, t: torch.Tensor, shape, index: int) -> int:
    if t.dtype is torch.int32 and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on GPU {index}, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}")


def _too_large(what: str, **sizes):
    """(ctypes would pass the lower 32 bits on.)"""
    raise ValueError(f"{what}: {', '.join(f'{k} = {v}' for k, v in sizes.items() if v >> 31 > 0)} does not fit 32 bits")


class Rope:
    """Cosines and sines of the positions' angles, fp32 [n_positions][rotary_dim / 2], and how values pair up
    (moe_rope): "halves" (i, i + rotary_dim / 2) or "neighbours" (2i, 2i + 1)."""

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, pairs: str = "halves"):
        _dense("Rope: cos", cos, torch.float32, cos.shape)
        _dense("Rope: sin", sin, torch.float32, cos.shape)
        if cos.dim() != 2 or cos.device != sin.device:
            raise ValueError(f"Rope: cos and sin must be [n_positions][rotary_dim / 2] on one device, got "
                             f"{tuple(cos.shape)} on {cos.device} and {sin.device}")
        self.cos, self.sin, self.index = cos, sin, cos.get_device()
        self.rotary_dim = 2 * cos.shape[1]
        self.c = moe_rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], self.rotary_dim, ROPE_PAIRS[pairs])
        self.at = ctypes.addressof(self.c)


class KvCache:
    """A paged key-value cache (moe_kv_cache) on given tensors k and v [n_pages][n_kv_heads][page_size][head_dim], of
    bf16, fp16 or (MXFP8) uint8 codes with scales uint8 [n_pages][n_kv_heads][page_size][head_dim / 32].  The last
    dimension is contiguous, the others may be strided (a cache kept token by token is given as a permuted view); k and v
    have the same strides.  KvCache.empty() allocates one, a head's tokens of a page next to each other."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        fmt = {t: f for f, t in KV_TYPES.items()}.get(k.dtype)
        if fmt is None or v.dtype != k.dtype:
            raise TypeError(f"KvCache: k and v must both be bfloat16, float16 or uint8, got {k.dtype} and {v.dtype}")
        self.fmt, self.tensors, self.device, self.index = fmt, (k, v, k_scales, v_scales), k.device, k.get_device()

        def strides(what, a, b, shape):
            if a is None or b is None or a.shape != shape or b.shape != shape or a.device != k.device \
                    or b.device != k.device or a.dtype != b.dtype:
                raise ValueError(f"KvCache: {what} must be {tuple(shape)} on {k.device}")
            sa, sb = a.stride(), b.stride()
            if any(x != y for x, y, n in zip(sa, sb, shape) if n > 1) or (sa[3] != 1 and shape[3] > 1):
                raise ValueError(f"KvCache: {what} must have the same strides and contiguous values, got {sa} and {sb}")
            return [x if n > 1 else 0 for x, n in zip(sa[:3], shape)]

        if k.dim() != 4:
            raise ValueError(f"KvCache: k must be [n_pages][n_kv_heads][page_size][head_dim], got {tuple(k.shape)}")
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        page, head, token = strides("k and v", k, v, k.shape)
        self.c = moe_kv_cache(fmt, self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, k.data_ptr(),
                              v.data_ptr(), page, head, token)
        if fmt == MOE_KV_MXFP8:
            if k_scales is None or k_scales.dtype != torch.uint8:
                raise ValueError("KvCache: uint8 codes need uint8 scales")
            page, head, token = strides("scales", k_scales, v_scales, k.shape[:3] + (self.head_dim // 32,))
            self.c.k_scales, self.c.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
            self.c.s_page_stride, self.c.s_head_stride, self.c.s_token_stride = page, head, token
        elif k_scales is not None or v_scales is not None:
            raise ValueError("KvCache: 16-bit values take no scales")
        self.act = torch.float16 if fmt == MOE_KV_FP16 else torch.bfloat16  # type of q and y
        self.at = ctypes.addressof(self.c)
        self._need = (None, 0)  # the last (B, heads, max_len) asked for and its workspace bytes

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, fmt: str = "bf16", device="cuda"):
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        make = lambda s, t: torch.empty(s, dtype=t, device=device)
        t = KV_TYPES[KV_FORMATS[fmt]]
        if fmt != "mxfp8":
            return cls(make(shape, t), make(shape, t))
        s = shape[:3] + (head_dim // 32,)
        return cls(make(shape, t), make(shape, t), make(s, torch.uint8), make(s, torch.uint8))


def moe_rope_cache(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                   rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                   cache: Optional[KvCache] = None, slots: Optional[torch.Tensor] = None, out=None):
    """q [T][n_q_heads][head_dim], k and v [T][n_kv_heads][head_dim] (bf16, fp16 or fp32, one type, strided tokens and
    heads) at int32 positions [T] -> (q, k, v) turned by the rope's angles (v as it is) in the cache's 16-bit type (bf16
    without a cache); the turned k, and v, also go to int32 slots [T] (page * page_size + token) of the cache.  q may be
    None, or k and v.  `out` gives the three buffers; a None there leaves that output out, and a buffer may be its input
    itself."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("moe_rope_cache: needs q or k")
    gpu = _gpu(x)
    T, _, D = x.shape
    if T >> 31:
        _too_large("moe_rope_cache", T=T)
    nq = 0 if q is None else q.shape[1]
    nkv = 0 if k is None else k.shape[1]
    if out is None:
        act = torch.bfloat16 if cache is None else cache.act
        out = tuple(None if t is None else torch.empty((T, n, D), dtype=act, device=x.device)
                    for t, n in ((q, nq), (k, nkv), (v if k is not None else None, nkv)))
    q_out, k_out, v_out = out
    qs, ks = (T, nq, D), (T, nkv, D)
    none = _NO_HEADS
    h = _packed((none if q is None else _heads("moe_rope_cache: q", q, qs, gpu))
                + (none if k is None else _heads("moe_rope_cache: k", k, ks, gpu))
                + (none if v is None else _heads("moe_rope_cache: v", v, ks, gpu))
                + (none if q_out is None else _heads("moe_rope_cache: q_out", q_out, qs, gpu))
                + (none if k_out is None else _heads("moe_rope_cache: k_out", k_out, ks, gpu))
                + (none if v_out is None else _heads("moe_rope_cache: v_out", v_out, ks, gpu)), 6)
    if rope is not None and rope.index != gpu or cache is not None and cache.index != gpu:
        raise ValueError(f"moe_rope_cache: the rope and the cache must be on GPU {gpu}")
    at, n = ctypes.addressof(h), _HEADS_BYTES
    _enqueue("moe_rope_cache", gpu, None if rope is None else rope.at,
             None if positions is None else _ints("moe_rope_cache: positions", positions, (T,), gpu), T, nq, nkv, D,
             None if q is None else at, None if k is None else at + n, None if v is None else at + 2 * n,
             None if q_out is None else at + 3 * n, None if k_out is None else at + 4 * n,
             None if v_out is None else at + 5 * n, None if cache is None else cache.at,
             None if slots is None else _ints("moe_rope_cache: slots", slots, (T,), gpu))
    return out


def moe_attention_prompt_workspace_bytes(Tq: int, Tk: int, n_seqs: int, n_q_heads: int, n_kv_heads: int,
                                         head_dim: int) -> int:
    return lib().moe_attention_prompt_workspace_bytes(Tq, Tk, n_seqs, n_q_heads, n_kv_heads, head_dim)


def _attention_out(what: str, q: torch.Tensor, out, want_lse: bool, gpu: int):
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device),
               torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if want_lse else None)
    y, lse = out
    h = _heads(f"{what}: out", y, q.shape, gpu)
    if lse is not None:
        _dense(f"{what}: lse", lse, torch.float32, q.shape[:2], gpu)
    return y, lse, h


def moe_attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                         cu_k: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = True,
                         window: int = 0, want_lse: bool = False, out=None, workspace=None):
    """Packed sequences: q [Tq][n_q_heads][head_dim], k and v [Tk][n_kv_heads][head_dim] (bf16 or fp16), sequence b's
    rows cu_q[b] .. cu_q[b+1] and keys cu_k[b] .. cu_k[b+1] (int32 [n + 1]; cu_k None: cu_q) -> (y like q, lse fp32
    [Tq][n_q_heads] or None).  scale None: head_dim ** -0.5.  Rows outside the sequences keep what `out` held."""
    gpu = _gpu(q)
    Tq, nq, D = q.shape
    Tk, nkv = k.shape[:2]
    n = cu_q.shape[0] - 1
    if (Tq | Tk | window) >> 31 > 0:
        _too_large("moe_attention_prompt", Tq=Tq, Tk=Tk, window=window)
    qh = _heads("moe_attention_prompt: q", q, (Tq, nq, D), gpu)
    kh = _heads("moe_attention_prompt: k", k, (Tk, nkv, D), gpu)
    vh = _heads("moe_attention_prompt: v", v, (Tk, nkv, D), gpu)
    y, lse, yh = _attention_out("moe_attention_prompt", q, out, want_lse, gpu)
    h = _packed(qh + kh + vh + yh, 4)
    cq = _ints("moe_attention_prompt: cu_q", cu_q, (n + 1,), gpu)
    ck = cq if cu_k is None else _ints("moe_attention_prompt: cu_k", cu_k, (n + 1,), gpu)
    ws = workspace
    if ws is None:
        ws = _workspace(moe_attention_prompt_workspace_bytes(Tq, Tk, n, nq, nkv, D), q.device)
    else:
        _on_gpu("moe_attention_prompt: workspace", ws, gpu)
    at, size = ctypes.addressof(h), _HEADS_BYTES
    _enqueue("moe_attention_prompt", gpu, at, at + size, at + 2 * size, cq, ck, n, Tq, Tk, nq, nkv, D,
             D ** -0.5 if scale is None else scale, int(bool(causal)), window, at + 3 * size,
             None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
             0 if ws is None else ws.numel())
    return y, lse


def moe_attention_decode_workspace_bytes(B: int, n_q_heads: int, cache: KvCache, max_len: int) -> int:
    key = (B, n_q_heads, max_len)
    last, need = cache._need
    if last != key:
        need = lib().moe_attention_decode_workspace_bytes(B, n_q_heads, cache.n_kv_heads, cache.head_dim, max_len)
        cache._need = (key, need)
    return need


def moe_attention_decode(q: torch.Tensor, cache: KvCache, page_table: torch.Tensor, lens: torch.Tensor,
                         max_len: Optional[int] = None, scale: Optional[float] = None, window: int = 0,
                         want_lse: bool = False, out=None, workspace=None):
    """One new token per sequence: q [B][n_q_heads][head_dim] over the lens[b] cached tokens (int32 [B]) on the pages
    page_table[b] (int32 [B][width], contiguous rows) -> (y like q, lse fp32 [B][n_q_heads] or None).  max_len (None: the
    table's width in tokens) bounds the lengths.  scale None: head_dim ** -0.5."""
    gpu = _gpu(q)
    B, nq, D = q.shape
    if cache.index != gpu:
        raise ValueError(f"moe_attention_decode: q is on GPU {gpu}, the cache on {cache.device}")
    qh = _heads("moe_attention_decode: q", q, (B, nq, cache.head_dim), gpu)
    y, lse, yh = _attention_out("moe_attention_decode", q, out, want_lse, gpu)
    h = _packed(qh + yh, 2)
    at = ctypes.addressof(h)
    if page_table.dtype is not torch.int32 or page_table.dim() != 2:
        raise ValueError(f"moe_attention_decode: page_table must be int32 [B][width], got {page_table.dtype}")
    width = page_table.shape[1]
    stride = _rows("moe_attention_decode: page_table", page_table, (B, width), gpu)
    if max_len is None:
        max_len = width * cache.page_size
    if (B | max_len | window) >> 31 > 0:
        _too_large("moe_attention_decode", B=B, max_len=max_len, window=window)
    ws = workspace
    if ws is None:
        need = moe_attention_decode_workspace_bytes(B, nq, cache, max_len)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _on_gpu("moe_attention_decode: workspace", ws, gpu)
    _enqueue("moe_attention_decode", gpu, at, B, nq, cache.at, page_table.data_ptr(), stride, width,
             _ints("moe_attention_decode: lens", lens, (B,), gpu), max_len, D ** -0.5 if scale is None else scale, window,
             at + _HEADS_BYTES, None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
             0 if ws is None else ws.numel())
    return y, lse


# ----------------------------------------------------------------------------------------------------
class MoELayer:
    """One routed-MoE layer with every intermediate buffer allocated once, so that forward() only
    enqueues the four library calls (capturable in a HIP graph)."""

    def __init__(self, W: ExpertWeights, T: int, top_k: int, n_shared: int = 0,
                 w_router: Optional[torch.Tensor] = None, logit_bias: Optional[torch.Tensor] = None,
                 mx=None):
        self.W, self.T, self.top_k, self.n_shared = W, T, top_k, n_shared
        self.mx = None if mx is None else _mx_fmt(mx)  # MX mode: activation format of the FFN
        self.w_router, self.logit_bias = w_router, logit_bias
        dev = W.device
        kt = top_k + n_shared
        self.k_total = kt
        H = W.hidden
        E = W.n_experts - n_shared
        self.dense = w_router is None  # all-active slices: caller-fixed ids j, weights 1
        if self.dense:
            self.ids = torch.arange(kt, dtype=torch.int32, device=dev).repeat(T, 1).contiguous()
            self.weights = torch.ones((T, kt), dtype=torch.float32, device=dev)
            self.route_ws = None
        else:
            self.ids = torch.empty((T, kt), dtype=torch.int32, device=dev)
            self.weights = torch.empty((T, kt), dtype=torch.float32, device=dev)
            self.route_ws = _workspace(moe_route_bucket_workspace_bytes(T, H, E, top_k, n_shared), dev)
        n = T * kt
        self.buckets = Buckets(torch.empty(W.n_experts, dtype=torch.int32, device=dev),
                               torch.empty(W.n_experts + 1, dtype=torch.int32, device=dev),
                               torch.empty(n, dtype=torch.int32, device=dev),
                               torch.empty(n, dtype=torch.int32, device=dev))
        self.bucket_ws = _workspace(moe_bucket_workspace_bytes(n, W.n_experts), dev)
        self.y_slots = torch.empty((n, H), dtype=torch.float32, device=dev)
        self.ffn_ws = _workspace(moe_expert_ffn_workspace_bytes(T, kt, W) if self.mx is None
                                 else moe_expert_ffn_mx_workspace_bytes(T, kt, W, self.mx), dev)
        self.y = torch.empty((T, H), dtype=torch.float32, device=dev)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if not self.dense and self.mx is None:
            # route, bucket and tile plan in one call, then the two FFN phases
            moe_route_bucket(x, self.w_router, self.top_k, self.logit_bias, self.n_shared, self.ids, self.weights,
                             self.buckets, self.W, self.ffn_ws, workspace=self.route_ws)
            moe_expert_ffn_gateup(x, self.W, self.buckets.offsets, self.buckets.sorted_slot, self.k_total, self.ffn_ws)
            moe_expert_ffn_down(self.T, self.W, self.buckets.offsets, self.buckets.sorted_slot, self.k_total,
                                self.ffn_ws, self.y_slots)
            return moe_combine(self.y_slots, self.weights, out=self.y)
        if not self.dense:
            moe_route(x, self.w_router, self.top_k, self.logit_bias, self.n_shared,
                      out=(self.ids, self.weights, None), workspace=self.route_ws)
        moe_bucket(self.ids, self.W.n_experts, out=self.buckets, workspace=self.bucket_ws)
        if self.mx is None:
            moe_expert_ffn(x, self.W, self.buckets.offsets, self.buckets.sorted_slot, self.k_total, out=self.y_slots,
                           workspace=self.ffn_ws)
        else:
            moe_expert_ffn_mx(x, self.W, self.mx, self.buckets.offsets, self.buckets.sorted_slot, self.k_total,
                              out=self.y_slots, workspace=self.ffn_ws)
        return moe_combine(self.y_slots, self.weights, out=self.y)


class MoEBlock:
    """The MoE half of a decoder block, its buffers allocated once for T tokens so that forward() only enqueues
    library calls (capturable in a HIP graph; a call that is given no residual_out allocates one): the attention output's projection (4-bit weights; left out
    without W_o), the residual addition and norm, routing by a rule, bucketing, the expert FFN and the combine.
    With mx ("fp8", "fp6", "fp4") the norm writes the MX codes that the expert FFN reads.

    forward(attn, residual) -> (y fp32 [T][H], residual_out): the next block's norm adds y to residual_out.

    Slots that a bias or logits that are not finite leave empty add nothing; a token none of whose logits is finite
    (NaN in its row, which residual_out shows) gets its shared experts alone, whose MX codes hold no NaN.  Passes of one block share its buffers, so they run one after
    another on one stream."""

    def __init__(self, W: ExpertWeights, T: int, rule: RouteRule, w_router: torch.Tensor, norm: RmsNorm,
                 W_o: Optional[LinearWeights] = None, mx=None):
        self.W, self.T, self.rule, self.w_router, self.norm, self.W_o = W, T, rule, w_router, norm, W_o
        self.mx = None if mx is None else _mx_fmt(mx)
        dev, H = W.device, W.hidden
        E = W.n_experts - rule.n_shared
        if w_router.shape != (E, H) or norm.hidden != H or (W_o is not None and W_o.n_out != H):
            raise ValueError(f"MoEBlock: hidden {H} and {E} routed experts do not fit the router, norm or projection")
        kt = self.k_total = rule.top_k + rule.n_shared
        n = T * kt
        act = torch.float16 if W.fmt == MOE_W_FP16 else torch.bfloat16
        self.a = None if W_o is None else torch.empty((T, H), dtype=torch.float32, device=dev)
        self.linear_ws = None if W_o is None else _workspace(moe_linear_workspace_bytes(T, W_o), dev)
        self.x = torch.empty((T, H), dtype=act, device=dev)
        self.codes = self.scales = None
        if self.mx is not None:
            self.codes = torch.empty((T, moe_mx_row_bytes(self.mx, H)), dtype=torch.uint8, device=dev)
            self.scales = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
        self.ids = torch.empty((T, kt), dtype=torch.int32, device=dev)
        self.weights = torch.empty((T, kt), dtype=torch.float32, device=dev)
        self.route_ws = _workspace(moe_route_workspace_bytes(T, H, E), dev)
        self.buckets = Buckets(torch.empty(W.n_experts, dtype=torch.int32, device=dev),
                               torch.empty(W.n_experts + 1, dtype=torch.int32, device=dev),
                               torch.empty(n, dtype=torch.int32, device=dev),
                               torch.empty(n, dtype=torch.int32, device=dev))
        self.bucket_ws = _workspace(moe_bucket_workspace_bytes(n, W.n_experts), dev)
        # whether the bias masks experts, so that slots may stay empty in every pass
        self.clear = rule.selection_bias is not None and not bool(torch.isfinite(rule.selection_bias).all())
        self.y_slots = torch.empty((n, H), dtype=torch.float32, device=dev)
        self.ffn_ws = _workspace(moe_expert_ffn_workspace_bytes(T, kt, W) if self.mx is None
                                 else moe_expert_ffn_mx_workspace_bytes(T, kt, W, self.mx), dev)
        self.y = torch.empty((T, H), dtype=torch.float32, device=dev)

    def forward(self, attn: torch.Tensor, residual: torch.Tensor, residual_out: Optional[torch.Tensor] = None):
        if attn.shape[0] != self.T:
            raise ValueError(f"MoEBlock: {attn.shape[0]} rows, built for {self.T}")
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        a = attn
        if self.W_o is not None:
            a = moe_linear(attn, self.W_o, out=self.a, workspace=self.linear_ws)
        moe_add_rms_norm(a, self.norm, residual, mx=self.mx, out=(self.x, residual_out, self.codes, self.scales))
        moe_route_grouped(self.x, self.w_router, self.rule, out=(self.ids, self.weights, None),
                          workspace=self.route_ws)
        b = moe_bucket(self.ids, self.W.n_experts, out=self.buckets, workspace=self.bucket_ws)
        if self.mx is None:
            moe_expert_ffn(self.x, self.W, b.offsets, b.sorted_slot, self.k_total, out=self.y_slots,
                           workspace=self.ffn_ws)
        else:
            moe_expert_ffn_mx_codes(self.codes, self.scales, self.W, self.mx, b.offsets, b.sorted_slot, self.k_total,
                                    out=self.y_slots, workspace=self.ffn_ws)
        return moe_combine(self.y_slots, self.weights, out=self.y), residual_out


class AttentionBlock:
    """The attention half of a decoder block, in front of MoEBlock: residual addition and norm, one 4-bit product for q,
    k and v (W_qkv: n_q_heads query heads, then n_kv_heads key and as many value heads), rotary positions and the cache
    write, attention.  Its row buffers are allocated once for up to T tokens, workspaces by each call, so a pass captures
    into a HIP graph.  Passes of one block share its buffers, so they run one after another on one stream.

    prompt(x, residual, positions, slots, cu) attends each sequence over its own rows, decode(x, residual, positions,
    slots, page_table, lens) each row over its cached tokens, its own (written to slots[b]) among them.  Both -> (attn
    [T'][n_q_heads * head_dim], residual_out), which MoEBlock.forward takes; x (an MoEBlock's y, or embeddings) and
    residual are [T'][hidden] for T' <= T tokens.  attn lies in the block's buffer: the next pass writes over it."""

    def __init__(self, W_qkv: LinearWeights, T: int, norm: RmsNorm, n_q_heads: int, cache: KvCache,
                 rope: Optional[Rope] = None, window: int = 0):
        D, nkv = cache.head_dim, cache.n_kv_heads
        if W_qkv.n_out != (n_q_heads + 2 * nkv) * D or W_qkv.k_in != norm.hidden:
            raise ValueError(f"AttentionBlock: {W_qkv.n_out} x {W_qkv.k_in} weights do not fit {n_q_heads} + 2 * {nkv} "
                             f"heads of {D} and a norm of {norm.hidden}")
        if cache.act is not torch.bfloat16:
            raise ValueError("AttentionBlock: 4-bit products take bf16 rows, so the cache is bf16 or mxfp8")
        self.W_qkv, self.T, self.norm, self.cache, self.rope, self.window = W_qkv, T, norm, cache, rope, window
        self.n_q_heads = n_q_heads
        empty = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=cache.device)
        self.x = empty(T, norm.hidden)
        self.qkv = torch.empty((T, W_qkv.n_out), dtype=torch.float32, device=cache.device)
        self.q, self.k, self.v, self.y = empty(T, n_q_heads, D), empty(T, nkv, D), empty(T, nkv, D), empty(T, n_q_heads, D)

    def _front(self, x, residual, positions, slots, residual_out, packed: bool):
        t = x.shape[0]
        if t > self.T:
            raise ValueError(f"AttentionBlock: {t} rows, built for {self.T}")
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        moe_add_rms_norm(x, self.norm, residual, out=(self.x[:t], residual_out, None, None))
        n, m = self.n_q_heads, self.cache.n_kv_heads
        qkv = moe_linear(self.x[:t], self.W_qkv, out=self.qkv[:t]).view(t, n + 2 * m, self.cache.head_dim)
        moe_rope_cache(qkv[:, :n], qkv[:, n:n + m], qkv[:, n + m:], self.rope,
                       None if self.rope is None else positions, self.cache, slots,
                       out=(self.q[:t], self.k[:t] if packed else None, self.v[:t] if packed else None))
        return t, residual_out

    def prompt(self, x: torch.Tensor, residual: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
               cu: torch.Tensor, residual_out: Optional[torch.Tensor] = None):
        t, residual_out = self._front(x, residual, positions, slots, residual_out, True)
        moe_attention_prompt(self.q[:t], self.k[:t], self.v[:t], cu, window=self.window, out=(self.y[:t], None))
        return self.y[:t].flatten(1), residual_out

    def decode(self, x: torch.Tensor, residual: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
               page_table: torch.Tensor, lens: torch.Tensor, max_len: Optional[int] = None,
               residual_out: Optional[torch.Tensor] = None):
        t, residual_out = self._front(x, residual, positions, slots, residual_out, False)
        moe_attention_decode(self.q[:t], self.cache, page_table, lens, max_len, window=self.window,
                             out=(self.y[:t], None))
        return self.y[:t].flatten(1), residual_out


class FixedShapeLayer:
    """A routed-MoE layer run at fixed row shapes (Cascadia Sec. 3.2): for each supported shape S
    the five calls (route, pad, bucket, expert FFN, combine) on S rows are captured once in a HIP
    graph; a call with T rows copies them into the shape's input buffer, writes T to the device
    row count, replays the graph of the smallest S >= T and returns the first T rows of y.  The
    padding rows carry zero routing weights and invalid ids, so they cost no expert work and
    change no real row.  Buffers are allocated once here; forward() allocates nothing."""

    def __init__(self, W: ExpertWeights, shapes, top_k: int, w_router: torch.Tensor,
                 logit_bias: Optional[torch.Tensor] = None, n_shared: int = 0):
        self.shapes = sorted(set(int(s) for s in shapes))
        self.W, self.top_k, self.n_shared = W, top_k, n_shared
        self.w_router, self.logit_bias = w_router, logit_bias
        dev = W.device
        S = self.shapes[-1]
        kt = top_k + n_shared
        self.k_total = kt
        H = W.hidden
        E = W.n_experts - n_shared
        self.x = torch.zeros((S, H), dtype=torch.bfloat16 if W.fmt == MOE_W_MXFP4 else torch.float16, device=dev)
        self.n_rows = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ids = torch.empty((S, kt), dtype=torch.int32, device=dev)
        self.weights = torch.empty((S, kt), dtype=torch.float32, device=dev)
        self.route_ws = _workspace(max(moe_route_workspace_bytes(s, H, E) for s in self.shapes), dev)
        self.buckets = Buckets(torch.empty(W.n_experts, dtype=torch.int32, device=dev),
                               torch.empty(W.n_experts + 1, dtype=torch.int32, device=dev),
                               torch.empty(S * kt, dtype=torch.int32, device=dev), None)
        self.bucket_ws = _workspace(max(moe_bucket_workspace_bytes(s * kt, W.n_experts) for s in self.shapes), dev)
        self.ffn_ws = _workspace(max(moe_expert_ffn_workspace_bytes(s, kt, W) for s in self.shapes), dev)
        self.y_slots = torch.empty((S * kt, H), dtype=torch.float32, device=dev)
        self.y = torch.empty((S, H), dtype=torch.float32, device=dev)
        self.graphs = {}

    def run_shape(self, S: int) -> None:
        """Enqueue the five calls for row shape S (eager; also what each graph holds)."""
        kt = self.k_total
        ids, w = self.ids[:S], self.weights[:S]
        moe_route(self.x[:S], self.w_router, self.top_k, self.logit_bias, self.n_shared, out=(ids, w, None),
                  workspace=self.route_ws)
        moe_pad_rows(self.n_rows, ids, w)
        b = Buckets(self.buckets.counts, self.buckets.offsets, self.buckets.sorted_slot[:S * kt], None)
        moe_bucket(ids, self.W.n_experts, out=b, workspace=self.bucket_ws)
        moe_expert_ffn(self.x[:S], self.W, b.offsets, b.sorted_slot, kt, out=self.y_slots[:S * kt],
                       workspace=self.ffn_ws)
        moe_combine(self.y_slots[:S * kt], w, out=self.y[:S])

    def capture(self) -> None:
        """Capture one graph per shape (after one eager pass of each on a side stream)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for S in self.shapes:
                self.run_shape(S)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for S in self.shapes:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.run_shape(S)
            self.graphs[S] = g
        torch.cuda.synchronize()

    def forward(self, x: torch.Tensor, use_graph: bool = True) -> torch.Tensor:
        """y[:T] for the T rows of x (a view into the layer's output buffer, valid until the next call)."""
        T = x.shape[0]
        S = moe_row_shape(T, self.shapes)
        if S < 0:
            raise ValueError(f"{T} rows exceed the largest supported row shape {self.shapes[-1]}")
        self.x[:T].copy_(x)
        self.n_rows.fill_(T)
        if use_graph:
            if not self.graphs:
                self.capture()
            self.graphs[S].replay()
        else:
            self.run_shape(S)
        return self.y[:T]


__all__ = ["moe_route", "moe_route_sigmoid", "moe_route_bucket", "moe_route_bucket_workspace_bytes", "moe_bucket", "moe_expert_ffn", "moe_expert_ffn_static", "moe_expert_ffn_f16",
           "moe_expert_ffn_f16_workspace_bytes", "moe_combine_restore", "moe_expert_ffn_plan", "moe_expert_ffn_gateup",
           "moe_expert_ffn_down", "moe_combine", "moe_mxfp4_dequant", "moe_mx_quantize", "moe_mx_row_bytes",
           "moe_expert_ffn_mx", "moe_expert_ffn_mx_workspace_bytes", "moe_stream_read", "moe_expert_ffn_mx_workspace_layout",
           "moe_route_workspace_bytes", "moe_bucket_workspace_bytes", "moe_expert_ffn_workspace_bytes",
           "moe_row_shape", "moe_pad_rows", "ExpertWeights", "Buckets", "MoELayer", "FixedShapeLayer", "MoEError",
           "moe_select_experts", "moe_route_grouped", "moe_add_rms_norm", "moe_linear", "moe_linear_workspace_bytes",
           "moe_expert_ffn_mx_codes", "RouteRule", "RmsNorm", "LinearWeights", "MoEBlock", "lib",
           "moe_rope_cache", "moe_attention_prompt", "moe_attention_prompt_workspace_bytes", "moe_attention_decode",
           "moe_attention_decode_workspace_bytes", "Rope", "KvCache", "AttentionBlock"]
