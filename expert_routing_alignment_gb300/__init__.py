"""Decode-time MoE layer for GB300 (sm_103a): Python binding of the C ABI.

Every function here marshals torch tensors into the C ABI of
``include/moe_gb300.h`` (``libmoe_gb300.so``) and returns; each step of the
layer runs in the library's CUDA kernels on the current torch stream (or the
stream passed in).  There is no fallback: if the library is missing or fails
to load, every call raises.

    import expert_routing_alignment_gb300 as moe
    ex = moe.Experts.from_tensors(moe.FMT_FP8_B128, E, H, I, gate, up, down)
    layer = moe.LayerDesc(top_k=8, block_size=16, routed=ex)
    ws = moe.alloc_workspace(layer, max_M=8)
    moe.moe_decode_layer(layer, x, out, ws, router_logits=logits)
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Optional, Sequence

import torch

from . import build as _build

MOE_OK = 0
MOE_EINVAL = 1
MOE_EUNSUPPORTED = 2
MOE_ECUDA = 3
MOE_ERR_BAD_ID = 0x1
MOE_ERR_BAD_POSITION = 0x4

FMT_FP8_B128 = 1
FMT_NVFP4_G16 = 2
FMT_NVFP4_GATE_UP = 3   # gate and up NVFP4_G16, down FP8_B128
PATH_AUTO = 0
PATH_SIMT = 1
PATH_TC = 2
PATH_SIMT_STAGED = 3
MOE_ERR_TIMEOUT = 0x2
MAX_EXPERTS = 1024
MAX_ROW_HIDDEN = 16384
DTYPE_BF16 = 1
DTYPE_F16 = 2
DTYPE_F32 = 3
DTYPE_E4M3 = 4
MAX_ROWS = 128
MAX_ROWS_TC = 4096   # M admitted on the tensor-core path (FP8 experts)
TOKEN_FORM_ROWS = 16   # tensor-core path: up to this M, x terms are kept by token
F4_TOKEN_COLUMNS_SMALL = 16   # NVFP4 tensor-core kernel: token columns for M <= 16
F4_TOKEN_COLUMNS = 32         # and for 16 < M <= 32 (its largest M)

LIB_PATH = _build.LIB


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        names = {1: "MOE_EINVAL", 2: "MOE_EUNSUPPORTED", 3: "MOE_ECUDA"}
        msg = f"{fn} failed: {names.get(status, status)}"
        if status == MOE_ECUDA:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


# --------------------------------------------------------------------------
# ctypes mirror of the header's structs
# --------------------------------------------------------------------------

class _Proj(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p)]


class _Experts(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("num_experts", ctypes.c_int), ("hidden", ctypes.c_int),
                ("inter", ctypes.c_int), ("gate", _Proj), ("up", _Proj), ("down", _Proj)]


class _LayerDesc(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int), ("block_size", ctypes.c_int), ("path", ctypes.c_int),
                ("routed", _Experts), ("shared", ctypes.POINTER(_Experts)),
                ("shared_gate", ctypes.c_void_p), ("router_weight", ctypes.c_void_p)]


class _WsView(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "topk_ids", "topk_w", "sorted_token_ids", "sorted_expert_ids", "expert_offsets",
        "token_to_perm", "active_experts", "active_count", "num_tokens_post_padded", "h",
        "h_shared", "y", "y_shared", "blend_counters", "router_logits", "shared_gate", "tc_x_terms", "tc_x_scale",
        "tc_h_terms", "tc_h_scale", "tc_done", "total_bytes")] + [
        ("max_total", ctypes.c_int), ("max_blocks", ctypes.c_int), ("cap", ctypes.c_int),
        ("tc_items", ctypes.c_size_t)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
EXPORTS = {
    "moe_version": (ctypes.c_char_p, []),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_cuda_error": (_I, []),
    "moe_align_sizes": (_I, [_I, _I, _I, _P, _P, _P]),
    "moe_align": (_I, [_P, _I, _I, _I, _I] + [_P] * 9),
    "moe_topk_softmax": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_router_logits": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "moe_grouped_gate_up": (_I, [ctypes.POINTER(_Experts), ctypes.POINTER(_Experts), _P, _I, _I,
                                 _P, _P, _P, _P, _P, _P, _I, _P]),
    "moe_grouped_down": (_I, [ctypes.POINTER(_Experts), ctypes.POINTER(_Experts), _P, _P, _I, _I,
                              _P, _P, _P, _P, _P, _P, _I, _P]),
    "moe_blend": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "moe_decode_layer_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(_LayerDesc), _I]),
    "moe_decode_layer_workspace_view": (_I, [ctypes.POINTER(_LayerDesc), _I,
                                             ctypes.POINTER(_WsView)]),
    "moe_decode_layer": (_I, [ctypes.POINTER(_LayerDesc), _P, _I, _P, _P, _P, _P, _P,
                              ctypes.c_size_t, _P, _P]),
    "moe_decode_layer_launches": (_I, [ctypes.POINTER(_LayerDesc), _I, _I]),
    "moe_decode_layer_noalloc": (_I, [ctypes.POINTER(_LayerDesc), _P, _I, _P, _P, _P, _P, _P,
                                      _P]),
    "moe_decode_experts": (_I, [ctypes.POINTER(_LayerDesc), _P, _I, _P, _P, ctypes.c_size_t, _P,
                                _P]),
    "moe_dispatch": (_I, [_P, _L, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _P]),
    "moe_dispatch_backward": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
    "moe_combine": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "moe_combine_backward": (_I, [_P, _L, _I, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P,
                                  _P]),
    "moe_topk_softmax_backward": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_add_rmsnorm": (_I, [_P, _L, _P, _L, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P, _P,
                             _P, _P]),
    "moe_add_rmsnorm_backward_workspace_bytes": (ctypes.c_size_t, [_I, _I]),
    "moe_add_rmsnorm_backward": (_I, [_P, _L, _P, _L, _P, _P, _P, _L, _I, _I, _I, _I, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "moe_decode_block": (_I, [ctypes.POINTER(_LayerDesc), _P, _P, _P, ctypes.c_float, _I, _P, _P,
                              _P, _P, ctypes.c_size_t, _P, _P]),
    "moe_quantize_nvfp4_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I]),
    "moe_quantize_nvfp4": (_I, [_P, _L, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P,
                                ctypes.c_size_t, _P]),
    "moe_dequantize_nvfp4": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_grouped_product_nvfp4": (_I, [ctypes.POINTER(_Proj), _I, _I, _I, _P, _P, _P, _I, _I, _I,
                                       _P, _P, _I, _I, _P, _P, _P]),
    "moe_grouped_gate_up_nvfp4": (_I, [ctypes.POINTER(_Proj), ctypes.POINTER(_Proj), _I, _I, _I,
                                       _P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _P, _P, _P]),
}

_lib: Optional[ctypes.CDLL] = None


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """The loaded library (built on first use when missing or stale)."""
    global _lib
    if _lib is None:
        if build_if_missing:
            _build.build()
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run expert_routing_alignment_gb300.build")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status, load().moe_last_cuda_error() if status == MOE_ECUDA else 0)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# --------------------------------------------------------------------------
# weight descriptors
# --------------------------------------------------------------------------

@dataclass
class Experts:
    """An expert set on the device (see moe_experts in the header).  Each
    projection is (codes, scale, global_scale or None)."""
    fmt: int
    num_experts: int
    hidden: int
    inter: int
    gate: Sequence
    up: Sequence
    down: Sequence
    _struct: _Experts = field(init=False, repr=False)

    def __post_init__(self):
        def proj(p):
            codes, scale, glob = (list(p) + [None])[:3]
            return _Proj(codes.data_ptr(), scale.data_ptr(),
                         None if glob is None else glob.data_ptr())
        self._struct = _Experts(self.fmt, self.num_experts, self.hidden, self.inter,
                                proj(self.gate), proj(self.up), proj(self.down))

    @staticmethod
    def from_synth(d) -> "Experts":
        """From a ``synth.ExpertData`` already on the device."""
        fmt = {"fp8": FMT_FP8_B128, "nvfp4": FMT_NVFP4_G16,
               "nvfp4_gate_up": FMT_NVFP4_GATE_UP}[d.fmt]
        t = lambda p: (p.codes, p.scale, p.glob)
        return Experts(fmt, d.E, d.H, d.I, t(d.gate), t(d.up), t(d.down))


@dataclass
class LayerDesc:
    top_k: int
    block_size: int
    routed: Experts
    shared: Optional[Experts] = None
    path: int = PATH_AUTO
    # bf16 [E, H] on the device: lets moe_decode_layer take x alone (hidden in)
    router_weight: Optional[torch.Tensor] = None
    # bf16 [H] on the device: gates the shared expert, sigmoid(x . shared_gate)
    shared_gate: Optional[torch.Tensor] = None
    _struct: _LayerDesc = field(init=False, repr=False)

    def __post_init__(self):
        sh = ctypes.pointer(self.shared._struct) if self.shared is not None else None
        self._struct = _LayerDesc(self.top_k, self.block_size, self.path, self.routed._struct, sh,
                                  _ptr(self.shared_gate), _ptr(self.router_weight))

    @property
    def num_experts(self) -> int:
        return self.routed.num_experts


# --------------------------------------------------------------------------
# entry points (same names as the C ABI)
# --------------------------------------------------------------------------

def moe_version() -> str:
    return load().moe_version().decode()


def moe_align_sizes(n: int, num_experts: int, block_size: int):
    a, b, c = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check("moe_align_sizes", load().moe_align_sizes(n, num_experts, block_size, ctypes.byref(a),
                                                      ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def alloc_align_outputs(n: int, num_experts: int, block_size: int, device="cuda") -> dict:
    max_total, max_blocks, cap = moe_align_sizes(n, num_experts, block_size)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(sorted_token_ids=torch.empty(max(max_total, 1), **i32),
                sorted_expert_ids=torch.empty(max(max_blocks, 1), **i32),
                expert_offsets=torch.empty(num_experts + 1, **i32),
                token_to_perm=torch.empty(max(n, 1), **i32),
                active_experts=torch.empty(max(cap, 1), **i32),
                active_count=torch.empty(1, **i32),
                num_tokens_post_padded=torch.empty(1, **i32),
                max_total=max_total, max_blocks=max_blocks, cap=cap)


def moe_align(topk_ids: torch.Tensor, num_experts: int, block_size: int,
              out: Optional[dict] = None, err_word: Optional[torch.Tensor] = None,
              stream=None) -> dict:
    """Alignment tables of the flat ids (int32 or int64, device), with their
    number as "num_slots" (buffers of ``out`` may be larger)."""
    ids = topk_ids.contiguous().view(-1)
    n = ids.numel()
    if out is None:
        out = alloc_align_outputs(n, num_experts, block_size, ids.device)
    _check("moe_align", load().moe_align(
        _ptr(ids), int(ids.dtype == torch.int64), n, num_experts, block_size,
        _ptr(out["sorted_token_ids"]), _ptr(out["sorted_expert_ids"]),
        _ptr(out["expert_offsets"]), _ptr(out["token_to_perm"]), _ptr(out["active_experts"]),
        _ptr(out["active_count"]), _ptr(out["num_tokens_post_padded"]), _ptr(err_word),
        _stream(stream)))
    out["num_slots"] = n
    return out


def moe_topk_softmax(logits: torch.Tensor, top_k: int, ids: Optional[torch.Tensor] = None,
                     w: Optional[torch.Tensor] = None, stream=None):
    M, E = logits.shape
    if ids is None:
        ids = torch.empty(M, top_k, dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty(M, top_k, dtype=torch.float32, device=logits.device)
    _check("moe_topk_softmax", load().moe_topk_softmax(_ptr(logits), M, E, top_k, _ptr(ids),
                                                       _ptr(w), _stream(stream)))
    return ids, w


def _dense(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> None:
    """The C entry points read plain row-major buffers: refuse anything else."""
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError(f"{name}: want a contiguous {dtype} tensor of shape {shape}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def moe_router_logits(x: torch.Tensor, router_weight: torch.Tensor,
                      logits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp32 logits [M, E] = x [M, H] (bf16) times router_weight [E, H] (bf16) transposed."""
    M, H = x.shape
    E = router_weight.shape[0]
    _dense("x", x, torch.bfloat16, (M, H))
    _dense("router_weight", router_weight, torch.bfloat16, (E, H))
    if logits is None:
        logits = torch.empty(M, E, dtype=torch.float32, device=x.device)
    _dense("logits", logits, torch.float32, (M, E))
    _check("moe_router_logits", load().moe_router_logits(_ptr(x), _ptr(router_weight), M, H, E,
                                                         _ptr(logits), _stream(stream)))
    return logits


def _sp(x: Optional[Experts]):
    return None if x is None else ctypes.pointer(x._struct)


def moe_grouped_gate_up(routed: Experts, shared: Optional[Experts], x: torch.Tensor, top_k: int,
                        tables: dict, h: torch.Tensor, h_shared: Optional[torch.Tensor] = None,
                        path: int = PATH_AUTO, stream=None) -> None:
    M = x.shape[0]
    _check("moe_grouped_gate_up", load().moe_grouped_gate_up(
        _sp(routed), _sp(shared), _ptr(x), M, top_k, _ptr(tables["expert_offsets"]),
        _ptr(tables["sorted_token_ids"]), _ptr(tables["active_experts"]),
        _ptr(tables["active_count"]), _ptr(h), _ptr(h_shared), path, _stream(stream)))


def moe_grouped_down(routed: Experts, shared: Optional[Experts], h: torch.Tensor,
                     h_shared: Optional[torch.Tensor], M: int, top_k: int, tables: dict,
                     y: torch.Tensor, y_shared: Optional[torch.Tensor] = None,
                     path: int = PATH_AUTO, stream=None) -> None:
    _check("moe_grouped_down", load().moe_grouped_down(
        _sp(routed), _sp(shared), _ptr(h), _ptr(h_shared), M, top_k,
        _ptr(tables["expert_offsets"]), _ptr(tables["sorted_token_ids"]),
        _ptr(tables["active_experts"]), _ptr(tables["active_count"]), _ptr(y), _ptr(y_shared),
        path, _stream(stream)))


def moe_blend(y: torch.Tensor, topk_w: torch.Tensor, token_to_perm: torch.Tensor,
              y_shared: Optional[torch.Tensor], out: torch.Tensor, top_k: int,
              x: Optional[torch.Tensor] = None, shared_gate: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """shared_gate (bf16 [H]) with x (bf16 [M, H]) gates the shared term by
    sigmoid(x[t] . shared_gate)."""
    M, H = out.shape
    if shared_gate is not None:
        if x is None:
            raise ValueError("shared_gate: x is required to compute the gate")
        _dense("x", x, torch.bfloat16, (M, H))
        _dense("shared_gate", shared_gate, torch.bfloat16, (H,))
    _check("moe_blend", load().moe_blend(_ptr(y), _ptr(topk_w), _ptr(token_to_perm),
                                         _ptr(y_shared), _ptr(x), _ptr(shared_gate), _ptr(out),
                                         M, top_k, H, _stream(stream)))


def workspace_bytes(layer: LayerDesc, max_M: int) -> int:
    nbytes = load().moe_decode_layer_workspace_bytes(ctypes.pointer(layer._struct), max_M)
    if nbytes == 0:
        raise MoeError("moe_decode_layer_workspace_bytes", MOE_EINVAL)
    return nbytes


def alloc_workspace(layer: LayerDesc, max_M: int, device="cuda") -> torch.Tensor:
    return torch.zeros(workspace_bytes(layer, max_M), dtype=torch.uint8, device=device)


def workspace_view(layer: LayerDesc, M: int, ws: torch.Tensor) -> dict:
    """Tensors aliasing the layer's intermediates inside the workspace."""
    v = _WsView()
    _check("moe_decode_layer_workspace_view",
           load().moe_decode_layer_workspace_view(ctypes.pointer(layer._struct), M,
                                                  ctypes.byref(v)))
    k, E = layer.top_k, layer.num_experts
    H, I = layer.routed.hidden, layer.routed.inter
    Is = layer.shared.inter if layer.shared is not None else 0

    def sl(off, count, dtype):
        nb = count * torch.tensor([], dtype=dtype).element_size()
        return ws[off: off + nb].view(dtype)

    tc = {}
    mt = v.max_total
    f4 = layer.routed.fmt in (FMT_NVFP4_G16, FMT_NVFP4_GATE_UP)
    if v.tc_h_terms and f4:
        # the NVFP4 tensor-core kernel: f16 h terms (hi, lo) [2][max_total][I],
        # the f16 x table [H/128][2][NT][64] of NT = 16 or 32 token columns
        nt = F4_TOKEN_COLUMNS_SMALL if M <= F4_TOKEN_COLUMNS_SMALL else F4_TOKEN_COLUMNS
        tc = dict(
            tc_h_terms=sl(v.tc_h_terms, 2 * mt * I, torch.float16).view(2, mt, I),
            tc_h_scale=sl(v.tc_h_scale, mt * (I // 128), torch.float32).view(mt, I // 128),
            tc_items=sl(v.tc_items, 4 * v.cap, torch.int32).view(v.cap, 4),
            tc_x_table=sl(v.tc_x_terms, nt * H, torch.float16).view(H // 128, 2, nt, 64),
            tc_x_scale=sl(v.tc_x_scale, nt, torch.float32))
    elif v.tc_h_terms:   # the FP8 tensor-core kernel's h terms and the active table
        tc = dict(
            tc_h_terms=sl(v.tc_h_terms, 3 * mt * I, torch.uint8).view(3, mt, I),
            tc_h_scale=sl(v.tc_h_scale, mt * (I // 128), torch.float32).view(mt, I // 128),
            tc_items=sl(v.tc_items, 4 * v.cap, torch.int32).view(v.cap, 4))
    if v.tc_x_terms and not f4 and M <= TOKEN_FORM_ROWS:   # x terms by token [H/128][2][16][128]
        tc.update(
            tc_x_table=sl(v.tc_x_terms, 2 * 16 * H, torch.uint8).view(H // 128, 2, 16, 128),
            tc_x_scale=sl(v.tc_x_scale, 16, torch.float32))
    elif v.tc_x_terms and not f4:   # x terms by sorted row [2][max_total][H]
        tc.update(
            tc_x_terms=sl(v.tc_x_terms, 2 * mt * H, torch.uint8).view(2, mt, H),
            tc_x_scale=sl(v.tc_x_scale, mt, torch.float32))

    return dict(
        topk_ids=sl(v.topk_ids, M * k, torch.int32), topk_w=sl(v.topk_w, M * k, torch.float32),
        sorted_token_ids=sl(v.sorted_token_ids, v.max_total, torch.int32),
        sorted_expert_ids=sl(v.sorted_expert_ids, v.max_blocks, torch.int32),
        expert_offsets=sl(v.expert_offsets, E + 1, torch.int32),
        token_to_perm=sl(v.token_to_perm, M * k, torch.int32),
        active_experts=sl(v.active_experts, v.cap, torch.int32),
        active_count=sl(v.active_count, 1, torch.int32),
        num_tokens_post_padded=sl(v.num_tokens_post_padded, 1, torch.int32),
        h=sl(v.h, v.max_total * I, torch.float32).view(v.max_total, I),
        h_shared=sl(v.h_shared, M * Is, torch.float32).view(M, Is),
        y=sl(v.y, v.max_total * H, torch.float32).view(v.max_total, H),
        y_shared=sl(v.y_shared, M * H, torch.float32).view(M, H),
        router_logits=sl(v.router_logits, M * E, torch.float32).view(M, E),
        shared_gate=sl(v.shared_gate, M, torch.float32),
        max_total=v.max_total, max_blocks=v.max_blocks, cap=v.cap, **tc)


def moe_decode_layer_launches(layer: LayerDesc, M: int, with_logits: int = 1) -> int:
    """Kernels one moe_decode_layer call enqueues (host only); with_logits 0:
    ids given, 1: logits given, 2: logits computed from x (hidden in)."""
    n = load().moe_decode_layer_launches(ctypes.pointer(layer._struct), M, int(with_logits))
    if n < 0:
        raise MoeError("moe_decode_layer_launches", MOE_EINVAL)
    return n


def moe_decode_layer(layer: LayerDesc, x: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                     router_logits: Optional[torch.Tensor] = None,
                     topk_ids: Optional[torch.Tensor] = None,
                     topk_w: Optional[torch.Tensor] = None,
                     err_word: Optional[torch.Tensor] = None, stream=None) -> None:
    M = x.shape[0]
    _check("moe_decode_layer", load().moe_decode_layer(
        ctypes.pointer(layer._struct), _ptr(x), M, _ptr(router_logits), _ptr(topk_ids),
        _ptr(topk_w), _ptr(out), _ptr(workspace), workspace.numel(), _ptr(err_word),
        _stream(stream)))


def moe_decode_experts(layer: LayerDesc, x: torch.Tensor, out: torch.Tensor,
                       workspace: torch.Tensor, err_word: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """The expert half of moe_decode_layer (grouped gate+up, down, blend) on
    the routing and alignment tables that an earlier moe_decode_layer call
    with the same layer and M left in this workspace, with this x."""
    M = x.shape[0]
    _check("moe_decode_experts", load().moe_decode_experts(
        ctypes.pointer(layer._struct), _ptr(x), M, _ptr(out), _ptr(workspace),
        workspace.numel(), _ptr(err_word), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20


def moe_decode_layer_noalloc(layer: LayerDesc, x: torch.Tensor, out: torch.Tensor,
                             router_logits: Optional[torch.Tensor] = None,
                             topk_ids: Optional[torch.Tensor] = None,
                             topk_w: Optional[torch.Tensor] = None,
                             err_word: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_decode_layer without a caller workspace, for callers that cannot
    allocate device memory: the library's fixed device array (32 MiB, shared
    by every call on the device) serves as the workspace."""
    M = x.shape[0]
    _check("moe_decode_layer_noalloc", load().moe_decode_layer_noalloc(
        ctypes.pointer(layer._struct), _ptr(x), M, _ptr(router_logits), _ptr(topk_ids),
        _ptr(topk_w), _ptr(out), _ptr(err_word), _stream(stream)))


# --------------------------------------------------------------------------
# tokens in expert order and back, the norm ahead of the router, gradients
# --------------------------------------------------------------------------

_FLOAT = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
# E4M3 rows: torch's float8 type, or the bytes
_ROWS = {**_FLOAT, torch.float8_e4m3fn: DTYPE_E4M3, torch.uint8: DTYPE_E4M3}

# These wrappers stand in front of kernels of a few microseconds, so they pass
# plain addresses, check each tensor once and ask for the current device and
# stream directly (a torch.cuda.Stream object costs more than the launch).
# torch has those two calls in a build with CUDA only, so they are looked up
# when a device tensor needs them, not when this module is imported.


def _on_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The kernels run on the current device: refuse tensors of any other."""
    dev = first.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"want CUDA tensors of the current device, got one on {first.device}")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"want tensors on one device, got {first.device} and {t.device}")
    return dev


def _handle(stream, dev: int) -> int:
    """The cudaStream_t of a stream argument; None: the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _kind(name: str, t: torch.Tensor, kinds: dict) -> int:
    kind = kinds.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name}: unsupported type {t.dtype}")
    return kind


def _at(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> int:
    """The address of a plain row-major buffer; anything else is refused."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {dtype} tensor of shape {shape}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _row_stride(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> int:
    """The distance of the rows of an input whose rows are dense."""
    if t.dtype is dtype and t.shape == shape:
        s0, s1 = t.stride()
        if s1 == 1 or shape[1] == 1:
            return s0 if shape[0] > 1 else shape[1]
    raise ValueError(f"{name}: want a {dtype} tensor of shape {shape} with dense rows, "
                     f"got {t.dtype} {tuple(t.shape)} strides {t.stride()}")


def _empty(shape: tuple, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """A new output: it belongs to the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else \
            torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _table(name: str, t: torch.Tensor, least: int) -> int:
    if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() < least or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous int32 tensor of at least {least} elements, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _num_rows(tables: dict) -> int:
    """Rows of the expert-order buffers: the tables' max_total."""
    n = tables["sorted_token_ids"].numel()
    return min(n, tables.get("max_total", n))


def _num_slots(tables: dict) -> Optional[int]:
    """The slots that the tables are of, which is also the slot that padding
    positions hold: moe_align's count, or as many as token_to_perm has."""
    n = tables.get("num_slots")
    if n is None:
        ttp = tables.get("token_to_perm")
        n = None if ttp is None else ttp.numel()
    return n


def _err(err_word: Optional[torch.Tensor]):
    if err_word is None:
        return None
    if err_word.dtype not in (torch.int32, torch.uint32) or err_word.numel() < 1:
        raise ValueError("err_word: want an int32 tensor")
    return err_word.data_ptr()


def moe_dispatch(x: torch.Tensor, tables: dict, top_k: int, rows: Optional[torch.Tensor] = None,
                 x_scale: Optional[torch.Tensor] = None,
                 rows_scale: Optional[torch.Tensor] = None,
                 err_word: Optional[torch.Tensor] = None, stream=None):
    """Token rows x [M, H] into expert order by moe_align's tables: rows
    [max_total, H], zeros in the padding, what was there behind the total
    (undefined in a new buffer).  E4M3 x (float8_e4m3fn, or the bytes) comes
    with x_scale fp32 [M, ceil(H / 128)]; then (rows, rows_scale)."""
    M, H = x.shape
    dtype, kind = x.dtype, _kind("x", x, _ROWS)
    xs = _row_stride("x", x, dtype, (M, H))
    ttp, sti = tables["token_to_perm"], tables["sorted_token_ids"]
    total, n_rows = tables["num_tokens_post_padded"], _num_rows(tables)
    t_at, s_at = _table("token_to_perm", ttp, M * top_k), _table("sorted_token_ids", sti, n_rows)
    n_at, e_at = _table("num_tokens_post_padded", total, 1), _err(err_word)
    if (kind == DTYPE_E4M3) != (x_scale is not None) or (rows_scale is not None
                                                         and x_scale is None):
        raise ValueError("x_scale, rows_scale: E4M3 rows have scales, others none")
    r_at = None if rows is None else _at("rows", rows, dtype, (n_rows, H))
    xs_at = rs_at = None
    if x_scale is not None:
        blocks = -(-H // 128)
        xs_at = _at("x_scale", x_scale, torch.float32, (M, blocks))
        if rows_scale is not None:
            rs_at = _at("rows_scale", rows_scale, torch.float32, (n_rows, blocks))
    dev = _on_device(x, ttp, sti, total, rows, x_scale, rows_scale, err_word)
    if r_at is None:
        rows = _empty((n_rows, H), dtype, x.device, stream)
        r_at = rows.data_ptr()
    if xs_at is not None and rs_at is None:
        rows_scale = _empty((n_rows, blocks), torch.float32, x.device, stream)
        rs_at = rows_scale.data_ptr()
    _check("moe_dispatch", load().moe_dispatch(
        x.data_ptr(), xs, xs_at, kind, M, top_k, H, t_at, s_at, n_at, n_rows, r_at, rs_at, e_at,
        _handle(stream, dev)))
    return rows if x_scale is None else (rows, rows_scale)


def moe_dispatch_backward(drows: torch.Tensor, tables: dict, M: int, top_k: int,
                          dx: Optional[torch.Tensor] = None,
                          err_word: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_dispatch: dx [M, H] = the sum over a token's slots of
    drows [max_total, H], fp32, rounded once."""
    dtype, kind, H = drows.dtype, _kind("drows", drows, _FLOAT), drows.shape[-1]
    ttp, n_rows = tables["token_to_perm"], _num_rows(tables)
    t_at, e_at = _table("token_to_perm", ttp, M * top_k), _err(err_word)
    r_at = _at("drows", drows, dtype, (n_rows, H))
    x_at = None if dx is None else _at("dx", dx, dtype, (M, H))
    dev = _on_device(drows, ttp, dx, err_word)
    if x_at is None:
        dx = _empty((M, H), dtype, drows.device, stream)
        x_at = dx.data_ptr()
    _check("moe_dispatch_backward", load().moe_dispatch_backward(
        r_at, kind, M, top_k, H, t_at, n_rows, x_at, e_at, _handle(stream, dev)))
    return dx


def moe_combine(rows: torch.Tensor, topk_w: torch.Tensor, tables: dict,
                out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                err_word: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [M, H] = sum_j topk_w[t, j] * rows[token_to_perm[t, j]], fp32, j
    ascending, rounded once to out's type (out_dtype, or rows')."""
    M, k = topk_w.shape
    kind, H = _kind("rows", rows, _FLOAT), rows.shape[-1]
    ttp, n_rows = tables["token_to_perm"], _num_rows(tables)
    t_at, e_at = _table("token_to_perm", ttp, M * k), _err(err_word)
    r_at = _at("rows", rows, rows.dtype, (n_rows, H))
    w_at = _at("topk_w", topk_w, torch.float32, (M, k))
    otype = out_dtype or (rows.dtype if out is None else out.dtype)
    okind = _FLOAT.get(otype)
    if okind is None:
        raise ValueError(f"out: unsupported type {otype}")
    o_at = None if out is None else _at("out", out, otype, (M, H))
    dev = _on_device(rows, topk_w, ttp, out, err_word)
    if o_at is None:
        out = _empty((M, H), otype, rows.device, stream)
        o_at = out.data_ptr()
    _check("moe_combine", load().moe_combine(
        r_at, kind, w_at, t_at, M, k, H, n_rows, okind, o_at, e_at, _handle(stream, dev)))
    return out


def moe_combine_backward(dout: torch.Tensor, rows: Optional[torch.Tensor], topk_w: torch.Tensor,
                         tables: dict, drows: Optional[torch.Tensor] = None,
                         dtopk_w: Optional[torch.Tensor] = None, want_drows: bool = True,
                         want_dtopk_w: bool = True, rows_dtype: Optional[torch.dtype] = None,
                         err_word: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_combine: (drows [max_total, H], dtopk_w [M, k]), None
    where it is not wanted.  drows has zeros in the padding and keeps what was
    there behind the total.  rows may be None when dtopk_w is not wanted: then
    drows has rows_dtype, or dout's type."""
    M, k = topk_w.shape
    okind, H = _kind("dout", dout, _FLOAT), dout.shape[-1]
    ds = _row_stride("dout", dout, dout.dtype, (M, H))
    ttp, sti = tables["token_to_perm"], tables["sorted_token_ids"]
    total, n_rows = tables["num_tokens_post_padded"], _num_rows(tables)
    t_at, s_at = _table("token_to_perm", ttp, M * k), _table("sorted_token_ids", sti, n_rows)
    n_at, e_at = _table("num_tokens_post_padded", total, 1), _err(err_word)
    w_at = _at("topk_w", topk_w, torch.float32, (M, k))
    r_at = None
    if rows is not None:
        rtype = rows.dtype
        r_at = _at("rows", rows, rtype, (n_rows, H))
    elif want_dtopk_w:
        raise ValueError("rows: needed for dtopk_w")
    else:
        rtype = rows_dtype or (drows.dtype if drows is not None else dout.dtype)
    if not want_drows and not want_dtopk_w:
        raise ValueError("neither drows nor dtopk_w is wanted")
    rkind = _FLOAT.get(rtype)
    if rkind is None:
        raise ValueError(f"rows: unsupported type {rtype}")
    if not want_drows:
        drows = None
    if not want_dtopk_w:
        dtopk_w = None
    dr_at = None if drows is None else _at("drows", drows, rtype, (n_rows, H))
    dw_at = None if dtopk_w is None else _at("dtopk_w", dtopk_w, torch.float32, (M, k))
    dev = _on_device(dout, rows, topk_w, ttp, sti, total, drows, dtopk_w, err_word)
    if want_drows and dr_at is None:
        drows = _empty((n_rows, H), rtype, dout.device, stream)
        dr_at = drows.data_ptr()
    if want_dtopk_w and dw_at is None:
        dtopk_w = _empty((M, k), torch.float32, dout.device, stream)
        dw_at = dtopk_w.data_ptr()
    _check("moe_combine_backward", load().moe_combine_backward(
        dout.data_ptr(), ds, okind, r_at, rkind, w_at, t_at, s_at, n_at, M, k, H, n_rows, dr_at,
        dw_at, e_at, _handle(stream, dev)))
    return drows, dtopk_w


def moe_topk_softmax_backward(topk_ids: torch.Tensor, topk_w: torch.Tensor,
                              dtopk_w: torch.Tensor, num_experts: int,
                              dlogits: Optional[torch.Tensor] = None,
                              err_word: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """Gradient of moe_topk_softmax: dlogits fp32 [M, E] from the weights'
    gradients dtopk_w [M, k]; 0 for every logit that was not selected."""
    M, k = shape = topk_w.shape
    i_at = _at("topk_ids", topk_ids, torch.int32, shape)
    w_at = _at("topk_w", topk_w, torch.float32, shape)
    d_at = _at("dtopk_w", dtopk_w, torch.float32, shape)
    l_at = None if dlogits is None else _at("dlogits", dlogits, torch.float32, (M, num_experts))
    e_at = _err(err_word)
    dev = _on_device(topk_ids, topk_w, dtopk_w, dlogits, err_word)
    if l_at is None:
        dlogits = _empty((M, num_experts), torch.float32, topk_w.device, stream)
        l_at = dlogits.data_ptr()
    _check("moe_topk_softmax_backward", load().moe_topk_softmax_backward(
        i_at, w_at, d_at, M, num_experts, k, l_at, e_at, _handle(stream, dev)))
    return dlogits


def _norm_output(name: str, dtype: torch.dtype, M: int, H: int) -> tuple:
    """(shape, type) of an output of moe_add_rmsnorm on rows of ``dtype``."""
    if name == "out" or name == "sum":
        return (M, H), dtype
    if name == "codes":
        return (M, H), torch.float8_e4m3fn
    if name == "scale":
        return (M, -(-H // 128)), torch.float32
    if name == "rstd":
        return (M,), torch.float32
    raise ValueError(f"no output {name!r}: want out, sum, codes, scale or rstd")


def alloc_add_rmsnorm_outputs(x: torch.Tensor, want: Sequence[str], stream=None) -> dict:
    """Buffers for moe_add_rmsnorm: "out", "sum" [M, H] of x's type, "codes"
    float8_e4m3fn [M, H] and "scale" fp32 [M, ceil(H / 128)], "rstd" fp32 [M]."""
    M, H = x.shape
    device = x.device
    return {name: _empty(*_norm_output(name, x.dtype, M, H), device, stream) for name in want}


def moe_add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                    residual: Optional[torch.Tensor] = None, want: Sequence[str] = ("out",),
                    out: Optional[dict] = None, stream=None) -> dict:
    """sum = x + residual (rounded to x's type), out = sum * rstd * weight with
    rstd = 1 / sqrt(mean(sum^2) + eps) by rows; "codes" and "scale" are out in
    E4M3 with a scale per 128 columns.  Writes the buffers of ``out``, or new
    ones for the outputs in ``want``, and returns them by name."""
    M, H = x.shape
    dtype, kind, wkind = x.dtype, _kind("x", x, _FLOAT), _kind("weight", weight, _FLOAT)
    xs = _row_stride("x", x, dtype, (M, H))
    rs, r_at = 0, None
    if residual is not None:
        rs, r_at = _row_stride("residual", residual, dtype, (M, H)), residual.data_ptr()
    w_at = _at("weight", weight, weight.dtype, (H,))
    at = {}
    if out is not None:
        for name, t in out.items():
            shape, otype = _norm_output(name, dtype, M, H)
            if name == "codes" and t.dtype is torch.uint8:
                otype = torch.uint8
            at[name] = _at(name, t, otype, shape)
        dev = _on_device(x, weight, residual, *out.values())
    else:
        dev, device, out = _on_device(x, weight, residual), x.device, {}
        for name in want:
            shape, otype = _norm_output(name, dtype, M, H)
            t = out[name] = _empty(shape, otype, device, stream)
            at[name] = t.data_ptr()
    get = at.get
    _check("moe_add_rmsnorm", load().moe_add_rmsnorm(
        x.data_ptr(), xs, r_at, rs, w_at, kind, wkind, M, H, eps, get("sum"), get("out"),
        get("codes"), get("scale"), get("rstd"), _handle(stream, dev)))
    return out


def add_rmsnorm_backward_workspace_bytes(M: int, hidden: int) -> int:
    nbytes = load().moe_add_rmsnorm_backward_workspace_bytes(M, hidden)
    if nbytes == 0:
        raise MoeError("moe_add_rmsnorm_backward_workspace_bytes", MOE_EINVAL)
    return nbytes


def moe_add_rmsnorm_backward(dout: torch.Tensor, sum: torch.Tensor, weight: torch.Tensor,
                             rstd: torch.Tensor, dsum: Optional[torch.Tensor] = None,
                             dx: Optional[torch.Tensor] = None,
                             dweight: Optional[torch.Tensor] = None, want_dweight: bool = True,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_add_rmsnorm from its "sum" and "rstd": (dx [M, H] of
    dout's type, dweight fp32 [H] or None).  dx is the gradient of x and of
    residual; dsum is the gradient that reaches "sum" from elsewhere.  The
    weight gradient needs a workspace (a new one when None)."""
    M, H = shape = dout.shape
    dtype, kind, wkind = dout.dtype, _kind("dout", dout, _FLOAT), _kind("weight", weight, _FLOAT)
    ds = _row_stride("dout", dout, dtype, shape)
    ss = _row_stride("sum", sum, dtype, shape)
    es, d_at = 0, None
    if dsum is not None:
        es, d_at = _row_stride("dsum", dsum, dtype, shape), dsum.data_ptr()
    w_at, r_at = _at("weight", weight, weight.dtype, (H,)), _at("rstd", rstd, torch.float32, (M,))
    x_at = None if dx is None else _at("dx", dx, dtype, shape)
    nbytes, g_at, ws_at = 0, None, None
    if not want_dweight:
        dweight = workspace = None
    else:
        if dweight is not None:
            g_at = _at("dweight", dweight, torch.float32, (H,))
        if workspace is not None:
            if not workspace.is_contiguous():
                raise ValueError("workspace: want a contiguous tensor")
            ws_at, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    dev = _on_device(dout, sum, weight, rstd, dsum, dx, dweight, workspace)
    if x_at is None:
        dx = _empty((M, H), dtype, dout.device, stream)
        x_at = dx.data_ptr()
    if want_dweight and g_at is None:
        dweight = _empty((H,), torch.float32, dout.device, stream)
        g_at = dweight.data_ptr()
    if want_dweight and workspace is None:
        nbytes = add_rmsnorm_backward_workspace_bytes(M, H)
        workspace = _empty((nbytes,), torch.uint8, dout.device, stream)
        ws_at = workspace.data_ptr()
    _check("moe_add_rmsnorm_backward", load().moe_add_rmsnorm_backward(
        dout.data_ptr(), ds, sum.data_ptr(), ss, w_at, r_at, d_at, es, kind, wkind, M, H, x_at,
        g_at, ws_at, nbytes, _handle(stream, dev)))
    return dx, dweight


def moe_decode_block(layer: LayerDesc, x: torch.Tensor, residual: Optional[torch.Tensor],
                     norm_weight: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                     eps: float = 1e-6, sum_out: Optional[torch.Tensor] = None,
                     normed: Optional[torch.Tensor] = None,
                     err_word: Optional[torch.Tensor] = None, stream=None):
    """The expert half of a block: sum = x + residual, normed = its RMS norm,
    out = moe_decode_layer(normed) with the layer's router weights.  Returns
    (sum, normed); sum_out may be residual's own buffer."""
    M, H = shape = x.shape
    bf16 = torch.bfloat16
    if H != layer.routed.hidden:
        raise ValueError(f"x: want rows of {layer.routed.hidden}, got {H}")
    x_at, o_at = _at("x", x, bf16, shape), _at("out", out, bf16, shape)
    r_at = None if residual is None else _at("residual", residual, bf16, shape)
    s_at = None if sum_out is None else _at("sum_out", sum_out, bf16, shape)
    n_at = None if normed is None else _at("normed", normed, bf16, shape)
    w_at, e_at = _at("norm_weight", norm_weight, bf16, (H,)), _err(err_word)
    dev = _on_device(x, residual, norm_weight, out, workspace, sum_out, normed, err_word)
    if s_at is None:
        sum_out = _empty((M, H), bf16, x.device, stream)
        s_at = sum_out.data_ptr()
    if n_at is None:
        normed = _empty((M, H), bf16, x.device, stream)
        n_at = normed.data_ptr()
    _check("moe_decode_block", load().moe_decode_block(
        ctypes.pointer(layer._struct), x_at, r_at, w_at, eps, M, s_at, n_at, o_at,
        workspace.data_ptr(), workspace.numel(), e_at, _handle(stream, dev)))
    return sum_out, normed


# --------------------------------------------------------------------------
# four-bit rows, and the products of four-bit rows and weights
# --------------------------------------------------------------------------

_U8, _E4M3, _F32 = torch.uint8, torch.float8_e4m3fn, torch.float32


def _bytes_at(name: str, t: torch.Tensor, shape: tuple) -> int:
    """The address of a dense buffer of bytes (scales: E4M3 values too)."""
    dtype = t.dtype
    if (dtype is not _U8 and dtype is not _E4M3) or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous uint8 tensor of shape {shape}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _packed(name: str, q) -> tuple:
    """(codes, scale, global_scale) of a dict of moe_quantize_nvfp4, or of the
    three tensors themselves."""
    if isinstance(q, dict):
        return q["codes"], q["scale"], q["global_scale"]
    if len(q) != 3:
        raise ValueError(f"{name}: want codes, scale and global_scale")
    return q


def _packed_at(name: str, q: tuple, codes_shape: tuple, scale_shape: tuple) -> tuple:
    """Their addresses."""
    codes, scale, glob = q
    if codes.dtype is not _U8:
        raise ValueError(f"{name} codes: want uint8, got {codes.dtype}")
    return (_bytes_at(name, codes, codes_shape), _bytes_at(name, scale, scale_shape),
            _at(name, glob, _F32, codes_shape[:1]))


def quantize_nvfp4_workspace_bytes(groups: int, rows: int, cols: int) -> int:
    nbytes = load().moe_quantize_nvfp4_workspace_bytes(groups, rows, cols)
    if nbytes == 0:
        raise MoeError("moe_quantize_nvfp4_workspace_bytes", MOE_EINVAL)
    return nbytes


def _quantized(name: str, dtype: torch.dtype, shape: tuple) -> tuple:
    """(shape, type) of an output of moe_quantize_nvfp4 on x."""
    if name == "codes":
        return (*shape[:-1], shape[-1] // 2), _U8
    if name == "scale":
        return (*shape[:-1], shape[-1] // 16), _U8
    if name == "global_scale":
        return shape[:1], _F32
    if name == "values":
        return shape, dtype
    raise ValueError(f"no output {name!r}: want codes, scale, global_scale or values")


def alloc_quantize_nvfp4_outputs(x: torch.Tensor,
                                 want: Sequence[str] = ("codes", "scale", "global_scale"),
                                 stream=None) -> dict:
    """Buffers for moe_quantize_nvfp4 of x."""
    shape, dtype, device = tuple(x.shape), x.dtype, x.device
    return {name: _empty(*_quantized(name, dtype, shape), device, stream) for name in want}


def moe_quantize_nvfp4(x: torch.Tensor, want: Sequence[str] = ("codes", "scale", "global_scale"),
                       global_scale: Optional[torch.Tensor] = None,
                       tables: Optional[dict] = None, out: Optional[dict] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """x in NVFP4: rows [M, H], each with a global scale of its own, or expert
    matrices [E, rows, cols], one for each expert; or under the scales that
    ``global_scale`` gives.  "codes" uint8 [..., H / 2], "scale" uint8 (E4M3)
    [..., H / 16], "global_scale" fp32 [M or E], and "values" of x's type and
    shape, what the codes stand for (for products of the user's own and
    gradients straight through the rounding).  With ``tables``, x's rows are in
    expert order and the padding rows are skipped.  Writes the buffers of
    ``out``, or new ones for the outputs in ``want``, and returns them by name."""
    dtype, kind, shape = x.dtype, _kind("x", x, _FLOAT), tuple(x.shape)
    if len(shape) == 2:
        groups, cols = shape
        rows, stride = 1, _row_stride("x", x, dtype, shape)
    elif len(shape) == 3:
        groups, rows, cols = shape
        s0, s1, s2 = x.stride()
        stride = s1 if rows > 1 else s0 if groups > 1 else cols
        if (s2 != 1 and cols > 1) or (groups > 1 and rows > 1 and s0 != rows * s1):
            raise ValueError(f"x: want evenly spaced dense rows, got strides {x.stride()}")
    else:
        raise ValueError(f"x: want [M, H] or [E, rows, cols], got {shape}")
    sti = s_at = g_at = None
    n = 0
    if tables is not None:
        sti = tables["sorted_token_ids"]
        if rows != 1 or len(shape) == 3 or _num_rows(tables) != groups:
            raise ValueError(f"x: want the tables' {_num_rows(tables)} rows, got {shape}")
        s_at, n = _table("sorted_token_ids", sti, groups), _num_slots(tables)
        if n is None:
            raise ValueError("tables: want num_slots or token_to_perm, the slots they are of")
    if global_scale is not None:
        g_at = _at("global_scale", global_scale, _F32, (groups,))
    at = {}
    if out is not None:
        for name, t in out.items():
            oshape, otype = _quantized(name, dtype, shape)
            at[name] = _bytes_at(name, t, oshape) if otype is _U8 else _at(name, t, otype, oshape)
        dev = _on_device(x, global_scale, workspace, sti, *out.values())
    else:
        dev, device, out = _on_device(x, global_scale, workspace, sti), x.device, {}
        for name in want:
            oshape, otype = _quantized(name, dtype, shape)
            if stream is None:   # as _empty, without a call
                t = torch.empty(oshape, dtype=otype, device=device)
            else:
                t = _empty(oshape, otype, device, stream)
            out[name] = t
            at[name] = t.data_ptr()
    nbytes, ws_at = 0, None
    if rows > 1 and g_at is None:
        if workspace is None:
            workspace = _empty((quantize_nvfp4_workspace_bytes(groups, rows, cols),), _U8, x.device,
                               stream)
        elif not workspace.is_contiguous():
            raise ValueError("workspace: want a contiguous tensor")
        ws_at, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    get = at.get
    _check("moe_quantize_nvfp4", load().moe_quantize_nvfp4(
        x.data_ptr(), stride, kind, groups, rows, cols, g_at, s_at, n, get("codes"), get("scale"),
        get("global_scale"), get("values"), ws_at, nbytes, _handle(stream, dev)))
    return out


def moe_dequantize_nvfp4(codes: torch.Tensor, scale: torch.Tensor, global_scale: torch.Tensor,
                         dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """The values of NVFP4 codes [M, H / 2] or [E, rows, cols / 2], of ``dtype``
    (or out's type): code * (scale * global_scale), rounded once."""
    lead, cols = tuple(codes.shape[:-1]), 2 * codes.shape[-1]
    if not 1 <= len(lead) <= 2:
        raise ValueError(f"codes: want [M, H / 2] or [E, rows, cols / 2], got {tuple(codes.shape)}")
    c_at, s_at, g_at = _packed_at("rows", (codes, scale, global_scale), (*lead, cols // 2),
                                  (*lead, cols // 16))
    if out is not None:
        dtype = out.dtype
    kind = _FLOAT.get(dtype)
    if kind is None:
        raise ValueError(f"out: unsupported type {dtype}")
    o_at = None if out is None else _at("out", out, dtype, (*lead, cols))
    dev = _on_device(codes, scale, global_scale, out)
    if o_at is None:
        out = _empty((*lead, cols), dtype, codes.device, stream)
        o_at = out.data_ptr()
    _check("moe_dequantize_nvfp4", load().moe_dequantize_nvfp4(
        c_at, s_at, g_at, lead[0], lead[1] if len(lead) == 2 else 1, cols, kind, o_at,
        _handle(stream, dev)))
    return out


def _grouped_nvfp4(fn: str, sets: tuple, rows, tables: dict, top_k: int, M: Optional[int],
                   out: Optional[torch.Tensor], out_dtype: Optional[torch.dtype], err_word,
                   stream) -> torch.Tensor:
    sets = [_packed("weight", w) for w in sets]
    shape = tuple(sets[0][0].shape)
    if len(shape) != 3:
        raise ValueError(f"weight codes: want [E, rows, cols / 2], got {shape}")
    E, R, C = shape
    C *= 2
    w_shape = (E, R, C // 16)
    projs = [_Proj(*_packed_at("weight", w, shape, w_shape)) for w in sets]
    codes, scale, glob = x = _packed("rows", rows)
    by_token, n_rows = M is None, _num_rows(tables)
    if by_token:
        M = codes.shape[0]
    slots = _num_slots(tables)
    if slots is not None and M * top_k != slots:
        raise ValueError(f"want the {slots} slots of the tables, got {M} tokens of {top_k}")
    n = M if by_token else n_rows
    x_at = _packed_at("rows", x, (n, C // 2), (n, C // 16))
    offs, sti = tables["expert_offsets"], tables["sorted_token_ids"]
    f_at, s_at = _table("expert_offsets", offs, E + 1), _table("sorted_token_ids", sti, n_rows)
    e_at = _err(err_word)
    otype = out_dtype or (torch.bfloat16 if out is None else out.dtype)
    okind = _FLOAT.get(otype)
    if okind is None:
        raise ValueError(f"out: unsupported type {otype}")
    o_at = None if out is None else _at("out", out, otype, (n_rows, R))
    dev = _on_device(codes, scale, glob, *sets[0], *(sets[1] if len(sets) > 1 else ()), offs, sti,
                     out, err_word)
    if o_at is None:
        out = _empty((n_rows, R), otype, codes.device, stream)
        o_at = out.data_ptr()
    _check(fn, getattr(load(), fn)(*map(ctypes.byref, projs), E, R, C, *x_at, by_token, M, top_k,
                                   f_at, s_at, n_rows, okind, o_at, e_at, _handle(stream, dev)))
    return out


def moe_grouped_product_nvfp4(weight, rows, tables: dict, top_k: int, M: Optional[int] = None,
                              out: Optional[torch.Tensor] = None,
                              out_dtype: Optional[torch.dtype] = None,
                              err_word: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """out [max_total, R] = each real position's row times its expert's matrix:
    weight (codes [E, R, C / 2], scale, global_scale) and rows (the same of
    moe_quantize_nvfp4, as its dict or in that order), four bits both, under
    scales without a sign, as the tensor cores take them.  Without M the rows are
    the tokens' own, read through the tables; with M, the number of tokens, they
    are in expert order, [max_total, C].  The tables are those of as many tokens
    and top_k (their "num_slots", or token_to_perm's length without it).  out has
    out_dtype (bf16 by default); its padding rows stay as they were (undefined in
    a new buffer)."""
    return _grouped_nvfp4("moe_grouped_product_nvfp4", (weight,), rows, tables, top_k, M, out,
                          out_dtype, err_word, stream)


def moe_grouped_gate_up_nvfp4(gate, up, rows, tables: dict, top_k: int, M: Optional[int] = None,
                              out: Optional[torch.Tensor] = None,
                              out_dtype: Optional[torch.dtype] = None,
                              err_word: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """moe_grouped_product_nvfp4 with two sets of the same sizes:
    out = silu(rows x gate) * (rows x up), in fp32 before its rounding."""
    return _grouped_nvfp4("moe_grouped_gate_up_nvfp4", (gate, up), rows, tables, top_k, M, out,
                          out_dtype, err_word, stream)
