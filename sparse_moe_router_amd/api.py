"""Python binding of libmoe.so -- argument marshalling only.

Each function has the name of the C entry point it calls and takes torch
tensors (device memory) instead of raw pointers.  Every step of the layer runs
in the HIP kernels behind the C ABI; nothing here computes.  If the library is
missing the binding raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")
# the same entry points with device range checks of caller-provided routing
# arrays (select it with use_debug_library)
DEBUG_LIB_PATH = os.path.join(_HERE, "libmoe_debug.so")

MOE_OK, MOE_E_ARG, MOE_E_UNSUPPORTED, MOE_E_WORKSPACE, MOE_E_DEVICE = range(5)
MOE_Q4_SYM_G32, MOE_Q2_ASYM_G32, MOE_Q3_SYM_G32 = 1, 2, 3
MOE_ACT_F32, MOE_ACT_BF16 = 0, 1
QFMT = {"q4_sym_g32": MOE_Q4_SYM_G32, "q2_asym_g32": MOE_Q2_ASYM_G32, "q3_sym_g32": MOE_Q3_SYM_G32}
CODE_BITS = {MOE_Q4_SYM_G32: 4, MOE_Q3_SYM_G32: 3, MOE_Q2_ASYM_G32: 2}
ACT = {"f32": MOE_ACT_F32, "bf16": MOE_ACT_BF16}

EXPORTS = ("moe_router_topk", "moe_permute", "moe_expert_ffn_q", "moe_expert_gate_up_q", "moe_expert_down_q",
           "moe_combine", "moe_layer_forward", "moe_layer_forward_noalloc",
           "moe_workspace_bytes", "moe_stack_forward", "moe_linear_q", "moe_beam_select", "moe_beam_workspace_bytes",
           "moe_beam_reorder", "moe_dequant", "moe_status_str", "moe_abi_version", "moe_range_checks")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg}")
        self.status = status


class c_qmat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("mins", ctypes.c_void_p)]


class c_experts(ctypes.Structure):
    _fields_ = [("gate", c_qmat), ("up", c_qmat), ("down", c_qmat), ("n", ctypes.c_int32)]


class c_layer(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("qfmt", ctypes.c_int32), ("act", ctypes.c_int32),
                ("router_w", ctypes.c_void_p), ("router_b", ctypes.c_void_p),
                ("routed", c_experts), ("shared", c_experts), ("hot_experts", ctypes.c_int32)]


class c_linear(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("qfmt", ctypes.c_int32), ("act", ctypes.c_int32),
                ("out", ctypes.c_int32), ("w", c_qmat), ("bias", ctypes.c_void_p)]


class c_beam(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("beams", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("n_out", ctypes.c_int32), ("act", ctypes.c_int32), ("eos", ctypes.c_int32)]


class c_state(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("chunk_bytes", ctypes.c_int64),
                ("chunks", ctypes.c_int64), ("src_row_stride", ctypes.c_int64), ("src_chunk_stride", ctypes.c_int64),
                ("dst_row_stride", ctypes.c_int64), ("dst_chunk_stride", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m sparse_moe_router_amd.build` "
                               "(there is no non-HIP fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        lp = ctypes.POINTER(c_layer)
        sigs = {
            "moe_router_topk": [lp, vp, i32, vp, vp, vp, vp, sz, vp],
            "moe_permute": [lp, vp, i32, vp, vp, vp, vp, sz, vp],
            "moe_expert_ffn_q": [lp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_expert_gate_up_q": [lp, vp, i32, vp, vp, vp, vp, vp, vp],
            "moe_expert_down_q": [lp, vp, vp, i32, vp, vp, vp, vp, vp, vp],
            "moe_combine": [lp, vp, vp, vp, vp, i32, vp, vp, vp, vp],
            "moe_layer_forward": [lp, vp, i32, vp, vp, vp, vp, vp, sz, vp],
            "moe_layer_forward_noalloc": [lp, vp, i32, vp, vp, vp, vp, vp],
            "moe_stack_forward": [lp, i32, vp, i32, vp, vp, sz, vp],
            "moe_dequant": [ctypes.POINTER(c_qmat), i32, i32, i32, vp, vp],
            "moe_linear_q": [ctypes.POINTER(c_linear), vp, ctypes.c_int64, i32, vp, ctypes.c_int64, vp],
            "moe_beam_select": [ctypes.POINTER(c_beam), vp, ctypes.c_int64, vp, vp, vp, ctypes.c_int64, vp, vp, vp, vp,
                                sz, vp],
            "moe_beam_reorder": [ctypes.POINTER(c_state), i32, vp, ctypes.c_int64, i32, i32, vp],
        }
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [lp, i32]
        L.moe_workspace_bytes.restype = sz
        L.moe_beam_workspace_bytes.argtypes = [ctypes.POINTER(c_beam)]
        L.moe_beam_workspace_bytes.restype = sz
        L.moe_status_str.argtypes = [ctypes.c_int]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = i32
        L.moe_range_checks.argtypes = []
        L.moe_range_checks.restype = i32
        _lib = L
    return _lib


def use_debug_library(debug: bool = True):
    """Route every later call to the debug library (or back to the release
    one).  Layer objects and workspaces stay valid across the switch."""
    global LIB_PATH, _lib
    path = DEBUG_LIB_PATH if debug else os.path.join(_HERE, "libmoe.so")
    if path != LIB_PATH:
        LIB_PATH, _lib = path, None


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status, lib().moe_status_str(status).decode())


def _need(name: str, t: Optional[torch.Tensor], n: int, dtype=None):
    """Type, dtype and size of one argument: at least ``n`` elements.

    Checked for every buffer before anything is marshalled: the C ABI receives
    bare pointers, so a buffer that is too small would turn into a device
    access out of bounds."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name}: {t.numel()} elements, at least {n} needed")


def _ptr(t: Optional[torch.Tensor], dtype=None, device=None) -> Optional[int]:
    """Device address of a contiguous tensor (on ``device`` when given)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError("tensor must live in device memory")
    if device is not None and t.device != device:
        raise ValueError(f"tensor on {t.device}, the layer's weights on {device}")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _act_dtype(act: int):
    return torch.bfloat16 if act == MOE_ACT_BF16 else torch.float32


class Layer:
    """A moe_layer descriptor over device tensors (kept alive by this object).

    routed / shared: dict(gate=(codes, scales, mins), up=(...), down=(...)) with
    codes uint8 [n][rows][...], scales and mins int16/uint16-bit fp16 planes
    [n][rows][cols/32] (mins None for the 4-bit format).
    """

    def __init__(self, *, hidden: int, inter: int, n_experts: int, top_k: int, qfmt, act,
                 router_w: torch.Tensor, router_b: Optional[torch.Tensor], routed: dict,
                 shared: Optional[dict] = None, hot_experts: int = 0):
        self.qfmt = QFMT.get(qfmt, qfmt)
        self.act = ACT.get(act, act)
        self.hidden, self.inter, self.n_experts, self.top_k = hidden, inter, n_experts, top_k
        self.act_dtype = _act_dtype(self.act)
        self.device = router_w.device
        self._keep = [router_w, router_b, routed, shared]
        if router_w.shape != (n_experts, hidden):
            raise ValueError("router_w must be [E][H]")
        if router_b is not None and router_b.shape != (n_experts,):
            raise ValueError("router_b must be [E]")
        if self.qfmt not in CODE_BITS:
            raise ValueError(f"unknown format {qfmt!r}")
        cb = CODE_BITS[self.qfmt]
        dev = self.device

        def qm(parts, n, rows, cols):
            codes, scales, mins = parts
            if codes.dtype != torch.uint8 or tuple(codes.shape) != (n, rows, cols * cb // 8):
                raise ValueError(f"codes must be uint8 [{n}][{rows}][{cols * cb // 8}], got {codes.dtype} {tuple(codes.shape)}")
            if scales.element_size() != 2 or tuple(scales.shape) != (n, rows, cols // 32):
                raise ValueError("scales must be 16-bit [n][rows][cols/32]")
            if (mins is None) != (self.qfmt != MOE_Q2_ASYM_G32):
                raise ValueError("mins are required for the 2-bit format only")
            if mins is not None and (mins.element_size() != 2 or tuple(mins.shape) != (n, rows, cols // 32)):
                raise ValueError("mins must be 16-bit [n][rows][cols/32]")
            return c_qmat(_ptr(codes, device=dev), _ptr(scales, device=dev), _ptr(mins, device=dev))

        def ex(d, n):
            if d is None:
                return c_experts(c_qmat(), c_qmat(), c_qmat(), 0)
            return c_experts(qm(d["gate"], n, inter, hidden), qm(d["up"], n, inter, hidden),
                             qm(d["down"], n, hidden, inter), n)

        self.c = c_layer(hidden, inter, n_experts, top_k, self.qfmt, self.act,
                         _ptr(router_w, torch.float32), _ptr(router_b, torch.float32, dev),
                         ex(routed, n_experts), ex(shared, 1), int(hot_experts))

    @property
    def ref(self):
        return ctypes.byref(self.c)


def moe_workspace_bytes(layer: Layer, T_max: int) -> int:
    return int(lib().moe_workspace_bytes(layer.ref, int(T_max)))


def workspace(layer: Layer, T_max: int, device=None) -> torch.Tensor:
    """A device workspace tensor of moe_workspace_bytes(layer, T_max) bytes."""
    n = moe_workspace_bytes(layer, T_max)
    if n == 0:
        raise MoeError("moe_workspace_bytes", MOE_E_ARG, "invalid layer descriptor or T")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _ws(layer: Layer, ws):
    return (None, 0) if ws is None else (_ptr(ws, torch.uint8, layer.device), ws.numel())


def _x(layer: Layer, x: torch.Tensor, T: int):
    if not isinstance(x, torch.Tensor) or x.dtype != layer.act_dtype or x.dim() != 2 or \
            x.shape[1] != layer.hidden or x.shape[0] < T:
        raise ValueError(f"x must be {layer.act_dtype} [>=T][{layer.hidden}]")
    return _ptr(x, device=layer.device)


def _p(layer: Layer, t, dtype=None):
    return _ptr(t, dtype, layer.device)


def moe_router_topk(layer: Layer, x, T, topk_ids, topk_w, logits=None, ws=None, stream=None):
    K, E = layer.top_k, layer.n_experts
    _need("topk_ids", topk_ids, T * K, torch.int32)
    _need("topk_w", topk_w, T * K, torch.float32)
    _need("logits", logits, T * E, torch.float32)
    w, wn = _ws(layer, ws)
    _check("moe_router_topk", lib().moe_router_topk(layer.ref, _x(layer, x, T), int(T), _p(layer, topk_ids),
                                                    _p(layer, topk_w), _p(layer, logits), w, wn, _stream(stream)))


def moe_permute(layer: Layer, topk_ids, T, expert_offsets, sorted_pairs, pair_pos, ws, stream=None):
    K, E = layer.top_k, layer.n_experts
    _need("topk_ids", topk_ids, T * K, torch.int32)
    _need("expert_offsets", expert_offsets, E + 1, torch.int32)
    _need("sorted_pairs", sorted_pairs, T * K, torch.int32)
    _need("pair_pos", pair_pos, T * K, torch.int32)
    w, wn = _ws(layer, ws)
    _check("moe_permute", lib().moe_permute(layer.ref, _p(layer, topk_ids), int(T), _p(layer, expert_offsets),
                                            _p(layer, sorted_pairs), _p(layer, pair_pos), w, wn, _stream(stream)))


def _routing_inputs(layer: Layer, T, topk_ids, expert_offsets, sorted_pairs):
    K, E = layer.top_k, layer.n_experts
    _need("topk_ids", topk_ids, T * K, torch.int32)
    _need("expert_offsets", expert_offsets, E + 1, torch.int32)
    _need("sorted_pairs", sorted_pairs, T * K, torch.int32)


def moe_expert_ffn_q(layer: Layer, x, T, topk_ids, expert_offsets, sorted_pairs, expert_out, shared_out=None,
                     h=None, shared_h=None, ws=None, stream=None):
    K, H, I = layer.top_k, layer.hidden, layer.inter
    _routing_inputs(layer, T, topk_ids, expert_offsets, sorted_pairs)
    _need("expert_out", expert_out, T * K * H, torch.float32)
    _need("shared_out", shared_out, T * H, torch.float32)
    _need("h", h, T * K * I, layer.act_dtype)
    _need("shared_h", shared_h, T * I, layer.act_dtype)
    w, wn = _ws(layer, ws)
    _check("moe_expert_ffn_q", lib().moe_expert_ffn_q(layer.ref, _x(layer, x, T), int(T), _p(layer, topk_ids),
                                                      _p(layer, expert_offsets), _p(layer, sorted_pairs),
                                                      _p(layer, expert_out), _p(layer, shared_out), _p(layer, h),
                                                      _p(layer, shared_h), w, wn, _stream(stream)))


def _gate_up_args(layer, x, T, topk_ids, expert_offsets, sorted_pairs, h, shared_h, stream):
    K, I = layer.top_k, layer.inter
    _routing_inputs(layer, T, topk_ids, expert_offsets, sorted_pairs)
    _need("h", h, T * K * I, layer.act_dtype)
    _need("shared_h", shared_h, T * I, layer.act_dtype)
    return (layer.ref, _x(layer, x, T), int(T), _p(layer, topk_ids), _p(layer, expert_offsets),
            _p(layer, sorted_pairs), _p(layer, h), _p(layer, shared_h), _stream(stream))


def moe_expert_gate_up_q(layer: Layer, x, T, topk_ids, expert_offsets, sorted_pairs, h, shared_h=None,
                         stream=None):
    _check("moe_expert_gate_up_q", lib().moe_expert_gate_up_q(
        *_gate_up_args(layer, x, T, topk_ids, expert_offsets, sorted_pairs, h, shared_h, stream)))


def moe_expert_down_q(layer: Layer, h, shared_h, T, topk_ids, expert_offsets, sorted_pairs, expert_out,
                      shared_out=None, stream=None):
    K, H, I = layer.top_k, layer.hidden, layer.inter
    _routing_inputs(layer, T, topk_ids, expert_offsets, sorted_pairs)
    _need("h", h, T * K * I, layer.act_dtype)
    _need("shared_h", shared_h, T * I, layer.act_dtype)
    _need("expert_out", expert_out, T * K * H, torch.float32)
    _need("shared_out", shared_out, T * H, torch.float32)
    _check("moe_expert_down_q", lib().moe_expert_down_q(layer.ref, _p(layer, h), _p(layer, shared_h), int(T),
                                                        _p(layer, topk_ids), _p(layer, expert_offsets),
                                                        _p(layer, sorted_pairs), _p(layer, expert_out),
                                                        _p(layer, shared_out), _stream(stream)))


def moe_combine(layer: Layer, expert_out, shared_out, pair_pos, topk_w, T, y, x_resid=None, x_next=None,
                stream=None):
    K, H = layer.top_k, layer.hidden
    _need("expert_out", expert_out, T * K * H, torch.float32)
    _need("shared_out", shared_out, T * H, torch.float32)
    _need("pair_pos", pair_pos, T * K, torch.int32)
    _need("topk_w", topk_w, T * K, torch.float32)
    _need("y", y, T * H, torch.float32)
    _need("x_resid", x_resid, T * H, layer.act_dtype)
    _need("x_next", x_next, T * H, layer.act_dtype)
    _check("moe_combine", lib().moe_combine(layer.ref, _p(layer, expert_out), _p(layer, shared_out),
                                            _p(layer, pair_pos), _p(layer, topk_w), int(T), _p(layer, y),
                                            _p(layer, x_resid), _p(layer, x_next), _stream(stream)))


def _layer_forward_args(layer, x, T, y, x_next, topk_ids, topk_w, ws, stream):
    K, H = layer.top_k, layer.hidden
    _need("y", y, T * H, torch.float32)
    _need("x_next", x_next, T * H, layer.act_dtype)
    _need("topk_ids", topk_ids, T * K, torch.int32)
    _need("topk_w", topk_w, T * K, torch.float32)
    w, wn = _ws(layer, ws)
    return (layer.ref, _x(layer, x, T), int(T), _p(layer, y), _p(layer, x_next), _p(layer, topk_ids),
            _p(layer, topk_w), w, wn, _stream(stream))


def moe_layer_forward(layer: Layer, x, T, y, x_next=None, topk_ids=None, topk_w=None, ws=None, stream=None):
    _check("moe_layer_forward", lib().moe_layer_forward(
        *_layer_forward_args(layer, x, T, y, x_next, topk_ids, topk_w, ws, stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20  # MOE_NOALLOC_SCRATCH_BYTES


def moe_layer_forward_noalloc(layer: Layer, x, T, y, x_next=None, topk_ids=None, topk_w=None, stream=None):
    """moe_layer_forward with the library's own device array in place of a workspace."""
    K, H = layer.top_k, layer.hidden
    _need("y", y, T * H, torch.float32)
    _need("x_next", x_next, T * H, layer.act_dtype)
    _need("topk_ids", topk_ids, T * K, torch.int32)
    _need("topk_w", topk_w, T * K, torch.float32)
    _check("moe_layer_forward_noalloc", lib().moe_layer_forward_noalloc(
        layer.ref, _x(layer, x, T), int(T), _p(layer, y), _p(layer, x_next), _p(layer, topk_ids),
        _p(layer, topk_w), _stream(stream)))


class Bound:
    """One entry point with its arguments checked and marshalled once.

    Calling it enqueues the same call again (same buffers, same stream) through
    the C ABI with no per-call Python checks, for loops where the host would
    otherwise take as long as the kernels.  It keeps the tensors it was given
    alive.  A non-OK status still raises MoeError."""

    def __init__(self, name: str, args: tuple, keep: tuple):
        self.name, self.args, self._keep = name, args, keep
        self.fn = getattr(lib(), name)

    def __call__(self):
        st = self.fn(*self.args)
        if st != MOE_OK:
            _check(self.name, st)


def bind_layer_forward(layer: Layer, x, T, y, x_next=None, topk_ids=None, topk_w=None, ws=None,
                       stream=None) -> Bound:
    """moe_layer_forward(...) as a Bound call."""
    return Bound("moe_layer_forward", _layer_forward_args(layer, x, T, y, x_next, topk_ids, topk_w, ws, stream),
                 (layer, x, y, x_next, topk_ids, topk_w, ws, stream))


def bind_expert_gate_up_q(layer: Layer, x, T, topk_ids, expert_offsets, sorted_pairs, h, shared_h=None,
                          stream=None) -> Bound:
    """moe_expert_gate_up_q(...) as a Bound call."""
    return Bound("moe_expert_gate_up_q",
                 _gate_up_args(layer, x, T, topk_ids, expert_offsets, sorted_pairs, h, shared_h, stream),
                 (layer, x, topk_ids, expert_offsets, sorted_pairs, h, shared_h, stream))


def moe_stack_forward(layers, x_inout, T, y_last=None, ws=None, stream=None):
    arr = (c_layer * len(layers))(*[l.c for l in layers])
    if not layers:
        _check("moe_stack_forward", lib().moe_stack_forward(arr, 0, None, int(T), None, None, 0, _stream(stream)))
        return
    L0 = layers[0]
    if any(l.device != L0.device for l in layers):
        raise ValueError("every layer of a stack must live on one device")
    _need("y_last", y_last, T * L0.hidden, torch.float32)
    w, wn = _ws(L0, ws)
    _check("moe_stack_forward", lib().moe_stack_forward(arr, len(layers), _x(L0, x_inout, T), int(T),
                                                        _p(L0, y_last), w, wn, _stream(stream)))


def moe_dequant(codes, scales, mins, qfmt, rows, cols, out, stream=None):
    q = QFMT.get(qfmt, qfmt)
    if q not in CODE_BITS:
        raise ValueError(f"unknown format {qfmt!r}")
    _need("codes", codes, rows * cols * CODE_BITS[q] // 8, torch.uint8)
    _need("scales", scales, rows * (cols // 32))
    _need("mins", mins, rows * (cols // 32))
    _need("out", out, rows * cols, torch.float32)
    dev = out.device
    m = c_qmat(_ptr(codes, device=dev), _ptr(scales, device=dev), _ptr(mins, device=dev))
    _check("moe_dequant", lib().moe_dequant(ctypes.byref(m), q, int(rows), int(cols), _ptr(out, torch.float32),
                                            _stream(stream)))


# ------------------------------------------------------------------ around the layer

def _need_rows(name: str, t: torch.Tensor, rows: int, cols: int, dtype):
    """Type, dtype and shape of a matrix of at least ``rows`` rows of ``cols``
    elements, each row contiguous (the row stride is the caller's)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be [>={rows}][{cols}], got {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: rows overlap (row stride {t.stride(0)}, {cols} columns)")


def _addr(name: str, t: torch.Tensor, device) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must live in device memory")
    if t.device != device:
        raise ValueError(f"{name}: tensor on {t.device}, expected {device}")
    return t.data_ptr()


class _DeviceBound(Bound):
    """A Bound call that makes its tensors' device current for the launch."""

    def __init__(self, name: str, args: tuple, keep: tuple, device: torch.device):
        super().__init__(name, args, keep)
        self.device = device

    def __call__(self):
        if torch.cuda.current_device() == self.device.index:
            st = self.fn(*self.args)
        else:
            with torch.cuda.device(self.device):
                st = self.fn(*self.args)
        if st != MOE_OK:
            _check(self.name, st)


def _stream_on(stream, device) -> Optional[int]:
    """The given stream, or the current one of the tensors' device."""
    return torch.cuda.current_stream(device).cuda_stream if stream is None else _stream(stream)


class Linear:
    """A moe_linear descriptor over device tensors (kept alive by this object):
    a matrix [rows][cols] in one of the packed formats.

    codes uint8 [rows][cols*bits/8]; scales and mins (2-bit format only) 16-bit
    planes [rows][cols/32]; bias fp32 [rows] or None.  ``act`` is the type of x,
    ``out`` that of y ("f32" or "bf16").  A one-matrix expert set ([1][rows][..])
    is taken as it is."""

    def __init__(self, *, rows: int, cols: int, qfmt, act, codes: torch.Tensor, scales: torch.Tensor,
                 mins: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, out="f32"):
        self.qfmt, self.act, self.out = QFMT.get(qfmt, qfmt), ACT.get(act, act), ACT.get(out, out)
        if self.qfmt not in CODE_BITS:
            raise ValueError(f"unknown format {qfmt!r}")
        for name, a in (("act", self.act), ("out", self.out)):
            if a not in (MOE_ACT_F32, MOE_ACT_BF16):
                raise ValueError(f"{name} must be 'f32' or 'bf16'")
        self.rows, self.cols = int(rows), int(cols)
        self.act_dtype, self.out_dtype = _act_dtype(self.act), _act_dtype(self.out)
        nb = self.cols * CODE_BITS[self.qfmt] // 8
        if codes.dtype != torch.uint8 or tuple(codes.shape) not in ((self.rows, nb), (1, self.rows, nb)):
            raise ValueError(f"codes must be uint8 [{self.rows}][{nb}], got {codes.dtype} {tuple(codes.shape)}")
        if (mins is None) != (self.qfmt != MOE_Q2_ASYM_G32):
            raise ValueError("mins are required for the 2-bit format only")
        ng = self.cols // 32
        for name, t in (("scales", scales), ("mins", mins)):
            if t is not None and (t.element_size() != 2 or tuple(t.shape) not in ((self.rows, ng), (1, self.rows, ng))):
                raise ValueError(f"{name} must be 16-bit [{self.rows}][{ng}]")
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (self.rows,)):
            raise ValueError(f"bias must be fp32 [{self.rows}]")
        self.device = codes.device
        self._keep = (codes, scales, mins, bias)
        dev = self.device
        self.c = c_linear(self.rows, self.cols, self.qfmt, self.act, self.out,
                          c_qmat(_ptr(codes, device=dev), _ptr(scales, device=dev), _ptr(mins, device=dev)),
                          _ptr(bias, device=dev))

    @property
    def ref(self):
        return ctypes.byref(self.c)


def _linear_args(lin: Linear, x, T, y, stream):
    T = int(T)
    _need_rows("x", x, T, lin.cols, lin.act_dtype)
    _need_rows("y", y, T, lin.rows, lin.out_dtype)
    return (lin.ref, _addr("x", x, lin.device), x.stride(0) if T > 1 else lin.cols, T, _addr("y", y, lin.device),
            y.stride(0) if T > 1 else lin.rows, _stream_on(stream, lin.device))


def bind_linear_q(lin: Linear, x, T, y, stream=None) -> Bound:
    """moe_linear_q(...) as a Bound call."""
    return _DeviceBound("moe_linear_q", _linear_args(lin, x, T, y, stream), (lin, x, y, stream), lin.device)


def moe_linear_q(lin: Linear, x, T, y, stream=None):
    """y[:T] = x[:T] W^T + bias.  x [>=T][cols] and y [>=T][rows] may have any
    row stride (x: rows at multiples of 16 bytes)."""
    bind_linear_q(lin, x, T, y, stream)()


class Beam:
    """A moe_beam descriptor: the shape of one beam search's step.  ``act`` is
    the type of the logits, ``eos`` the token finished beams are carried on with."""

    def __init__(self, *, batch: int, beams: int, vocab: int, n_out: int, act="f32", eos: int = -1):
        self.batch, self.beams, self.vocab, self.n_out, self.eos = int(batch), int(beams), int(vocab), int(n_out), int(eos)
        self.act = ACT.get(act, act)
        self.c = c_beam(self.batch, self.beams, self.vocab, self.n_out, self.act, self.eos)

    @property
    def ref(self):
        return ctypes.byref(self.c)


def moe_beam_workspace_bytes(beam: Beam) -> int:
    return int(lib().moe_beam_workspace_bytes(beam.ref))


def beam_workspace(beam: Beam, device=None) -> torch.Tensor:
    """A device workspace tensor of moe_beam_workspace_bytes(beam) bytes."""
    n = moe_beam_workspace_bytes(beam)
    if n == 0:
        raise MoeError("moe_beam_workspace_bytes", MOE_E_ARG, "invalid beam descriptor")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _beam_args(beam: Beam, logits, scores, out_score, out_parent, out_token, finished, allowed, ws, stream):
    rows, n = beam.batch * beam.beams, beam.batch * beam.n_out
    if not isinstance(logits, torch.Tensor):
        raise TypeError(f"logits: expected a torch.Tensor, got {type(logits).__name__}")
    dev = logits.device
    _need("scores", scores, rows, torch.float32)
    _need("out_score", out_score, n, torch.float32)
    _need("out_parent", out_parent, n, torch.int32)
    _need("out_token", out_token, n, torch.int32)
    _need("finished", finished, rows, torch.uint8)
    ld_allowed = 0
    if allowed is not None:
        words = (beam.vocab + 31) // 32
        if allowed.dim() != 2 or allowed.shape[0] not in (1, rows) or allowed.shape[1] != words:
            raise ValueError(f"allowed must be int32 [1 or {rows}][{words}], got {tuple(allowed.shape)}")
        ld_allowed = allowed.stride(0) if allowed.shape[0] > 1 else 0
        _need_rows("allowed", allowed, allowed.shape[0], words, torch.int32)
    _need_rows("logits", logits, rows, beam.vocab, _act_dtype(beam.act))
    lp = _addr("logits", logits, dev)
    ap = None if allowed is None else _addr("allowed", allowed, dev)
    w, wn = (None, 0) if ws is None else (_ptr(ws, torch.uint8, dev), ws.numel())
    return (beam.ref, lp, logits.stride(0) if rows > 1 else beam.vocab, _ptr(scores, None, dev), _ptr(finished, None, dev),
            ap, ld_allowed, _ptr(out_score, None, dev), _ptr(out_parent, None, dev), _ptr(out_token, None, dev), w, wn,
            _stream_on(stream, dev))


def bind_beam_select(beam: Beam, logits, scores, out_score, out_parent, out_token, finished=None, allowed=None, ws=None,
                     stream=None) -> Bound:
    """moe_beam_select(...) as a Bound call."""
    return _DeviceBound("moe_beam_select",
                        _beam_args(beam, logits, scores, out_score, out_parent, out_token, finished, allowed, ws, stream),
                        (beam, logits, scores, out_score, out_parent, out_token, finished, allowed, ws, stream),
                        logits.device)


def moe_beam_select(beam: Beam, logits, scores, out_score, out_parent, out_token, finished=None, allowed=None, ws=None,
                    stream=None):
    """The n_out best continuations of each sequence.  logits [batch*beams][vocab]
    (any row stride), scores [batch][beams]; finished uint8 [batch][beams];
    allowed int32 bit masks [1 or batch*beams][(vocab+31)//32]."""
    bind_beam_select(beam, logits, scores, out_score, out_parent, out_token, finished, allowed, ws, stream)()


def _pieces(t: torch.Tensor):
    """(contiguous elements, count, element stride) of a row of a state tensor:
    one row is ``count`` equally spaced runs of contiguous elements."""
    dims = [(n, s) for n, s in zip(t.shape[1:], t.stride()[1:]) if n != 1]
    run = 1
    while dims and dims[-1][1] == run:
        run *= dims.pop()[0]
    if not dims:
        return run, 1, 0
    count, stride = dims[-1]
    for n, s in reversed(dims[:-1]):
        if s != stride * count:
            raise ValueError("state: a row must be equally spaced contiguous pieces")
        count *= n
    return run, count, stride


def _state(src: torch.Tensor, dst: torch.Tensor, rows: int, device) -> c_state:
    for name, t in (("state", src), ("dst", dst)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dim() < 1 or t.shape[0] != rows:
            raise ValueError(f"{name} must have {rows} rows (batch * beams), got {tuple(t.shape)}")
    if src.shape != dst.shape or src.dtype != dst.dtype:
        raise ValueError("a state and its dst must have the same shape and type")
    if src.numel() == 0:
        return c_state()
    (r0, n0, s0), (r1, n1, s1) = _pieces(src), _pieces(dst)
    run = min(r0, r1)
    if r0 > run:  # a contiguous row next to one in pieces
        if n0 != 1:
            raise ValueError("state: the pieces of a state and its dst must match")
        n0, s0 = r0 // run, run
    if r1 > run:
        if n1 != 1:
            raise ValueError("state: the pieces of a state and its dst must match")
        n1, s1 = r1 // run, run
    if n0 != n1:
        raise ValueError("state: the pieces of a state and its dst must match")
    for t in (src, dst):
        if not t.is_cuda:
            raise ValueError("state: tensor must live in device memory")
        if t.device != device:
            raise ValueError(f"state: tensor on {t.device}, expected {device}")
    e = src.element_size()
    return c_state(src.data_ptr(), dst.data_ptr(), run * e, n0, src.stride(0) * e, s0 * e, dst.stride(0) * e, s1 * e)


def bind_beam_reorder(states, parent, batch: int, beams: int, dst=None, stream=None) -> Bound:
    """moe_beam_reorder(...) as a Bound call."""
    states = list(states)
    dst = states if dst is None else list(dst)
    if len(dst) != len(states):
        raise ValueError(f"{len(states)} states, {len(dst)} destinations")
    rows = int(batch) * int(beams)
    dev = parent.device
    if parent.dtype != torch.int32 or parent.dim() != 2 or parent.shape[0] < batch or parent.shape[1] < beams:
        raise ValueError(f"parent must be int32 [>={batch}][>={beams}], got {parent.dtype} {tuple(parent.shape)}")
    _need_rows("parent", parent, int(batch), parent.shape[1], torch.int32)
    arr = (c_state * len(states))(*[_state(s, d, rows, dev) for s, d in zip(states, dst)])
    pp = _addr("parent", parent, dev)
    return _DeviceBound("moe_beam_reorder", (arr, len(states), pp, parent.stride(0) if batch > 1 else int(beams),
                                             int(batch), int(beams), _stream_on(stream, dev)),
                        (states, dst, parent, stream), dev)


def moe_beam_reorder(states, parent, batch: int, beams: int, dst=None, stream=None):
    """Every state's row b * beams + i becomes its row b * beams + parent[b][i],
    in place or written to ``dst``.  states: tensors [batch*beams][...] whose
    rows are contiguous or equally spaced contiguous pieces (a cache's filled
    part, cache[:, :, :length], is); parent int32 [batch][>= beams]."""
    bind_beam_reorder(states, parent, batch, beams, dst, stream)()


def moe_abi_version() -> int:
    return int(lib().moe_abi_version())


def moe_range_checks() -> int:
    return int(lib().moe_range_checks())
