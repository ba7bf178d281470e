"""Python binding of libmoeep: the single-GPU expert-parallel MoE layer path
(route -> layout -> dispatch -> grouped SwiGLU FFN -> combine) on MI355X.

Each function here has the name of the C entry point it marshals (see
include/moeep.h for the full contract).  Tensors are torch device tensors
used only as memory; the binding checks shapes and dtypes, allocates outputs
the caller did not provide, passes ``data_ptr()`` and the current HIP stream,
and raises :class:`MoeError` with the library's message on a non-OK status.
All compute happens in the HIP kernels of ``libmoeep.so``; there is no other
code path.  Build the library with ``python -m combine_grouped_gemm_amd.build``.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = ["MoeError", "lib", "library_path", "moe_version", "moe_route",
           "moe_layout_workspace_bytes", "moe_layout", "moe_layout_noalloc", "moe_dispatch",
           "moe_ffn_workspace_bytes", "moe_ffn_gate_up", "moe_ffn_down",
           "moe_grouped_ffn", "moe_combine", "moe_layout_masked", "moe_ffn_gate_up_masked",
           "moe_ffn_down_masked", "moe_grouped_ffn_masked", "moe_route_mapped", "moe_eplb_place", "moe_route_shared",
           "moe_route_scored", "moe_quant_rows", "moe_quant_rows_masked",
           "moe_checkpoint_rows", "moe_checkpoint_values", "moe_ffn_gate_up_train", "moe_swiglu_backward",
           "moe_ffn_dgrad", "moe_ffn_wgrad", "moe_route_backward",
           "moe_weight_ld", "moe_packed_weight_bytes", "moe_pack_weights",
           "MOE_F32", "MOE_BF16", "MOE_FP8_E4M3", "MOE_FP8_E4M3_PO2", "MOE_INT8", "MOE_CKPT8", "MOE_W_PACKED",
           "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_SCORE_PICKS",
           "MOE_GATHER_NONE", "MOE_GATHER_X", "MOE_GATHER_DY",
           "MoELayer"]

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP = 0, 1, 2, 3
MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_FP8_E4M3_PO2, MOE_INT8, MOE_CKPT8 = 0, 1, 2, 3, 4, 5
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID, MOE_SCORE_PICKS = 0, 1, 2
MOE_GATHER_NONE, MOE_GATHER_X, MOE_GATHER_DY = 0, 1, 2
MOE_W_PACKED = 0x100
FP8_BLOCK = 128
CKPT_BLOCK = 128             # columns of a row that share a scale in an 8-bit checkpoint
MAX_SEGMENTS = 64
INT8_MAX_COLS = 131056       # largest H and I of int8 operands (exact int32 sums)

_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_FP8_E4M3,
       torch.int8: MOE_INT8}
_TORCH = {v: k for k, v in _DT.items()}
_NAMES = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8": MOE_FP8_E4M3, "int8": MOE_INT8}
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoeep.so")
_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


def _status_name(s):
    return {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
            3: "MOE_ERR_HIP"}.get(s, f"status {s}")


def lib() -> ctypes.CDLL:
    """The loaded libmoeep.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"libmoeep.so is missing at {library_path}; build it with "
                           "'python -m combine_grouped_gemm_amd.build'")
    L = ctypes.CDLL(library_path)
    P, I, Z, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int
    F = ctypes.c_float
    sig = {
        "moe_status_string": ([I], ctypes.c_char_p),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_version": ([], ctypes.c_char_p),
        "moe_route": ([P, I, I, I, P, P, P], S),
        "moe_layout_workspace_bytes": ([I, I, I], Z),
        "moe_layout": ([P, I, I, I, I, I, P, P, P, P, I, P, Z, P], S),
        "moe_layout_noalloc": ([P, I, I, I, I, I, P, P, P, P, I, P], S),
        "moe_dispatch": ([P, P, I, I, I, P, I, P, I, P, I, P], S),
        "moe_ffn_workspace_bytes": ([I, I, I], Z),
        "moe_ffn_gate_up": ([P, P, P, I, I, I, I, I, P, P, P, P, I, P, P, I, P], S),
        "moe_ffn_down": ([P, P, P, I, I, I, I, I, P, P, I, P, I, I, P], S),
        "moe_grouped_ffn": ([P, P, P, I, I, I, I, I, P, P, P, P, P, P, I, P, I, P, Z, I, P], S),
        "moe_combine": ([P, I, I, P, P, I, I, I, P, I, P], S),
        "moe_layout_masked": ([P, I, I, I, I, I, P, P, P, P, I, P, Z, P], S),
        "moe_route_mapped": ([P, I, I, I, P, P, P, P], S),
        "moe_eplb_place": ([P, I, I, P], S),
        "moe_route_shared": ([P, I, I, I, I, P, P, P], S),
        "moe_route_scored": ([P, I, P, I, I, I, I, I, I, I, I, F, P, I, P, P, P], S),
        "moe_quant_rows": ([P, I, P, I, I, I, P, P, P], S),
        "moe_quant_rows_masked": ([P, I, P, I, I, I, P, P, P], S),
        "moe_checkpoint_rows": ([P, I, P, I, I, I, P, P, P], S),
        "moe_checkpoint_values": ([P, P, P, I, I, I, P, I, P], S),
        "moe_ffn_gate_up_train": ([P, P, I, I, I, I, I, P, P, I, P, P, P, P, P, I, P], S),
        "moe_swiglu_backward": ([P, I, P, P, P, P, I, I, P, P, I, I, P, P, P, P, P], S),
        "moe_ffn_dgrad": ([P, P, P, I, I, P, I, I, I, I, I, P, P, I, P, I, P], S),
        "moe_ffn_wgrad": ([P, P, P, I, P, P, I, I, I, P, I, I, I, I, I, P, P, P, P, I, I, P], S),
        "moe_route_backward": ([P, I, P, P, I, I, I, I, I, F, P, I, P, P], S),
        "moe_weight_ld": ([I, I], I),
        "moe_packed_weight_bytes": ([I, I, I, I], Z),
        "moe_pack_weights": ([P, I, I, I, I, P, P], S),
    }
    # the masked FFN calls take (m, E_local, cap_per_expert) where the others take
    # (offsets, E_local, cap_rows): same argument types
    for name in ("moe_ffn_gate_up", "moe_ffn_down", "moe_grouped_ffn"):
        sig[name + "_masked"] = sig[name]
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _lib = L
    return L


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, lib().moe_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current device, and the current stream of a device as an integer:
# torch.cuda.current_stream() builds an object for it, which costs as much as the rest
# of a call
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(stream):
    if stream is None:
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _call(fn, t, stream, *args):
    """One library call with t's device current, on `stream` (None: that device's current stream)."""
    index = t.get_device()
    if index != _current_device():
        with torch.cuda.device(index):
            return _call(fn, t, stream, *args)
    if stream is None:
        status = fn(*args, _raw_stream(index))
    else:
        if isinstance(stream, torch.cuda.Stream) and stream.device_index != index:
            raise ValueError(f"stream must be of the tensors' device {t.device} (got one of cuda:{stream.device_index})")
        status = fn(*args, _stream(stream))
    if status != MOE_OK:
        _check(status)


def _new(shape, dtype, device, stream, scratch=False):
    """An output or workspace (scratch) the caller did not give, allocated for the stream
    that uses it: memory of another stream may still be in use there, and a workspace freed
    on return would go to that stream's next allocation while the call is still running.
    For an output the current stream, where the caller goes on, is noted as a user too: what
    it still reads when the tensor is dropped is not written by the given stream's next call."""
    if stream is None or _stream(stream) == _raw_stream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    current = torch.cuda.current_stream(device)
    if device.index == _current_device():
        # what torch.cuda.stream() does, at a third of its time
        torch.cuda.set_stream(stream)
        try:
            t = torch.empty(shape, dtype=dtype, device=device)
        finally:
            torch.cuda.set_stream(current)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(current)
    return t


def _dev(t, name, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {t.dim()})")
    return t


def _need(t, name, numel=None, shape=None):
    """Caller-provided tensors must cover what the kernels index: the C ABI
    cannot see sizes, so an undersized tensor would be written out of bounds
    on the device.  Raises ValueError before any library call."""
    if t is None:
        return
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} needs at least {numel} elements (got {t.numel()})")


def _same_device(t, name, *others):
    """Every tensor of a call lives on the device of its first one (None: not given)."""
    index = t.get_device()
    for o in others:
        if o is not None and o.get_device() != index:
            raise ValueError(f"all tensors must be on {name}'s device {t.device} (got {o.device})")


def _dtype_code(d):
    if isinstance(d, str):
        return _NAMES[d]
    if isinstance(d, torch.dtype):
        return _DT[d]
    return int(d)


def moe_version() -> str:
    return lib().moe_version().decode()


# ----------------------------------------------------------------------------
def moe_route(logits, K: int, topk_ids=None, topk_w=None, stream=None):
    """Top-K expert ids (B, K) int32 and renormalised softmax gates (B, K) fp32."""
    _dev(logits, "logits", torch.float32, 2)
    B, E = logits.shape
    if topk_ids is None:
        topk_ids = _new((B, K), torch.int32, logits.device, stream)
    if topk_w is None:
        topk_w = _new((B, K), torch.float32, logits.device, stream)
    _dev(topk_ids, "topk_ids", torch.int32)
    _dev(topk_w, "topk_w", torch.float32)
    _need(topk_ids, "topk_ids", shape=(B, K))
    _need(topk_w, "topk_w", shape=(B, K))
    _same_device(logits, "logits", topk_ids, topk_w)
    _call(lib().moe_route, logits, stream, _ptr(logits), B, E, K, _ptr(topk_ids), _ptr(topk_w))
    return topk_ids, topk_w


def moe_route_mapped(logits, K: int, phys_of_logical, topk_ids=None, topk_w=None, stream=None):
    """moe_route with the chosen expert ids written through a placement map
    (phys_of_logical: (E,) int32 device tensor)."""
    _dev(logits, "logits", torch.float32, 2)
    _dev(phys_of_logical, "phys_of_logical", torch.int32, 1)
    B, E = logits.shape
    if phys_of_logical.numel() != E:
        raise ValueError("phys_of_logical needs E entries")
    if topk_ids is None:
        topk_ids = _new((B, K), torch.int32, logits.device, stream)
    if topk_w is None:
        topk_w = _new((B, K), torch.float32, logits.device, stream)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    _dev(topk_w, "topk_w", torch.float32, 2)
    _need(topk_ids, "topk_ids", shape=(B, K))
    _need(topk_w, "topk_w", shape=(B, K))
    _same_device(logits, "logits", phys_of_logical, topk_ids, topk_w)
    _call(lib().moe_route_mapped, logits, stream, _ptr(logits), B, E, K, _ptr(phys_of_logical), _ptr(topk_ids),
          _ptr(topk_w))
    return topk_ids, topk_w


def moe_route_shared(logits, K: int, n_shared: int, topk_ids=None, topk_w=None, stream=None):
    """moe_route plus n_shared always-on experts: ids / gates (B, K + n_shared),
    the last n_shared columns E, E+1, ... with gate 1."""
    _dev(logits, "logits", torch.float32, 2)
    B, E = logits.shape
    Kt = K + n_shared
    if topk_ids is None:
        topk_ids = _new((B, Kt), torch.int32, logits.device, stream)
    if topk_w is None:
        topk_w = _new((B, Kt), torch.float32, logits.device, stream)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    _dev(topk_w, "topk_w", torch.float32, 2)
    if topk_ids.shape != (B, Kt) or topk_w.shape != (B, Kt):
        raise ValueError(f"outputs must be ({B}, {Kt})")
    _same_device(logits, "logits", topk_ids, topk_w)
    _call(lib().moe_route_shared, logits, stream, _ptr(logits), B, E, K, int(n_shared), _ptr(topk_ids), _ptr(topk_w))
    return topk_ids, topk_w


def moe_route_scored(logits, K: int, score: str = "sigmoid", bias=None, n_groups: int = 1, topk_groups: int = 1,
                     group_top: int = 2, renorm: bool = True, scale: float = 1.0, phys_of_logical=None,
                     n_shared: int = 0, topk_ids=None, topk_w=None, stream=None):
    """Top-K experts by ``score`` ('sigmoid' or 'softmax' over all experts) plus
    ``bias`` (E,) inside the ``topk_groups`` best of ``n_groups`` expert groups
    (a group scores the sum of its ``group_top`` best); weights are the picks'
    scores, renormalised and scaled.  logits (B, E) fp32 or bf16; ids / weights
    (B, K + n_shared); slots that find no unmasked expert get id -1, weight 0."""
    _dev(logits, "logits", None, 2)
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits must be float32 or bfloat16 (got {logits.dtype})")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)} (got {score!r})")
    B, E = logits.shape
    Kt = K + n_shared
    dev = logits.device
    if bias is not None:
        _dev(bias, "bias", torch.float32, 1)
        _need(bias, "bias", shape=(E,))
    if phys_of_logical is not None:
        _dev(phys_of_logical, "phys_of_logical", torch.int32, 1)
        _need(phys_of_logical, "phys_of_logical", shape=(E,))
    if topk_ids is None:
        topk_ids = _new((B, max(Kt, 0)), torch.int32, dev, stream)
    else:
        _dev(topk_ids, "topk_ids", torch.int32)
        _need(topk_ids, "topk_ids", shape=(B, Kt))
    if topk_w is None:
        topk_w = _new((B, max(Kt, 0)), torch.float32, dev, stream)
    else:
        _dev(topk_w, "topk_w", torch.float32)
        _need(topk_w, "topk_w", shape=(B, Kt))
    _same_device(logits, "logits", bias, phys_of_logical, topk_ids, topk_w)
    _call(lib().moe_route_scored, logits, stream, logits.data_ptr(), _DT[logits.dtype], _ptr(bias), B, E, K,
          _SCORES[score], n_groups, topk_groups, group_top, 1 if renorm else 0, scale, _ptr(phys_of_logical), n_shared,
          topk_ids.data_ptr(), topk_w.data_ptr())
    return topk_ids, topk_w


def moe_eplb_place(load, n_groups: int):
    """Host expert placement: load (E,) activation counts (any integer
    array-like) -> phys_of_logical (E,) int32 CPU tensor."""
    load = torch.as_tensor(load).to(torch.int64).contiguous().cpu()
    if load.dim() != 1:
        raise ValueError("load must be 1-D")
    phys = torch.empty(load.numel(), dtype=torch.int32)
    _check(lib().moe_eplb_place(load.data_ptr(), load.numel(), int(n_groups), phys.data_ptr()))
    return phys


def moe_layout_workspace_bytes(B: int, K: int, E: int) -> int:
    return int(lib().moe_layout_workspace_bytes(B, K, E))


def _check_layout_outputs(B, K, E, E_loc, cap_rows, counts, offsets, row_of, src_of):
    _need(counts, "counts", numel=E)
    _need(offsets, "offsets", numel=max(E_loc, 0) + 1)
    _need(row_of, "row_of", numel=B * K)
    _need(src_of, "src_of", numel=cap_rows)


def moe_layout(topk_ids, E: int, e_begin: int, e_end: int, cap_rows: int, counts=None,
               offsets=None, row_of=None, src_of=None, ws=None, stream=None) -> dict:
    """counts (E), offsets (E_loc+1), row_of (B, K), src_of (cap_rows), all int32."""
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    B, K = topk_ids.shape
    dev = topk_ids.device
    E_loc = e_end - e_begin
    counts = _new(E, torch.int32, dev, stream) if counts is None else counts
    offsets = _new(max(E_loc, 0) + 1, torch.int32, dev, stream) if offsets is None else offsets
    row_of = _new((B, K), torch.int32, dev, stream) if row_of is None else row_of
    src_of = _new(max(cap_rows, 1), torch.int32, dev, stream) if src_of is None else src_of
    need = moe_layout_workspace_bytes(B, K, E)
    if ws is None:
        ws = _new(max(need, 256), torch.uint8, dev, stream, scratch=True)
    for n, t in (("counts", counts), ("offsets", offsets), ("row_of", row_of), ("src_of", src_of)):
        _dev(t, n, torch.int32)
    _check_layout_outputs(B, K, E, E_loc, cap_rows, counts, offsets, row_of, src_of)
    _dev(ws, "ws")
    _same_device(topk_ids, "topk_ids", counts, offsets, row_of, src_of, ws)
    _call(lib().moe_layout, topk_ids, stream, _ptr(topk_ids), B, K, E, e_begin, e_end, _ptr(counts), _ptr(offsets),
          _ptr(row_of), _ptr(src_of), cap_rows, _ptr(ws), ws.numel() * ws.element_size())
    return {"counts": counts, "offsets": offsets, "row_of": row_of, "src_of": src_of}


LAYOUT_NOALLOC_SCRATCH_BYTES = 4 << 20


def moe_layout_noalloc(topk_ids, E: int, e_begin: int, e_end: int, cap_rows: int, counts=None,
                       offsets=None, row_of=None, src_of=None, stream=None) -> dict:
    """moe_layout without a workspace argument: the library's own per-GPU
    scratch (LAYOUT_NOALLOC_SCRATCH_BYTES) holds the chunk histograms, and
    the call allocates nothing on the device when every output is given.
    Batches needing more workspace than that raise MoeError; calls that
    overlap on one GPU race on the shared scratch."""
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    B, K = topk_ids.shape
    dev = topk_ids.device
    E_loc = e_end - e_begin
    counts = _new(E, torch.int32, dev, stream) if counts is None else counts
    offsets = _new(max(E_loc, 0) + 1, torch.int32, dev, stream) if offsets is None else offsets
    row_of = _new((B, K), torch.int32, dev, stream) if row_of is None else row_of
    src_of = _new(max(cap_rows, 1), torch.int32, dev, stream) if src_of is None else src_of
    for n, t in (("counts", counts), ("offsets", offsets), ("row_of", row_of), ("src_of", src_of)):
        _dev(t, n, torch.int32)
    _check_layout_outputs(B, K, E, E_loc, cap_rows, counts, offsets, row_of, src_of)
    _same_device(topk_ids, "topk_ids", counts, offsets, row_of, src_of)
    _call(lib().moe_layout_noalloc, topk_ids, stream, _ptr(topk_ids), B, K, E, e_begin, e_end, _ptr(counts),
          _ptr(offsets), _ptr(row_of), _ptr(src_of), cap_rows)
    return {"counts": counts, "offsets": offsets, "row_of": row_of, "src_of": src_of}


def moe_layout_masked(topk_ids, E: int, e_begin: int, e_end: int, cap_per_expert: int, counts=None,
                      m=None, row_of=None, src_of=None, ws=None, stream=None) -> dict:
    """Fixed-capacity layout: counts (E), m (E_loc), row_of (B, K),
    src_of (E_loc * cap_per_expert), all int32."""
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    B, K = topk_ids.shape
    dev = topk_ids.device
    E_loc = e_end - e_begin
    counts = _new(E, torch.int32, dev, stream) if counts is None else counts
    m = _new(max(E_loc, 1), torch.int32, dev, stream) if m is None else m
    row_of = _new((B, K), torch.int32, dev, stream) if row_of is None else row_of
    if src_of is None:
        src_of = _new(max(E_loc * cap_per_expert, 1), torch.int32, dev, stream)
    need = moe_layout_workspace_bytes(B, K, E)
    if ws is None:
        ws = _new(max(need, 256), torch.uint8, dev, stream, scratch=True)
    for n, t in (("counts", counts), ("m", m), ("row_of", row_of), ("src_of", src_of)):
        _dev(t, n, torch.int32)
    _need(counts, "counts", numel=E)
    _need(m, "m", numel=max(E_loc, 0))
    _need(row_of, "row_of", numel=B * K)
    _need(src_of, "src_of", numel=max(E_loc, 0) * cap_per_expert)
    _dev(ws, "ws")
    _same_device(topk_ids, "topk_ids", counts, m, row_of, src_of, ws)
    _call(lib().moe_layout_masked, topk_ids, stream, _ptr(topk_ids), B, K, E, e_begin, e_end, _ptr(counts), _ptr(m),
          _ptr(row_of), _ptr(src_of), cap_per_expert, _ptr(ws), ws.numel() * ws.element_size())
    return {"counts": counts, "m": m, "row_of": row_of, "src_of": src_of}


def moe_dispatch(seg_x, row_of, cap_rows: int, xd_dtype=None, xd=None, xd_scales=None,
                 stream=None):
    """Scatter the token rows of the segments into xd (cap_rows, H); fp8
    storage also fills xd_scales (cap_rows, ceil(H/128)), int8 storage
    xd_scales (cap_rows,)."""
    if isinstance(seg_x, torch.Tensor):
        seg_x = [seg_x]
    seg_x = list(seg_x)
    if not 1 <= len(seg_x) <= MAX_SEGMENTS:
        raise ValueError(f"need 1..{MAX_SEGMENTS} segments")
    x_dt = seg_x[0].dtype
    H = seg_x[0].shape[1]
    for i, s in enumerate(seg_x):
        _dev(s, f"seg_x[{i}]", x_dt, 2)
        if s.shape[1] != H:
            raise ValueError("all segments need the same H")
    _dev(row_of, "row_of", torch.int32, 2)
    K = row_of.shape[1]
    dev = row_of.device
    xd_code = _DT[x_dt] if xd_dtype is None else _dtype_code(xd_dtype)
    if xd is None:
        xd = _new((max(cap_rows, 1), H), _TORCH[xd_code], dev, stream)
    if xd_code == MOE_FP8_E4M3 and xd_scales is None:
        xd_scales = _new((max(cap_rows, 1), -(-H // FP8_BLOCK)), torch.float32, dev, stream)
    if xd_code == MOE_INT8 and xd_scales is None:
        xd_scales = _new(max(cap_rows, 1), torch.float32, dev, stream)
    _dev(xd, "xd")
    B = sum(int(t.shape[0]) for t in seg_x)
    _need(row_of, "row_of", shape=(B, K))
    if xd.dtype != _TORCH[xd_code]:
        raise ValueError(f"xd must be {_TORCH[xd_code]} (got {xd.dtype})")
    _need(xd, "xd", numel=cap_rows * H)
    if xd_code in (MOE_FP8_E4M3, MOE_INT8):
        _dev(xd_scales, "xd_scales", torch.float32)
        _need(xd_scales, "xd_scales", numel=cap_rows * _scale_cols(xd_code, H))
    _same_device(row_of, "row_of", xd, xd_scales if xd_code in (MOE_FP8_E4M3, MOE_INT8) else None, *seg_x)
    ptrs = (ctypes.c_void_p * len(seg_x))(*[s.data_ptr() for s in seg_x])
    rows = (ctypes.c_int32 * len(seg_x))(*[s.shape[0] for s in seg_x])
    _call(lib().moe_dispatch, row_of, stream, ptrs, rows, len(seg_x), _DT[x_dt], H, _ptr(row_of), K, _ptr(xd), xd_code, _ptr(xd_scales), cap_rows)
    return xd, xd_scales


def _scale_cols(code, cols):
    """fp32 scales of a quantised row of ``cols`` elements: fp8 one per block, int8 one."""
    return -(-cols // FP8_BLOCK) if code == MOE_FP8_E4M3 else 1


def moe_quant_rows(x, rows=None, cap_per_expert=None, q=None, scales=None, stream=None, E_loc=None):
    """int8 codes (cap_rows, cols) and a scale (cap_rows,) for each valid row of x
    (fp32 or bf16).  rows: the contiguous layout's offsets (E_loc + 1), or with
    cap_per_expert the masked layout's m (E_loc) (moe_quant_rows_masked); None
    quantises every row, e.g. weight rows (a scale for each output channel).
    E_loc: the local experts, when rows is a longer buffer (default: as many as it
    describes; the FFN calls take them from the weights).
    Other rows of given q and scales are left as they were."""
    _dev(x, "x", None, 2)
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"x must be float32 or bfloat16 (got {x.dtype})")
    cap, cols = x.shape
    third = cap
    if rows is None:
        if cap_per_expert is not None:
            raise ValueError("cap_per_expert needs the masked layout's m")
        if E_loc is not None:
            raise ValueError("E_loc needs the layout's offsets or m")
        E_loc = 0
    else:
        name, last = ("offsets", 1) if cap_per_expert is None else ("m", 0)
        _dev(rows, name, torch.int32, 1)
        if E_loc is None:
            E_loc = max(rows.numel() - last, 1)       # an empty tensor's null pointer would mean all rows
        if E_loc < 1:
            raise ValueError(f"E_loc must be positive (got {E_loc})")
        _need(rows, name, numel=E_loc + last)
        third = _rows_arg(rows, cap_per_expert, E_loc, cap)
    if q is None:
        q = _new((cap, cols), torch.int8, x.device, stream)
    if scales is None:
        scales = _new(cap, torch.float32, x.device, stream)
    _dev(q, "q", torch.int8)
    _dev(scales, "scales", torch.float32)
    _need(q, "q", shape=(cap, cols))
    _need(scales, "scales", numel=cap)
    _same_device(x, "x", rows, q, scales)
    fn = lib().moe_quant_rows if cap_per_expert is None else lib().moe_quant_rows_masked
    _call(fn, x, stream, _ptr(x), _DT[x.dtype], _ptr(rows), E_loc, third, cols, _ptr(q), _ptr(scales))
    return q, scales


def moe_quant_rows_masked(x, m, cap_per_expert, **kw):
    """moe_quant_rows over the masked layout (rows [j*cap_per_expert, +m[j]))."""
    return moe_quant_rows(x, m, cap_per_expert=cap_per_expert, **kw)


def moe_ffn_workspace_bytes(cap_rows: int, I: int, act_dtype) -> int:
    return int(lib().moe_ffn_workspace_bytes(cap_rows, I, _dtype_code(act_dtype)))


def moe_weight_ld(cols: int, w_dtype) -> int:
    """Row pitch (elements) of packed weights with rows of ``cols`` elements."""
    ld = int(lib().moe_weight_ld(int(cols), _dtype_code(w_dtype)))
    if ld < 0:
        raise ValueError(f"no packed pitch for cols={cols}, dtype={w_dtype}")
    return ld


def moe_packed_weight_bytes(E_local: int, rows: int, cols: int, w_dtype) -> int:
    return int(lib().moe_packed_weight_bytes(E_local, rows, cols, _dtype_code(w_dtype)))


def moe_pack_weights(w, out=None, stream=None):
    """w (E_local, rows, cols) -> (E_local, rows, moe_weight_ld(cols)), rows
    unchanged and the padding zero: the layout the FFN calls read when given
    weights with the packed pitch (results identical to the dense weights)."""
    _dev(w, "w", ndim=3)
    E_loc, rows, cols = w.shape
    code = _DT[w.dtype]
    ld = moe_weight_ld(cols, code)
    if out is None:
        out = _new((E_loc, rows, ld), w.dtype, w.device, stream)
    _dev(out, "out", w.dtype)
    _need(out, "out", shape=(E_loc, rows, ld))
    _same_device(w, "w", out)
    _call(lib().moe_pack_weights, w, stream, _ptr(w), E_loc, rows, cols, code, _ptr(out))
    return out


def _w_packed(w, in_dim, act, name):
    """Layout of weight tensor w (E_local, out, last): False if last is the
    input dim (dense), True if it is the packed pitch, None when the packed
    pitch equals the input dim (both layouts are the same)."""
    ld = moe_weight_ld(in_dim, act)
    last = w.shape[2]
    if last == in_dim:
        return None if ld == in_dim else False
    if last == ld:
        return True
    raise ValueError(f"{name} must have {in_dim} columns (dense) or {ld} (packed), got {last}")


def _pack_flag(*layouts):
    """MOE_W_PACKED if the call's weights are packed; all of one call's
    weights share one layout."""
    seen = {x for x in layouts if x is not None}
    if len(seen) > 1:
        raise ValueError("the weights of one call must be all packed or all dense")
    return MOE_W_PACKED if seen == {True} else 0


def _rows_arg(rows, cap_per_expert, E_loc, n_rows):
    """(pointer tensor, third int argument) of the row description: offsets
    (E_loc+1) of the contiguous layout, or m (E_loc) of the masked one."""
    _dev(rows, "offsets" if cap_per_expert is None else "m", torch.int32, 1)
    if cap_per_expert is None:
        return n_rows
    if n_rows != E_loc * cap_per_expert:
        raise ValueError(f"masked layout needs E_loc * cap_per_expert = {E_loc * cap_per_expert} rows, "
                         f"got {n_rows}")
    return int(cap_per_expert)


def _check_ffn(a, a_scales, rows, cap_per_expert, E_loc, Kdim, cap, act, also, **tensors):
    """Shapes of the FFN operands: the activation rows (cap, Kdim) [+ fp8 or
    int8 scales], the row description (offsets E_loc + 1, or m E_loc), and each
    named (tensor, shape or minimum element count) pair; one device for all, `also` too."""
    if a.shape[1] != Kdim:
        raise ValueError(f"activations must have {Kdim} columns (got {a.shape[1]})")
    _need(rows, "offsets" if cap_per_expert is None else "m",
          numel=E_loc + 1 if cap_per_expert is None else E_loc)
    if act in (MOE_FP8_E4M3, MOE_INT8):
        if a_scales is None:
            raise ValueError("fp8 activations need their block scales" if act == MOE_FP8_E4M3
                             else "int8 activations need their row scales")
        _dev(a_scales, "activation scales", torch.float32)
        _need(a_scales, "activation scales", numel=cap * _scale_cols(act, Kdim))
    if act == MOE_INT8:
        for name, (t, _) in tensors.items():
            if name.startswith("w_") and name.endswith("_scales"):
                if t is None:
                    raise ValueError(f"int8 weights need {name}")
                _dev(t, name, torch.float32)
    _same_device(a, "activations", a_scales if act in (MOE_FP8_E4M3, MOE_INT8) else None, rows, *also)
    index = a.get_device()
    for name, (t, want) in tensors.items():
        if t is None:
            continue
        _dev(t, name)
        if t.get_device() != index:
            _same_device(a, "activations", t)
        if isinstance(want, tuple):
            _need(t, name, shape=want)
        else:
            _need(t, name, numel=want)


def _w_scales(act, scales, E_loc, rows, cols):
    """(weight scales, their shape) of a quantised weight (E_loc, rows, cols) for _check_ffn."""
    if act == MOE_FP8_E4M3:
        return scales, (E_loc, rows, -(-cols // FP8_BLOCK))
    return (scales, (E_loc, rows)) if act == MOE_INT8 else (None, None)


def _h_dtype_for(xd):
    """Storage of gate/up's output: the activations' own, but bf16 for int8 (moe_quant_rows
    makes its int8 rows, whose scale takes a whole row)."""
    return torch.bfloat16 if xd.dtype == torch.int8 else xd.dtype


def _w_code(act, w_scales_pow2):
    """Weight dtype code: fp8 weights whose block scales are all powers of two
    are declared as MOE_FP8_E4M3_PO2."""
    if w_scales_pow2 and act != MOE_FP8_E4M3:
        raise ValueError("w_scales_pow2 applies to fp8 weights only")
    return MOE_FP8_E4M3_PO2 if w_scales_pow2 else act


def moe_ffn_gate_up(xd, xd_scales, offsets, w_gate, w_up, w_gate_scales=None, w_up_scales=None,
                    h=None, h_scales=None, expected_rows=0, stream=None, cap_per_expert=None,
                    w_scales_pow2=False):
    """h = silu(Xd Wg^T) * (Xd Wu^T) per local expert -> (cap_rows, I) [+ scales].
    expected_rows: rows a local expert is expected to get (tile-shape hint only).
    With cap_per_expert given, ``offsets`` is the masked layout's m and the call
    is moe_ffn_gate_up_masked.  w_scales_pow2: the fp8 weight scales are all
    powers of two (weight dtype MOE_FP8_E4M3_PO2).  int8: xd_scales (cap_rows,),
    weight scales (E_loc, I), h is bf16 and h_scales None (see moe_quant_rows)."""
    _dev(xd, "xd", ndim=2)
    _dev(w_gate, "w_gate", xd.dtype, 3)
    _dev(w_up, "w_up", xd.dtype, 3)
    E_loc, I, H = w_gate.shape[0], w_gate.shape[1], xd.shape[1]
    cap = xd.shape[0]
    third = _rows_arg(offsets, cap_per_expert, E_loc, cap)
    act = _DT[xd.dtype]
    packed = _pack_flag(_w_packed(w_gate, H, act, "w_gate"))
    if h is None:
        h = _new((cap, I), _h_dtype_for(xd), xd.device, stream)
    if act == MOE_FP8_E4M3 and h_scales is None:
        h_scales = _new((cap, -(-I // FP8_BLOCK)), torch.float32, xd.device, stream)
    if h.dtype != _h_dtype_for(xd):
        raise ValueError(f"h must be {_h_dtype_for(xd)} (got {h.dtype})")
    nbI = -(-I // FP8_BLOCK)
    fp8 = act == MOE_FP8_E4M3
    _check_ffn(xd, xd_scales, offsets, cap_per_expert, E_loc, H, cap, act, (w_gate,),
               w_up=(w_up, tuple(w_gate.shape)), h=(h, cap * I),
               h_scales=(h_scales if fp8 else None, cap * nbI),
               w_gate_scales=_w_scales(act, w_gate_scales, E_loc, I, H),
               w_up_scales=_w_scales(act, w_up_scales, E_loc, I, H))
    fn = lib().moe_ffn_gate_up if cap_per_expert is None else lib().moe_ffn_gate_up_masked
    _call(fn, xd, stream, _ptr(xd), _ptr(xd_scales), _ptr(offsets), E_loc, third, H, I, act,
          _ptr(w_gate), _ptr(w_up), _ptr(w_gate_scales), _ptr(w_up_scales),
          _w_code(act, w_scales_pow2) | packed, _ptr(h), _ptr(h_scales), int(expected_rows))
    return h, h_scales


def _y_dtype_for(act):
    return torch.float32 if act == MOE_F32 else torch.bfloat16


def moe_ffn_down(h, h_scales, offsets, w_down, w_down_scales=None, y=None, y_dtype=None,
                 expected_rows=0, stream=None, cap_per_expert=None, w_scales_pow2=False):
    """y = h Wd^T per local expert -> (cap_rows, H).  cap_per_expert and
    w_scales_pow2: as in moe_ffn_gate_up (moe_ffn_down_masked).  int8: h_scales
    (cap_rows,), weight scales (E_loc, H), y bf16 (the default) or fp32."""
    _dev(h, "h", ndim=2)
    _dev(w_down, "w_down", h.dtype, 3)
    E_loc, H, I = w_down.shape[0], w_down.shape[1], h.shape[1]
    cap = h.shape[0]
    third = _rows_arg(offsets, cap_per_expert, E_loc, cap)
    act = _DT[h.dtype]
    packed = _pack_flag(_w_packed(w_down, I, act, "w_down"))
    y_dtype = _y_dtype_for(act) if y_dtype is None else y_dtype
    if y is None:
        y = _new((cap, H), y_dtype, h.device, stream)
    _check_ffn(h, h_scales, offsets, cap_per_expert, E_loc, I, cap, act, (w_down,), y=(y, cap * H),
               w_down_scales=_w_scales(act, w_down_scales, E_loc, H, I))
    fn = lib().moe_ffn_down if cap_per_expert is None else lib().moe_ffn_down_masked
    _call(fn, h, stream, _ptr(h), _ptr(h_scales), _ptr(offsets), E_loc, third, H, I, act,
          _ptr(w_down), _ptr(w_down_scales), _w_code(act, w_scales_pow2) | packed, _ptr(y), _DT[y.dtype],
          int(expected_rows))
    return y


def moe_grouped_ffn(xd, xd_scales, offsets, w_gate, w_up, w_down, w_gate_scales=None,
                    w_up_scales=None, w_down_scales=None, y=None, y_dtype=None, ws=None,
                    expected_rows=0, stream=None, cap_per_expert=None, w_scales_pow2=False):
    """Both FFN stages (int8: and the quantisation of h between them) with h held
    in the workspace ``ws``.  cap_per_expert
    and w_scales_pow2: as in moe_ffn_gate_up (moe_grouped_ffn_masked)."""
    _dev(xd, "xd", ndim=2)
    for n, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _dev(w, n, xd.dtype, 3)
    E_loc, I, H = w_gate.shape[0], w_gate.shape[1], xd.shape[1]
    cap = xd.shape[0]
    third = _rows_arg(offsets, cap_per_expert, E_loc, cap)
    act = _DT[xd.dtype]
    packed = _pack_flag(_w_packed(w_gate, H, act, "w_gate"), _w_packed(w_down, I, act, "w_down"))
    y_dtype = _y_dtype_for(act) if y_dtype is None else y_dtype
    if y is None:
        y = _new((cap, H), y_dtype, xd.device, stream)
    need = moe_ffn_workspace_bytes(cap, I, act)
    if ws is None:
        ws = _new(max(need, 256), torch.uint8, xd.device, stream, scratch=True)
    _dev(ws, "ws")
    _check_ffn(xd, xd_scales, offsets, cap_per_expert, E_loc, H, cap, act, (w_gate, ws),
               w_up=(w_up, tuple(w_gate.shape)), w_down=(w_down, (E_loc, H, w_down.shape[2])),
               y=(y, cap * H),
               w_gate_scales=_w_scales(act, w_gate_scales, E_loc, I, H),
               w_up_scales=_w_scales(act, w_up_scales, E_loc, I, H),
               w_down_scales=_w_scales(act, w_down_scales, E_loc, H, I))
    fn = lib().moe_grouped_ffn if cap_per_expert is None else lib().moe_grouped_ffn_masked
    _call(fn, xd, stream, _ptr(xd), _ptr(xd_scales), _ptr(offsets), E_loc, third, H, I, act,
          _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(w_gate_scales),
          _ptr(w_up_scales), _ptr(w_down_scales), _w_code(act, w_scales_pow2) | packed, _ptr(y),
          _DT[y.dtype], _ptr(ws), ws.numel() * ws.element_size(), int(expected_rows))
    return y


def moe_ffn_gate_up_masked(xd, xd_scales, m, cap_per_expert, w_gate, w_up, **kw):
    """moe_ffn_gate_up over the masked layout (rows [j*cap_per_expert, +m[j]))."""
    return moe_ffn_gate_up(xd, xd_scales, m, w_gate, w_up, cap_per_expert=cap_per_expert, **kw)


def moe_ffn_down_masked(h, h_scales, m, cap_per_expert, w_down, **kw):
    """moe_ffn_down over the masked layout."""
    return moe_ffn_down(h, h_scales, m, w_down, cap_per_expert=cap_per_expert, **kw)


def moe_grouped_ffn_masked(xd, xd_scales, m, cap_per_expert, w_gate, w_up, w_down, **kw):
    """moe_grouped_ffn over the masked layout."""
    return moe_grouped_ffn(xd, xd_scales, m, w_gate, w_up, w_down, cap_per_expert=cap_per_expert, **kw)


def moe_combine(y, row_of, topk_w, out=None, out_dtype=None, stream=None):
    """out[t] = sum_k topk_w[t,k] * y[row_of[t,k]] over local slots -> (B, H)."""
    _dev(y, "y", ndim=2)
    _dev(row_of, "row_of", torch.int32, 2)
    _dev(topk_w, "topk_w", torch.float32, 2)
    B, K = row_of.shape
    H = y.shape[1]
    if out is None:
        out = _new((B, H), y.dtype if out_dtype is None else out_dtype, y.device, stream)
    _dev(out, "out")
    _need(topk_w, "topk_w", shape=(B, K))
    _need(out, "out", numel=B * H)
    _same_device(y, "y", row_of, topk_w, out)
    _call(lib().moe_combine, y, stream, _ptr(y), _DT[y.dtype], y.shape[0], _ptr(row_of), _ptr(topk_w), B, K, H,
          _ptr(out), _DT[out.dtype])
    return out


# ----------------------------------------------------------------------------
# training step (contiguous layout, fp32 or bf16)
# ----------------------------------------------------------------------------
def _blocks(cols):
    """Scales of a checkpointed row."""
    return -(-cols // CKPT_BLOCK)


def _train_type(t, name):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be float32 or bfloat16 (got {t.dtype})")


def _is(t, name, dtype, shape, first, index):
    """t is a device tensor of this type and shape on the device (index) of the call's first
    tensor (a name).  One expression for what holds as a rule: the single checks and
    their messages cost a call of ten small tensors as much as its launch."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return
    _dev(t, name, dtype, len(shape))
    _need(t, name, shape=shape)
    if t.get_device() != index:
        raise ValueError(f"all tensors must be on {first}'s device cuda:{index} (got {t.device})")


def _out(t, name, dtype, shape, like, first, index, stream):
    """The caller's tensor after its checks, or a new one."""
    if t is None:
        return _new(shape, dtype, like.device, stream)
    _is(t, name, dtype, shape, first, index)
    return t


def _offsets(offsets, E_loc, first, index):
    """Local experts of the contiguous layout's offsets (None, all rows: 0)."""
    if offsets is None:
        if E_loc is not None:
            raise ValueError("E_loc needs the layout's offsets")
        return 0
    _dev(offsets, "offsets", torch.int32, 1)
    E_loc = max(offsets.numel() - 1, 1) if E_loc is None else E_loc
    if E_loc < 1:
        raise ValueError(f"E_loc must be positive (got {E_loc})")
    _need(offsets, "offsets", numel=E_loc + 1)
    if offsets.get_device() != index:
        raise ValueError(f"all tensors must be on {first}'s device cuda:{index} (got {offsets.device})")
    return E_loc


def moe_checkpoint_rows(x, offsets=None, q=None, scales=None, stream=None, E_loc=None):
    """8-bit checkpoint of the rows of x (fp32 or bf16): int8 codes (cap_rows, cols)
    and a power-of-two scale for each 128 columns of a row, (cap_rows,
    ceil(cols/128)).  offsets: the contiguous layout's (E_loc + 1), None for all rows;
    other rows of given q and scales are left as they were.  E_loc: as in
    moe_quant_rows."""
    _dev(x, "x", None, 2)
    _train_type(x, "x")
    cap, cols = x.shape
    index = x.get_device()
    E_loc = _offsets(offsets, E_loc, "x", index)
    q = _out(q, "q", torch.int8, (cap, cols), x, "x", index, stream)
    scales = _out(scales, "scales", torch.float32, (cap, _blocks(cols)), x, "x", index, stream)
    _call(lib().moe_checkpoint_rows, x, stream, x.data_ptr(), _DT[x.dtype], _ptr(offsets), E_loc, cap, cols, q.data_ptr(),
          scales.data_ptr())
    return q, scales


def moe_checkpoint_values(q, scales, offsets=None, out=None, out_dtype=torch.bfloat16, stream=None, E_loc=None):
    """The values (cap_rows, cols) that a checkpoint stands for, exact in bf16 and fp32;
    offsets and E_loc as in moe_checkpoint_rows."""
    _dev(q, "q", torch.int8, 2)
    cap, cols = q.shape
    index = q.get_device()
    _is(scales, "scales", torch.float32, (cap, _blocks(cols)), "q", index)
    E_loc = _offsets(offsets, E_loc, "q", index)
    out = _out(out, "out", out_dtype if out is None else out.dtype, (cap, cols), q, "q", index, stream)
    _train_type(out, "out")
    _call(lib().moe_checkpoint_values, q, stream, q.data_ptr(), scales.data_ptr(), _ptr(offsets), E_loc, cap, cols,
          out.data_ptr(), _DT[out.dtype])
    return out


def moe_ffn_gate_up_train(xd, offsets, w_gate, w_up, h=None, gate_q=None, gate_scales=None, up_q=None, up_scales=None,
                          expected_rows=0, stream=None):
    """moe_ffn_gate_up (fp32 or bf16) that also leaves gate and up, before SwiGLU, as
    8-bit checkpoints -> h (cap_rows, I), (gate_q, gate_scales), (up_q, up_scales)."""
    _dev(xd, "xd", ndim=2)
    _train_type(xd, "xd")
    index, dt = xd.get_device(), xd.dtype
    _dev(w_gate, "w_gate", dt, 3)
    (E_loc, I, _), (cap, H) = w_gate.shape, xd.shape
    _is(w_gate, "w_gate", dt, w_gate.shape, "xd", index)
    _is(w_up, "w_up", dt, w_gate.shape, "xd", index)
    act = _DT[dt]
    packed = _pack_flag(_w_packed(w_gate, H, act, "w_gate"))
    _offsets(offsets, E_loc, "xd", index)
    h = _out(h, "h", dt, (cap, I), xd, "xd", index, stream)
    gate_q = _out(gate_q, "gate_q", torch.int8, (cap, I), xd, "xd", index, stream)
    up_q = _out(up_q, "up_q", torch.int8, (cap, I), xd, "xd", index, stream)
    gate_scales = _out(gate_scales, "gate_scales", torch.float32, (cap, _blocks(I)), xd, "xd", index, stream)
    up_scales = _out(up_scales, "up_scales", torch.float32, (cap, _blocks(I)), xd, "xd", index, stream)
    _call(lib().moe_ffn_gate_up_train, xd, stream, _ptr(xd), _ptr(offsets), E_loc, cap, H, I, act, _ptr(w_gate),
          _ptr(w_up), act | packed, _ptr(h), _ptr(gate_q), _ptr(gate_scales), _ptr(up_q), _ptr(up_scales),
          int(expected_rows))
    return h, (gate_q, gate_scales), (up_q, up_scales)


def moe_swiglu_backward(dh, gate_q, gate_scales, up_q, up_scales, row_of, topk_w, dgate=None, dup=None, hw=None,
                        dtopk_w=None, stream=None):
    """From dh (cap_rows, I), the gradient of h before the routing weights, and the
    checkpoints of gate and up: dgate, dup, hw = topk_w * h (cap_rows, I) and dtopk_w
    (B, K).  Rows that no slot of row_of names are left as they were."""
    _dev(dh, "dh", ndim=2)
    _train_type(dh, "dh")
    index, dt, rows = dh.get_device(), dh.dtype, dh.shape
    cap, I = rows
    blocks = (cap, _blocks(I))
    _is(gate_q, "gate_q", torch.int8, rows, "dh", index)
    _is(up_q, "up_q", torch.int8, rows, "dh", index)
    _is(gate_scales, "gate_scales", torch.float32, blocks, "dh", index)
    _is(up_scales, "up_scales", torch.float32, blocks, "dh", index)
    _dev(row_of, "row_of", torch.int32, 2)
    slots = row_of.shape
    _is(row_of, "row_of", torch.int32, slots, "dh", index)
    _is(topk_w, "topk_w", torch.float32, slots, "dh", index)
    dgate = _out(dgate, "dgate", dt, rows, dh, "dh", index, stream)
    dup = _out(dup, "dup", dt, rows, dh, "dh", index, stream)
    hw = _out(hw, "hw", dt, rows, dh, "dh", index, stream)
    dtopk_w = _out(dtopk_w, "dtopk_w", torch.float32, slots, dh, "dh", index, stream)
    _call(lib().moe_swiglu_backward, dh, stream, dh.data_ptr(), _DT[dt], gate_q.data_ptr(), gate_scales.data_ptr(),
          up_q.data_ptr(), up_scales.data_ptr(), cap, I, row_of.data_ptr(), topk_w.data_ptr(), slots[0], slots[1],
          dgate.data_ptr(), dup.data_ptr(), hw.data_ptr(), dtopk_w.data_ptr())
    return dgate, dup, hw, dtopk_w


def moe_ffn_dgrad(dy, offsets, w, dy2=None, w2=None, src_of=None, slots_per_token=1, dx=None, in_dim=None,
                  expected_rows=0, stream=None):
    """dx[r] = dy[r] W_j (+ dy2[r] W2_j) for the rows of every local expert -> (cap_rows,
    in_dim); w, w2 (E_loc, out_dim, in_dim), or packed (E_loc, out_dim, pitch) with
    in_dim given (or dx).  src_of (cap_rows,): row r reads dy's row src_of[r] //
    slots_per_token (a token's gradient); None: row r itself."""
    _dev(dy, "dy", ndim=2)
    _train_type(dy, "dy")
    index, dt = dy.get_device(), dy.dtype
    _dev(w, "w", dt, 3)
    _is(w, "w", dt, w.shape, "dy", index)
    E_loc, out_dim = w.shape[0], w.shape[1]
    if dy.shape[1] != out_dim:
        raise ValueError(f"dy must have {out_dim} columns (got {dy.shape[1]})")
    _offsets(offsets, E_loc, "dy", index)
    if (dy2 is None) != (w2 is None):
        raise ValueError("dy2 and w2 come together")
    if dy2 is not None:
        _is(dy2, "dy2", dt, dy.shape, "dy", index)
        _is(w2, "w2", dt, w.shape, "dy", index)
    if in_dim is None:
        in_dim = w.shape[2] if dx is None else dx.shape[-1]
    act = _DT[dt]
    packed = _pack_flag(_w_packed(w, in_dim, act, "w"))
    if src_of is None:
        cap = dy.shape[0]
    else:
        _dev(src_of, "src_of", torch.int32, 1)
        cap = src_of.numel() if dx is None else dx.shape[0]
        _need(src_of, "src_of", numel=cap)
        _is(src_of, "src_of", torch.int32, src_of.shape, "dy", index)
    dx = _out(dx, "dx", dt, (cap, in_dim), dy, "dy", index, stream)
    _call(lib().moe_ffn_dgrad, dy, stream, _ptr(dy), _ptr(dy2), _ptr(src_of), int(slots_per_token), dy.shape[0],
          _ptr(offsets), E_loc, cap, out_dim, in_dim, act, _ptr(w), _ptr(w2), act | packed, _ptr(dx),
          int(expected_rows))
    return dx


_GATHER = {None: MOE_GATHER_NONE, "x": MOE_GATHER_X, "dy": MOE_GATHER_DY}


def moe_ffn_wgrad(dy, x, offsets, x_scales=None, dy2=None, src_of=None, slots_per_token=1, gather=None, base=None,
                  base2=None, dw=None, dw2=None, dw_dtype=torch.float32, expected_rows=0, stream=None, E_loc=None):
    """dw_j = base_j + sum over expert j's rows of dy[r]^T x[r] -> (E_loc, out_dim, in_dim)
    fp32, or bf16 beside bf16 activations; with dy2 a pair (dw, dw2) that shares x.
    x: dy's type, or the int8 codes of a checkpoint with x_scales.  gather 'x' or
    'dy': that operand holds tokens, and row r reads its row src_of[r] //
    slots_per_token.  base may be dw itself (accumulation over micro-batches)."""
    _dev(dy, "dy", ndim=2)
    _train_type(dy, "dy")
    index, dt = dy.get_device(), dy.dtype
    _dev(x, "x", ndim=2)
    _is(x, "x", x.dtype, x.shape, "dy", index)
    out_dim, in_dim = dy.shape[1], x.shape[1]
    if x.dtype not in (dt, torch.int8):
        raise ValueError(f"x must be {dt} or a checkpoint's int8 (got {x.dtype})")
    if (x.dtype == torch.int8) != (x_scales is not None):
        raise ValueError("x_scales belong to a checkpoint's int8 x")
    if x_scales is not None:
        _is(x_scales, "x_scales", torch.float32, (x.shape[0], _blocks(in_dim)), "dy", index)
    if dy2 is not None:
        _is(dy2, "dy2", dt, dy.shape, "dy", index)
    elif dw2 is not None or base2 is not None:
        raise ValueError("dw2 and base2 belong to dy2")
    if gather not in _GATHER:
        raise ValueError(f"gather must be None, 'x' or 'dy' (got {gather!r})")
    if offsets is None:
        raise ValueError("offsets must be a torch.Tensor")
    E_loc = _offsets(offsets, (dw.shape[0] if dw is not None and dw.dim() == 3 else None) if E_loc is None else E_loc,
                     "dy", index)
    cap, src_rows = (x.shape[0], dy.shape[0]) if gather == "dy" else (dy.shape[0], x.shape[0])
    if gather is None:
        if src_rows != cap:
            raise ValueError(f"dy and x must have the same rows (got {cap} and {src_rows})")
    else:
        if src_of is None:
            raise ValueError("a gathered operand needs src_of")
        _dev(src_of, "src_of", torch.int32, 1)
        _need(src_of, "src_of", numel=cap)
        _is(src_of, "src_of", torch.int32, src_of.shape, "dy", index)
    shape = (E_loc, out_dim, in_dim)
    dw = _out(dw, "dw", dw_dtype if dw is None else dw.dtype, shape, dy, "dy", index, stream)
    if dy2 is not None:
        dw2 = _out(dw2, "dw2", dw.dtype, shape, dy, "dy", index, stream)
    for name, t in (("base", base), ("base2", base2)):
        if t is not None:
            _is(t, name, dw.dtype, shape, "dy", index)
    _call(lib().moe_ffn_wgrad, dy, stream, _ptr(dy), _ptr(dy2), _ptr(x),
          MOE_CKPT8 if x.dtype == torch.int8 else _DT[x.dtype], _ptr(x_scales), _ptr(src_of) if gather else None,
          int(slots_per_token), src_rows, _GATHER[gather], _ptr(offsets), E_loc, cap, out_dim, in_dim, _DT[dt],
          _ptr(base), _ptr(base2), _ptr(dw), _ptr(dw2), _DT.get(dw.dtype, -1), int(expected_rows))
    return dw if dy2 is None else (dw, dw2)


_BACK_SCORES = {"picks": MOE_SCORE_PICKS, **_SCORES}


def moe_route_backward(logits, topk_ids, dtopk_w, score: str = "picks", renorm: bool = True, scale: float = 1.0,
                       phys_of_logical=None, n_shared: int = 0, dlogits=None, stream=None):
    """dlogits (B, E) fp32 from the gradient dtopk_w (B, K + n_shared) of the routing
    weights.  score 'picks': moe_route and its variants; 'sigmoid' or 'softmax':
    moe_route_scored with its renorm, scale, placement map and shared slots."""
    _dev(logits, "logits", None, 2)
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits must be float32 or bfloat16 (got {logits.dtype})")
    if score not in _BACK_SCORES:
        raise ValueError(f"score must be one of {sorted(_BACK_SCORES)} (got {score!r})")
    B, E = logits.shape
    index = logits.get_device()
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    Kt = topk_ids.shape[1]
    _is(topk_ids, "topk_ids", torch.int32, (B, Kt), "logits", index)
    _is(dtopk_w, "dtopk_w", torch.float32, (B, Kt), "logits", index)
    if phys_of_logical is not None:
        _is(phys_of_logical, "phys_of_logical", torch.int32, (E,), "logits", index)
    dlogits = _out(dlogits, "dlogits", torch.float32, (B, E), logits, "logits", index, stream)
    _call(lib().moe_route_backward, logits, stream, logits.data_ptr(), _DT[logits.dtype], topk_ids.data_ptr(),
          dtopk_w.data_ptr(), B, E, Kt - n_shared, _BACK_SCORES[score], 1 if renorm else 0, scale,
          _ptr(phys_of_logical), n_shared, dlogits.data_ptr())
    return dlogits


from .layer import MoELayer  # noqa: E402  (uses the functions above)
