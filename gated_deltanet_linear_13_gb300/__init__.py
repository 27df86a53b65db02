"""gated_deltanet_linear_13_gb300 -- Python binding of libgdn.so (GB300 / sm_103a).

The gated delta rule (Gated DeltaNet) behind a C ABI (``include/gdn.h``):
``gdn_chunk_prefill``, ``gdn_decode_step``, ``causal_conv1d_update``, ``gdn_state_checkpoint``.
This module only marshals torch tensors into pointers and sizes: every step of the path runs
in the CUDA kernels of ``libgdn.so``.  It checks shapes, dtypes, devices and contiguity
before handing raw pointers to the library (a wrong size would otherwise let a kernel read
past a buffer).  The usual call of the serving step's operators is checked and marshalled by a
native part (``csrc/marshal.cpp``), whatever it leaves by the checks here, and all of it where that
part is missing or belongs to another torch.  If ``libgdn.so`` is missing loading it fails: there is
no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")
HEAD_DIM = 128

GDN_OK = 0
GDN_F32, GDN_BF16 = 0, 1
GDN_KV_BF16, GDN_KV_E4M3 = 0, 1
GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}   # gdn_rope_scaling in include/gdn.h
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARGUMENT", 2: "GDN_ERR_UNSUPPORTED",
                3: "GDN_ERR_WORKSPACE", 4: "GDN_ERR_CUDA", 5: "GDN_ERR_DEVICE_TIMEOUT",
                6: "GDN_ERR_DEVICE_INDEX"}

EXPORTED = ("gdn_prefill_workspace_size", "gdn_chunk_prefill", "gdn_decode_step",
            "causal_conv1d_update", "gdn_state_checkpoint", "gdn_chunk_prefill_noalloc",
            "gdn_chunk_prefill_snapshots", "gdn_chunk_prefill_gated", "gdn_decode_step_gated",
            "gdn_prefill_varlen_workspace_size", "gdn_chunk_prefill_varlen", "gdn_decode_multi",
            "gdn_get_device_error", "gdn_status_string", "gdn_version",
            "gdn_selftest_device_timeout", "gdn_chunk_prefill_ex",
            "gdn_kv_cache_append", "gdn_kv_cache_read", "gdn_prefix_attention_workspace_size",
            "gdn_prefix_attention", "gdn_token_logprobs_workspace_size", "gdn_token_logprobs",
            "gdn_qk_norm_rope", "gdn_rope_phase_steps", "gdn_page_plan", "gdn_page_release",
            "gdn_verify_tokens_workspace_size", "gdn_verify_tokens")
NOALLOC_SCRATCH_BYTES = 64 << 20   # GDN_NOALLOC_SCRATCH_BYTES in include/gdn.h


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class GdnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("chunk_size", ctypes.c_int32),
                ("conv_width", ctypes.c_int32), ("num_slots", ctypes.c_int32)]


class GdnOpts(ctypes.Structure):
    _fields_ = [("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("qk_l2norm", ctypes.c_int32), ("l2_eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("conv_silu", ctypes.c_int32),
                ("gates_precomputed", ctypes.c_int32)]


class GdnOutGate(ctypes.Structure):
    _fields_ = [("z", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


class GdnPrefillExt(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("snap_every", ctypes.c_int32),
                ("snap_state", ctypes.c_void_p), ("snap_conv_state", ctypes.c_void_p),
                ("num_snap_slots", ctypes.c_int32), ("snap_slots", ctypes.c_void_p),
                ("prev_workspace", ctypes.c_void_p)]


class GdnKvCache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("format", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p)]


class GdnRope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int),
                ("amplitude", ctypes.c_float), ("phase_steps", ctypes.c_void_p)]


class GdnPagePool(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p)]


_vp = ctypes.c_void_p
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (raises OSError when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"libgdn.so not found at {path}: build it with "
                      "`python -m gated_deltanet_linear_13_gb300.build_lib`")
    L = ctypes.CDLL(path)
    dp, op = ctypes.POINTER(GdnDims), ctypes.POINTER(GdnOpts)
    L.gdn_prefill_workspace_size.restype = ctypes.c_size_t
    L.gdn_prefill_workspace_size.argtypes = [dp, op]
    L.gdn_chunk_prefill.restype = ctypes.c_int
    L.gdn_chunk_prefill.argtypes = [dp, op] + [_vp] * 14 + [ctypes.c_size_t, _vp]
    L.gdn_chunk_prefill_snapshots.restype = ctypes.c_int
    L.gdn_chunk_prefill_snapshots.argtypes = ([dp, op] + [_vp] * 13 +
                                              [ctypes.c_int32, _vp, _vp, ctypes.c_int32, _vp,
                                               _vp, ctypes.c_size_t, _vp])
    gp = ctypes.POINTER(GdnOutGate)
    L.gdn_chunk_prefill_gated.restype = ctypes.c_int
    L.gdn_chunk_prefill_gated.argtypes = [dp, op] + [_vp] * 13 + [gp, _vp, ctypes.c_size_t, _vp]
    L.gdn_chunk_prefill_ex.restype = ctypes.c_int
    L.gdn_chunk_prefill_ex.argtypes = ([dp, op] + [_vp] * 13 +
                                       [ctypes.POINTER(GdnPrefillExt), _vp, ctypes.c_size_t, _vp])
    L.gdn_decode_step_gated.restype = ctypes.c_int
    L.gdn_decode_step_gated.argtypes = [dp, op] + [_vp] * 13 + [gp, _vp]
    L.gdn_prefill_varlen_workspace_size.restype = ctypes.c_size_t
    L.gdn_prefill_varlen_workspace_size.argtypes = [dp, op]
    L.gdn_chunk_prefill_varlen.restype = ctypes.c_int
    L.gdn_chunk_prefill_varlen.argtypes = [dp, op] + [_vp] * 14 + [gp, _vp, ctypes.c_size_t, _vp]
    L.gdn_decode_multi.restype = ctypes.c_int
    L.gdn_decode_multi.argtypes = [dp, op] + [_vp] * 15 + [ctypes.c_int32, _vp, _vp]
    L.gdn_chunk_prefill_noalloc.restype = ctypes.c_int
    L.gdn_chunk_prefill_noalloc.argtypes = [dp, op] + [_vp] * 13 + [_vp]
    L.gdn_decode_step.restype = ctypes.c_int
    L.gdn_decode_step.argtypes = [dp, op] + [_vp] * 13 + [_vp]
    L.causal_conv1d_update.restype = ctypes.c_int
    L.causal_conv1d_update.argtypes = ([ctypes.c_int32] * 4 + [ctypes.c_int] + [_vp] * 4 +
                                       [ctypes.c_int32, _vp, ctypes.c_int32, _vp, _vp])
    L.gdn_state_checkpoint.restype = ctypes.c_int
    L.gdn_state_checkpoint.argtypes = ([ctypes.c_int32, dp, ctypes.c_int] + [_vp] * 4 +
                                       [ctypes.c_int32, _vp, _vp, ctypes.c_int32, _vp])
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cp = ctypes.POINTER(GdnKvCache)
    L.gdn_kv_cache_append.restype = ctypes.c_int
    L.gdn_kv_cache_append.argtypes = [cp, i32, ctypes.c_int, _vp, i64, _vp, i64, _vp, _vp]
    L.gdn_kv_cache_read.restype = ctypes.c_int
    L.gdn_kv_cache_read.argtypes = [cp, i32, _vp, ctypes.c_int, _vp, _vp, _vp]
    L.gdn_prefix_attention_workspace_size.restype = sz
    L.gdn_prefix_attention_workspace_size.argtypes = [i32] * 5
    L.gdn_prefix_attention.restype = ctypes.c_int
    L.gdn_prefix_attention.argtypes = ([cp] + [i32] * 3 + [_vp, i64, _vp, i32, _vp, i32, _vp,
                                       ctypes.c_float, ctypes.c_int] + [_vp] * 3 + [sz, _vp])
    L.gdn_token_logprobs_workspace_size.restype = sz
    L.gdn_token_logprobs_workspace_size.argtypes = [i32, i32, ctypes.c_int, i32]
    L.gdn_token_logprobs.restype = ctypes.c_int
    L.gdn_token_logprobs.argtypes = ([i32, i32, ctypes.c_int, _vp, i64, _vp, ctypes.c_float, _vp,
                                      _vp, i32] + [_vp] * 3 + [sz, _vp])
    f32, f64 = ctypes.c_float, ctypes.c_double
    L.gdn_qk_norm_rope.restype = ctypes.c_int
    L.gdn_qk_norm_rope.argtypes = ([i32] * 4 + [ctypes.c_int, _vp, i64, i64, _vp, i64, _vp, _vp,
                                    f32, _vp, ctypes.POINTER(GdnRope), _vp, i64, _vp, cp, _vp,
                                    i64, _vp, _vp])
    L.gdn_rope_phase_steps.restype = ctypes.c_int
    L.gdn_rope_phase_steps.argtypes = ([i32, f64, ctypes.c_int] + [f64] * 4 +
                                       [ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(f32)])
    pp = ctypes.POINTER(GdnPagePool)
    L.gdn_page_plan.restype = ctypes.c_int
    L.gdn_page_plan.argtypes = [pp, i32, _vp, _vp, _vp, i32, i32] + [_vp] * 6
    L.gdn_page_release.restype = ctypes.c_int
    L.gdn_page_release.argtypes = [pp, i32, _vp, _vp, _vp]
    L.gdn_verify_tokens_workspace_size.restype = sz
    L.gdn_verify_tokens_workspace_size.argtypes = [i32, i32, i32, ctypes.c_int, i32]
    L.gdn_verify_tokens.restype = ctypes.c_int
    L.gdn_verify_tokens.argtypes = ([i32] * 3 + [ctypes.c_int, _vp, i64, _vp, _vp, i64] +
                                    [_vp] * 7 + [sz, _vp])
    L.gdn_get_device_error.restype = ctypes.c_int
    L.gdn_get_device_error.argtypes = [_vp]
    L.gdn_selftest_device_timeout.restype = ctypes.c_int
    L.gdn_selftest_device_timeout.argtypes = [ctypes.c_uint32, _vp]
    L.gdn_status_string.restype = ctypes.c_char_p
    L.gdn_status_string.argtypes = [ctypes.c_int]
    L.gdn_version.restype = ctypes.c_int32
    L.gdn_version.argtypes = []
    _bind_marshal(L)
    _lib = L
    return L


class _NoNative:
    """In the place of the binding's native part: leaves every call to the checks in Python."""

    @staticmethod
    def qk_norm_rope(*args):
        return None

    page_plan = page_release = verify_tokens = qk_norm_rope


_native = _NoNative


def _bind_marshal(L: ctypes.CDLL) -> None:
    """The binding's native part (csrc/marshal.cpp), on the functions of this library, if it is
    there and was built against this torch (whose tensors it reads)."""
    global _native
    _native = _NoNative
    try:
        from . import _marshal as m
    except ImportError:
        return
    if getattr(m, "torch_version", None) != str(torch.__version__):
        return
    m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
             (L.gdn_qk_norm_rope, L.gdn_page_plan, L.gdn_page_release, L.gdn_verify_tokens)),
           getattr(torch._C, "_cuda_getCurrentRawStream", None))
    _native = m


# ---------------------------------------------------------------- marshalling helpers

def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: Optional[torch.Tensor], name: str, shape, dtype, device):
    if (t is not None and t.dtype is dtype and t.shape == shape and t.device == device and
            t.is_contiguous()):
        return                       # the usual case, ahead of finding out what is wrong
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_of(stream, device: torch.device) -> int:
    """The raw stream; by default the current one of the tensors' device (a lookup without the
    Stream object, whose making costs as much as a launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return _stream(stream)


def _workspace(need: int, device: torch.device, stream) -> torch.Tensor:
    """A call's own workspace, from the pool of the stream that it runs on, so that the memory
    goes to nobody else before the call is through."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        raw = _stream(stream)
        stream = (torch.cuda.ExternalStream(raw, device=device) if raw
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):                  # (None: the current one)
        return torch.empty(need, dtype=torch.uint8, device=device)


def _workspace_bytes(workspace: torch.Tensor, device: torch.device) -> int:
    """The bytes of a caller's workspace, which the kernels take as one piece of the device's."""
    if workspace.device != device:
        raise ValueError(f"workspace: on {workspace.device}, expected {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.nbytes


def _check(status: int, where: str):
    if status != GDN_OK:
        raise GDNError(status, where)


def _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state, state, state_slots,
                num_slots_hint):
    B, T, Hv = a.shape
    W = 0 if conv_weight is None else conv_weight.shape[1]
    if W > 0:
        Hk = num_k_heads
        C = (2 * Hk + Hv) * HEAD_DIM
        if q.shape != (B, T, C):
            raise ValueError(f"x: shape {tuple(q.shape)}, expected {(B, T, C)}")
    else:
        Hk = q.shape[2]
    num_slots = state.shape[0]
    if state_slots is None and num_slots < B:
        raise ValueError("state has fewer rows than the batch and no state_slots given")
    return B, T, Hk, Hv, W, num_slots


def _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    in_t = q.dtype
    d = HEAD_DIM
    C = (2 * Hk + Hv) * d
    if W > 0:
        if k is not None or v is not None:
            raise ValueError("with a conv, pass the pre-conv x as q and k = v = None")
        _need(conv_weight, "conv_weight", (C, W), in_t, dev)
        if conv_bias is not None:
            _need(conv_bias, "conv_bias", (C,), in_t, dev)
        if W > 1:
            _need(conv_state, "conv_state", (num_slots, W - 1, C), in_t, dev)
    else:
        _need(q, "q", (B, T, Hk, d), in_t, dev)
        _need(k, "k", (B, T, Hk, d), in_t, dev)
        _need(v, "v", (B, T, Hv, d), in_t, dev)
    gt = torch.float32 if gates_precomputed else in_t
    _need(a, "a", (B, T, Hv), gt, dev)
    _need(b, "b", (B, T, Hv), gt, dev)
    if not gates_precomputed:
        _need(A_log, "A_log", (Hv,), torch.float32, dev)
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", (Hv,), torch.float32, dev)
    _need(state, "state", (num_slots, Hv, d, d), torch.float32, dev)
    if state_slots is not None:
        _need(state_slots, "state_slots", (B,), torch.int32, dev)
    if out.device != dev or not out.is_contiguous() or tuple(out.shape) != (B, T, Hv, d):
        raise ValueError(f"out: expected contiguous {(B, T, Hv, d)} on {dev}")


def _opts(in_dtype, out_dtype, qk_l2norm, eps, scale, conv_silu, gates_precomputed):
    return GdnOpts(in_dtype, out_dtype, int(qk_l2norm), float(eps), float(scale),
                   int(conv_silu), int(gates_precomputed))


# ---------------------------------------------------------------- public API

def gdn_prefill_workspace_size(batch: int, seqlen: int, num_k_heads: int, num_v_heads: int,
                               conv_width: int, in_dtype=torch.bfloat16) -> int:
    L = load_library()
    dims = GdnDims(batch, seqlen, num_k_heads, num_v_heads, HEAD_DIM, 64, conv_width, 0)
    dt = GDN_BF16 if in_dtype == torch.bfloat16 else GDN_F32
    opts = _opts(dt, dt, 1, 1e-6, 1.0, 1, 0)
    return int(L.gdn_prefill_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))


def gdn_chunk_prefill(q, k, v, a, b, A_log, dt_bias, state, out, *, num_k_heads=None,
                      conv_weight=None, conv_bias=None, conv_state=None, state_slots=None,
                      scale: float = 1.0, eps: float = 1e-6, qk_l2norm: bool = True,
                      conv_silu: bool = True, gates_precomputed: bool = False,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Chunked prefill (see gdn_chunk_prefill in include/gdn.h).  With a conv, ``q`` is the
    pre-conv x [B,T,C_conv] and ``k = v = None``.  ``state`` (and ``conv_state``) are updated
    in place; ``out`` [B,T,Hv,128] is written.  Returns ``out``."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    dims = GdnDims(B, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    need = int(L.gdn_prefill_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = L.gdn_chunk_prefill(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(v),
                             _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(conv_weight),
                             _ptr(conv_bias), _ptr(state), _ptr(conv_state), _ptr(state_slots),
                             _ptr(out), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_prefill")
    return out


def gdn_chunk_prefill_snapshots(q, k, v, a, b, A_log, dt_bias, state, out, *, snap_every: int,
                                snap_state, snap_slots, snap_conv_state=None, num_k_heads=None,
                                conv_weight=None, conv_bias=None, conv_state=None,
                                state_slots=None, scale: float = 1.0, eps: float = 1e-6,
                                qk_l2norm: bool = True, conv_silu: bool = True,
                                gates_precomputed: bool = False,
                                workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """gdn_chunk_prefill over the whole prompt in one call, recording the state after every
    ``snap_every`` tokens (see gdn_chunk_prefill_snapshots in include/gdn.h): snapshot j of
    row b goes to bank row ``snap_slots[b, j]`` of ``snap_state`` [n, Hv, 128, 128] (and of
    ``snap_conv_state`` [n, W-1, C_conv] with a conv), j < T // snap_every.  Returns ``out``."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    dev = q.device
    n_snap = T // snap_every if snap_every > 0 else 0
    nb = snap_state.shape[0]
    _need(snap_state, "snap_state", (nb, Hv, HEAD_DIM, HEAD_DIM), torch.float32, dev)
    _need(snap_slots, "snap_slots", (B, n_snap), torch.int32, dev)
    if W > 1:
        _need(snap_conv_state, "snap_conv_state", (nb, W - 1, (2 * Hk + Hv) * HEAD_DIM),
              q.dtype, dev)
    dims = GdnDims(B, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    need = int(L.gdn_prefill_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = L.gdn_chunk_prefill_snapshots(
        ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
        _ptr(A_log), _ptr(dt_bias), _ptr(conv_weight), _ptr(conv_bias), _ptr(state),
        _ptr(conv_state), _ptr(state_slots), _ptr(out), int(snap_every), _ptr(snap_state),
        _ptr(snap_conv_state), nb, _ptr(snap_slots), _ptr(workspace), ws_bytes,
        _stream(stream))
    _check(st, "gdn_chunk_prefill_snapshots")
    return out


def gdn_chunk_prefill_noalloc(q, k, v, a, b, A_log, dt_bias, state, out, *, num_k_heads=None,
                              conv_weight=None, conv_bias=None, conv_state=None,
                              state_slots=None, scale: float = 1.0, eps: float = 1e-6,
                              qk_l2norm: bool = True, conv_silu: bool = True,
                              gates_precomputed: bool = False, stream=None) -> torch.Tensor:
    """gdn_chunk_prefill without a workspace, for callers that cannot allocate: the library's
    fixed device scratch array (NOALLOC_SCRATCH_BYTES per GPU) holds the call's workspace.  Raises GDNError(GDN_ERR_WORKSPACE) when the call needs more than that.
    Calls that overlap on the GPU share that array and must be serialised."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    dims = GdnDims(B, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    st = L.gdn_chunk_prefill_noalloc(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k),
                                     _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                     _ptr(conv_weight), _ptr(conv_bias), _ptr(state),
                                     _ptr(conv_state), _ptr(state_slots), _ptr(out),
                                     _stream(stream))
    _check(st, "gdn_chunk_prefill_noalloc")
    return out


def gdn_decode_step(q, k, v, a, b, A_log, dt_bias, state, out, *, num_k_heads=None,
                    conv_weight=None, conv_bias=None, conv_state=None, state_slots=None,
                    scale: float = 1.0, eps: float = 1e-6, qk_l2norm: bool = True,
                    conv_silu: bool = True, gates_precomputed: bool = False,
                    stream=None) -> torch.Tensor:
    """One decode step for B sequences (T = 1), fused into one kernel launch."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    if T != 1:
        raise ValueError("gdn_decode_step takes exactly one token per sequence")
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    dims = GdnDims(B, 1, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    st = L.gdn_decode_step(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(v),
                           _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(conv_weight),
                           _ptr(conv_bias), _ptr(state), _ptr(conv_state), _ptr(state_slots),
                           _ptr(out), _stream(stream))
    _check(st, "gdn_decode_step")
    return out


def _out_gate(gate_z, gate_weight, gate_eps, out, in_dtype) -> GdnOutGate:
    dev = out.device
    _need(gate_z, "gate_z", tuple(out.shape), in_dtype, dev)
    _need(gate_weight, "gate_weight", (HEAD_DIM,), torch.float32, dev)
    return GdnOutGate(_ptr(gate_z), _ptr(gate_weight), float(gate_eps))


def gdn_chunk_prefill_gated(q, k, v, a, b, A_log, dt_bias, state, out, *, gate_z, gate_weight,
                            gate_eps: float = 1e-6, num_k_heads=None, conv_weight=None,
                            conv_bias=None, conv_state=None, state_slots=None,
                            scale: float = 1.0, eps: float = 1e-6, qk_l2norm: bool = True,
                            conv_silu: bool = True, gates_precomputed: bool = False,
                            workspace: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """gdn_chunk_prefill with the gated RMS norm on the output (see gdn_out_gate in
    include/gdn.h): out = gate_weight * o / sqrt(mean(o^2) + gate_eps) * silu(gate_z) per
    (token, value head); gate_z has the shape of out and the input dtype."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    gate = _out_gate(gate_z, gate_weight, gate_eps, out, q.dtype)
    dims = GdnDims(B, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    need = int(L.gdn_prefill_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = L.gdn_chunk_prefill_gated(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                   _ptr(conv_weight), _ptr(conv_bias), _ptr(state),
                                   _ptr(conv_state), _ptr(state_slots), _ptr(out),
                                   ctypes.byref(gate), _ptr(workspace), ws_bytes,
                                   _stream(stream))
    _check(st, "gdn_chunk_prefill_gated")
    return out


def gdn_chunk_prefill_ex(q, k, v, a, b, A_log, dt_bias, state, out, *, num_k_heads=None,
                         conv_weight=None, conv_bias=None, conv_state=None, state_slots=None,
                         scale: float = 1.0, eps: float = 1e-6, qk_l2norm: bool = True,
                         conv_silu: bool = True, gates_precomputed: bool = False,
                         gate_z=None, gate_weight=None, gate_eps: float = 1e-6,
                         snap_every: int = 0, snap_state=None, snap_slots=None,
                         snap_conv_state=None, prev_workspace: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """gdn_chunk_prefill with any of its optional parts (see gdn_chunk_prefill_ex in
    include/gdn.h): the gated output norm (``gate_z``, ``gate_weight``), in-call snapshots
    (``snap_every`` > 0, as gdn_chunk_prefill_snapshots), and ``prev_workspace``: the
    workspace of the previous prefill call of the same sequences on this stream, which this
    call continues (its kernels may then start while that call finishes; pass the two
    workspaces alternately).  Returns ``out``."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    dev = q.device
    ext = GdnPrefillExt()
    gate = None
    if gate_z is not None or gate_weight is not None:
        gate = _out_gate(gate_z, gate_weight, gate_eps, out, q.dtype)
        ext.gate = ctypes.cast(ctypes.pointer(gate), ctypes.c_void_p)
    if snap_every:
        n_snap = T // snap_every if snap_every > 0 else 0
        nb = snap_state.shape[0]
        _need(snap_state, "snap_state", (nb, Hv, HEAD_DIM, HEAD_DIM), torch.float32, dev)
        _need(snap_slots, "snap_slots", (B, n_snap), torch.int32, dev)
        if W > 1:
            _need(snap_conv_state, "snap_conv_state", (nb, W - 1, (2 * Hk + Hv) * HEAD_DIM),
                  q.dtype, dev)
        ext.snap_every = int(snap_every)
        ext.snap_state = _ptr(snap_state)
        ext.snap_conv_state = _ptr(snap_conv_state)
        ext.num_snap_slots = nb
        ext.snap_slots = _ptr(snap_slots)
    ext.prev_workspace = _ptr(prev_workspace)
    dims = GdnDims(B, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    need = int(L.gdn_prefill_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = L.gdn_chunk_prefill_ex(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k),
                                _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                _ptr(conv_weight), _ptr(conv_bias), _ptr(state),
                                _ptr(conv_state), _ptr(state_slots), _ptr(out),
                                ctypes.byref(ext), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_prefill_ex")
    return out


def gdn_prefill_varlen_workspace_size(num_seqs: int, total_tokens: int, num_k_heads: int,
                                      num_v_heads: int, conv_width: int,
                                      in_dtype=torch.bfloat16) -> int:
    L = load_library()
    dims = GdnDims(num_seqs, total_tokens, num_k_heads, num_v_heads, HEAD_DIM, 64, conv_width, 0)
    dt = GDN_BF16 if in_dtype == torch.bfloat16 else GDN_F32
    opts = _opts(dt, dt, 1, 1e-6, 1.0, 1, 0)
    return int(L.gdn_prefill_varlen_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))


def gdn_chunk_prefill_varlen(q, k, v, a, b, A_log, dt_bias, state, out, *, cu_seqlens,
                             num_k_heads=None, conv_weight=None, conv_bias=None,
                             conv_state=None, state_slots=None, gate_z=None, gate_weight=None,
                             gate_eps: float = 1e-6, scale: float = 1.0, eps: float = 1e-6,
                             qk_l2norm: bool = True, conv_silu: bool = True,
                             gates_precomputed: bool = False,
                             workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """Prefill of a packed variable-length batch (see gdn_chunk_prefill_varlen in
    include/gdn.h): every tensor has the layout of a one-sequence call over all T packed
    tokens ([1, T, ...]); sequence n is tokens cu_seqlens[n] .. cu_seqlens[n+1] - 1 and uses
    state row state_slots[n] (or n).  Optional gated output norm (gate_z shaped like out)."""
    L = load_library()
    _, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, None, None)
    if a.shape[0] != 1:
        raise ValueError("a packed batch has all its tokens in one row: a must be [1, T, Hv]")
    N = cu_seqlens.numel() - 1
    if N < 0:
        raise ValueError("cu_seqlens needs N + 1 >= 1 entries")
    _need(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, q.device)
    if state_slots is None and num_slots < N:
        raise ValueError("state has fewer rows than sequences and no state_slots given")
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 None, out, 1, T, Hk, Hv, W, num_slots, gates_precomputed)
    if state_slots is not None:
        _need(state_slots, "state_slots", (N,), torch.int32, q.device)
    gate = None
    if gate_z is not None:
        gate = _out_gate(gate_z, gate_weight, gate_eps, out, q.dtype)
    dims = GdnDims(N, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    need = int(L.gdn_prefill_varlen_workspace_size(ctypes.byref(dims), ctypes.byref(opts)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = L.gdn_chunk_prefill_varlen(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k),
                                    _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                    _ptr(conv_weight), _ptr(conv_bias), _ptr(state),
                                    _ptr(conv_state), _ptr(state_slots), _ptr(cu_seqlens),
                                    _ptr(out), None if gate is None else ctypes.byref(gate),
                                    _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_prefill_varlen")
    return out


def gdn_decode_multi(q, k, v, a, b, A_log, dt_bias, state, out, *, num_k_heads=None,
                     conv_weight=None, conv_bias=None, conv_state=None, state_slots=None,
                     snap_state=None, snap_conv_state=None, snap_slots=None,
                     scale: float = 1.0, eps: float = 1e-6, qk_l2norm: bool = True,
                     conv_silu: bool = True, gates_precomputed: bool = False,
                     stream=None) -> torch.Tensor:
    """A decode step over T <= 16 tokens per sequence (see gdn_decode_multi in
    include/gdn.h); inputs shaped as for gdn_chunk_prefill with seqlen T.  With snap_slots
    [B, T] the state (and conv state) after every token go to those rows of snap_state
    (snap_conv_state)."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    nb = 0
    if snap_slots is not None:
        dev = q.device
        nb = snap_state.shape[0]
        _need(snap_slots, "snap_slots", (B, T), torch.int32, dev)
        _need(snap_state, "snap_state", (nb, Hv, HEAD_DIM, HEAD_DIM), torch.float32, dev)
        if W > 1:
            _need(snap_conv_state, "snap_conv_state", (nb, W - 1, (2 * Hk + Hv) * HEAD_DIM),
                  q.dtype, dev)
    dims = GdnDims(B, T, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    st = L.gdn_decode_multi(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(v),
                            _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(conv_weight),
                            _ptr(conv_bias), _ptr(state), _ptr(conv_state), _ptr(state_slots),
                            _ptr(out), _ptr(snap_state), _ptr(snap_conv_state), nb,
                            _ptr(snap_slots), _stream(stream))
    _check(st, "gdn_decode_multi")
    return out


def gdn_decode_step_gated(q, k, v, a, b, A_log, dt_bias, state, out, *, gate_z, gate_weight,
                          gate_eps: float = 1e-6, num_k_heads=None, conv_weight=None,
                          conv_bias=None, conv_state=None, state_slots=None, scale: float = 1.0,
                          eps: float = 1e-6, qk_l2norm: bool = True, conv_silu: bool = True,
                          gates_precomputed: bool = False, stream=None) -> torch.Tensor:
    """gdn_decode_step with the gated RMS norm on the output (gate_z shaped like out)."""
    L = load_library()
    B, T, Hk, Hv, W, num_slots = _layer_dims(q, k, v, a, num_k_heads, conv_weight, conv_state,
                                             state, state_slots, None)
    if T != 1:
        raise ValueError("gdn_decode_step_gated takes exactly one token per sequence")
    _check_layer(q, k, v, a, b, A_log, dt_bias, conv_weight, conv_bias, state, conv_state,
                 state_slots, out, B, T, Hk, Hv, W, num_slots, gates_precomputed)
    gate = _out_gate(gate_z, gate_weight, gate_eps, out, q.dtype)
    dims = GdnDims(B, 1, Hk, Hv, HEAD_DIM, 64, W, num_slots)
    opts = _opts(_dt(q), _dt(out), qk_l2norm, eps, scale, conv_silu, gates_precomputed)
    st = L.gdn_decode_step_gated(ctypes.byref(dims), ctypes.byref(opts), _ptr(q), _ptr(k),
                                 _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
                                 _ptr(conv_weight), _ptr(conv_bias), _ptr(state),
                                 _ptr(conv_state), _ptr(state_slots), _ptr(out),
                                 ctypes.byref(gate), _stream(stream))
    _check(st, "gdn_decode_step_gated")
    return out


def causal_conv1d_update(x, weight, conv_state, y, *, bias=None, state_slots=None,
                         silu: bool = True, stream=None) -> torch.Tensor:
    """Standalone causal depthwise conv with carried state: x, y [B,T,C]; weight [C,W];
    conv_state [num_slots, W-1, C] updated in place."""
    L = load_library()
    B, T, C = x.shape
    W = weight.shape[1]
    dev, dt = x.device, x.dtype
    _need(x, "x", (B, T, C), dt, dev)
    _need(y, "y", (B, T, C), dt, dev)
    _need(weight, "weight", (C, W), dt, dev)
    if bias is not None:
        _need(bias, "bias", (C,), dt, dev)
    ns = conv_state.shape[0]
    _need(conv_state, "conv_state", (ns, W - 1, C), dt, dev)
    if state_slots is not None:
        _need(state_slots, "state_slots", (B,), torch.int32, dev)
    st = L.causal_conv1d_update(B, T, C, W, _dt(x), _ptr(x), _ptr(weight), _ptr(bias),
                                _ptr(conv_state), ns, _ptr(state_slots), int(silu), _ptr(y),
                                _stream(stream))
    _check(st, "causal_conv1d_update")
    return y


def gdn_state_checkpoint(op: str, state, conv_state, slot_state, slot_conv_state, rows, slots,
                         *, num_k_heads: int, stream=None) -> None:
    """op 'save' (live rows -> bank slots) or 'restore' (bank slots -> live rows)."""
    L = load_library()
    opc = {"save": 0, "restore": 1}[op]
    ns, Hv, d, _ = state.shape
    nb = slot_state.shape[0]
    dev = state.device
    _need(state, "state", (ns, Hv, d, d), torch.float32, dev)
    _need(slot_state, "slot_state", (nb, Hv, d, d), torch.float32, dev)
    W = 0
    cdt = GDN_BF16
    if conv_state is not None:
        W = conv_state.shape[1] + 1
        C = conv_state.shape[2]
        if C != (2 * num_k_heads + Hv) * d:
            raise ValueError("conv_state channels do not match the head geometry")
        _need(conv_state, "conv_state", (ns, W - 1, C), conv_state.dtype, dev)
        _need(slot_conv_state, "slot_conv_state", (nb, W - 1, C), conv_state.dtype, dev)
        cdt = _dt(conv_state)
    n = rows.shape[0]
    _need(rows, "rows", (n,), torch.int32, dev)
    _need(slots, "slots", (n,), torch.int32, dev)
    dims = GdnDims(ns, 1, num_k_heads, Hv, d, 64, W, ns)
    st = L.gdn_state_checkpoint(opc, ctypes.byref(dims), cdt, _ptr(state), _ptr(conv_state),
                                _ptr(slot_state), _ptr(slot_conv_state), nb, _ptr(rows),
                                _ptr(slots), n, _stream(stream))
    _check(st, "gdn_state_checkpoint")


# ---------------------------------------------------------------- full-attention layers

def _kv_cache(k_cache, v_cache, k_exp, v_exp):
    """(C struct, device) of a paged cache [num_pages, H, page_size, D]: bf16, or float8_e4m3fn
    codes with uint8 exponents [num_pages, H, page_size]."""
    dev, shape, dtype = k_cache.device, k_cache.shape, k_cache.dtype
    if (dtype is torch.float8_e4m3fn and len(shape) == 4 and v_cache is not None and
            k_exp is not None and v_exp is not None and v_cache.dtype is dtype and
            v_cache.shape == shape and k_exp.dtype is torch.uint8 and v_exp.dtype is torch.uint8 and
            k_exp.shape == v_exp.shape == shape[:3] and
            dev == v_cache.device == k_exp.device == v_exp.device and dev.type == "cuda" and
            k_cache.is_contiguous() and v_cache.is_contiguous() and k_exp.is_contiguous() and
            v_exp.is_contiguous()):                  # the usual case at once
        return GdnKvCache(shape[0], shape[2], shape[1], shape[3], GDN_KV_E4M3, k_cache.data_ptr(),
                          v_cache.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr()), dev
    if (dtype is torch.bfloat16 and len(shape) == 4 and v_cache is not None and k_exp is None and
            v_exp is None and v_cache.dtype is dtype and v_cache.shape == shape and
            dev == v_cache.device and dev.type == "cuda" and k_cache.is_contiguous() and
            v_cache.is_contiguous()):
        return GdnKvCache(shape[0], shape[2], shape[1], shape[3], GDN_KV_BF16, k_cache.data_ptr(),
                          v_cache.data_ptr(), None, None), dev
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if len(shape) != 4:
        raise ValueError(f"k_cache: shape {tuple(shape)}, expected 4 dimensions")
    f8 = dtype is torch.float8_e4m3fn
    if not f8 and dtype is not torch.bfloat16:
        raise TypeError(f"k_cache: dtype {dtype}, expected bfloat16 or float8_e4m3fn")
    _need(k_cache, "k_cache", shape, dtype, dev)
    _need(v_cache, "v_cache", shape, dtype, dev)
    pages, heads, page_size, d = shape
    if f8:
        _need(k_exp, "k_exp", shape[:3], torch.uint8, dev)
        _need(v_exp, "v_exp", shape[:3], torch.uint8, dev)
        return GdnKvCache(pages, page_size, heads, d, GDN_KV_E4M3, k_cache.data_ptr(),
                          v_cache.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr()), dev
    if k_exp is not None or v_exp is not None:
        raise ValueError("a bf16 cache has no exponents: k_exp and v_exp must be None")
    return GdnKvCache(pages, page_size, heads, d, GDN_KV_BF16, k_cache.data_ptr(),
                      v_cache.data_ptr(), None, None), dev


def _token_stride(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """The token stride (elements) of t [..., H, D], whose heads are dense and whose leading
    dimensions lie one token after the other."""
    H, D = shape[-2:]
    if t.shape == shape and t.dtype is dtype and t.device == device:
        if t.is_contiguous():
            return H * D
        strides = t.stride()
        if len(shape) == 3 and strides[2] == 1 and strides[1] == D and shape[0] > 1:
            return strides[0]                        # slices of wider rows
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    strides = t.stride()
    if (D > 1 and strides[-1] != 1) or (H > 1 and strides[-2] != D):
        raise ValueError(f"{name}: the last two dimensions must be dense")
    lead, stride = [(n, s) for n, s in zip(shape[:-2], strides) if n > 1], H * D
    if lead:
        stride = lead[-1][1]
        for (_, s), (n, inner) in zip(lead[:-1], lead[1:]):
            if s != n * inner:
                raise ValueError(f"{name}: tokens must lie at one stride")
    return stride


def gdn_kv_cache_append(k, v, k_cache, v_cache, slots, *, k_exp=None, v_exp=None,
                        stream=None) -> None:
    """Write n tokens' keys and values k, v [n, H, D] (bf16 or fp32; slices of wider rows are
    fine) to their ``slots`` [n] of the paged cache k_cache, v_cache [num_pages, H, page_size,
    D]: bf16, or float8_e4m3fn with k_exp, v_exp (see gdn_kv_cache_append in include/gdn.h)."""
    L = load_library()
    c, dev = _kv_cache(k_cache, v_cache, k_exp, v_exp)
    n = slots.shape[0]
    shape = (n, c.num_kv_heads, c.head_dim)
    _need(slots, "slots", (n,), torch.int32, dev)
    dt = _dt(k)
    ks = _token_stride(k, "k", shape, k.dtype, dev)
    vs = _token_stride(v, "v", shape, k.dtype, dev)
    st = L.gdn_kv_cache_append(ctypes.byref(c), n, dt, k.data_ptr(), ks, v.data_ptr(), vs,
                               slots.data_ptr(), _stream_of(stream, dev))
    _check(st, "gdn_kv_cache_append")


def gdn_kv_cache_read(k_cache, v_cache, slots, k_out, v_out, *, k_exp=None, v_exp=None,
                      stream=None):
    """Gather ``slots`` [n] of the cache into k_out, v_out [n, H, D] (bf16 or fp32); negative
    slots read as zeros.  Returns (k_out, v_out)."""
    L = load_library()
    c, dev = _kv_cache(k_cache, v_cache, k_exp, v_exp)
    n = slots.shape[0]
    _need(slots, "slots", (n,), torch.int32, dev)
    dt = _dt(k_out)
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        _need(t, name, (n, c.num_kv_heads, c.head_dim), k_out.dtype, dev)
    st = L.gdn_kv_cache_read(ctypes.byref(c), n, slots.data_ptr(), dt, k_out.data_ptr(),
                             v_out.data_ptr(), _stream_of(stream, dev))
    _check(st, "gdn_kv_cache_read")
    return k_out, v_out


def gdn_prefix_attention_workspace_size(batch: int, seqlen: int, num_heads: int,
                                        num_kv_heads: int, head_dim: int) -> int:
    return int(load_library().gdn_prefix_attention_workspace_size(batch, seqlen, num_heads,
                                                                  num_kv_heads, head_dim))


def gdn_prefix_attention(q, k_cache, v_cache, out, *, pages, kv_len, prefix_pages=None,
                         prefix_len: int = 0, k_exp=None, v_exp=None,
                         scale: Optional[float] = None, lse=None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of T new tokens of each of B sequences that share a prefix (see
    gdn_prefix_attention in include/gdn.h).  q [B, T, Hq, D] bf16, the cache as in
    gdn_kv_cache_append, prefix_pages [>= ceil(prefix_len / page_size)], pages [B, max_pages],
    kv_len [B] (own tokens, the T new ones included), out [B, T, Hq, D] bf16 or fp32, lse
    [B, T, Hq] fp32 or None; scale defaults to 1 / sqrt(D).  Returns ``out``."""
    L = load_library()
    c, dev = _kv_cache(k_cache, v_cache, k_exp, v_exp)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q: shape {tuple(shape)}, expected 4 dimensions")
    B, T, Hq, D = shape
    if D == c.head_dim and q.dtype is torch.bfloat16 and q.device == dev and q.is_contiguous():
        qs = Hq * D
    else:
        qs = _token_stride(q, "q", (B, T, Hq, c.head_dim), torch.bfloat16, dev)
    dt = _dt(out)
    _need(out, "out", shape, out.dtype, dev)
    i32 = torch.int32
    if pages.dim() != 2:
        raise ValueError(f"pages: shape {tuple(pages.shape)}, expected (B, max_pages)")
    max_pages = pages.shape[1]
    _need(pages, "pages", (B, max_pages), i32, dev)
    _need(kv_len, "kv_len", (B,), i32, dev)
    pp = None
    if prefix_len:
        if prefix_len < 0:
            raise ValueError("prefix_len must not be negative")
        if prefix_pages is None:
            raise ValueError("prefix_pages is required")
        n = prefix_pages.numel()
        _need(prefix_pages, "prefix_pages", (n,), i32, dev)
        if n * c.page_size < prefix_len:
            raise ValueError("prefix_pages holds fewer tokens than prefix_len")
        pp = prefix_pages.data_ptr()
    if lse is not None:
        _need(lse, "lse", shape[:3], torch.float32, dev)
    if workspace is None:
        need = int(L.gdn_prefix_attention_workspace_size(B, T, Hq, c.num_kv_heads, D))
        workspace = _workspace(need, dev, stream)
    st = L.gdn_prefix_attention(ctypes.byref(c), B, T, Hq, q.data_ptr(), qs, pp, prefix_len,
                                pages.data_ptr(), max_pages, kv_len.data_ptr(),
                                D ** -0.5 if scale is None else scale, dt, out.data_ptr(),
                                _ptr(lse), workspace.data_ptr(),
                                _workspace_bytes(workspace, dev), _stream_of(stream, dev))
    _check(st, "gdn_prefix_attention")
    return out


def gdn_token_logprobs_workspace_size(rows: int, vocab: int, top_k: int = 0,
                                      dtype=torch.bfloat16) -> int:
    dt = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(load_library().gdn_token_logprobs_workspace_size(rows, vocab, dt, top_k))


def gdn_token_logprobs(logits, targets, logprobs, entropy=None, *, top_ids=None,
                       top_logprobs=None, scale: float = 1.0,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Log probabilities of ``targets`` [N] (int32; negative: none, 0 is written) under logits
    [N, V] (bf16 or fp32, rows may be slices of wider ones), the rows' ``entropy`` [N] and, with
    top_ids int32 / top_logprobs fp32 [N, k], the k most likely tokens (see gdn_token_logprobs
    in include/gdn.h).  ``targets`` and ``logprobs`` may both be None."""
    L = load_library()
    if logits.dim() != 2:
        raise ValueError(f"logits: shape {tuple(logits.shape)}, expected (N, V)")
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    N, V = logits.shape
    dt = _dt(logits)
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits: rows must be dense")
    if (targets is None) != (logprobs is None):
        raise ValueError("targets and logprobs go together")
    if targets is not None:
        _need(targets, "targets", (N,), torch.int32, dev)
        _need(logprobs, "logprobs", (N,), torch.float32, dev)
    if entropy is not None:
        _need(entropy, "entropy", (N,), torch.float32, dev)
    k = 0
    if top_ids is not None or top_logprobs is not None:
        if top_ids is None or top_logprobs is None:
            raise ValueError("top_ids and top_logprobs go together")
        k = top_ids.shape[1] if top_ids.dim() == 2 else -1
        _need(top_ids, "top_ids", (N, k), torch.int32, dev)
        _need(top_logprobs, "top_logprobs", (N, k), torch.float32, dev)
    if workspace is None:
        need = int(L.gdn_token_logprobs_workspace_size(N, V, dt, k))
        if need:
            workspace = _workspace(need, dev, stream)
    ws_bytes = 0 if workspace is None else _workspace_bytes(workspace, dev)
    st = L.gdn_token_logprobs(N, V, dt, _ptr(logits), logits.stride(0) if N > 1 else V,
                              _ptr(targets), float(scale), _ptr(logprobs), _ptr(entropy), k,
                              _ptr(top_ids), _ptr(top_logprobs), _ptr(workspace), ws_bytes,
                              _stream_of(stream, dev))
    _check(st, "gdn_token_logprobs")


def gdn_rope_phase_steps(rotary_dim: int, base: float = 10000.0, *,
                         scaling: Optional[str] = None, factor: float = 1.0,
                         original_context: float = 0.0, beta_fast: float = 32.0,
                         beta_slow: float = 1.0, device="cuda"):
    """(phase steps, amplitude) of a rotation for gdn_qk_norm_rope: int64 [rotary_dim / 2] on
    ``device`` (the bits of the 64-bit steps) and a float.  ``scaling``: None, "linear", "ntk" or
    "yarn" (see gdn_rope_phase_steps in include/gdn.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling: {scaling!r}, expected one of {list(ROPE_SCALINGS)}")
    steps = (ctypes.c_uint64 * max(1, rotary_dim // 2))()
    amplitude = ctypes.c_float()
    st = load_library().gdn_rope_phase_steps(rotary_dim, base, ROPE_SCALINGS[scaling], factor,
                                             original_context, beta_fast, beta_slow, steps,
                                             ctypes.byref(amplitude))
    _check(st, "gdn_rope_phase_steps")
    signed = [x - (1 << 64) if x >> 63 else x for x in steps][:rotary_dim // 2]
    return torch.tensor(signed, dtype=torch.int64, device=device), amplitude.value


def _head_strides(t: torch.Tensor, name: str, shape):
    """The token and head strides (elements) of t [n, H, D] with dense vectors."""
    n, H, D = shape
    token, head, element = t.stride()
    if element != 1 and D > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    if H == 1:
        head = D
    return token if n > 1 else (H - 1) * head + D, head


def gdn_qk_norm_rope(q, k, positions, phase_steps, q_out, k_out=None, *, q_weight=None,
                     k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                     amplitude: float = 1.0, v=None, k_cache=None, v_cache=None, slots=None,
                     k_exp=None, v_exp=None, stream=None) -> None:
    """RMS norm of query and key heads q [n, Hq, D], k [n, H, D] (bf16 or fp32; q's heads may lie
    apart, tokens too), rotated by their ``positions`` [n] (int32; see gdn_qk_norm_rope in
    include/gdn.h) into q_out [n, Hq, D] and k_out [n, H, D].  ``phase_steps`` int64
    [rotary_dim / 2] and ``amplitude`` come from gdn_rope_phase_steps; None turns nothing.  With a
    cache (as in gdn_kv_cache_append) the keys and the values v [n, H, D] go to ``slots`` [n], and
    k_out may be None."""
    L = _lib or load_library()
    st = _native.qk_norm_rope(q, k, positions, phase_steps, q_out, k_out, q_weight, k_weight, eps,
                              interleaved, amplitude, v, k_cache, v_cache, slots, k_exp, v_exp,
                              None if stream is None else _stream(stream))
    if st is not None:
        return _check(st, "gdn_qk_norm_rope")
    # anything unusual, with what is wrong
    dev, dtype, shape, kshape = q.device, q.dtype, q.shape, k.shape
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if len(shape) != 3 or len(kshape) != 3:
        raise ValueError("q and k must have 3 dimensions: tokens, heads, elements")
    dt = _dt(q)
    n, Hq, D = shape
    H = kshape[1]
    qs, qh = _head_strides(q, "q", shape)
    kshape = (n, H, D)
    ks = _token_stride(k, "k", kshape, dtype, dev)
    if (q_out.shape == shape and q_out.dtype is dtype and q_out.device == dev and
            q_out.is_contiguous()):
        qo = Hq * D
    else:
        qo = _token_stride(q_out, "q_out", shape, dtype, dev)
    r, pp, sp = 0, None, None
    if phase_steps is not None:
        r = 2 * phase_steps.numel()
        _need(phase_steps, "phase_steps", (r // 2,), torch.int64, dev)
        _need(positions, "positions", (n,), torch.int32, dev)
        if r:
            pp, sp = positions.data_ptr(), phase_steps.data_ptr()
    qw = kw = ko = None
    if q_weight is not None:
        _need(q_weight, "q_weight", (D,), torch.float32, dev)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _need(k_weight, "k_weight", (D,), torch.float32, dev)
        kw = k_weight.data_ptr()
    if k_out is not None:
        _need(k_out, "k_out", kshape, dtype, dev)
        ko = k_out.data_ptr()
    cache, vp, vs, slot = None, None, 0, None
    if k_cache is not None:
        c, cdev = _kv_cache(k_cache, v_cache, k_exp, v_exp)
        if cdev != dev:
            raise ValueError(f"k_cache: on {cdev}, expected {dev}")
        if v is None:
            raise ValueError("v is required")
        vs = _token_stride(v, "v", kshape, dtype, dev)
        _need(slots, "slots", (n,), torch.int32, dev)
        cache, vp, slot = ctypes.byref(c), v.data_ptr(), slots.data_ptr()
    elif ko is None:
        raise ValueError("k_out or a cache is required")
    elif v is not None or slots is not None or v_cache is not None:
        raise ValueError("v, v_cache and slots go with k_cache")
    rope = GdnRope(r, GDN_ROPE_INTERLEAVED if interleaved else GDN_ROPE_HALF, amplitude, sp)
    st = L.gdn_qk_norm_rope(n, Hq, H, D, dt, q.data_ptr(), qs, qh, k.data_ptr(), ks, qw, kw, eps,
                            pp, ctypes.byref(rope), q_out.data_ptr(), qo, ko, cache, vp, vs, slot,
                            _stream_of(stream, dev))
    if st:
        _check(st, "gdn_qk_norm_rope")


def _page_pool(table, held, free_pages, free_count, page_size):
    """(C struct, device) of a pool: table [num_rows, max_pages], held [num_rows], free_pages
    [num_pages], free_count [1], all int32."""
    dev, i32, tshape, fshape = table.device, torch.int32, table.shape, free_pages.shape
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if len(tshape) != 2 or len(fshape) != 1:
        raise ValueError("table must have 2 dimensions and free_pages 1")
    rows, columns = tshape
    pages = fshape[0]
    if (held.shape == (rows,) and free_count.shape == (1,) and
            i32 is table.dtype is held.dtype is free_pages.dtype is free_count.dtype and
            dev == held.device == free_pages.device == free_count.device and
            table.is_contiguous() and held.is_contiguous() and free_pages.is_contiguous()):
        return GdnPagePool(pages, page_size, rows, columns, table.data_ptr(), held.data_ptr(),
                           free_pages.data_ptr(), free_count.data_ptr()), dev
    _need(table, "table", (rows, columns), i32, dev)
    _need(held, "held", (rows,), i32, dev)
    _need(free_pages, "free_pages", (pages,), i32, dev)
    _need(free_count, "free_count", (1,), i32, dev)
    return GdnPagePool(pages, page_size, rows, columns, table.data_ptr(), held.data_ptr(),
                       free_pages.data_ptr(), free_count.data_ptr()), dev


def gdn_page_plan(kv_len, new_len, slots=None, positions=None, cu_seqlens=None, kv_len_out=None,
                  pages=None, *, table, held, free_pages, free_count, page_size: int, rows=None,
                  position_offset: int = 0, stream=None) -> None:
    """Pages, ``slots`` and ``positions`` [capacity] for new_len [B] more tokens of each of B
    requests that have kv_len [B] (see gdn_page_plan in include/gdn.h).  The pool (table
    [num_rows, max_pages], held [num_rows], free_pages [num_pages], free_count [1]; int32) is
    updated in place; cu_seqlens [B + 1], kv_len_out [B] and the block tables ``pages``
    [B, max_pages] are written where given.  Request b is row rows[b] (or b) of the pool."""
    L = _lib or load_library()
    st = _native.page_plan(kv_len, new_len, slots, positions, cu_seqlens, kv_len_out, pages, table,
                           held, free_pages, free_count, page_size, rows, position_offset,
                           None if stream is None else _stream(stream))
    if st is not None:
        return _check(st, "gdn_page_plan")
    # anything unusual, with what is wrong
    p, dev = _page_pool(table, held, free_pages, free_count, page_size)
    i32 = torch.int32
    shape = kv_len.shape
    B = shape[0]
    if rows is None and B > p.num_rows:
        raise ValueError("the pool has fewer rows than the batch and no rows given")
    if not (len(shape) == 1 and new_len.shape == shape and i32 is kv_len.dtype is new_len.dtype and
            dev == kv_len.device == new_len.device and kv_len.is_contiguous() and
            new_len.is_contiguous()):
        _need(kv_len, "kv_len", (B,), i32, dev)
        _need(new_len, "new_len", (B,), i32, dev)
    capacity = 0x7fffffff                            # (nothing to be written a token)
    sp = pp = rp = cp = op = tp = None
    if slots is not None:
        capacity = slots.shape[0]
        _need(slots, "slots", (capacity,), i32, dev)
        sp = slots.data_ptr()
    if positions is not None:
        if slots is None:
            capacity = positions.shape[0]
        _need(positions, "positions", (capacity,), i32, dev)
        pp = positions.data_ptr()
    if rows is not None:
        _need(rows, "rows", shape, i32, dev)
        rp = rows.data_ptr()
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", (B + 1,), i32, dev)
        cp = cu_seqlens.data_ptr()
    if kv_len_out is not None:
        _need(kv_len_out, "kv_len_out", shape, i32, dev)
        op = kv_len_out.data_ptr()
    if pages is not None:
        _need(pages, "pages", (B, p.max_pages), i32, dev)
        tp = pages.data_ptr()
    st = L.gdn_page_plan(ctypes.byref(p), B, rp, kv_len.data_ptr(), new_len.data_ptr(), capacity,
                         position_offset, sp, pp, cp, op, tp, _stream_of(stream, dev))
    if st:
        _check(st, "gdn_page_plan")


def gdn_page_release(keep_len, *, table, held, free_pages, free_count, page_size: int, rows=None,
                     stream=None) -> None:
    """Requests keep the pages of their first keep_len [B] tokens and give the others back (see
    gdn_page_release in include/gdn.h); the pool as in gdn_page_plan."""
    L = _lib or load_library()
    st = _native.page_release(keep_len, table, held, free_pages, free_count, page_size, rows,
                              None if stream is None else _stream(stream))
    if st is not None:
        return _check(st, "gdn_page_release")
    # anything unusual, with what is wrong
    p, dev = _page_pool(table, held, free_pages, free_count, page_size)
    B = keep_len.shape[0]
    if rows is None and B > p.num_rows:
        raise ValueError("the pool has fewer rows than the batch and no rows given")
    _need(keep_len, "keep_len", (B,), torch.int32, dev)
    rp = None
    if rows is not None:
        _need(rows, "rows", (B,), torch.int32, dev)
        rp = rows.data_ptr()
    st = L.gdn_page_release(ctypes.byref(p), B, rp, keep_len.data_ptr(), _stream_of(stream, dev))
    if st:
        _check(st, "gdn_page_release")


def gdn_verify_tokens_workspace_size(batch: int, num_drafts: int, vocab: int,
                                     dtype=torch.bfloat16, draft_logits: bool = True) -> int:
    dt = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(load_library().gdn_verify_tokens_workspace_size(batch, num_drafts, vocab, dt,
                                                               int(draft_logits)))


def _row_stride(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """The row stride (elements) of t [B, T, V]: rows dense, one after the other."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return shape[2]
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    B, T, V = shape
    outer, row, element = t.stride()
    if V > 1 and element != 1:
        raise ValueError(f"{name}: rows must be dense")
    if T == 1:
        return outer if B > 1 else V
    if B > 1 and outer != T * row:
        raise ValueError(f"{name}: rows must lie at one stride")
    return row


def gdn_verify_tokens(target_logits, tokens, accepted, *, clocks, draft_ids=None,
                      draft_logits=None, accept_u=None, scale=None, logprobs=None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Verify T drafted tokens ``draft_ids`` [B, T] (int32; negative ones end a row) of each of B
    sequences under target_logits [B, T + 1, V] (bf16 or fp32) and draft_logits [B, T, V] (or
    None: the drafts have no distribution), from uniform ``accept_u`` [B, T] and exponential
    ``clocks`` [B, V] numbers; ``scale`` [B] fp32 inverse temperatures (inf: greedy; negative: left
    out) or None.  Writes tokens [B, T + 1] (int32: the accepted drafts, the token behind them,
    then -1), accepted [B] (int32) and logprobs [B, T + 1] (fp32) or None.  T = 0 draws one token
    a sequence.  See gdn_verify_tokens in include/gdn.h."""
    L = _lib or load_library()
    if workspace is not None:
        st = _native.verify_tokens(target_logits, tokens, accepted, clocks, draft_ids, draft_logits,
                                   accept_u, scale, logprobs, workspace,
                                   None if stream is None else _stream(stream))
        if st is not None:
            return _check(st, "gdn_verify_tokens")
    # a workspace to be made, or anything unusual, with what is wrong
    if target_logits.dim() != 3:
        raise ValueError(f"target_logits: shape {tuple(target_logits.shape)}, expected (B, T + 1, V)")
    dev = target_logits.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    B, T1, V = target_logits.shape
    T = T1 - 1
    dtype, f32 = target_logits.dtype, torch.float32
    dt = _dt(target_logits)
    ts = _row_stride(target_logits, "target_logits", (B, T1, V), dtype, dev)
    ds = 0
    if T > 0:
        _need(draft_ids, "draft_ids", (B, T), torch.int32, dev)
        _need(accept_u, "accept_u", (B, T), f32, dev)
        if draft_logits is not None:
            ds = _row_stride(draft_logits, "draft_logits", (B, T, V), dtype, dev)
    elif draft_ids is not None or draft_logits is not None or accept_u is not None:
        raise ValueError("one row a sequence has no drafts: draft_ids, draft_logits and accept_u "
                         "must be None")
    _need(clocks, "clocks", (B, V), f32, dev)
    if scale is not None:
        _need(scale, "scale", (B,), f32, dev)
    _need(tokens, "tokens", (B, T1), torch.int32, dev)
    _need(accepted, "accepted", (B,), torch.int32, dev)
    if logprobs is not None:
        _need(logprobs, "logprobs", (B, T1), f32, dev)
    if workspace is None:
        need = int(L.gdn_verify_tokens_workspace_size(B, T, V, dt, int(draft_logits is not None)))
        workspace = _workspace(need, dev, stream)
    st = L.gdn_verify_tokens(B, T, V, dt, target_logits.data_ptr(), ts, _ptr(draft_ids),
                             _ptr(draft_logits), ds, _ptr(accept_u), clocks.data_ptr(),
                             _ptr(scale), tokens.data_ptr(), accepted.data_ptr(), _ptr(logprobs),
                             workspace.data_ptr(), _workspace_bytes(workspace, dev),
                             _stream_of(stream, dev))
    _check(st, "gdn_verify_tokens")


def gdn_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status code."""
    return int(load_library().gdn_get_device_error(_stream(stream)))


def gdn_selftest_device_timeout(max_iters: int = 1024, stream=None) -> None:
    """Enqueue the bounded-wait self-test (a wait that nothing ends, on no copy or MMA): the
    next gdn_get_device_error() returns GDN_ERR_DEVICE_TIMEOUT."""
    st = load_library().gdn_selftest_device_timeout(int(max_iters), _stream(stream))
    _check(st, "gdn_selftest_device_timeout")


def gdn_status_string(status: int) -> str:
    return load_library().gdn_status_string(int(status)).decode()
