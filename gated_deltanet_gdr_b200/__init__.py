"""B200 (sm_100a) gated delta rule: Python binding of libgdr.so.

The functions here only check and marshal arguments (torch tensors to device
pointers and sizes) and call the C ABI declared in ``include/gdr.h``; every
step of the computation runs in the library's CUDA kernels.  PyTorch supplies
device memory and streams.  If the compiled library is missing, importing the
binding's functions raises: there is no fallback.

    out, final_state = chunk_fwd(q, k, v, beta, g, initial_state, actual_seq_lengths, scale)
    out, state_pool  = recurrent_step(q, k, v, beta, g, gk, state_pool, ssm_state_indices,
                                      actual_seq_lengths, num_accepted_tokens, scale)

Beside the rule: the causal conv1d before it (``conv1d``, ``conv1d_bwd``), the gated linear recurrence with one scalar
state per channel (``scan_fwd``, ``scan_bwd``, ``scan_step``), and the slots of the state pools (``slot_copy``,
``slot_fork``, ``slot_compact``, ``slot_free``).

Layouts are BNSD: q, k (B, Nk, S, Dk); v (B, Nv, S, Dv); beta, g (B, Nv, S).
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr.so")

GDR_OK, GDR_ERR_SHAPE, GDR_ERR_DTYPE, GDR_ERR_NULL, GDR_ERR_ALIGN, GDR_ERR_UNSUPPORTED, GDR_ERR_DEVICE, \
    GDR_ERR_LAUNCH, GDR_ERR_WORKSPACE = range(9)
GDR_F32, GDR_BF16, GDR_F16 = 0, 1, 2
DEVERR_SLOT_INDEX, DEVERR_LENGTH, DEVERR_TIMEOUT = 0x1, 0x2, 0x4

# Every symbol the C header declares (checked by the ABI test).
EXPORTED = ("gdr_chunk_fwd_workspace", "gdr_chunk_fwd", "gdr_chunk_fwd_noalloc", "gdr_recurrent_step", "gdr_recurrent_step_spec", "gdr_conv1d",
            "gdr_conv1d_bwd", "gdr_conv1d_bwd_workspace", "gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step",
            "gdr_slot_copy", "gdr_slot_fork", "gdr_slot_compact", "gdr_slot_free",
            "gdr_prologue_apply", "gdr_get_error", "gdr_debug_set_wait_limit", "gdr_debug_timeout_site",
            "gdr_debug_set_chunk_schedule",
            "gdr_status_string", "gdr_version")


class GdrPrologueStruct(ctypes.Structure):
    _fields_ = [("l2norm_qk", ctypes.c_int), ("eps", ctypes.c_float), ("beta_logits", ctypes.c_int),
                ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class GdrPoolStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("slot_bytes", ctypes.c_size_t)]


class GdrEpilogueStruct(ctypes.Structure):
    _fields_ = [("z", ctypes.c_void_p), ("norm_w", ctypes.c_void_p), ("eps", ctypes.c_float)]


_lib = None
_quick = None  # the compiled marshalling of the short calls, once the library is loaded (see below)
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load libgdr.so (built in-tree by ``python -m gated_deltanet_gdr_b200.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgdr.so is not built ({LIB_PATH} missing); run "
                               "`python -m gated_deltanet_gdr_b200.build` -- there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.gdr_chunk_fwd_workspace.restype = ctypes.c_size_t
        L.gdr_chunk_fwd_workspace.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        L.gdr_chunk_fwd.restype = i32
        L.gdr_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, i32, i32,
                                    ctypes.POINTER(GdrPrologueStruct), ctypes.POINTER(GdrEpilogueStruct), vp, vp, vp,
                                    ctypes.c_size_t, vp]
        L.gdr_chunk_fwd_noalloc.restype = i32
        L.gdr_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, i32, i32,
                                            ctypes.POINTER(GdrPrologueStruct), ctypes.POINTER(GdrEpilogueStruct),
                                            vp, vp, vp]
        L.gdr_recurrent_step.restype = i32
        L.gdr_recurrent_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, f32, i32, i32, i32, i32, i32,
                                         i32, i32, i32, ctypes.POINTER(GdrPrologueStruct),
                                         ctypes.POINTER(GdrEpilogueStruct), vp, vp]
        L.gdr_recurrent_step_spec.restype = i32
        L.gdr_recurrent_step_spec.argtypes = L.gdr_recurrent_step.argtypes
        L.gdr_conv1d.restype = i32
        L.gdr_conv1d.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]
        L.gdr_conv1d_bwd.restype = i32
        L.gdr_conv1d_bwd.argtypes = [vp] * 9 + [i32] * 8 + [vp] * 5 + [ctypes.c_size_t, vp]
        L.gdr_conv1d_bwd_workspace.restype = ctypes.c_size_t
        L.gdr_conv1d_bwd_workspace.argtypes = [i32] * 7
        L.gdr_scan_fwd.restype = i32
        L.gdr_scan_fwd.argtypes = [vp] * 4 + [i32] * 7 + [vp] * 4
        L.gdr_scan_bwd.restype = i32
        L.gdr_scan_bwd.argtypes = [vp] * 6 + [i32] * 7 + [vp] * 4
        L.gdr_scan_step.restype = i32
        L.gdr_scan_step.argtypes = [vp, vp, vp, i32, vp, vp, vp] + [i32] * 8 + [vp, vp]
        pools = ctypes.POINTER(GdrPoolStruct)
        L.gdr_slot_copy.restype = i32
        L.gdr_slot_copy.argtypes = [pools, i32, i32, vp, vp, i32, vp]
        L.gdr_slot_fork.restype = i32
        L.gdr_slot_fork.argtypes = [pools, i32, i32, vp, vp, i32, vp, vp]
        L.gdr_slot_compact.restype = i32
        L.gdr_slot_compact.argtypes = [pools, i32, i32, vp, vp, vp, vp]
        L.gdr_slot_free.restype = i32
        L.gdr_slot_free.argtypes = [pools, i32, i32, vp, i32, vp, vp]
        L.gdr_prologue_apply.restype = i32
        L.gdr_prologue_apply.argtypes = [vp, vp, vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                         vp]
        L.gdr_get_error.restype = i32
        L.gdr_get_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
        L.gdr_debug_set_wait_limit.restype = i32
        L.gdr_debug_set_wait_limit.argtypes = [ctypes.c_ulonglong]
        L.gdr_debug_timeout_site.restype = i32
        L.gdr_debug_timeout_site.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.gdr_debug_set_chunk_schedule.restype = i32
        L.gdr_debug_set_chunk_schedule.argtypes = [i32]
        L.gdr_status_string.restype = ctypes.c_char_p
        L.gdr_status_string.argtypes = [i32]
        L.gdr_version.restype = i32
        L.gdr_version.argtypes = []
        _load_marshal(L)
        _lib = L
        return L


def _load_marshal(L) -> None:
    """Loads the extension _marshal and gives it the addresses of the C entries.  Without it, or with another torch than
    it was compiled against (whose tensors may be laid out differently), the short calls are marshalled in Python: the
    same checks and the same kernels, some microseconds later."""
    global _quick
    try:
        from . import _marshal as m
    except ImportError:
        return
    if m.torch_version != torch.__version__:
        return
    entries = ("gdr_scan_fwd", "gdr_scan_bwd", "gdr_scan_step", "gdr_conv1d_bwd", "gdr_conv1d_bwd_workspace",
               "gdr_slot_copy", "gdr_slot_fork", "gdr_slot_compact", "gdr_slot_free")
    m.bind(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in entries))
    _quick = m


@dataclass
class Prologue:
    """Fused pre-processing (see ``gdr_prologue`` in include/gdr.h): l2norm of raw
    q/k with eps inside the sqrt, beta from logits, g from raw a via A_log/dt_bias."""
    l2norm_qk: bool = True
    eps: float = 1e-6
    beta_logits: bool = True
    A_log: Optional[torch.Tensor] = None
    dt_bias: Optional[torch.Tensor] = None

    def as_struct(self) -> GdrPrologueStruct:
        return GdrPrologueStruct(int(self.l2norm_qk), float(self.eps), int(self.beta_logits), _ptr(self.A_log),
                                 _ptr(self.dt_bias))


@dataclass
class Epilogue:
    """Fused output epilogue (see ``gdr_epilogue`` in include/gdr.h): each valid out row o
    becomes o / sqrt(mean(o^2) + eps) * norm_w * silu(z) (the layer's gated RMSNorm)."""
    z: torch.Tensor  # (B, Nv, S, Dv), the dtype of q
    norm_w: torch.Tensor  # (Dv,) fp32
    eps: float = 1e-6

    def as_struct(self) -> GdrEpilogueStruct:
        return GdrEpilogueStruct(_ptr(self.z), _ptr(self.norm_w), float(self.eps))


def _check_epilogue(epi, B, Nv, S, Dv, dt):
    if epi is None:
        return None
    _dev(epi.z, "epilogue.z", dt, (B, Nv, S, Dv))
    _dev(epi.norm_w, "epilogue.norm_w", torch.float32, (Dv,))
    return epi.as_struct()


def _check(status: int, what: str):
    if status == GDR_OK:
        return
    msg = f"{what}: {lib().gdr_status_string(status).decode()} (status {status})"
    if status == GDR_ERR_SHAPE:
        raise ValueError(msg)
    raise RuntimeError(msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return GDR_F32
    if dt == torch.bfloat16:
        return GDR_BF16
    if dt == torch.float16:
        return GDR_F16
    raise RuntimeError(f"unsupported dtype {dt}; use torch.float32, torch.bfloat16 or torch.float16")


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise RuntimeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index != cur:  # the kernels run on the current device and would read this pointer there
        raise RuntimeError(f"{name} is on {t.device}, but the call runs on the current device cuda:{cur}")
    if dtype is not None and t.dtype != dtype:
        raise RuntimeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")
    return t


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    if s.device.index != torch.cuda.current_device():
        raise RuntimeError(f"the stream is on {s.device}, but the call runs on the current device "
                           f"cuda:{torch.cuda.current_device()}")
    return ctypes.c_void_p(s.cuda_stream)


def _chunk_checked(q, k, v, beta, g, initial_state, actual_seq_lengths, prologue, out, final_state,
                   output_final_state):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be (B, Nk, S, Dk) and v (B, Nv, S, Dv)")
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    dt = q.dtype
    _dtype_code(dt)
    _dev(q, "q", dt)
    _dev(k, "k", dt, (B, Nk, S, Dk))
    _dev(v, "v", dt, (B, Nv, S, Dv))
    _dev(beta, "beta", dt, (B, Nv, S))
    _dev(g, "g", torch.float32, (B, Nv, S))
    _dev(initial_state, "initial_state", dt, (B, Nv, Dk, Dv))
    _dev(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Nv, S, Dv), dtype=dt, device=q.device)
    _dev(out, "out", dt, (B, Nv, S, Dv))
    if output_final_state and final_state is None:
        final_state = torch.empty((B, Nv, Dk, Dv), dtype=dt, device=q.device)
    _dev(final_state, "final_state", dt, (B, Nv, Dk, Dv))
    if prologue is not None:
        _dev(prologue.A_log, "A_log", torch.float32, (Nv,))
        _dev(prologue.dt_bias, "dt_bias", torch.float32, (Nv,))
    return out, final_state


def chunk_fwd_workspace_bytes(B: int, Nk: int, Nv: int, S: int, Dk: int, Dv: int, dtype: torch.dtype) -> int:
    """Bytes of workspace the fastest schedule of ``gdr_chunk_fwd`` wants for these sizes
    (``gdr_chunk_fwd_workspace``; 0 when it wants none)."""
    return int(lib().gdr_chunk_fwd_workspace(B, Nk, Nv, S, Dk, Dv, _dtype_code(dtype)))


def _workspace(q, v, workspace):
    """The caller's workspace (a CUDA uint8 tensor), or a new one of the size the call needs."""
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    need = chunk_fwd_workspace_bytes(B, Nk, Nv, S, Dk, Dv, q.dtype)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _dev(workspace, "workspace", torch.uint8)
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; the call needs {need}")
    return workspace


def chunk_fwd(q, k, v, beta, g=None, initial_state=None, actual_seq_lengths=None, scale: float = 1.0, *,
              prologue: Optional[Prologue] = None, epilogue: Optional[Epilogue] = None, out=None, final_state=None,
              output_final_state: bool = True, workspace=None, stream=None):
    """Chunked prefill (``gdr_chunk_fwd``).  Returns (out, final_state or None).  ``workspace`` (uint8, at least
    ``chunk_fwd_workspace_bytes`` bytes) is allocated per call when not given and the sizes ask for one."""
    out, final_state = _chunk_checked(q, k, v, beta, g, initial_state, actual_seq_lengths, prologue, out,
                                      final_state, output_final_state)
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    pro = prologue.as_struct() if prologue is not None else None
    epi = _check_epilogue(epilogue, B, Nv, S, Dv, q.dtype)
    ws = _workspace(q, v, workspace)
    st = lib().gdr_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(initial_state),
                             _ptr(actual_seq_lengths), float(scale), B, Nk, Nv, S, Dk, Dv, _dtype_code(q.dtype),
                             ctypes.byref(pro) if pro is not None else None,
                             ctypes.byref(epi) if epi is not None else None, _ptr(out), _ptr(final_state),
                             _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    _check(st, "gdr_chunk_fwd")
    return out, final_state


def _decode_checked(q, k, v, beta, g, gk, state_pool, ssm_state_indices, actual_seq_lengths, num_accepted_tokens,
                    out):
    if q.dim() != 4 or v.dim() != 4 or state_pool.dim() != 4:
        raise ValueError("q, k (B, Nk, S, Dk), v (B, Nv, S, Dv), state_pool (slots, Nv, Dk, Dv)")
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    dt = q.dtype
    _dtype_code(dt)
    _dtype_code(state_pool.dtype)
    _dev(q, "q", dt)
    _dev(k, "k", dt, (B, Nk, S, Dk))
    _dev(v, "v", dt, (B, Nv, S, Dv))
    _dev(beta, "beta", dt, (B, Nv, S))
    _dev(g, "g", torch.float32, (B, Nv, S))
    _dev(gk, "gk", torch.float32, (B, Nv, S, Dk))
    _dev(state_pool, "state_pool", state_pool.dtype, (state_pool.shape[0], Nv, Dk, Dv))
    if ssm_state_indices is None or ssm_state_indices.numel() != B * S:
        raise ValueError("ssm_state_indices must hold B * S int32 slot indices, one per flattened token")
    _dev(ssm_state_indices.reshape(-1), "ssm_state_indices", torch.int32)
    _dev(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,))
    _dev(num_accepted_tokens, "num_accepted_tokens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Nv, S, Dv), dtype=dt, device=q.device)
    _dev(out, "out", dt, (B, Nv, S, Dv))
    return out


def recurrent_step(q, k, v, beta, g, gk, state_pool, ssm_state_indices, actual_seq_lengths,
                   num_accepted_tokens=None, scale: float = 1.0, *, prologue: Optional[Prologue] = None,
                   epilogue: Optional[Epilogue] = None, out=None, per_token: bool = False, stream=None):
    """Recurrent decode over a slot pool (``gdr_recurrent_step``), updating
    ``state_pool`` in place.  Returns (out, state_pool).  ``per_token=True`` calls
    ``gdr_recurrent_step_spec`` (speculative decoding: start from the slot of token
    A - 1, every token's state to its own slot)."""
    out = _decode_checked(q, k, v, beta, g, gk, state_pool, ssm_state_indices, actual_seq_lengths,
                          num_accepted_tokens, out)
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    pro = prologue.as_struct() if prologue is not None else None
    epi = _check_epilogue(epilogue, B, Nv, S, Dv, q.dtype)
    fn = lib().gdr_recurrent_step_spec if per_token else lib().gdr_recurrent_step
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(gk), _ptr(state_pool),
                                  int(state_pool.shape[0]), _ptr(ssm_state_indices), _ptr(actual_seq_lengths),
                                  _ptr(num_accepted_tokens), float(scale), B, Nk, Nv, S, Dk, Dv,
                                  _dtype_code(q.dtype), _dtype_code(state_pool.dtype),
                                  ctypes.byref(pro) if pro is not None else None,
                                  ctypes.byref(epi) if epi is not None else None, _ptr(out), _stream(stream))
    _check(st, "gdr_recurrent_step_spec" if per_token else "gdr_recurrent_step")
    return out, state_pool


class PreparedCall:
    """A C-ABI call with its arguments checked and marshalled once.

    Calling the object launches the library's kernels again on the same buffers
    (which the caller keeps alive and may refill in place) with no Python-side
    argument work, for serving loops and for timing the kernels alone.  Raises
    like the one-shot functions if the library reports an error.
    """

    def __init__(self, fn, args, what, result):
        self._fn, self._args, self._what, self.result = fn, args, what, result

    def __call__(self):
        st = self._fn(*self._args)
        if st != GDR_OK:
            _check(st, self._what)
        return self.result


def prepare_chunk_fwd(q, k, v, beta, g=None, initial_state=None, actual_seq_lengths=None, scale: float = 1.0, *,
                      prologue: Optional[Prologue] = None, epilogue: Optional[Epilogue] = None, out=None,
                      final_state=None, workspace=None, stream=None) -> PreparedCall:
    """Check and marshal a gdr_chunk_fwd call once; see chunk_fwd for the arguments (the workspace, if not given,
    is allocated once here and kept by the prepared call)."""
    out, final_state = _chunk_checked(q, k, v, beta, g, initial_state, actual_seq_lengths, prologue, out,
                                      final_state, True)
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    pro = prologue.as_struct() if prologue is not None else None
    epi = _check_epilogue(epilogue, B, Nv, S, Dv, q.dtype)
    ws = _workspace(q, v, workspace)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(initial_state), _ptr(actual_seq_lengths),
            ctypes.c_float(scale), B, Nk, Nv, S, Dk, Dv, _dtype_code(q.dtype),
            ctypes.pointer(pro) if pro is not None else None, ctypes.pointer(epi) if epi is not None else None,
            _ptr(out), _ptr(final_state), _ptr(ws), ctypes.c_size_t(0 if ws is None else ws.numel()),
            _stream(stream))
    call = PreparedCall(lib().gdr_chunk_fwd, args, "gdr_chunk_fwd", (out, final_state))
    call._keep = (pro, prologue, epi, epilogue, ws)
    return call


def prepare_recurrent_step(q, k, v, beta, g, gk, state_pool, ssm_state_indices, actual_seq_lengths,
                           num_accepted_tokens=None, scale: float = 1.0, *, prologue: Optional[Prologue] = None,
                           epilogue: Optional[Epilogue] = None, out=None, per_token: bool = False,
                           stream=None) -> PreparedCall:
    """Check and marshal a gdr_recurrent_step call once; see recurrent_step for the arguments."""
    out = _decode_checked(q, k, v, beta, g, gk, state_pool, ssm_state_indices, actual_seq_lengths,
                          num_accepted_tokens, out)
    B, Nk, S, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[3]
    pro = prologue.as_struct() if prologue is not None else None
    epi = _check_epilogue(epilogue, B, Nv, S, Dv, q.dtype)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(gk), _ptr(state_pool), int(state_pool.shape[0]),
            _ptr(ssm_state_indices), _ptr(actual_seq_lengths), _ptr(num_accepted_tokens), ctypes.c_float(scale), B,
            Nk, Nv, S, Dk, Dv, _dtype_code(q.dtype), _dtype_code(state_pool.dtype),
            ctypes.pointer(pro) if pro is not None else None, ctypes.pointer(epi) if epi is not None else None,
            _ptr(out), _stream(stream))
    name = "gdr_recurrent_step_spec" if per_token else "gdr_recurrent_step"
    call = PreparedCall(getattr(lib(), name), args, name, (out, state_pool))
    call._keep = (pro, prologue, epi, epilogue)
    return call


def _conv1d_checked(x, weight, bias, conv_state, actual_seq_lengths, Nk, Nv, Dk, Dv, q, k, v, conv_state_out,
                    output_state, stream):
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be (B, S, C) and weight (C, K)")
    B, S, C = x.shape
    K = weight.shape[1]
    if C != 2 * Nk * Dk + Nv * Dv:
        raise ValueError(f"x has {C} channels; 2 * Nk * Dk + Nv * Dv = {2 * Nk * Dk + Nv * Dv}")
    dt = x.dtype
    code = _dtype_code(dt)
    _dev(x, "x", dt)
    _dev(weight, "weight", dt, (C, K))
    _dev(bias, "bias", dt, (C,))
    _dev(conv_state, "conv_state", dt, (B, C, K))
    _dev(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,))
    outs = []
    for name, t, shape in (("q", q, (B, Nk, S, Dk)), ("k", k, (B, Nk, S, Dk)), ("v", v, (B, Nv, S, Dv))):
        t = torch.empty(shape, dtype=dt, device=x.device) if t is None else t
        outs.append(_dev(t, name, dt, shape))
    if output_state and conv_state_out is None:
        conv_state_out = torch.empty((B, C, K), dtype=dt, device=x.device)
    _dev(conv_state_out, "conv_state_out", dt, (B, C, K))
    args = (_ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(actual_seq_lengths), B, S, Nk, Nv, Dk, Dv, K,
            code, _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(conv_state_out), _stream(stream))
    return args, (outs[0], outs[1], outs[2], conv_state_out)


def conv1d(x, weight, bias=None, conv_state=None, actual_seq_lengths=None, *, Nk: int, Nv: int, Dk: int, Dv: int,
           q=None, k=None, v=None, conv_state_out=None, output_state: bool = True, stream=None):
    """Depthwise causal conv1d + SiLU over the fused q/k/v channels (``gdr_conv1d``).

    x (B, S, C) channels last with C = 2 * Nk * Dk + Nv * Dv, weight (C, K) taps oldest first, bias (C,) or
    None, conv_state (B, C, K) or None (zeros).  Returns (q (B, Nk, S, Dk), k, v (B, Nv, S, Dv), new state
    (B, C, K) or None).  Pass ``conv_state_out=conv_state`` to update the state in place (decode)."""
    args, res = _conv1d_checked(x, weight, bias, conv_state, actual_seq_lengths, Nk, Nv, Dk, Dv, q, k, v,
                                conv_state_out, output_state, stream)
    _check(lib().gdr_conv1d(*args), "gdr_conv1d")
    return res


def prepare_conv1d(x, weight, bias=None, conv_state=None, actual_seq_lengths=None, *, Nk: int, Nv: int, Dk: int,
                   Dv: int, q=None, k=None, v=None, conv_state_out=None, output_state: bool = True,
                   stream=None) -> "PreparedCall":
    """Check and marshal a gdr_conv1d call once; see conv1d for the arguments."""
    args, res = _conv1d_checked(x, weight, bias, conv_state, actual_seq_lengths, Nk, Nv, Dk, Dv, q, k, v,
                                conv_state_out, output_state, stream)
    return PreparedCall(lib().gdr_conv1d, args, "gdr_conv1d", res)


# ---- the conv1d's gradient, the gated linear recurrence and the state slots -------------------------------------
#
# These calls marshal for short kernels (a decode step, a handful of slots), where a microsecond of checks is a
# measurable share.  The ordinary case (dense tensors on the current device, the current stream) is checked and marshalled
# in C++ (csrc/marshal.cpp), which answers None to anything else.  The functions below then say what is wrong, or make
# the call on another stream: each looks at the current device and stream once, checks a tensor in one expression (``_dev`` names
# what is wrong with it only when something is), and passes plain integers to the C entry.  With ``stream=`` another than
# the current stream, the tensors a call allocates belong to that stream, and the allocator is told which streams use what.

_CODES = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16, torch.float16: GDR_F16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _ready():
    """Whether the compiled marshalling is there, after loading the library."""
    if _lib is None:
        lib()
    return _quick


def _result(r, what):
    if type(r) is int:  # a status
        _check(r, what)
    return r


class _Call:
    """The device and stream of one call, and the tensors it touches on another stream than the current one."""
    __slots__ = ("dev", "stream", "other", "used")

    def __init__(self, stream):
        self.dev = torch.cuda.current_device()
        self.stream = _raw_stream(self.dev)
        self.other = None
        if stream is not None and stream.device.index != self.dev:  # (default streams have one handle on every device)
            raise RuntimeError(f"the stream is on {stream.device}, but the call runs on the current device "
                               f"cuda:{self.dev}")
        if stream is not None and stream.cuda_stream != self.stream:
            self.other, self.stream, self.used = stream, stream.cuda_stream, []

    def ptr(self, t, name, dtype, shape):
        """Address of a dense tensor of that type and shape on the current device; None for None."""
        if t is None:
            return None
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == self.dev
                and t.is_contiguous()):
            _dev(t, name, dtype, shape)
        if self.other is not None:
            self.used.append(t)
        return t.data_ptr()

    def out(self, t, name, ref, dtype=None, shape=None):
        """The output t (checked) or, for None, a new one: as the dense tensor ref, or of a type and shape of its own
        on ref's device.  Returns the tensor and its address."""
        if t is not None:
            return t, self.ptr(t, name, dtype or ref.dtype, ref.shape if shape is None else shape)
        if self.other is None:
            t = torch.empty_like(ref) if shape is None else ref.new_empty(shape, dtype=dtype)
        else:
            with torch.cuda.stream(self.other):
                t = torch.empty_like(ref) if shape is None else ref.new_empty(shape, dtype=dtype)
            t.record_stream(torch.cuda.current_stream())
        return t, t.data_ptr()

    def done(self, status, what):
        if self.other is not None:
            for t in self.used:
                t.record_stream(self.other)
        if status != GDR_OK:
            _check(status, what)


def _int_sizes(shape, name):
    """The sizes of a tensor that go to the C entries as int (ctypes would cut larger ones off)."""
    if any(n >= 1 << 31 for n in shape):
        raise ValueError(f"{name} must have sizes below 2^31, got {tuple(shape)}")
    return shape


def _sizes(x, name):
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError(f"{name} must be a (B, N, S, D) tensor")
    return _int_sizes(x.shape, name)


def _code(dt):
    c = _CODES.get(dt)
    return _dtype_code(dt) if c is None else c


def _gate_code(x, g):
    if not isinstance(g, torch.Tensor) or (g.dtype is not torch.float32 and g.dtype is not x.dtype):
        raise RuntimeError("g must be a float32 tensor or have the dtype of x")
    return _code(g.dtype)


def scan_checkpoint_shape(B: int, N: int, S: int, D: int):
    """Shape of the fp32 ``checkpoints`` of ``scan_fwd``: the state before every 64th token."""
    return (B, N, (S + 63) // 64, D)


def _scan_fwd_args(x, g, initial_state, actual_seq_lengths, mix, out, final_state, output_final_state, checkpoints,
                   output_checkpoints, stream):
    B, N, S, D = _sizes(x, "x")
    dt, code = x.dtype, _code(x.dtype)
    gcode = _gate_code(x, g)
    c = _Call(stream)
    px, pg = c.ptr(x, "x", dt, x.shape), c.ptr(g, "g", g.dtype, x.shape)
    pi = c.ptr(initial_state, "initial_state", torch.float32, (B, N, D))
    pl = c.ptr(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,))
    out, po = c.out(out, "out", x)
    pf = pc = None
    if final_state is not None or output_final_state:
        final_state, pf = c.out(final_state, "final_state", x, torch.float32, (B, N, D))
    if checkpoints is not None or output_checkpoints:
        checkpoints, pc = c.out(checkpoints, "checkpoints", x, torch.float32, scan_checkpoint_shape(B, N, S, D))
    args = (px, pg, pi, pl, B, N, S, D, code, gcode, 1 if mix else 0, po, pf, pc, c.stream)
    return c, args, (out, final_state, checkpoints)


def scan_fwd(x, g, initial_state=None, actual_seq_lengths=None, *, mix: bool = False, out=None, final_state=None,
             output_final_state: bool = True, checkpoints=None, output_checkpoints: bool = False, stream=None):
    """Gated linear recurrence over a sequence (``gdr_scan_fwd``): h_t = exp(g_t) h_{t-1} + x_t per channel, or
    + (1 - exp(g_t)) x_t with ``mix``.

    x (B, N, S, D) in fp32, bf16 or fp16, g (B, N, S, D) log-decay in fp32 or the dtype of x, initial_state fp32
    (B, N, D) or None.  Returns (out, final_state or None, checkpoints or None); ``output_checkpoints`` keeps the fp32
    states that ``scan_bwd`` needs.  ``final_state`` may be ``initial_state`` (in-place update)."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.scan_fwd(x, g, initial_state, actual_seq_lengths, out, final_state, checkpoints, bool(mix),
                              bool(output_final_state), bool(output_checkpoints), dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_scan_fwd")
    c, args, res = _scan_fwd_args(x, g, initial_state, actual_seq_lengths, mix, out, final_state, output_final_state,
                                  checkpoints, output_checkpoints, stream)
    c.done((_lib or lib()).gdr_scan_fwd(*args), "gdr_scan_fwd")
    return res


def prepare_scan_fwd(x, g, initial_state=None, actual_seq_lengths=None, *, mix: bool = False, out=None,
                     final_state=None, output_final_state: bool = True, checkpoints=None,
                     output_checkpoints: bool = False, stream=None) -> PreparedCall:
    """Check and marshal a gdr_scan_fwd call once; see scan_fwd for the arguments."""
    c, args, res = _scan_fwd_args(x, g, initial_state, actual_seq_lengths, mix, out, final_state, output_final_state,
                                  checkpoints, output_checkpoints, stream)
    c.done(GDR_OK, "gdr_scan_fwd")
    return PreparedCall((_lib or lib()).gdr_scan_fwd, args, "gdr_scan_fwd", res)


def scan_bwd(x, g, checkpoints, dout, dfinal_state=None, actual_seq_lengths=None, *, mix: bool = False, dx=None,
             dg=None, dinitial_state=None, output_dinitial_state: bool = True, stream=None):
    """Gradient of ``scan_fwd`` (``gdr_scan_bwd``) from the checkpoints it kept, for the gradients dout (B, N, S, D) of
    out and dfinal_state (B, N, D) of final_state.  Returns (dx, dg, dinitial_state or None)."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.scan_bwd(x, g, checkpoints, dout, dfinal_state, actual_seq_lengths, dx, dg, dinitial_state, bool(mix),
                              bool(output_dinitial_state), dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_scan_bwd")
    B, N, S, D = _sizes(x, "x")
    dt, code = x.dtype, _code(x.dtype)
    gcode = _gate_code(x, g)
    c = _Call(stream)
    px, pg = c.ptr(x, "x", dt, x.shape), c.ptr(g, "g", g.dtype, x.shape)
    pc = c.ptr(checkpoints, "checkpoints", torch.float32, scan_checkpoint_shape(B, N, S, D))
    pd = c.ptr(dout, "dout", dt, x.shape)
    pf = c.ptr(dfinal_state, "dfinal_state", torch.float32, (B, N, D))
    pl = c.ptr(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,))
    dx, px_ = c.out(dx, "dx", x)
    dg, pg_ = c.out(dg, "dg", g)
    pi_ = None
    if dinitial_state is not None or output_dinitial_state:
        dinitial_state, pi_ = c.out(dinitial_state, "dinitial_state", x, torch.float32, (B, N, D))
    st = (_lib or lib()).gdr_scan_bwd(px, pg, pc, pd, pf, pl, B, N, S, D, code, gcode, 1 if mix else 0, px_, pg_, pi_,
                                      c.stream)
    c.done(st, "gdr_scan_bwd")
    return dx, dg, dinitial_state


def _scan_step_args(x, g, state_pool, ssm_state_indices, actual_seq_lengths, num_accepted_tokens, mix, out, per_token,
                    stream):
    B, N, S, D = _sizes(x, "x")
    dt, code = x.dtype, _code(x.dtype)
    gcode = _gate_code(x, g)
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 3:
        raise ValueError("state_pool must be a (slots, N, D) tensor")
    if not isinstance(ssm_state_indices, torch.Tensor) or ssm_state_indices.numel() != B * S:
        raise ValueError("ssm_state_indices must hold B * S int32 slot indices, one per flattened token")
    slots = _int_sizes(state_pool.shape, "state_pool")[0]
    c = _Call(stream)
    px, pg = c.ptr(x, "x", dt, x.shape), c.ptr(g, "g", g.dtype, x.shape)
    pp = c.ptr(state_pool, "state_pool", torch.float32, (slots, N, D))
    ps = c.ptr(ssm_state_indices, "ssm_state_indices", torch.int32, ssm_state_indices.shape)
    pl = c.ptr(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,))
    pa = c.ptr(num_accepted_tokens, "num_accepted_tokens", torch.int32, (B,))
    out, po = c.out(out, "out", x)
    args = (px, pg, pp, slots, ps, pl, pa, B, N, S, D, code, gcode, 1 if mix else 0, 1 if per_token else 0, po,
            c.stream)
    return c, args, (out, state_pool)


def scan_step(x, g, state_pool, ssm_state_indices, actual_seq_lengths=None, num_accepted_tokens=None, *,
              mix: bool = False, out=None, per_token: bool = False, stream=None):
    """The recurrence for decode over a pool of fp32 states (slots, N, D) (``gdr_scan_step``), updating it in place:
    x, g (B, N, S, D) with S <= 8, index and length arrays as in ``recurrent_step``.  Returns (out, state_pool)."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.scan_step(x, g, state_pool, ssm_state_indices, actual_seq_lengths, num_accepted_tokens, out, bool(mix),
                               bool(per_token), dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_scan_step")
    c, args, res = _scan_step_args(x, g, state_pool, ssm_state_indices, actual_seq_lengths, num_accepted_tokens, mix,
                                   out, per_token, stream)
    c.done((_lib or lib()).gdr_scan_step(*args), "gdr_scan_step")
    return res


def prepare_scan_step(x, g, state_pool, ssm_state_indices, actual_seq_lengths=None, num_accepted_tokens=None, *,
                      mix: bool = False, out=None, per_token: bool = False, stream=None) -> PreparedCall:
    """Check and marshal a gdr_scan_step call once; see scan_step for the arguments."""
    c, args, res = _scan_step_args(x, g, state_pool, ssm_state_indices, actual_seq_lengths, num_accepted_tokens, mix,
                                   out, per_token, stream)
    c.done(GDR_OK, "gdr_scan_step")
    return PreparedCall((_lib or lib()).gdr_scan_step, args, "gdr_scan_step", res)


def conv1d_bwd_workspace_bytes(B: int, S: int, Nk: int, Nv: int, Dk: int, Dv: int, K: int) -> int:
    """Bytes of workspace ``gdr_conv1d_bwd`` needs for these sizes."""
    return int((_lib or lib()).gdr_conv1d_bwd_workspace(B, S, Nk, Nv, Dk, Dv, K))


def conv1d_bwd(x, weight, dq, dk, dv, bias=None, conv_state=None, actual_seq_lengths=None, dconv_state_out=None, *,
               dx=None, dweight=None, dbias=None, dconv_state=None, workspace=None, stream=None):
    """Gradient of ``conv1d`` (``gdr_conv1d_bwd``) for the gradients dq, dk (B, Nk, S, Dk) and dv (B, Nv, S, Dv) of its
    outputs and dconv_state_out (B, C, K) or None of its new state.  Returns (dx (B, S, C), dweight fp32 (C, K), dbias
    fp32 (C,), dconv_state (B, C, K)); ``workspace`` (uint8) is allocated per call when not given."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.conv1d_bwd(x, weight, dq, dk, dv, bias, conv_state, actual_seq_lengths, dconv_state_out, dx, dweight, dbias,
                                dconv_state, workspace, dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_conv1d_bwd")
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be (B, S, C) and weight (C, K)")
    B, S, C = _int_sizes(x.shape, "x")
    K = _int_sizes(weight.shape, "weight")[1]
    _, Nk, _, Dk = _sizes(dq, "dq")
    _, Nv, _, Dv = _sizes(dv, "dv")
    if C != 2 * Nk * Dk + Nv * Dv:
        raise ValueError(f"x has {C} channels; 2 * Nk * Dk + Nv * Dv = {2 * Nk * Dk + Nv * Dv}")
    dt, code = x.dtype, _code(x.dtype)
    c = _Call(stream)
    ins = (c.ptr(x, "x", dt, x.shape), c.ptr(weight, "weight", dt, (C, K)), c.ptr(bias, "bias", dt, (C,)),
           c.ptr(conv_state, "conv_state", dt, (B, C, K)),
           c.ptr(actual_seq_lengths, "actual_seq_lengths", torch.int32, (B,)), c.ptr(dq, "dq", dt, (B, Nk, S, Dk)),
           c.ptr(dk, "dk", dt, (B, Nk, S, Dk)), c.ptr(dv, "dv", dt, (B, Nv, S, Dv)),
           c.ptr(dconv_state_out, "dconv_state_out", dt, (B, C, K)))
    need = (_lib or lib()).gdr_conv1d_bwd_workspace(B, S, Nk, Nv, Dk, Dv, K)
    if workspace is not None and workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; the call needs {need}")
    pw = None
    if workspace is not None or need:
        workspace, pw = c.out(workspace, "workspace", x, torch.uint8, (need,) if workspace is None else workspace.shape)
    dx, px = c.out(dx, "dx", x)
    dweight, pdw = c.out(dweight, "dweight", x, torch.float32, (C, K))
    dbias, pdb = c.out(dbias, "dbias", x, torch.float32, (C,))
    dconv_state, pds = c.out(dconv_state, "dconv_state", x, dt, (B, C, K))
    st = (_lib or lib()).gdr_conv1d_bwd(*ins, B, S, Nk, Nv, Dk, Dv, K, code, px, pdw, pdb, pds, pw,
                                        0 if workspace is None else workspace.numel(), c.stream)
    c.done(st, "gdr_conv1d_bwd")
    return dx, dweight, dbias, dconv_state


def _pools(c, pools):
    """The C array of a list of pools (tensors whose first dimension is the slots), and their number of slots."""
    pools = [pools] if isinstance(pools, torch.Tensor) else list(pools)
    if not pools:
        raise ValueError("pools must name at least one tensor")
    arr = (GdrPoolStruct * len(pools))()
    slots = None
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor) or t.dim() < 1:
            raise ValueError("a pool must be a tensor whose first dimension is the slots")
        if slots is None:
            slots = _int_sizes(t.shape[:1], f"pools[{i}]")[0]
        elif t.shape[0] != slots:
            raise ValueError(f"all pools must have {slots} slots, pool {i} has {t.shape[0]}")
        arr[i].data = c.ptr(t, f"pools[{i}]", t.dtype, t.shape)
        arr[i].slot_bytes = t.element_size() * (t.numel() // slots if slots else 0)
    return arr, len(pools), slots


def _list_i32(c, t, name, n=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be a one-dimensional int32 tensor")
    _int_sizes(t.shape, name)
    return c.ptr(t, name, torch.int32, t.shape if n is None else (n,))


def slot_copy(pools, src, dst, *, stream=None):
    """pool[dst[i]] = pool[src[i]] in every pool (``gdr_slot_copy``).  ``pools``: one tensor (slots, ...) or a list of
    up to 64 of any types with the same number of slots; src, dst int32 (n), -1 for no move.  A move whose target is
    another move's source or an earlier move's target is skipped and flagged (``get_error``).  Returns pools."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.slot_copy(pools, src, dst, dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_slot_copy")
    c = _Call(stream)
    arr, n_pools, slots = _pools(c, pools)
    ps = _list_i32(c, src, "src")
    st = (_lib or lib()).gdr_slot_copy(arr, n_pools, slots, ps, _list_i32(c, dst, "dst", src.shape[0]), src.shape[0], c.stream)
    c.done(st, "gdr_slot_copy")
    return pools


def slot_fork(pools, slot_table, parents, *, new_slot_table=None, stream=None):
    """Beam reordering (``gdr_slot_fork``): row i continues from row parents[i] (-1: from nothing).  The lowest
    child of a row keeps its slot, the others get copies in the slots of the rows without a child.  Returns the
    new slot of every row (int32)."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.slot_fork(pools, slot_table, parents, new_slot_table, dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_slot_fork")
    c = _Call(stream)
    arr, n_pools, slots = _pools(c, pools)
    pt = _list_i32(c, slot_table, "slot_table")
    n = slot_table.shape[0]
    pp = _list_i32(c, parents, "parents", n)
    new_slot_table, pn = c.out(new_slot_table, "new_slot_table", slot_table)
    st = (_lib or lib()).gdr_slot_fork(arr, n_pools, slots, pt, pp, n, pn, c.stream)
    c.done(st, "gdr_slot_fork")
    return new_slot_table


def slot_compact(pools, live, *, new_slot=None, n_live=None, stream=None):
    """Moves the live slots (live int32 (slots), non-zero) at or above their count into the free slots below it
    (``gdr_slot_compact``).  Returns (new_slot int32 (slots): where each slot went, -1 for free ones; n_live int32
    (1,))."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.slot_compact(pools, live, new_slot, n_live, dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_slot_compact")
    c = _Call(stream)
    arr, n_pools, slots = _pools(c, pools)
    pl = _list_i32(c, live, "live", slots)
    new_slot, pn = c.out(new_slot, "new_slot", live)
    n_live, pc = c.out(n_live, "n_live", live, torch.int32, (1,))
    st = (_lib or lib()).gdr_slot_compact(arr, n_pools, slots, pl, pn, pc, c.stream)
    c.done(st, "gdr_slot_compact")
    return new_slot, n_live


def slot_free(pools, idx, live=None, *, stream=None):
    """Sets the slots idx (int32 (n), -1 for none) of every pool to zero and, with ``live``, marks them free
    (``gdr_slot_free``).  Returns pools."""
    if stream is None and (_quick or _ready()):
        dev = torch.cuda.current_device()
        r = _quick.slot_free(pools, idx, live, dev, _raw_stream(dev))
        if r is not None:
            return _result(r, "gdr_slot_free")
    c = _Call(stream)
    arr, n_pools, slots = _pools(c, pools)
    pi = _list_i32(c, idx, "idx")
    pl = None if live is None else _list_i32(c, live, "live", slots)
    st = (_lib or lib()).gdr_slot_free(arr, n_pools, slots, pi, idx.shape[0], pl, c.stream)
    c.done(st, "gdr_slot_free")
    return pools


def prologue(q=None, k=None, b=None, a=None, A_log=None, dt_bias=None, eps: float = 1e-6, *, stream=None):
    """Stand-alone prologue (``gdr_prologue_apply``): returns a dict with q_hat,
    k_hat (l2norm, eps inside the sqrt), beta = sigmoid(b) and
    g = -exp(A_log) * softplus(a + dt_bias) for whichever inputs are given."""
    ref = next(t for t in (q, k, b) if t is not None) if any(t is not None for t in (q, k, b)) else None
    dt = ref.dtype if ref is not None else torch.float32
    code = _dtype_code(dt)
    if q is not None or k is not None:
        B, Nk, S, Dk = (q if q is not None else k).shape
    else:
        B, Nk, S, Dk = (b if b is not None else a).shape[0], 1, (b if b is not None else a).shape[2], 16
    Nv = (b if b is not None else a).shape[1] if (b is not None or a is not None) else Nk
    res = {}
    for name, t in (("q", q), ("k", k)):
        if t is not None:
            _dev(t, name, dt, (B, Nk, S, Dk))
            res[name + "_hat"] = torch.empty_like(t)
    if b is not None:
        _dev(b, "b", dt, (B, Nv, S))
        res["beta"] = torch.empty_like(b)
    if a is not None:
        _dev(a, "a", torch.float32, (B, Nv, S))
        _dev(A_log, "A_log", torch.float32, (Nv,))
        _dev(dt_bias, "dt_bias", torch.float32, (Nv,))
        res["g"] = torch.empty_like(a)
    st = lib().gdr_prologue_apply(_ptr(q), _ptr(k), _ptr(b), _ptr(a), _ptr(A_log), _ptr(dt_bias), float(eps), B, Nk,
                                  Nv, S, Dk, code, _ptr(res.get("q_hat")), _ptr(res.get("k_hat")),
                                  _ptr(res.get("beta")), _ptr(res.get("g")), _stream(stream))
    _check(st, "gdr_prologue_apply")
    return res


def get_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    v = ctypes.c_int(0)
    _check(lib().gdr_get_error(_stream(stream), ctypes.byref(v)), "gdr_get_error")
    return v.value


def version() -> int:
    return int(lib().gdr_version())


def take_timeout_site() -> dict:
    """Diagnostic: the first bounded wait of the tensor-core prefill that ran out since the last read (cleared by
    the read), as {"warp", "barrier", "parity", "cta"}, or {} if none."""
    v = ctypes.c_uint(0)
    _check(lib().gdr_debug_timeout_site(ctypes.byref(v)), "gdr_debug_timeout_site")
    x = v.value
    if not x:
        return {}
    return {"warp": (x >> 24) & 0x3F, "barrier": (x >> 16) & 0xFF, "parity": (x >> 15) & 1, "cta": x & 0x7FFF}


# schedules of the tensor-core prefill for ``set_chunk_schedule``
SCHEDULE_AUTO, SCHEDULE_ONE_KERNEL, SCHEDULE_TWO_KERNELS = 0, 1, 2


def set_chunk_schedule(schedule: int) -> None:
    """Diagnostic: which schedule of the tensor-core prefill the workspace query sizes for later calls
    (``gdr_debug_set_chunk_schedule``): SCHEDULE_AUTO by shape, or one of the two always."""
    _check(lib().gdr_debug_set_chunk_schedule(int(schedule)), "gdr_debug_set_chunk_schedule")


def set_wait_limit_ns(ns: int) -> None:
    """Diagnostic: the limit of the tensor-core prefill's bounded waits for later calls (0: the default, 1 s)."""
    _check(lib().gdr_debug_set_wait_limit(int(ns)), "gdr_debug_set_wait_limit")
