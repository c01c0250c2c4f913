"""ctypes binding of libattn.so (include/attn.h), argument marshalling only.

The functions named like the C entry points (``attn_fwd``, ``attn_bwd``, ...)
take torch tensors (or raw device addresses as ints) and pass their data
pointers, sizes and the CUDA stream straight through; every step of the
computation runs in the library's CUDA kernels. ``forward``/``backward``
additionally allocate the outputs (and the backward workspace) with torch.

There is no fallback: if libattn.so is missing or a call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

__all__ = [
    "LIB_PATH", "EXPORTED_SYMBOLS", "AttnError", "load_library",
    "ATTN_OK", "ATTN_ERR_INVALID_ARG", "ATTN_ERR_UNSUPPORTED", "ATTN_ERR_MISALIGNED", "ATTN_ERR_CUDA",
    "ATTN_ERR_TIMEOUT", "ATTN_ERR_WORKSPACE", "ATTN_F32", "ATTN_BF16",
    "attn_fwd", "attn_fwd_f32_blocked", "attn_fwd_splitkv", "attn_fwd_splitkv_splits",
    "attn_fwd_splitkv_workspace_size", "attn_bwd", "attn_bwd_phase", "attn_bwd_workspace_size", "attn_bwd_dq_splits",
    "attn_bwd_noalloc", "ATTN_NOALLOC_SCRATCH_BYTES", "attn_online_softmax_step", "attn_device_status",
    "attn_selftest_wait_timeout", "attn_strerror", "attn_last_cuda_error", "attn_version",
    "attn_fwd_scored", "attn_fwd_scored_workspace_size", "attn_bwd_scored", "attn_bwd_scored_workspace_size",
    "attn_rope_init", "attn_rope", "AttnScore", "AttnRope",
    "forward", "backward", "forward_scored", "backward_scored", "rope_plan", "rope",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn.so")

ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_MISALIGNED = 0, 1, 2, 3
ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT, ATTN_ERR_WORKSPACE = 4, 5, 6
ATTN_F32, ATTN_BF16 = 0, 1

_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t



class AttnScore(ctypes.Structure):
    """attn_score_t: how the scored attention changes and masks its scores (device addresses, 0 for none)."""
    _fields_ = [("softcap", _F), ("causal", _I), ("slopes", _P), ("q_pos", _P), ("key_begin", _P), ("key_end", _P)]


class AttnRope(ctypes.Structure):
    """attn_rope_t: a plan of rotary positions (see rope_plan)."""
    _fields_ = [("rot", _I), ("interleaved", _I), ("mscale", _F), ("reserved", _I), ("turns", ctypes.c_uint64 * 128)]


_STRIDES = ctypes.c_longlong * 12

# name -> (restype, argtypes); must list every function of include/attn.h
_SIGNATURES = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "attn_fwd_f32_blocked": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "attn_fwd_splitkv": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P, _SZ, _P]),
    "attn_fwd_splitkv_splits": (_I, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "attn_fwd_splitkv_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "attn_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "attn_bwd_dq_splits": (_I, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P, _SZ, _P]),
    "attn_bwd_phase": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P, _SZ,
                            _I, _P]),
    "attn_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P]),
    "attn_fwd_scored": (_I, [_P] * 5 + [_I] * 7 + [_F, ctypes.POINTER(AttnScore), _I, _P, _SZ, _P]),
    "attn_fwd_scored_workspace_size": (_SZ, [_I] * 8),
    "attn_bwd_scored": (_I, [_P] * 9 + [_I] * 7 + [_F, ctypes.POINTER(AttnScore), _I, _P, _SZ, _P]),
    "attn_bwd_scored_workspace_size": (_SZ, [_I] * 8),
    "attn_rope_init": (_I, [ctypes.POINTER(AttnRope), _I, _I] + [ctypes.c_double] * 6),
    "attn_rope": (_I, [ctypes.POINTER(AttnRope)] + [_P] * 4 + [ctypes.POINTER(ctypes.c_longlong), _P] + [_I] * 7 + [_P]),
    "attn_online_softmax_step": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "attn_device_status": (_I, [_P]),
    "attn_selftest_wait_timeout": (_I, [_I, _P]),
    "attn_strerror": (ctypes.c_char_p, [_I]),
    "attn_last_cuda_error": (_I, []),
    "attn_version": (_I, []),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)

_lib: Optional[ctypes.CDLL] = None


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = attn_strerror(status) if _lib is not None else str(status)
        extra = ""
        if status == ATTN_ERR_CUDA and _lib is not None:
            extra = f" (cuda error {_lib.attn_last_cuda_error()})"
        super().__init__(f"{where}: {msg}{extra} [status {status}]")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libattn.so once; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m exact_tiled_softmax_attn_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t) -> int:
    if isinstance(t, int):
        return t
    if t.dtype == torch.float32:
        return ATTN_F32
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def attn_strerror(status: int) -> str:
    return load_library().attn_strerror(status).decode()


def attn_last_cuda_error() -> int:
    return load_library().attn_last_cuda_error()


def attn_version() -> int:
    return load_library().attn_version()


def attn_fwd(Q, K, V, O, LSE, B, H, Tq, Tk, d, dv, scale, causal, dtype, stream=None, check=True) -> int:
    st = load_library().attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Tq, Tk, d, dv,
                                 float(scale), int(causal), int(dtype), _stream(stream))
    if check:
        _check(st, "attn_fwd")
    return st


def attn_fwd_f32_blocked(Q, K, V, O, LSE, B, H, Tq, Tk, d, dv, scale, causal, block_n, stream=None,
                         check=True) -> int:
    st = load_library().attn_fwd_f32_blocked(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Tq, Tk, d, dv,
                                             float(scale), int(causal), int(block_n), _stream(stream))
    if check:
        _check(st, "attn_fwd_f32_blocked")
    return st


def attn_fwd_splitkv(Q, K, V, O, LSE, B, H, Tq, Tk, d, dv, scale, causal, dtype, num_splits, workspace,
                     workspace_bytes, stream=None, check=True) -> int:
    st = load_library().attn_fwd_splitkv(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Tq, Tk, d, dv,
                                         float(scale), int(causal), int(dtype), int(num_splits), _ptr(workspace),
                                         int(workspace_bytes), _stream(stream))
    if check:
        _check(st, "attn_fwd_splitkv")
    return st


def attn_fwd_splitkv_splits(B, H, Tq, Tk, d, dv, dtype, num_splits) -> int:
    return load_library().attn_fwd_splitkv_splits(B, H, Tq, Tk, d, dv, int(dtype), int(num_splits))


def attn_fwd_splitkv_workspace_size(B, H, Tq, Tk, d, dv, dtype, num_splits) -> int:
    return load_library().attn_fwd_splitkv_workspace_size(B, H, Tq, Tk, d, dv, int(dtype), int(num_splits))


def attn_online_softmax_step(m, l, acc, scores, v_block, n, bs, dv, stream=None, check=True) -> int:
    st = load_library().attn_online_softmax_step(_ptr(m), _ptr(l), _ptr(acc), _ptr(scores), _ptr(v_block), int(n),
                                                 int(bs), int(dv), _stream(stream))
    if check:
        _check(st, "attn_online_softmax_step")
    return st


def attn_bwd_workspace_size(B, H, Tq, Tk, d, dv, dtype, deterministic) -> int:
    return load_library().attn_bwd_workspace_size(B, H, Tq, Tk, d, dv, int(dtype), int(deterministic))


def attn_bwd_dq_splits(B, H, Tq, Tk, d, dv, dtype, deterministic) -> int:
    return load_library().attn_bwd_dq_splits(B, H, Tq, Tk, d, dv, int(dtype), int(deterministic))


def attn_bwd(Q, K, V, O, LSE, dO, dQ, dK, dV, B, H, Tq, Tk, d, dv, scale, causal, dtype, deterministic,
             workspace, workspace_bytes, stream=None, check=True) -> int:
    st = load_library().attn_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _ptr(dO), _ptr(dQ), _ptr(dK),
                                 _ptr(dV), B, H, Tq, Tk, d, dv, float(scale), int(causal), int(dtype),
                                 int(deterministic), _ptr(workspace), int(workspace_bytes), _stream(stream))
    if check:
        _check(st, "attn_bwd")
    return st


def attn_bwd_phase(Q, K, V, O, LSE, dO, dQ, dK, dV, B, H, Tq, Tk, d, dv, scale, causal, dtype, deterministic,
                   workspace, workspace_bytes, phase, stream=None, check=True) -> int:
    st = load_library().attn_bwd_phase(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _ptr(dO), _ptr(dQ),
                                       _ptr(dK), _ptr(dV), B, H, Tq, Tk, d, dv, float(scale), int(causal),
                                       int(dtype), int(deterministic), _ptr(workspace), int(workspace_bytes),
                                       int(phase), _stream(stream))
    if check:
        _check(st, "attn_bwd_phase")
    return st


def attn_bwd_noalloc(Q, K, V, O, LSE, dO, dQ, dK, dV, B, H, Tq, Tk, d, dv, scale, causal, dtype, deterministic,
                     stream=None, check=True) -> int:
    """attn_bwd with the library's static scratch buffer instead of a workspace."""
    st = load_library().attn_bwd_noalloc(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _ptr(dO), _ptr(dQ),
                                         _ptr(dK), _ptr(dV), B, H, Tq, Tk, d, dv, float(scale), int(causal),
                                         int(dtype), int(deterministic), _stream(stream))
    if check:
        _check(st, "attn_bwd_noalloc")
    return st


ATTN_NOALLOC_SCRATCH_BYTES = 64 << 20


def attn_fwd_scored(Q, K, V, O, LSE, B, H, Hkv, Tq, Tk, d, dv, scale, score, dtype, workspace, workspace_bytes,
                    stream=None, check=True) -> int:
    """`score`: an AttnScore, or None for plain scores without a mask."""
    st = load_library().attn_fwd_scored(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, H, Hkv, Tq, Tk, d, dv,
                                        scale, score, dtype, _ptr(workspace), workspace_bytes, _stream(stream))
    if check:
        _check(st, "attn_fwd_scored")
    return st


def attn_fwd_scored_workspace_size(B, H, Hkv, Tq, Tk, d, dv, dtype) -> int:
    return load_library().attn_fwd_scored_workspace_size(B, H, Hkv, Tq, Tk, d, dv, dtype)


def attn_bwd_scored(Q, K, V, O, LSE, dO, dQ, dK, dV, B, H, Hkv, Tq, Tk, d, dv, scale, score, dtype, workspace,
                    workspace_bytes, stream=None, check=True) -> int:
    st = load_library().attn_bwd_scored(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _ptr(dO), _ptr(dQ), _ptr(dK),
                                        _ptr(dV), B, H, Hkv, Tq, Tk, d, dv, scale, score, dtype, _ptr(workspace),
                                        workspace_bytes, _stream(stream))
    if check:
        _check(st, "attn_bwd_scored")
    return st


def attn_bwd_scored_workspace_size(B, H, Hkv, Tq, Tk, d, dv, dtype) -> int:
    return load_library().attn_bwd_scored_workspace_size(B, H, Hkv, Tq, Tk, d, dv, dtype)


def attn_rope_init(plan, rot, interleaved, theta, factor, original_length, low_turns, high_turns, mscale,
                   check=True) -> int:
    st = load_library().attn_rope_init(plan, rot, interleaved, theta, factor, original_length, low_turns, high_turns,
                                       mscale)
    if check:
        _check(st, "attn_rope_init")
    return st


def attn_rope(plan, Q, Qout, K, Kout, strides, pos, B, H, Hkv, T, d, inverse, dtype, stream=None, check=True) -> int:
    """`strides`: 12 element strides (batch, head, token of Q, Qout, K, Kout)."""
    st = load_library().attn_rope(plan, _ptr(Q), _ptr(Qout), _ptr(K), _ptr(Kout), _STRIDES(*strides), _ptr(pos), B, H,
                                  Hkv, T, d, inverse, dtype, _stream(stream))
    if check:
        _check(st, "attn_rope")
    return st


def attn_device_status(stream=None) -> int:
    return load_library().attn_device_status(_stream(stream))


def attn_selftest_wait_timeout(limit_ms: int, stream=None) -> int:
    return load_library().attn_selftest_wait_timeout(int(limit_ms), _stream(stream))


# ------------------------------------------------------------------ helpers

def _shape(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("expected [B, H, T, d] tensors")
    B, H, Tq, d = q.shape
    Tk, dv = k.shape[2], v.shape[3]
    if tuple(k.shape) != (B, H, Tk, d) or tuple(v.shape) != (B, H, Tk, dv):
        raise ValueError("Q, K, V shapes disagree")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return B, H, Tq, Tk, d, dv


def forward(q, k, v, causal: bool = False, scale: Optional[float] = None, stream=None,
            num_splits: Optional[int] = None):
    """O, LSE = attention(q, k, v). Allocates O (q.dtype) and LSE (fp32) with torch.

    num_splits selects the split-KV forward (0 = automatic, n >= 1 = that many
    key splits); None is the plain forward."""
    B, H, Tq, Tk, d, dv = _shape(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty(B, H, Tq, dv, dtype=q.dtype, device=q.device)
    lse = torch.empty(B, H, Tq, dtype=torch.float32, device=q.device)
    dt = _dtype_code(q)
    if num_splits is None:
        attn_fwd(q, k, v, o, lse, B, H, Tq, Tk, d, dv, scale, causal, dt, stream)
    else:
        nbytes = attn_fwd_splitkv_workspace_size(B, H, Tq, Tk, d, dv, dt, num_splits)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
        attn_fwd_splitkv(q, k, v, o, lse, B, H, Tq, Tk, d, dv, scale, causal, dt, num_splits, ws, ws.numel(),
                         stream)
    return o, lse


def backward(q, k, v, o, lse, do, causal: bool = False, scale: Optional[float] = None,
             deterministic: bool = False, stream=None, workspace=None):
    """dQ, dK, dV. Allocates the gradients and (unless given) the workspace with torch."""
    B, H, Tq, Tk, d, dv = _shape(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dt = _dtype_code(q)
    ws_bytes = attn_bwd_workspace_size(B, H, Tq, Tk, d, dv, dt, int(deterministic))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dvv = torch.empty_like(v)
    attn_bwd(q, k, v, o, lse, do, dq, dk, dvv, B, H, Tq, Tk, d, dv, scale, causal, dt, int(deterministic),
             workspace, workspace.numel(), stream)
    return dq, dk, dvv


# The current stream's handle without building a torch.cuda.Stream for it (3 us of a small call's 15).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _call_on(index, stream, call, *args):
    """call(stream handle, *args) with CUDA device `index`, and a stream given for the call, made current, so that
    what the call allocates belongs to the stream its kernels run on."""
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    if stream is None:
        if index == torch.cuda.current_device():
            return call(_raw_stream(index), *args)
        with torch.cuda.device(index):
            return call(_raw_stream(index), *args)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=index)
    elif stream.device.index != index:
        raise ValueError("the stream must be one of the tensors' device")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return call(stream.cuda_stream, *args)


_workspace_size = functools.lru_cache(maxsize=4096)(
    lambda fn, *shape: getattr(load_library(), fn)(*shape))   # a rule of the shapes


def _row_array(name, t, rows, dev):
    """The address of an optional int32 [B, Tq] array of row values."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != rows or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous int32 {list(rows)} tensor on Q's device")
    return t.data_ptr()


def _scored_args(q, k, v, causal, scale, softcap, slopes, q_pos, key_begin, key_end):
    """Checks shapes, types and devices; (shape arguments, scale, AttnScore, device index)."""
    qs, ks, vs = q.shape, k.shape, v.shape
    if len(qs) != 4 or len(ks) != 4 or len(vs) != 4:
        raise ValueError("expected [B, H, T, d] tensors")
    B, H, Tq, d = qs
    _, Hkv, Tk, dv = vs
    if ks[0] != B or vs[0] != B or ks[1] != Hkv or ks[2] != Tk or ks[3] != d:
        raise ValueError("Q, K, V shapes disagree")
    if Hkv == 0 or H % Hkv:
        raise ValueError("the number of query heads must be a multiple of the number of key heads")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("tensors must be contiguous")
    dev, dtype = q.get_device(), q.dtype
    if k.dtype != dtype or v.dtype != dtype or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("Q, K and V must have one dtype and device")
    rows = (B, Tq)
    if slopes is not None:
        if slopes.dtype != torch.float32 or slopes.shape != (H,) or not slopes.is_contiguous() or \
                slopes.get_device() != dev:
            raise ValueError("slopes must be a contiguous fp32 [H] tensor on Q's device")
        slopes = slopes.data_ptr()
    score = AttnScore(softcap, 1 if causal else 0, slopes, _row_array("q_pos", q_pos, rows, dev),
                      _row_array("key_begin", key_begin, rows, dev), _row_array("key_end", key_end, rows, dev))
    shape = (B, H, Hkv, Tq, Tk, d, dv)
    return shape, 1.0 / math.sqrt(d) if scale is None else scale, score, _dtype_code(q), dev


def _check_workspace(given, dev):
    # (its address and size go to the library as they are: a view that repeats memory, or host memory, would be written)
    if given is not None and (given.dtype != torch.uint8 or not given.is_contiguous() or given.get_device() != dev):
        raise ValueError("workspace must be a contiguous uint8 tensor on Q's device")


def _workspace(given, nbytes, device):
    return torch.empty(nbytes or 1, dtype=torch.uint8, device=device) if given is None else given


def forward_scored(q, k, v, causal: bool = False, scale: Optional[float] = None, softcap: float = 0.0, slopes=None,
                   q_pos=None, key_begin=None, key_end=None, stream=None, workspace=None):
    """O, LSE of the scored attention: q [B, H, Tq, d], k [B, Hkv, Tk, d], v [B, Hkv, Tk, dv].

    Scores scale * q.k are capped by softcap * tanh(. / softcap) where softcap > 0, lowered by slopes[h] *
    |q_pos - key| where slopes ([H] fp32) is given, and limited to keys [key_begin, key_end) of each query row
    (int32 [B, Tq], shared by the heads) and, with causal, to keys at or before q_pos (default: the row index).
    Allocates O, LSE and, unless given, the workspace (uint8, attn_fwd_scored_workspace_size bytes)."""
    shape, scale, score, dt, dev = _scored_args(q, k, v, causal, scale, softcap, slopes, q_pos, key_begin, key_end)
    _check_workspace(workspace, dev)
    B, H, _, Tq, _, _, dv = shape

    def call(handle):
        device = q.device
        o = torch.empty((B, H, Tq, dv), dtype=q.dtype, device=device)
        lse = torch.empty((B, H, Tq), dtype=torch.float32, device=device)
        ws = _workspace(workspace, _workspace_size("attn_fwd_scored_workspace_size", *shape, dt), device)
        _check(load_library().attn_fwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                              *shape, scale, score, dt, ws.data_ptr(), ws.numel(), handle),
               "attn_fwd_scored")
        return o, lse
    return _call_on(dev, stream, call)


def backward_scored(q, k, v, o, lse, do, causal: bool = False, scale: Optional[float] = None, softcap: float = 0.0,
                    slopes=None, q_pos=None, key_begin=None, key_end=None, stream=None, workspace=None):
    """dQ, dK, dV of forward_scored's O (same arguments; dK and dV summed over the heads that share them)."""
    shape, scale, score, dt, dev = _scored_args(q, k, v, causal, scale, softcap, slopes, q_pos, key_begin, key_end)
    _check_workspace(workspace, dev)
    B, H, _, Tq, _, _, dv = shape
    for name, t, want, dtype in (("O", o, (B, H, Tq, dv), q.dtype), ("dO", do, (B, H, Tq, dv), q.dtype),
                                 ("LSE", lse, (B, H, Tq), torch.float32)):
        if t.shape != want or t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"{name} must be a contiguous {dtype} {list(want)} tensor on Q's device")

    def call(handle):
        dq, dk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = _workspace(workspace, _workspace_size("attn_bwd_scored_workspace_size", *shape, dt), q.device)
        _check(load_library().attn_bwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                              do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dvv.data_ptr(), *shape,
                                              scale, score, dt, ws.data_ptr(), ws.numel(), handle), "attn_bwd_scored")
        return dq, dk, dvv
    return _call_on(dev, stream, call)


def rope_plan(rot: int, interleaved: bool = False, theta: float = 10000.0, factor: float = 1.0,
              original_length: float = 0.0, low_turns: float = 1.0, high_turns: float = 4.0,
              mscale: float = 1.0) -> AttnRope:
    """A plan for rope(): `rot` rotated elements a head, pairs (i, i + rot/2) or, interleaved, (2i, 2i + 1).

    `factor` stretches the context: every frequency is divided by it, or, with original_length > 0, only those
    of pairs that make fewer than high_turns turns over it (wholly below low_turns)."""
    plan = AttnRope()
    attn_rope_init(plan, int(rot), int(interleaved), theta, factor, original_length, low_turns, high_turns, mscale)
    return plan


def rope(q, k, plan: AttnRope, pos=None, inverse: bool = False, out=None, stream=None):
    """Rotary positions of q [B, H, T, d] and k [B, Hkv, T, d] (any strides, last dimension contiguous).

    pos: int32 [B, T] positions (default: the token index); inverse turns back, which is the gradient. Returns
    new contiguous tensors, or writes `out` = (q_out, k_out), which may be (q, k) themselves."""
    qs, ks = q.shape, k.shape
    dev, dtype = q.get_device(), q.dtype
    if len(qs) != 4 or len(ks) != 4 or k.dtype != dtype or k.get_device() != dev:
        raise ValueError("expected two [B, H, T, d] tensors of one dtype and device")
    B, H, T, d = qs
    Hkv = ks[1]
    if ks[0] != B or ks[2] != T or ks[3] != d:
        raise ValueError("Q and K shapes disagree")
    where = _row_array("pos", pos, (B, T), dev)
    q0, q1, q2, q3 = q.stride()
    k0, k1, k2, k3 = k.stride()
    if (q3 != 1 or k3 != 1) and d > 1:
        raise ValueError("the last dimension must be contiguous")
    if out is None:
        c = T * d
        strides = _STRIDES(q0, q1, q2, H * c, c, d, k0, k1, k2, Hkv * c, c, d)
    else:
        a, b = out
        if a.shape != qs or b.shape != ks or a.dtype != dtype or b.dtype != dtype or a.get_device() != dev or \
                b.get_device() != dev or (d > 1 and (a.stride(3) != 1 or b.stride(3) != 1)):
            raise ValueError("outputs must have the shapes, dtype and device of Q and K and contiguous rows")
        strides = _STRIDES(q0, q1, q2, *a.stride()[:3], k0, k1, k2, *b.stride()[:3])

    def call(handle):
        a, b = out or (torch.empty(qs, dtype=dtype, device=q.device), torch.empty(ks, dtype=dtype, device=q.device))
        _check(load_library().attn_rope(plan, q.data_ptr(), a.data_ptr(), k.data_ptr(), b.data_ptr(), strides, where,
                                        B, H, Hkv, T, d, 1 if inverse else 0, _dtype_code(q), handle), "attn_rope")
        return a, b
    return _call_on(dev, stream, call)
