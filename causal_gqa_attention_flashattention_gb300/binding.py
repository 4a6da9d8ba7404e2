"""ctypes binding for libneattn.so (C ABI in include/ne_attn.h).

Argument marshalling only: every step of the attention runs in the CUDA
library.  PyTorch supplies device memory and the current stream.  If the
library has not been built, or its kernels cannot run on this device, the
calls raise; there is no other implementation to fall back to.
"""
import collections
import ctypes
import importlib.util
import os

import torch

from .build import bind_path

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libneattn.so")

NE_OK = 0
ERR_WORKSPACE = -5
O_FP32 = 1       # flag bits, see include/ne_attn.h
GRAD_FP32 = 2
PRECISE_QK = 4
QK_ROTATED = 8
ROPE_HALF = 16
FP8 = 32
_lib = None


class NeAttnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = lib().ne_attn_status_string(status).decode() if _lib is not None else str(status)
        super().__init__("%s failed with status %d: %s" % (fn, status, msg))


def lib():
    """Loads the in-tree CUDA library (built by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libneattn.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.ne_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
        L.ne_attn_fwd.restype = i
        L.ne_attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
        L.ne_attn_fwd_ex.restype = i
        L.ne_attn_fwd_workspace_size.argtypes = [i, i, i, i, i, i]
        L.ne_attn_fwd_workspace_size.restype = sz
        L.ne_attn_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
        L.ne_attn_bwd_workspace_size.restype = sz
        L.ne_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
        L.ne_attn_bwd.restype = i
        L.ne_attn_check_status.argtypes = [vp]
        L.ne_attn_check_status.restype = i
        L.ne_attn_status_string.argtypes = [i]
        L.ne_attn_status_string.restype = ctypes.c_char_p
        L.ne_attn_debug_timeout_probe.argtypes = [i, vp]
        L.ne_attn_debug_timeout_probe.restype = i
        L.ne_attn_profile_start.argtypes = [i]
        L.ne_attn_profile_start.restype = i
        L.ne_attn_profile_stop.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong)]
        L.ne_attn_profile_stop.restype = i
        L.ne_attn_profile_detach.argtypes = []
        L.ne_attn_profile_detach.restype = i
        L.ne_attn_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong)]
        L.ne_attn_profile_read.restype = i
        L.ne_attn_kv_append.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        L.ne_attn_kv_append.restype = i
        L.ne_attn_decode_workspace_size.argtypes = [i, i, i, i, i, i]
        L.ne_attn_decode_workspace_size.restype = sz
        L.ne_attn_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp, sz, vp]
        L.ne_attn_decode.restype = i
        ip = ctypes.POINTER(ctypes.c_int)
        L.ne_attn_debug_fwd_schedule.argtypes = [i, i, i, i, i, ip, i, ip, ip]
        L.ne_attn_debug_fwd_schedule.restype = i
        L.ne_attn_qkv_workspace_size.argtypes = [i, i, i, i, i, i, i]
        L.ne_attn_qkv_workspace_size.restype = sz
        L.ne_attn_qkv_rmsnorm.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, f, i, vp, sz, vp]
        L.ne_attn_qkv_rmsnorm.restype = i
        ll = ctypes.c_longlong
        L.ne_attn_qk_norm.argtypes = [vp, vp, vp, vp, i, i, i, i, i, ll, ll, f, f, i, vp, sz, vp]
        L.ne_attn_qk_norm.restype = i
        L.ne_attn_qk_norm_bwd_workspace_size.argtypes = [i, i, i, i, i]
        L.ne_attn_qk_norm_bwd_workspace_size.restype = sz
        L.ne_attn_qk_norm_bwd.argtypes = [vp] * 10 + [i] * 5 + [ll] * 4 + [f, i, vp, sz, vp]
        L.ne_attn_qk_norm_bwd.restype = i
        L.ne_attn_kv_append_paged.argtypes = [vp] * 8 + [i] * 7 + [ll] * 3 + [f, f, i, vp]
        L.ne_attn_kv_append_paged.restype = i
        L.ne_attn_decode_paged_workspace_size.argtypes = [i, i, i, i, i, i]
        L.ne_attn_decode_paged_workspace_size.restype = sz
        L.ne_attn_decode_paged.argtypes = [vp] * 9 + [i] * 8 + [ll, ll, i, f, f, i, vp, sz, vp]
        L.ne_attn_decode_paged.restype = i
        L.ne_attn_paged_plan.argtypes = [vp] * 13 + [i] * 6 + [ll, vp]
        L.ne_attn_paged_plan.restype = i
        L.ne_attn_paged_plan_ex.argtypes = [vp] * 14 + [i] * 6 + [ll, vp]
        L.ne_attn_paged_plan_ex.restype = i
        L.ne_attn_kv_append_slots.argtypes = [vp] * 7 + [i] * 6 + [ll] * 3 + [f, f, i, vp]
        L.ne_attn_kv_append_slots.restype = i
        L.ne_attn_decode_tree_workspace_size.argtypes = [i, i, i, i, i]
        L.ne_attn_decode_tree_workspace_size.restype = sz
        L.ne_attn_decode_tree.argtypes = [vp] * 10 + [i] * 8 + [ll] * 3 + [f, f, i, vp, sz, vp]
        L.ne_attn_decode_tree.restype = i
        L.ne_attn_kv_keep_paged.argtypes = [vp] * 8 + [i] * 8 + [ll, vp]
        L.ne_attn_kv_keep_paged.restype = i
        _lib = L
    return _lib


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, st):
    if st != NE_OK:
        raise NeAttnError(fn, st)


def _ptr(t):
    return ctypes.c_void_p(None if t is None else t.data_ptr())


def _shape(q, k):
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    return B, T, Hq, Hkv, D


def fwd_workspace_size(B, T, Hq, Hkv, D, precise=False, fp8=False):
    flags = (PRECISE_QK if precise else 0) | (FP8 if fp8 else 0)
    return int(lib().ne_attn_fwd_workspace_size(B, T, Hq, Hkv, D, flags))


def attn_fwd(q, k, v, rope_base=10000.0, o=None, lse=None, o_dtype=torch.bfloat16, precise=False,
             workspace=None, rope_half=False, qk_rotated=False, Hq=None, fp8=False, stream=None):
    """o, lse = causal GQA attention of q [B,T,Hq,D], k/v [B,T,Hkv,D] (bf16, CUDA).

    o_dtype: bfloat16 or float32.  precise: hi+lo split of the rotated q, k
    for the logits (NE_ATTN_PRECISE_QK).  workspace: a uint8 CUDA tensor of at
    least fwd_workspace_size bytes (the rotated fp16 q, k land there); if None
    one is allocated for the call.  qk_rotated: `workspace` already holds the
    rotated q and k (written by qkv_rmsnorm with rotated=True); q and k may
    then be None, with the number of query heads given as Hq.  fp8: the
    e4m3 forward (NE_ATTN_FP8; D = 64, about 3e-2 relative error in o).
    """
    if qk_rotated and workspace is None:
        raise ValueError("qk_rotated needs the workspace that holds the rotated q and k")
    if q is None:
        if not qk_rotated or Hq is None:
            raise ValueError("q may be None only with qk_rotated and Hq")
        B, T, Hkv, D = v.shape
    else:
        B, T, Hq, Hkv, D = _shape(q, k)
    if o is None:
        o = torch.empty((B, T, Hq, D), dtype=o_dtype, device=v.device)
    if lse is None:
        # precise mode stores the LSE and its fp32 remainder: lse[0] is the LSE
        shape = (2, B, Hq, T) if precise else (B, Hq, T)
        lse = torch.empty(shape, dtype=torch.float32, device=v.device)
    assert lse.numel() == (2 if precise else 1) * B * Hq * T and o.shape == (B, T, Hq, D)
    for t in (q, k, v):
        assert t is None or (t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous())
    assert o.dtype in (torch.bfloat16, torch.float32) and o.is_contiguous()
    assert lse.dtype == torch.float32 and lse.is_contiguous()
    flags = ((O_FP32 if o.dtype == torch.float32 else 0) | (PRECISE_QK if precise else 0)
             | (ROPE_HALF if rope_half else 0) | (QK_ROTATED if qk_rotated else 0) | (FP8 if fp8 else 0))
    if workspace is None:
        n = fwd_workspace_size(B, T, Hq, Hkv, D, precise, fp8)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=v.device)
    assert workspace.dtype == torch.uint8 and workspace.is_cuda
    _check("ne_attn_fwd_ex", lib().ne_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                                  B, T, Hq, Hkv, D, float(rope_base), flags,
                                                  _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, lse


def bwd_workspace_size(B, T, Hq, Hkv, D, precise=False):
    return int(lib().ne_attn_bwd_workspace_size(B, T, Hq, Hkv, D, PRECISE_QK if precise else 0))


def alloc_workspace(B, T, Hq, Hkv, D, precise=False, device="cuda"):
    n = bwd_workspace_size(B, T, Hq, Hkv, D, precise)
    if n == 0:
        raise ValueError("unsupported shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def attn_bwd(q, k, v, o, lse, dout, rope_base=10000.0, grad_dtype=torch.bfloat16, precise=False,
             dq=None, dk=None, dv=None, workspace=None, qk_rotated=False, rope_half=False, stream=None):
    """dq, dk, dv of the causal GQA attention given the forward's o and lse.

    o may be bfloat16 or float32; grad_dtype selects the gradient dtype.
    qk_rotated: `workspace` was also the forward's workspace (for these q, k)
    and still holds its rotated q and k (NE_ATTN_QK_ROTATED).
    """
    if qk_rotated and workspace is None:
        raise ValueError("qk_rotated needs the workspace the forward wrote")
    if (q is None or k is None) and not qk_rotated:
        raise ValueError("q and k may be None only with qk_rotated")
    B, T, Hq, D = dout.shape
    Hkv = v.shape[2]
    if grad_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("grad_dtype must be bfloat16 or float32")
    if dq is None:
        dq = torch.empty(dout.shape, dtype=grad_dtype, device=v.device)
    if dk is None:
        dk = torch.empty(v.shape, dtype=grad_dtype, device=v.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=grad_dtype, device=v.device)
    if workspace is None:
        workspace = alloc_workspace(B, T, Hq, Hkv, D, precise, v.device)
    for t in (q, k, v, dout):
        assert t is None or (t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous())
    assert o.dtype in (torch.bfloat16, torch.float32) and o.is_contiguous()
    assert lse.dtype == torch.float32 and lse.numel() == (2 if precise else 1) * B * Hq * T
    for t in (dq, dk, dv):
        assert t.dtype == grad_dtype and t.is_contiguous()
    flags = ((O_FP32 if o.dtype == torch.float32 else 0) | (GRAD_FP32 if grad_dtype == torch.float32 else 0)
             | (PRECISE_QK if precise else 0) | (QK_ROTATED if qk_rotated else 0) | (ROPE_HALF if rope_half else 0))
    _check("ne_attn_bwd", lib().ne_attn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
        B, T, Hq, Hkv, D, float(rope_base), flags, _ptr(workspace), workspace.numel(), _stream(stream)))
    return dq, dk, dv


def check_status(stream=None):
    """Synchronises the stream; raises if a kernel reported a device-side timeout."""
    _check("ne_attn_check_status", lib().ne_attn_check_status(_stream(stream)))


def status_of_last_kernels(stream=None):
    """Like check_status but returns the raw status code (and clears it)."""
    return int(lib().ne_attn_check_status(_stream(stream)))


KERNEL_KINDS = ("fwd", "bwd_prep", "bwd_dkdv", "bwd_dq", "fwd_rope", "kv_append", "decode", "decode_aux",
                "qkv_prep", "qkv", "qk_norm", "qk_norm_bwd", "kv_append_paged", "decode_paged",
                "decode_prefix", "paged_plan", "decode_tree", "kv_keep")


def profile_start(capacity):
    """Brackets each library kernel launch with CUDA events (see ne_attn_profile_start)."""
    _check("ne_attn_profile_start", lib().ne_attn_profile_start(int(capacity)))


def profile_stop():
    """Returns {kernel kind: (total device ms, launches)} for the launches since profile_start."""
    ms = (ctypes.c_double * len(KERNEL_KINDS))()
    n = (ctypes.c_longlong * len(KERNEL_KINDS))()
    _check("ne_attn_profile_stop", lib().ne_attn_profile_stop(ms, n))
    return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(KERNEL_KINDS)}


def profile_stop_deferred():
    """Closes a profile whose launches were captured into a CUDA graph: the
    events run (and are timed) each time the graph replays.  Returns a handle
    for profile_read, which reads the times of the most recent replay."""
    _check("ne_attn_profile_detach", lib().ne_attn_profile_detach())
    return True


def profile_read(handle):
    ms = (ctypes.c_double * len(KERNEL_KINDS))()
    n = (ctypes.c_longlong * len(KERNEL_KINDS))()
    _check("ne_attn_profile_read", lib().ne_attn_profile_read(ms, n))
    return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(KERNEL_KINDS)}


def debug_timeout_probe(limit_us, stream=None):
    _check("ne_attn_debug_timeout_probe", lib().ne_attn_debug_timeout_probe(int(limit_us), _stream(stream)))


def fwd_bwd_host(q, k, v, dout, rope_base=10000.0, grad_dtype=torch.bfloat16, o_dtype=torch.bfloat16,
                 precise=False, device="cuda", stream=None):
    """End-to-end call on host (CPU) bfloat16 tensors: copies in, forward +
    backward, copies out.  Pinned host memory makes the copies asynchronous.
    Returns host tensors (o, lse, dq, dk, dv).
    """
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.stream(s):
        qd = q.to(device, non_blocking=True)
        kd = k.to(device, non_blocking=True)
        vd = v.to(device, non_blocking=True)
        dod = dout.to(device, non_blocking=True)
        ws = alloc_workspace(*_shape(qd, kd), precise=precise, device=device)
        o, lse = attn_fwd(qd, kd, vd, rope_base, o_dtype=o_dtype, precise=precise, workspace=ws, stream=s)
        dq, dk, dv = attn_bwd(qd, kd, vd, o, lse, dod, rope_base, grad_dtype, precise=precise, workspace=ws,
                              qk_rotated=not precise, stream=s)
        out = [t.to("cpu", non_blocking=False) for t in (o, lse, dq, dk, dv)]
    return tuple(out)


def kv_cache(B, Tcap, Hkv, D, device):
    """Empty head-major key (fp16, rotated) and value (bf16) caches [B, Hkv, Tcap, D]."""
    return (torch.zeros((B, Hkv, Tcap, D), dtype=torch.float16, device=device),
            torch.zeros((B, Hkv, Tcap, D), dtype=torch.bfloat16, device=device))


def kv_append(k_new, v_new, k_cache, v_cache, pos0, rope_base=10000.0, rope_half=False, stream=None):
    """Writes positions pos0 .. pos0 + Tn - 1 of the caches from k_new, v_new [B,Tn,Hkv,D] (bf16)."""
    B, Tn, Hkv, D = k_new.shape
    Tcap = k_cache.shape[2]
    for t in (k_new, v_new):
        assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous()
    assert k_cache.dtype == torch.float16 and v_cache.dtype == torch.bfloat16
    assert k_cache.is_contiguous() and v_cache.is_contiguous() and k_cache.shape == v_cache.shape
    _check("ne_attn_kv_append", lib().ne_attn_kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                                        B, Tn, pos0, Tcap, Hkv, D, float(rope_base),
                                                        ROPE_HALF if rope_half else 0, _stream(stream)))


def decode_workspace_size(B, Tq, Tkv, Hq, Hkv, D):
    return int(lib().ne_attn_decode_workspace_size(B, Tq, Tkv, Hq, Hkv, D))


def attn_decode(q, k_cache, v_cache, Tkv, rope_base=10000.0, o=None, lse=None, o_dtype=torch.bfloat16,
                workspace=None, rope_half=False, stream=None):
    """o, lse for the Tq new queries q [B,Tq,Hq,D] (bf16, positions Tkv-Tq .. Tkv-1)
    against cache positions 0 .. Tkv-1 (see ne_attn_decode)."""
    B, Tq, Hq, D = q.shape
    Hkv, Tcap = k_cache.shape[1], k_cache.shape[2]
    assert q.dtype == torch.bfloat16 and q.is_cuda and q.is_contiguous()
    assert k_cache.dtype == torch.float16 and v_cache.dtype == torch.bfloat16
    if o is None:
        o = torch.empty(q.shape, dtype=o_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device)
    assert o.dtype in (torch.bfloat16, torch.float32) and o.is_contiguous()
    assert lse.dtype == torch.float32 and lse.is_contiguous() and lse.numel() == B * Hq * Tq
    if workspace is None:
        workspace = torch.empty(max(decode_workspace_size(B, Tq, Tkv, Hq, Hkv, D), 1), dtype=torch.uint8,
                                device=q.device)
    flags = (O_FP32 if o.dtype == torch.float32 else 0) | (ROPE_HALF if rope_half else 0)
    _check("ne_attn_decode", lib().ne_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                                                  B, Tq, Tkv, Tcap, Hq, Hkv, D, float(rope_base), flags,
                                                  _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, lse


def qkv_workspace_size(B, T, C, Hq, Hkv, D, rotated=False, rope_half=False):
    flags = (QK_ROTATED if rotated else 0) | (ROPE_HALF if rope_half else 0)
    return int(lib().ne_attn_qkv_workspace_size(B, T, C, Hq, Hkv, D, flags))


def qkv_rmsnorm(x, norm_w, w_qkv, Hq, Hkv, D, eps=1e-5, rope_base=10000.0, rotated=False, rope_half=False,
                write_qk=True, q=None, k=None, v=None, rstd=None, workspace=None, stream=None):
    """RMSNorm of x [B,T,C] and the fused projection w_qkv [(Hq+2Hkv)D, C] (bf16, CUDA).

    Returns (q, k, v, rstd, workspace): q [B,T,Hq,D], k and v [B,T,Hkv,D]
    (bf16; q and k are None when write_qk is False), rstd [B,T] fp32.
    rotated: also write the rotated q, k (fp16) at the start of `workspace`
    (allocated here if None; at least qkv_workspace_size bytes), where
    attn_fwd / attn_bwd with qk_rotated=True take them.
    """
    B, T, C = x.shape
    N = (Hq + 2 * Hkv) * D
    assert norm_w.shape == (C,) and w_qkv.shape == (N, C)
    for t in (x, norm_w, w_qkv):
        assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous()
    if not write_qk and not rotated:
        raise ValueError("write_qk=False needs rotated=True")
    dev = x.device
    if write_qk:
        q = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=dev) if q is None else q
        k = torch.empty((B, T, Hkv, D), dtype=torch.bfloat16, device=dev) if k is None else k
    else:
        q = k = None
    v = torch.empty((B, T, Hkv, D), dtype=torch.bfloat16, device=dev) if v is None else v
    rstd = torch.empty((B, T), dtype=torch.float32, device=dev) if rstd is None else rstd
    for t in (q, k, v):
        assert t is None or (t.dtype == torch.bfloat16 and t.is_contiguous())
    assert rstd.dtype == torch.float32 and rstd.numel() == B * T
    if workspace is None:
        n = qkv_workspace_size(B, T, C, Hq, Hkv, D, rotated, rope_half)
        if n == 0:
            raise ValueError("unsupported shape")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    flags = (QK_ROTATED if rotated else 0) | (ROPE_HALF if rope_half else 0)
    _check("ne_attn_qkv_rmsnorm", lib().ne_attn_qkv_rmsnorm(
        _ptr(x), _ptr(norm_w), _ptr(w_qkv), _ptr(q), _ptr(k), _ptr(v), _ptr(rstd), B, T, C, Hq, Hkv, D,
        float(eps), float(rope_base), flags, _ptr(workspace), workspace.numel(), _stream(stream)))
    return q, k, v, rstd, workspace


def rotated_qk(workspace, B, T, Hq, Hkv, D):
    """Views of the rotated fp16 q [B,T,Hq,D] and k [B,T,Hkv,D] at the start of a
    forward / backward / projection workspace (NE_ATTN_QK_ROTATED layout)."""
    at = (B * T * Hq * D + 127) // 128 * 128  # each array starts on 256 bytes
    if workspace.numel() % 2:
        workspace = workspace[:-1]
    w = workspace.view(torch.float16)
    first = w.storage_offset()
    return (w.as_strided((B, T, Hq, D), (T * Hq * D, Hq * D, D, 1), first),
            w.as_strided((B, T, Hkv, D), (T * Hkv * D, Hkv * D, D, 1), first + at))


# ------------------------------------------------------------------ query/key norms, paged cache
def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on(stream, call, x, *args):
    """call(x, *args) with `stream`, of x's device, as the current stream: what it allocates then belongs to it."""
    if stream.device != x.device:
        raise ValueError("stream must be of the call's device")
    with torch.cuda.stream(stream):
        return call(x, *args)


def _call(name, device, args):
    """Status of library function `name` with `device`'s current stream as its last argument."""
    index = device.index
    # no Python around the device and the stream: a call right after a launch finds the caches cold
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call(name, device, args)
    return getattr(_lib or lib(), name)(*args, torch._C._cuda_getCurrentRawStream(index))


def _run(name, device, *args):
    st = _call(name, device, args)
    if st != NE_OK:
        raise NeAttnError(name, st)


def _optr(t):
    return None if t is None else t.data_ptr()


def _head_rows(t, name, dtype=torch.bfloat16, device=None):
    """Row stride (values between positions) of t [B, T, H, D] or [N, H, D]: heads
    contiguous, positions evenly spaced."""
    s, n = t.stride(), t.shape
    if t.dtype != dtype or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError("%s must be %s on the call's CUDA device" % (name, dtype))
    H, D = n[-2], n[-1]
    ok = s[-1] == 1 and (H == 1 or s[-2] == D)
    if len(n) == 3:
        row = s[0] if n[0] > 1 else H * D
    else:
        row = s[1] if n[1] > 1 else (s[0] if n[0] > 1 else H * D)
        ok = ok and (n[0] == 1 or n[1] == 1 or s[0] == n[1] * s[1])
    if not ok:
        raise ValueError("%s: the heads of a position must be contiguous and the positions evenly spaced" % name)
    return row


def _vector(t, D, name, device):
    if t.dtype != torch.bfloat16 or t.device != device or t.shape != (D,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous bfloat16 [%d] on the call's device" % (name, D))


def _int32(t, name, device, shape):
    if t.dtype != torch.int32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 %s on the call's device" % (name, list(shape)))


def _bytes(workspace, device):
    # its size is counted in numel(): an expanded tensor has more of those than bytes
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8 on the call's device")


def _run_ws(name, device, args, workspace, size):
    """_run with the workspace as the last arguments: the caller's; without one NULL (the
    library's own for the stream) or, where a capture needs one, a tensor of the capture's own."""
    if workspace is None:
        st = _call(name, device, args + (None, 0))
        if st == NE_OK:
            return
        if st != ERR_WORKSPACE:
            raise NeAttnError(name, st)
        workspace = torch.empty(size(), dtype=torch.uint8, device=device)
    else:
        _bytes(workspace, device)
    _run(name, device, *args, workspace.data_ptr(), workspace.numel())


def qk_norm(q, k, q_weight, k_weight, eps=1e-6, rope_base=10000.0, rope_half=False, workspace=None, stream=None):
    """RMS norm of every head of q [B,T,Hq,D] and k [B,T,Hkv,D] (bf16) with weights
    [D], then the rotary embedding, in one pass (ne_attn_qk_norm).

    q and k may be slices of a fused projection's rows.  The rotated fp16 q and k
    land at the start of `workspace` (a uint8 CUDA tensor of at least
    fwd_workspace_size bytes; one of that size is allocated if None), which is
    returned: attn_fwd takes it with qk_rotated=True (q and k then None), rotated_qk
    views it.  attn_bwd needs more room: for training give alloc_workspace's, which
    attn_fwd and attn_bwd then both take with qk_rotated=True.
    """
    if stream is not None:
        return _on(stream, qk_norm, q, k, q_weight, k_weight, eps, rope_base, rope_half, workspace)
    B, T, Hq, D = q.shape
    Hkv, dev = k.shape[2], q.device
    _need(k.shape == (B, T, Hkv, D), "k must be [B, T, Hkv, D] like q")
    qs, ks = _head_rows(q, "q"), _head_rows(k, "k", device=dev)
    _vector(q_weight, D, "q_weight", dev)
    _vector(k_weight, D, "k_weight", dev)
    if workspace is None:
        n = (B * T * Hq * D + 127) // 128 * 256 + (B * T * Hkv * D + 127) // 128 * 256  # as rotated_qk
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        _bytes(workspace, dev)
        n = workspace.numel()
    _run("ne_attn_qk_norm", dev, q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(),
         B, T, Hq, Hkv, D, qs, ks, eps, rope_base, ROPE_HALF if rope_half else 0, workspace.data_ptr(), n)
    return workspace


def qk_norm_bwd(q, k, q_weight, k_weight, dqn, dkn, eps=1e-6, dq=None, dk=None, workspace=None, stream=None):
    """Backward of qk_norm: dq, dk (the type of dqn and dkn), dq_weight, dk_weight (fp32 [D])
    from dqn [B,T,Hq,D] and dkn [B,T,Hkv,D], the dq and dk of attn_bwd with qk_rotated=True
    (bf16 or fp32, contiguous).  dq and dk may be given: slices of a fused projection's
    gradient, or dqn and dkn themselves."""
    if stream is not None:
        return _on(stream, qk_norm_bwd, q, k, q_weight, k_weight, dqn, dkn, eps, dq, dk, workspace)
    B, T, Hq, D = q.shape
    Hkv, dev, dt = k.shape[2], q.device, dqn.dtype
    _need(k.shape == (B, T, Hkv, D), "k must be [B, T, Hkv, D] like q")
    _need(dt in (torch.bfloat16, torch.float32), "dqn and dkn must be bfloat16 or float32")
    qs, ks = _head_rows(q, "q"), _head_rows(k, "k", device=dev)
    _vector(q_weight, D, "q_weight", dev)
    _vector(k_weight, D, "k_weight", dev)
    for t, like, name in ((dqn, q, "dqn"), (dkn, k, "dkn")):
        _need(t.dtype == dt and t.device == dev and t.shape == like.shape and t.is_contiguous(),
              "%s must be contiguous, of the shape of its input and of one type with the other" % name)
    if dq is None:
        dq, dqs = torch.empty(q.shape, dtype=dt, device=dev), Hq * D
    else:
        _need(dq.shape == q.shape, "dq must have the shape of q")
        dqs = _head_rows(dq, "dq", dt, dev)
    if dk is None:
        dk, dks = torch.empty(k.shape, dtype=dt, device=dev), Hkv * D
    else:
        _need(dk.shape == k.shape, "dk must have the shape of k")
        dks = _head_rows(dk, "dk", dt, dev)
    dqw = torch.empty(D, dtype=torch.float32, device=dev)
    dkw = torch.empty(D, dtype=torch.float32, device=dev)
    args = (q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(), dqn.data_ptr(), dkn.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dqw.data_ptr(), dkw.data_ptr(), B, T, Hq, Hkv, D, qs, ks, dqs, dks, eps,
            GRAD_FP32 if dt == torch.float32 else 0)
    _run_ws("ne_attn_qk_norm_bwd", dev, args, workspace,
            lambda: int(lib().ne_attn_qk_norm_bwd_workspace_size(B, T, Hq, Hkv, D)))
    return dq, dk, dqw, dkw


def paged_cache(num_pages, page_size, Hkv, D, device):
    """Empty page pools [num_pages, Hkv, page_size, D]: rotated keys (fp16) and values (bf16)."""
    shape = (num_pages, Hkv, page_size, D)
    return (torch.zeros(shape, dtype=torch.float16, device=device),
            torch.zeros(shape, dtype=torch.bfloat16, device=device))


def _pools(k_pages, v_pages, Hkv, D, device):
    """(number of pages, page size, page stride) of the two pools."""
    shape = k_pages.shape
    P, H, page, d = shape
    if v_pages.shape != shape or H != Hkv or d != D:
        raise ValueError("pools must be [num_pages, Hkv, page_size, D]")
    if (k_pages.dtype != torch.float16 or v_pages.dtype != torch.bfloat16 or k_pages.device != device
            or v_pages.device != device):
        raise ValueError("pools must be float16 keys and bfloat16 values on the call's CUDA device")
    sk, sv = k_pages.stride(), v_pages.stride()
    stride = sk[0] if P > 1 else H * page * D
    inner = (page * D, D, 1)
    if sk[1:] != inner or sv != sk:
        # strides of dimensions of one do not matter
        for t in (sk, sv):
            if t[3] != 1 or t[2] != D or (H > 1 and t[1] != page * D) or (P > 1 and t[0] != stride):
                raise ValueError("pools must be contiguous inside a page and have one page stride")
    return P, page, stride


def kv_append_paged(k_new, v_new, k_pages, v_pages, page_table, pos0, cu_new=None, k_weight=None, eps=1e-6,
                    rope_base=10000.0, rope_half=False, stream=None):
    """Writes new keys and values [N,Hkv,D] (bf16, rows may be strided) into a paged cache
    (ne_attn_kv_append_paged).

    page_table int32 [B, max_pages], pos0 int32 [B] (the first new position of each
    sequence) and cu_new int32 [B + 1] (its rows; None: N / B each) are CUDA tensors.
    k_weight [D]: the keys are normalised first.  Bad pages are found by check_status."""
    if stream is not None:
        return _on(stream, kv_append_paged, k_new, v_new, k_pages, v_pages, page_table, pos0, cu_new, k_weight, eps,
                   rope_base, rope_half)
    N, Hkv, D = k_new.shape
    dev = k_new.device
    _need(v_new.shape == k_new.shape, "k_new and v_new must have one shape")
    ks, vs = _head_rows(k_new, "k_new"), _head_rows(v_new, "v_new", device=dev)
    P, page, stride = _pools(k_pages, v_pages, Hkv, D, dev)
    B, width = page_table.shape
    _int32(page_table, "page_table", dev, (B, width))
    _int32(pos0, "pos0", dev, (B,))
    if cu_new is not None:
        _int32(cu_new, "cu_new", dev, (B + 1,))
    if k_weight is not None:
        _vector(k_weight, D, "k_weight", dev)
    if N == 0:
        return
    _run("ne_attn_kv_append_paged", dev, k_new.data_ptr(), v_new.data_ptr(), _optr(k_weight),
         k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), pos0.data_ptr(), _optr(cu_new), N, B, Hkv, D,
         page, P, width, stride, ks, vs, eps, rope_base, ROPE_HALF if rope_half else 0)


def decode_paged_workspace_size(B, Tq, Hq, Hkv, D, prefix_len=0):
    return int(lib().ne_attn_decode_paged_workspace_size(B, Tq, Hq, Hkv, D, prefix_len))


def _outputs(o, lse, o_dtype, B, Tq, Hq, D, dev):
    if o is None:
        o = torch.empty((B, Tq, Hq, D), dtype=o_dtype, device=dev)
    elif o.device != dev or not o.is_contiguous() or o.shape != (B, Tq, Hq, D):
        raise ValueError("o must be a contiguous [B, Tq, Hq, D] on the call's device")
    else:
        o_dtype = o.dtype
    if lse is None:
        lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=dev)
    elif lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous() or lse.shape != (B, Hq, Tq):
        raise ValueError("lse must be a contiguous float32 [B, Hq, Tq] on the call's device")
    fp32 = o_dtype == torch.float32
    if not fp32 and o_dtype != torch.bfloat16:
        raise ValueError("o must be bfloat16 or float32")
    return o, lse, fp32


def attn_decode_paged(q, k_pages, v_pages, page_table, kv_len, q_weight=None, eps=1e-6, rope_base=10000.0,
                      prefix_table=None, prefix_len=0, o=None, lse=None, o_dtype=torch.bfloat16, workspace=None,
                      rope_half=False, stream=None):
    """o, lse for the newest Tq tokens q [B,Tq,Hq,D] (bf16) of every sequence over a paged
    cache (ne_attn_decode_paged).

    kv_len int32 [B] counts the cached positions, the new tokens' own included (0: an
    idle slot, whose o is 0 and lse -inf).  q_weight [D]: the queries are normalised
    first.  prefix_table int32 and prefix_len: the first prefix_len positions (whole
    pages) of every sequence are these pages, read once for the batch."""
    if stream is not None:
        return _on(stream, attn_decode_paged, q, k_pages, v_pages, page_table, kv_len, q_weight, eps, rope_base,
                   prefix_table, prefix_len, o, lse, o_dtype, workspace, rope_half)
    B, Tq, Hq, D = q.shape
    Hkv, dev = k_pages.shape[1], q.device
    qs = _head_rows(q, "q")
    P, page, stride = _pools(k_pages, v_pages, Hkv, D, dev)
    width = page_table.shape[1]
    _int32(page_table, "page_table", dev, (B, width))
    _int32(kv_len, "kv_len", dev, (B,))
    if q_weight is not None:
        _vector(q_weight, D, "q_weight", dev)
    if prefix_len:
        _need(prefix_table is not None and prefix_table.dim() == 1 and prefix_table.numel() * page >= prefix_len,
              "prefix_table must hold the pages of prefix_len positions")
        _int32(prefix_table, "prefix_table", dev, prefix_table.shape)
    o, lse, fp32 = _outputs(o, lse, o_dtype, B, Tq, Hq, D, dev)
    args = (q.data_ptr(), None if q_weight is None else q_weight.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
            page_table.data_ptr(), kv_len.data_ptr(), prefix_table.data_ptr() if prefix_len else None, o.data_ptr(),
            lse.data_ptr(), B, Tq, Hq, Hkv, D, page, P, width, stride, qs, prefix_len, eps, rope_base,
            (O_FP32 if fp32 else 0) | (ROPE_HALF if rope_half else 0))
    _run_ws("ne_attn_decode_paged", dev, args, workspace,
            lambda: decode_paged_workspace_size(B, Tq, Hq, Hkv, D, prefix_len))
    return o, lse


# ------------------------------------------------------------------ drafted trees over the paged cache
class PagedPlan(collections.namedtuple("PagedPlan", "kv_len held span cu_new slots positions")):
    """What paged_plan returns.  new_len [B], the positions that each sequence was granted, is an attribute beside the tuple."""
    new_len = None


_bind = None
BIND_PATH = bind_path()  # for this interpreter and this torch


def _compiled():
    """The compiled part of the binding (csrc/bind.cpp), which has the library's entry points from here."""
    global _bind
    if _bind is None:
        L = lib()
        if not os.path.exists(BIND_PATH):
            raise RuntimeError("the compiled part of the binding is not built (%s); run __graft_entry__.build()" % BIND_PATH)
        spec = importlib.util.spec_from_file_location("_neattn_bind", BIND_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        names = ("ne_attn_paged_plan_ex", "ne_attn_kv_append_slots", "ne_attn_decode_tree",
                 "ne_attn_decode_tree_workspace_size", "ne_attn_kv_keep_paged")
        m.init(dict({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names},
                    OutOfMemoryError=torch.OutOfMemoryError))
        _bind = m
    return _bind


def paged_plan(page_table, free_pages, held, free_span, kv_len, new_len, rows, page_size, parents=None, kv_len_out=None,
               held_out=None, span_out=None, stream=None, new_len_out=None):
    """Block tables and slot maps from lengths, on the device (ne_attn_paged_plan).

    Sequence b has kv_len[b] positions, holds the first held[b] pages of its row of page_table [B, max_pages] and
    is to have new_len[b] more; free_pages [num_pages] is a ring whose entries free_span = (first, count) are free.
    All are int32 CUDA tensors; page_table and free_pages are changed in place.  rows: how many new rows the
    call maps, those past the sum of new_len being padding.  parents [B, Tq] or [Tq]: the new tokens are trees.

    Returns PagedPlan(kv_len [B], held [B], span [2], cu_new [B + 1], slots [rows], positions [rows]): the new
    lengths and pages held (a sequence whose pages the ring no longer has keeps its old ones), where each
    sequence's rows begin, and the place (-1: none) and rotary position of every row for kv_append_slots.  Its new_len
    [B] is what each sequence was granted, 0 where refused: the tree_len of attn_decode_tree and kv_keep_paged.
    held_out, span_out and new_len_out may be held, free_span and new_len themselves; kv_len_out may not lie on kv_len,
    the table, the ring or parents."""
    if stream is not None:
        return _on(stream, paged_plan, page_table, free_pages, held, free_span, kv_len, new_len, rows, page_size, parents,
                   kv_len_out, held_out, span_out, None, new_len_out)
    r = (_bind or _compiled()).plan(page_table, free_pages, held, free_span, kv_len, new_len, rows, page_size, parents, kv_len_out,
                                    held_out, span_out, new_len_out)
    if type(r) is int:
        raise NeAttnError("ne_attn_paged_plan", r)
    p = PagedPlan._make(r[:6])
    p.new_len = r[6]
    return p


def kv_append_slots(k_new, v_new, k_pages, v_pages, slots, positions, capacity, k_weight=None, eps=1e-6,
                    rope_base=10000.0, rope_half=False, stream=None):
    """Writes new keys and values [N,Hkv,D] (bf16, rows may be strided) to given places of a paged cache
    (ne_attn_kv_append_slots): row n to slot slots[n] (int32 [N], negative: nowhere), its key normalised with k_weight
    [D] unless None and rotated at positions[n] (int32 [N], below `capacity`).  paged_plan gives both.
    Bad slots and positions are found by check_status."""
    if stream is not None:
        return _on(stream, kv_append_slots, k_new, v_new, k_pages, v_pages, slots, positions, capacity, k_weight, eps,
                   rope_base, rope_half)
    st = (_bind or _compiled()).append(k_new, v_new, k_pages, v_pages, slots, positions, capacity, k_weight, eps, rope_base, rope_half)
    if st != NE_OK:
        raise NeAttnError("ne_attn_kv_append_slots", st)


def decode_tree_workspace_size(B, Tq, Hq, Hkv, D):
    return int(lib().ne_attn_decode_tree_workspace_size(B, Tq, Hq, Hkv, D))


def attn_decode_tree(q, k_pages, v_pages, page_table, kv_len, parents, tree_len=None, q_weight=None, eps=1e-6,
                     rope_base=10000.0, o=None, lse=None, o_dtype=torch.bfloat16, workspace=None, rope_half=False,
                     stream=None):
    """o, lse for a tree of drafted tokens q [B,Tq,Hq,D] (bf16) of every sequence over a paged cache
    (ne_attn_decode_tree).

    kv_len int32 [B] counts the cached positions, the tree's tree_len[b] own included (int32 [B]; None: Tq; after a plan
    what it granted, new_len, as a refused sequence has no tree at its end).  parents
    int32 [B, Tq] or [Tq] (one tree for all): the token each hangs on, -1 for the context.  A token sees the
    positions before the tree, its ancestors and itself; tokens past tree_len, and idle slots (kv_len 0), get o = 0
    and lse = -inf.  q_weight [D]: the queries are normalised first."""
    if stream is not None:
        return _on(stream, attn_decode_tree, q, k_pages, v_pages, page_table, kv_len, parents, tree_len, q_weight, eps,
                   rope_base, o, lse, o_dtype, workspace, rope_half)
    if o_dtype is not torch.bfloat16 and o_dtype is not torch.float32 and o is None:
        raise ValueError("o must be bfloat16 or float32")
    r = (_bind or _compiled()).decode_tree(q, k_pages, v_pages, page_table, kv_len, parents, tree_len, q_weight, eps, rope_base, o, lse,
                                           o_dtype is torch.float32, workspace, rope_half)
    if type(r) is int:
        raise NeAttnError("ne_attn_decode_tree", r)
    return r


def kv_keep_paged(k_pages, v_pages, page_table, kv_len, tree_len, path, path_len, kv_len_out=None, stream=None):
    """Keeps the accepted path of every sequence's tree (ne_attn_kv_keep_paged): the keys and values of its tokens
    path[b, :path_len[b]] (int32 [B, width] and [B], rising) move to the positions right behind the context, in place.

    kv_len int32 [B] counts the cached positions, the tree's tree_len (int32 [B], or one number for all) included; one of 0
    keeps nothing and its length, whatever its path holds;
    returns the new lengths (kv_len_out if given, which may lie on none of the tensors read).  The pools of several layers with one
    table may be passed as one [num_pages, layers * Hkv, page_size, D]."""
    if stream is not None:
        return _on(stream, kv_keep_paged, k_pages, v_pages, page_table, kv_len, tree_len, path, path_len, kv_len_out)
    r = (_bind or _compiled()).keep(k_pages, v_pages, page_table, kv_len, tree_len, path, path_len, kv_len_out)
    if type(r) is int:
        raise NeAttnError("ne_attn_kv_keep_paged", r)
    return r


class HostStepPipeline:
    """Forward + backward steps on host tensors, with the copies of one step
    overlapping the compute of the others.

    Inputs go up on one stream, the library's kernels run on a second, results
    come down on a third; `depth` device buffer sets rotate, and CUDA events
    order each set's reuse (a set is refilled only after its previous results
    have come down).  Host tensors should be pinned so the copies run
    asynchronously.  submit() only enqueues work; synchronize() waits for all
    of it and raises if a kernel reported a device-side timeout.  precise:
    split precision (NE_ATTN_PRECISE_QK) with an fp32 o, for inputs with very
    large logits; lse then holds the LSE and its remainder ([2 B, Hq, T]).
    """

    def __init__(self, B, T, Hq, Hkv, D, rope_base=10000.0, depth=3, grad_dtype=torch.float32,
                 o_dtype=torch.bfloat16, device="cuda", precise=False):
        self.shape = (B, T, Hq, Hkv, D)
        self.rope_base = float(rope_base)
        self.grad_dtype = grad_dtype
        self.precise = bool(precise)
        if self.precise:
            o_dtype = torch.float32
        self.device = torch.device(device)
        self.up = torch.cuda.Stream(self.device)
        self.comp = torch.cuda.Stream(self.device)
        self.down = torch.cuda.Stream(self.device)
        self.sets = []
        for _ in range(depth):
            def bf(h):
                return torch.empty((B, T, h, D), dtype=torch.bfloat16, device=self.device)
            self.sets.append(dict(
                q=bf(Hq), k=bf(Hkv), v=bf(Hkv), do=bf(Hq),
                o=torch.empty((B, T, Hq, D), dtype=o_dtype, device=self.device),
                lse=torch.empty(((2 if self.precise else 1) * B, Hq, T), dtype=torch.float32, device=self.device),
                dq=torch.empty((B, T, Hq, D), dtype=grad_dtype, device=self.device),
                dk=torch.empty((B, T, Hkv, D), dtype=grad_dtype, device=self.device),
                dv=torch.empty((B, T, Hkv, D), dtype=grad_dtype, device=self.device),
                ws=alloc_workspace(B, T, Hq, Hkv, D, precise=self.precise, device=self.device),
                up_done=torch.cuda.Event(), comp_done=torch.cuda.Event(), down_done=torch.cuda.Event(),
                used=False))
        self.n = 0

    def submit(self, q, k, v, dout, out):
        """Enqueue one step: q, k, v, dout are host bf16 tensors; `out` maps
        o, lse, dq, dk, dv to host tensors that receive the results."""
        s = self.sets[self.n % len(self.sets)]
        self.n += 1
        if s["used"]:
            self.up.wait_event(s["down_done"])  # the set's last results have come down
        with torch.cuda.stream(self.up):
            for name, src in (("q", q), ("k", k), ("v", v), ("do", dout)):
                s[name].copy_(src, non_blocking=True)
            s["up_done"].record(self.up)
        self.comp.wait_event(s["up_done"])
        attn_fwd(s["q"], s["k"], s["v"], self.rope_base, o=s["o"], lse=s["lse"], workspace=s["ws"],
                 o_dtype=s["o"].dtype, precise=self.precise, stream=self.comp)
        attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], self.rope_base, grad_dtype=self.grad_dtype,
                 dq=s["dq"], dk=s["dk"], dv=s["dv"], workspace=s["ws"], qk_rotated=not self.precise,
                 precise=self.precise, stream=self.comp)
        s["comp_done"].record(self.comp)
        self.down.wait_event(s["comp_done"])
        with torch.cuda.stream(self.down):
            for name in ("o", "lse", "dq", "dk", "dv"):
                out[name].copy_(s[name], non_blocking=True)
            s["down_done"].record(self.down)
        s["used"] = True

    def synchronize(self):
        self.down.synchronize()
        check_status(self.comp)


def fwd_schedule(B, Hkv, G, nt, nsm):
    """The persistent forward's work items per CTA (host computation, no GPU):
    a list of `grid` lists of items (b, (h0, i0), (h1, i1) or None), each CTA's
    items in the order it runs them."""
    k, grid = ctypes.c_int(0), ctypes.c_int(0)
    lib().ne_attn_debug_fwd_schedule(B, Hkv, G, nt, nsm, None, 0, ctypes.byref(grid), ctypes.byref(k))
    n = max(1, 4 * grid.value * k.value)
    buf = (ctypes.c_int * n)()
    _check("ne_attn_debug_fwd_schedule",
           lib().ne_attn_debug_fwd_schedule(B, Hkv, G, nt, nsm, buf, n, ctypes.byref(grid), ctypes.byref(k)))
    out = []
    for c in range(grid.value):
        row = []
        for j in range(k.value):
            b, hh, i0, i1 = buf[4 * (c * k.value + j):4 * (c * k.value + j) + 4]
            if b < 0:
                continue
            h0, h1 = hh & 0xFFFF, (hh >> 16) - 1
            row.append((b, (h0, i0), (h1, i1) if h1 >= 0 else None))
        out.append(row)
    return out
