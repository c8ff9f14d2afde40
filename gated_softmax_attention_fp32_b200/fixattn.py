"""Python binding of libfixattn.so (include/fix_attn.h): argument marshalling only.

Every step of FiX attention runs in the library's CUDA kernels; this module
allocates the output tensors and the workspace with PyTorch, passes raw device
pointers and the current CUDA stream through ctypes, and turns status codes
into exceptions.  There is no fallback: if the library is missing or the
device is not a B200 (sm_100), calls raise.

Names mirror the C ABI: ``fix_attn_fwd``, ``fix_attn_bwd``,
``fix_attn_workspace_bytes``, ``fix_attn_device_status``; ``fix_attn`` wraps
the pair in a ``torch.autograd.Function`` with the FiX README's argument order
("Quick Start": q, k, v, g, then cu_seqlens / o_norm_weight).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

__all__ = ["load", "Problem", "fix_attn_fwd", "fix_attn_bwd", "fix_attn_workspace_bytes",
           "fix_attn_decode", "fix_attn_rotary", "fix_rotary", "fix_attn_append_paged",
           "fix_attn_decode_paged", "fix_attn_decode_paged_workspace",
           "fix_attn_device_status", "fix_attn", "training_workspace", "FixStatusError", "LIB_PATH",
           "EXPORTS"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfixattn.so")
EXPORTS = ("fix_attn_workspace_bytes", "fix_attn_fwd", "fix_attn_bwd", "fix_attn_device_status",
           "fix_attn_kernel_count", "fix_attn_status_string", "fix_attn_fwd_noalloc",
           "fix_attn_noalloc_device_status", "fix_attn_decode_workspace_bytes",
           "fix_attn_decode", "fix_attn_rotary", "fix_attn_append_paged",
           "fix_attn_decode_paged_workspace_bytes", "fix_attn_decode_paged")
FIX_ERR_PAGE = 12
NOALLOC_MAX_WORKSPACE_BYTES = 16 * 1024 * 1024
FIX_FLAG_REUSE_FWD_WORKSPACE = 1
FIX_FLAG_NO_NORM = 2
FIX_FLAG_SCALAR_GATE = 4
STAGES = ("fwd_prefix", "fwd_attn", "bwd_prefix", "bwd_pre", "bwd_dq", "bwd_dkv", "bwd_dg",
          "bwd_finish")

ALGOS = {"auto": 0, "simt": 1, "tc": 2}
_lib = None


class Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim_k", ctypes.c_int32), ("head_dim_v", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("algo", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("events", ctypes.c_void_p)]


class Rotation(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class PageCache(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("k_pages", ctypes.c_void_p),
                ("v_pages", ctypes.c_void_p), ("g_pages", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class FixStatusError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (code {code})")


def load():
    """Load libfixattn.so (once).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"FiX CUDA library not built: {LIB_PATH} is missing "
                           "(run python -m gated_softmax_attention_fp32_b200.build)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(Problem)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.fix_attn_workspace_bytes.argtypes = [P, ctypes.c_int]
    lib.fix_attn_workspace_bytes.restype = sz
    lib.fix_attn_fwd.argtypes = [P] + [vp] * 11 + [sz, vp]
    lib.fix_attn_fwd.restype = ctypes.c_int
    lib.fix_attn_bwd.argtypes = [P] + [vp] * 17 + [sz, vp]
    lib.fix_attn_bwd.restype = ctypes.c_int
    lib.fix_attn_fwd_noalloc.argtypes = [P] + [vp] * 10 + [vp]
    lib.fix_attn_fwd_noalloc.restype = ctypes.c_int
    lib.fix_attn_device_status.argtypes = [vp, vp]
    lib.fix_attn_device_status.restype = ctypes.c_int
    lib.fix_attn_noalloc_device_status.argtypes = [vp]
    lib.fix_attn_noalloc_device_status.restype = ctypes.c_int
    lib.fix_attn_decode_workspace_bytes.argtypes = [P]
    lib.fix_attn_decode_workspace_bytes.restype = sz
    lib.fix_attn_decode.argtypes = [P] + [vp] * 9 + [sz, vp]
    lib.fix_attn_decode.restype = ctypes.c_int
    i64 = ctypes.c_int64
    R, C = ctypes.POINTER(Rotation), ctypes.POINTER(PageCache)
    lib.fix_attn_rotary.argtypes = [P, R, vp, vp, i64, vp, i64, vp, vp, ctypes.c_int, vp]
    lib.fix_attn_rotary.restype = ctypes.c_int
    lib.fix_attn_append_paged.argtypes = [P, C, R] + [vp, i64] * 4 + [vp, vp, vp]
    lib.fix_attn_append_paged.restype = ctypes.c_int
    lib.fix_attn_decode_paged_workspace_bytes.argtypes = [P, C]
    lib.fix_attn_decode_paged_workspace_bytes.restype = sz
    lib.fix_attn_decode_paged.argtypes = [P, C] + [vp] * 5 + [sz, vp]
    lib.fix_attn_decode_paged.restype = ctypes.c_int
    lib.fix_attn_kernel_count.argtypes = [P, ctypes.c_int]
    lib.fix_attn_kernel_count.restype = ctypes.c_int
    lib.fix_attn_status_string.argtypes = [ctypes.c_int]
    lib.fix_attn_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().fix_attn_status_string(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_problem(q, k, v, cu_seqlens=None, cu_seqlens_host=None, scale=None, eps=1e-6,
                 y_dtype=torch.bfloat16, algo="auto", events=None, o_norm=True,
                 scalar_gate=False):
    """Build the C problem descriptor from [B,T,H,D] tensors.  Returns
    (Problem, keepalive) where keepalive holds the host cu_seqlens tensor and
    the event-handle array.  ``events``: optional list of 2*len(STAGES)
    ``torch.cuda.Event(enable_timing=True)`` recorded around each stage.
    ``o_norm=False`` sets FIX_FLAG_NO_NORM, ``scalar_gate`` (g of shape
    [B,T,Hkv]) FIX_FLAG_SCALAR_GATE."""
    B, T, Hq, Dk = q.shape
    Hkv, Dv = v.shape[2], v.shape[3]
    p = Problem()
    p.batch, p.seqlen, p.num_q_heads, p.num_kv_heads = B, T, Hq, Hkv
    p.head_dim_k, p.head_dim_v = Dk, Dv
    p.y_dtype = 1 if y_dtype == torch.float32 else 0
    p.algo = ALGOS[algo]
    p.flags = (0 if o_norm else FIX_FLAG_NO_NORM) | (FIX_FLAG_SCALAR_GATE if scalar_gate else 0)
    p.scale = float(scale) if scale is not None else 0.0
    p.eps = float(eps)
    keep = None
    if cu_seqlens is not None:
        if cu_seqlens_host is None:
            cu_seqlens_host = cu_seqlens.detach().to("cpu")
        keep = cu_seqlens_host.to(torch.int64).contiguous()
        p.num_seqs = keep.numel() - 1
        p.cu_seqlens = cu_seqlens.data_ptr()
        p.cu_seqlens_host = keep.data_ptr()
    else:
        p.num_seqs = 0
    if events is not None:
        assert len(events) == 2 * len(STAGES)
        arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
        p.events = ctypes.cast(arr, ctypes.c_void_p)
        keep = (keep, arr)
    return p, keep


def fix_attn_workspace_bytes(problem: Problem, backward: bool) -> int:
    return int(load().fix_attn_workspace_bytes(ctypes.byref(problem), int(bool(backward))))


def fix_attn_kernel_count(problem: Problem, backward: bool) -> int:
    return int(load().fix_attn_kernel_count(ctypes.byref(problem), int(bool(backward))))


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def fix_attn_fwd(q, k, v, g, o_norm_weight, cu_seqlens=None, cu_seqlens_host=None, scale=None,
                 eps=1e-6, y_dtype=torch.bfloat16, save=True, algo="auto", workspace=None,
                 out=None, stream=None, events=None, o_gate=None, o_norm=True):
    """Forward.  Returns (y, saved) with saved = (o, m, rstd) or None.  g of
    shape [B,T,Hkv] is a scalar gate; ``o_gate`` [B,T,Hq,Dv] bf16 gates the
    output with swish; ``o_norm=False`` drops the RMSNorm (o_norm_weight may
    then be None)."""
    lib = load()
    p, keep = make_problem(q, k, v, cu_seqlens, cu_seqlens_host, scale, eps, y_dtype, algo,
                           events, o_norm, g.dim() == 3)
    B, T, Hq, _ = q.shape
    Dv = v.shape[3]
    dev = q.device
    y = out if out is not None else torch.empty(B, T, Hq, Dv, device=dev, dtype=y_dtype)
    saved = None
    if save:
        saved = (torch.empty(B, T, Hq, Dv, device=dev, dtype=torch.float32),
                 torch.empty(B, T, Hq, device=dev, dtype=torch.float32),
                 torch.empty(B, T, Hq, device=dev, dtype=torch.float32))
    nbytes = fix_attn_workspace_bytes(p, False)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), device=dev, dtype=torch.uint8)
    s = lib.fix_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o_norm_weight),
                         _ptr(o_gate), _ptr(y),
                         *(map(_ptr, saved) if saved else (None, None, None)),
                         _ptr(workspace), workspace.numel(), _stream(stream))
    if s != 0:
        raise FixStatusError(s, "fix_attn_fwd")
    del keep
    return y, saved


def fix_attn_fwd_noalloc(q, k, v, g, o_norm_weight, y, saved, cu_seqlens=None,
                         cu_seqlens_host=None, scale=None, eps=1e-6, algo="auto", stream=None,
                         o_gate=None, o_norm=True):
    """Forward into caller-provided ``y`` and ``saved`` = (o, m, rstd) or None,
    with the library's own fixed device workspace (no allocation by anyone)."""
    lib = load()
    p, keep = make_problem(q, k, v, cu_seqlens, cu_seqlens_host, scale, eps, y.dtype, algo,
                           None, o_norm, g.dim() == 3)
    s = lib.fix_attn_fwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(o_norm_weight), _ptr(o_gate), _ptr(y),
                                 *(map(_ptr, saved) if saved else (None, None, None)),
                                 _stream(stream))
    if s != 0:
        raise FixStatusError(s, "fix_attn_fwd_noalloc")
    del keep
    return y, saved


def fix_attn_bwd(q, k, v, g, o_norm_weight, dy, saved, cu_seqlens=None, cu_seqlens_host=None,
                 scale=None, eps=1e-6, algo="auto", workspace=None, stream=None, events=None,
                 out=None, reuse_forward_workspace=False, o_gate=None, o_norm=True):
    """Backward of sum(dy * y).  Returns dq, dk, dv, dg, dw, d_o_gate (the last
    None without an output gate; dw None without the norm and no ``out``)
    (``out`` may supply those six tensors).  ``reuse_forward_workspace``:
    ``workspace`` is the one the matching training forward used (sized for the
    backward, see ``training_workspace``) and has not been written since; the
    backward then reuses the forward's gate prefix results
    (FIX_FLAG_REUSE_FWD_WORKSPACE)."""
    lib = load()
    p, keep = make_problem(q, k, v, cu_seqlens, cu_seqlens_host, scale, eps, torch.bfloat16, algo,
                           events, o_norm, g.dim() == 3)
    if reuse_forward_workspace:
        if workspace is None:
            raise ValueError("reuse_forward_workspace needs the forward's workspace")
        p.flags |= FIX_FLAG_REUSE_FWD_WORKSPACE
    if out is not None:
        dq, dk, dv, dg, dw = out[:5]
        dz = out[5] if len(out) > 5 else None
    else:
        dq = torch.empty_like(q)
        dk = torch.empty_like(k)
        dv = torch.empty_like(v)
        dg = torch.empty_like(g)
        dw = torch.empty_like(o_norm_weight) if o_norm_weight is not None else None
        dz = None
    if o_gate is not None and dz is None:
        dz = torch.empty_like(o_gate)
    nbytes = fix_attn_workspace_bytes(p, True)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), device=q.device, dtype=torch.uint8)
    o_s, m_s, r_s = saved
    s = lib.fix_attn_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o_norm_weight),
                         _ptr(o_gate), _ptr(dy), _ptr(o_s), _ptr(m_s), _ptr(r_s), _ptr(dq),
                         _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dw), _ptr(dz), _ptr(workspace),
                         workspace.numel(), _stream(stream))
    if s != 0:
        raise FixStatusError(s, "fix_attn_bwd")
    del keep
    return dq, dk, dv, dg, dw, dz


def training_workspace(q, k, v, cu_seqlens=None, cu_seqlens_host=None, algo="auto", g=None,
                       o_norm=True):
    """A workspace sized for the backward, to pass to a training forward and
    then to its backward with ``reuse_forward_workspace=True``."""
    p, keep = make_problem(q, k, v, cu_seqlens, cu_seqlens_host, None, 1e-6, torch.bfloat16, algo,
                           None, o_norm, g is not None and g.dim() == 3)
    n = fix_attn_workspace_bytes(p, True)
    del keep
    return torch.empty(max(n, 1), device=q.device, dtype=torch.uint8)


def fix_attn_decode(q, k_cache, v_cache, g_cache, seqlens, o_norm_weight=None, scale=None,
                    eps=1e-6, y_dtype=torch.bfloat16, o_gate=None, o_norm=True, workspace=None,
                    out=None, stream=None):
    """One new query per sequence against its cache.  q [B,Hq,Dk];
    k_cache [B,Tmax,Hkv,Dk], v_cache [B,Tmax,Hkv,Dv] bf16; g_cache
    [B,Tmax,Hkv,Dv] (or [B,Tmax,Hkv]) f32; seqlens int32 [B] on the device
    (tokens per cache, the new one included).  Returns y [B,Hq,Dv]."""
    lib = load()
    B, Hq, Dk = q.shape
    Tmax, Hkv, Dv = v_cache.shape[1], v_cache.shape[2], v_cache.shape[3]
    p = Problem()
    p.batch, p.seqlen, p.num_q_heads, p.num_kv_heads = B, Tmax, Hq, Hkv
    p.head_dim_k, p.head_dim_v = Dk, Dv
    p.y_dtype = 1 if y_dtype == torch.float32 else 0
    p.flags = (0 if o_norm else FIX_FLAG_NO_NORM) | (FIX_FLAG_SCALAR_GATE if g_cache.dim() == 3 else 0)
    p.scale = float(scale) if scale is not None else 0.0
    p.eps = float(eps)
    y = out if out is not None else torch.empty(B, Hq, Dv, device=q.device, dtype=y_dtype)
    nbytes = int(lib.fix_attn_decode_workspace_bytes(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), device=q.device, dtype=torch.uint8)
    s = lib.fix_attn_decode(ctypes.byref(p), _ptr(seqlens), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                            _ptr(g_cache), _ptr(o_norm_weight), _ptr(o_gate), _ptr(y),
                            _ptr(workspace), workspace.numel(), _stream(stream))
    if s != 0:
        raise FixStatusError(s, "fix_attn_decode")
    return y


# The checks below run on every call of a decode step, whose kernels take a
# few microseconds: they ask a tensor for no more than they need (dtype and
# device index by identity and number, not torch.device objects).
_Tensor = torch.Tensor
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
# (absent where torch was built without CUDA: the package imports there, and
# every call refuses its tensors before it needs these)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _bad_tensor(name, t, dtype, index):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _tensor(name, t, dtype, index):
    """A tensor argument of the right type on the call's GPU."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index:
        _bad_tensor(name, t, dtype, index)


def _dense(name, t, dtype, index, shape):
    _tensor(name, t, dtype, index)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dense_like(t):
    """An uninitialised dense tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _token_stride(name, t, inner):
    """Elements between consecutive tokens of a [B,T,...] tensor whose inner
    dims (``inner`` elements) are dense: a dense tensor or a slice of a fused
    projection's output.  Anything else raises."""
    if t.is_contiguous():
        return inner
    B, T, shape, st = t.shape[0], t.shape[1], t.shape, t.stride()
    dense, run = True, 1
    for i in range(t.dim() - 1, 1, -1):
        dense = dense and (shape[i] == 1 or st[i] == run)
        run *= shape[i]
    s = st[1] if T > 1 else st[0] if B > 1 else inner
    _need(dense and s >= inner and (B <= 1 or T <= 1 or st[0] == T * s),
          f"{name}: heads must be dense and tokens evenly spaced (got shape {tuple(shape)}, "
          f"strides {tuple(st)}); pass {name}.contiguous()")
    return s


def _cuda_index(name, t):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    return index


def _elsewhere(index, stream):
    """A context that makes device ``index`` current, and ``stream`` where one
    is given (so that what is allocated meanwhile belongs to the stream that
    uses it); None where the call is at home already."""
    if stream is not None:
        _need(stream.device.index == index,
              f"the stream is on {stream.device}, the tensors on cuda:{index}")
        return torch.cuda.stream(stream)                   # sets the device too
    if _current_device() != index:
        return torch.cuda.device(index)
    return None


def _rotation(inv_freq, Dk, interleaved, index):
    _tensor("inv_freq", inv_freq, torch.float32, index)
    _need(inv_freq.dim() == 1 and inv_freq.is_contiguous(), "inv_freq must be a dense vector")
    rot = 2 * inv_freq.numel()
    if rot % 16 or rot < 16 or rot > Dk:
        raise ValueError("inv_freq must hold rot_dim/2 frequencies, rot_dim a multiple of 16 in "
                         f"[16, {Dk}]")
    return Rotation(inv_freq.data_ptr(), rot, 1 if interleaved else 0)


def _token_problem(q_heads, k_heads, B, T, Dk, Dv, cu_seqlens, index, scalar=False):
    p = Problem(B, T, q_heads, k_heads, Dk, Dv, 0, 0, 0, FIX_FLAG_SCALAR_GATE if scalar else 0)
    if cu_seqlens is not None:
        _tensor("cu_seqlens", cu_seqlens, torch.int64, index)
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2 and cu_seqlens.is_contiguous(),
              "cu_seqlens must be a dense int64 vector of S + 1 entries")
        _need(B == 1, "packed sequences use a batch of 1")
        p.num_seqs = cu_seqlens.numel() - 1
        p.cu_seqlens = cu_seqlens.data_ptr()
    return p


def _rotary_plan(q, k, inv_freq, cu_seqlens, positions, interleaved, index):
    """Checks a rotation's arguments: (Problem, Rotation, positions' address)."""
    _tensor("q", q, _bf16, index)
    qd = q.shape
    _need(len(qd) == 4, "q must be [B,T,Hq,Dk]")
    B, T, Hq, Dk = qd
    Hkv = Hq
    if k is not None:
        _tensor("k", k, _bf16, index)
        kd = k.shape
        if len(kd) != 4 or kd[0] != B or kd[1] != T or kd[3] != Dk:
            raise ValueError("k must be [B,T,Hkv,Dk] with q's B, T and Dk")
        Hkv = kd[2]
    r = _rotation(inv_freq, Dk, interleaved, index)
    p = _token_problem(Hq, Hkv, B, T, Dk, Dk, cu_seqlens, index)
    if positions is None:
        return p, r, None
    _dense("positions", positions, _i32, index, (B, T))
    return p, r, positions.data_ptr()


def _rotate(plan, q, qs, k, ks, q_out, k_out, inverse, index):
    p, r, positions = plan
    s = load().fix_attn_rotary(
        p, r, positions, q.data_ptr(), qs, None if k is None else k.data_ptr(), ks,
        q_out.data_ptr(), None if k is None else k_out.data_ptr(), 1 if inverse else 0,
        _raw_stream(index))
    if s != 0:
        raise FixStatusError(s, "fix_attn_rotary")
    return q_out, k_out


def fix_attn_rotary(q, k, inv_freq, cu_seqlens=None, positions=None, interleaved=False,
                    inverse=False, out=None, stream=None):
    """Rotates q [B,T,Hq,Dk] and k [B,T,Hkv,Dk] (or None) by position: the
    channel pair i at position p turns by p * inv_freq[i] (``inv_freq`` float32
    [rot_dim/2] on the device; pairs (i, i + rot_dim/2), or (2i, 2i + 1) with
    ``interleaved``; channels from rot_dim on are copied).  Positions are t,
    the index within the sequence for packed tokens (B = 1, int64
    ``cu_seqlens`` on the device; tokens behind the last sequence are copied),
    or int32 ``positions`` [B,T].  q and k may be views of one projection's
    output.  ``inverse`` turns back (the gradient).  Returns new dense (q, k),
    or ``out`` = (q_out, k_out), which may be dense inputs themselves."""
    index = _cuda_index("q", q)
    ctx = _elsewhere(index, stream)
    if ctx is not None:
        with ctx:
            return fix_attn_rotary(q, k, inv_freq, cu_seqlens, positions, interleaved, inverse, out)
    plan = _rotary_plan(q, k, inv_freq, cu_seqlens, positions, interleaved, index)
    qs = _token_stride("q", q, q.shape[2] * q.shape[3])
    ks = _token_stride("k", k, k.shape[2] * k.shape[3]) if k is not None else 0
    if out is None:
        q_out = _dense_like(q)
        k_out = _dense_like(k) if k is not None else None
    else:
        q_out, k_out = out
        _dense("out[0]", q_out, _bf16, index, q.shape)
        _need((k is None) == (k_out is None), "out[1] goes with k")
        if k is not None:
            _dense("out[1]", k_out, _bf16, index, k.shape)
    return _rotate(plan, q, qs, k, ks, q_out, k_out, inverse, index)


def _page_cache(k_pages, v_pages, g_pages, page_table, seqlens, status, S, index):
    """(PageCache, Hkv, Dk, Dv, scalar gate)."""
    try:
        right = (k_pages.dtype is _bf16 and v_pages.dtype is _bf16 and g_pages.dtype is _f32
                 and page_table.dtype is _i32 and seqlens.dtype is _i32
                 and k_pages.get_device() == v_pages.get_device() == g_pages.get_device()
                 == page_table.get_device() == seqlens.get_device() == index)
    except AttributeError:
        right = False
    if not right:
        _tensor("k_pages", k_pages, _bf16, index)
        _tensor("v_pages", v_pages, _bf16, index)
        _tensor("g_pages", g_pages, _f32, index)
        _tensor("page_table", page_table, _i32, index)
        _tensor("seqlens", seqlens, _i32, index)
    kd, vd, gd, td = k_pages.shape, v_pages.shape, g_pages.shape, page_table.shape
    if len(kd) != 4 or not k_pages.is_contiguous():
        raise ValueError("k_pages must be a dense [num_pages,page_size,Hkv,Dk]")
    P, ps, Hkv, Dk = kd
    if len(vd) != 4 or not v_pages.is_contiguous() or vd[0] != P or vd[1] != ps or vd[2] != Hkv:
        raise ValueError("v_pages must be a dense [num_pages,page_size,Hkv,Dv]")
    Dv = vd[3]
    scalar = len(gd) == 3
    if (gd != (P, ps, Hkv) if scalar else gd != vd) or not g_pages.is_contiguous():
        raise ValueError("g_pages must be a dense [num_pages,page_size,Hkv,Dv] or "
                         "[num_pages,page_size,Hkv]")
    if len(td) != 2 or td[0] != S or not page_table.is_contiguous():
        raise ValueError(f"page_table must be a dense [{S},max_pages]")
    if seqlens.shape != (S,) or not seqlens.is_contiguous():
        raise ValueError(f"seqlens must be a dense [{S}]")
    sp = None
    if status is not None:
        _tensor("status", status, _i32, index)
        _need(status.numel() == 1, "status must hold one int32")
        sp = status.data_ptr()
    return (PageCache(ps, P, td[1], page_table.data_ptr(), seqlens.data_ptr(),
                      k_pages.data_ptr(), v_pages.data_ptr(), g_pages.data_ptr(), sp),
            Hkv, Dk, Dv, scalar)


def fix_attn_append_paged(k, v, g, k_pages, v_pages, g_pages, page_table, seqlens,
                          cu_seqlens=None, q=None, inv_freq=None, interleaved=False,
                          return_k=False, status=None, stream=None):
    """Appends new tokens k [B,T,Hkv,Dk], v [B,T,Hkv,Dv] bf16 and g [B,T,Hkv,Dv]
    (or [B,T,Hkv]) f32 to a paged cache: k_pages [num_pages,page_size,Hkv,Dk],
    v_pages and g_pages likewise, int32 ``page_table`` [S,max_pages], int32
    ``seqlens`` [S] (lengths with the new tokens; S = B, or packed B = 1 with
    int64 ``cu_seqlens`` [S+1], all on the device).  The last token of
    sequence b takes position seqlens[b] - 1.  With ``inv_freq`` the keys, and
    ``q`` [B,T,Hq,Dk], are rotated by position as in ``fix_attn_rotary``.
    Tokens at negative positions are padding and not stored.  Returns (q, k)
    rotated: None without ``q`` / unless ``return_k``.  ``status`` (int32 [1])
    is set to FIX_ERR_PAGE if a token had no page (it is skipped)."""
    index = _cuda_index("k", k)
    ctx = _elsewhere(index, stream)
    if ctx is not None:
        with ctx:
            return fix_attn_append_paged(k, v, g, k_pages, v_pages, g_pages, page_table, seqlens,
                                         cu_seqlens, q, inv_freq, interleaved, return_k, status)
    try:
        right = (k.dtype is _bf16 and v.dtype is _bf16 and g.dtype is _f32
                 and v.get_device() == g.get_device() == index)
    except AttributeError:
        right = False
    if not right:
        _tensor("k", k, _bf16, index)
        _tensor("v", v, _bf16, index)
        _tensor("g", g, _f32, index)
    kd, vd, gd = k.shape, v.shape, g.shape
    if len(kd) != 4 or len(vd) != 4 or vd[0] != kd[0] or vd[1] != kd[1] or vd[2] != kd[2]:
        raise ValueError("k and v must be [B,T,Hkv,Dk] and [B,T,Hkv,Dv]")
    B, T, Hkv, Dk = kd
    Dv = vd[3]
    scalar = len(gd) == 3
    if gd != (B, T, Hkv) if scalar else gd != vd:
        raise ValueError("g must be [B,T,Hkv,Dv] or [B,T,Hkv]")
    Hq, qs, qp = Hkv, 0, None
    if q is not None:
        _tensor("q", q, _bf16, index)
        _need(q.dim() == 4, "q must be [B,T,Hq,Dk]")
        Bq, Tq, Hq, Dkq = q.shape
        _need(Bq == B and Tq == T and Dkq == Dk, "q must have k's B, T and Dk")
        qs = 0 if q.is_contiguous() else _token_stride("q", q, Hq * Dk)
        qp = q.data_ptr()
    _need(inv_freq is not None or (q is None and not return_k),
          "q and return_k go with inv_freq")
    p = _token_problem(Hq, Hkv, B, T, Dk, Dv, cu_seqlens, index, scalar)
    c, Hp, Dkp, Dvp, sp = _page_cache(k_pages, v_pages, g_pages, page_table, seqlens, status,
                                      p.num_seqs if cu_seqlens is not None else B, index)
    _need(Hp == Hkv and Dkp == Dk and Dvp == Dv and sp == scalar,
          "the pages must have the tokens' heads, dims and gate")
    r = _rotation(inv_freq, Dk, interleaved, index) if inv_freq is not None else None
    ks = 0 if k.is_contiguous() else _token_stride("k", k, Hkv * Dk)    # 0: dense
    vs = 0 if v.is_contiguous() else _token_stride("v", v, Hkv * Dv)
    gs = 0 if g.is_contiguous() else _token_stride("g", g, Hkv if scalar else Hkv * Dv)
    q_out = _dense_like(q) if q is not None else None
    k_out = _dense_like(k) if return_k else None
    s = load().fix_attn_append_paged(
        p, c, r, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, g.data_ptr(), gs,
        None if q_out is None else q_out.data_ptr(), None if k_out is None else k_out.data_ptr(),
        _raw_stream(index))
    if s != 0:
        raise FixStatusError(s, "fix_attn_append_paged")
    return q_out, k_out


def _paged_problem(q, k_pages, v_pages, g_pages, page_table, seqlens, scale, eps, y_dtype, o_norm,
                   status):
    index = _cuda_index("q", q)
    _tensor("q", q, _bf16, index)
    _need(q.dim() == 3 and q.is_contiguous(), "q must be a dense [B,Hq,Dk]")
    _need(y_dtype is torch.bfloat16 or y_dtype is torch.float32,
          "y_dtype must be bfloat16 or float32")
    B, Hq, Dk = q.shape
    c, Hkv, Dkp, Dv, scalar = _page_cache(k_pages, v_pages, g_pages, page_table, seqlens, status,
                                          B, index)
    _need(Dkp == Dk, "q must have the pages' Dk")
    p = Problem(B, 1, Hq, Hkv, Dk, Dv, 0, 1 if y_dtype is torch.float32 else 0, 0,
                (0 if o_norm else FIX_FLAG_NO_NORM) | (FIX_FLAG_SCALAR_GATE if scalar else 0),
                None, None, 0.0 if scale is None else scale, eps)
    return index, p, c, (B, Hq, Dv)


def fix_attn_decode_paged_workspace(q, k_pages, v_pages, g_pages, page_table, seqlens):
    """A workspace for ``fix_attn_decode_paged`` calls of this shape that do
    not overlap (uint8 tensor; needs no initialisation)."""
    index, p, c, _ = _paged_problem(q, k_pages, v_pages, g_pages, page_table, seqlens, None, 1e-6,
                                    torch.bfloat16, True, None)
    return torch.empty(max(load().fix_attn_decode_paged_workspace_bytes(p, c), 1),
                       dtype=torch.uint8, device=q.device)


def fix_attn_decode_paged(q, k_pages, v_pages, g_pages, page_table, seqlens, o_norm_weight=None,
                          scale=None, eps=1e-6, y_dtype=torch.bfloat16, o_gate=None, o_norm=True,
                          workspace=None, out=None, status=None, stream=None):
    """One new query per sequence, q [B,Hq,Dk], against a paged cache (see
    ``fix_attn_append_paged``; the new token is in it): the last row of
    ``fix_attn`` on each sequence, as ``fix_attn_decode`` computes it from a
    contiguous cache.  int32 ``seqlens`` [B] on the device; length 0 gives 0.
    ``status`` (int32 [1]) is set to FIX_ERR_PAGE if a token had no page (it
    is left out).  Returns y [B,Hq,Dv]."""
    ctx = _elsewhere(_cuda_index("q", q), stream)
    if ctx is not None:
        with ctx:
            return fix_attn_decode_paged(q, k_pages, v_pages, g_pages, page_table, seqlens,
                                         o_norm_weight, scale, eps, y_dtype, o_gate, o_norm,
                                         workspace, out, status)
    index, p, c, shape = _paged_problem(q, k_pages, v_pages, g_pages, page_table, seqlens, scale,
                                        eps, y_dtype, o_norm, status)
    _need(o_norm_weight is not None or not o_norm, "o_norm=True needs o_norm_weight")
    wp = zp = None
    if o_norm_weight is not None:
        _dense("o_norm_weight", o_norm_weight, _bf16, index, shape[2:])
        wp = o_norm_weight.data_ptr()
    if o_gate is not None:
        _dense("o_gate", o_gate, _bf16, index, shape)
        zp = o_gate.data_ptr()
    lib = load()
    if out is None:
        out = q.new_empty(shape) if y_dtype is torch.bfloat16 else q.new_empty(shape, dtype=y_dtype)
    else:
        _dense("out", out, y_dtype, index, shape)
    if workspace is None:
        # in q's type: a plain new_empty is the cheapest allocation
        nbytes = lib.fix_attn_decode_paged_workspace_bytes(p, c)
        workspace = q.new_empty((nbytes + 1) // 2)
    else:
        _tensor("workspace", workspace, torch.uint8, index)
        _need(workspace.is_contiguous(), "workspace must be contiguous")
        nbytes = workspace.numel()
    s = lib.fix_attn_decode_paged(p, c, q.data_ptr(), wp, zp, out.data_ptr(), workspace.data_ptr(),
                                  nbytes, _raw_stream(index))
    if s != 0:
        raise FixStatusError(s, "fix_attn_decode_paged")
    return out


def fix_attn_device_status(workspace, stream=None) -> int:
    return int(load().fix_attn_device_status(_ptr(workspace), _stream(stream)))


def fix_attn_noalloc_device_status(stream=None) -> int:
    """Device status word of the last fix_attn_fwd_noalloc call on the current
    device (synchronises the stream)."""
    return int(load().fix_attn_noalloc_device_status(_stream(stream)))


def _check(ws, where):
    s = fix_attn_device_status(ws)
    if s != 0:
        raise FixStatusError(s, where)


class _FixAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, w, z, cu_seqlens, cu_host, scale, eps, algo, o_norm, check):
        ws = training_workspace(q, k, v, cu_seqlens, cu_host, algo, g, o_norm)
        y, saved = fix_attn_fwd(q, k, v, g, w, cu_seqlens, cu_host, scale, eps, save=True,
                                algo=algo, workspace=ws, o_gate=z, o_norm=o_norm)
        if check:
            _check(ws, "fix_attn forward (device status)")
        ctx.save_for_backward(q, k, v, g, w, z, *saved)
        ctx.cfg = (cu_seqlens, cu_host, scale, eps, algo, o_norm, check)
        ctx.ws = ws
        return y

    @staticmethod
    def backward(ctx, dy):
        q, k, v, g, w, z, o_s, m_s, r_s = ctx.saved_tensors
        cu, cu_host, scale, eps, algo, o_norm, check = ctx.cfg
        dq, dk, dv, dg, dw, dz = fix_attn_bwd(q, k, v, g, w, dy.to(torch.bfloat16).contiguous(),
                                              (o_s, m_s, r_s), cu, cu_host, scale, eps, algo,
                                              workspace=ctx.ws, reuse_forward_workspace=True,
                                              o_gate=z, o_norm=o_norm)
        if check:
            _check(ctx.ws, "fix_attn backward (device status)")
        ctx.ws = None
        return dq, dk, dv, dg, dw, dz, None, None, None, None, None, None, None


def _aligned(t):
    """A gradient as autograd hands it over, dense and on a 16-byte boundary."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _replan(saved, interleaved, sizes, rot_dim, index):
    """A plan of the same sizes for what the saved tensors are by now: copies,
    under saved-tensor hooks."""
    inv_freq, cu_seqlens, positions = saved
    if (inv_freq.dtype is not _f32 or inv_freq.get_device() != index or inv_freq.dim() != 1
            or 2 * inv_freq.numel() != rot_dim or not inv_freq.is_contiguous()):
        _dense("inv_freq", inv_freq, _f32, index, (rot_dim // 2,))
    if sizes.num_seqs:
        _dense("cu_seqlens", cu_seqlens, torch.int64, index, (sizes.num_seqs + 1,))
        sizes = Problem.from_buffer_copy(sizes)
        sizes.cu_seqlens = cu_seqlens.data_ptr()
    if positions is not None:
        _dense("positions", positions, _i32, index, (sizes.batch, sizes.seqlen))
        positions = positions.data_ptr()
    return sizes, Rotation(inv_freq.data_ptr(), rot_dim, 1 if interleaved else 0), positions


class _FixRotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, inv_freq, cu_seqlens, positions, interleaved, inverse):
        index = _cuda_index("q", q)
        ctx.save_for_backward(inv_freq, cu_seqlens, positions)
        with _elsewhere(index, None) or contextlib.nullcontext():
            plan = _rotary_plan(q, k, inv_freq, cu_seqlens, positions, interleaved, index)
            # of this plan the backward takes the sizes, not the addresses:
            # under saved-tensor hooks (checkpoints, offload) the tensors may
            # be gone by then
            ctx.cfg = (interleaved, inverse, plan[0], plan[1].rot_dim)
            return _rotate(plan, q, _token_stride("q", q, q.shape[2] * q.shape[3]), k,
                           _token_stride("k", k, k.shape[2] * k.shape[3]), _dense_like(q),
                           _dense_like(k), inverse, index)

    @staticmethod
    def backward(ctx, dq, dk):
        # the rotation is linear and orthogonal: its gradient is the rotation
        # back (itself differentiable)
        saved = ctx.saved_tensors            # raises where one was changed since
        interleaved, inverse, sizes, rot_dim = ctx.cfg
        dq, dk = _aligned(dq), _aligned(dk)
        index = dq.get_device()
        plan = _replan(saved, interleaved, sizes, rot_dim, index)
        if torch.is_grad_enabled():
            dq, dk = _FixRotary.apply(dq, dk, *saved, interleaved, not inverse)
        else:
            dq, dk = _rotate(plan, dq, 0, dk, 0, _dense_like(dq), _dense_like(dk), not inverse, index)
        return dq, dk, None, None, None, None, None


def fix_rotary(q, k, inv_freq, cu_seqlens=None, positions=None, interleaved=False):
    """``fix_attn_rotary`` of q and k, differentiable in both: the rotation
    that a model trains with before ``fix_attn``, the same that
    ``fix_attn_append_paged`` applies when it serves.  Forward and backward may
    be captured into a CUDA graph, as PyTorch's own operations may: not while
    an uncaptured autograd graph of the same leaves is alive."""
    _need(k is not None, "fix_rotary needs q and k")
    return _FixRotary.apply(q, k, inv_freq, cu_seqlens, positions, bool(interleaved), False)


def fix_attn(q, k, v, g, o_norm_weight=None, cu_seqlens=None, cu_seqlens_host=None, scale=None,
             eps=1e-6, algo="auto", o_gate=None, o_norm=True, check_status=True):
    """FiX attention, differentiable, with the FiX README's arguments ("Quick
    Start"): y = RMSNorm(FiX attention(q, k, v, g)) * o_norm_weight
    [* swish(o_gate)]; with ``o_norm=False`` the output is the attention
    average o_t / l_t [* swish(o_gate)].  g [B,T,Hkv,Dv] (element-wise gate)
    or [B,T,Hkv] (scalar gate).  ``check_status`` reads the device status
    word after the forward and after the backward (each read synchronises
    the stream) and raises FixStatusError if a bounded device wait expired;
    pass False to keep the calls asynchronous."""
    if o_norm and o_norm_weight is None:
        raise ValueError("o_norm=True needs o_norm_weight")
    return _FixAttn.apply(q, k, v, g, o_norm_weight, o_gate, cu_seqlens, cu_seqlens_host, scale,
                          eps, algo, o_norm, check_status)
