"""Thin Python binding of libsinkattn.so (ctypes; argument marshalling only).

Every computation runs in the CUDA library; this module only checks tensor
metadata, allocates outputs with torch, and passes raw device pointers and
the current CUDA stream through the C ABI declared in ``include/sinkattn.h``.
There is no fallback: if the library is missing or the device is not a B200
(sm_100a), calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import warnings
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsinkattn.so")

BF16, FP16, FP32 = 0, 1, 2
OK = 0
ERR_NAMES = {1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "WORKSPACE", 5: "TIMEOUT",
             6: "BOUNDS", 7: "PLAN"}

_c = ctypes
_vp = _c.c_void_p
_i = _c.c_int
_sz = _c.c_size_t


class CMask(_c.Structure):
    """Mirror of ``sinkattn_mask``."""
    _fields_ = [("causal", _c.c_int32), ("n_sink", _c.c_int32), ("window", _c.c_int32),
                ("cu_seqlens", _vp), ("n_seq", _c.c_int32), ("max_seqlen", _c.c_int32),
                ("block_indices", _vp), ("n_qblk", _c.c_int32), ("block_q", _c.c_int32),
                ("block_k", _c.c_int32), ("max_blocks", _c.c_int32)]


class CPagedCache(_c.Structure):
    """Mirror of ``sinkattn_paged_cache``."""
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("block_table", _vp), ("cache_seqlens", _vp), ("B", _c.c_int32),
                ("n_pages", _c.c_int32), ("page_size", _c.c_int32), ("max_pages", _c.c_int32),
                ("Hkv", _c.c_int32), ("D", _c.c_int32)]


class SinkAttnError(RuntimeError):
    def __init__(self, fn, code, detail=None):
        msg = f"{fn} failed: {ERR_NAMES.get(code, code)} ({error_string(code)})"
        super().__init__(msg if detail is None else f"{msg}: {detail}")
        self.code = code


_lib = None


def lib():
    """Load libsinkattn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m learnable_sink_b200.build` (nvcc, sm_100a)")
        L = _c.CDLL(LIB_PATH)
        M = _c.POINTER(CMask)
        L.sinkattn_plan_bytes.restype = _sz
        L.sinkattn_plan_bytes.argtypes = [_i, _i, _i, M]
        L.sinkattn_plan.argtypes = [_i, _i, _i, M, _vp, _sz, _vp]
        L.sinkattn_fwd.argtypes = [_i, _i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, M, _vp, _sz,
                                   _vp, _vp, _vp, _vp]
        L.sinkattn_fwd_ex.argtypes = [_i, _i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, M, _vp,
                                      _sz, _vp, _vp, _vp, _vp, _vp]
        L.sinkattn_bwd_workspace_bytes.restype = _sz
        L.sinkattn_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, M]
        L.sinkattn_bwd.argtypes = [_i, _i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _vp, M, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.sinkattn_bwd_ex.argtypes = [_i, _i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, M, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _sz,
                                      _vp]
        L.sinkattn_gate_importance_workspace_bytes.restype = _sz
        L.sinkattn_gate_importance_workspace_bytes.argtypes = [_i, _i]
        L.sinkattn_gate_importance.argtypes = [_i, _i, _vp, _vp, _vp, _sz, _vp]
        L.sinkattn_gate_vanilla.argtypes = [_i, _i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, M,
                                            _vp, _vp]
        L.sinkattn_decode_workspace_bytes.restype = _sz
        L.sinkattn_decode_workspace_bytes.argtypes = [_i, _i, _i, _i]
        L.sinkattn_decode_num_splits.argtypes = [_i, _i, _i, _i, _i, _i]
        L.sinkattn_decode.argtypes = [_i, _i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, _i, _i,
                                      _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]
        L.sinkattn_decode_fp8_num_splits.argtypes = [_i, _i, _i, _i, _i, _i]
        L.sinkattn_decode_fp8.argtypes = [_i, _i, _i, _i, _c.c_float, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _i, _vp,
                                          _sz, _vp]
        L.sinkattn_cache_append_fp8.argtypes = [_i, _i, _i, _i, _i] + [_vp] * 9 + [_vp]
        L.sinkattn_cache_append.argtypes = [_i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]
        L.sinkattn_cache_fill.argtypes = [_i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _vp]
        P, ll = _c.POINTER(CPagedCache), _c.c_longlong
        append = [_i, _i, _i, P, _vp, ll, _vp, ll, _vp, ll, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]
        L.sinkattn_paged_append.argtypes = append
        L.sinkattn_paged_append_fp8.argtypes = append
        L.sinkattn_paged_decode_workspace_bytes.restype = _sz
        L.sinkattn_paged_decode_workspace_bytes.argtypes = [_i, _i, _i, _i]
        paged = [_i, _i, _c.c_float, _vp, P, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.sinkattn_paged_decode.argtypes = paged
        L.sinkattn_paged_decode_fp8.argtypes = paged
        L.sinkattn_set_kernel_events.argtypes = [_i, _vp, _vp]
        L.sinkattn_selftest_timeout.argtypes = [_vp]
        L.sinkattn_get_status.argtypes = [_vp]
        L.sinkattn_clear_status.argtypes = [_vp]
        L.sinkattn_error_string.restype = _c.c_char_p
        L.sinkattn_error_string.argtypes = [_i]
        L.sinkattn_version.argtypes = []
        _lib = L
    return _lib


_short = None


class _PythonWay:
    """Stands in for the extension where it cannot be used: every call is declined, and the
    Python path makes it."""

    @staticmethod
    def paged_append(*args):
        return -1

    paged_decode = paged_append


def _short_way():
    """The paged calls' short way (csrc/binding.cpp): it checks the tensors and
    makes the C ABI call in one step, or declines (-1) without a launch.  Without the
    extension, or with one that was built for another torch, the Python path makes every
    call (the same kernels, some microseconds of host time more)."""
    global _short
    if _short is None:
        why = None
        try:
            from . import _binding
            if not torch.__version__.startswith(_binding.torch_version):  # 2.11.0+cu128, 2.12.0a0
                why = f"was built for torch {_binding.torch_version}"
        except (ImportError, AttributeError) as e:
            why = f"is missing or does not load ({e})"
        if why is not None:
            warnings.warn(f"learnable_sink_b200/_binding.so {why}: build it with `python -m "
                          "learnable_sink_b200.build`; the paged calls take longer on the host "
                          "without it", RuntimeWarning, stacklevel=4)
            _short = _PythonWay
            return _short
        L = lib()
        _binding.bind(*(_c.cast(f, _vp).value for f in (
            L.sinkattn_paged_append, L.sinkattn_paged_append_fp8,
            L.sinkattn_paged_decode, L.sinkattn_paged_decode_fp8)))
        _short = _binding
    return _short


def error_string(code: int) -> str:
    return lib().sinkattn_error_string(code).decode()


def _check(fn, code):
    if code != OK:
        raise SinkAttnError(fn, code)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else _vp(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return _vp(s.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return FP16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16, float16 or float32")


@dataclass
class Mask:
    """Mask descriptor.  ``cu_seqlens`` / ``block_indices`` are int32 CUDA
    tensors; ``max_seqlen`` must bound every sequence length."""
    cu_seqlens: torch.Tensor
    max_seqlen: int
    causal: bool = True
    n_sink: int = 0
    window: int = 0
    block_indices: Optional[torch.Tensor] = None
    block_q: int = 64
    block_k: int = 64

    def c(self) -> CMask:
        bi = self.block_indices
        return CMask(int(bool(self.causal)), int(self.n_sink), int(self.window),
                     self.cu_seqlens.data_ptr(), int(self.cu_seqlens.numel() - 1),
                     int(self.max_seqlen), None if bi is None else bi.data_ptr(),
                     0 if bi is None else int(bi.shape[1]), int(self.block_q), int(self.block_k),
                     0 if bi is None else int(bi.shape[2]))

    @staticmethod
    def from_spec(spec, device="cuda") -> "Mask":
        """From :class:`learnable_sink_b200.workloads.MaskSpec` (CPU tensors)."""
        bi = spec.block_indices
        return Mask(cu_seqlens=spec.cu_seqlens.to(device=device, dtype=torch.int32).contiguous(),
                    max_seqlen=max(1, spec.max_seqlen), causal=spec.causal, n_sink=spec.n_sink,
                    window=spec.window,
                    block_indices=None if bi is None else bi.to(device=device, dtype=torch.int32).contiguous(),
                    block_q=spec.block_q, block_k=spec.block_k)


class Plan:
    """Tile schedule built on the device from a mask (reusable by fwd/bwd)."""

    def __init__(self, T_tot: int, Hq: int, Hkv: int, mask: Mask, stream=None):
        self.T_tot, self.Hq, self.Hkv, self.mask = T_tot, Hq, Hkv, mask
        self._cm = mask.c()
        nbytes = lib().sinkattn_plan_bytes(T_tot, Hq, Hkv, _c.byref(self._cm))
        if nbytes == 0:
            raise SinkAttnError("sinkattn_plan_bytes", 1)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=mask.cu_seqlens.device)
        self.rebuild(stream)

    def rebuild(self, stream=None) -> None:
        """Rebuild the schedule in place (e.g. after the mask arrays changed)."""
        _check("sinkattn_plan", lib().sinkattn_plan(self.T_tot, self.Hq, self.Hkv,
                                                    _c.byref(self._cm), _ptr(self.buf),
                                                    self.buf.numel(), _stream(stream)))

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


def _want(fn, ok, detail):
    """Metadata the C ABI cannot see through raw pointers (element types and
    extents); a mismatch would make a kernel read or write outside a buffer,
    so it is refused here as SINKATTN_ERR_INVALID_ARG before any launch."""
    if not ok:
        raise SinkAttnError(fn, 1, detail)


def _same_type(fn, ref, **ts):
    for name, t in ts.items():
        if t is not None:
            _want(fn, t.dtype == ref.dtype, f"{name} is {t.dtype}, expected {ref.dtype}")


def _shape(fn, name, t, shape, dtype=None):
    if t is None:
        return
    _want(fn, tuple(t.shape) == tuple(shape),
          f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None:
        _want(fn, t.dtype == dtype, f"{name} is {t.dtype}, expected {dtype}")


def _attn_meta(fn, q, k, v, mask):
    _want(fn, q.dim() == 3 and k.dim() == 3 and v.dim() == 3, "q, k, v must be [T, H, D]")
    _same_type(fn, q, k=k, v=v)
    _want(fn, tuple(k.shape) == tuple(v.shape), "k and v shapes differ")
    _want(fn, q.shape[0] == k.shape[0] and q.shape[2] == k.shape[2],
          f"q {tuple(q.shape)} and k {tuple(k.shape)} disagree on T or D")
    _want(fn, mask.cu_seqlens.dtype == torch.int32, "cu_seqlens must be int32")
    if mask.block_indices is not None:
        _want(fn, mask.block_indices.dtype == torch.int32, "block_indices must be int32")


def _ring_meta(fn, k_cache, v_cache, ref, B, D, n_sink, window):
    _same_type(fn, ref, k_cache=k_cache, v_cache=v_cache)
    _want(fn, tuple(k_cache.shape) == tuple(v_cache.shape), "k_cache and v_cache shapes differ")
    S_ = int(n_sink) + int(window)
    _want(fn, k_cache.shape[0] == B and k_cache.shape[1] == S_ and k_cache.shape[3] == D,
          f"caches have shape {tuple(k_cache.shape)}, expected [{B}, n_sink + window = {S_}, "
          f"Hkv, {D}]")


def _contig(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def fwd(q, k, v, sink, mask: Mask, plan: Plan, scale: Optional[float] = None, stream=None,
        out=None, lse=None, sink_s=None, lse_orig=None):
    """Forward.  Returns (out [T,Hq,D], lse_new [T,Hq] fp32, sink_s [T,Hq] fp32).
    With ``lse_orig`` (fp32 [T,Hq]) also writes the LSE over the visible keys
    alone, before the sink joins (sinkattn_fwd_ex)."""
    _attn_meta("sinkattn_fwd", q, k, v, mask)
    T, Hq, D = q.shape
    _shape("sinkattn_fwd", "learnable_sink", sink, (Hq,), torch.float32)
    _shape("sinkattn_fwd", "out", out, q.shape, q.dtype)
    for name, t in (("lse", lse), ("sink_s", sink_s), ("lse_orig", lse_orig)):
        _shape("sinkattn_fwd", name, t, (T, Hq), torch.float32)
    _contig(q, k, v, sink)
    Hkv = k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(T, Hq, dtype=torch.float32, device=q.device) if lse is None else lse
    sink_s = torch.empty(T, Hq, dtype=torch.float32, device=q.device) if sink_s is None else sink_s
    cm = mask.c()
    if lse_orig is None:
        _check("sinkattn_fwd", lib().sinkattn_fwd(
            _dt(q), T, Hq, Hkv, D, scale, _ptr(q), _ptr(k), _ptr(v), _ptr(sink), _c.byref(cm),
            _ptr(plan.buf), plan.nbytes, _ptr(out), _ptr(lse), _ptr(sink_s), _stream(stream)))
    else:
        _contig(lse_orig)
        _check("sinkattn_fwd_ex", lib().sinkattn_fwd_ex(
            _dt(q), T, Hq, Hkv, D, scale, _ptr(q), _ptr(k), _ptr(v), _ptr(sink), _c.byref(cm),
            _ptr(plan.buf), plan.nbytes, _ptr(out), _ptr(lse), _ptr(sink_s), _ptr(lse_orig),
            _stream(stream)))
    return out, lse, sink_s


def bwd_workspace_bytes(q, k, mask: Mask) -> int:
    T, Hq, D = q.shape
    cm = mask.c()
    return int(lib().sinkattn_bwd_workspace_bytes(_dt(q), T, Hq, k.shape[1], D, _c.byref(cm)))


def bwd(q, k, v, out, dout, lse, sink, mask: Mask, plan: Plan, scale: Optional[float] = None,
        stream=None, workspace=None, dq=None, dk=None, dv=None, dsink=None, d_sink_s=None):
    """Backward.  Returns (dq, dk, dv, dsink or None).  ``d_sink_s`` [T, Hq]
    float32 is an optional upstream gradient of the gate sink_s."""
    _attn_meta("sinkattn_bwd", q, k, v, mask)
    T, Hq, D = q.shape
    _same_type("sinkattn_bwd", q, out=out, dout=dout, dq=dq, dk=dk, dv=dv)
    for name, t in (("out", out), ("dout", dout), ("dq", dq)):
        _shape("sinkattn_bwd", name, t, q.shape)
    for name, t in (("dk", dk), ("dv", dv)):
        _shape("sinkattn_bwd", name, t, k.shape)
    for name, t in (("lse", lse), ("d_sink_s", d_sink_s)):
        _shape("sinkattn_bwd", name, t, (T, Hq), torch.float32)
    for name, t in (("learnable_sink", sink), ("dsink", dsink)):
        _shape("sinkattn_bwd", name, t, (Hq,), torch.float32)
    _contig(q, k, v, out, dout, lse, sink, d_sink_s)
    Hkv = k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    cm = mask.c()
    nws = lib().sinkattn_bwd_workspace_bytes(_dt(q), T, Hq, Hkv, D, _c.byref(cm))
    if workspace is None:
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dsink is None and sink is not None:
        dsink = torch.empty(Hq, dtype=torch.float32, device=q.device)
    _check("sinkattn_bwd_ex", lib().sinkattn_bwd_ex(
        _dt(q), T, Hq, Hkv, D, scale, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
        _ptr(d_sink_s), _ptr(sink), _c.byref(cm), _ptr(plan.buf), plan.nbytes, _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(dsink), _ptr(workspace), workspace.numel(), _stream(stream)))
    return dq, dk, dv, dsink


def gate_importance(sink_s, stream=None, workspace=None, imp=None):
    """Per-head mean gate Imp [Hq] of sink_s [T, Hq] float32."""
    _want("sinkattn_gate_importance", sink_s.dim() == 2 and sink_s.dtype == torch.float32,
          "sink_s must be float32 [T, Hq]")
    T, Hq = sink_s.shape
    _shape("sinkattn_gate_importance", "imp", imp, (Hq,), torch.float32)
    _contig(sink_s)
    nws = int(lib().sinkattn_gate_importance_workspace_bytes(T, Hq))
    if workspace is None:
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=sink_s.device)
    imp = torch.empty(Hq, dtype=torch.float32, device=sink_s.device) if imp is None else imp
    _check("sinkattn_gate_importance", lib().sinkattn_gate_importance(
        T, Hq, _ptr(sink_s), _ptr(imp), _ptr(workspace), workspace.numel(), _stream(stream)))
    return imp


def gate_vanilla(q, k, lse, mask: Mask, scale: Optional[float] = None, stream=None, gate=None):
    """Gate sigma(LSE_not0 - q.k_0 scale) [T, Hq] of a sink-free model whose
    sink is each sequence's first token; ``lse`` is the sink-free LSE."""
    _attn_meta("sinkattn_gate_vanilla", q, k, k, mask)
    T, Hq, D = q.shape
    for name, t in (("lse", lse), ("gate", gate)):
        _shape("sinkattn_gate_vanilla", name, t, (T, Hq), torch.float32)
    _contig(q, k, lse, gate)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    cm = mask.c()
    gate = torch.empty(T, Hq, dtype=torch.float32, device=q.device) if gate is None else gate
    _check("sinkattn_gate_vanilla", lib().sinkattn_gate_vanilla(
        _dt(q), T, Hq, k.shape[1], D, scale, _ptr(q), _ptr(k), _ptr(lse), _c.byref(cm),
        _ptr(gate), _stream(stream)))
    return gate


def decode_num_splits(B, Hq, Hkv, D, n_sink, window) -> int:
    return int(lib().sinkattn_decode_num_splits(B, Hq, Hkv, D, n_sink, window))


def decode_workspace_bytes(B, Hq, D, num_splits) -> int:
    return int(lib().sinkattn_decode_workspace_bytes(B, Hq, D, num_splits))


def decode(q, k_cache, v_cache, cache_seqlens, n_sink: int, window: int, sink,
           scale: Optional[float] = None, num_splits: int = 0, stream=None, workspace=None,
           out=None, lse=None, sink_s=None):
    """Ring-buffer decode.  Returns (out [B,Hq,D], lse_new [B,Hq], sink_s [B,Hq])."""
    fn = "sinkattn_decode"
    _want(fn, q.dim() == 3 and k_cache.dim() == 4, "q must be [B, Hq, D], caches [B, S, Hkv, D]")
    B, Hq, D = q.shape
    _ring_meta(fn, k_cache, v_cache, q, B, D, n_sink, window)
    _shape(fn, "cache_seqlens", cache_seqlens, (B,), torch.int32)
    _shape(fn, "learnable_sink", sink, (Hq,), torch.float32)
    _shape(fn, "out", out, q.shape, q.dtype)
    for name, t in (("lse", lse), ("sink_s", sink_s)):
        _shape(fn, name, t, (B, Hq), torch.float32)
    _contig(q, k_cache, v_cache, cache_seqlens, sink)
    Hkv = k_cache.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if num_splits <= 0:
        num_splits = decode_num_splits(B, Hq, Hkv, D, n_sink, window)
    nws = decode_workspace_bytes(B, Hq, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device) if lse is None else lse
    sink_s = torch.empty(B, Hq, dtype=torch.float32, device=q.device) if sink_s is None else sink_s
    _check("sinkattn_decode", lib().sinkattn_decode(
        _dt(q), B, Hq, Hkv, D, scale, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_seqlens),
        int(n_sink), int(window), _ptr(sink), _ptr(out), _ptr(lse), _ptr(sink_s), int(num_splits),
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return out, lse, sink_s


def decode_fp8_num_splits(B, Hq, Hkv, D, n_sink, window) -> int:
    return int(lib().sinkattn_decode_fp8_num_splits(B, Hq, Hkv, D, n_sink, window))


def decode_fp8(q, k_sink, v_sink, k_win, v_win, k_scale, v_scale, cache_seqlens, n_sink: int,
               window: int, sink, scale: Optional[float] = None, num_splits: int = 0,
               stream=None, workspace=None, out=None, lse=None, sink_s=None):
    """Ring-buffer decode over a mixed-precision cache: bf16 sink slots
    k_sink/v_sink [B, n_sink, Hkv, D], FP8 E4M3 window slots k_win/v_win
    [B, window, Hkv, D] (uint8 codes, or torch.float8_e4m3fn) with per-KV-head
    float32 scales k_scale/v_scale [Hkv].  Returns (out [B,Hq,D] bf16,
    lse_new [B,Hq], sink_s [B,Hq])."""
    fn = "sinkattn_decode_fp8"
    _want(fn, q.dim() == 3 and q.dtype == torch.bfloat16, "q must be bfloat16 [B, Hq, D]")
    B, Hq, D = q.shape
    _want(fn, k_win.dim() == 4 and k_win.element_size() == 1 and v_win.element_size() == 1,
          "k_win / v_win must be 1-byte [B, window, Hkv, D] E4M3 codes")
    Hkv = k_win.shape[2]
    _shape(fn, "k_win", k_win, (B, window, Hkv, D))
    _shape(fn, "v_win", v_win, (B, window, Hkv, D))
    for name, t in (("k_sink", k_sink), ("v_sink", v_sink)):
        _shape(fn, name, t, (B, n_sink, Hkv, D), torch.bfloat16)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _shape(fn, name, t, (Hkv,), torch.float32)
    _shape(fn, "cache_seqlens", cache_seqlens, (B,), torch.int32)
    _shape(fn, "learnable_sink", sink, (Hq,), torch.float32)
    _shape(fn, "out", out, q.shape, q.dtype)
    for name, t in (("lse", lse), ("sink_s", sink_s)):
        _shape(fn, name, t, (B, Hq), torch.float32)
    _contig(q, k_sink, v_sink, k_win, v_win, k_scale, v_scale, cache_seqlens, sink)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if num_splits <= 0:
        num_splits = decode_fp8_num_splits(B, Hq, Hkv, D, n_sink, window)
    nws = decode_workspace_bytes(B, Hq, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device) if lse is None else lse
    sink_s = torch.empty(B, Hq, dtype=torch.float32, device=q.device) if sink_s is None else sink_s
    _check(fn, lib().sinkattn_decode_fp8(
        B, Hq, Hkv, D, scale, _ptr(q), _ptr(k_sink), _ptr(v_sink), _ptr(k_win), _ptr(v_win),
        _ptr(k_scale), _ptr(v_scale), _ptr(cache_seqlens), int(n_sink), int(window), _ptr(sink),
        _ptr(out), _ptr(lse), _ptr(sink_s), int(num_splits), _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return out, lse, sink_s


def cache_append(k_new, v_new, cache_seqlens, k_cache, v_cache, n_sink: int, window: int,
                 stream=None) -> None:
    """Write one new token per sequence (k_new/v_new [B, Hkv, D]) into its ring
    slot; cache_seqlens [B] int32 already counts the new token."""
    fn = "sinkattn_cache_append"
    _want(fn, k_new.dim() == 3 and k_cache.dim() == 4, "k_new must be [B, Hkv, D]")
    B, Hkv, D = k_new.shape
    _shape(fn, "v_new", v_new, k_new.shape, k_new.dtype)
    _ring_meta(fn, k_cache, v_cache, k_new, B, D, n_sink, window)
    _want(fn, k_cache.shape[2] == Hkv, "k_new and the caches disagree on Hkv")
    _shape(fn, "cache_seqlens", cache_seqlens, (B,), torch.int32)
    _contig(k_new, v_new, cache_seqlens, k_cache, v_cache)
    _check("sinkattn_cache_append", lib().sinkattn_cache_append(
        _dt(k_new), B, Hkv, D, int(n_sink), int(window), _ptr(k_new), _ptr(v_new),
        _ptr(cache_seqlens), _ptr(k_cache), _ptr(v_cache), _stream(stream)))


def cache_append_fp8(k_new, v_new, cache_seqlens, k_sink, v_sink, k_win, v_win, k_scale,
                     v_scale, n_sink: int, window: int, stream=None) -> None:
    """Write one new bf16 token per sequence (k_new/v_new [B, Hkv, D]) into
    the mixed-precision cache of decode_fp8: a sink slot as it is, a window
    row as E4M3 codes of value / scale; cache_seqlens [B] int32 already
    counts the new token."""
    fn = "sinkattn_cache_append_fp8"
    _want(fn, k_new.dim() == 3 and k_new.dtype == torch.bfloat16, "k_new must be bf16 [B, Hkv, D]")
    B, Hkv, D = k_new.shape
    _shape(fn, "v_new", v_new, k_new.shape, k_new.dtype)
    for name, t in (("k_sink", k_sink), ("v_sink", v_sink)):
        _shape(fn, name, t, (B, n_sink, Hkv, D), torch.bfloat16)
    for name, t in (("k_win", k_win), ("v_win", v_win)):
        if t is not None:
            _want(fn, t.element_size() == 1, f"{name} must hold 1-byte E4M3 codes")
        _shape(fn, name, t, (B, window, Hkv, D))
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _shape(fn, name, t, (Hkv,), torch.float32)
    _shape(fn, "cache_seqlens", cache_seqlens, (B,), torch.int32)
    _contig(k_new, v_new, cache_seqlens, k_sink, v_sink, k_win, v_win, k_scale, v_scale)
    _check(fn, lib().sinkattn_cache_append_fp8(
        B, Hkv, D, int(n_sink), int(window), _ptr(k_new), _ptr(v_new), _ptr(cache_seqlens),
        _ptr(k_sink), _ptr(v_sink), _ptr(k_win), _ptr(v_win), _ptr(k_scale), _ptr(v_scale),
        _stream(stream)))


def cache_fill(k, v, cu_seqlens, k_cache, v_cache, n_sink: int, window: int,
               cache_seqlens_out=None, stream=None) -> None:
    """Write a packed prefill (k/v [T_tot, Hkv, D], sequences by cu_seqlens)
    into the ring caches [n_seq, S, Hkv, D]; optionally store the lengths."""
    fn = "sinkattn_cache_fill"
    _want(fn, k.dim() == 3 and k_cache.dim() == 4 and cu_seqlens.dim() == 1,
          "k must be [T, Hkv, D], caches [n_seq, S, Hkv, D], cu_seqlens [n_seq + 1]")
    T, Hkv, D = k.shape
    n_seq = cu_seqlens.numel() - 1
    _shape(fn, "v", v, k.shape, k.dtype)
    _want(fn, cu_seqlens.dtype == torch.int32, "cu_seqlens must be int32")
    _ring_meta(fn, k_cache, v_cache, k, n_seq, D, n_sink, window)
    _want(fn, k_cache.shape[2] == Hkv, "k and the caches disagree on Hkv")
    _shape(fn, "cache_seqlens_out", cache_seqlens_out, (n_seq,), torch.int32)
    _contig(k, v, cu_seqlens, k_cache, v_cache, cache_seqlens_out)
    n_seq = cu_seqlens.numel() - 1
    _check("sinkattn_cache_fill", lib().sinkattn_cache_fill(
        _dt(k), n_seq, T, Hkv, D, int(n_sink), int(window), _ptr(cu_seqlens), _ptr(k), _ptr(v),
        _ptr(k_cache), _ptr(v_cache), _ptr(cache_seqlens_out), _stream(stream)))


class PagedCache:
    """A paged K/V cache (see ``sinkattn_paged_cache``): pools ``k_pages`` /
    ``v_pages`` [n_pages, Hkv, page_size, D] in bfloat16 or float16, or E4M3
    codes (torch.float8_e4m3fn or uint8) with float32 scales ``k_scale`` /
    ``v_scale`` [n_pages, Hkv]; ``block_table`` int32 [B, max_pages] and
    ``cache_seqlens`` int32 [B], which counts a call's new tokens.  The tensors
    are checked once, here, and kept: their contents may change between calls, the
    attributes and the tensors' storage (``set_``, ``resize_``) may not (other tensors
    are another PagedCache)."""

    __slots__ = ("k_pages", "v_pages", "block_table", "cache_seqlens", "k_scale", "v_scale",
                 "device", "B", "Hkv", "D", "_c", "_ref", "_dev", "_at", "_kind")

    def __init__(self, k_pages, v_pages, block_table, cache_seqlens, k_scale=None, v_scale=None):
        fn = "PagedCache"
        _want(fn, k_pages.dim() == 4, "pages must be [n_pages, Hkv, page_size, D]")
        _same_type(fn, k_pages, v_pages=v_pages)
        _shape(fn, "v_pages", v_pages, k_pages.shape)
        n_pages, Hkv, page_size, D = k_pages.shape
        coded = k_pages.element_size() == 1
        if coded:
            _want(fn, k_pages.dtype in (torch.float8_e4m3fn, torch.uint8),
                  f"pages are {k_pages.dtype}, expected float8_e4m3fn or uint8 codes")
            _want(fn, k_scale is not None and v_scale is not None, "8-bit pages need scales")
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                _shape(fn, name, t, (n_pages, Hkv), torch.float32)
        else:
            _want(fn, k_pages.dtype in (torch.bfloat16, torch.float16),
                  f"pages are {k_pages.dtype}, expected bfloat16, float16 or 8-bit codes")
            _want(fn, k_scale is None and v_scale is None, "scales go with 8-bit pages")
        _want(fn, page_size in (16, 32, 64, 128), f"page_size {page_size}: 16, 32, 64 or 128")
        _want(fn, D in (64, 128), f"D {D}: 64 or 128")
        _want(fn, block_table.dim() == 2 and block_table.dtype == torch.int32
              and block_table.numel() > 0, "block_table must be int32 [B, max_pages]")
        B, max_pages = block_table.shape
        _shape(fn, "cache_seqlens", cache_seqlens, (B,), torch.int32)
        ts = (k_pages, v_pages, block_table, cache_seqlens, k_scale, v_scale)
        _contig(*ts)
        _one_device(fn, *ts)
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.block_table, self.cache_seqlens = block_table, cache_seqlens
        self.device, self.B, self.Hkv, self.D = k_pages.device, B, Hkv, D
        self._dev = k_pages.get_device()
        self._c = CPagedCache(k_pages.data_ptr(), v_pages.data_ptr(),
                              None if k_scale is None else k_scale.data_ptr(),
                              None if v_scale is None else v_scale.data_ptr(),
                              block_table.data_ptr(), cache_seqlens.data_ptr(), B, n_pages,
                              page_size, max_pages, Hkv, D)
        self._ref = _c.byref(self._c)
        self._at = _c.addressof(self._c)
        self._kind = 2 if coded else int(k_pages.dtype == torch.float16)

    def __setattr__(self, name, value):
        # the calls read the descriptor that was built with the tensors: a tensor put
        # in their place would go unseen
        if hasattr(self, "_kind"):
            raise AttributeError(f"PagedCache.{name} is fixed; build another PagedCache")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        # nor may a tensor be let go of: the descriptor holds its address
        raise AttributeError(f"PagedCache.{name} is fixed; build another PagedCache")


def _one_device(fn, *ts):
    dev = ts[0].device
    for t in ts:
        if t is not None and t.device != dev:
            raise SinkAttnError(fn, 1, f"tensors on {dev} and {t.device}")


def _current(fn, dev):
    """The library launches on the current device."""
    if dev != torch.cuda.current_device():
        raise SinkAttnError(fn, 1, f"tensors on cuda:{dev}, current device "
                                   f"cuda:{torch.cuda.current_device()}")


# torch.cuda.current_stream() builds an object around this handle (3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(dev)


_CODE = {torch.bfloat16: BF16, torch.float16: FP16}

# The paged calls serve single tokens, where the host's time counts: their checks
# are plain comparisons, and what was wrong is put in words only once one fails.


def _plain(t, shape, dtype, dev):
    """t (if any) is contiguous, of this shape and type, on device dev."""
    return t is None or (t.shape == shape and t.dtype == dtype and t.get_device() == dev
                         and t.is_contiguous())


def _refuse_plain(fn, name, t, shape, dtype, dev):
    _shape(fn, name, t, shape, dtype)
    _contig(t)
    raise SinkAttnError(fn, 1, f"{name} is on {t.device}, the cache on cuda:{dev}")


def _token_stride(fn, name, t, shape, dtype, dev):
    """Checks a packed [T, H, D] input whose tokens may be strided (a view of a
    fused projection); returns its token stride in elements."""
    T, H, D = shape
    if t.shape != shape or t.dtype != dtype:
        _shape(fn, name, t, shape, dtype)
    s0, s1, s2 = t.stride()
    row = H * D
    if T <= 1:
        s0 = row
    if (s2 == 1 and (s1 == D or H == 1) and s0 >= row and not s0 % 8 and not t.data_ptr() % 16
            and t.get_device() == dev):
        return s0
    if t.get_device() != dev:
        raise SinkAttnError(fn, 1, f"{name} is on {t.device}, the cache on cuda:{dev}")
    if s2 != 1 or (H != 1 and s1 != D):
        raise SinkAttnError(fn, 1, f"{name}: a token's heads must be contiguous")
    raise SinkAttnError(fn, 1, f"{name}: tokens must be 16-byte aligned and not overlap")


def _paged_append(fn, call, coded, k, v, cache, cu_new, rope, interleaved, q, q_out, k_out, stream):
    if k.dim() != 3:
        raise SinkAttnError(fn, 1, "k must be [T, Hkv, D]")
    dev, D, B, dt = cache._dev, cache.D, cache.B, k.dtype
    if coded:
        _want(fn, cache.k_scale is not None, "the cache is not an 8-bit cache")
    elif cache.k_pages.dtype != dt:
        raise SinkAttnError(fn, 1, f"k is {dt}, the pages {cache.k_pages.dtype}")
    T = k.shape[0]
    kv = (T, cache.Hkv, D)
    ks = _token_stride(fn, "k", k, kv, dt, dev)
    vs = _token_stride(fn, "v", v, kv, dt, dev)
    Hq = qs = rot = n_pos = 0
    q_ptr = qo_ptr = ko_ptr = cu_ptr = rope_ptr = None
    if q is not None:
        if q.dim() != 3:
            raise SinkAttnError(fn, 1, "q must be [T, Hq, D]")
        Hq = q.shape[1]
        shape = (T, Hq, D)
        qs = _token_stride(fn, "q", q, shape, dt, dev)
        if (q_out.shape != shape or q_out.dtype != dt or q_out.get_device() != dev
              or not q_out.is_contiguous()):
            _refuse_plain(fn, "q_out", q_out, shape, dt, dev)
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise SinkAttnError(fn, 1, "q_out without q")
    if k_out is not None:
        if not _plain(k_out, kv, dt, dev):
            _refuse_plain(fn, "k_out", k_out, kv, dt, dev)
        ko_ptr = k_out.data_ptr()
    if cu_new is None:
        if T != B:
            raise SinkAttnError(fn, 1, f"{T} tokens for {B} sequences without cu_new")
    else:
        if not _plain(cu_new, (B + 1,), torch.int32, dev):
            _refuse_plain(fn, "cu_new", cu_new, (B + 1,), torch.int32, dev)
        cu_ptr = cu_new.data_ptr()
    if rope is not None:
        if (rope.dim() != 2 or rope.dtype != torch.float32 or rope.get_device() != dev
                or not rope.is_contiguous()):
            raise SinkAttnError(fn, 1, "rope must be float32 [n_pos, rot_dim], contiguous, on the "
                                       "cache's device")
        n_pos, rot = rope.shape
        if n_pos < 1 or rot % 16 or not 16 <= rot <= D:
            raise SinkAttnError(fn, 1, f"rot_dim {rot}: a multiple of 16 up to {D}")
        n_pos = min(n_pos, 2 ** 31 - 1)  # no position lies past it
        rope_ptr = rope.data_ptr()
    if dev != torch.cuda.current_device():
        _current(fn, dev)
    rc = call(_CODE.get(dt) if dt in _CODE else _dt(k), T, Hq, cache._ref, k.data_ptr(), ks,
              v.data_ptr(), vs, q_ptr, qs, cu_ptr, rope_ptr, rot, n_pos, 1 if interleaved else 0,
              qo_ptr, ko_ptr, _handle(stream, dev))
    if rc:
        raise SinkAttnError(fn, rc)
    return q_out


_APPEND = ("sinkattn_paged_append", "sinkattn_paged_append_fp8")
_DECODE = ("sinkattn_paged_decode", "sinkattn_paged_decode_fp8")


_AS_IS = contextlib.nullcontext()


def _allocating(stream):
    """What a call on `stream` allocates belongs to that stream: memory of the current
    one may still be in use there, and would go back to it before the kernel ends."""
    return _AS_IS if stream is None else torch.cuda.stream(stream)


def _append_call(coded, k, v, cache, cu_new, rope, interleaved, q, q_out, k_out, stream):
    if q_out is None and q is not None:
        with _allocating(stream):
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if stream is None:
        rc = (_short or _short_way()).paged_append(cache._at, coded, cache._kind, cache._dev, k, v,
                                                   cu_new, rope, interleaved, q, q_out, k_out)
        if rc == 0:
            return q_out
        if rc > 0:
            raise SinkAttnError(_APPEND[coded], rc)
    return _paged_append(_APPEND[coded], getattr(lib(), _APPEND[coded]), coded, k, v, cache, cu_new,
                         rope, interleaved, q, q_out, k_out, stream)


def paged_append(k, v, cache: PagedCache, cu_new=None, rope=None, interleaved: bool = False,
                 q=None, q_out=None, k_out=None, stream=None):
    """Append packed new tokens (k/v [T, Hkv, D], sequences by cu_new int32
    [B + 1]; without it one token per sequence) as the last positions that
    cache.cache_seqlens counts, keys rotated by ``rope`` [n_pos, rot_dim]
    (cosines, then sines; pairs half a rot_dim apart, or neighbours when
    interleaved).  ``q`` [T, Hq, D] is rotated into q_out, the rotated keys also
    go to k_out if given.  k, v and q may be views with strided tokens.
    Returns q_out."""
    return _append_call(0, k, v, cache, cu_new, rope, interleaved, q, q_out, k_out, stream)


def paged_append_fp8(k, v, cache: PagedCache, cu_new=None, rope=None, interleaved: bool = False,
                     q=None, q_out=None, k_out=None, stream=None):
    """paged_append into an 8-bit cache: E4M3 codes with a power-of-two scale for
    each page and KV head, which grows (the page's earlier codes with it) when
    new rows need it."""
    return _append_call(1, k, v, cache, cu_new, rope, interleaved, q, q_out, k_out, stream)


def paged_decode_workspace_bytes(B, Hq, Hkv, D) -> int:
    return int(lib().sinkattn_paged_decode_workspace_bytes(B, Hq, Hkv, D))


def _decode_call(coded, q, cache, sink, n_sink, window, scale, stream, workspace, out, lse, sink_s):
    if out is None or lse is None or sink_s is None or workspace is None:
        if q.dim() != 3:
            raise SinkAttnError(_DECODE[coded], 1, "q must be [B, Hq, D]")
        B, Hq, D = q.shape
        with _allocating(stream):
            if out is None:
                out = torch.empty_like(q, memory_format=torch.contiguous_format)
            if lse is None:
                lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
            if sink_s is None:
                sink_s = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
            if workspace is None:
                workspace = torch.empty(max(paged_decode_workspace_bytes(B, Hq, cache.Hkv, D), 16),
                                        dtype=torch.uint8, device=q.device)
    if stream is None:
        rc = (_short or _short_way()).paged_decode(cache._at, coded, cache._kind, cache._dev, q, sink,
                                                   n_sink, window, scale, workspace, out, lse, sink_s)
        if rc == 0:
            return out, lse, sink_s
        if rc > 0:
            raise SinkAttnError(_DECODE[coded], rc)
    return _paged_decode(_DECODE[coded], getattr(lib(), _DECODE[coded]), coded, q, cache, sink, n_sink,
                         window, scale, stream, workspace, out, lse, sink_s)


def _int32(fn, name, x):
    """ctypes would keep the low 32 bits of anything larger."""
    if int(x) != x or not 0 <= x < 2 ** 31:
        raise SinkAttnError(fn, 1, f"{name} {x}: a whole number in [0, 2^31)")
    return int(x)


def _paged_decode(fn, call, coded, q, cache, sink, n_sink, window, scale, stream, workspace, out,
                  lse, sink_s):
    if q.dim() != 3 or q.shape[0] != cache.B or q.shape[2] != cache.D:
        raise SinkAttnError(fn, 1, f"q {tuple(q.shape)} and the cache disagree on B or D: "
                                   f"[{cache.B}, Hq, {cache.D}]")
    B, Hq, D = shape = q.shape
    dev, dt = cache._dev, q.dtype
    if coded:
        _want(fn, cache.k_scale is not None, "the cache is not an 8-bit cache")
    elif cache.k_pages.dtype != dt:
        raise SinkAttnError(fn, 1, f"k_pages is {cache.k_pages.dtype}, expected {dt}")
    f32, rows = torch.float32, (B, Hq)
    if not (out.shape == shape and out.dtype == dt and lse.shape == rows and lse.dtype == f32
            and sink_s.shape == rows and sink_s.dtype == f32
            and q.get_device() == out.get_device() == lse.get_device() == sink_s.get_device()
            == workspace.get_device() == dev
            and q.is_contiguous() and out.is_contiguous() and lse.is_contiguous()
            and sink_s.is_contiguous() and workspace.is_contiguous()
            and _plain(sink, (Hq,), f32, dev)):
        for name, t, want, kind in (("q", q, shape, dt), ("out", out, shape, dt),
                                    ("lse", lse, rows, f32), ("sink_s", sink_s, rows, f32),
                                    ("learnable_sink", sink, (Hq,), f32),
                                    ("workspace", workspace, workspace.shape, workspace.dtype)):
            if not _plain(t, want, kind, dev):
                _refuse_plain(fn, name, t, want, kind, dev)
    n_sink, window = _int32(fn, "n_sink", n_sink), _int32(fn, "window", window)
    if dev != torch.cuda.current_device():
        _current(fn, dev)
    rc = call(_CODE.get(dt) if dt in _CODE else _dt(q), Hq, D ** -0.5 if scale is None else float(scale),
              q.data_ptr(), cache._ref, n_sink, window, None if sink is None else sink.data_ptr(),
              out.data_ptr(), lse.data_ptr(), sink_s.data_ptr(), workspace.data_ptr(),
              workspace.nbytes, _handle(stream, dev))
    if rc:
        raise SinkAttnError(fn, rc)
    return out, lse, sink_s


def paged_decode(q, cache: PagedCache, sink, n_sink: int = 0, window: int = 0,
                 scale: Optional[float] = None, stream=None, workspace=None, out=None, lse=None,
                 sink_s=None):
    """One query token per sequence (q [B, Hq, D]) over a paged 16-bit cache;
    with window > 0 only the first n_sink and the last ``window`` positions are
    visible.  Returns (out [B,Hq,D], lse_new [B,Hq], sink_s [B,Hq])."""
    return _decode_call(0, q, cache, sink, n_sink, window, scale, stream, workspace, out, lse, sink_s)


def paged_decode_fp8(q, cache: PagedCache, sink, n_sink: int = 0, window: int = 0,
                     scale: Optional[float] = None, stream=None, workspace=None, out=None,
                     lse=None, sink_s=None):
    """paged_decode over an 8-bit cache (q and out bfloat16 or float16)."""
    return _decode_call(1, q, cache, sink, n_sink, window, scale, stream, workspace, out, lse, sink_s)


KERNEL_FWD, KERNEL_BWD, KERNEL_DECODE, KERNEL_GATE = 0, 1, 2, 3


def set_kernel_events(which: int, start=None, stop=None) -> None:
    """Have later calls record torch.cuda.Event ``start``/``stop`` around their
    main kernel (events must already have been recorded once, so that torch
    has created them).  Pass None, None to stop."""
    sp = None if start is None else _vp(start.cuda_event)
    ep = None if stop is None else _vp(stop.cuda_event)
    _check("sinkattn_set_kernel_events", lib().sinkattn_set_kernel_events(int(which), sp, ep))


def selftest_timeout(stream=None) -> None:
    """Launch the bounded-wait self-test kernel (see include/sinkattn.h)."""
    _check("sinkattn_selftest_timeout", lib().sinkattn_selftest_timeout(_stream(stream)))


def get_status(stream=None) -> int:
    return int(lib().sinkattn_get_status(_stream(stream)))


def clear_status(stream=None) -> None:
    _check("sinkattn_clear_status", lib().sinkattn_clear_status(_stream(stream)))
