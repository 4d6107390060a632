"""Python binding of libfa.so: the C-ABI entry points under the same names.

Argument marshalling only -- every step of the attention runs in the CUDA
kernels behind the C ABI. Tensors are torch CUDA tensors (torch provides the
device memory and the stream); nothing here computes attention, and there is
no fallback: if the library is missing or the call fails, an exception says so.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "fa.h")

FA_OK = 0
FA_FP16, FA_BF16, FA_FP8_E4M3, FA_INT8 = 0, 1, 2, 3
_DTYPE = {torch.float16: FA_FP16, torch.bfloat16: FA_BF16}
_CACHE_DTYPE = {**_DTYPE, torch.float8_e4m3fn: FA_FP8_E4M3, torch.int8: FA_INT8}

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} ({status})")


def header_functions():
    """Names of the functions include/fa.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(fa_\w+)\s*\(", text, flags=re.M)))


def lib():
    """Load libfa.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.fa_fwd.restype = i
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp, i, i, i, vp]
        L.fa_fp8_prep.restype = i
        L.fa_fp8_prep.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
        L.fa_fwd_fp8.restype = i
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_varlen_blocks.restype = i
        L.fa_varlen_blocks.argtypes = [vp, i, vp, vp]
        L.fa_fp8_prep_varlen.restype = i
        L.fa_fp8_prep_varlen.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, i, i, vp, vp, vp, vp,
                                         i, i, i, i, i, vp]
        L.fa_fwd_fp8_varlen.restype = i
        L.fa_fwd_fp8_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, vp, vp, vp, vp, i, i, i, i, i,
                                        f, i, vp]
        L.fa_fwd_paged.restype = i
        L.fa_fwd_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp, i, i, vp,
                                   ctypes.c_size_t, i, vp]
        L.fa_bwd_workspace_size.restype = ctypes.c_size_t
        L.fa_bwd_workspace_size.argtypes = [i, i]
        L.fa_bwd.restype = i
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp, i, i, vp,
                             ctypes.c_size_t, i, vp]
        L.fa_fwd_splitkv_workspace_size.restype = ctypes.c_size_t
        L.fa_fwd_splitkv_workspace_size.argtypes = [i, i, i, i, i, i]
        L.fa_fwd_splitkv.restype = i
        L.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, ctypes.c_size_t, i, vp]
        L.fa_rope.restype = i
        L.fa_rope.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, i, i, vp, i, vp]
        L.fa_kv_append.restype = i
        L.fa_kv_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp, i, i, i, vp]
        L.fa_kv_read.restype = i
        L.fa_kv_read.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, vp]
        L.fa_fwd_kvcache_workspace_size.restype = ctypes.c_size_t
        L.fa_fwd_kvcache_workspace_size.argtypes = [i, i, i, i, i, i, i]
        L.fa_fwd_kvcache.restype = i
        L.fa_fwd_kvcache.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, vp, i, vp,
                                     ctypes.c_size_t, i, i, vp]
        L.fa_fwd_prefix.restype = i
        L.fa_fwd_prefix.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, vp, i, vp,
                                    ctypes.c_size_t, i, i, vp]
        L.fa_get_device_status.restype = i
        L.fa_get_device_status.argtypes = [vp, ctypes.POINTER(i)]
        L.fa_strerror.restype = ctypes.c_char_p
        L.fa_strerror.argtypes = [i]
        L.fa_version.restype = i
        L.fa_version.argtypes = []
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().fa_strerror(int(status)).decode()


def fa_version() -> int:
    return lib().fa_version()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def fa_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale, causal, cu_seqlens_q=None, cu_seqlens_k=None,
           total_q=0, total_k=0, dtype=None, stream=None, check=True) -> int:
    """Raw entry point: pointers from the tensors, sizes as given. Returns the
    status; raises FAError when ``check`` and the status is not FA_OK."""
    if dtype is None:
        dtype = _DTYPE[q.dtype]
    st = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(H), int(Sq), int(Sk),
                      int(D), float(scale), int(bool(causal)), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                      int(total_q), int(total_k), int(dtype), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd")
    return st


def fa_fwd_splitkv_workspace_size(B, H, Sq, Sk, D, num_splits) -> int:
    return int(lib().fa_fwd_splitkv_workspace_size(int(B), int(H), int(Sq), int(Sk), int(D), int(num_splits)))


def fa_fwd_splitkv(q, k, v, o, lse, B, H, Sq, Sk, D, scale, causal, num_splits, workspace, workspace_bytes,
                   dtype=None, stream=None, check=True) -> int:
    """Raw entry point: split-KV forward with a caller-owned workspace."""
    if dtype is None:
        dtype = _DTYPE[q.dtype]
    st = lib().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(H), int(Sq), int(Sk),
                              int(D), float(scale), int(bool(causal)), int(num_splits), _ptr(workspace),
                              int(workspace_bytes), int(dtype), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_splitkv")
    return st


def fa_fwd_splitkv_noalloc(q, k, v, o, lse, B, H, Sq, Sk, D, scale, causal, num_splits, dtype=None,
                           stream=None, check=True) -> int:
    """Raw entry point: split-KV forward whose scratch is the library's own
    fixed array, for callers that cannot allocate device memory."""
    L = lib()
    fn = L.fa_fwd_splitkv_noalloc
    vp, i = ctypes.c_void_p, ctypes.c_int
    fn.restype = i
    fn.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, ctypes.c_float, i, i, i, vp]
    if dtype is None:
        dtype = _DTYPE[q.dtype]
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(H), int(Sq), int(Sk), int(D), float(scale),
            int(bool(causal)), int(num_splits), int(dtype), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_splitkv_noalloc")
    return st


def attention_forward_splitkv(q, k, v, *, batch, causal=False, scale=None, num_splits=0, workspace=None,
                              out=None, lse=None, stream=None):
    """Allocate O, LSE and (unless given) the workspace with torch and call
    ``fa_fwd_splitkv``. q ``[B*Sq, H, D]``, k/v ``[B*Sk, H, D]``."""
    B = batch
    H, D = q.shape[1], q.shape[2]
    Sq, Sk = q.shape[0] // B, k.shape[0] // B
    if scale is None:
        scale = D ** -0.5
    nbytes = fa_fwd_splitkv_workspace_size(B, H, Sq, Sk, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Sq), device=q.device, dtype=torch.float32)
    fa_fwd_splitkv(q, k, v, out, lse, B, H, Sq, Sk, D, scale, causal, num_splits, workspace,
                   workspace.numel() * workspace.element_size(), stream=stream)
    return out, lse


def fa_fp8_prep(q, k, v, q8, k8, v8, q_scale, k_scale, v_scale, sigma, B, H, Sq, Sk, D, in_dtype=None,
                stream=None, check=True) -> int:
    """Raw entry point: Hadamard rotation (``sigma`` int8 +-1, or None for
    none) and per-128-row-block e4m3 quantisation of Q, K (rotated) and V."""
    if in_dtype is None:
        in_dtype = _DTYPE[q.dtype]
    st = lib().fa_fp8_prep(_ptr(q), _ptr(k), _ptr(v), int(in_dtype), _ptr(q8), _ptr(k8), _ptr(v8),
                           _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), _ptr(sigma), int(B), int(H), int(Sq),
                           int(Sk), int(D), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fp8_prep")
    return st


def fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B, H, Sq, Sk, D, scale, causal, stream=None,
               check=True) -> int:
    """Raw entry point: attention on e4m3 codes with block scales; bf16 O."""
    st = lib().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), _ptr(o),
                          _ptr(lse), int(B), int(H), int(Sq), int(Sk), int(D), float(scale), int(bool(causal)),
                          _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_fp8")
    return st


def fa_varlen_blocks(cu_seqlens, B, cu_blocks, stream=None, check=True) -> int:
    """Raw entry point: cu_blocks[b] = sum of ceil(L / 128) over the first b sequences."""
    st = lib().fa_varlen_blocks(_ptr(cu_seqlens), int(B), _ptr(cu_blocks), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_varlen_blocks")
    return st


def fa_fp8_prep_varlen(q, k, v, q8, k8, v8, q_scale, k_scale, v_scale, sigma, B, H, cu_seqlens_q,
                       cu_seqlens_k, cu_blocks_q, cu_blocks_k, total_q, total_k, max_seqlen_q, max_seqlen_k, D,
                       in_dtype=None, stream=None, check=True) -> int:
    """Raw entry point: ``fa_fp8_prep`` over packed variable-length sequences."""
    if in_dtype is None:
        in_dtype = _DTYPE[(q if q is not None else k).dtype]
    st = lib().fa_fp8_prep_varlen(_ptr(q), _ptr(k), _ptr(v), int(in_dtype), _ptr(q8), _ptr(k8), _ptr(v8),
                                  _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), _ptr(sigma), int(B), int(H),
                                  _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(cu_blocks_q), _ptr(cu_blocks_k),
                                  int(total_q), int(total_k), int(max_seqlen_q), int(max_seqlen_k), int(D),
                                  _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fp8_prep_varlen")
    return st


def fa_fwd_fp8_varlen(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B, H, cu_seqlens_q, cu_seqlens_k,
                      cu_blocks_q, cu_blocks_k, total_q, total_k, max_seqlen_q, max_seqlen_k, D, scale, causal,
                      stream=None, check=True) -> int:
    """Raw entry point: ``fa_fwd_fp8`` over packed variable-length sequences."""
    st = lib().fa_fwd_fp8_varlen(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale),
                                 _ptr(o), _ptr(lse), int(B), int(H), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                 _ptr(cu_blocks_q), _ptr(cu_blocks_k), int(total_q), int(total_k),
                                 int(max_seqlen_q), int(max_seqlen_k), int(D), float(scale), int(bool(causal)),
                                 _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_fp8_varlen")
    return st


def _fp8_side_varlen(x, cu, H, dev, stream, names):
    """e4m3 codes, block offsets and scale arrays of one packed side."""
    B = cu.numel() - 1
    total = x.shape[0]
    cb = torch.empty(B + 1, dtype=torch.int32, device=dev)
    fa_varlen_blocks(cu, B, cb, stream=stream)
    nb = total // 128 + B   # upper bound on cu_blocks[B]
    out = {n: torch.empty((nb, H), dtype=torch.float32, device=dev) for n in names[1:]}
    out[names[0]] = cb
    return out


def fp8_prepare_varlen(q, k, v, sigma, *, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, stream=None):
    """Varlen ``fp8_prepare``: q ``[total_q, H, D]``, k/v ``[total_k, H, D]``
    16-bit, ``cu_seqlens_*`` int32 CUDA tensors. Either side may be None (q,
    or k and v): that side is skipped, so a K/V cache is prepared once and
    reused. Scale arrays ``[n_blocks, H]`` are allocated at their upper bound
    ``total // 128 + B`` rows; the first ``cu_blocks[B]`` rows are written."""
    ref = q if q is not None else k
    H, D = ref.shape[1], ref.shape[2]
    dev = ref.device
    B = (cu_seqlens_q if cu_seqlens_q is not None else cu_seqlens_k).numel() - 1
    out = {"B": B, "H": H, "D": D, "varlen": True}
    if q is not None:
        out.update(_fp8_side_varlen(q, cu_seqlens_q, H, dev, stream, ("cu_blocks_q", "q_scale")))
        out.update(q8=torch.empty(q.shape, dtype=torch.uint8, device=dev), cu_seqlens_q=cu_seqlens_q,
                   total_q=q.shape[0], max_seqlen_q=max_seqlen_q)
    if k is not None:
        out.update(_fp8_side_varlen(k, cu_seqlens_k, H, dev, stream, ("cu_blocks_k", "k_scale", "v_scale")))
        out.update(k8=torch.empty(k.shape, dtype=torch.uint8, device=dev),
                   v8=torch.empty(v.shape, dtype=torch.uint8, device=dev), cu_seqlens_k=cu_seqlens_k,
                   total_k=k.shape[0], max_seqlen_k=max_seqlen_k)
    g = out.get
    fa_fp8_prep_varlen(q, k, v, g("q8"), g("k8"), g("v8"), g("q_scale"), g("k_scale"), g("v_scale"), sigma, B, H,
                       g("cu_seqlens_q"), g("cu_seqlens_k"), g("cu_blocks_q"), g("cu_blocks_k"), g("total_q", 0),
                       g("total_k", 0), g("max_seqlen_q", 0) if q is not None else 0,
                       g("max_seqlen_k", 0) if k is not None else 0, D,
                       in_dtype=_DTYPE[ref.dtype], stream=stream)
    return out


def fp8_prepare(q, k, v, sigma, *, batch, stream=None):
    """Allocate the e4m3 tensors and block scales and call ``fa_fp8_prep``.
    q ``[B*Sq, H, D]``, k/v ``[B*Sk, H, D]`` 16-bit. Returns a dict."""
    B = batch
    H, D = q.shape[1], q.shape[2]
    Sq, Sk = q.shape[0] // B, k.shape[0] // B
    dev = q.device
    out = {"q8": torch.empty(q.shape, dtype=torch.uint8, device=dev),
           "k8": torch.empty(k.shape, dtype=torch.uint8, device=dev),
           "v8": torch.empty(v.shape, dtype=torch.uint8, device=dev),
           "q_scale": torch.empty((B, H, (Sq + 127) // 128), dtype=torch.float32, device=dev),
           "k_scale": torch.empty((B, H, (Sk + 127) // 128), dtype=torch.float32, device=dev),
           "v_scale": torch.empty((B, H, (Sk + 127) // 128), dtype=torch.float32, device=dev),
           "B": B, "H": H, "Sq": Sq, "Sk": Sk, "D": D}
    fa_fp8_prep(q, k, v, out["q8"], out["k8"], out["v8"], out["q_scale"], out["k_scale"], out["v_scale"],
                sigma, B, H, Sq, Sk, D, stream=stream)
    return out


def fp8_attention_forward(prep, *, causal=False, scale=None, out=None, lse=None, stream=None):
    """Attention on the output of ``fp8_prepare`` (or of ``fp8_prepare_varlen``,
    or a dict merging a Q preparation with a K/V one); returns (O bf16, LSE
    fp32 ``[B, H, Sq]``, varlen ``[H, total_q]``)."""
    if prep.get("varlen"):
        p = prep
        H, D = p["H"], p["D"]
        if scale is None:
            scale = D ** -0.5
        dev = p["q8"].device
        if out is None:
            out = torch.empty((p["total_q"], H, D), dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.empty((H, p["total_q"]), dtype=torch.float32, device=dev)
        fa_fwd_fp8_varlen(p["q8"], p["k8"], p["v8"], p["q_scale"], p["k_scale"], p["v_scale"], out, lse, p["B"], H,
                          p["cu_seqlens_q"], p["cu_seqlens_k"], p["cu_blocks_q"], p["cu_blocks_k"], p["total_q"],
                          p["total_k"], p["max_seqlen_q"], p["max_seqlen_k"], D, scale, causal, stream=stream)
        return out, lse
    B, H, Sq, Sk, D = prep["B"], prep["H"], prep["Sq"], prep["Sk"], prep["D"]
    if scale is None:
        scale = D ** -0.5
    dev = prep["q8"].device
    if out is None:
        out = torch.empty((B * Sq, H, D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=dev)
    fa_fwd_fp8(prep["q8"], prep["k8"], prep["v8"], prep["q_scale"], prep["k_scale"], prep["v_scale"], out, lse,
               B, H, Sq, Sk, D, scale, causal, stream=stream)
    return out, lse


def fa_get_device_status(stream=None, check=True):
    raw = ctypes.c_int(0)
    st = lib().fa_get_device_status(_stream(stream), ctypes.byref(raw))
    if check and st != FA_OK:
        raise FAError(st, f"device status word 0x{raw.value:x}")
    return st, raw.value


def attention_forward(q, k, v, *, causal=False, scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
                      max_seqlen_q=None, max_seqlen_k=None, batch=None, out=None, lse=None, stream=None):
    """Allocate O and LSE and call ``fa_fwd``.

    Fixed length: q ``[B*Sq, H, D]`` (or ``[B, Sq, H, D]``), k/v likewise; give
    ``batch`` when passing the flattened form. Varlen: ``cu_seqlens_*`` int32
    CUDA tensors and ``max_seqlen_*``. Returns (O, LSE) with LSE fp32
    ``[B, H, Sq]`` (fixed) or ``[H, total_q]`` (varlen).
    """
    if q.dim() == 4:
        B, Sq, H, D = q.shape
        Sk = k.shape[1]
        q, k, v = q.reshape(B * Sq, H, D), k.reshape(B * Sk, H, D), v.reshape(B * Sk, H, D)
    else:
        H, D = q.shape[1], q.shape[2]
        if cu_seqlens_q is None:
            B = batch
            Sq, Sk = q.shape[0] // B, k.shape[0] // B
        else:
            B = cu_seqlens_q.numel() - 1
            Sq, Sk = max_seqlen_q, max_seqlen_k
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors")
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        shape = (H, q.shape[0]) if cu_seqlens_q is not None else (B, H, Sq)
        lse = torch.empty(shape, device=q.device, dtype=torch.float32)
    fa_fwd(q, k, v, out, lse, B, H, Sq, Sk, D, scale, causal, cu_seqlens_q, cu_seqlens_k,
           q.shape[0], k.shape[0], stream=stream)
    return out, lse


def fa_bwd_workspace_size(H, total_q) -> int:
    return int(lib().fa_bwd_workspace_size(int(H), int(total_q)))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, Sq, Sk, D, scale, causal, cu_seqlens_q=None,
           cu_seqlens_k=None, total_q=0, total_k=0, workspace=None, workspace_bytes=0, dtype=None, stream=None,
           check=True) -> int:
    """Raw entry point: dQ, dK, dV of the attention forward for upstream gradient dO."""
    if dtype is None:
        dtype = _DTYPE[q.dtype]
    st = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                      int(B), int(H), int(Sq), int(Sk), int(D), float(scale), int(bool(causal)),
                      _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(total_q), int(total_k), _ptr(workspace),
                      int(workspace_bytes), int(dtype), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_bwd")
    return st


def attention_backward(q, k, v, o, lse, dout, *, causal=False, scale=None, cu_seqlens_q=None, cu_seqlens_k=None,
                       max_seqlen_q=None, max_seqlen_k=None, batch=None, workspace=None, stream=None):
    """Allocate dQ, dK, dV (and the scratch) and call ``fa_bwd``. Arguments
    as ``attention_forward``; ``o`` and ``lse`` are its outputs, ``dout`` the
    gradient of ``o``. Returns (dQ, dK, dV)."""
    H, D = q.shape[1], q.shape[2]
    if cu_seqlens_q is None:
        B = batch
        Sq, Sk = q.shape[0] // B, k.shape[0] // B
    else:
        B = cu_seqlens_q.numel() - 1
        Sq, Sk = max_seqlen_q, max_seqlen_k
    if scale is None:
        scale = D ** -0.5
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = fa_bwd_workspace_size(H, q.shape[0])
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, Sq, Sk, D, scale, causal, cu_seqlens_q, cu_seqlens_k,
           q.shape[0], k.shape[0], workspace, workspace.numel() * workspace.element_size(), stream=stream)
    return dq, dk, dv


def fa_fwd_paged(q, k_cache, v_cache, block_table, seqlens_k, o, lse, B, H, Sq, D, num_pages, page_size, max_pages,
                 scale, causal, num_splits=1, workspace=None, workspace_bytes=0, cu_seqlens_q=None, total_q=0,
                 dtype=None, stream=None, check=True) -> int:
    """Raw entry point: attention over K/V held in a paged cache."""
    if dtype is None:
        dtype = _DTYPE[q.dtype]
    st = lib().fa_fwd_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seqlens_k), _ptr(o),
                            _ptr(lse), int(B), int(H), int(Sq), int(D), int(num_pages), int(page_size),
                            int(max_pages), float(scale), int(bool(causal)), _ptr(cu_seqlens_q), int(total_q),
                            int(num_splits), _ptr(workspace), int(workspace_bytes), int(dtype), _stream(stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_paged")
    return st


def attention_forward_paged(q, k_cache, v_cache, block_table, seqlens_k, *, causal=False, scale=None, num_splits=1,
                            cu_seqlens_q=None, max_seqlen_q=None, out=None, lse=None, stream=None):
    """Allocate O, LSE (and the split workspace) and call ``fa_fwd_paged``.
    q ``[B*Sq, H, D]`` (or packed ``[total_q, H, D]`` with ``cu_seqlens_q``
    and ``max_seqlen_q``); caches ``[num_pages, page_size, H, D]``;
    block_table int32 ``[B, max_pages]``; seqlens_k int32 ``[B]``. Returns
    (O, LSE ``[B, H, Sq]``, packed ``[H, total_q]``)."""
    B, max_pages = block_table.shape
    num_pages, page_size, H, D = k_cache.shape
    Sq = q.shape[0] // B if cu_seqlens_q is None else max_seqlen_q
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        shape = (B, H, Sq) if cu_seqlens_q is None else (H, q.shape[0])
        lse = torch.empty(shape, device=q.device, dtype=torch.float32)
    ws, ws_bytes = None, 0
    if num_splits != 1:
        ws_bytes = fa_fwd_splitkv_workspace_size(B, H, Sq, max_pages * page_size, D, num_splits)
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    fa_fwd_paged(q, k_cache, v_cache, block_table, seqlens_k, out, lse, B, H, Sq, D, num_pages, page_size, max_pages,
                 scale, causal, num_splits, ws, ws_bytes, cu_seqlens_q=cu_seqlens_q, total_q=q.shape[0],
                 stream=stream)
    return out, lse


# --------------------------------------------------------------------------
# rotary positions with several axes
# --------------------------------------------------------------------------
def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _current_device() -> int:
    """Index of the current CUDA device."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _on(device, *tensors):
    """True if every tensor (or None) is on CUDA device number ``device``."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            return False
    return True


def _handle(stream, device):
    """cudaStream_t of ``stream``, or of the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(stream, shape, dtype, device):
    """A new tensor that belongs to ``stream`` (memory that a call allocates and
    gives back must not be handed on while its kernels still run there)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(stream, x):
    """A new contiguous tensor of x's shape and type, as ``_empty``."""
    if stream is None and x.is_contiguous():
        return torch.empty_like(x)
    return _empty(stream, x.shape, x.dtype, x.device)


def _addr(t):
    return None if t is None else t.data_ptr()


class RotaryPlan(NamedTuple):
    """Frequencies and axes of the pairs of a head; made by ``rotary_plan``."""
    rot_dim: int
    n_axes: int
    interleaved: bool
    inv_freq: ctypes.Array
    axis: ctypes.Array


@functools.lru_cache(maxsize=64)
def rotary_plan(rot_dim, sections, *, base=10000.0, interleaved=False, cyclic=False, per_axis=False, inv_freq=None):
    """Plan of a rotation of the first ``rot_dim`` elements of a head.

    ``sections`` (a tuple) gives the number of pairs that each axis turns,
    ``rot_dim / 2`` in all: the first ``sections[0]`` pairs follow axis 0 and
    so on, or, with ``cyclic``, the axes take pairs in turn while they have
    any left. Pair j turns at ``base ** (-2 j / rot_dim)`` per position; with
    ``per_axis`` every axis has the whole range of frequencies (pair i of the
    n of an axis: ``base ** (-i / n)``); ``inv_freq`` (a tuple of rot_dim / 2
    numbers) gives them outright. ``interleaved``: pair j is elements
    (2j, 2j + 1) instead of (j, j + rot_dim / 2).
    """
    sections = tuple(int(n) for n in sections)
    _need(rot_dim >= 2 and rot_dim % 2 == 0 and rot_dim <= 256, "rot_dim must be even, 2 to 256")
    _need(0 < len(sections) <= 127 and min(sections) >= 0 and sum(sections) == rot_dim // 2,
          "sections must be non-negative and add up to rot_dim / 2")
    axis, index = [], []
    if cyclic:
        used = [0] * len(sections)
        while len(axis) < rot_dim // 2:
            for a, n in enumerate(sections):
                if used[a] < n:
                    axis.append(a)
                    index.append(used[a])
                    used[a] += 1
    else:
        for a, n in enumerate(sections):
            axis += [a] * n
            index += range(n)
    if inv_freq is None:
        if per_axis:
            inv_freq = [base ** (-i / sections[a]) for a, i in zip(axis, index)]
        else:
            inv_freq = [base ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)]
    _need(len(inv_freq) == rot_dim // 2 and all(math.isfinite(f) for f in inv_freq),
          "inv_freq must hold rot_dim / 2 finite numbers")
    return RotaryPlan(rot_dim, len(sections), bool(interleaved), (ctypes.c_double * len(axis))(*inv_freq),
                      (ctypes.c_byte * len(axis))(*axis))


def fa_rope(q, k, q_out, k_out, positions, T, Hq, Hk, D, rot_dim, n_axes, inv_freq, axis, interleaved, inverse,
            strides=None, dtype=None, stream=None, check=True) -> int:
    """Raw entry point: rotary positions; ``inv_freq``, ``axis`` and
    ``strides`` are ctypes arrays."""
    ref = q if q is not None else k
    st = lib().fa_rope(_addr(q), _addr(k), _addr(q_out), _addr(k_out), positions.data_ptr(), T, Hq, Hk, D, rot_dim, n_axes,
                       inv_freq, axis, interleaved, inverse, strides, _DTYPE[ref.dtype] if dtype is None else dtype,
                       _handle(stream, ref.get_device()))
    if check and st != FA_OK:
        raise FAError(st, "fa_rope")
    return st


_Strides8 = ctypes.c_longlong * 8
_Strides4 = ctypes.c_longlong * 4


def _rotary(q, k, positions, plan, out, stream, inverse):
    # (single-token calls are bound by this function: checks are written out,
    # and the library is called without the raw wrapper)
    ref = k if q is None else q
    if ref is None:
        raise ValueError("q or k must be given")
    dev = _current_device()
    if ref.get_device() != dev or positions.get_device() != dev:
        raise ValueError("q, k and positions must be on the current CUDA device")
    rot_dim, n_axes, interleaved, inv_freq, axis = plan
    dtype = _DTYPE.get(ref.dtype)
    shape = ref.shape
    if dtype is None or len(shape) != 3:
        raise ValueError("q and k must be fp16 or bf16 [T, H, D]")
    T, H, D = shape
    if rot_dim > D:
        raise ValueError("the plan rotates more than a head holds")
    if positions.dtype != torch.int32 or positions.shape != (n_axes, T) or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int32 tensor of shape {(n_axes, T)}")
    dense = ref.is_contiguous()
    Hk = H
    if q is None:
        H = 0
    elif k is None:
        Hk = 0
    else:
        kshape = k.shape
        if k.get_device() != dev or k.dtype != q.dtype or len(kshape) != 3 or kshape[0] != T or kshape[2] != D:
            raise ValueError("q and k must be [T, H, D] of one type on one device")
        Hk = kshape[1]
        dense = dense and k.is_contiguous()
    if out is None:
        qo, ko = None if q is None else _empty_like(stream, q), None if k is None else _empty_like(stream, k)
    else:
        qo, ko = out
        for x, y in ((q, qo), (k, ko)):
            if (x is None) != (y is None) or (x is not None and (y.shape != x.shape or y.dtype != x.dtype
                                                                  or y.get_device() != dev)):
                raise ValueError("out must have the inputs' shapes, type and device")
            dense = dense and (y is None or y.is_contiguous())
    strides = None
    if not dense:
        st = []
        for x in (q, qo, k, ko):
            xt, xh, xd = (0, 0, 1) if x is None else x.stride()
            if xd != 1:
                raise ValueError("D must be contiguous")
            st += (xt, xh)
        strides = _Strides8(*st)
    st = (_lib or lib()).fa_rope(None if q is None else q.data_ptr(), None if k is None else k.data_ptr(),
                                 None if q is None else qo.data_ptr(), None if k is None else ko.data_ptr(),
                                 positions.data_ptr(), T, H, Hk, D, rot_dim, n_axes, inv_freq, axis, interleaved, inverse,
                                 strides, dtype, _handle(stream, dev))
    if st != FA_OK:
        raise FAError(st, "fa_rope")
    return qo, ko


def rotary_forward(q, k, positions, plan, *, out=None, stream=None):
    """Rotate q ``[T, Hq, D]`` and k ``[T, Hk, D]`` (either may be None; any
    strides with D contiguous) by ``positions``, int32 ``[n_axes, T]``, as
    ``plan`` says. ``out``: a pair of tensors to write, (q, k) itself for in
    place. Returns the rotated pair."""
    return _rotary(q, k, positions, plan, out, stream, 0)


def rotary_backward(dq, dk, positions, plan, *, out=None, stream=None):
    """Gradients of ``rotary_forward``'s q and k for the gradients of its
    outputs; arguments as there."""
    return _rotary(dq, dk, positions, plan, out, stream, 1)


# --------------------------------------------------------------------------
# the paged K/V cache: written, read back, attended to
# --------------------------------------------------------------------------
class KVCache(NamedTuple):
    """A paged cache: k, v ``[num_pages, page_size, Hk, D]`` fp16, bf16,
    float8_e4m3fn or int8; for the 8-bit types also k_scale, v_scale fp32
    ``[num_pages, Hk, page_size]`` (value = code * scale)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def kv_cache(num_pages, page_size, H, D, *, dtype=torch.float8_e4m3fn, device=None):
    """An empty cache (zeros) of ``H`` K/V heads."""
    _need(dtype in _CACHE_DTYPE, "a cache is fp16, bf16, float8_e4m3fn or int8")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    shape = (num_pages, page_size, H, D)
    if dtype in _DTYPE:
        return KVCache(*(torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)))
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
    ks, vs = (torch.zeros((num_pages, H, page_size), dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


def _cache_args(cache, block_table, seqlens_k, dev):
    """Checks a cache and its tables; returns (num_pages, page_size, H, D, B,
    max_pages, cache dtype)."""
    k, v, ks, vs = cache
    kt = k.dtype
    cd = _CACHE_DTYPE.get(kt)
    shape = k.shape
    if (cd is None or len(shape) != 4 or v.shape != shape or v.dtype != kt or not k.is_contiguous()
            or not v.is_contiguous()):
        raise ValueError("cache k and v must be contiguous [num_pages, page_size, H, D] of one cache type")
    num_pages, page_size, H, D = shape
    if cd >= FA_FP8_E4M3:
        scales = (num_pages, H, page_size)
        if (ks is None or vs is None or ks.shape != scales or vs.shape != scales or ks.dtype != torch.float32
                or vs.dtype != torch.float32 or not ks.is_contiguous() or not vs.is_contiguous()):
            raise ValueError("an 8-bit cache needs contiguous fp32 scales [num_pages, H, page_size]")
        if ks.get_device() != dev or vs.get_device() != dev:
            raise ValueError("the cache must be on the current CUDA device")
    table = block_table.shape
    if len(table) != 2 or block_table.dtype != torch.int32 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [B, max_pages]")
    B, max_pages = table
    if seqlens_k.shape != (B,) or seqlens_k.dtype != torch.int32 or not seqlens_k.is_contiguous():
        raise ValueError("seqlens_k must be a contiguous int32 [B]")
    if (k.get_device() != dev or v.get_device() != dev or block_table.get_device() != dev
            or seqlens_k.get_device() != dev):
        raise ValueError("the cache and its tables must be on the current CUDA device")
    return num_pages, page_size, H, D, B, max_pages, cd


def _rows_per_seq(T, B, cu, max_seqlen, name, dev):
    """Rows of each sequence: T / B, or the bound of the packed form."""
    if cu is None:
        if T and (B == 0 or T % B):
            raise ValueError(f"{name} has {T} rows, not a multiple of {B} sequences")
        return T // B if B else 0
    if cu.shape != (B + 1,) or cu.dtype != torch.int32 or not cu.is_contiguous() or cu.get_device() != dev:
        raise ValueError("cu_seqlens must be a contiguous int32 [B + 1] on the current CUDA device")
    if max_seqlen is None:
        raise ValueError("packed rows need max_seqlen_q")
    if T and B and max_seqlen < 1:
        raise ValueError(f"{name} has {T} rows, but max_seqlen_q is {max_seqlen}")
    return max_seqlen


def fa_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, B, H, Sq, D, num_pages, page_size,
                 max_pages, strides=None, cu_seqlens_q=None, total_q=0, dtype=None, cache_dtype=None, stream=None,
                 check=True) -> int:
    """Raw entry point: the newest keys and values into their pages."""
    st = lib().fa_kv_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale),
                            _addr(v_scale), block_table.data_ptr(), seqlens_k.data_ptr(), B, H, Sq, D, num_pages, page_size,
                            max_pages, strides, _addr(cu_seqlens_q), total_q, _DTYPE[k.dtype] if dtype is None else dtype,
                            _CACHE_DTYPE[k_cache.dtype] if cache_dtype is None else cache_dtype,
                            _handle(stream, k.get_device()))
    if check and st != FA_OK:
        raise FAError(st, "fa_kv_append")
    return st


def kv_cache_append(k, v, cache, block_table, seqlens_k, *, cu_seqlens_q=None, max_seqlen_q=None, stream=None):
    """Write the newest keys and values, k and v ``[B*Sq, H, D]`` (or packed
    ``[total_q, H, D]`` with ``cu_seqlens_q`` and ``max_seqlen_q``; any
    strides with D contiguous), into the pages of their sequences, quantised
    if the cache is 8-bit. ``seqlens_k`` counts the new keys too. Returns the
    cache."""
    dev = _current_device()
    num_pages, page_size, H, D, B, max_pages, cd = _cache_args(cache, block_table, seqlens_k, dev)
    shape = k.shape
    dtype = _DTYPE.get(k.dtype)
    if dtype is None or v.dtype != k.dtype or len(shape) != 3 or shape[1] != H or shape[2] != D or v.shape != shape:
        raise ValueError("k and v must be [T, H, D] of one 16-bit type, with the cache's heads")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("k and v must be on the current CUDA device")
    T = shape[0]
    Sq = _rows_per_seq(T, B, cu_seqlens_q, max_seqlen_q, "k", dev)
    strides = None
    if not (k.is_contiguous() and v.is_contiguous()):
        kt, kh, kd = k.stride()
        vt, vh, vd = v.stride()
        if kd != 1 or vd != 1:
            raise ValueError("D must be contiguous")
        strides = _Strides4(kt, kh, vt, vh)
    fa_kv_append(k, v, cache[0], cache[1], cache[2], cache[3], block_table, seqlens_k, B, H, Sq, D, num_pages, page_size,
                 max_pages, strides, cu_seqlens_q, T, dtype, cd, stream)
    return cache


def fa_kv_read(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, cu_seqlens_k, k, v, B, H, D, num_pages,
               page_size, max_pages, total_k, dtype=None, cache_dtype=None, stream=None, check=True) -> int:
    """Raw entry point: cached keys and values back into packed tensors."""
    st = lib().fa_kv_read(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale), block_table.data_ptr(),
                          seqlens_k.data_ptr(), cu_seqlens_k.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, D, num_pages,
                          page_size, max_pages, total_k, _DTYPE[k.dtype] if dtype is None else dtype,
                          _CACHE_DTYPE[k_cache.dtype] if cache_dtype is None else cache_dtype,
                          _handle(stream, k.get_device()))
    if check and st != FA_OK:
        raise FAError(st, "fa_kv_read")
    return st


def kv_cache_read(cache, block_table, seqlens_k, cu_seqlens_k, *, total_k, dtype=None, out=None, stream=None):
    """The first ``cu_seqlens_k[b+1] - cu_seqlens_k[b]`` keys and values of
    every sequence as packed ``[total_k, H, D]`` tensors of ``dtype`` (default:
    the cache's own for a 16-bit one, else bf16), as ``attention_forward``
    takes them. ``out``: a pair of tensors to write."""
    dev = _current_device()
    num_pages, page_size, H, D, B, max_pages, cd = _cache_args(cache, block_table, seqlens_k, dev)
    if cu_seqlens_k.shape != (B + 1,) or cu_seqlens_k.dtype != torch.int32 or not cu_seqlens_k.is_contiguous():
        raise ValueError("cu_seqlens_k must be a contiguous int32 [B + 1]")
    shape = (total_k, H, D)
    if cu_seqlens_k.get_device() != dev:
        raise ValueError("cu_seqlens_k must be on the current CUDA device")
    if out is None:
        if dtype is None:
            dtype = cache.k.dtype if cd < FA_FP8_E4M3 else torch.bfloat16
        elif dtype not in _DTYPE:
            raise ValueError("dtype must be fp16 or bf16")
        device = cache[0].device
        k, v = _empty(stream, shape, dtype, device), _empty(stream, shape, dtype, device)
    else:
        k, v = out
        if (k.dtype not in _DTYPE or v.dtype != k.dtype or k.shape != shape or v.shape != shape or not k.is_contiguous()
                or not v.is_contiguous()):
            raise ValueError("out must be two contiguous [total_k, H, D] tensors of one 16-bit type")
        if k.get_device() != dev or v.get_device() != dev:
            raise ValueError("out must be on the current CUDA device")
    fa_kv_read(cache[0], cache[1], cache[2], cache[3], block_table, seqlens_k, cu_seqlens_k, k, v, B, H, D, num_pages,
               page_size, max_pages, total_k, _DTYPE[k.dtype], cd, stream)
    return k, v


def fa_fwd_kvcache_workspace_size(B, Hq, Hk, Sq, D, total_q=0, prefix_len=0) -> int:
    return int(lib().fa_fwd_kvcache_workspace_size(int(B), int(Hq), int(Hk), int(Sq), int(D), int(total_q),
                                                   int(prefix_len)))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(device, B, Hq, Hk, Sq, D, total_q, prefix_len):
    """``fa_fwd_kvcache_workspace_size`` on the current device, ``device``."""
    return fa_fwd_kvcache_workspace_size(B, Hq, Hk, Sq, D, total_q, prefix_len)


def fa_fwd_kvcache(q, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, o, lse, B, Hq, Hk, Sq, D, num_pages,
                   page_size, max_pages, scale, causal, workspace, workspace_bytes, cu_seqlens_q=None, total_q=0,
                   dtype=None, cache_dtype=None, stream=None, check=True) -> int:
    """Raw entry point: attention of a few query rows over a paged cache."""
    st = lib().fa_fwd_kvcache(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                              block_table.data_ptr(), seqlens_k.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hk, Sq, D,
                              num_pages, page_size, max_pages, scale, causal, _addr(cu_seqlens_q), total_q,
                              workspace.data_ptr(), workspace_bytes, _DTYPE[q.dtype] if dtype is None else dtype,
                              _CACHE_DTYPE[k_cache.dtype] if cache_dtype is None else cache_dtype,
                              _handle(stream, q.get_device()))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_kvcache")
    return st


def fa_fwd_prefix(q, k_cache, v_cache, k_scale, v_scale, prefix_pages, prefix_len, block_table, seqlens_k, o, lse, B,
                  Hq, Hk, Sq, D, num_pages, page_size, max_pages, scale, causal, workspace, workspace_bytes,
                  cu_seqlens_q=None, total_q=0, dtype=None, cache_dtype=None, stream=None, check=True) -> int:
    """Raw entry point: the same for a batch that shares its first keys."""
    st = lib().fa_fwd_prefix(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale), _addr(v_scale),
                             _addr(prefix_pages), prefix_len, block_table.data_ptr(), seqlens_k.data_ptr(), o.data_ptr(),
                             lse.data_ptr(), B, Hq, Hk, Sq, D, num_pages, page_size, max_pages, scale, causal,
                             _addr(cu_seqlens_q), total_q, workspace.data_ptr(), workspace_bytes,
                             _DTYPE[q.dtype] if dtype is None else dtype,
                             _CACHE_DTYPE[k_cache.dtype] if cache_dtype is None else cache_dtype,
                             _handle(stream, q.get_device()))
    if check and st != FA_OK:
        raise FAError(st, "fa_fwd_prefix")
    return st


def _attention_kvcache(q, cache, prefix_pages, prefix_len, block_table, seqlens_k, causal, scale, cu_seqlens_q,
                       max_seqlen_q, out, lse, workspace, stream):
    dev = _current_device()
    num_pages, page_size, Hk, D, B, max_pages, cd = _cache_args(cache, block_table, seqlens_k, dev)
    k, v, ks, vs = cache
    dtype = _DTYPE.get(q.dtype)
    shape = q.shape
    if dtype is None or len(shape) != 3 or shape[2] != D or shape[1] % Hk or not q.is_contiguous():
        raise ValueError("q must be contiguous fp16 or bf16 [T, Hq, D], Hq a multiple of the cache's heads")
    T, Hq, _ = shape
    Sq = _rows_per_seq(T, B, cu_seqlens_q, max_seqlen_q, "q", dev)
    if prefix_pages is not None:
        n = -(-prefix_len // page_size)
        if prefix_pages.shape != (n,) or prefix_pages.dtype != torch.int32 or not prefix_pages.is_contiguous():
            raise ValueError(f"prefix_pages must be a contiguous int32 [{n}]")
        if prefix_pages.get_device() != dev:
            raise ValueError("every tensor must be on the current CUDA device")
    if q.get_device() != dev or not (out is lse is workspace is None or _on(dev, out, lse, workspace)):
        raise ValueError("every tensor must be on the current CUDA device")
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty_like(stream, q)
    elif out.shape != shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must be like q")
    shape = (B, Hq, Sq) if cu_seqlens_q is None else (Hq, T)
    if lse is None:
        lse = _empty(stream, shape, torch.float32, k.device)
    elif lse.shape != shape or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous fp32 {shape}")
    if workspace is None:
        nbytes = _workspace_bytes(dev, B, Hq, Hk, Sq, D, T, prefix_len) or 1
        workspace = _empty(stream, nbytes, torch.uint8, k.device)
    elif workspace.is_contiguous():
        nbytes = workspace.numel() * workspace.element_size()
    else:
        raise ValueError("workspace must be contiguous")
    # (single-token calls are bound by this function: the library is called
    # without the raw wrappers)
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), None if ks is None else ks.data_ptr(),
            None if vs is None else vs.data_ptr())
    tail = (block_table.data_ptr(), seqlens_k.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hk, Sq, D, num_pages,
            page_size, max_pages, D ** -0.5 if scale is None else scale, 1 if causal else 0,
            None if cu_seqlens_q is None else cu_seqlens_q.data_ptr(), T, workspace.data_ptr(), nbytes, dtype, cd,
            _handle(stream, dev))
    if prefix_pages is None:
        st = (_lib or lib()).fa_fwd_kvcache(*head, *tail)
    else:
        st = (_lib or lib()).fa_fwd_prefix(*head, prefix_pages.data_ptr(), prefix_len, *tail)
    if st != FA_OK:
        raise FAError(st, "fa_fwd_kvcache" if prefix_pages is None else "fa_fwd_prefix")
    return out, lse


def attention_forward_kvcache(q, cache, block_table, seqlens_k, *, causal=False, scale=None, cu_seqlens_q=None,
                              max_seqlen_q=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of q ``[B*Sq, Hq, D]`` (or packed ``[total_q, Hq, D]`` with
    ``cu_seqlens_q`` and ``max_seqlen_q``) over a paged ``KVCache`` whose heads
    are shared by ``Hq / Hk`` query heads each; a few rows per sequence
    (decoding). block_table int32 ``[B, max_pages]``, seqlens_k int32 ``[B]``.
    Allocates what is not given (workspace: ``fa_fwd_kvcache_workspace_size``
    bytes). Returns (O, LSE ``[B, Hq, Sq]``, packed ``[Hq, total_q]``)."""
    return _attention_kvcache(q, cache, None, 0, block_table, seqlens_k, causal, scale, cu_seqlens_q, max_seqlen_q, out,
                              lse, workspace, stream)


def attention_forward_prefix(q, cache, prefix_pages, prefix_len, block_table, seqlens_k, *, causal=False, scale=None,
                             cu_seqlens_q=None, max_seqlen_q=None, out=None, lse=None, workspace=None, stream=None):
    """``attention_forward_kvcache`` for a batch whose sequences all begin with
    the ``prefix_len`` keys in ``prefix_pages`` (int32 ``[ceil(prefix_len /
    page_size)]``): these are read once for the whole batch. block_table and
    seqlens_k name each sequence's own keys, which follow."""
    _need(prefix_len >= 0, "prefix_len must not be negative")
    _need(prefix_pages is not None or prefix_len == 0, "a prefix needs prefix_pages")
    return _attention_kvcache(q, cache, prefix_pages, prefix_len, block_table, seqlens_k, causal, scale, cu_seqlens_q,
                              max_seqlen_q, out, lse, workspace, stream)
