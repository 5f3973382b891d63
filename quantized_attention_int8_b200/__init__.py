"""INT8-QK / FP8-PV quantized attention for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI in ``include/sage.h`` (``libsage_b200.so``,
built in-tree by ``python quantized_attention_int8_b200/build_lib.py``).  The
functions keep the C entry points' names and only marshal arguments: torch
supplies device memory and the current CUDA stream, and every step of the
computation runs in the library's CUDA kernels.  There is no CPU fallback: if
the library is missing, importing this package fails.

    from quantized_attention_int8_b200 import sage_attn
    out = sage_attn(q, k, v, tensor_layout="HND", is_causal=False)

mirrors the ``sageattn(q, k, v, tensor_layout, is_causal, sm_scale)`` call of
the SageAttention README ("How to Use"); ``pv_accum_dtype`` selects "fp32" or
"fp16+fp32" accumulation of the P.V product (qwbw.cn article, pitfalls) and
``pv_dtype`` its operands: "fp8" (E4M3, the INT8-QK / FP8-PV kernel) or "fp16"
(the INT8-QK / FP16-PV kernel of the README's "Available APIs"); ``qk_quant_gran``
the Q scale granularity ("per_block", "per_warp", "per_thread") and ``smooth_v``
optional V smoothing (see ``sage_opts`` in include/sage.h).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sys

import torch

__all__ = [
    "SageError", "sage_attn", "sage_quantize", "sage_attn_quantized", "sage_qk_int32", "sage_check_status",
    "sage_workspace_bytes", "sage_device_supported", "sage_status_string", "padded_dim", "LIB_PATH", "capi",
    "sage_attn_noalloc", "SAGE_NOALLOC_MAX_BYTES", "load_checked", "CHECKED_LIB_PATH", "BINDING_PATH", "pv_mode", "sage_attn_varlen", "SageOpts", "opts",
    "sage_qk_norm_rope", "sage_kv_cache", "sage_cache_append", "sage_cache_gather", "sage_attn_decode",
    "sageattn", "sageattn_qk_int8_pv_fp8_cuda", "sageattn_qk_int8_pv_fp16_cuda", "sageattn_varlen",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsage_b200.so")
# the same library compiled with -DSAGE_CHECKED: every kernel store tests its extent first
CHECKED_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsage_b200_checked.so")

# the compiled binding of the serving calls (csrc/binding.cpp), of this Python and this torch; loaded by the first of them
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                            f"_sage_binding.{sys.implementation.cache_tag}-torch{torch.__version__}.so")

SAGE_OK, SAGE_ERR_INVALID_ARG, SAGE_ERR_UNSUPPORTED, SAGE_ERR_ARCH, SAGE_ERR_CUDA, SAGE_ERR_OOM, \
    SAGE_ERR_TIMEOUT, SAGE_ERR_BOUNDS = range(8)
SAGE_HND, SAGE_NHD = 0, 1
SAGE_FP16, SAGE_BF16, SAGE_FP32 = 0, 1, 2
SAGE_PV_FP32, SAGE_PV_FP16_FP32, SAGE_PV16_FP32, SAGE_PV16_FP16_FP32, SAGE_PV16_FP16 = 0, 1, 2, 3, 6

_LAYOUTS = {"HND": SAGE_HND, "NHD": SAGE_NHD}
_DTYPES = {torch.float16: SAGE_FP16, torch.bfloat16: SAGE_BF16, torch.float32: SAGE_FP32}
_PV = {("fp8", "fp32"): SAGE_PV_FP32, ("fp8", "fp16+fp32"): SAGE_PV_FP16_FP32,
       ("fp8", "fp32+fp16"): SAGE_PV_FP16_FP32,
       ("fp16", "fp32"): SAGE_PV16_FP32, ("fp16", "fp16+fp32"): SAGE_PV16_FP16_FP32,
       ("fp16", "fp16"): SAGE_PV16_FP16}


def pv_mode(pv_dtype: str = "fp8", pv_accum_dtype: str = "fp32") -> int:
    """The sage_pv_mode value for P.V operands ``pv_dtype`` and accumulation ``pv_accum_dtype``.

    "fp32+fp16" is the README's spelling of the two-level (fp16 tile, fp32 total)
    accumulation of the FP8 kernel.  "fp16" (pure fp16 accumulation with FP16 operands,
    the fastest and least overflow-safe option on the GPUs the pages target) maps to
    SAGE_PV16_FP16, which the library rejects with SAGE_ERR_UNSUPPORTED: on sm_100a a
    tcgen05 MMA issues at the same rate with an F16 or an F32 accumulator, so fp16
    accumulation would buy no speed and only add error and overflow risk.
    """
    try:
        return _PV[(pv_dtype, pv_accum_dtype)]
    except KeyError:
        raise ValueError(f"unsupported pv_dtype / pv_accum_dtype {pv_dtype!r} / {pv_accum_dtype!r}") from None


class SageOpts(ctypes.Structure):
    """The C ``sage_opts``: query tokens per Q scale (128, 32 or 1) and V smoothing (0 / 1)."""
    _fields_ = [("q_gran", ctypes.c_int), ("smooth_v", ctypes.c_int)]


_GRANS = {"per_block": 128, "per_warp": 32, "per_thread": 1}


def opts(qk_quant_gran: str = "per_block", smooth_v: bool = False) -> SageOpts:
    """SageOpts for a granularity name ("per_block", "per_warp", "per_thread") and V smoothing."""
    if qk_quant_gran not in _GRANS:
        raise ValueError(f"qk_quant_gran must be one of {sorted(_GRANS)}, got {qk_quant_gran!r}")
    return SageOpts(_GRANS[qk_quant_gran], 1 if smooth_v else 0)


class SageNormRope(ctypes.Structure):
    """The C ``sage_norm_rope``: RMS norm of the heads and their position rotation."""
    _fields_ = [("norm", ctypes.c_int), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int), ("cos_sin", ctypes.c_void_p),
                ("n_pos", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int)]


class SageKVCache(ctypes.Structure):
    """The C ``sage_kv_cache``: the four arrays of a paged cache and their sizes."""
    _fields_ = [("k8", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("v8", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int)]


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python quantized_attention_int8_b200/build_lib.py` "
            "(this package has no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    sig = {
        "sage_attn": ([P, P, P, P, I, I, I, I, I, I, I, I, F, I, P], I),
        "sage_workspace_bytes": ([I, I, I, I, I], Z),
        "sage_quantize": ([P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, P, P], I),
        "sage_attn_quantized": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P, P], I),
        "sage_qk_int32": ([P, P, I, I, I, I, I, P, I, P, P], I),
        "sage_check_status": ([P], I),
        "sage_status_string": ([I], ctypes.c_char_p),
        "sage_device_supported": ([], I),
        "sage_attn_noalloc": ([P, P, P, P, I, I, I, I, I, I, I, I, F, I, P], I),
        "sage_attn_ex": ([P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P, P], I),
        "sage_selftest_wait_timeout": ([I, P], I),
        "sage_mma_probe": ([I, I, ctypes.POINTER(ctypes.c_double), P], I),
        "sage_test_inject": ([I, I], None),
        "sage_test_out_limit": ([ctypes.c_longlong], None),
        "sage_checked_build": ([], I),
        "sage_qk_norm_rope": ([P, P, P, P, P, P, L, I, I, I, I, I, I, P, P], I),
        "sage_cache_append": ([P, P, P, P, P, P, P, L, I, P, P, P, I, I, I, I, P, P], I),
        "sage_cache_gather": ([P, P, L, I, P, P, P, P, P, I, I, I, P], I),
        "sage_attn_decode": ([P, L, L, P, P, L, I, P, P, I, I, I, I, F, P], I),
        "sage_attn_varlen": ([P, P, P, P, P, P, I, I, I, ctypes.c_longlong, ctypes.c_longlong, I, I, I, I, I, F, I, P,
                              P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    # the addresses that the compiled binding of the serving calls takes
    lib.serving = {name: ctypes.cast(getattr(lib, name), P).value
                   for name in ("sage_qk_norm_rope", "sage_cache_append", "sage_cache_gather", "sage_attn_decode")}
    return lib


_binding = None


def _serving():
    """The compiled binding, loaded on first use: nothing else in the package needs it."""
    global _binding
    if _binding is None:
        if not os.path.exists(BINDING_PATH):
            raise ImportError(f"{BINDING_PATH} is not built; run `python quantized_attention_int8_b200/build_lib.py` "
                              "(the serving calls need it)")
        spec = importlib.util.spec_from_file_location("_sage_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _binding = module
    return _binding


capi = _load()


def load_checked() -> ctypes.CDLL:
    """The checked build (``libsage_b200_checked.so``) with the same signatures as ``capi``.

    Its kernels test every global store against the buffer it belongs to, skip one that falls
    outside and report it through ``sage_check_status`` (SAGE_ERR_BOUNDS).  A second, independent
    copy of the library: its device state (error words, no-alloc workspace) is its own."""
    return _load(CHECKED_LIB_PATH)


class SageError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {sage_status_string(status)} (status {status})")


def sage_status_string(status: int) -> str:
    return capi.sage_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != SAGE_OK:
        raise SageError(status, where)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def padded_dim(d: int) -> int:
    if d > 256:
        raise ValueError("head_dim > 256 is not supported")
    return 64 if d <= 64 else (128 if d <= 128 else 256)


def _shape(q: torch.Tensor, k: torch.Tensor, layout: str):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be 4-D")
    if layout == "HND":
        B, Hq, N, d = q.shape
        Hkv, Nk = k.shape[1], k.shape[2]
    elif layout == "NHD":
        B, N, Hq, d = q.shape
        Hkv, Nk = k.shape[2], k.shape[1]
    else:
        raise ValueError(f"tensor_layout must be 'HND' or 'NHD', got {layout!r}")
    return B, Hq, Hkv, N, Nk, d


def _check_tensors(q, k, v):
    for t in (q, k, v):
        if not t.is_cuda:
            raise ValueError("q, k, v must be CUDA tensors (no CPU path exists)")
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    if not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share one dtype")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")


def _check_inputs_nk(q, k, v, layout):
    """(B, Hq, Hkv, Nq, Nk, d) of q and k, v, which may differ in length."""
    _check_tensors(q, k, v)
    B, Hq, Hkv, N, Nk, d = _shape(q, k, layout)
    kshape = (B, Hkv, Nk, d) if layout == "HND" else (B, Nk, Hkv, d)
    if tuple(k.shape) != kshape:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected {kshape}")
    return B, Hq, Hkv, N, Nk, d


def _check_inputs(q, k, v, layout):
    """(B, Hq, Hkv, N, d) of q, k, v of one length."""
    B, Hq, Hkv, N, Nk, d = _check_inputs_nk(q, k, v, layout)
    if Nk != N:
        raise ValueError(f"q has {N} tokens and k, v {Nk}; this entry point needs equal lengths")
    return B, Hq, Hkv, N, d


def sage_attn(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None, pv_accum_dtype="fp32", out=None,
              pv_dtype="fp8", qk_quant_gran="per_block", smooth_v=False):
    """Quantized attention of fp16/bf16 q (B,Hq,Nq,d), k/v (B,Hkv,Nk,d) (HND; NHD stores (B,N,H,d)).

    Nq may differ from Nk (then the causal mask is aligned bottom-right); non-default
    qk_quant_gran / smooth_v, or Nq != Nk, go through sage_attn_ex."""
    B, Hq, Hkv, N, Nk, d = _check_inputs_nk(q, k, v, tensor_layout)
    o = opts(qk_quant_gran, smooth_v)
    if out is None:
        out = torch.empty_like(q)
    scale = float(sm_scale) if sm_scale is not None else 0.0
    mode = pv_mode(pv_dtype, pv_accum_dtype)
    if Nk == N and o.q_gran == 128 and not o.smooth_v:
        st = capi.sage_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq, Hkv, N, d,
                            _DTYPES[q.dtype], _LAYOUTS[tensor_layout], int(bool(is_causal)), scale, mode, _stream())
        _check(st, "sage_attn")
    else:
        st = capi.sage_attn_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq, Hkv, N, Nk, d,
                               _DTYPES[q.dtype], _LAYOUTS[tensor_layout], int(bool(is_causal)), scale, mode,
                               ctypes.byref(o), _stream())
        _check(st, "sage_attn_ex")
    return out


def sage_attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, is_causal=False,
                     sm_scale=None, pv_accum_dtype="fp32", out=None, pv_dtype="fp8", qk_quant_gran="per_block",
                     smooth_v=False):
    """Packed batch: q (total_q, Hq, d), k/v (total_k, Hkv, d), cu_seqlens_* int32 CUDA tensors of
    B + 1 offsets (sequence b = tokens cu[b] .. cu[b+1]-1).  Each sequence attends to its own keys
    (causal: aligned bottom-right per sequence).  A bad offset table raises SageError from the
    status check after the launch."""
    _check_tensors(q, k, v)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("varlen q, k, v must be 3-D (tokens, heads, head_dim)")
    total_q, Hq, d = q.shape
    total_k, Hkv, dk = k.shape
    if dk != d:
        raise ValueError("q and k must have the same head_dim")
    for c in (cu_seqlens_q, cu_seqlens_k):
        if not (c.is_cuda and c.dtype == torch.int32 and c.dim() == 1 and c.is_contiguous()):
            raise ValueError("cu_seqlens must be contiguous 1-D int32 CUDA tensors")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both hold B + 1 >= 2 offsets")
    B = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    st = capi.sage_attn_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), cu_seqlens_q.data_ptr(),
                               cu_seqlens_k.data_ptr(), B, int(max_seqlen_q), int(max_seqlen_k), total_q, total_k,
                               Hq, Hkv, d, _DTYPES[q.dtype], int(bool(is_causal)),
                               float(sm_scale) if sm_scale is not None else 0.0, pv_mode(pv_dtype, pv_accum_dtype),
                               ctypes.byref(opts(qk_quant_gran, smooth_v)), _stream())
    _check(st, "sage_attn_varlen")
    return out


SAGE_NOALLOC_MAX_BYTES = 64 << 20


def sage_attn_noalloc(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None, pv_accum_dtype="fp32", out=None,
                      pv_dtype="fp8"):
    """sage_attn with no device allocation inside the library (for callers that cannot
    allocate at call time); the caller supplies ``out`` or torch allocates it here.  The
    library's static workspace holds problems up to SAGE_NOALLOC_MAX_BYTES of workspace
    (larger ones raise SageError with SAGE_ERR_INVALID_ARG); calls that may overlap on the
    GPU must be ordered by the caller."""
    B, Hq, Hkv, N, d = _check_inputs(q, k, v, tensor_layout)
    if out is None:
        out = torch.empty_like(q)
    st = capi.sage_attn_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, Hq, Hkv, N, d,
                                _DTYPES[q.dtype], _LAYOUTS[tensor_layout], int(bool(is_causal)),
                                float(sm_scale) if sm_scale is not None else 0.0, pv_mode(pv_dtype, pv_accum_dtype),
                        _stream())
    _check(st, "sage_attn_noalloc")
    return out


# ---------------------------------------------------------------------------------------------
# Serving: head norm and rotation, the paged cache, one-token attention (include/sage.h, "Serving").
# None of these record gradients.  They go through a compiled binding (csrc/binding.cpp), which checks the
# tensors, allocates the outputs and calls the same C functions: at a decode step's sizes the checks and
# conversions took longer in Python than the kernels.
# ---------------------------------------------------------------------------------------------
def sage_qk_norm_rope(q, k, positions=None, cos_sin=None, q_weight=None, k_weight=None, tensor_layout="HND", norm=True,
                      eps=1e-6, interleaved=False, q_out=None, k_out=None):
    """RMS norm of every query and key head and its position rotation in one launch; returns (q_out, k_out).

    q (B,Hq,N,d), k (B,Hkv,N,d) (HND; NHD stores (B,N,H,d)), or packed tokens (T,H,d); channels contiguous,
    otherwise any strides (slices of a fused projection).  k may be None.  cos_sin float32 (n_pos, rot): row p
    holds the rot/2 cosines of position p's angles, then the sines; channels i and i + rot/2 turn together, or
    2i and 2i + 1 with interleaved; None: no rotation.  positions int32 (N,) or (B,N), default 0..N-1; one
    outside the table leaves its token unwritten and is reported by sage_check_status.  Weights (d,) in fp16,
    bf16 or fp32.  q_out may be q and k_out may be k; outputs that overlap q, k or each other otherwise are refused
    (slices side by side of one fused tensor do not)."""
    if tensor_layout not in _LAYOUTS:
        raise ValueError(f"tensor_layout must be 'HND' or 'NHD', got {tensor_layout!r}")
    r = _serving().qk_norm_rope(capi.serving["sage_qk_norm_rope"], q, k, positions, tensor_layout == "HND", cos_sin,
                                q_weight, k_weight, norm, eps, interleaved, q_out, k_out)
    if type(r) is int:
        _check(r, "sage_qk_norm_rope")
    return r


def sage_kv_cache(num_pages, num_kv_heads, head_dim, page_size=64, device="cuda") -> dict:
    """An empty paged cache: k8 int8 and v8 uint8 (E4M3 codes) (num_pages, Hkv, page_size, dc) with
    dc = 16 * ceil(head_dim / 16), ks and vs float32 (num_pages, Hkv, page_size)."""
    shape = (num_pages, num_kv_heads, page_size)
    dc = (head_dim + 15) // 16 * 16
    return dict(k8=torch.zeros((*shape, dc), dtype=torch.int8, device=device),
                ks=torch.zeros(shape, dtype=torch.float32, device=device),
                v8=torch.zeros((*shape, dc), dtype=torch.uint8, device=device),
                vs=torch.zeros(shape, dtype=torch.float32, device=device))


def sage_cache_append(cache, k, v, page_table, seq_lens, cu_seqlens=None, q=None, cos_sin=None, q_weight=None,
                      k_weight=None, norm=False, eps=1e-6, interleaved=False, k_mean=None, q_out=None):
    """Quantizes new tokens k, v (T,Hkv,d) into the paged cache (a dict as sage_kv_cache returns).

    page_table int32 (B, max_pages), seq_lens int32 (B,): lengths with the new tokens; cu_seqlens int32 (B+1,): each
    sequence's tokens in the packed k and v, None: one token per sequence (length 0: an empty slot, skipped).
    norm, weights, cos_sin, interleaved: as sage_qk_norm_rope, on the keys at their positions, and on q (T,Hq,d),
    which is returned (q_out; None without q).  k_mean float32 (Hkv,d) is subtracted from the keys before
    they are coded.  Channels contiguous, other strides free.  Bad pages and positions are skipped and reported
    by sage_check_status.  q_out may be q; it must not overlap k, v or the cache (refused)."""
    r = _serving().cache_append(capi.serving["sage_cache_append"], cache["k8"], cache["ks"], cache["v8"], cache["vs"], k, v,
                                page_table, seq_lens, cu_seqlens, q, cos_sin, q_weight, k_weight, norm, eps, interleaved,
                                k_mean, q_out)
    if type(r) is int:
        _check(r, "sage_cache_append")
    return r


def sage_cache_gather(cache, page_table, cu_seqlens, total, head_dim, dtype=torch.float16, starts=None, k_mean=None,
                      k_out=None, v_out=None):
    """Reads cached tokens back as (k, v), each (total, Hkv, head_dim) of ``dtype``: token i of sequence b (rows
    cu_seqlens[b] .. cu_seqlens[b+1]-1) is position starts[b] + i (starts None: 0).  k_mean is added to the keys.
    Rows behind the last sequence, and rows of bad pages, are left unwritten."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    r = _serving().cache_gather(capi.serving["sage_cache_gather"], cache["k8"], cache["ks"], cache["v8"], cache["vs"],
                                page_table, cu_seqlens, total, head_dim, code, starts, k_mean, k_out, v_out)
    if type(r) is int:
        _check(r, "sage_cache_gather")
    return r


def sage_attn_decode(q, cache, page_table, seq_lens, max_seqlen, sm_scale=None, out=None):
    """Attention of one new token per sequence, q (B,Hq,d), over its cached tokens: out (B,Hq,d).

    seq_lens int32 (B,): the cached keys each query sees (0: zeros); max_seqlen bounds them (a longer sequence gets
    zeros and is reported by sage_check_status).  q may be strided (channels contiguous)."""
    r = _serving().attn_decode(capi.serving["sage_attn_decode"], cache["k8"], cache["ks"], cache["v8"], cache["vs"], q,
                               page_table, seq_lens, max_seqlen, 0.0 if sm_scale is None else sm_scale, out)
    if type(r) is int:
        _check(r, "sage_attn_decode")
    return r


def sage_workspace_bytes(B, Hq, Hkv, N, d) -> int:
    return int(capi.sage_workspace_bytes(B, Hq, Hkv, N, d))


def sage_quantize(q, k, v, tensor_layout="HND", pv_accum_dtype="fp32", pv_dtype="fp8", qk_quant_gran="per_block",
                  smooth_v=False) -> dict:
    """The quantize/smooth pass alone; returns the codes and scales as CUDA tensors.

    Layouts (Np = 128*ceil(N/128), dp = padded head dim): q8 int8 (B,Hq,Np,dp),
    qs f32 (B,Hq,Np/128), k8 int8 (B,Hkv,Np,dp), ks f32 (B,Hkv,Np/128),
    km f32 (B,Hkv,dp), v8t (B,Hkv,dp,Np) uint8 E4M3 codes (pv_dtype "fp8") or
    float16 codes (pv_dtype "fp16"), vs f32 (B,Hkv,dp), vm f32 (B,Hkv,dp) (V's token mean
    with smooth_v, else zeros); qs has Np / q_gran entries per head.
    """
    mode = pv_mode(pv_dtype, pv_accum_dtype)
    o = opts(qk_quant_gran, smooth_v)
    B, Hq, Hkv, N, d = _check_inputs(q, k, v, tensor_layout)
    dp, nb = padded_dim(d), (N + 127) // 128
    Np = nb * 128
    dev = q.device
    z = dict(
        q8=torch.empty((B, Hq, Np, dp), dtype=torch.int8, device=dev),
        qs=torch.empty((B, Hq, Np // o.q_gran), dtype=torch.float32, device=dev),
        k8=torch.empty((B, Hkv, Np, dp), dtype=torch.int8, device=dev),
        ks=torch.empty((B, Hkv, nb), dtype=torch.float32, device=dev),
        km=torch.empty((B, Hkv, dp), dtype=torch.float32, device=dev),
        v8t=torch.empty((B, Hkv, dp, Np), dtype=torch.float16 if pv_dtype == "fp16" else torch.uint8, device=dev),
        vs=torch.empty((B, Hkv, dp), dtype=torch.float32, device=dev),
        vm=torch.zeros((B, Hkv, dp), dtype=torch.float32, device=dev),
    )
    st = capi.sage_quantize(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, Hq, Hkv, N, d, _DTYPES[q.dtype],
                            _LAYOUTS[tensor_layout], mode, ctypes.byref(o),
                            *(z[n].data_ptr() for n in ("q8", "qs", "k8", "ks", "km", "v8t", "vs", "vm")), _stream())
    _check(st, "sage_quantize")
    z.update(B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, pv_dtype=pv_dtype, qk_quant_gran=qk_quant_gran, smooth_v=bool(smooth_v))
    return z


def sage_attn_quantized(z: dict, out_dtype=torch.float16, tensor_layout="HND", is_causal=False, sm_scale=None,
                        pv_accum_dtype="fp32", out=None):
    """The fused attention kernel alone on quantized buffers (the dict sage_quantize returns;
    its ``pv_dtype`` entry selects the P.V operands)."""
    B, Hq, Hkv, N, d = (z[n] for n in ("B", "Hq", "Hkv", "N", "d"))
    if out is None:
        shape = (B, Hq, N, d) if tensor_layout == "HND" else (B, N, Hq, d)
        out = torch.empty(shape, dtype=out_dtype, device=z["q8"].device)
    o = opts(z.get("qk_quant_gran", "per_block"), z.get("smooth_v", False))
    vm = z.get("vm")
    st = capi.sage_attn_quantized(*(z[n].data_ptr() for n in ("q8", "qs", "k8", "ks", "v8t", "vs")),
                                  vm.data_ptr() if vm is not None else None,
                                  out.data_ptr(), B, Hq, Hkv, N, d, _DTYPES[out.dtype], _LAYOUTS[tensor_layout],
                                  int(bool(is_causal)), float(sm_scale) if sm_scale is not None else 0.0,
                                  pv_mode(z.get("pv_dtype", "fp8"), pv_accum_dtype), ctypes.byref(o), _stream())
    _check(st, "sage_attn_quantized")
    return out


def sage_qk_int32(z: dict, tiles) -> torch.Tensor:
    """int32 Q8.K8^T of 128x128 tiles; tiles = list of (b, hq, q_tile, k_tile)."""
    t = torch.as_tensor(tiles, dtype=torch.int32).reshape(-1, 4).to(z["q8"].device).contiguous()
    out = torch.empty((t.shape[0], 128, 128), dtype=torch.int32, device=z["q8"].device)
    st = capi.sage_qk_int32(z["q8"].data_ptr(), z["k8"].data_ptr(), z["B"], z["Hq"], z["Hkv"], z["N"], z["d"],
                            t.data_ptr(), t.shape[0], out.data_ptr(), _stream())
    _check(st, "sage_qk_int32")
    return out


def sage_check_status() -> None:
    _check(capi.sage_check_status(_stream()), "sage_check_status")


def sage_device_supported() -> bool:
    return bool(capi.sage_device_supported())


# ---------------------------------------------------------------------------------------------
# The entry-point names of the SageAttention README ("How to Use": sageattn(q, k, v,
# tensor_layout="HND", is_causal=False); "Available APIs": the INT8-QK kernels with FP8 or FP16
# P.V and the varlen one), mapped onto the calls above.
# ---------------------------------------------------------------------------------------------
def sageattn(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None, **kw):
    """sage_attn under the README's name (FP8 P.V with fp32 accumulation unless told otherwise)."""
    return sage_attn(q, k, v, tensor_layout, is_causal, sm_scale, **kw)


def sageattn_qk_int8_pv_fp8_cuda(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None,
                                 pv_accum_dtype="fp32", qk_quant_gran="per_block", smooth_v=False, out=None):
    """INT8 Q.K^T and FP8 (E4M3) P.V; pv_accum_dtype "fp32" or "fp16+fp32" / "fp32+fp16"."""
    return sage_attn(q, k, v, tensor_layout, is_causal, sm_scale, pv_accum_dtype, out=out, pv_dtype="fp8",
                     qk_quant_gran=qk_quant_gran, smooth_v=smooth_v)


def sageattn_qk_int8_pv_fp16_cuda(q, k, v, tensor_layout="HND", is_causal=False, sm_scale=None,
                                  pv_accum_dtype="fp32", qk_quant_gran="per_block", smooth_v=False, out=None):
    """INT8 Q.K^T and FP16 P.V; pv_accum_dtype "fp32", "fp16+fp32" or "fp16" (see pv_mode)."""
    return sage_attn(q, k, v, tensor_layout, is_causal, sm_scale, pv_accum_dtype, out=out, pv_dtype="fp16",
                     qk_quant_gran=qk_quant_gran, smooth_v=smooth_v)


def sageattn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, is_causal=False, sm_scale=None,
                    pv_dtype="fp16", **kw):
    """sage_attn_varlen under the README's name; FP16 P.V by default, as the README lists it."""
    return sage_attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, is_causal, sm_scale,
                            pv_dtype=pv_dtype, **kw)
