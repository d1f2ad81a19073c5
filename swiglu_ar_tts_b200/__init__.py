"""Python binding of libarops.so: per-token decode operators for B200 (sm_100a).

Thin ctypes wrappers with the names of the C entry points in ``include/arops.h``
(``arops_rmsnorm`` -> ``rmsnorm`` and so on).  They check that the tensors are
CUDA, contiguous and of one dtype, then pass ``data_ptr()`` values, sizes and
torch's current CUDA stream to the library.  Every step of every operator runs
in the library's CUDA kernels; there is no fallback of any kind.  If the shared
library has not been built, every call raises.

Build the library with ``python -m swiglu_ar_tts_b200.build``.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

__all__ = [
    "rmsnorm", "add_rmsnorm", "layernorm", "add_layernorm", "mrope_qk", "mrope_kv_append",
    "mrope_paged_append", "paged_attention", "shared_prefix_attention",
    "attention_workspace", "attention_prepare",
    "swiglu", "set_pdl",
    "set_streaming", "set_topk_cluster", "topk_sample", "topk_sample_workspace", "topk_sample_prepare",
    "device_errors", "launch_count",
    "lib", "lib_path", "ArOpsError", "DTYPES",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libarops.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA = 0, 1, 2, 3
DTYPES = {torch.float32: 0, torch.bfloat16: 1}

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32


class _PagedCache(ctypes.Structure):
    """arops_paged_cache"""
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("num_pages", _i64), ("page_size", _i32),
                ("n_kv_heads", _i32), ("head_dim", _i32), ("dtype", ctypes.c_int)]


class _PagedBatch(ctypes.Structure):
    """arops_paged_batch"""
    _fields_ = [("q_start", _vp), ("kv_lens", _vp), ("block_table", _vp), ("n_seqs", _i32),
                ("max_pages", _i32)]


class _AttentionOptions(ctypes.Structure):
    """arops_attention_options"""
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", _i32),
                ("slopes", _vp), ("bidir_lens", _vp)]


class _PrefixGroups(ctypes.Structure):
    """arops_prefix_groups"""
    _fields_ = [("group_start", _vp), ("prefix_lens", _vp), ("prefix_table", _vp),
                ("n_groups", _i32), ("max_prefix_pages", _i32)]


# The same structures as bytes.  The tensor wrappers pass these: packing is a
# quarter of the cost of a Structure, and refuses a number that a field cannot
# hold where a Structure would cut it to the field's bits.
_pack_cache = struct.Struct("@PPqiiii").pack
_pack_batch = struct.Struct("@PPPii").pack
_pack_options = struct.Struct("@ffiPP").pack
_pack_groups = struct.Struct("@PPPii").pack
_pack_sections = struct.Struct("@iii").pack
_pack_sizes = struct.Struct("@qii").pack
_append_call = _attention_call = _shared_call = None  # set by lib()


class ArOpsError(RuntimeError):
    """A non-OK status from libarops; ``status`` holds the code."""

    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded libarops.so (loaded on first use; raises if it is missing)."""
    global _lib, _append_call, _attention_call, _shared_call
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with `python -m swiglu_ar_tts_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        L.arops_rmsnorm.argtypes = [_vp, _vp, _vp, _i64, _i64, ctypes.c_float, ctypes.c_int, _vp]
        L.arops_add_rmsnorm.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_float,
                                        ctypes.c_int, _vp]
        L.arops_mrope_qk.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                     ctypes.POINTER(_i32), ctypes.c_float, ctypes.c_int, _vp]
        L.arops_swiglu.argtypes = [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp]
        L.arops_mrope_kv_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32,
                                            _i32, _i32, _i64, _i64, ctypes.POINTER(_i32),
                                            ctypes.c_float, ctypes.c_int, _vp]
        L.arops_mrope_kv_append.restype = ctypes.c_int
        L.arops_layernorm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_float,
                                      ctypes.c_int, _vp]
        L.arops_add_layernorm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                          ctypes.c_float, ctypes.c_int, _vp]
        for fn in ("arops_rmsnorm", "arops_add_rmsnorm", "arops_mrope_qk", "arops_swiglu",
                   "arops_layernorm", "arops_add_layernorm"):
            getattr(L, fn).restype = ctypes.c_int
        L.arops_topk_sample_workspace.argtypes = [_i64, _i64, _i32, ctypes.POINTER(ctypes.c_size_t)]
        L.arops_topk_sample_workspace.restype = ctypes.c_int
        L.arops_topk_sample_prepare.argtypes = [_vp, ctypes.c_size_t, _vp]
        L.arops_topk_sample_prepare.restype = ctypes.c_int
        L.arops_topk_sample.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i32, ctypes.c_float,
                                        ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        L.arops_topk_sample.restype = ctypes.c_int
        cache, batch = ctypes.POINTER(_PagedCache), ctypes.POINTER(_PagedBatch)
        options, groups = ctypes.POINTER(_AttentionOptions), ctypes.POINTER(_PrefixGroups)
        L.arops_mrope_paged_append.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, cache,
                                               batch, _vp, _vp, ctypes.c_float, _vp, _i64, _i32,
                                               ctypes.POINTER(_i32), ctypes.c_float, _vp]
        L.arops_attention_workspace.argtypes = [_i64, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)]
        L.arops_paged_attention_workspace.argtypes = L.arops_attention_workspace.argtypes
        L.arops_attention_prepare.argtypes = [_vp, ctypes.c_size_t, _vp]
        L.arops_paged_attention.argtypes = [_vp, _i64, _vp, cache, batch, options, _i64, _i32, _vp,
                                            ctypes.c_size_t, _vp]
        L.arops_shared_prefix_attention.argtypes = [_vp, _i64, _vp, cache, batch, groups, options,
                                                    _i32, _vp, ctypes.c_size_t, _vp]
        for fn in ("arops_mrope_paged_append", "arops_attention_workspace",
                   "arops_paged_attention_workspace", "arops_attention_prepare",
                   "arops_paged_attention", "arops_shared_prefix_attention"):
            getattr(L, fn).restype = ctypes.c_int
        packed = {t: ctypes.c_char_p for t in (cache, batch, options, groups, ctypes.POINTER(_i32))}

        def with_bytes(name):
            fn = L[name]  # a function object of its own
            fn.argtypes = [packed.get(t, t) for t in getattr(L, name).argtypes]
            fn.restype = ctypes.c_int
            return fn

        _append_call = with_bytes("arops_mrope_paged_append")
        _attention_call = with_bytes("arops_paged_attention")
        _shared_call = with_bytes("arops_shared_prefix_attention")
        L.arops_set_pdl.argtypes = [ctypes.c_int]
        L.arops_set_pdl.restype = ctypes.c_int
        L.arops_set_streaming.argtypes = [ctypes.c_int]
        L.arops_set_streaming.restype = ctypes.c_int
        L.arops_set_topk_cluster.argtypes = [ctypes.c_int]
        L.arops_set_topk_cluster.restype = ctypes.c_int
        L.arops_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
        L.arops_device_errors.restype = ctypes.c_int
        L.arops_launch_count.restype = ctypes.c_uint64
        L.arops_status_string.argtypes = [ctypes.c_int]
        L.arops_status_string.restype = ctypes.c_char_p
        L.arops_last_error.restype = ctypes.c_char_p
        L.arops_version.restype = ctypes.c_int
        _lib = L
        return L


def _check(status: int) -> None:
    if status != OK:
        L = lib()
        raise ArOpsError(status, f"{L.arops_status_string(status).decode()}: "
                                 f"{L.arops_last_error().decode()}")


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dtype_code(*ts: torch.Tensor) -> int:
    dt = ts[0].dtype
    if dt not in DTYPES:
        raise TypeError(f"unsupported dtype {dt}; use torch.float32 or torch.bfloat16")
    for t in ts:
        if t.dtype != dt:
            raise TypeError(f"dtype mismatch: {t.dtype} vs {dt}")
    return DTYPES[dt]


def _check_tensors(named) -> None:
    """Every (name, tensor) is a contiguous CUDA tensor on the first one's device:
    the kernels receive raw pointers and run on that device."""
    dev = None
    for name, t in named:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """y = gamma * x / sqrt(mean(x^2, -1) + eps); ``out`` may be ``x``."""
    hidden = x.shape[-1]
    if out is None:
        out = torch.empty_like(x)
    _check_tensors((("x", x), ("gamma", gamma), ("out", out)))
    if gamma.shape != (hidden,) or out.shape != x.shape:
        raise ValueError("shape mismatch")
    code = _dtype_code(x, gamma, out)
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device):
        _check(lib().arops_rmsnorm(x.data_ptr(), gamma.data_ptr(), out.data_ptr(), rows, hidden,
                                   float(eps), code, _stream(x)))
    return out


def add_rmsnorm(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                y: torch.Tensor | None = None, residual_out: torch.Tensor | None = None):
    """residual_out = x + residual (rounded to the dtype); y = RMSNorm(residual_out).

    ``residual_out`` defaults to ``residual`` (updated in place); ``y`` defaults to
    a new tensor.  Returns ``(y, residual_out)``."""
    hidden = x.shape[-1]
    if y is None:
        y = torch.empty_like(x)
    if residual_out is None:
        residual_out = residual
    _check_tensors((("x", x), ("residual", residual), ("gamma", gamma), ("y", y),
                    ("residual_out", residual_out)))
    if (residual.shape != x.shape or y.shape != x.shape or residual_out.shape != x.shape
            or gamma.shape != (hidden,)):
        raise ValueError("shape mismatch")
    code = _dtype_code(x, residual, gamma, y, residual_out)
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device):
        _check(lib().arops_add_rmsnorm(x.data_ptr(), residual.data_ptr(), residual_out.data_ptr(),
                                       gamma.data_ptr(), y.data_ptr(), rows, hidden, float(eps),
                                       code, _stream(x)))
    return y, residual_out


def layernorm(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float = 1e-6,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """y = gamma * (x - mean) / sqrt(var + eps) + beta over the last dimension."""
    hidden = x.shape[-1]
    if out is None:
        out = torch.empty_like(x)
    _check_tensors((("x", x), ("gamma", gamma), ("beta", beta), ("out", out)))
    if gamma.shape != (hidden,) or beta.shape != (hidden,) or out.shape != x.shape:
        raise ValueError("shape mismatch")
    code = _dtype_code(x, gamma, beta, out)
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device):
        _check(lib().arops_layernorm(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                                     out.data_ptr(), rows, hidden, float(eps), code, _stream(x)))
    return out


def add_layernorm(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor,
                  beta: torch.Tensor, eps: float = 1e-6, y: torch.Tensor | None = None,
                  residual_out: torch.Tensor | None = None):
    """residual_out = x + residual (rounded); y = LayerNorm(residual_out).
    ``residual_out`` defaults to ``residual`` (in place).  Returns ``(y, residual_out)``."""
    hidden = x.shape[-1]
    if y is None:
        y = torch.empty_like(x)
    if residual_out is None:
        residual_out = residual
    _check_tensors((("x", x), ("residual", residual), ("gamma", gamma), ("beta", beta), ("y", y),
                    ("residual_out", residual_out)))
    if (residual.shape != x.shape or y.shape != x.shape or residual_out.shape != x.shape
            or gamma.shape != (hidden,) or beta.shape != (hidden,)):
        raise ValueError("shape mismatch")
    code = _dtype_code(x, residual, gamma, beta, y, residual_out)
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device):
        _check(lib().arops_add_layernorm(x.data_ptr(), residual.data_ptr(),
                                         residual_out.data_ptr(), gamma.data_ptr(),
                                         beta.data_ptr(), y.data_ptr(), rows, hidden, float(eps),
                                         code, _stream(x)))
    return y, residual_out


def mrope_qk(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor, sections=(24, 20, 20),
             theta: float = 1e6, q_out: torch.Tensor | None = None,
             k_out: torch.Tensor | None = None):
    """Multi-section rotary embedding of q [T, Hq, D] and k [T, Hk, D] with int32
    position ids pos [3, T] (rows t, h, w).  Outputs default to the inputs
    (rotation in place).  Returns ``(q_out, k_out)``."""
    if q_out is None:
        q_out = q
    if k_out is None:
        k_out = k
    _check_tensors((("q", q), ("k", k), ("pos", pos), ("q_out", q_out), ("k_out", k_out)))
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    tokens, hq, d = q.shape
    if k.shape[0] != tokens or k.shape[2] != d or q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("shape mismatch")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (3, tokens):
        raise ValueError("pos must be int32 [3, tokens]")
    code = _dtype_code(q, k, q_out, k_out)
    sec = (_i32 * 3)(*[int(s) for s in sections])
    with torch.cuda.device(q.device):
        _check(lib().arops_mrope_qk(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
                                    pos.data_ptr(), tokens, hq, k.shape[1], d, sec, float(theta),
                                    code, _stream(q)))
    return q_out, k_out


def mrope_kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                    cache_loc: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    sections=(24, 20, 20), theta: float = 1e6,
                    q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate q (into ``q_out``, default in place) and k with M-RoPE and write
    the rotated k and the unrotated v of token t into slot
    (cache_loc[0, t], cache_loc[1, t]) of k_cache / v_cache
    [cache_rows, n_kv_heads, max_seq, head_dim].  Returns ``q_out``."""
    if q_out is None:
        q_out = q
    _check_tensors((("q", q), ("k", k), ("v", v), ("pos", pos), ("cache_loc", cache_loc),
                    ("k_cache", k_cache), ("v_cache", v_cache), ("q_out", q_out)))
    tokens, hq, d = q.shape
    hk = k.shape[1]
    if (k.shape != (tokens, hk, d) or v.shape != k.shape or q_out.shape != q.shape
            or k_cache.dim() != 4 or k_cache.shape[1] != hk or k_cache.shape[3] != d
            or v_cache.shape != k_cache.shape):
        raise ValueError("shape mismatch")
    if pos.dtype != torch.int32 or tuple(pos.shape) != (3, tokens):
        raise ValueError("pos must be int32 [3, tokens]")
    if cache_loc.dtype != torch.int32 or tuple(cache_loc.shape) != (2, tokens):
        raise ValueError("cache_loc must be int32 [2, tokens]")
    code = _dtype_code(q, k, v, q_out, k_cache, v_cache)
    sec = (_i32 * 3)(*[int(s) for s in sections])
    with torch.cuda.device(q.device):
        _check(lib().arops_mrope_kv_append(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), pos.data_ptr(), cache_loc.data_ptr(), tokens, hq, hk, d,
            k_cache.shape[0], k_cache.shape[2], sec, float(theta), code, _stream(q)))
    return q_out


# The paged-cache calls are made a few times a layer with a dozen tensors each:
# their checks are one pass of cheap comparisons, and only a failed one looks
# for the words to say what is wrong.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


def _launch(device: int, fn, *args) -> None:
    """fn(*args, the device's current stream), with `device` current."""
    if torch.cuda.current_device() == device:
        status = fn(*args, _stream_of(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream_of(device))
    if status != OK:
        _check(status)


def _device_of(name: str, t: torch.Tensor) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _reject(name: str, t: torch.Tensor, device: int, dtype: torch.dtype, shape) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} is {list(t.shape)}, not {list(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _need(name: str, t: torch.Tensor, device: int, dtype: torch.dtype, shape) -> None:
    """A dense tensor of this device, type and shape (None: any)."""
    if (t.get_device() != device or t.dtype != dtype or not t.is_contiguous()
            or (shape is not None and t.shape != shape)):
        _reject(name, t, device, dtype, shape)


def _pack(pack, *values) -> bytes:
    try:
        return pack(*values)
    except (struct.error, OverflowError, TypeError) as e:
        raise ValueError(f"an argument is not of its type or range: {e}") from None


def _token_stride(name: str, t: torch.Tensor) -> int:
    """Elements between the tokens of a [tokens, heads, head_dim] tensor whose
    heads are dense (a slice of a packed projection is)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    if t.numel() == 0:
        return h * d
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name}'s heads must be dense (strides {t.stride()})")
    if n > 1 and st < h * d:
        raise ValueError(f"{name}'s tokens overlap (strides {t.stride()})")
    return st if n > 1 else h * d


def _pool(k_pages: torch.Tensor, v_pages: torch.Tensor, device: int, dtype: torch.dtype,
          head_dim: int) -> tuple[bytes, int]:
    """arops_paged_cache of the two pools, and their heads."""
    code = DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; use torch.float32 or torch.bfloat16")
    if k_pages.dim() != 4:
        raise ValueError("k_pages and v_pages must be [pages, n_kv_heads, page_size, head_dim]")
    n, hk, page, d = k_pages.shape
    if d != head_dim:
        raise ValueError(f"the pages hold heads of {d}, q heads of {head_dim}")
    _need("k_pages", k_pages, device, dtype, None)
    _need("v_pages", v_pages, device, dtype, k_pages.shape)
    return _pack(_pack_cache, k_pages.data_ptr(), v_pages.data_ptr(), n, page, hk, d, code), hk


def _table(name: str, t: torch.Tensor, device: int, rows: int) -> int:
    """Checks an int32 [rows, pages] table; returns its pages a row."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be int32 [{rows}, pages]")
    width = t.shape[1]
    _need(name, t, device, torch.int32, (rows, width))
    return width


def mrope_paged_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                       q_start: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                       k_pages: torch.Tensor, v_pages: torch.Tensor, sections=(24, 20, 20),
                       theta: float = 1e6, gamma_q: torch.Tensor | None = None,
                       gamma_k: torch.Tensor | None = None, eps: float = 1e-6,
                       q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Normalise (where a weight [D] is given) and rotate q [T, Hq, D] into
    ``q_out`` (default in place) and k [T, Hk, D] into its slot of the paged
    cache k_pages/v_pages [pages, Hk, page_size, D], and copy v into its slot.
    Sequence s owns tokens q_start[s]..q_start[s+1] and, after the call,
    kv_lens[s] cache positions in the pages block_table[s]; its tokens are the
    last of them.  q, k and v may be slices of one packed projection (dense
    heads, any token stride).  Returns ``q_out``."""
    device, dtype = _device_of("q", q), q.dtype
    sq, sk, sv = _token_stride("q", q), _token_stride("k", k), _token_stride("v", v)
    tokens, hq, d = q.shape
    if q_out is None:
        q_out, so = q, sq
    else:
        so = _token_stride("q_out", q_out)
        if q_out.get_device() != device or q_out.dtype != dtype or q_out.shape != q.shape:
            _reject("q_out", q_out, device, dtype, q.shape)
    cache, hk = _pool(k_pages, v_pages, device, dtype, d)
    shape = (tokens, hk, d)
    if k.get_device() != device or k.dtype != dtype or k.shape != shape:
        _reject("k", k, device, dtype, shape)
    if v.get_device() != device or v.dtype != dtype or v.shape != shape:
        _reject("v", v, device, dtype, shape)
    gq = gk = None
    if gamma_q is not None:
        _need("gamma_q", gamma_q, device, dtype, (d,))
        gq = gamma_q.data_ptr()
    if gamma_k is not None:
        _need("gamma_k", gamma_k, device, dtype, (d,))
        gk = gamma_k.data_ptr()
    n = kv_lens.numel()
    i32 = torch.int32
    _need("pos", pos, device, i32, (3, tokens))
    _need("q_start", q_start, device, i32, (n + 1,))
    _need("kv_lens", kv_lens, device, i32, (n,))
    pages = _table("block_table", block_table, device, n)
    batch = _pack(_pack_batch, q_start.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), n,
                  pages)
    lib()
    _launch(device, _append_call, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv,
            q_out.data_ptr(), so, cache, batch, gq, gk, eps, pos.data_ptr(), tokens, hq,
            _pack(_pack_sections, *sections), theta)
    return q_out


def attention_workspace(tokens: int, n_q_heads: int, head_dim: int,
                        shared_prefix: bool = True) -> int:
    """Bytes of device workspace that paged_attention and
    shared_prefix_attention need for this many query tokens; paged_attention
    alone (``shared_prefix=False``) needs fewer where there are many."""
    n = ctypes.c_size_t(0)
    _pack(_pack_sizes, tokens, n_q_heads, head_dim)  # ctypes would cut them to their bits
    fn = lib().arops_attention_workspace if shared_prefix else lib().arops_paged_attention_workspace
    _check(fn(tokens, n_q_heads, head_dim, ctypes.byref(n)))
    return int(n.value)


def attention_prepare(workspace: torch.Tensor) -> torch.Tensor:
    """Clears the arrival counters of a new attention workspace (a uint8 device
    tensor) on the current stream; needed once, before its first use."""
    _check_tensors((("workspace", workspace),))
    with torch.cuda.device(workspace.device):
        _check(lib().arops_attention_prepare(workspace.data_ptr(),
                                             workspace.numel() * workspace.element_size(),
                                             _stream(workspace)))
    return workspace


def _options(scale, softcap, window, slopes: int, bidir_lens: int) -> bytes:
    """arops_attention_options; a cap that is no longer one as a float is refused."""
    packed = _pack(_pack_options, scale, softcap, window, slopes, bidir_lens)
    if softcap != 0 and abs(softcap) < 2.0 ** -149:
        raise ValueError(f"softcap {softcap} is 0, which is no cap, as a float")
    return packed


def _attention_args(q, k_pages, v_pages, q_start, kv_lens, block_table, scale, softcap, window,
                    slopes, bidir_lens, workspace, out):
    """Checks and arguments that both attention operators share (q_start: None
    where every sequence has one token)."""
    device, dtype = _device_of("q", q), q.dtype
    stride = _token_stride("q", q)
    tokens, hq, d = q.shape
    cache, _ = _pool(k_pages, v_pages, device, dtype, d)
    if out is None:
        out = torch.empty(tokens, hq, d, dtype=dtype, device=q.device)
    else:
        _need("out", out, device, dtype, q.shape)
    n = kv_lens.numel()
    _need("kv_lens", kv_lens, device, torch.int32, (n,))
    pages = _table("block_table", block_table, device, n)
    starts = slope_ptr = bidir_ptr = 0
    if q_start is not None:
        _need("q_start", q_start, device, torch.int32, (n + 1,))
        starts = q_start.data_ptr()
    if slopes is not None:
        _need("slopes", slopes, device, torch.float32, (hq,))
        slope_ptr = slopes.data_ptr()
    if bidir_lens is not None:
        _need("bidir_lens", bidir_lens, device, torch.int32, (n,))
        bidir_ptr = bidir_lens.data_ptr()
    options = _options(d ** -0.5 if scale is None else scale, softcap, window, slope_ptr, bidir_ptr)
    batch = _pack(_pack_batch, starts, kv_lens.data_ptr(), block_table.data_ptr(), n, pages)
    if workspace is None:
        size = attention_workspace(tokens, hq, d, shared_prefix=q_start is None)
        workspace = attention_prepare(torch.empty(size, dtype=torch.uint8, device=q.device))
    elif workspace.get_device() != device or not workspace.is_contiguous():
        _reject("workspace", workspace, device, workspace.dtype, None)
    lib()
    return device, stride, cache, batch, options, workspace, out


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    q_start: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                    scale: float | None = None, softcap: float = 0.0, window: int = 0,
                    slopes: torch.Tensor | None = None, bidir_lens: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of q [T, Hq, D] (dense heads, any token stride) over the paged
    cache [pages, Hk, page_size, D]: sequence s owns tokens
    q_start[s]..q_start[s+1], the last of its kv_lens[s] positions, in the pages
    block_table[s].  Causal; the first bidir_lens[s] positions are seen by all
    of the sequence's queries; ``window`` > 0 hides keys that far back;
    ``softcap`` > 0 caps scores by a tanh; ``slopes`` [Hq] subtracts
    slope * distance.  ``scale`` defaults to D ** -0.5.  ``workspace`` is a
    uint8 tensor of attention_workspace() bytes (``shared_prefix=False`` is
    enough here), cleared once (attention_prepare); allocated and cleared here
    if omitted."""
    device, stride, cache, batch, options, workspace, out = _attention_args(
        q, k_pages, v_pages, q_start, kv_lens, block_table, scale, softcap, window, slopes,
        bidir_lens, workspace, out)
    tokens, hq, _ = q.shape
    _launch(device, _attention_call, q.data_ptr(), stride, out.data_ptr(), cache, batch, options,
            tokens, hq, workspace.data_ptr(), workspace.nbytes)
    return out


def shared_prefix_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                            group_start: torch.Tensor, prefix_lens: torch.Tensor,
                            prefix_table: torch.Tensor, kv_lens: torch.Tensor,
                            block_table: torch.Tensor, scale: float | None = None,
                            softcap: float = 0.0, window: int = 0,
                            slopes: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention of candidates that share a prompt: query s of q
    [n_seqs, Hq, D] sees the prefix_lens[g] positions of its group (sequences
    group_start[g]..group_start[g+1], pages prefix_table[g]) and then its own
    kv_lens[s] positions (pages block_table[s]), at whose end it stands.
    Options, workspace and ``out`` as for paged_attention."""
    device, stride, cache, batch, options, workspace, out = _attention_args(
        q, k_pages, v_pages, None, kv_lens, block_table, scale, softcap, window, slopes, None,
        workspace, out)
    if q.shape[0] != kv_lens.numel():
        raise ValueError("q must hold one token per sequence")
    n = prefix_lens.numel()
    _need("group_start", group_start, device, torch.int32, (n + 1,))
    _need("prefix_lens", prefix_lens, device, torch.int32, (n,))
    pages = _table("prefix_table", prefix_table, device, n)
    groups = _pack(_pack_groups, group_start.data_ptr(), prefix_lens.data_ptr(),
                   prefix_table.data_ptr(), n, pages)
    _launch(device, _shared_call, q.data_ptr(), stride, out.data_ptr(), cache, batch, groups,
            options, q.shape[1], workspace.data_ptr(), workspace.nbytes)
    return out


def swiglu(gate: torch.Tensor, up: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """out = silu(gate) * up (fp32 math); ``out`` may be ``gate`` or ``up``."""
    if out is None:
        out = torch.empty_like(gate)
    _check_tensors((("gate", gate), ("up", up), ("out", out)))
    if up.shape != gate.shape or out.shape != gate.shape:
        raise ValueError("shape mismatch")
    code = _dtype_code(gate, up, out)
    inter = gate.shape[-1] if gate.dim() else 1
    rows = gate.numel() // inter if inter else 0
    with torch.cuda.device(gate.device):
        _check(lib().arops_swiglu(gate.data_ptr(), up.data_ptr(), out.data_ptr(), rows, inter,
                                  code, _stream(gate)))
    return out


def topk_sample_workspace(rows: int, vocab: int, top_k: int) -> int:
    """Bytes of device workspace that topk_sample needs for this shape."""
    n = ctypes.c_size_t(0)
    _check(lib().arops_topk_sample_workspace(rows, vocab, top_k, ctypes.byref(n)))
    return int(n.value)


def topk_sample_prepare(workspace: torch.Tensor) -> torch.Tensor:
    """Clears the arrival counters of a new sampling workspace (a uint8 device
    tensor) on the current stream; needed once, before its first use."""
    _check_tensors((("workspace", workspace),))
    with torch.cuda.device(workspace.device):
        _check(lib().arops_topk_sample_prepare(workspace.data_ptr(),
                                               workspace.numel() * workspace.element_size(),
                                               _stream(workspace)))
    return workspace


def topk_sample(logits: torch.Tensor, gumbel: torch.Tensor, top_k: int, temperature: float = 1.0,
                workspace: torch.Tensor | None = None, token_out: torch.Tensor | None = None,
                prob_out: torch.Tensor | None = None):
    """Gumbel-max sample from softmax(logits / temperature) restricted to the
    top_k logits of each row.  logits [rows, vocab] (bf16/f32); gumbel
    [rows, top_k] float32 Gumbel(0,1) draws, draw j for the j-th largest logit.
    Returns (token int32 [rows], probability float32 [rows]).  ``workspace`` is
    a uint8 device tensor of at least topk_sample_workspace() bytes whose
    counters were cleared once (topk_sample_prepare); allocated and cleared
    here if omitted."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    if token_out is None:
        token_out = torch.empty(rows, dtype=torch.int32, device=logits.device)
    if prob_out is None:
        prob_out = torch.empty(rows, dtype=torch.float32, device=logits.device)
    need = topk_sample_workspace(rows, vocab, top_k) if rows else 0
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=logits.device)
        if rows:
            topk_sample_prepare(workspace)
    _check_tensors((("logits", logits), ("gumbel", gumbel), ("token_out", token_out),
                    ("prob_out", prob_out), ("workspace", workspace)))
    if gumbel.dtype != torch.float32 or tuple(gumbel.shape) != (rows, top_k):
        raise ValueError("gumbel must be float32 [rows, top_k]")
    if token_out.dtype != torch.int32 or prob_out.dtype != torch.float32:
        raise ValueError("token_out must be int32 and prob_out float32")
    code = _dtype_code(logits)
    with torch.cuda.device(logits.device):
        _check(lib().arops_topk_sample(logits.data_ptr(), gumbel.data_ptr(), token_out.data_ptr(),
                                       prob_out.data_ptr(), rows, vocab, int(top_k),
                                       float(temperature), code, workspace.data_ptr(),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(logits)))
    return token_out, prob_out


def set_pdl(enable: bool) -> bool:
    """Turn programmatic dependent launch on or off; returns the old setting."""
    return bool(lib().arops_set_pdl(1 if enable else 0))


def set_streaming(enable: bool) -> bool:
    """Choose the shared-memory streaming kernels or the register kernels (the
    default); returns the old setting.  Both give results within tolerance."""
    return bool(lib().arops_set_streaming(1 if enable else 0))


def set_topk_cluster(mode) -> int:
    """Which kernels top-k sampling may take: 0 (or False) the slice kernel
    only; 1 (or True, the default) the cluster kernels, registers for calls
    whose rows' 16-CTA clusters are all resident at once and shared memory for
    the rest; 2 the shared-memory cluster kernel for every call; 3 the
    streaming kernel (one CTA a row) for 16-byte-aligned rows.  Returns the
    old mode.  Every kernel gives identical results."""
    return int(lib().arops_set_topk_cluster(int(mode)))


def device_errors(clear: bool = True) -> int:
    """Device-side error bits (1: a bulk-copy wait timed out; 2: a KV-cache slot
    out of range was skipped; 4: a sampling workspace's counters were not
    cleared); synchronises the device."""
    v = ctypes.c_uint32(0)
    _check(lib().arops_device_errors(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


def launch_count() -> int:
    """Kernels launched by libarops in this process so far."""
    return int(lib().arops_launch_count())
