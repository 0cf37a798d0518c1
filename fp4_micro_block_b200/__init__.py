"""Python binding of ``libfp4q.so``, the sm_100a micro-block FP4 quantizer.

The entry points below carry the C names of ``include/fp4q.h`` and only
marshal arguments: torch tensors become device pointers, the current torch CUDA
stream becomes the ``stream`` argument, and a non-zero status raises
``Fp4qError``.  Every step of the computation runs in the library's kernels;
there is no CPU or PyTorch fallback.  The library is loaded on first use; if it
has not been built, that first call raises ImportError (build it with
``python -m fp4_micro_block_b200.build``).

Helpers at the bottom (``quantize_nvfp4`` ...) only allocate the output tensors
with torch and call the entry points.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FP4Q_LIBRARY selects another build of the library (a variant made with
# `python -m fp4_micro_block_b200.build --define ... --out ...`).
LIB_PATH = os.environ.get("FP4Q_LIBRARY") or os.path.join(_HERE, "libfp4q.so")

# enum values of include/fp4q.h
FP4Q_OK, FP4Q_ERR_INVALID_ARG, FP4Q_ERR_UNSUPPORTED, FP4Q_ERR_ALIGNMENT, FP4Q_ERR_CUDA, \
    FP4Q_ERR_DEVICE = range(6)
FP4Q_NVFP4, FP4Q_MXFP4, FP4Q_NVFP4_DUAL, FP4Q_INT4 = 0, 1, 2, 3
FP4Q_SCALES_LINEAR, FP4Q_SCALES_SWIZZLED = 0, 1
FP4Q_TSCALE_DYNAMIC, FP4Q_TSCALE_STATIC = 0, 1
FP4Q_FP8_ROW, FP4Q_FP8_TILE = 0, 1
FP4Q_WORKSPACE_BYTES = 16384

EXPORTED = [
    "fp4q_quantize_nvfp4", "fp4q_quantize_nvfp4_noalloc", "fp4q_quantize_mxfp4", "fp4q_hadamard_quantize", "fp4q_arc_quantize",
    "fp4q_dequantize", "fp4q_workspace_bytes", "fp4q_scales_bytes", "fp4q_status_string",
    "fp4q_device_error", "fp4q_selftest_div", "fp4q_gemm_nvfp4", "fp4q_hadamard_quantize_signed",
    "fp4q_dequantize_signed", "fp4q_quantize_fp8", "fp4q_gemm_fp8", "fp4q_kv_append_fp8", "fp4q_attention_fp8",
    "fp4q_attention_fp8_workspace_bytes",
]


class Fp4qError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def _load() -> C.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m fp4_micro_block_b200.build`")
    return declare(C.CDLL(LIB_PATH))


def declare(L: C.CDLL) -> C.CDLL:
    """Sets the argument and result types of the C entry points on a loaded library."""
    p, i64, f32, i32, sz = C.c_void_p, C.c_int64, C.c_float, C.c_int, C.c_size_t
    sigs = {
        "fp4q_quantize_nvfp4": (i32, [p, i64, i64, i64, p, p, p, i32, i32, p, sz, p]),
        "fp4q_quantize_nvfp4_noalloc": (i32, [p, i64, i64, i64, p, p, p, i32, p]),
        "fp4q_quantize_mxfp4": (i32, [p, i64, i64, i64, p, p, i32, p]),
        "fp4q_hadamard_quantize": (i32, [p, i64, i64, i64, i32, i32, p, p, p, i32, i32, p, sz, p]),
        "fp4q_arc_quantize": (i32, [p, i64, i64, i64, p, f32, p, p, i64, i32, p, p, p, i32, i32, p, sz, p]),
        "fp4q_dequantize": (i32, [i32, p, p, p, i64, i64, i32, i32, p, p]),
        "fp4q_workspace_bytes": (sz, [i64, i64]),
        "fp4q_scales_bytes": (i64, [i64, i64, i32]),
        "fp4q_status_string": (C.c_char_p, [i32]),
        "fp4q_device_error": (i32, []),
        "fp4q_selftest_div": (i32, [p, p, i64, p, p, p]),
        "fp4q_gemm_nvfp4": (i32, [p, p, p, p, p, p, i64, i64, i64, p, i32, p]),
        "fp4q_hadamard_quantize_signed": (i32, [p, i64, i64, i64, i32, p, i32, p, p, p, i32, i32, p, sz, p]),
        "fp4q_dequantize_signed": (i32, [i32, p, p, p, i64, i64, i32, i32, p, p, p]),
        "fp4q_quantize_fp8": (i32, [p, i64, i64, i64, i32, p, i64, p, i64, p, i64, p, i64, p]),
        "fp4q_gemm_fp8": (i32, [p, i64, p, i64, p, i64, p, i64, i32, i64, i64, i64, p, i64, i32, p]),
        "fp4q_kv_append_fp8": (i32, [p, i64, p, i64, i64, p, p, p, i64, i64, p]),
        "fp4q_attention_fp8": (i32, [p, i64, i64, i32, p, p, p, i64, i64, i64, i32, f32, p, i64, p, p, sz, p]),
        "fp4q_attention_fp8_workspace_bytes": (sz, [i64, i64, i64, i32, i32, i32]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


class Fp4qKvCache(C.Structure):
    """fp4q_kv_cache of the header."""

    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("num_pages", C.c_int64), ("num_kv_heads", C.c_int32), ("page_size", C.c_int32),
                ("head_dim", C.c_int32), ("block_table", C.c_void_p), ("table_stride", C.c_int64)]


class _Lazy:
    """Loads libfp4q.so on first attribute access."""

    _cdll = None

    def __getattr__(self, name):
        if _Lazy._cdll is None:
            _Lazy._cdll = _load()
        fn = getattr(_Lazy._cdll, name)
        self.__dict__[name] = fn  # later uses find it without this call
        return fn


_lib = _Lazy()


def lib():
    return _lib


def status_string(status: int) -> str:
    return _lib.fp4q_status_string(int(status)).decode()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("fp4q entry points take CUDA tensors")
    return t.data_ptr()


def _ws_bytes(workspace) -> int:
    """Bytes of a workspace (None: 0), which is written as one run from its pointer on."""
    if workspace is None:
        return 0
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str) -> int:
    if status != FP4Q_OK:
        raise Fp4qError(status, where)
    return status


def _ld(x: torch.Tensor) -> int:
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major view (unit column stride)")
    return x.stride(0)


# ----------------------------------------------------------------------------- C entry points

def fp4q_workspace_bytes(M: int = 0, K: int = 0) -> int:
    return int(_lib.fp4q_workspace_bytes(M, K))


def fp4q_scales_bytes(M: int, ncols: int, layout: int = FP4Q_SCALES_LINEAR) -> int:
    return int(_lib.fp4q_scales_bytes(M, ncols, layout))


def fp4q_quantize_nvfp4(x, codes, scales, tensor_scale, mode=FP4Q_TSCALE_DYNAMIC,
                        layout=FP4Q_SCALES_LINEAR, workspace=None, stream=None):
    M, K = x.shape
    ws_bytes = _ws_bytes(workspace)
    return _check(_lib.fp4q_quantize_nvfp4(_ptr(x), M, K, _ld(x), _ptr(codes), _ptr(scales),
                                           _ptr(tensor_scale), mode, layout, _ptr(workspace),
                                           ws_bytes, _stream(stream)), "fp4q_quantize_nvfp4")


def fp4q_quantize_nvfp4_noalloc(x, codes, scales, tensor_scale, layout=FP4Q_SCALES_LINEAR,
                                stream=None):
    M, K = x.shape
    return _check(_lib.fp4q_quantize_nvfp4_noalloc(_ptr(x), M, K, _ld(x), _ptr(codes), _ptr(scales),
                                                   _ptr(tensor_scale), layout, _stream(stream)),
                  "fp4q_quantize_nvfp4_noalloc")


def fp4q_quantize_mxfp4(x, codes, scales, layout=FP4Q_SCALES_LINEAR, stream=None):
    M, K = x.shape
    return _check(_lib.fp4q_quantize_mxfp4(_ptr(x), M, K, _ld(x), _ptr(codes), _ptr(scales),
                                           layout, _stream(stream)), "fp4q_quantize_mxfp4")


def fp4q_hadamard_quantize(x, had_size, fmt, codes, scales, scale_fp32,
                           mode=FP4Q_TSCALE_DYNAMIC, layout=FP4Q_SCALES_LINEAR,
                           workspace=None, stream=None):
    M, K = x.shape
    ws_bytes = _ws_bytes(workspace)
    return _check(_lib.fp4q_hadamard_quantize(_ptr(x), M, K, _ld(x), int(had_size), int(fmt),
                                              _ptr(codes), _ptr(scales), _ptr(scale_fp32), mode,
                                              layout, _ptr(workspace), ws_bytes, _stream(stream)),
                  "fp4q_hadamard_quantize")


def fp4q_arc_quantize(x, gamma, eps, perm, outliers, fmt, codes, scales, tensor_scale,
                      mode=FP4Q_TSCALE_DYNAMIC, layout=FP4Q_SCALES_LINEAR, workspace=None,
                      stream=None):
    M, K = x.shape
    S = 0 if outliers is None else outliers.numel()
    ws_bytes = _ws_bytes(workspace)
    return _check(_lib.fp4q_arc_quantize(_ptr(x), M, K, _ld(x), _ptr(gamma), float(eps), _ptr(perm),
                                         _ptr(outliers), S, int(fmt), _ptr(codes), _ptr(scales),
                                         _ptr(tensor_scale), mode, layout, _ptr(workspace),
                                         ws_bytes, _stream(stream)), "fp4q_arc_quantize")


def fp4q_dequantize(fmt, codes, scales, scale_fp32, M, K, y, layout=FP4Q_SCALES_LINEAR,
                    inv_had_size=0, stream=None):
    return _check(_lib.fp4q_dequantize(int(fmt), _ptr(codes), _ptr(scales), _ptr(scale_fp32), M, K,
                                       layout, int(inv_had_size), _ptr(y), _stream(stream)),
                  "fp4q_dequantize")


def fp4q_gemm_nvfp4(a_codes, a_scales, a_scale, b_codes, b_scales, b_scale, K, d, stream=None):
    """d [M, N] (float32 or bfloat16) = a_scale b_scale (A B^T) of two NVFP4
    tensors in the quantizers' output form (SWIZZLED scale buffers)."""
    M, N = d.shape
    if d.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("d must be float32 or bfloat16")
    return _check(_lib.fp4q_gemm_nvfp4(_ptr(a_codes), _ptr(a_scales), _ptr(a_scale), _ptr(b_codes),
                                       _ptr(b_scales), _ptr(b_scale), M, N, K, _ptr(d),
                                       int(d.dtype == torch.bfloat16), _stream(stream)),
                  "fp4q_gemm_nvfp4")


def _host_words(signs):
    """A host uint32 pattern (numpy array or sequence) as a ctypes pointer, kept alive by the caller."""
    import numpy as np
    arr = np.ascontiguousarray(np.asarray(signs, dtype=np.uint32))
    return arr, arr.ctypes.data


def fp4q_hadamard_quantize_signed(x, had_size, signs, fmt, codes, scales, scale_fp32,
                                  mode=FP4Q_TSCALE_DYNAMIC, layout=FP4Q_SCALES_LINEAR,
                                  workspace=None, stream=None):
    M, K = x.shape
    ws_bytes = _ws_bytes(workspace)
    keep, sp = _host_words(signs)
    return _check(_lib.fp4q_hadamard_quantize_signed(_ptr(x), M, K, _ld(x), int(had_size), sp, int(fmt),
                                                     _ptr(codes), _ptr(scales), _ptr(scale_fp32), mode,
                                                     layout, _ptr(workspace), ws_bytes, _stream(stream)),
                  "fp4q_hadamard_quantize_signed")


def fp4q_dequantize_signed(fmt, codes, scales, scale_fp32, M, K, y, signs, layout=FP4Q_SCALES_LINEAR,
                           inv_had_size=0, stream=None):
    keep, sp = _host_words(signs)
    return _check(_lib.fp4q_dequantize_signed(int(fmt), _ptr(codes), _ptr(scales), _ptr(scale_fp32), M, K,
                                              layout, int(inv_had_size), sp, _ptr(y), _stream(stream)),
                  "fp4q_dequantize_signed")


def fp4q_device_error() -> int:
    return int(_lib.fp4q_device_error())


def fp4q_selftest_div(x, d, q_fast, q_ieee, stream=None):
    return _check(_lib.fp4q_selftest_div(_ptr(x), _ptr(d), x.numel(), _ptr(q_fast), _ptr(q_ieee),
                                         _stream(stream)), "fp4q_selftest_div")


# ----------------------------------------------------------------------------- 8-bit entry points

# A call costs the host about as much as its kernel costs the GPU, so these keep
# to cheap tensor queries.

def _device(where, *tensors):
    """The CUDA device index that all of them (but None) are on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: tensors on {tensors[0].device} and {t.device}")
    if dev < 0:
        raise ValueError("fp4q entry points take CUDA tensors")
    return dev


def _launch(where, dev, fn, args, stream):
    """fn(*args, stream) with device `dev` current (the library launches on the current
    device, and the default stream is that device's current one)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != FP4Q_OK:
        raise Fp4qError(status, where)
    return status


def _want(t, name, dtypes, *shape):
    """A tensor argument's type and shape (None: any size) against what the call takes."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d).replace('torch.', '') for d in dtypes)}, not {t.dtype}")
    got = t.shape
    if got != shape and (len(got) != len(shape) or any(w is not None and w != n for w, n in zip(shape, got))):
        raise ValueError(f"{name} must have shape {tuple('any' if w is None else w for w in shape)}, not {tuple(got)}")


_CODES = (torch.uint8, torch.float8_e4m3fn)
_F32, _I32, _BF16 = (torch.float32,), (torch.int32,), (torch.bfloat16,)
_NO_SIZE = C.c_size_t(-1).value
_KV = struct.Struct("<5q3i4x2q")  # fp4q_kv_cache


def _row_stride(t, name, unit):
    """Row stride of a 2-D row-major view; for a single row, whose stride says nothing, the next multiple of `unit`."""
    ld, step = t.stride()
    rows, cols = t.shape
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must be a row-major view (unit column stride)")
    return ld if rows > 1 else -(-cols // unit) * unit


def _fp8_rows(n, block):
    return n if block == FP4Q_FP8_ROW else -(-n // 128)


def _fp8_side(codes, scales, rows, cols, block, what):
    """Codes [rows, cols] and scales [ceil(cols/128), rows or tile rows]: their strides."""
    n = rows if block == FP4Q_FP8_ROW else -(-rows // 128)
    kb = -(-cols // 128)
    if codes.dtype not in _CODES or scales.dtype is not torch.float32 or codes.shape != (rows, cols) or scales.shape != (kb, n):
        _want(codes, what, _CODES, rows, cols)
        _want(scales, what, _F32, kb, n)
    ld, step = codes.stride()
    lds, steps = scales.stride()
    if (step != 1 and cols > 1) or (steps != 1 and n > 1):
        raise ValueError(f"{what} must be row-major views (unit column stride)")
    # (a single row's stride says nothing)
    return ld if rows > 1 else -(-cols // 16) * 16, lds if kb > 1 else -(-n // 4) * 4


def fp4q_quantize_fp8(x, block, codes=None, scales=None, codes_t=None, scales_t=None, stream=None):
    """E4M3 codes and block-128 scales of bf16 x [M, K] and / or of its transpose."""
    _want(x, "x", _BF16, None, None)
    M, K = x.shape
    if (codes is None) != (scales is None) or (codes_t is None) != (scales_t is None):
        raise ValueError("fp4q_quantize_fp8: codes and scales go together")
    dev = _device("fp4q_quantize_fp8", x, codes, scales, codes_t, scales_t)
    c = s = ct = st = None
    ldc = lds = ldct = ldst = 0
    if codes is not None:
        ldc, lds = _fp8_side(codes, scales, M, K, block, "codes / scales")
        c, s = codes.data_ptr(), scales.data_ptr()
    if codes_t is not None:
        ldct, ldst = _fp8_side(codes_t, scales_t, K, M, block, "codes_t / scales_t")
        ct, st = codes_t.data_ptr(), scales_t.data_ptr()
    return _launch("fp4q_quantize_fp8", dev, _lib.fp4q_quantize_fp8,
                   (x.data_ptr(), M, K, _row_stride(x, "x", 8), block, c, ldc, s, lds, ct, ldct, st, ldst), stream)


def fp4q_gemm_fp8(a_codes, a_scales, b_codes, b_scales, b_block, d, stream=None):
    """d [M, N] (float32 or bfloat16) = A B^T of two fp4q_quantize_fp8 outputs (A: row blocks)."""
    bf16 = d.dtype is torch.bfloat16
    if not bf16 or len(d.shape) != 2:
        _want(d, "d", (torch.float32, torch.bfloat16), None, None)
    M, N = d.shape
    K = a_codes.shape[-1]
    dev = _device("fp4q_gemm_fp8", d, a_codes, a_scales, b_codes, b_scales)
    lda, ldas = _fp8_side(a_codes, a_scales, M, K, FP4Q_FP8_ROW, "A's codes / scales")
    ldb, ldbs = _fp8_side(b_codes, b_scales, N, K, b_block, "B's codes / scales")
    return _launch("fp4q_gemm_fp8", dev, _lib.fp4q_gemm_fp8,
                   (a_codes.data_ptr(), lda, a_scales.data_ptr(), ldas, b_codes.data_ptr(), ldb, b_scales.data_ptr(), ldbs,
                    b_block, M, N, K, d.data_ptr(), _row_stride(d, "d", 1), bf16), stream)


def _kv_cache(k_cache, v_cache, k_scale, v_scale, block_table):
    """The bytes of an fp4q_kv_cache, its head count, head dim and batch."""
    shape = k_cache.shape
    if (len(shape) != 4 or v_cache.shape != shape or k_scale.shape != shape[:2] or v_scale.shape != shape[:2] or
            len(block_table.shape) != 2 or k_cache.dtype not in _CODES or v_cache.dtype not in _CODES or
            k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32 or block_table.dtype is not torch.int32):
        _want(k_cache, "k_cache", _CODES, None, None, None, None)
        _want(v_cache, "v_cache", _CODES, *shape)
        _want(k_scale, "k_scale", _F32, *shape[:2])
        _want(v_scale, "v_scale", _F32, *shape[:2])
        _want(block_table, "block_table", _I32, None, None)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and
            v_scale.is_contiguous() and block_table.is_contiguous()):
        raise ValueError("the cache, its scales and the block table must be contiguous")
    pages, heads, page, dim = shape
    B, width = block_table.shape
    return _KV.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads, page,
                    dim, block_table.data_ptr(), width), heads, dim, B


def _ragged(cu, lens, B, name):
    if cu.dtype is not torch.int32 or lens.dtype is not torch.int32 or cu.shape != (B + 1,) or lens.shape != (B,):
        _want(cu, name, _I32, B + 1)
        _want(lens, "lens", _I32, B)
    if not (cu.is_contiguous() and lens.is_contiguous()):
        raise ValueError(f"{name} and lens must be contiguous")


def _tokens(t, name, T, heads, dim):
    """bf16 [T, heads, dim] whose heads and dims are contiguous: the stride between tokens."""
    if t.dtype is not torch.bfloat16 or t.shape != (T, heads, dim):
        _want(t, name, _BF16, T, heads, dim)
    st, sh, sd = t.stride()
    if (dim > 1 and sd != 1) or (heads > 1 and sh != dim):
        raise ValueError(f"{name}: heads and dims of a token must be contiguous")
    return st if T > 1 else heads * dim


def fp4q_kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_new, lens, max_new, stream=None):
    """Writes the new tokens k, v [tokens, Hkv, D] (bf16) at the end of their sequences."""
    dev = _device("fp4q_kv_append_fp8", k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_new, lens)
    cache, heads, dim, B = _kv_cache(k_cache, v_cache, k_scale, v_scale, block_table)
    T = k.shape[0]
    ldk, ldv = _tokens(k, "k", T, heads, dim), _tokens(v, "v", T, heads, dim)
    _ragged(cu_new, lens, B, "cu_new")
    return _launch("fp4q_kv_append_fp8", dev, _lib.fp4q_kv_append_fp8,
                   (k.data_ptr(), ldk, v.data_ptr(), ldv, T, cache, cu_new.data_ptr(), lens.data_ptr(), B, int(max_new)), stream)


def fp4q_attention_fp8_workspace_bytes(batch, max_q, max_len, num_q_heads, num_kv_heads, head_dim):
    n = _lib.fp4q_attention_fp8_workspace_bytes(int(batch), int(max_q), int(max_len), num_q_heads, num_kv_heads, head_dim)
    if n == _NO_SIZE:
        raise Fp4qError(FP4Q_ERR_INVALID_ARG, "fp4q_attention_fp8_workspace_bytes")
    return n


def fp4q_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, lens, max_q, max_len, o, lse=None,
                       causal=True, softmax_scale=None, workspace=None, stream=None):
    """o [tokens, Hq, D] (bf16) = attention of q [tokens, Hq, D] (bf16) over the cache."""
    ws_bytes = _ws_bytes(workspace)
    dev = _device("fp4q_attention_fp8", q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, lens, o, lse, workspace)
    cache, _, dim, B = _kv_cache(k_cache, v_cache, k_scale, v_scale, block_table)
    T, Hq, _ = q.shape
    ldq, ldo = _tokens(q, "q", T, Hq, dim), _tokens(o, "o", T, Hq, dim)
    _ragged(cu_q, lens, B, "cu_q")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()):
        _want(lse, "lse", _F32, T, Hq)
        raise ValueError("lse must be contiguous")
    scale = dim ** -0.5 if softmax_scale is None else float(softmax_scale)
    return _launch("fp4q_attention_fp8", dev, _lib.fp4q_attention_fp8,
                   (q.data_ptr(), ldq, T, Hq, cache, cu_q.data_ptr(), lens.data_ptr(), B, int(max_q), int(max_len), bool(causal),
                    scale, o.data_ptr(), ldo, None if lse is None else lse.data_ptr(),
                    None if workspace is None else workspace.data_ptr(), ws_bytes), stream)


# ----------------------------------------------------------------------------- allocating helpers

def _block(fmt: int) -> int:
    return 32 if fmt == FP4Q_MXFP4 else 16


def alloc_outputs(M: int, K: int, fmt: int, layout: int = FP4Q_SCALES_LINEAR, device="cuda",
                  ncols: int | None = None):
    """codes [M, K/2] u8, scales (linear [M, ncols] or the padded tiled buffer),
    and the fp32 scale(s): 1 float (NVFP4, INT4), [M, K/128] (dual) or None (MXFP4)."""
    ncols = K // _block(fmt) if ncols is None else ncols
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=device)
    if layout == FP4Q_SCALES_LINEAR:
        scales = torch.empty((M, ncols), dtype=torch.uint8, device=device)
    else:
        scales = torch.empty(fp4q_scales_bytes(M, ncols, layout), dtype=torch.uint8, device=device)
    if fmt in (FP4Q_NVFP4, FP4Q_INT4):
        sf = torch.zeros(1, dtype=torch.float32, device=device)
    elif fmt == FP4Q_NVFP4_DUAL:
        sf = torch.empty((M, K // 128), dtype=torch.float32, device=device)
    else:
        sf = None
    return codes, scales, sf


def workspace(device="cuda") -> torch.Tensor:
    return torch.empty(FP4Q_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def quantize_nvfp4(x, tensor_scale=None, layout=FP4Q_SCALES_LINEAR, ws=None):
    """NVFP4 of bf16 x; dynamic tensor scale unless `tensor_scale` (1-float tensor) is given."""
    M, K = x.shape
    codes, scales, sf = alloc_outputs(M, K, FP4Q_NVFP4, layout, x.device)
    mode = FP4Q_TSCALE_DYNAMIC
    if tensor_scale is not None:
        sf.copy_(tensor_scale.reshape(1))
        mode = FP4Q_TSCALE_STATIC
    ws = workspace(x.device) if (ws is None and mode == FP4Q_TSCALE_DYNAMIC) else ws
    fp4q_quantize_nvfp4(x, codes, scales, sf, mode, layout, ws)
    return codes, scales, sf


def quantize_mxfp4(x, layout=FP4Q_SCALES_LINEAR):
    M, K = x.shape
    codes, scales, _ = alloc_outputs(M, K, FP4Q_MXFP4, layout, x.device)
    fp4q_quantize_mxfp4(x, codes, scales, layout)
    return codes, scales


def hadamard_quantize(x, had_size, fmt=FP4Q_NVFP4, tensor_scale=None, layout=FP4Q_SCALES_LINEAR,
                      ws=None, signs=None):
    """Block Hadamard (with `signs`: the random-sign rotation) + quantization."""
    M, K = x.shape
    codes, scales, sf = alloc_outputs(M, K, fmt, layout, x.device)
    mode = FP4Q_TSCALE_DYNAMIC
    if fmt == FP4Q_NVFP4 and tensor_scale is not None:
        sf.copy_(tensor_scale.reshape(1))
        mode = FP4Q_TSCALE_STATIC
    if fmt == FP4Q_NVFP4 and mode == FP4Q_TSCALE_DYNAMIC and ws is None:
        ws = workspace(x.device)
    if signs is None:
        fp4q_hadamard_quantize(x, had_size, fmt, codes, scales, sf, mode, layout, ws)
    else:
        fp4q_hadamard_quantize_signed(x, had_size, signs, fmt, codes, scales, sf, mode, layout, ws)
    return codes, scales, sf


def arc_quantize(x, gamma, perm, outliers, eps=1e-6, tensor_scale=None,
                 layout=FP4Q_SCALES_LINEAR, ws=None, fmt=FP4Q_NVFP4):
    """ARCQuant path; returns (codes, scales, tensor scale (NVFP4, INT4) or None (MXFP4))."""
    M, K = x.shape
    S = 0 if outliers is None else outliers.numel()
    codes, scales, sf = alloc_outputs(M, K + S, fmt, layout, x.device)
    mode = FP4Q_TSCALE_DYNAMIC
    if fmt in (FP4Q_NVFP4, FP4Q_INT4):
        if tensor_scale is not None:
            sf.copy_(tensor_scale.reshape(1))
            mode = FP4Q_TSCALE_STATIC
        ws = workspace(x.device) if (ws is None and mode == FP4Q_TSCALE_DYNAMIC) else ws
    fp4q_arc_quantize(x, gamma, eps, perm, outliers, fmt, codes, scales, sf, mode, layout, ws)
    return codes, scales, sf


def dequantize(fmt, codes, scales, scale_fp32, K, layout=FP4Q_SCALES_LINEAR, inv_had_size=0, signs=None):
    M = codes.shape[0]
    y = torch.empty((M, K), dtype=torch.bfloat16, device=codes.device)
    if signs is None:
        fp4q_dequantize(fmt, codes, scales, scale_fp32, M, K, y, layout, inv_had_size)
    else:
        fp4q_dequantize_signed(fmt, codes, scales, scale_fp32, M, K, y, signs, layout, inv_had_size)
    return y


def gemm_nvfp4(a_codes, a_scales, a_scale, b_codes, b_scales, b_scale, K, out_dtype=torch.float32):
    """Allocates D [M, N] and calls fp4q_gemm_nvfp4."""
    d = torch.empty((a_codes.shape[0], b_codes.shape[0]), dtype=out_dtype, device=a_codes.device)
    fp4q_gemm_nvfp4(a_codes, a_scales, a_scale, b_codes, b_scales, b_scale, K, d)
    return d


def alloc_fp8(rows, cols, block=FP4Q_FP8_ROW, device="cuda"):
    """codes [rows, cols] u8 and scales [ceil(cols/128), rows or ceil(rows/128)] f32, as views of
    buffers whose rows are 16-byte aligned."""
    n = _fp8_rows(rows, block)
    codes = torch.empty_strided((rows, cols), (-(-cols // 16) * 16, 1), dtype=torch.uint8, device=device)
    scales = torch.empty_strided((-(-cols // 128), n), (-(-n // 4) * 4, 1), dtype=torch.float32, device=device)
    return codes, scales


def quantize_fp8(x, block=FP4Q_FP8_ROW, transpose=False):
    """(codes, scales) of bf16 x [M, K]; with transpose=True also those of its transpose:
    (codes, scales, codes_t, scales_t), all from one read of x."""
    M, K = x.shape
    out = alloc_fp8(M, K, block, x.device) + (alloc_fp8(K, M, block, x.device) if transpose else ())
    fp4q_quantize_fp8(x, block, *out)
    return out


def gemm_fp8(a_codes, a_scales, b_codes, b_scales, b_block=FP4Q_FP8_TILE, out_dtype=torch.bfloat16):
    """Allocates D [M, N] and calls fp4q_gemm_fp8."""
    d = torch.empty((a_codes.shape[0], b_codes.shape[0]), dtype=out_dtype, device=a_codes.device)
    fp4q_gemm_fp8(a_codes, a_scales, b_codes, b_scales, b_block, d)
    return d


def alloc_kv_cache(num_pages, num_kv_heads, page_size, head_dim, device="cuda"):
    """k_cache, v_cache (u8 [num_pages, Hkv, page_size, D]) and k_scale, v_scale (f32 [num_pages, Hkv])."""
    codes = [torch.zeros((num_pages, num_kv_heads, page_size, head_dim), dtype=torch.uint8, device=device)
             for _ in range(2)]
    scales = [torch.zeros((num_pages, num_kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    return (*codes, *scales)


def kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_new, lens, max_new):
    """fp4q_kv_append_fp8; returns the cache tensors, updated in place."""
    fp4q_kv_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_new, lens, max_new)
    return k_cache, v_cache, k_scale, v_scale


def attention_fp8_workspace(q, k_cache, batch, max_q, max_len):
    """Scratch for attention_fp8 calls of these sizes (None: none is needed)."""
    sizes = (batch, max_q, max_len, q.shape[1], k_cache.shape[1], k_cache.shape[3])
    if torch._C._cuda_getDevice() == q.get_device():
        n = fp4q_attention_fp8_workspace_bytes(*sizes)
    else:
        with torch.cuda.device(q.device):
            n = fp4q_attention_fp8_workspace_bytes(*sizes)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, lens, max_q, max_len, causal=True,
                  softmax_scale=None, ws=None):
    """(o [tokens, Hq, D] bf16, lse [tokens, Hq] f32); tokens that belong to no sequence are left unset."""
    o = torch.empty_like(q, memory_format=torch.contiguous_format)  # (1.4 us of the host; torch.empty 2.4)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if ws is None:
        ws = attention_fp8_workspace(q, k_cache, block_table.shape[0], max_q, max_len)
    fp4q_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, lens, max_q, max_len, o, lse, causal,
                       softmax_scale, ws)
    return o, lse
