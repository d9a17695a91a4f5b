"""BitDelta on GB300: Python binding of the C-ABI library ``libbitdelta.so``.

The method (web page "BitDelta: serving 14 Zen models from one GPU cluster",
sections "The mathematical foundation" and "Serving architecture"):
compress a fine-tuned matrix to one f32 scale alpha = mean|W_ft - W_base| and
one sign bit per weight, and serve many variants from one resident base with a
fused linear y = x (W_base + alpha_v sign(delta_v))^T that never writes the
reconstructed weights to memory.

This module only marshals arguments: every step runs in the library's CUDA
kernels.  The first use loads the library and raises ImportError if it is
missing (build it with ``python -m bit_delta_compressed_gb300.build``); there
is no CPU fallback.

Two layers:
* ``lib`` and the functions named like the C entry points
  (``bitdelta_compress``, ``bitdelta_linear``, ...) take raw integers
  (device pointers, sizes, a stream handle) exactly as the C ABI does;
* ``compress``, ``compress_rows`` and ``linear`` take torch CUDA tensors,
  allocate outputs and workspace with torch, and call the C ABI on the
  current torch stream.
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libbitdelta.so"

BD_OK, BD_ERR_NULL, BD_ERR_ALIGN, BD_ERR_SHAPE, BD_ERR_DTYPE, BD_ERR_VARIANT, \
    BD_ERR_WORKSPACE, BD_ERR_CUDA, BD_ERR_TIMEOUT, BD_ERR_UNSUPPORTED, BD_ERR_SLOT = range(11)
BD_F32, BD_BF16 = 0, 1
BD_PATH_AUTO, BD_PATH_SIMT, BD_PATH_DECODE_TC, BD_PATH_PREFILL_TC, BD_PATH_DECODE_FOLD, BD_PATH_DECODE_WEFF = range(6)
MAX_VARIANTS = 64
PATHS = {"auto": BD_PATH_AUTO, "simt": BD_PATH_SIMT, "decode_tc": BD_PATH_DECODE_TC,
         "prefill_tc": BD_PATH_PREFILL_TC, "decode_fold": BD_PATH_DECODE_FOLD,
         "decode_weff": BD_PATH_DECODE_WEFF}

# name -> (restype, argtypes), in the order of include/bitdelta.h
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_ST = ctypes.c_int
_F32 = ctypes.c_float


class KVCacheDesc(ctypes.Structure):
    """``bd_kv_cache``: one layer's key/value cache as the C ABI takes it."""
    _fields_ = [("k", _P), ("v", _P), ("slots", _I64), ("capacity", _I64), ("kv_heads", _I32), ("head_dim", _I32),
                ("stride_slot", _I64), ("stride_token", _I64), ("stride_head", _I64)]


class KVCache4Desc(ctypes.Structure):
    """``bd_kv_cache4``: one layer's 4-bit cache as the C ABI takes it."""
    _fields_ = [("data", _P), ("slots", _I64), ("capacity", _I64), ("kv_heads", _I32), ("head_dim", _I32),
                ("stride_slot", _I64), ("stride_head", _I64)]


SIGNATURES = {
    "bitdelta_compress_workspace": (_SZ, [_I64, _I64]),
    "bitdelta_compress": (_ST, [_P, _P, _ST, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "bitdelta_compress_rows": (_ST, [_P, _P, _ST, _I64, _I64, _P, _P, _P]),
    "bitdelta_compress_noalloc": (_ST, [_P, _P, _ST, _I64, _I64, _P, _P, _P]),
    "bitdelta_reconstruct": (_ST, [_P, _P, _I32, _P, _I64, _I64, _P, _P]),
    "bitdelta_linear_workspace": (_SZ, [_I64, _I64, _I64, _I32]),
    "bitdelta_linear": (_ST, [_P, _P, _I64, _I64, _I64, _P, _P, _P, _I32, _P, _ST, _P, _SZ, _P]),
    "bitdelta_linear_ex": (_ST, [_P, _P, _I64, _I64, _I64, _P, _P, _P, _I32, _P, _ST, _P, _SZ,
                                 _P, _ST]),
    "bitdelta_group": (_ST, [_P, _I64, _I32, _P, _SZ, _P]),
    "bitdelta_linear_grouped": (_ST, [_P, _I64, _I64, _I64, _P, _P, _P, _I32, _P, _ST, _P, _SZ,
                                      _P, _ST]),
    "bitdelta_linear_rows": (_ST, [_P, _P, _I64, _I64, _I64, _P, _P, _P, _I32, _P, _ST, _P, _SZ,
                                   _P, _ST]),
    "bitdelta_attn_workspace": (_SZ, [_I64, _I64, _I32, _I32, _I32, _I64]),
    "bitdelta_attn_decode": (_ST, [_P, _I64, _I64, _I32, _P, _P, _P, _I32, _I32, _F32, _P, _P, _P, _SZ, _P]),
    "bitdelta_attn_decode_prefix": (_ST, [_P, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _F32,
                                          _P, _P, _P, _SZ, _P]),
    "bitdelta_attn_prefill": (_ST, [_P, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32,
                                    _F32, _P, _P, _SZ, _P]),
    "bitdelta_evict_workspace": (_SZ, [_I64, _I32, _I64]),
    "bitdelta_cache_evict": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "bitdelta_cache4_bytes": (_SZ, [_I64, _I64, _I32, _I32]),
    "bitdelta_cache4_write": (_ST, [_P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "bitdelta_cache4_read": (_ST, [_P, _I64, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "bitdelta_attn4_workspace": (_SZ, [_I64, _I64, _I32, _I32, _I32, _I64]),
    "bitdelta_attn4_decode": (_ST, [_P, _I64, _I64, _I32, _P, _P, _P, _I32, _I32, _F32, _P, _P, _SZ, _P]),
    "bitdelta_attn4_prefill": (_ST, [_P, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _I64, _I32, _I32, _F32, _P, _P, _SZ, _P]),
    "bitdelta_device_status": (_ST, [_P, _P]),
    "bitdelta_check_bounded_wait": (_ST, [_P, ctypes.c_uint32, ctypes.c_int, _P]),
    "bitdelta_launch_count": (ctypes.c_uint64, []),
    "bitdelta_status_string": (ctypes.c_char_p, [_ST]),
    "bitdelta_abi_version": (ctypes.c_int, []),
}


class BitDeltaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (status %d)" % (where, status_string(code), code))


_LIB = None


def get_lib() -> ctypes.CDLL:
    """The loaded library; raises ImportError if it has not been built."""
    global _LIB
    if _LIB is None:
        if not LIB_PATH.exists():
            raise ImportError("libbitdelta.so is not built (%s); run "
                              "`python -m bit_delta_compressed_gb300.build`" % LIB_PATH)
        lib = ctypes.CDLL(str(LIB_PATH))
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def __getattr__(name):
    # `lib` and the raw C entry points resolve on first use, so the build
    # submodule can be imported before the library exists.
    if name == "lib":
        return get_lib()
    if name in SIGNATURES:
        return getattr(get_lib(), name)
    raise AttributeError(name)


def status_string(code: int) -> str:
    return get_lib().bitdelta_status_string(int(code)).decode()


def check(code: int, where: str) -> None:
    if code != BD_OK:
        raise BitDeltaError(code, where)


# -- torch layer ---------------------------------------------------------------

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(stream=None) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    torch = _torch()
    try:                                          # 0.1 us; the Stream object takes 3
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return int(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t == torch.float32:
        return BD_F32
    if t == torch.bfloat16:
        return BD_BF16
    raise TypeError("unsupported dtype %s" % t)


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def _workspace(ws, device: int):
    """A workspace's address and bytes; `device` is the index of the other tensors'."""
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the CUDA device of the other tensors")
    return ws.data_ptr(), ws.numel()


def compress_workspace(N: int, K: int, device=None):
    torch = _torch()
    n = int(get_lib().bitdelta_compress_workspace(N, K))
    if n == 0:
        raise BitDeltaError(BD_ERR_SHAPE, "bitdelta_compress_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def compress(w_ft, w_base, workspace=None, alpha_out=None, bits_out=None, stream=None):
    """(alpha [1] f32, bits int32 [N, K/32]) for one fine-tuned matrix."""
    torch = _torch()
    _need_cuda(w_ft, w_base)
    if w_ft.shape != w_base.shape or w_ft.dtype != w_base.dtype or w_ft.dim() != 2:
        raise ValueError("w_ft and w_base must be 2-D of one shape and dtype")
    N, K = w_ft.shape
    dev = w_ft.device
    ws = compress_workspace(N, K, dev) if workspace is None else workspace
    alpha = torch.empty(1, dtype=torch.float32, device=dev) if alpha_out is None else alpha_out
    bits = torch.empty((N, K // 32), dtype=torch.int32, device=dev) if bits_out is None else bits_out
    check(get_lib().bitdelta_compress(w_ft.data_ptr(), w_base.data_ptr(), _dtype_code(w_ft.dtype), N, K,
                                alpha.data_ptr(), bits.data_ptr(), *_workspace(ws, w_ft.get_device()),
                                _stream(stream)), "bitdelta_compress")
    return alpha, bits


def compress_rows(w_ft, w_base, stream=None):
    """(alpha [N] f32, bits int32 [N, K/32]) with one scale per output row."""
    torch = _torch()
    _need_cuda(w_ft, w_base)
    N, K = w_ft.shape
    alpha = torch.empty(N, dtype=torch.float32, device=w_ft.device)
    bits = torch.empty((N, K // 32), dtype=torch.int32, device=w_ft.device)
    check(get_lib().bitdelta_compress_rows(w_ft.data_ptr(), w_base.data_ptr(), _dtype_code(w_ft.dtype),
                                     N, K, alpha.data_ptr(), bits.data_ptr(), _stream(stream)),
          "bitdelta_compress_rows")
    return alpha, bits


def reconstruct(w_base, alpha, bits, out=None, stream=None):
    """bf16 W_eff [N, K] = nearest bf16 of W_base + alpha * s (``alpha``: a
    float32 tensor of 1 or N values; see ``bitdelta_reconstruct``)."""
    torch = _torch()
    _need_cuda(w_base, alpha, bits)
    N, K = w_base.shape
    if alpha.dtype != torch.float32 or alpha.numel() not in (1, N) or not alpha.is_contiguous():
        raise ValueError("alpha must be a contiguous float32 tensor of 1 or N values")
    per_row = 1 if (alpha.numel() == N and N != 1) else 0
    out = torch.empty((N, K), dtype=torch.bfloat16, device=w_base.device) if out is None else out
    check(get_lib().bitdelta_reconstruct(w_base.data_ptr(), alpha.data_ptr(), per_row, bits.data_ptr(), N, K,
                                         out.data_ptr(), _stream(stream)), "bitdelta_reconstruct")
    return out


def linear_workspace(M: int, N: int, K: int, V: int, device=None):
    torch = _torch()
    n = int(get_lib().bitdelta_linear_workspace(M, N, K, V))
    if n == 0:
        raise BitDeltaError(BD_ERR_SHAPE, "bitdelta_linear_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def bits_pointer_array(bits_list):
    """HOST array of the variants' device pointers, as the C ABI takes it."""
    arr = (ctypes.c_void_p * max(1, len(bits_list)))(*[b.data_ptr() for b in bits_list])
    return arr


def linear(x, variant_ids, w_base, alphas, bits_list, out_dtype=None, workspace=None,
           out=None, path: str = "auto", stream=None, bits_ptrs=None):
    """y [M, N] = per-token fused BitDelta linear (see ``bitdelta_linear``)."""
    torch = _torch()
    _need_cuda(x, variant_ids, w_base)
    M, K = x.shape
    N = w_base.shape[0]
    V = len(bits_list)
    if V > MAX_VARIANTS:
        raise ValueError("at most %d variants" % MAX_VARIANTS)
    out_dtype = out_dtype or torch.float32
    y = torch.empty((M, N), dtype=out_dtype, device=x.device) if out is None else out
    ws = linear_workspace(M, N, K, V, x.device) if workspace is None else workspace
    ptrs = bits_pointer_array(bits_list) if bits_ptrs is None else bits_ptrs
    al = alphas.data_ptr() if V > 0 else None
    check(get_lib().bitdelta_linear_ex(x.data_ptr(), variant_ids.data_ptr(), M, N, K, w_base.data_ptr(),
                                 al, ctypes.cast(ptrs, ctypes.c_void_p), V, y.data_ptr(),
                                 _dtype_code(out_dtype), *_workspace(ws, x.get_device()),
                                 _stream(stream), PATHS[path]), "bitdelta_linear")
    return y


def linear_rows(x, variant_ids, w_base, alpha_rows, bits_list, out_dtype=None, workspace=None,
                out=None, path: str = "auto", stream=None, bits_ptrs=None):
    """y [M, N] with one scale per (variant, output row): ``alpha_rows`` is a
    float32 [V, N] device tensor (see ``bitdelta_linear_rows``)."""
    torch = _torch()
    _need_cuda(x, variant_ids, w_base)
    M, K = x.shape
    N = w_base.shape[0]
    V = len(bits_list)
    if V > MAX_VARIANTS:
        raise ValueError("at most %d variants" % MAX_VARIANTS)
    if V > 0 and (alpha_rows.dtype != torch.float32 or alpha_rows.numel() != V * N
                  or not alpha_rows.is_contiguous()):
        raise ValueError("alpha_rows must be a contiguous float32 [V, N] tensor")
    out_dtype = out_dtype or torch.float32
    y = torch.empty((M, N), dtype=out_dtype, device=x.device) if out is None else out
    ws = linear_workspace(M, N, K, V, x.device) if workspace is None else workspace
    ptrs = bits_pointer_array(bits_list) if bits_ptrs is None else bits_ptrs
    al = alpha_rows.data_ptr() if V > 0 else None
    check(get_lib().bitdelta_linear_rows(x.data_ptr(), variant_ids.data_ptr(), M, N, K, w_base.data_ptr(),
                                         al, ctypes.cast(ptrs, ctypes.c_void_p), V, y.data_ptr(),
                                         _dtype_code(out_dtype), *_workspace(ws, x.get_device()),
                                         _stream(stream), PATHS[path]), "bitdelta_linear_rows")
    return y


def group(variant_ids, V: int, workspace, stream=None) -> None:
    """Group one batch's tokens by variant into ``workspace``."""
    _need_cuda(variant_ids)
    check(get_lib().bitdelta_group(variant_ids.data_ptr(), variant_ids.numel(), V,
                                   *_workspace(workspace, variant_ids.get_device()), _stream(stream)),
          "bitdelta_group")


def linear_grouped(x, w_base, alphas, bits_ptrs, V: int, y, workspace, path: str = "auto",
                   stream=None) -> None:
    """The fused linear on a batch grouped by ``group`` (outputs into ``y``).
    ``bits_ptrs`` is the host pointer array from ``bits_pointer_array``."""
    M, K = x.shape
    N = w_base.shape[0]
    al = alphas.data_ptr() if V > 0 else None
    check(get_lib().bitdelta_linear_grouped(x.data_ptr(), M, N, K, w_base.data_ptr(), al,
                                            ctypes.cast(bits_ptrs, ctypes.c_void_p), V,
                                            y.data_ptr(), _dtype_code(y.dtype),
                                            *_workspace(workspace, x.get_device()),
                                            _stream(stream), PATHS[path]),
          "bitdelta_linear_grouped")


# -- attention over a key/value cache -----------------------------------------------

# (A decode step of one request takes a few microseconds on the GPU: what a call
# asks of its tensors it asks once, and the cache's description is packed, not built
# as an object.)
_DESC = struct.Struct("@PPqqiiqqq")        # KVCacheDesc's layout


def _desc_of(k, v):
    torch = _torch()
    shape, strides = k.shape, k.stride()
    if len(shape) != 4 or v.shape != shape or v.stride() != strides:
        raise ValueError("k and v must be 4-D [slots, capacity, kv_heads, head_dim] of one shape and strides")
    if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16:
        raise TypeError("the cache must be bfloat16")
    S, C, H, D = shape
    ss, st, sh, sd = strides
    dev = k.get_device()                   # -1 on the CPU
    if dev < 0 or v.get_device() != dev or sd != 1:
        raise ValueError("the cache must be CUDA tensors on one device with contiguous head_dim")
    # the stride of a dimension of one entry is never used, and torch leaves it open
    return shape, dev, _DESC.pack(k.data_ptr(), v.data_ptr(), S, C, H, D, ss if S > 1 else D, st if C > 1 else D,
                             sh if H > 1 else D)


def _int32(name, t, dev, *shape):
    if t is None:
        return None
    if t.dtype is not _torch().int32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s on the cache's device" % (name, shape))
    return t.data_ptr()


def _attn_args(q, D, out, dev):
    torch = _torch()
    shape, strides = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != D or q.dtype is not torch.bfloat16 or q.get_device() != dev:
        raise ValueError("q must be a bf16 tensor [rows, q_heads, head_dim] on the cache's device")
    T, H, _ = shape
    if strides[2] != 1 or (H > 1 and strides[1] != D):
        raise ValueError("the heads of a row of q must be contiguous")
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    elif out.shape != shape or out.dtype is not torch.bfloat16 or out.get_device() != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor of q's shape on the cache's device")
    return T, H, strides[0] if T > 1 else H * D, out


def _weights_ptr(weights, dev, S, H, C):
    if weights is None:
        return None
    if (weights.dtype is not _torch().float32 or weights.shape != (S, H, C) or weights.get_device() != dev
            or not weights.is_contiguous()):
        raise ValueError("weights must be contiguous float32 [slots, kv_heads, capacity] on the cache's device")
    return weights.data_ptr()


def _mask_args(window, sinks):
    """As the C ABI's int32 has them: a number beyond it means no more than the largest
    (no position reaches it), and one below zero stays one."""
    return max(-1, min(window, 0x7FFFFFFF)), max(-1, min(sinks, 0x7FFFFFFF))


def _prefix_args(prefix_ids, prefix_slots, prefix_lens, dev, B):
    if prefix_ids is None and prefix_slots is None and prefix_lens is None:
        return None, None, None, 0
    if prefix_ids is None or prefix_slots is None or prefix_lens is None:
        raise ValueError("prefix_ids, prefix_slots and prefix_lens go together")
    P = prefix_slots.numel()
    return (_int32("prefix_ids", prefix_ids, dev, B), _int32("prefix_slots", prefix_slots, dev, P),
            _int32("prefix_lens", prefix_lens, dev, P), P)


def attn_workspace(tokens: int, batch: int, q_heads: int, kv_heads: int, head_dim: int, weigh_len: int = 0,
                   device=None):
    """Zeroed workspace for attention calls of at most ``tokens`` query rows and
    ``batch`` requests; ``weigh_len``: the cache's capacity if decode
    accumulates weights."""
    torch = _torch()
    n = int(get_lib().bitdelta_attn_workspace(tokens, batch, q_heads, kv_heads, head_dim, weigh_len))
    if n == 0:
        raise BitDeltaError(BD_ERR_SHAPE, "bitdelta_attn_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def attn_decode(q, k_cache, v_cache, lens, workspace, slots=None, window: int = 0, sinks: int = 0, scale=None,
                weights=None, out=None, stream=None):
    """Attention of one new token a request: q [B, q_heads, head_dim] bf16 on the
    cache [slots, capacity, kv_heads, head_dim] (see ``bitdelta_attn_decode``).
    ``weights`` (f32 [slots, kv_heads, capacity]) is added to in place;
    ``scale`` defaults to head_dim ** -0.5.  Returns out [B, q_heads, head_dim]."""
    return attn_decode_prefix(q, k_cache, v_cache, lens, None, None, None, workspace, slots=slots, window=window,
                              sinks=sinks, scale=scale, weights=weights, out=out, stream=stream)


def attn_decode_prefix(q, k_cache, v_cache, lens, prefix_ids, prefix_slots, prefix_lens, workspace, slots=None,
                       window: int = 0, sinks: int = 0, scale=None, weights=None, out=None, stream=None):
    """``attn_decode`` for requests that share prefixes: request b's keys follow
    the ``prefix_lens[p]`` keys in slot ``prefix_slots[p]``, p = ``prefix_ids[b]``
    (-1: none), which are read once for up to 256 rows, requests times heads of a
    group (see ``bitdelta_attn_decode_prefix``)."""
    (S, C, Hk, D), dev, desc = _desc_of(k_cache, v_cache)
    B, H, stride, out = _attn_args(q, D, out, dev)
    rest = (*_mask_args(window, sinks), D ** -0.5 if scale is None else scale, _weights_ptr(weights, dev, S, Hk, C), out.data_ptr(),
            *_workspace(workspace, dev), _stream(stream))
    ids, pslots, plens, P = _prefix_args(prefix_ids, prefix_slots, prefix_lens, dev, B)
    lib = get_lib()
    if P == 0:
        code = lib.bitdelta_attn_decode(q.data_ptr(), stride, B, H, desc, _int32("slots", slots, dev, B),
                                        _int32("lens", lens, dev, B), *rest)
    else:
        code = lib.bitdelta_attn_decode_prefix(q.data_ptr(), stride, B, H, desc, _int32("slots", slots, dev, B),
                                               _int32("lens", lens, dev, B), ids, pslots, plens, P, *rest)
    if code != BD_OK:
        check(code, "bitdelta_attn_decode" if P == 0 else "bitdelta_attn_decode_prefix")
    return out


def attn_prefill(q, k_cache, v_cache, cu_q, lens, workspace, slots=None, window: int = 0, sinks: int = 0, scale=None,
                 prefix_ids=None, prefix_slots=None, prefix_lens=None, out=None, stream=None):
    """Causal attention of several new tokens a request: rows ``cu_q[b]`` to
    ``cu_q[b+1]`` of q [T, q_heads, head_dim] are request b's newest tokens,
    whose keys are the last of its ``lens[b]`` keys in the cache (see
    ``bitdelta_attn_prefill``).  Returns out [T, q_heads, head_dim]."""
    (_, _, _, D), dev, desc = _desc_of(k_cache, v_cache)
    T, H, stride, out = _attn_args(q, D, out, dev)
    B = lens.numel()
    ids, pslots, plens, P = _prefix_args(prefix_ids, prefix_slots, prefix_lens, dev, B)
    check(get_lib().bitdelta_attn_prefill(q.data_ptr(), stride, T, B, H, desc, _int32("slots", slots, dev, B),
                                          _int32("cu_q", cu_q, dev, B + 1), _int32("lens", lens, dev, B), ids, pslots, plens, P,
                                          *_mask_args(window, sinks), D ** -0.5 if scale is None else scale, out.data_ptr(),
                                          *_workspace(workspace, dev), _stream(stream)),
          "bitdelta_attn_prefill")
    return out


def evict_workspace(n: int, kv_heads: int, capacity: int, device=None):
    torch = _torch()
    b = int(get_lib().bitdelta_evict_workspace(n, kv_heads, capacity))
    if b == 0:
        raise BitDeltaError(BD_ERR_SHAPE, "bitdelta_evict_workspace")
    return torch.zeros(b, dtype=torch.uint8, device=device)


def cache_evict(k_cache, v_cache, weights, lens, src, dst, budget: int, workspace, sinks: int = 0, recent: int = 0,
                kept=None, stream=None) -> None:
    """Move requests from slots ``src`` to slots ``dst``, keeping the first
    ``sinks``, the last ``recent`` and the heaviest other keys, ``budget`` in
    all, of every head (see ``bitdelta_cache_evict``).  ``lens`` holds a length
    for every slot.  ``kept`` (int32 [n, kv_heads, budget]) receives the kept
    keys' old places."""
    (S, C, H, _), dev, desc = _desc_of(k_cache, v_cache)
    n = src.numel()
    if weights is None:
        raise ValueError("weights are needed")
    check(get_lib().bitdelta_cache_evict(desc, _weights_ptr(weights, dev, S, H, C), _int32("lens", lens, dev, S),
                                         _int32("src", src, dev, n), _int32("dst", dst, dev, n), n, budget, sinks, recent,
                                         _int32("kept", kept, dev, n, H, budget), *_workspace(workspace, dev),
                                         _stream(stream)), "bitdelta_cache_evict")


# -- a key/value cache held in 4 bits ------------------------------------------------

_DESC4 = struct.Struct("@Pqqiiqq")         # KVCache4Desc's layout


def cache4(slots: int, capacity: int, kv_heads: int, head_dim: int, device=None):
    """An empty 4-bit cache, uint8 [slots, kv_heads, capacity / 16, 17 * head_dim]
    (see ``bd_kv_cache4``): blocks of 16 tokens of one head; ``capacity`` a multiple of 16."""
    torch = _torch()
    if int(get_lib().bitdelta_cache4_bytes(slots, capacity, kv_heads, head_dim)) == 0:
        raise BitDeltaError(BD_ERR_SHAPE, "bitdelta_cache4_bytes")
    return torch.zeros((slots, kv_heads, capacity // 16, 17 * head_dim), dtype=torch.uint8, device=device)


def _desc4_of(cache):
    shape, strides = cache.shape, cache.stride()
    if len(shape) != 4 or shape[3] not in (17 * 64, 17 * 128):
        raise ValueError("the cache must be 4-D [slots, kv_heads, capacity / 16, 17 * head_dim], head_dim 64 or 128")
    if cache.dtype is not _torch().uint8:
        raise TypeError("the cache must be uint8")
    S, H, N, W = shape
    ss, sh, sn, sb = strides
    dev = cache.get_device()
    if dev < 0 or sb != 1 or (N > 1 and sn != W):
        raise ValueError("the cache must be a CUDA tensor whose blocks of a head follow one another")
    # the stride of a dimension of one entry is never used, and torch leaves it open
    return (H, W // 17), dev, _DESC4.pack(cache.data_ptr(), S, 16 * N, H, W // 17, ss if S > 1 else W, sh if H > 1 else W)


def _rows4(name, t, H, D, dev):
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != H or shape[2] != D or t.dtype is not _torch().bfloat16 or t.get_device() != dev:
        raise ValueError("%s must be a bf16 tensor [rows, kv_heads, head_dim] on the cache's device" % name)
    if strides[2] != 1 or (H > 1 and strides[1] != D):
        raise ValueError("the heads of a row of %s must be contiguous" % name)
    return shape[0], t.data_ptr(), strides[0] if shape[0] > 1 else H * D


def _move4(entry, k, v, cache, lens, workspace, slots, cu_q, stream):
    (H, D), dev, desc = _desc4_of(cache)
    T, k_ptr, k_stride = _rows4("k", k, H, D, dev)
    rows, v_ptr, v_stride = _rows4("v", v, H, D, dev)
    B = lens.numel()
    if rows != T or (cu_q is None and T != B):
        raise ValueError("k and v must have one number of rows, without cu_q one for each request")
    code = getattr(get_lib(), entry)(k_ptr, k_stride, v_ptr, v_stride, T, B, desc, _int32("slots", slots, dev, B),
                                     _int32("cu_q", cu_q, dev, B + 1), _int32("lens", lens, dev, B),
                                     *_workspace(workspace, dev), _stream(stream))
    if code != BD_OK:
        check(code, entry)


def cache4_write(k, v, cache, lens, workspace, slots=None, cu_q=None, stream=None) -> None:
    """Quantise new tokens into a 4-bit cache: rows ``cu_q[b]`` to ``cu_q[b+1]``
    of k and v [T, kv_heads, head_dim] bf16 become the last of request b's ``lens[b]`` keys
    (without ``cu_q`` one row a request; see ``bitdelta_cache4_write``)."""
    _move4("bitdelta_cache4_write", k, v, cache, lens, workspace, slots, cu_q, stream)


def cache4_read(k, v, cache, lens, workspace, slots=None, cu_q=None, stream=None):
    """Read keys and values back into rows of k and v: what ``cache4_write`` of the
    same arguments would have written, as the cache holds it (see ``bitdelta_cache4_read``).  Returns k, v."""
    _move4("bitdelta_cache4_read", k, v, cache, lens, workspace, slots, cu_q, stream)
    return k, v


def _longest(n):
    """As the C ABI's int64 has it: a number beyond what it takes stays one."""
    return max(-1, min(n, 1 << 40))


def attn4_workspace(tokens: int, batch: int, q_heads: int, kv_heads: int, head_dim: int, longest: int = 0, device=None):
    """Zeroed workspace for attention calls on a 4-bit cache of at most ``tokens`` query
    rows and ``batch`` requests; ``longest``: the most keys of a request that
    ``attn4_prefill`` serves (0: decode only)."""
    torch = _torch()
    n = int(get_lib().bitdelta_attn4_workspace(tokens, batch, q_heads, kv_heads, head_dim, _longest(longest)))
    if n == 0:
        raise BitDeltaError(BD_ERR_SHAPE, "bitdelta_attn4_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def attn4_decode(q, cache, lens, workspace, slots=None, window: int = 0, sinks: int = 0, scale=None, out=None, stream=None):
    """``attn_decode`` on a 4-bit cache (see ``bitdelta_attn4_decode``)."""
    (_, D), dev, desc = _desc4_of(cache)
    B, H, stride, out = _attn_args(q, D, out, dev)
    code = get_lib().bitdelta_attn4_decode(q.data_ptr(), stride, B, H, desc, _int32("slots", slots, dev, B),
                                           _int32("lens", lens, dev, B), *_mask_args(window, sinks),
                                           D ** -0.5 if scale is None else scale, out.data_ptr(),
                                           *_workspace(workspace, dev), _stream(stream))
    if code != BD_OK:
        check(code, "bitdelta_attn4_decode")
    return out


def attn4_prefill(q, cache, cu_q, lens, workspace, longest: int, slots=None, window: int = 0, sinks: int = 0, scale=None,
                  out=None, stream=None):
    """``attn_prefill`` on a 4-bit cache, for requests of at most ``longest`` keys, what the
    workspace was made for or less (see ``bitdelta_attn4_prefill``)."""
    (_, D), dev, desc = _desc4_of(cache)
    T, H, stride, out = _attn_args(q, D, out, dev)
    B = lens.numel()
    check(get_lib().bitdelta_attn4_prefill(q.data_ptr(), stride, T, B, H, desc, _int32("slots", slots, dev, B),
                                           _int32("cu_q", cu_q, dev, B + 1), _int32("lens", lens, dev, B), _longest(longest),
                                           *_mask_args(window, sinks), D ** -0.5 if scale is None else scale, out.data_ptr(),
                                           *_workspace(workspace, dev), _stream(stream)), "bitdelta_attn4_prefill")
    return out


def device_status(workspace, stream=None) -> int:
    """Synchronise, read and clear the status word of a workspace."""
    return int(get_lib().bitdelta_device_status(workspace.data_ptr(), _stream(stream)))
