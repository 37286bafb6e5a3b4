"""TQ4_1S weight codec and fused dequant-GEMV for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI in ``include/tq.h`` (``libtq.so``, built
in-tree by ``dequant_gemv_tq4_b200/build.py``).  Every step of the path runs in
the library's CUDA kernels; this module only marshals arguments.  PyTorch is
used for device memory and streams.  There is no CPU fallback: if the
library cannot be loaded, every call raises.

Two layers:
  * ``tq_*`` functions with the C names and raw integer pointers (what the
    ABI tests call);
  * tensor helpers (``quantize``, ``dequantize``, ``prerotate``, ``gemm``,
    ``gemv``, ``gemm_xrot``; ``rope``, ``kv_append``, ``kv_read``,
    ``kv_attention``, ``kv_commit`` for the key/value cache) that allocate
    outputs with torch and pass ``data_ptr()`` and the current CUDA stream.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
_DTYPE_CODE = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}
STATUS_NAMES = {0: "TQ_OK", 1: "TQ_ERR_INVALID_ARG", 2: "TQ_ERR_SHAPE", 3: "TQ_ERR_ALIGNMENT",
                4: "TQ_ERR_DTYPE", 5: "TQ_ERR_WORKSPACE", 6: "TQ_ERR_CUDA", 7: "TQ_ERR_UNSUPPORTED",
                8: "TQ_ERR_TIMEOUT"}
TQ_MAX_BATCH = 8


class GemmDesc(ctypes.Structure):
    """Mirror of ``tq_gemm_desc`` in include/tq.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("X", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("Y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64)]


class DequantDesc(ctypes.Structure):
    """Mirror of ``tq_dequant_desc`` in include/tq.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("w_out", ctypes.c_void_p), ("ldo", ctypes.c_int64)]


class Nvfp4GemmDesc(ctypes.Structure):
    """Mirror of ``tq_nvfp4_gemm_desc`` in include/tq.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("X", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


TQ_NVFP4_TENSOR_BYTES = 16

_lock = threading.Lock()
_lib = None


class KvCache(ctypes.Structure):
    """Mirror of ``tq_kv_cache`` in include/tq.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("batch", ctypes.c_int64), ("pages_per_seq", ctypes.c_int64),
                ("page_table_ld", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    """Mirror of ``tq_rope_desc`` in include/tq.h."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("scale", ctypes.c_float)]


class TQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load_library() -> ctypes.CDLL:
    """Load libtq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtq.so not built ({LIB_PATH}); run dequant_gemv_tq4_b200/build.py")
        lib = ctypes.CDLL(LIB_PATH)
        P, I64, SZ, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        sig = {
            "tq_status_string": ([I], ctypes.c_char_p),
            "tq_codes_bytes": ([I64, I64], SZ),
            "tq_scales_bytes": ([I64, I64], SZ),
            "tq_xrot_bytes": ([I64, I64], SZ),
            "tq_gemm_workspace_bytes": ([I64, I64, I64], SZ),
            "tq_quantize": ([P, I, I64, I64, I64, P, P, P], I),
            "tq_dequantize": ([P, P, I64, I64, P, I, I64, P], I),
            "tq_dequantize_batch": ([ctypes.POINTER(DequantDesc), I, I, P], I),
            "tq_prerotate": ([P, I, I64, I64, I64, P, P], I),
            "tq_gemm": ([P, P, I64, I64, P, I, I64, I64, P, I, I64, P, SZ, P], I),
            "tq_gemv": ([P, P, I64, I64, P, I, P, I, P, SZ, P], I),
            "tq_gemm_xrot": ([P, P, I64, I64, P, I64, P, I, I64, P, SZ, P], I),
            "tq_gemm_batch_workspace_bytes": ([ctypes.POINTER(GemmDesc), I, I64], SZ),
            "tq_gemm_batch": ([ctypes.POINTER(GemmDesc), I, I64, I, I, P, SZ, P], I),
            "tq_workspace_status": ([P, I, P], I),
            "tq_debug_set_flags": ([ctypes.c_uint32], None),
            "tq_gemv_static_scratch": ([P, P, I64, I64, P, I, P, I, P], I),
            "tq_static_scratch_status": ([I, P], I),
            "tq_gemm_prefill_workspace_bytes": ([I64, I64], SZ),
            "tq_gemm_prefill": ([P, P, I64, I64, P, I, I64, I64, P, I, I64, P, SZ, P], I),
            "tq_prefill_xrot_bytes": ([I64, I64], SZ),
            "tq_prerotate_plain": ([P, I, I64, I64, I64, P, P], I),
            "tq_gemm_prefill_xrot": ([P, P, I64, I64, P, I64, P, I, I64, P, SZ, P], I),
            "tq_rope": ([P, P, I, I64, I64, I64, I64, I64, I64, I64, P, ctypes.POINTER(RopeDesc), P], I),
            "tq_kv_codes_bytes": ([I64, I64, I64, I64], SZ),
            "tq_kv_scales_bytes": ([I64, I64, I64, I64], SZ),
            "tq_kv_append": ([ctypes.POINTER(KvCache), P, P, I64, P, I64, I64, P, I64, I64, I, P,
                              ctypes.POINTER(RopeDesc), P], I),
            "tq_kv_read": ([ctypes.POINTER(KvCache), P, P, I64, P, I64, I64, P, I64, I64, I, P], I),
            "tq_kv_attention_workspace_bytes": ([I64, I64, I64, I64, I64], SZ),
            "tq_kv_attention": ([ctypes.POINTER(KvCache), P, P, I64, P, I, I64, I64, I64, P, I, I64, I64, I64, I64,
                                 I64, ctypes.c_float, P, SZ, P], I),
            "tq_kv_commit": ([ctypes.POINTER(KvCache), I64, I64, I64, P, P, I64, I64, P], I),
            "tq_nvfp4_scales_bytes": ([I64, I64], SZ),
            "tq_nvfp4_quantize": ([P, I, I64, I64, I64, P, P, P, P], I),
            "tq_nvfp4_dequantize": ([P, P, P, I64, I64, P, I, I64, P], I),
            "tq_nvfp4_gemm": ([P, P, P, I64, I64, P, I, I64, I64, P, I, I64, P, SZ, P], I),
            "tq_nvfp4_gemm_batch_workspace_bytes": ([ctypes.POINTER(Nvfp4GemmDesc), I, I64], SZ),
            "tq_nvfp4_gemm_batch": ([ctypes.POINTER(Nvfp4GemmDesc), I, I64, I, I, P, SZ, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise TQError(status, where)


# ---------------------------------------------------------------------------
# raw C-ABI layer (integer pointers)
# ---------------------------------------------------------------------------
def status_string(status: int) -> str:
    return load_library().tq_status_string(int(status)).decode()


def tq_codes_bytes(n: int, k: int) -> int:
    return int(load_library().tq_codes_bytes(n, k))


def tq_scales_bytes(n: int, k: int) -> int:
    return int(load_library().tq_scales_bytes(n, k))


def tq_xrot_bytes(m: int, k: int) -> int:
    return int(load_library().tq_xrot_bytes(m, k))


def tq_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(load_library().tq_gemm_workspace_bytes(m, n, k))


def tq_quantize(w, wt, n, k, ldw, codes, scales, stream) -> int:
    return load_library().tq_quantize(w, wt, n, k, ldw, codes, scales, stream)


def tq_dequantize(codes, scales, n, k, w_out, ot, ldo, stream) -> int:
    return load_library().tq_dequantize(codes, scales, n, k, w_out, ot, ldo, stream)


def tq_dequantize_batch(descs, count, ot, stream) -> int:
    return load_library().tq_dequantize_batch(descs, count, ot, stream)


def tq_prerotate(X, xt, m, k, ldx, xrot, stream) -> int:
    return load_library().tq_prerotate(X, xt, m, k, ldx, xrot, stream)


def tq_gemm(codes, scales, n, k, X, xt, m, ldx, Y, yt, ldy, workspace, ws_bytes, stream) -> int:
    return load_library().tq_gemm(codes, scales, n, k, X, xt, m, ldx, Y, yt, ldy, workspace, ws_bytes, stream)


def tq_gemv(codes, scales, n, k, x, xt, y, yt, workspace, ws_bytes, stream) -> int:
    return load_library().tq_gemv(codes, scales, n, k, x, xt, y, yt, workspace, ws_bytes, stream)


def tq_gemm_xrot(codes, scales, n, k, xrot, m, Y, yt, ldy, workspace, ws_bytes, stream) -> int:
    return load_library().tq_gemm_xrot(codes, scales, n, k, xrot, m, Y, yt, ldy, workspace, ws_bytes, stream)


def tq_gemm_batch_workspace_bytes(descs, count, m) -> int:
    return int(load_library().tq_gemm_batch_workspace_bytes(descs, count, m))


def tq_gemm_batch(descs, count, m, xt, yt, workspace, ws_bytes, stream) -> int:
    return load_library().tq_gemm_batch(descs, count, m, xt, yt, workspace, ws_bytes, stream)


def tq_workspace_status(workspace, clear, stream) -> int:
    return load_library().tq_workspace_status(workspace, clear, stream)


def tq_debug_set_flags(flags: int) -> None:
    load_library().tq_debug_set_flags(flags)


def tq_gemv_static_scratch(codes, scales, n, k, x, xt, y, yt, stream) -> int:
    """GEMV without a workspace argument, for callers that cannot allocate
    device memory: the scratch is a fixed array inside the library (see
    include/tq.h).  Calls that overlap on the GPU must not share it."""
    return load_library().tq_gemv_static_scratch(codes, scales, n, k, x, xt, y, yt, stream)


def tq_static_scratch_status(clear, stream) -> int:
    """Timeout flag of the last tq_gemv_static_scratch call (synchronises)."""
    return load_library().tq_static_scratch_status(clear, stream)


def tq_gemm_prefill_workspace_bytes(m: int, k: int) -> int:
    return int(load_library().tq_gemm_prefill_workspace_bytes(m, k))


def tq_prefill_xrot_bytes(m: int, k: int) -> int:
    return int(load_library().tq_prefill_xrot_bytes(m, k))


def tq_prerotate_plain(X, xt, m, k, ldx, xrot, stream) -> int:
    return load_library().tq_prerotate_plain(X, xt, m, k, ldx, xrot, stream)


def tq_gemm_prefill_xrot(codes, scales, n, k, xrot, m, Y, yt, ldy, workspace, ws_bytes, stream) -> int:
    return load_library().tq_gemm_prefill_xrot(codes, scales, n, k, xrot, m, Y, yt, ldy, workspace, ws_bytes, stream)


def tq_gemm_prefill(codes, scales, n, k, X, xt, m, ldx, Y, yt, ldy, workspace, ws_bytes, stream) -> int:
    return load_library().tq_gemm_prefill(codes, scales, n, k, X, xt, m, ldx, Y, yt, ldy, workspace, ws_bytes,
                                          stream)


def tq_nvfp4_scales_bytes(n: int, k: int) -> int:
    return int(load_library().tq_nvfp4_scales_bytes(n, k))


def tq_nvfp4_quantize(w, wt, n, k, ldw, codes, scales, tensor_scale, stream) -> int:
    return load_library().tq_nvfp4_quantize(w, wt, n, k, ldw, codes, scales, tensor_scale, stream)


def tq_nvfp4_dequantize(codes, scales, tensor_scale, n, k, w_out, ot, ldo, stream) -> int:
    return load_library().tq_nvfp4_dequantize(codes, scales, tensor_scale, n, k, w_out, ot, ldo, stream)


def tq_nvfp4_gemm(codes, scales, tensor_scale, n, k, X, xt, m, ldx, Y, yt, ldy, workspace, ws_bytes, stream) -> int:
    return load_library().tq_nvfp4_gemm(codes, scales, tensor_scale, n, k, X, xt, m, ldx, Y, yt, ldy, workspace,
                                        ws_bytes, stream)


def tq_nvfp4_gemm_batch_workspace_bytes(descs, count, m) -> int:
    return int(load_library().tq_nvfp4_gemm_batch_workspace_bytes(descs, count, m))


def tq_nvfp4_gemm_batch(descs, count, m, xt, yt, workspace, ws_bytes, stream) -> int:
    return load_library().tq_nvfp4_gemm_batch(descs, count, m, xt, yt, workspace, ws_bytes, stream)


def tq_rope(x, out, t, tokens, heads, dim, x_token_stride, x_head_stride, out_token_stride, out_head_stride,
            positions, rope, stream) -> int:
    return load_library().tq_rope(x, out, t, tokens, heads, dim, x_token_stride, x_head_stride, out_token_stride,
                                  out_head_stride, positions, rope, stream)


def tq_kv_codes_bytes(pages: int, kv_heads: int, head_dim: int, page_size: int) -> int:
    return int(load_library().tq_kv_codes_bytes(pages, kv_heads, head_dim, page_size))


def tq_kv_scales_bytes(pages: int, kv_heads: int, head_dim: int, page_size: int) -> int:
    return int(load_library().tq_kv_scales_bytes(pages, kv_heads, head_dim, page_size))


def tq_kv_append(cache, seqs, places, tokens, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, t,
                 positions, rope, stream) -> int:
    return load_library().tq_kv_append(cache, seqs, places, tokens, k, k_token_stride, k_head_stride, v,
                                       v_token_stride, v_head_stride, t, positions, rope, stream)


def tq_kv_read(cache, seqs, places, tokens, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, t,
               stream) -> int:
    return load_library().tq_kv_read(cache, seqs, places, tokens, k, k_token_stride, k_head_stride, v,
                                     v_token_stride, v_head_stride, t, stream)


def tq_kv_attention_workspace_bytes(batch: int, tree: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load_library().tq_kv_attention_workspace_bytes(batch, tree, heads, kv_heads, head_dim))


def tq_kv_attention(cache, lens, parents, parents_ld, q, qt, q_batch_stride, q_token_stride, q_head_stride, out, ot,
                    out_batch_stride, out_token_stride, out_head_stride, tree, heads, scale, workspace, ws_bytes,
                    stream) -> int:
    return load_library().tq_kv_attention(cache, lens, parents, parents_ld, q, qt, q_batch_stride, q_token_stride,
                                          q_head_stride, out, ot, out_batch_stride, out_token_stride,
                                          out_head_stride, tree, heads, scale, workspace, ws_bytes, stream)


def tq_kv_commit(cache, layers, code_layer_stride, scale_layer_stride, lens, path, path_ld, steps, stream) -> int:
    return load_library().tq_kv_commit(cache, layers, code_layer_stride, scale_layer_stride, lens, path, path_ld,
                                       steps, stream)


# ---------------------------------------------------------------------------
# tensor helpers
# ---------------------------------------------------------------------------
def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _device(device):
    """The device that was asked for (0 is one), else the current one."""
    return torch.cuda.current_device() if device is None else device


def _dt(t: torch.dtype) -> int:
    if t not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {t}")
    return _DTYPE_CODE[t]


def superblocks(k: int) -> int:
    return (k // 32 + 3) // 4


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return t.stride(0)


def workspace(m: int, n: int, k: int, device=None) -> torch.Tensor:
    """A workspace tensor for gemm/gemv/gemm_xrot of these sizes (zero-filled)."""
    nbytes = tq_gemm_workspace_bytes(m, n, k)
    if nbytes == 0:
        raise ValueError("invalid sizes for workspace query")
    return torch.zeros(nbytes, dtype=torch.uint8, device=_device(device))


def tiles(n: int) -> int:
    return (n + 15) // 16


def quantize(w: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
             stream=None):
    """Encode W (n x k, fp32/bf16/fp16, on the GPU).  Returns the packed planes
    (codes uint8 [T*NSB*1024], scales int16 [T*NSB*128] holding fp16 bit
    patterns), T = ceil(n/16), in the tile-major layout of include/tq.h."""
    n, k = w.shape
    if codes is None:
        codes = torch.empty(tq_codes_bytes(n, k), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(tq_scales_bytes(n, k) // 2, dtype=torch.int16, device=w.device)
    _check(tq_quantize(w.data_ptr(), _dt(w.dtype), n, k, _ld(w), codes.data_ptr(), scales.data_ptr(),
                       _stream(stream)), "tq_quantize")
    return codes, scales


def dequantize(codes: torch.Tensor, scales: torch.Tensor, n: int, k: int, dtype=torch.bfloat16,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((n, k), dtype=dtype, device=codes.device)
    _check(tq_dequantize(codes.data_ptr(), scales.data_ptr(), n, k, out.data_ptr(), _dt(out.dtype), _ld(out),
                         _stream(stream)), "tq_dequantize")
    return out


def dequant_descs(items):
    """items: sequence of (codes, scales, n, k, out [n, k]) -> ctypes array."""
    arr = (DequantDesc * len(items))()
    for i, (codes, scales, n, k, out) in enumerate(items):
        arr[i] = DequantDesc(codes.data_ptr(), scales.data_ptr(), n, k, out.data_ptr(), _ld(out))
    return arr


def dequantize_batch(items, stream=None, descs=None):
    """Dequantise every (codes, scales, n, k, out) in one launch (outputs of one dtype)."""
    dts = {it[4].dtype for it in items}
    if len(dts) != 1:
        raise ValueError("dequantize_batch: every output needs the same dtype")
    if descs is None:
        descs = dequant_descs(items)
    _check(tq_dequantize_batch(descs, len(items), _dt(dts.pop()), _stream(stream)), "tq_dequantize_batch")


def prerotate(X: torch.Tensor, xrot: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    X2 = X.view(1, -1) if X.dim() == 1 else X
    m, k = X2.shape
    if xrot is None:
        xrot = torch.empty(tq_xrot_bytes(m, k) // 2, dtype=torch.int16, device=X.device)
    _check(tq_prerotate(X2.data_ptr(), _dt(X2.dtype), m, k, _ld(X2), xrot.data_ptr(), _stream(stream)),
           "tq_prerotate")
    return xrot


def gemm(codes, scales, n: int, k: int, X: torch.Tensor, dtype=torch.float32, out=None, ws=None,
         stream=None) -> torch.Tensor:
    """Y[m, n] = X[m, k] @ w~[n, k]^T (w~ = the dequantised weights), fused."""
    X2 = X.view(1, -1) if X.dim() == 1 else X
    m = X2.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=X.device)
    if ws is None:
        ws = workspace(m, n, k, X.device)
    _check(tq_gemm(codes.data_ptr(), scales.data_ptr(), n, k, X2.data_ptr(), _dt(X2.dtype), m, _ld(X2),
                   out.data_ptr(), _dt(out.dtype), _ld(out), ws.data_ptr(), ws.numel(), _stream(stream)),
           "tq_gemm")
    return out


def prefill_workspace(m: int, k: int, device=None) -> torch.Tensor:
    nbytes = tq_gemm_prefill_workspace_bytes(m, k)
    if nbytes == 0:
        raise ValueError("invalid sizes for workspace query")
    return torch.zeros(nbytes, dtype=torch.uint8, device=_device(device))


def gemm_prefill(codes, scales, n: int, k: int, X: torch.Tensor, dtype=torch.float32, out=None, ws=None,
                 stream=None) -> torch.Tensor:
    """Y[m, n] = X[m, k] @ w~[n, k]^T on the tensor-core prefill path (any m)."""
    X2 = X.view(1, -1) if X.dim() == 1 else X
    m = X2.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=X.device)
    if ws is None:
        ws = prefill_workspace(m, k, X.device)
    _check(tq_gemm_prefill(codes.data_ptr(), scales.data_ptr(), n, k, X2.data_ptr(), _dt(X2.dtype), m, _ld(X2),
                           out.data_ptr(), _dt(out.dtype), _ld(out), ws.data_ptr(), ws.numel(), _stream(stream)),
           "tq_gemm_prefill")
    return out


def prerotate_plain(X: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """Plain row-major fp16 pre-rotation of X (m x k) for the prefill product."""
    X2 = X.view(1, -1) if X.dim() == 1 else X
    m, k = X2.shape
    if out is None:
        out = torch.empty((m, k), dtype=torch.float16, device=X.device)
    _check(tq_prerotate_plain(X2.data_ptr(), _dt(X2.dtype), m, k, _ld(X2), out.data_ptr(), _stream(stream)),
           "tq_prerotate_plain")
    return out


def gemm_prefill_xrot(codes, scales, n: int, k: int, xrot: torch.Tensor, dtype=torch.float32, out=None, ws=None,
                      stream=None) -> torch.Tensor:
    """The tensor-core product over an activation from ``prerotate_plain``."""
    m = xrot.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=xrot.device)
    if ws is None:
        ws = torch.zeros(256, dtype=torch.uint8, device=xrot.device)
    _check(tq_gemm_prefill_xrot(codes.data_ptr(), scales.data_ptr(), n, k, xrot.data_ptr(), m, out.data_ptr(),
                                _dt(out.dtype), _ld(out), ws.data_ptr(), ws.numel(), _stream(stream)),
           "tq_gemm_prefill_xrot")
    return out


def gemv(codes, scales, n: int, k: int, x: torch.Tensor, dtype=torch.float32, out=None, ws=None,
         stream=None) -> torch.Tensor:
    """y[n] = w~[n, k] @ x[k], fused (m = 1)."""
    if out is None:
        out = torch.empty((n,), dtype=dtype, device=x.device)
    if ws is None:
        ws = workspace(1, n, k, x.device)
    _check(tq_gemv(codes.data_ptr(), scales.data_ptr(), n, k, x.data_ptr(), _dt(x.dtype), out.data_ptr(),
                   _dt(out.dtype), ws.data_ptr(), ws.numel(), _stream(stream)), "tq_gemv")
    return out


def gemm_xrot(codes, scales, n: int, k: int, xrot: torch.Tensor, m: int, dtype=torch.float32, out=None,
              ws=None, stream=None) -> torch.Tensor:
    """The fused product with an activation pre-rotated by ``prerotate`` (m <= 32)."""
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=xrot.device)
    if ws is None:
        ws = workspace(m, n, k, xrot.device)
    _check(tq_gemm_xrot(codes.data_ptr(), scales.data_ptr(), n, k, xrot.data_ptr(), m, out.data_ptr(),
                        _dt(out.dtype), _ld(out), ws.data_ptr(), ws.numel(), _stream(stream)), "tq_gemm_xrot")
    return out


def batch_descs(items):
    """items: sequence of (codes, scales, n, k, X [m, k], Y [m, n]) -> ctypes array."""
    arr = (GemmDesc * len(items))()
    for i, (codes, scales, n, k, X, Y) in enumerate(items):
        X2 = X.view(1, -1) if X.dim() == 1 else X
        Y2 = Y.view(1, -1) if Y.dim() == 1 else Y
        arr[i] = GemmDesc(codes.data_ptr(), scales.data_ptr(), n, k, X2.data_ptr(), _ld(X2), Y2.data_ptr(), _ld(Y2))
    return arr


def batch_workspace(items, m: int, device=None) -> torch.Tensor:
    descs = batch_descs(items)
    nbytes = tq_gemm_batch_workspace_bytes(descs, len(items), m)
    if nbytes == 0:
        raise ValueError("invalid batch for workspace query")
    return torch.zeros(nbytes, dtype=torch.uint8, device=_device(device))


def gemm_batch(items, m: int = 1, ws=None, stream=None, descs=None):
    """Fused products for several matrices in two launches (one pre-rotation
    per distinct input, one product launch).  items as in ``batch_descs``;
    the outputs Y are written in place.  All X share one dtype, all Y too."""
    if descs is None:
        descs = batch_descs(items)
    X0, Y0 = items[0][4], items[0][5]
    if ws is None:
        ws = batch_workspace(items, m, X0.device)
    _check(tq_gemm_batch(descs, len(items), m, _dt(X0.dtype), _dt(Y0.dtype), ws.data_ptr(), ws.numel(),
                         _stream(stream)), "tq_gemm_batch")
    return [it[5] for it in items]


def workspace_status(ws: torch.Tensor, clear: bool = True, stream=None) -> int:
    """0 (TQ_OK) or 8 (TQ_ERR_TIMEOUT) for the last product that used ``ws``."""
    return tq_workspace_status(ws.data_ptr(), 1 if clear else 0, _stream(stream))


# ---------------------------------------------------------------------------
# NVFP4 comparison codec (tensor helpers)
# ---------------------------------------------------------------------------
def nvfp4_quantize(w: torch.Tensor, stream=None):
    """Encode W (n x k) as NVFP4.  Returns (codes uint8 [tq_codes_bytes],
    scales uint8 [tq_nvfp4_scales_bytes] of E4M3 bytes, tensor block float32[4]
    holding g at [0] and amax|W| at [1])."""
    n, k = w.shape
    codes = torch.empty(tq_codes_bytes(n, k), dtype=torch.uint8, device=w.device)
    scales = torch.empty(tq_nvfp4_scales_bytes(n, k), dtype=torch.uint8, device=w.device)
    tensor = torch.empty(TQ_NVFP4_TENSOR_BYTES // 4, dtype=torch.float32, device=w.device)
    _check(tq_nvfp4_quantize(w.data_ptr(), _dt(w.dtype), n, k, _ld(w), codes.data_ptr(), scales.data_ptr(),
                             tensor.data_ptr(), _stream(stream)), "tq_nvfp4_quantize")
    return codes, scales, tensor


def nvfp4_dequantize(codes, scales, tensor, n: int, k: int, dtype=torch.bfloat16, out=None,
                     stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((n, k), dtype=dtype, device=codes.device)
    _check(tq_nvfp4_dequantize(codes.data_ptr(), scales.data_ptr(), tensor.data_ptr(), n, k, out.data_ptr(),
                               _dt(out.dtype), _ld(out), _stream(stream)), "tq_nvfp4_dequantize")
    return out


def nvfp4_gemm(codes, scales, tensor, n: int, k: int, X: torch.Tensor, dtype=torch.float32, out=None, ws=None,
               stream=None) -> torch.Tensor:
    """Y[m, n] = X[m, k] @ w~[n, k]^T for NVFP4 weights (m <= 32), fused."""
    X2 = X.view(1, -1) if X.dim() == 1 else X
    m = X2.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=X.device)
    if ws is None:
        ws = workspace(m, n, k, X.device)
    _check(tq_nvfp4_gemm(codes.data_ptr(), scales.data_ptr(), tensor.data_ptr(), n, k, X2.data_ptr(),
                         _dt(X2.dtype), m, _ld(X2), out.data_ptr(), _dt(out.dtype), _ld(out), ws.data_ptr(),
                         ws.numel(), _stream(stream)), "tq_nvfp4_gemm")
    return out


def nvfp4_batch_descs(items):
    """items: sequence of (codes, scales, tensor, n, k, X [m, k], Y [m, n])."""
    arr = (Nvfp4GemmDesc * len(items))()
    for i, (codes, scales, tensor, n, k, X, Y) in enumerate(items):
        X2 = X.view(1, -1) if X.dim() == 1 else X
        Y2 = Y.view(1, -1) if Y.dim() == 1 else Y
        arr[i] = Nvfp4GemmDesc(codes.data_ptr(), scales.data_ptr(), tensor.data_ptr(), n, k, X2.data_ptr(),
                               _ld(X2), Y2.data_ptr(), _ld(Y2))
    return arr


def nvfp4_batch_workspace(items, m: int, device=None) -> torch.Tensor:
    descs = nvfp4_batch_descs(items)
    nbytes = tq_nvfp4_gemm_batch_workspace_bytes(descs, len(items), m)
    if nbytes == 0:
        raise ValueError("invalid batch for workspace query")
    return torch.zeros(nbytes, dtype=torch.uint8, device=_device(device))


def nvfp4_gemm_batch(items, m: int = 1, ws=None, stream=None, descs=None):
    """NVFP4 products for several matrices in two launches; outputs in place."""
    if descs is None:
        descs = nvfp4_batch_descs(items)
    X0, Y0 = items[0][5], items[0][6]
    if ws is None:
        ws = nvfp4_batch_workspace(items, m, X0.device)
    _check(tq_nvfp4_gemm_batch(descs, len(items), m, _dt(X0.dtype), _dt(Y0.dtype), ws.data_ptr(), ws.numel(),
                               _stream(stream)), "tq_nvfp4_gemm_batch")
    return [it[6] for it in items]


# ---------------------------------------------------------------------------
# key/value cache (tensor helpers)
# ---------------------------------------------------------------------------
def _bad(name: str, t: torch.Tensor, what: str):
    raise ValueError(f"{name}: expected {what}, got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _ints(t: torch.Tensor, name: str, device, shape) -> int:
    """Address of a contiguous int32 tensor of this shape."""
    if t.dtype is not torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        _bad(name, t, f"a contiguous int32 tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, device, shape):
    """Strides of a head operand, whose last one is 1."""
    st = t.stride()
    if t.shape != shape or t.device != device or (st[-1] != 1 and shape[-1] > 1):
        _bad(name, t, f"shape {tuple(shape)} on {device} with unit stride in the last dimension")
    return st


def _elsewhere(device, stream):
    """The context that a call has to run in, None if that is the current one:
    the library launches on the current device, and memory that a call allocates
    belongs to the stream that the call runs on."""
    if device.type != "cuda":
        raise ValueError("expected CUDA tensors")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream: expected one of {device}, got one of {stream.device}")
        return torch.cuda.stream(stream)
    return None if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _raw_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, layers: int | None = None, device=None):
    """A zero-filled pool of pages: (codes uint8 [pages, 2, kv_heads, page_size,
    head_dim / 2], scales int16 [pages, 2, kv_heads, page_size, head_dim / 16]),
    both with a leading dimension ``layers`` if that is given."""
    nbytes = tq_kv_codes_bytes(pages, kv_heads, head_dim, page_size)
    if nbytes == 0 and pages != 0:
        raise ValueError("kv_cache: head_dim is a multiple of 32 up to 256, page_size a power of two from 16 to 1024")
    lead = () if layers is None else (layers,)
    device = _device(device)
    codes = torch.zeros((*lead, pages, 2, kv_heads, page_size, head_dim // 2), dtype=torch.uint8, device=device)
    scales = torch.zeros((*lead, pages, 2, kv_heads, page_size, head_dim // 16), dtype=torch.int16, device=device)
    return codes, scales


def _cache(codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, layers: bool = False) -> KvCache:
    """The C description of one layer's cache (of layer 0, with ``layers``)."""
    shape, device = codes.shape, codes.device
    if len(shape) != 5 + layers or shape[-4] != 2 or codes.dtype is not torch.uint8:
        _bad("codes", codes, "uint8 [pages, 2, kv_heads, page_size, head_dim / 2]")
    half = shape[-1]
    if scales.dtype is not torch.int16 or scales.shape != (*shape[:-1], half // 8) or scales.device != device:
        _bad("scales", scales, f"int16 [pages, 2, kv_heads, page_size, head_dim / 16] on {device}")
    one_layer = layers and shape[0]
    if not (codes[0] if one_layer else codes).is_contiguous():
        _bad("codes", codes, "a contiguous tensor")
    if not (scales[0] if one_layer else scales).is_contiguous():
        _bad("scales", scales, "a contiguous tensor")
    if page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.device != device:
        _bad("page_table", page_table, f"int32 [batch, pages of a sequence] on {device}")
    batch, per_seq = page_table.shape
    ld, one = page_table.stride()
    if one != 1 and per_seq > 1:
        _bad("page_table", page_table, "unit stride in the last dimension")
    return KvCache(codes.data_ptr(), scales.data_ptr(), shape[-5], page_table.data_ptr(), batch, per_seq,
                   ld if batch > 1 else per_seq, shape[-3], 2 * half, shape[-2])


def _rope_desc(inv_freq: torch.Tensor, device, interleaved=False, scale=1.0, inverse=False) -> RopeDesc:
    if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or inv_freq.device != device or \
            not inv_freq.is_contiguous():
        _bad("inv_freq", inv_freq, f"a contiguous float32 vector on {device}")
    return RopeDesc(inv_freq.data_ptr(), 2 * inv_freq.shape[0], interleaved, inverse, scale)


def rope_frequencies(rot_dim: int, theta: float = 10000.0, factor: float = 1.0, scaling: str = "none",
                     original_context: int = 8192, low: float = 1.0, high: float = 4.0,
                     device=None) -> torch.Tensor:
    """Angles per position of ``rope``, theta^(-2i/rot_dim) for i < rot_dim / 2,
    computed in 64 bits, as a float32 vector on the GPU.  ``scaling`` lengthens
    the context by ``factor``:
      "linear"   every frequency divided by factor;
      "ntk"      theta multiplied by factor^(rot_dim / (rot_dim - 2));
      "by_parts" a frequency that turns more than ``high`` times over
                 original_context stays, one that turns fewer than ``low``
                 times is divided by factor, between them a linear blend."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim: a positive even number")
    if theta <= 0 or factor <= 0:
        raise ValueError("theta and factor: positive numbers")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim of at least 4")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freq = theta ** (-2.0 * torch.arange(rot_dim // 2, dtype=torch.float64) / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if not high > low:
            raise ValueError("by_parts: high has to be above low")
        turns = original_context * freq / (2.0 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / factor)
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(torch.float32).to(_device(device))


def rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False,
         scale: float = 1.0, inverse: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of x [tokens, heads, dim]: the first 2 * len(inv_freq)
    elements of each head rotated by positions[token] * inv_freq, the rest
    unchanged.  ``inverse`` rotates back (the gradient).  ``out`` may be x."""
    if x.dim() != 3:
        _bad("x", x, "[tokens, heads, dim]")
    dev = x.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return rope(x, positions, inv_freq, interleaved, scale, inverse, out)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype is not x.dtype:
        _bad("out", out, f"{x.dtype}")
    shape = x.shape
    xs, os_ = _heads(x, "x", dev, shape), _heads(out, "out", dev, shape)
    st = tq_rope(x.data_ptr(), out.data_ptr(), _dt(x.dtype), shape[0], shape[1], shape[2], xs[0], xs[1], os_[0],
                 os_[1], _ints(positions, "positions", dev, shape[:1]),
                 _rope_desc(inv_freq, dev, interleaved, scale, inverse), _raw_stream(dev))
    if st:
        _check(st, "tq_rope")
    return out


def kv_append(codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, seqs: torch.Tensor,
              places: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope=None, interleaved: bool = False,
              rope_scale: float = 1.0, stream=None) -> None:
    """Writes the records of keys k and values v [n, kv_heads, head_dim]: token i
    goes to place places[i] of sequence seqs[i].  ``rope`` = (positions,
    inv_freq) rotates the keys on their way in."""
    dev = codes.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv_append(codes, scales, page_table, seqs, places, k, v, rope, interleaved, rope_scale)
    cache = _cache(codes, scales, page_table)
    one = seqs.shape
    n = seqs.numel()
    shape = (n, cache.kv_heads, cache.head_dim)
    if k.dtype is not v.dtype:
        _bad("v", v, f"{k.dtype}")
    ks, vs = _heads(k, "k", dev, shape), _heads(v, "v", dev, shape)
    pos = desc = None
    if rope is not None:
        pos, desc = _ints(rope[0], "positions", dev, (n,)), _rope_desc(rope[1], dev, interleaved, rope_scale)
    st = tq_kv_append(cache, _ints(seqs, "seqs", dev, (n,)), _ints(places, "places", dev, one), n, k.data_ptr(), ks[0],
                      ks[1], v.data_ptr(), vs[0], vs[1], _dt(k.dtype), pos, desc, _raw_stream(dev))
    if st:
        _check(st, "tq_kv_append")


def kv_read(codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, seqs: torch.Tensor,
            places: torch.Tensor, dtype=None, k: torch.Tensor | None = None,
            v: torch.Tensor | None = None, stream=None):
    """(keys, values) [n, kv_heads, head_dim] of the tokens at places[i] of seqs[i],
    of ``dtype`` (that of k or v if one is given, else bfloat16)."""
    for name, t in (("k", k), ("v", v)):
        if t is not None and dtype is not None and t.dtype is not dtype:
            _bad(name, t, f"{dtype}")
    dev = codes.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv_read(codes, scales, page_table, seqs, places, dtype, k, v)
    cache = _cache(codes, scales, page_table)
    n = seqs.numel()
    shape = (n, cache.kv_heads, cache.head_dim)
    if k is None and v is None:
        k, v = scales.new_empty((2, *shape), dtype=dtype or torch.bfloat16).unbind(0)
    elif k is None:
        k = torch.empty(shape, dtype=v.dtype, device=dev)
    elif v is None:
        v = torch.empty(shape, dtype=k.dtype, device=dev)
    if k.dtype is not v.dtype:
        _bad("v", v, f"{k.dtype}")
    ks, vs = _heads(k, "k", dev, shape), _heads(v, "v", dev, shape)
    st = tq_kv_read(cache, _ints(seqs, "seqs", dev, (n,)), _ints(places, "places", dev, (n,)), n, k.data_ptr(), ks[0],
                    ks[1], v.data_ptr(), vs[0], vs[1], _dt(k.dtype), _raw_stream(dev))
    if st:
        _check(st, "tq_kv_read")
    return k, v


def kv_attention_workspace(batch: int, tree: int, heads: int, kv_heads: int, head_dim: int,
                           device=None) -> torch.Tensor:
    """A workspace tensor for ``kv_attention`` of these sizes."""
    device = _device(device)
    with torch.cuda.device(device):  # the size goes by the device's number of SMs
        nbytes = tq_kv_attention_workspace_bytes(batch, tree, heads, kv_heads, head_dim)
    if nbytes == 0:
        raise ValueError("invalid sizes for workspace query")
    return torch.empty(nbytes, dtype=torch.uint8, device=_device(device))


def kv_attention(codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                 q: torch.Tensor, parents: torch.Tensor | None = None, scale: float | None = None, dtype=None,
                 out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of q [batch, tree, heads, head_dim] over the cache: every row
    sees the lens[b] tokens of its sequence, its own drafted token (record at
    place lens[b] + i) and that token's ancestors by ``parents`` [batch, tree]
    (None: a chain).  ``scale`` defaults to head_dim^-0.5, ``dtype`` to out's if
    that is given, else to q's.
    Whether a wait expired can be asked of a workspace that was passed
    (``workspace_status(ws)``); one that the call allocates is gone with it."""
    if out is not None and dtype is not None and out.dtype is not dtype:
        _bad("out", out, f"{dtype}")
    dev = codes.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv_attention(codes, scales, page_table, lens, q, parents, scale, dtype, out, ws)
    cache = _cache(codes, scales, page_table)
    if q.dim() != 4:
        _bad("q", q, "[batch, tree, heads, head_dim]")
    batch, tree, heads, dim = q.shape
    shape = (cache.batch, tree, heads, cache.head_dim)
    if out is None:
        out = torch.empty_like(q, dtype=dtype, memory_format=torch.contiguous_format)
    qs, os_ = _heads(q, "q", dev, shape), _heads(out, "out", dev, shape)
    if ws is None:
        nbytes = tq_kv_attention_workspace_bytes(batch, tree, heads, cache.kv_heads, dim)
        if nbytes == 0:
            raise ValueError("kv_attention: invalid sizes (heads is a multiple of kv_heads, up to 64 drafted tokens)")
        ws = codes.new_empty((nbytes,))
    else:
        if ws.device != dev or not ws.is_contiguous():
            _bad("ws", ws, f"a contiguous tensor on {dev}")
        nbytes = ws.numel() * ws.element_size()
    par = None if parents is None else _ints(parents, "parents", dev, (batch, tree))
    st = tq_kv_attention(cache, _ints(lens, "lens", dev, (batch,)), par, tree, q.data_ptr(), _dt(q.dtype), qs[0],
                         qs[1], qs[2], out.data_ptr(), _dt(out.dtype), os_[0], os_[1], os_[2], tree, heads,
                         dim ** -0.5 if scale is None else scale, ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check(st, "tq_kv_attention")
    return out


def kv_commit(codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
              path: torch.Tensor, stream=None) -> None:
    """Moves the records of accepted drafted tokens together: record
    lens[b] + path[b, i] to place lens[b] + i, for increasing path[b] up to its
    first entry that does not increase (-1).  codes and scales of one layer, or
    with a leading dimension of layers that share the page table."""
    dev = codes.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return kv_commit(codes, scales, page_table, lens, path)
    layered = codes.dim() == 6
    cache = _cache(codes, scales, page_table, layered)
    layers, cs, ss = (codes.shape[0], codes.stride(0), scales.stride(0)) if layered else (1, 0, 0)
    batch, steps = cache.batch, path.shape[-1]
    st = tq_kv_commit(cache, layers, cs, ss, _ints(lens, "lens", dev, (batch,)),
                      _ints(path, "path", dev, (batch, steps)), steps, steps, _raw_stream(dev))
    if st:
        _check(st, "tq_kv_commit")
