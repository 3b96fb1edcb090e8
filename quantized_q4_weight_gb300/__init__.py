"""Python binding of libqgemv (include/qgemv.h): the Q4_0-weight x
Q8_0-activation decode GEMV on one GB300.

Argument marshalling only: every step runs in the library's CUDA kernels.
Most calls go through ctypes; those of the decode step between its GEMVs
(rope_kv, attn_prefix, logits_rules) through the compiled _binding.so,
because their kernels are shorter than the marshalling.
Tensors supply device pointers; work is enqueued on the current torch CUDA
stream.  The library is loaded from this directory (libqgemv.so, built by
``quantized_q4_weight_gb300._build.build()``); if it is missing, every call
raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

QK = 32
Q4_0_BYTES = 18
W_GGML, W_PACKED = 0, 1

STATUS = {0: "QGEMV_OK", 1: "QGEMV_ERR_INVALID_ARG", 2: "QGEMV_ERR_MISALIGNED", 3: "QGEMV_ERR_UNSUPPORTED",
          4: "QGEMV_ERR_WORKSPACE", 5: "QGEMV_ERR_CUDA", 6: "QGEMV_ERR_TIMEOUT", 7: "QGEMV_ERR_BAD_ID",
          8: "QGEMV_ERR_INTERNAL"}


class QgemvError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class SeqItem(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class SeqF32Item(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class SeqEpItem(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p)]


class GatherMatrix(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("expert_stride", ctypes.c_int64), ("xq", ctypes.c_void_p),
                ("xq_stride", ctypes.c_int64), ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class GatherF32Matrix(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("expert_stride", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64), ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


F32, F16, BF16 = 0, 1, 2
_DTYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "yarn": 3}


class KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int), ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("layout", ctypes.c_int), ("scaling", ctypes.c_int),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("orig_len", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("mscale", ctypes.c_double)]


class RopePlan(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_uint64 * 128), ("mscale", ctypes.c_float), ("rot_dim", ctypes.c_int),
                ("layout", ctypes.c_int)]

    @property
    def address(self) -> int:
        """Where this plan lies, for a direct call of the C function (a copy lies elsewhere)."""
        return ctypes.addressof(self)


class AttnBatchStruct(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("n_q", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("prefix_len", ctypes.c_int), ("prefix_pages", ctypes.c_void_p), ("suffix_len", ctypes.c_void_p),
                ("suffix_pages", ctypes.c_void_p), ("suffix_pages_stride", ctypes.c_int64),
                ("max_suffix", ctypes.c_int), ("scale", ctypes.c_float)]


class LogitsSpec(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("vocab", ctypes.c_int64), ("history", ctypes.c_void_p),
                ("history_stride", ctypes.c_int64), ("history_len", ctypes.c_void_p), ("max_history", ctypes.c_int),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("bias_len", ctypes.c_void_p), ("max_bias", ctypes.c_int), ("mask", ctypes.c_void_p),
                ("mask_stride", ctypes.c_int64)]


_lib = None

_VP, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "qgemv_status_string": ([_I32], ctypes.c_char_p),
    "qgemv_version": ([], _I32),
    "qgemv_q4_0_bytes": ([_I64, _I64], _SZ),
    "qgemv_xq_bytes": ([_I32, _I64], _SZ),
    "qgemv_pack_q4_0": ([_VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_unpack_q4_0": ([_VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_quantize_q8_0": ([_VP, _VP, _I32, _I64, _I32, _VP], _I32),
    "qgemv_workspace_bytes": ([_I64, _I64, _I32], _SZ),
    "qgemv_q4_0": ([_VP, _I32, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_q4_0_f32": ([_VP, _I32, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_q4_0_argmax": ([_VP, _I32, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_q4_0_argmax_f32": ([_VP, _I32, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_q4_0_argmax_noalloc": ([_VP, _I32, _VP, _VP, _VP, _I64, _I64, _I32, _VP], _I32),
    "qgemv_q4_0_top2": ([_VP, _I32, _VP, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_q4_0_top2_f32": ([_VP, _I32, _VP, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_verify_commit": ([_VP, _VP, _I32, _I32, _VP, _VP], _I32),
    "qgemv_q4_0_verify_f32": ([_VP, _I32, _VP, _VP, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_ffn_workspace_bytes": ([_I64, _I64, _I32], _SZ),
    "qgemv_q4_0_ffn": ([_VP, _VP, _VP, _I32, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_q4_0_ffn_residual": ([_VP, _VP, _VP, _I32, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_debug_silu_mul_q8": ([_VP, _VP, _VP, _I32, _I64, _VP], _I32),
    "qgemv_pack_q8_0": ([_VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_unpack_q8_0": ([_VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_requant_f32_q4_0": ([_VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_requant_q8_0_q4_0": ([_VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_q8_0_workspace_bytes": ([_I64, _I64, _I32], _SZ),
    "qgemv_q8_0": ([_VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_seq_workspace_bytes": ([ctypes.POINTER(SeqItem), _I32, _I32], _SZ),
    "qgemv_q4_0_seq": ([ctypes.POINTER(SeqItem), _I32, _I32, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_seq_f32_workspace_bytes": ([ctypes.POINTER(SeqF32Item), _I32, _I32], _SZ),
    "qgemv_q4_0_seq_f32": ([ctypes.POINTER(SeqF32Item), _I32, _I32, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_seq_ep_workspace_bytes": ([ctypes.POINTER(SeqEpItem), _I32, _I32, _I32], _SZ),
    "qgemv_q4_0_seq_ep": ([ctypes.POINTER(SeqEpItem), _I32, _I32, _I32, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_gather_workspace_bytes": ([ctypes.POINTER(GatherMatrix), _I32, _I32, _I32], _SZ),
    "qgemv_q4_0_gather": ([ctypes.POINTER(GatherMatrix), _I32, _VP, _I32, _I32, _I32, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_gather_f32_workspace_bytes": ([ctypes.POINTER(GatherF32Matrix), _I32, _I32, _I32], _SZ),
    "qgemv_q4_0_gather_f32": ([ctypes.POINTER(GatherF32Matrix), _I32, _VP, _I32, _I32, _I32, _I32, _VP, _SZ, _VP],
                              _I32),
    "qgemv_gs64_bytes": ([_I64, _I64], _SZ),
    "qgemv_pack_gs64": ([_VP, _VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_unpack_gs64": ([_VP, _VP, _VP, _I64, _I64, _VP], _I32),
    "qgemv_quantize_vec_i8": ([_VP, _VP, _VP, _I32, _I64, _VP], _I32),
    "qgemv_gs64_workspace_bytes": ([_I64, _I64, _I32], _SZ),
    "qgemv_gs64": ([_VP, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_gs64_f32": ([_VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ, _VP], _I32),
    "qgemv_rope_init": ([ctypes.POINTER(RopeConfig), ctypes.POINTER(RopePlan)], _I32),
    "qgemv_rope_kv": ([_VP, _VP, _VP, _VP, _I32, _I64, _I64, _I64, _VP, _VP, _I64, _I32, _I32, _VP, _I32, _I64, _VP,
                       _VP], _I32),
    "qgemv_attn_workspace_bytes": ([_VP, _VP], _SZ),
    "qgemv_attn_prefix": ([_VP, _I64, _I64, _VP, _VP, _VP, _I32, _I64, _I64, _VP, _VP, _SZ, _VP], _I32),
    "qgemv_logits_workspace_bytes": ([_VP], _SZ),
    "qgemv_logits_rules": ([_VP, _I32, _I64, _VP, _VP, _I64, _VP, _VP, _VP, _SZ, _VP], _I32),
    "qgemv_debug_block_isums": ([_VP, _I32, _VP, _VP, _I64, _I64, _I32, _VP], _I32),
    "qgemv_debug_block_isums_tc": ([_VP, _I32, _VP, _VP, _I64, _I64, _I32, _I32, _VP], _I32),
    "qgemv_debug_stream_read": ([_VP, _SZ, _I32, _I32, _I32, _I32, _VP, _VP], _I32),
    "qgemv_set_tuning": ([_I32, _I32, _I32, _I32], _I32),
    "qgemv_set_tc_min_tokens": ([_I32], _I32),
    "qgemv_set_ffn_fused": ([_I32], _I32),
    "qgemv_device_status": ([ctypes.POINTER(ctypes.c_int)], _I32),
}


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"libqgemv is not built ({_build.LIB} missing): run "
                               "quantized_q4_weight_gb300._build.build() first")
        L = ctypes.CDLL(_build.LIB)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


_ext = None


def _load_binding():
    """The compiled binding (raises if it has not been built)."""
    global _ext
    if _ext is None:
        lib()
        if not os.path.exists(_build.BINDING):
            raise RuntimeError(f"the binding is not built ({_build.BINDING} missing): run "
                               "quantized_q4_weight_gb300._build.build() first")
        from . import _binding as ext
        _ext = ext
    return _ext


def _check(code: int, what: str):
    if code != 0:
        raise QgemvError(code, what)


def _stream(stream=None):
    """A stream's handle; by default the current stream's (read as a number:
    building a Stream object takes longer than a small kernel)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _result(shape, dtype, beside, stream):
    """A new tensor on `beside`'s device for a call on `stream` (None: the current one),
    from that stream's memory: a block that the current stream has just let go may
    still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=beside.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=beside.device)


def _ptr(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors"
    return t.data_ptr()


# ----------------------------------------------------------------- sizes

def q4_0_bytes(N: int, K: int) -> int:
    return int(lib().qgemv_q4_0_bytes(N, K))


def xq_bytes(R: int, K: int) -> int:
    return int(lib().qgemv_xq_bytes(R, K))


def workspace_bytes(N: int, K: int, T: int) -> int:
    return int(lib().qgemv_workspace_bytes(N, K, T))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled workspace (the library keeps its counters at zero)."""
    return torch.zeros(max(int(nbytes), 16384), dtype=torch.uint8, device=device or "cuda")


# ----------------------------------------------------------------- calls

def pack_q4_0(w_ggml: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    out = out if out is not None else _result(q4_0_bytes(N, K), torch.uint8, w_ggml, stream)
    _check(lib().qgemv_pack_q4_0(_ptr(w_ggml), _ptr(out), N, K, _stream(stream)), "qgemv_pack_q4_0")
    return out


def unpack_q4_0(w_packed: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None):
    out = out if out is not None else _result(q4_0_bytes(N, K), torch.uint8, w_packed, stream)
    _check(lib().qgemv_unpack_q4_0(_ptr(w_packed), _ptr(out), N, K, _stream(stream)), "qgemv_unpack_q4_0")
    return out


def quantize_q8_0(x: torch.Tensor, R: int, K: int, batch: int = 1, out: torch.Tensor | None = None, stream=None):
    """x fp32 [batch, R, K] (any shape with that many elements) -> planar Q8_0 bytes."""
    assert x.dtype == torch.float32 and x.numel() == batch * R * K
    out = out if out is not None else _result(batch * xq_bytes(R, K), torch.uint8, x, stream)
    _check(lib().qgemv_quantize_q8_0(_ptr(x), _ptr(out), R, K, batch, _stream(stream)), "qgemv_quantize_q8_0")
    return out


def gemv(W, layout: int, xq, N: int, K: int, T: int, ws, y=None, stream=None) -> torch.Tensor:
    y = y if y is not None else _result((T, N), torch.float32, W, stream)
    _check(lib().qgemv_q4_0(_ptr(W), layout, _ptr(xq), _ptr(y), N, K, T, _ptr(ws), ws.numel(), _stream(stream)),
           "qgemv_q4_0")
    return y


def gemv_f32(W, layout: int, x, N: int, K: int, T: int, ws, y=None, stream=None) -> torch.Tensor:
    y = y if y is not None else _result((T, N), torch.float32, W, stream)
    _check(lib().qgemv_q4_0_f32(_ptr(W), layout, _ptr(x), _ptr(y), N, K, T, _ptr(ws), ws.numel(), _stream(stream)),
           "qgemv_q4_0_f32")
    return y


def gemv_argmax(W, layout: int, xq, N: int, K: int, T: int, ws, y=None, idx=None, stream=None):
    idx = idx if idx is not None else _result(T, torch.int64, W, stream)
    _check(lib().qgemv_q4_0_argmax(_ptr(W), layout, _ptr(xq), _ptr(y), _ptr(idx), N, K, T, _ptr(ws), ws.numel(),
                                   _stream(stream)), "qgemv_q4_0_argmax")
    return idx


def gemv_argmax_f32(W, layout: int, x, N: int, K: int, T: int, ws, y=None, idx=None, stream=None):
    """Argmax of W . x over rows for fp32 x[T][K] (quantised inside the kernel)."""
    idx = idx if idx is not None else _result(T, torch.int64, W, stream)
    _check(lib().qgemv_q4_0_argmax_f32(_ptr(W), layout, _ptr(x), _ptr(y), _ptr(idx), N, K, T, _ptr(ws), ws.numel(),
                                       _stream(stream)), "qgemv_q4_0_argmax_f32")
    return idx


def gemv_top2(W, layout: int, xq, N: int, K: int, T: int, ws, y=None, idx2=None, val2=None, stream=None):
    """The two best rows per token and their outputs: (idx2 int64 [T][2], val2 fp32 [T][2])."""
    idx2 = idx2 if idx2 is not None else _result((T, 2), torch.int64, W, stream)
    val2 = val2 if val2 is not None else _result((T, 2), torch.float32, W, stream)
    _check(lib().qgemv_q4_0_top2(_ptr(W), layout, _ptr(xq), _ptr(y), _ptr(idx2), _ptr(val2), N, K, T, _ptr(ws),
                                 ws.numel(), _stream(stream)), "qgemv_q4_0_top2")
    return idx2, val2


def gemv_top2_f32(W, layout: int, x, N: int, K: int, T: int, ws, y=None, idx2=None, val2=None, stream=None):
    """gemv_top2 for fp32 x[T][K] (quantised inside the kernel)."""
    idx2 = idx2 if idx2 is not None else _result((T, 2), torch.int64, W, stream)
    val2 = val2 if val2 is not None else _result((T, 2), torch.float32, W, stream)
    _check(lib().qgemv_q4_0_top2_f32(_ptr(W), layout, _ptr(x), _ptr(y), _ptr(idx2), _ptr(val2), N, K, T, _ptr(ws),
                                     ws.numel(), _stream(stream)), "qgemv_q4_0_top2_f32")
    return idx2, val2


def verify_f32(W, layout: int, x, tokens, N: int, K: int, T: int, ws, idx2=None, val2=None, n_commit=None,
               stream=None):
    """A verify step in one launch: the top-2 rows of W . x per position and the
    committed count of the verify rule on (tokens, idx2[:, 0])."""
    idx2 = idx2 if idx2 is not None else _result((T, 2), torch.int64, W, stream)
    val2 = val2 if val2 is not None else _result((T, 2), torch.float32, W, stream)
    n_commit = n_commit if n_commit is not None else _result(1, torch.int32, W, stream)
    _check(lib().qgemv_q4_0_verify_f32(_ptr(W), layout, _ptr(x), _ptr(tokens), _ptr(idx2), _ptr(val2), _ptr(n_commit),
                                       N, K, T, _ptr(ws), ws.numel(), _stream(stream)), "qgemv_q4_0_verify_f32")
    return idx2, val2, n_commit


def verify_commit(tokens, pred, n_commit=None, stream=None):
    """Committed predictions of one verify step (int32 device scalar): tokens[0]
    is the current token, tokens[1:] the drafts, pred[t] the prediction after
    tokens[:t+1] (int64 device tensors; pred may be a strided column such as
    idx2[:, 0] of gemv_top2)."""
    T = tokens.numel()
    assert pred.dim() == 1 and pred.numel() == T and tokens.is_contiguous()
    n_commit = n_commit if n_commit is not None else _result(1, torch.int32, tokens, stream)
    _check(lib().qgemv_verify_commit(_ptr(tokens), ctypes.c_void_p(pred.data_ptr()), pred.stride(0), T,
                                     _ptr(n_commit), _stream(stream)), "qgemv_verify_commit")
    return n_commit


def ffn_workspace_bytes(d_model: int, d_ff: int, T: int) -> int:
    return int(lib().qgemv_ffn_workspace_bytes(d_model, d_ff, T))


def ffn(W_gate, W_up, W_down, layout: int, x, d_model: int, d_ff: int, T: int, ws, y=None, stream=None):
    """y[T][d_model] = W_down . Q8_0(SiLU(W_gate . x) * (W_up . x)) for fp32 x[T][d_model]."""
    y = y if y is not None else _result((T, d_model), torch.float32, x, stream)
    _check(lib().qgemv_q4_0_ffn(_ptr(W_gate), _ptr(W_up), _ptr(W_down), layout, _ptr(x), _ptr(y), d_model, d_ff, T,
                                _ptr(ws), ws.numel(), _stream(stream)), "qgemv_q4_0_ffn")
    return y


def ffn_residual(W_gate, W_up, W_down, layout: int, x, residual, d_model: int, d_ff: int, T: int, ws, y=None,
                 stream=None):
    """y = residual + W_down . Q8_0(SiLU(W_gate . x) * (W_up . x)); residual may be y."""
    y = y if y is not None else _result((T, d_model), torch.float32, x, stream)
    _check(lib().qgemv_q4_0_ffn_residual(_ptr(W_gate), _ptr(W_up), _ptr(W_down), layout, _ptr(x), _ptr(residual),
                                         _ptr(y), d_model, d_ff, T, _ptr(ws), ws.numel(), _stream(stream)),
           "qgemv_q4_0_ffn_residual")
    return y


def silu_mul_q8(g, u, T: int, F: int, hq=None, stream=None):
    """Test hook: planar Q8_0 codes of SiLU(g) * u (g, u fp32 [T][F])."""
    hq = hq if hq is not None else _result(xq_bytes(T, F), torch.uint8, g, stream)
    _check(lib().qgemv_debug_silu_mul_q8(_ptr(g), _ptr(u), _ptr(hq), T, F, _stream(stream)), "qgemv_debug_silu_mul_q8")
    return hq


def q8_0_bytes(N: int, K: int) -> int:
    return 34 * N * (K // QK)


def pack_q8_0(w_ggml: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """GGML Q8_0 weights (uint8 [34 N K/32]) -> the device layout (same bytes)."""
    out = out if out is not None else _result(q8_0_bytes(N, K), torch.uint8, w_ggml, stream)
    _check(lib().qgemv_pack_q8_0(_ptr(w_ggml), _ptr(out), N, K, _stream(stream)), "qgemv_pack_q8_0")
    return out


def unpack_q8_0(w_packed: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None):
    out = out if out is not None else _result(q8_0_bytes(N, K), torch.uint8, w_packed, stream)
    _check(lib().qgemv_unpack_q8_0(_ptr(w_packed), _ptr(out), N, K, _stream(stream)), "qgemv_unpack_q8_0")
    return out


def requant_f32_q4_0(w: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 weights [N][K] -> GGML Q4_0 blocks (uint8 [18 N K/32]), GGML's q4_0 encoder."""
    out = out if out is not None else _result(q4_0_bytes(N, K), torch.uint8, w, stream)
    _check(lib().qgemv_requant_f32_q4_0(_ptr(w), _ptr(out), N, K, _stream(stream)), "qgemv_requant_f32_q4_0")
    return out


def requant_q8_0_q4_0(w_q8: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None, stream=None):
    """GGML Q8_0 weights (uint8 [34 N K/32]) -> GGML Q4_0 blocks (uint8 [18 N K/32])."""
    out = out if out is not None else _result(q4_0_bytes(N, K), torch.uint8, w_q8, stream)
    _check(lib().qgemv_requant_q8_0_q4_0(_ptr(w_q8), _ptr(out), N, K, _stream(stream)), "qgemv_requant_q8_0_q4_0")
    return out


def q8_0_workspace_bytes(N: int, K: int, T: int) -> int:
    return int(lib().qgemv_q8_0_workspace_bytes(N, K, T))


def gemv_q8_0(W, xq, N: int, K: int, T: int, ws=None, y=None, stream=None) -> torch.Tensor:
    """y[T][N] for packed Q8_0 weights and planar Q8_0 activations."""
    y = y if y is not None else _result((T, N), torch.float32, W, stream)
    _check(lib().qgemv_q8_0(_ptr(W), _ptr(xq), _ptr(y), N, K, T, _ptr(ws), 0 if ws is None else ws.numel(),
                            _stream(stream)), "qgemv_q8_0")
    return y


def seq_items(entries) -> ctypes.Array:
    """entries: iterable of (W, xq, y, N, K) with CUDA tensors."""
    entries = list(entries)
    arr = (SeqItem * len(entries))()
    for i, (W, xq, y, N, K) in enumerate(entries):
        arr[i] = SeqItem(W.data_ptr(), xq.data_ptr(), y.data_ptr(), N, K)
    return arr


def seq_workspace_bytes(items: ctypes.Array, T: int) -> int:
    return int(lib().qgemv_seq_workspace_bytes(items, len(items), T))


def gemv_seq(items: ctypes.Array, layout: int, T: int, ws, stream=None):
    _check(lib().qgemv_q4_0_seq(items, len(items), layout, T, _ptr(ws), ws.numel(), _stream(stream)),
           "qgemv_q4_0_seq")


def seq_f32_items(entries) -> ctypes.Array:
    """entries: iterable of (W, x, y, N, K) with CUDA tensors (x fp32 [T, K])."""
    entries = list(entries)
    arr = (SeqF32Item * len(entries))()
    for i, (W, x, y, N, K) in enumerate(entries):
        arr[i] = SeqF32Item(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K)
    return arr


def seq_f32_workspace_bytes(items: ctypes.Array, T: int) -> int:
    return int(lib().qgemv_seq_f32_workspace_bytes(items, len(items), T))


def gemv_seq_f32(items: ctypes.Array, layout: int, T: int, ws, stream=None):
    _check(lib().qgemv_q4_0_seq_f32(items, len(items), layout, T, _ptr(ws), ws.numel(), _stream(stream)),
           "qgemv_q4_0_seq_f32")


def seq_ep_items(entries) -> ctypes.Array:
    """entries: iterable of (W, x, y, N, K, bias, residual) with CUDA tensors;
    x planar Q8_0 or fp32 [T, K] (the call's x_f32 says which); bias [N] and
    residual [T, N] fp32 or None (residual may be y)."""
    entries = list(entries)
    arr = (SeqEpItem * len(entries))()
    for i, (W, x, y, N, K, b, r) in enumerate(entries):
        arr[i] = SeqEpItem(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K,
                           None if b is None else b.data_ptr(), None if r is None else r.data_ptr())
    return arr


def seq_ep_workspace_bytes(items: ctypes.Array, T: int, x_f32: bool = False) -> int:
    return int(lib().qgemv_seq_ep_workspace_bytes(items, len(items), T, int(x_f32)))


def gemv_seq_ep(items: ctypes.Array, layout: int, T: int, ws, x_f32: bool = False, stream=None):
    """y = W . x + bias + residual for every item, in one launch per 200 items."""
    _check(lib().qgemv_q4_0_seq_ep(items, len(items), layout, T, int(x_f32), _ptr(ws), ws.numel(), _stream(stream)),
           "qgemv_q4_0_seq_ep")


def gather_mats(entries) -> ctypes.Array:
    """entries: (W, expert_stride_bytes, xq, xq_stride_bytes, y, y_stride_floats, N, K)."""
    entries = list(entries)
    arr = (GatherMatrix * len(entries))()
    for i, (W, ws_, xq, xs, y, ys, N, K) in enumerate(entries):
        arr[i] = GatherMatrix(W.data_ptr(), ws_, xq.data_ptr(), xs, y.data_ptr(), ys, N, K)
    return arr


def gather_workspace_bytes(mats: ctypes.Array, n_ids: int, T: int) -> int:
    return int(lib().qgemv_gather_workspace_bytes(mats, len(mats), n_ids, T))


def gemv_gather(mats: ctypes.Array, ids, n_experts: int, layout: int, T: int, ws, stream=None):
    _check(lib().qgemv_q4_0_gather(mats, len(mats), _ptr(ids), ids.numel(), n_experts, layout, T, _ptr(ws),
                                   ws.numel(), _stream(stream)), "qgemv_q4_0_gather")


def gather_f32_mats(entries) -> ctypes.Array:
    """entries: (W, expert_stride_bytes, x, x_stride_bytes, y, y_stride_floats, N, K), x fp32."""
    entries = list(entries)
    arr = (GatherF32Matrix * len(entries))()
    for i, (W, ws_, x, xs, y, ys, N, K) in enumerate(entries):
        arr[i] = GatherF32Matrix(W.data_ptr(), ws_, x.data_ptr(), xs, y.data_ptr(), ys, N, K)
    return arr


def gather_f32_workspace_bytes(mats: ctypes.Array, n_ids: int, T: int) -> int:
    return int(lib().qgemv_gather_f32_workspace_bytes(mats, len(mats), n_ids, T))


def gemv_gather_f32(mats: ctypes.Array, ids, n_experts: int, layout: int, T: int, ws, stream=None):
    _check(lib().qgemv_q4_0_gather_f32(mats, len(mats), _ptr(ids), ids.numel(), n_experts, layout, T, _ptr(ws),
                                       ws.numel(), _stream(stream)), "qgemv_q4_0_gather_f32")


# ---------------------------------------------- between the GEMVs of a step

def rope_plan(rot_dim: int, base: float, layout: str = "half", scaling: str = "plain", factor: float = 1.0,
              orig_len: float = 0.0, low: float | None = None, high: float | None = None,
              mscale: float = 0.0) -> RopePlan:
    """Frequencies of rotary positions (host; keep it across calls).  low and
    high default to 1 and 4 for "bands", 1 and 32 for "yarn"; mscale 0 means
    1, for "yarn" 0.1 ln(factor) + 1."""
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"rope_plan: layout {layout!r}, scaling {scaling!r}")
    cfg = RopeConfig(rot_dim, ROPE_LAYOUTS[layout], ROPE_SCALINGS[scaling], base, factor, orig_len,
                     1.0 if low is None else low, (4.0 if scaling == "bands" else 32.0) if high is None else high, mscale)
    plan = RopePlan()
    _check(lib().qgemv_rope_init(ctypes.byref(cfg), ctypes.byref(plan)), "qgemv_rope_init")
    return plan


class _Described:
    """Has `struct`, what the C call takes."""

    @property
    def address(self) -> int:
        return ctypes.addressof(self.struct)


class KvCache(_Described):
    """A paged cache: k and v f16 or bf16 tensors [pages][page_size][heads][head_dim]
    of the same strides (elements of a head contiguous).  For pages laid out
    [pages][heads][page_size][head_dim] pass k.transpose(1, 2), v.transpose(1, 2)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.stride(3) != 1:
            raise ValueError("KvCache: k and v [pages][page_size][heads][head_dim] of one type and the same strides")
        assert k.is_cuda and v.is_cuda and k.dtype in (torch.float16, torch.bfloat16)
        self.k, self.v = k, v
        self.struct = KvCacheStruct(k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], k.shape[0], k.shape[1], k.shape[2],
                                    k.shape[3], k.stride(0), k.stride(1), k.stride(2))


def _i32(x, what: str, n: int):
    if x is None:
        return None
    if x.dtype is not torch.int32 or not x.is_cuda or not x.is_contiguous() or x.numel() < n:
        raise ValueError(f"{what}: a contiguous int32 CUDA tensor of {n}")
    return x.data_ptr()


def rope_kv(plan: RopePlan, xq, xk, xv, pos, slots=None, cache: KvCache | None = None, out=None, stream=None):
    """Rotate q [tokens][heads][head_dim] into `out` (default: a new tensor of the
    cache's type, or of q's without a cache) and k, v [tokens][kv heads][head_dim] into
    the cache rows `slots` (-1: none).  xq, or xk and xv, may be None.  Returns out.
    In this call and those below a result made by the call is `stream`'s memory, as of
    tensors made with that stream current."""
    r = (_ext or _load_binding()).rope_kv(plan, xq, xk, xv, pos, slots, None if cache is None else cache.struct, out,
                                          None if stream is None else stream.cuda_stream)
    if type(r) is int:
        _check(r, "qgemv_rope_kv")
    return r


class AttnBatch(_Described):
    """Sequences that share a prefix, over a cache (see qgemv_attn_batch): the
    tables and lengths are device tensors that later calls read again, so a
    decode loop updates them in place.  scale None: 1 / sqrt(head_dim)."""

    def __init__(self, n_seqs: int, n_q: int, n_heads: int, cache: KvCache, prefix_len: int, prefix_pages, suffix_len,
                 suffix_pages, max_suffix: int, scale: float | None = None):
        page = cache.struct.page_size
        own = 0
        if max_suffix > 0:
            if suffix_pages.dim() != 2 or suffix_pages.shape[0] != n_seqs or suffix_pages.stride(1) != 1 or \
                    suffix_pages.shape[1] * page < max_suffix or not suffix_pages.is_cuda or \
                    suffix_pages.dtype != torch.int32:
                raise ValueError("AttnBatch: suffix_pages int32 [n_seqs][pages that hold max_suffix rows]")
            own = suffix_pages.data_ptr()
        self.cache, self.tables = cache, (prefix_pages, suffix_len, suffix_pages)
        self.n_seqs, self.n_q, self.n_heads = n_seqs, n_q, n_heads
        self.struct = AttnBatchStruct(
            n_seqs, n_q, n_heads, prefix_len,
            _i32(prefix_pages, "AttnBatch: prefix_pages", -(-prefix_len // page)) if prefix_len else None,
            _i32(suffix_len, "AttnBatch: suffix_len", n_seqs), own, suffix_pages.stride(0) if own else 0, max_suffix,
            0.0 if scale is None else scale)

    def workspace_bytes(self) -> int:
        return int(lib().qgemv_attn_workspace_bytes(self.address, self.cache.address))


def attn_prefix(xq, batch: AttnBatch, ws, out=None, lse=None, stream=None):
    """Attention of q [n_seqs][n_q][heads][head_dim] (or [tokens][heads][head_dim]) over the
    batch's contexts; out (the cache's type or fp32, q's shape; default: a new tensor
    of the cache's type); lse fp32 [tokens][heads] or None."""
    r = (_ext or _load_binding()).attn_prefix(xq, batch.cache.struct, batch.struct, ws, out, lse,
                                              None if stream is None else stream.cuda_stream)
    if type(r) is int:
        _check(r, "qgemv_attn_prefix")
    return r


class LogitsRules(_Described):
    """Rules on logits of `rows` rows over `vocab` tokens (see
    qgemv_logits_spec): device tensors that later calls read again, so a
    decode loop appends to `history` and counts up `history_len` in place.
    history int64 [rows][most], history_len int32 [rows]; repetition, frequency, presence
    fp32 [rows]; bias_ids int64, bias fp32 [rows][most], bias_len int32 [rows];
    mask int32 [rows][vocab / 32 rounded up] (or one row for all)."""

    def __init__(self, rows: int, vocab: int, history=None, history_len=None, repetition=None, frequency=None,
                 presence=None, bias_ids=None, bias=None, bias_len=None, mask=None):
        self.rows, self.vocab = rows, vocab
        self.tensors = (history, history_len, repetition, frequency, presence, bias_ids, bias, bias_len, mask)

        def table(x, dtype, what, one_row=False):
            if x is None:
                return None, 0, 0
            if not x.is_cuda or x.dtype != dtype or x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1) or \
                    (x.shape[0] != rows and not (one_row and x.shape[0] == 1)):
                raise ValueError(f"LogitsRules: {what} [rows][..] {dtype}")
            return x.data_ptr(), x.stride(0) if x.shape[0] > 1 and x.shape[1] > 0 else 0, x.shape[1]

        def list_at(address, lengths):
            # A list without columns has no memory, but its rule is on: any address
            # tells the library so, and nothing is read there.
            return address if address or lengths is None else lengths.data_ptr() & ~7

        def row(x, what):
            if x is None:
                return None
            if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous() or x.numel() != rows:
                raise ValueError(f"LogitsRules: {what} fp32 [rows]")
            return x.data_ptr()

        hp, hs, hn = table(history, torch.int64, "history")
        hp = None if history is None else list_at(hp, history_len)
        ip, is_, n_ids = table(bias_ids, torch.int64, "bias_ids")
        bp, bs, bn = table(bias, torch.float32, "bias")
        ip, bp = (None if bias_ids is None else list_at(ip, bias_len)), (None if bias is None else list_at(bp, bias_len))
        mp, ms, mn = table(mask, torch.int32, "mask", one_row=True)
        if (is_, n_ids) != (bs, bn) or (mask is not None and mn * 32 < vocab):
            raise ValueError("LogitsRules: bias_ids and bias of one shape and stride; mask with a bit per token")
        self.struct = LogitsSpec(rows, vocab, hp, hs, _i32(history_len, "LogitsRules: history_len", rows), hn,
                                 row(repetition, "repetition"), row(frequency, "frequency"), row(presence, "presence"),
                                 ip, bp, bs, _i32(bias_len, "LogitsRules: bias_len", rows), bn, mp, ms)

    def workspace_bytes(self) -> int:
        return int(lib().qgemv_logits_workspace_bytes(self.address))


def logits_rules(x, rules: LogitsRules, ws, out=None, idx=None, val=None, stream=None):
    """Apply the rules to x [rows][vocab] (fp32, f16, bf16); out (None: not
    written; may be x) receives the results in x's type.  Returns each row's best
    token (int64, -1 for none) and its value (fp32); a loop that passes idx and val
    saves their allocation, 0.5 to 1 us a call."""
    r = (_ext or _load_binding()).logits_rules(x, rules.struct, ws, out, idx, val,
                                               None if stream is None else stream.cuda_stream)
    if type(r) is int:
        _check(r, "qgemv_logits_rules")
    return r


def block_isums(W, layout: int, xq, N: int, K: int, T: int, stream=None) -> torch.Tensor:
    out = _result((T, N, K // QK), torch.int32, W, stream)
    _check(lib().qgemv_debug_block_isums(_ptr(W), layout, _ptr(xq), _ptr(out), N, K, T, _stream(stream)),
           "qgemv_debug_block_isums")
    return out


def gs64_bytes(N: int, K: int) -> int:
    return int(lib().qgemv_gs64_bytes(N, K))


def pack_gs64(wq, wscale, N: int, K: int, stream=None) -> torch.Tensor:
    """Row planes (nibbles [N][K/64][32] uint8, scales [N][K/64] fp32) -> packed device layout."""
    out = _result(gs64_bytes(N, K), torch.uint8, wq, stream)
    _check(lib().qgemv_pack_gs64(_ptr(wq), _ptr(wscale), _ptr(out), N, K, _stream(stream)), "qgemv_pack_gs64")
    return out


def unpack_gs64(W, N: int, K: int, stream=None):
    wq = _result((N, K // 64, 32), torch.uint8, W, stream)
    ws = _result((N, K // 64), torch.float32, W, stream)
    _check(lib().qgemv_unpack_gs64(_ptr(W), _ptr(wq), _ptr(ws), N, K, _stream(stream)), "qgemv_unpack_gs64")
    return wq, ws


def quantize_vec_i8(x, R: int, K: int, stream=None):
    """fp32 x [R][K] -> (int8 codes [R][K], fp32 scales [R]), one scale per row."""
    q = _result((R, K), torch.int8, x, stream)
    s = _result(R, torch.float32, x, stream)
    _check(lib().qgemv_quantize_vec_i8(_ptr(x), _ptr(q), _ptr(s), R, K, _stream(stream)), "qgemv_quantize_vec_i8")
    return q, s


def quantize_vec_i8_into(x, q, s, R: int, K: int, stream=None):
    """quantize_vec_i8 into existing buffers."""
    _check(lib().qgemv_quantize_vec_i8(_ptr(x), _ptr(q), _ptr(s), R, K, _stream(stream)), "qgemv_quantize_vec_i8")


def gs64_workspace_bytes(N: int, K: int, T: int) -> int:
    return int(lib().qgemv_gs64_workspace_bytes(N, K, T))


def gemv_gs64(W, q, s, N: int, K: int, T: int, ws=None, y=None, stream=None) -> torch.Tensor:
    if y is None:
        y = _result((T, N), torch.float32, W, stream)
    _check(lib().qgemv_gs64(_ptr(W), _ptr(q), _ptr(s), _ptr(y), N, K, T, _ptr(ws) if ws is not None else None,
                            ws.numel() if ws is not None else 0, _stream(stream)), "qgemv_gs64")
    return y


def gemv_gs64_f32(W, x, N: int, K: int, T: int, ws=None, y=None, stream=None) -> torch.Tensor:
    """gs64 GEMV on fp32 activations, quantised per vector inside the launch."""
    if y is None:
        y = _result((T, N), torch.float32, W, stream)
    _check(lib().qgemv_gs64_f32(_ptr(W), _ptr(x), _ptr(y), N, K, T, _ptr(ws) if ws is not None else None,
                                ws.numel() if ws is not None else 0, _stream(stream)), "qgemv_gs64_f32")
    return y


def block_isums_tc(W, layout: int, xq, N: int, K: int, T: int, f16_image: bool, stream=None) -> torch.Tensor:
    """The tensor-core path's block sums (see qgemv_debug_block_isums_tc)."""
    out = _result((T, N, K // QK), torch.int32, W, stream)
    _check(lib().qgemv_debug_block_isums_tc(_ptr(W), layout, _ptr(xq), _ptr(out), N, K, T, 1 if f16_image else 0,
                                            _stream(stream)), "qgemv_debug_block_isums_tc")
    return out


def stream_read(src, method: int, warps: int, depth: int, stage_bytes: int, sink, stream=None):
    """Measurement hook: stream all of `src` once (see qgemv_debug_stream_read)."""
    _check(lib().qgemv_debug_stream_read(_ptr(src), src.numel() * src.element_size(), method, warps, depth,
                                         stage_bytes, _ptr(sink), _stream(stream)), "qgemv_debug_stream_read")


def set_tuning(ctas_per_sm: int = 0, waves: int = 0, mma_min_T: int = 0, ring_depth: int = 0):
    """Tuning of the streaming kernel (0 = default for each); results are unchanged."""
    _check(lib().qgemv_set_tuning(ctas_per_sm, waves, mma_min_T, ring_depth), "qgemv_set_tuning")


def set_ffn_fused(on: bool = True):
    """The decode FFN step as one fused launch where it applies (else always three launches)."""
    _check(lib().qgemv_set_ffn_fused(1 if on else 0), "qgemv_set_ffn_fused")


def set_tc_min_T(tc_min_T: int = 0):
    """Token count from which packed sequences run on the tcgen05 kernel (0 = default: never; 1..8; 9 = never)."""
    _check(lib().qgemv_set_tc_min_tokens(tc_min_T), "qgemv_set_tc_min_tokens")


def device_status() -> int:
    """Read and clear the device status word (synchronises)."""
    code = ctypes.c_int(0)
    _check(lib().qgemv_device_status(ctypes.byref(code)), "qgemv_device_status")
    return int(code.value)
