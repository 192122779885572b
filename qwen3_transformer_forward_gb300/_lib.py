"""ctypes binding of libqw (the C ABI declared in include/qw.h).

Argument marshalling only: every wrapper checks nothing numerical, passes
device pointers, sizes and the current CUDA stream, and raises QwError on a
non-zero status.  There is no fallback: without the built library on a
CUDA device every call fails loudly.
"""
from __future__ import annotations

import ctypes as C
import os
from pathlib import Path
from typing import Optional

import torch

_LIB_PATH = Path(__file__).resolve().parent / "libqw.so"
_lib = None

QW_OK, QW_ERR_INVALID_ARG, QW_ERR_SHAPE, QW_ERR_DTYPE, QW_ERR_CUDA, QW_ERR_TIMEOUT, QW_ERR_WORKSPACE = range(7)
QW_BF16, QW_F32, QW_I8, QW_E4M3 = range(4)
QW_GEMM_COLUMN, QW_GEMM_ROW_REDUCE = 0, 1
QW_EPI_NONE, QW_EPI_SILU_MUL = 0, 1

_p, _i64, _i32, _f32, _f64, _sz = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_double, C.c_size_t

# name -> (restype, argtypes); mirrors include/qw.h
SIGNATURES = {
    "qw_abi_version": (C.c_int, []),
    "qw_last_error_string": (C.c_char_p, []),
    "qw_device_error": (C.c_int, [_p]),
    "qw_embed_vocab": (C.c_int, [_p, _i64, _p, _i64, _i64, _i32, _p, _p, _i32, _p]),
    "qw_add_rmsnorm": (C.c_int, [_p, _p, _p, _p, _f32, _i64, _i64, _p, _i32, _p]),
    "qw_rope_cos_sin_table": (C.c_int, [_p, _i64, _i32, _f64]),
    "qw_qkv_norm_rope_store_kv": (C.c_int, [_p, _i64, _i32, _i32, _i32, _i32, _p, _p, _i64, _p, _p, _f32, _p, _p,
                                            _p, _i64, _p, _p, _i32, _p]),
    "qw_gemm_add_rmsnorm": (C.c_int, [_p, _p, _i64, _i64, _i64, _i32, _p, _p, _f32, _p, _i32, _p]),
    "qw_qkv_gemm_norm_rope_store_kv": (C.c_int, [_p, _p, _i64, _i64, _i32, _i32, _i32, _i32, _p, _p, _i64, _p, _p,
                                                 _f32, _p, _p, _p, _i64, _p, _p, _i32, _p]),
    "qw_attention_prefill": (C.c_int, [_p, _p, _p, _i64, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _f32, _p, _i32, _p]),
    "qw_attention_decode": (C.c_int, [_p, _p, _p, _i64, _p, _p, _i32, _i32, _i32, _i32, _i32, _f32, _p, _p, _sz,
                                      _i32, _i32, _p]),
    "qw_attention_decode_workspace_size": (C.c_size_t, [_i32, _i32, _i32, _i32]),
    "qw_attention_decode_paged": (C.c_int, [_p, _p, _p, _i64, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32,
                                            _p, _p, _sz, _i32, _i32, _p]),
    "qw_attention_prefill_paged": (C.c_int, [_p, _p, _p, _i64, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                             _f32, _p, _i32, _p]),
    "qw_kv8_append": (C.c_int, [_p, _i64, _i32, _i32, _i32, _i32, _p, _p, _i64, _p, _p, _f32, _p, _p, _p, _i32, _i32, _i32,
                                _p, _p, _p, _p, _i64, _i32, _p, _p, _i32, _i32, _p]),
    "qw_kv8_read": (C.c_int, [_p, _p, _p, _p, _i64, _i32, _i32, _i32, _p, _i64, _p, _p, _p, _i32, _i32, _p]),
    "qw_attention_decode_kv8": (C.c_int, [_p, _p, _p, _p, _p, _i64, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                          _f32, _i32, _i32, _p, _p, _sz, _i32, _i32, _p]),
    "qw_attention_decode_kv8_workspace_size": (C.c_size_t, [_i32, _i32, _i32, _i32]),
    "qw_attention_prefill_kv8": (C.c_int, [_p, _p, _p, _p, _p, _i64, _i32, _p, _p, _p, _i32, _i32, _i32, _i64, _i32, _i32,
                                           _i32, _i32, _i32, _f32, _i32, _i32, _p, _p, _sz, _i32, _i32, _p]),
    "qw_attention_prefill_kv8_workspace_size": (C.c_size_t, [_i32, _i64, _i32, _i32, _i32, _i32]),
    "qw_attention_decode_rope": (C.c_int, [_p, _i32, _i32, _i32, _i32, _p, _p, _i64, _p, _p, _f32, _p, _p, _p, _i64,
                                           _p, _p, _p, _i32, _i32, _f32, _p, _p, _sz, _i32, _i32, _p]),
    "qw_attention_decode_static": (C.c_int, [_p, _p, _p, _i64, _p, _p, _i32, _i32, _i32, _i32, _i32, _f32, _p, _i32,
                                             _p]),
    "qw_attention_decode_static_scratch_bytes": (C.c_size_t, []),
    "qw_gemm": (C.c_int, [_p, _p, _p, _i64, _i64, _i64, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "qw_gemm_workspace_size": (C.c_size_t, [_i64, _i64, _i64, _i32, _i32, _i32, _i32]),
    "qw_silu_mul": (C.c_int, [_p, _p, _i64, _i64, _i32, _i32, _p]),
    "qw_lm_head": (C.c_int, [_p, _i64, _p, _i64, _p, _i64, _i64, _i32, _p, _p, _p, _sz, _i32, _p]),
    "qw_lm_head_workspace_size": (C.c_size_t, [_i64, _i64, _i64, _i32, _i32]),
    "qw_argmax": (C.c_int, [_p, _i64, _i64, _p, _i32, _p]),
    "qw_sample": (C.c_int, [_p, _i64, _i64, _p, _p, _p, _p, _p, _sz, _i32, _p]),
    "qw_sample_workspace_size": (C.c_size_t, [_i64, _i64]),
    "qw_selftest_wait_timeout": (C.c_int, [_p]),
    "qw_add_rmsnorm_gemm": (C.c_int, [_p, _p, _p, _p, _f32, _p, _p, _i64, _i64, _i64, _i32, _i32, _i32, _p]),
    "qw_decode_layers": (C.c_int, [_p, _i32, _p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _p,
                                   _i64, _i64, _f32, _f32, _p, _p, _p, _p, _sz, _p]),
    "qw_decode_layers_workspace_size": (C.c_size_t, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32]),
}

# field order of qw_decode_layer (include/qw.h)
DECODE_LAYER_FIELDS = ("input_layernorm", "qkv", "q_norm", "k_norm", "o_proj", "post_attention_layernorm", "gate_up",
                       "down", "k_cache", "v_cache")


class QwError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[qw status {code}] {msg}")
        self.code = code


def lib_path() -> Path:
    return _LIB_PATH


def load(path: Optional[os.PathLike] = None):
    """Loads libqw.so (built in-tree by build.py) and declares every signature."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path is not None else _LIB_PATH
    if not p.exists():
        raise QwError(-1, f"{p} is missing: build it with qwen3_transformer_forward_gb300.build.build()")
    lib = C.CDLL(str(p))
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(rc: int):
    if rc != QW_OK:
        raise QwError(rc, load().qw_last_error_string().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return t.data_ptr()


def _dev_ptr(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise QwError(QW_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise QwError(QW_ERR_INVALID_ARG, f"{name} must be contiguous")
    return t.data_ptr()


# torch.cuda.current_stream() builds a Stream object: 2.9 us of a call of about 10, the raw handle 0.3
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return QW_BF16
    if t == torch.float32:
        return QW_F32
    raise QwError(QW_ERR_DTYPE, f"unsupported dtype {t}")


# ----------------------------------------------------------------------------
# thin wrappers (same names as the C entry points, without the qw_ prefix)
# ----------------------------------------------------------------------------

def abi_version() -> int:
    return load().qw_abi_version()


def device_error(stream=None):
    _check(load().qw_device_error(_stream(stream)))


def embed_vocab(ids, table, tp, out, err_count=None, stream=None):
    T, H = out.shape
    _check(load().qw_embed_vocab(_dev_ptr(ids, "ids"), T, _dev_ptr(table, "table"), table.shape[0], H, tp,
                                 _dev_ptr(out, "out"), _dev_ptr(err_count, "err_count"), dtype_code(table.dtype),
                                 _stream(stream)))


def add_rmsnorm(x, residual_in, residual_out, gamma, eps, y, stream=None):
    T, H = x.shape
    _check(load().qw_add_rmsnorm(_dev_ptr(x, "x"), _dev_ptr(residual_in, "residual_in"),
                                 _dev_ptr(residual_out, "residual_out"), _dev_ptr(gamma, "gamma"), eps, T, H,
                                 _dev_ptr(y, "y"), dtype_code(x.dtype), _stream(stream)))


def rope_cos_sin_table(max_position: int, rotary_dim: int, theta: float) -> torch.Tensor:
    """Host-side table [max_position, rotary_dim] (float32, CPU tensor)."""
    out = torch.empty((max_position, rotary_dim), dtype=torch.float32)
    _check(load().qw_rope_cos_sin_table(out.data_ptr(), max_position, rotary_dim, theta))
    return out


def qkv_norm_rope_store_kv(qkv, n_heads, n_kv_heads, head_dim, tp, positions, cos_sin, q_gamma, k_gamma, eps,
                           slot_mapping, k_cache, v_cache, q_out, err_count=None, stream=None):
    T = qkv.shape[0]
    _check(load().qw_qkv_norm_rope_store_kv(
        _dev_ptr(qkv, "qkv"), T, n_heads, n_kv_heads, head_dim, tp, _dev_ptr(positions, "positions"),
        _dev_ptr(cos_sin, "cos_sin"), cos_sin.shape[0], _dev_ptr(q_gamma, "q_gamma"), _dev_ptr(k_gamma, "k_gamma"),
        eps, _dev_ptr(slot_mapping, "slot_mapping"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
        k_cache.shape[0], _dev_ptr(q_out, "q_out"), _dev_ptr(err_count, "err_count"), dtype_code(qkv.dtype),
        _stream(stream)))


def gemm_add_rmsnorm(A, W, residual, gamma, eps, y, tp, stream=None):
    """Row-parallel GEMM whose output is added to the residual in place, then RMSNorm into y (qw_gemm_add_rmsnorm)."""
    M, K = A.shape
    N = residual.shape[1]
    _check(load().qw_gemm_add_rmsnorm(_dev_ptr(A, "A"), _dev_ptr(W, "W"), M, N, K, tp, _dev_ptr(residual, "residual"),
                                      _dev_ptr(gamma, "gamma"), eps, _dev_ptr(y, "y"), dtype_code(A.dtype),
                                      _stream(stream)))


def qkv_gemm_norm_rope_store_kv(A, W, n_heads, n_kv_heads, head_dim, tp, positions, cos_sin, q_gamma, k_gamma, eps,
                                slot_mapping, k_cache, v_cache, q_out, err_count=None, stream=None):
    """Merged QKV GEMM with QK-RMSNorm + RoPE + KV store as its epilogue (qw_qkv_gemm_norm_rope_store_kv)."""
    T, H = A.shape
    _check(load().qw_qkv_gemm_norm_rope_store_kv(
        _dev_ptr(A, "A"), _dev_ptr(W, "W"), T, H, n_heads, n_kv_heads, head_dim, tp, _dev_ptr(positions, "positions"),
        _dev_ptr(cos_sin, "cos_sin"), cos_sin.shape[0], _dev_ptr(q_gamma, "q_gamma"), _dev_ptr(k_gamma, "k_gamma"), eps,
        _dev_ptr(slot_mapping, "slot_mapping"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
        k_cache.shape[0], _dev_ptr(q_out, "q_out"), _dev_ptr(err_count, "err_count"), dtype_code(A.dtype),
        _stream(stream)))


def attention_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k, seq_base, max_seqlen_q, n_heads, n_kv_heads, head_dim,
                      scale, out, stream=None):
    n_seqs = cu_seqlens_q.shape[0] - 1
    _check(load().qw_attention_prefill(
        _dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), k.shape[0], _dev_ptr(cu_seqlens_q, "cu_seqlens_q"),
        _dev_ptr(cu_seqlens_k, "cu_seqlens_k"), _dev_ptr(seq_base, "seq_base"), n_seqs, max_seqlen_q, n_heads,
        n_kv_heads, head_dim, scale, _dev_ptr(out, "out"), dtype_code(q.dtype), _stream(stream)))


def attention_decode_workspace_size(B, max_context, n_heads, head_dim) -> int:
    return load().qw_attention_decode_workspace_size(B, max_context, n_heads, head_dim)


QW_DECODE_HISTORY_READY = 1


def attention_decode(q, k_cache, v_cache, context_lens, seq_base, max_context, n_heads, n_kv_heads, head_dim, scale,
                     out, workspace=None, stream=None, history_ready=False):
    """history_ready: the previous kernel on the stream writes only q and each sequence's last cache row
    (see QW_DECODE_HISTORY_READY in qw.h)."""
    B = q.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_attention_decode(
        _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), k_cache.shape[0],
        _dev_ptr(context_lens, "context_lens"), _dev_ptr(seq_base, "seq_base"), B, max_context, n_heads, n_kv_heads,
        head_dim, scale, _dev_ptr(out, "out"), _dev_ptr(workspace, "workspace"), ws_bytes, dtype_code(q.dtype),
        QW_DECODE_HISTORY_READY if history_ready else 0, _stream(stream)))


def attention_decode_rope(qkv, n_heads, n_kv_heads, head_dim, tp, positions, cos_sin, q_gamma, k_gamma, eps,
                          slot_mapping, k_cache, v_cache, err_count, context_lens, seq_base, max_context, scale, out,
                          workspace, stream=None, history_ready=False):
    """QK-norm + RoPE + KV store of one decode token per sequence, then decode attention, in one launch."""
    B = qkv.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_attention_decode_rope(
        _dev_ptr(qkv, "qkv"), n_heads, n_kv_heads, head_dim, tp, _dev_ptr(positions, "positions"),
        _dev_ptr(cos_sin, "cos_sin"), cos_sin.shape[0], _dev_ptr(q_gamma, "q_gamma"), _dev_ptr(k_gamma, "k_gamma"),
        eps, _dev_ptr(slot_mapping, "slot_mapping"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"),
        k_cache.shape[0], _dev_ptr(err_count, "err_count"), _dev_ptr(context_lens, "context_lens"),
        _dev_ptr(seq_base, "seq_base"), B, max_context, scale, _dev_ptr(out, "out"), _dev_ptr(workspace, "workspace"),
        ws_bytes, dtype_code(qkv.dtype), QW_DECODE_HISTORY_READY if history_ready else 0, _stream(stream)))


def attention_decode_paged(q, k_cache, v_cache, context_lens, block_table, block_size, max_context, n_heads,
                           n_kv_heads, head_dim, scale, out, workspace, stream=None, history_ready=False):
    """Decode attention over a paged cache: block_table int32 [B, max_blocks]."""
    B = q.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_attention_decode_paged(
        _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), k_cache.shape[0],
        _dev_ptr(context_lens, "context_lens"), _dev_ptr(block_table, "block_table"), block_table.shape[1],
        block_size, B, max_context, n_heads, n_kv_heads, head_dim, scale, _dev_ptr(out, "out"),
        _dev_ptr(workspace, "workspace"), ws_bytes, dtype_code(q.dtype), QW_DECODE_HISTORY_READY if history_ready else 0,
        _stream(stream)))


def attention_prefill_paged(q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_table, block_size, max_seqlen_q,
                            n_heads, n_kv_heads, head_dim, scale, out, stream=None):
    """Causal prefill attention with every key read from a paged cache (prefix-cache prefill)."""
    n_seqs = cu_seqlens_q.shape[0] - 1
    _check(load().qw_attention_prefill_paged(
        _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), k_cache.shape[0],
        _dev_ptr(cu_seqlens_q, "cu_seqlens_q"), _dev_ptr(cu_seqlens_k, "cu_seqlens_k"),
        _dev_ptr(block_table, "block_table"), block_table.shape[1], block_size, n_seqs, max_seqlen_q, n_heads,
        n_kv_heads, head_dim, scale, _dev_ptr(out, "out"), dtype_code(q.dtype), _stream(stream)))


_KV_CODES = {torch.int8: QW_I8, torch.float8_e4m3fn: QW_E4M3}


def kv_code(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
            scale_block: int) -> int:
    """kv_dtype of an 8-bit cache; the library sees pointers only, so the tensors' types and sizes are checked here."""
    kind = k_cache.dtype
    code = _KV_CODES.get(kind)
    if code is None or v_cache.dtype is not kind:
        raise QwError(QW_ERR_DTYPE, f"caches must both be int8 or float8_e4m3fn, not {k_cache.dtype} and {v_cache.dtype}")
    if k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32:
        raise QwError(QW_ERR_DTYPE, "scales must be float32")
    shape = k_cache.shape
    want = (shape[0] // scale_block if scale_block > 0 else -1, shape[1])
    if v_cache.shape != shape or k_scale.shape != want or v_scale.shape != want:
        raise QwError(QW_ERR_SHAPE, f"caches {tuple(shape)} and {tuple(v_cache.shape)} need scales of {want}, not "
                                    f"{tuple(k_scale.shape)} and {tuple(v_scale.shape)}")
    return code


def _kv8_check(k_cache, n_kv_heads, head_dim, n_seqs, context_lens, block_table, x, y, x_heads, y_heads):
    """Types and sizes of a call on the 8-bit cache: x (tokens of x_heads heads) goes in, y (y_heads) comes out."""
    _, nkv, hd = k_cache.shape
    if nkv != n_kv_heads or hd != head_dim:
        raise QwError(QW_ERR_SHAPE, f"the cache holds {(nkv, hd)} per token, not {(n_kv_heads, head_dim)}")
    if context_lens.dtype is not torch.int32 or block_table.dtype is not torch.int32:
        raise QwError(QW_ERR_DTYPE, f"context_lens and block_table must be int32, not {context_lens.dtype}, {block_table.dtype}")
    rows, tokens, dtype = block_table.shape[0], x.shape[0], x.dtype
    if context_lens.numel() < n_seqs or rows < n_seqs:
        raise QwError(QW_ERR_SHAPE, f"{context_lens.numel()} context_lens and {rows} block table rows for {n_seqs} sequences")
    if y.dtype is not dtype:
        raise QwError(QW_ERR_DTYPE, f"the output's type {y.dtype} is not the input's, {dtype}")
    if x.numel() != tokens * x_heads * hd or y.numel() < tokens * y_heads * hd:
        raise QwError(QW_ERR_SHAPE, f"{tuple(x.shape)} in and {tuple(y.shape)} out are not {tokens} tokens of {x_heads} and "
                                    f"{y_heads} heads")


def _kv8_err(err_count):
    if err_count is None:
        return
    if err_count.dtype is not torch.int32:
        raise QwError(QW_ERR_DTYPE, f"err_count must be int32, not {err_count.dtype}")
    if err_count.numel() == 0:
        raise QwError(QW_ERR_SHAPE, "err_count is empty")


def _kv8_seqs(cu_seqlens_q) -> int:
    if cu_seqlens_q.dtype is not torch.int32:
        raise QwError(QW_ERR_DTYPE, f"cu_seqlens_q must be int32, not {cu_seqlens_q.dtype}")
    return cu_seqlens_q.shape[0] - 1


def kv8_append(qkv, n_heads, n_kv_heads, head_dim, tp, positions, cos_sin, q_gamma, k_gamma, eps, cu_seqlens_q,
               context_lens, block_table, block_size, k_cache, v_cache, k_scale, v_scale, scale_block, q_out,
               err_count=None, stream=None):
    """QK-norm + RoPE, q out, k and v quantised into an 8-bit paged cache; cu_seqlens_q None: one token per sequence."""
    kv = kv_code(k_cache, v_cache, k_scale, v_scale, scale_block)
    n_seqs = context_lens.shape[0] if cu_seqlens_q is None else _kv8_seqs(cu_seqlens_q)
    _kv8_check(k_cache, n_kv_heads, head_dim, n_seqs, context_lens, block_table, qkv, q_out, n_heads + 2 * n_kv_heads,
               n_heads)
    if positions.dtype != torch.int64 or cos_sin.dtype != torch.float32 or q_gamma.dtype != qkv.dtype or k_gamma.dtype != qkv.dtype:
        raise QwError(QW_ERR_DTYPE, "positions must be int64, cos_sin float32, gammas of qkv's type")
    if positions.numel() < qkv.shape[0] or cos_sin.numel() != cos_sin.shape[0] * head_dim:
        raise QwError(QW_ERR_SHAPE, f"{positions.numel()} positions and cos_sin {tuple(cos_sin.shape)} for {qkv.shape[0]} tokens")
    if q_gamma.numel() < head_dim or k_gamma.numel() < head_dim:
        raise QwError(QW_ERR_SHAPE, f"gammas of {q_gamma.numel()} and {k_gamma.numel()} weights for heads of {head_dim}")
    _kv8_err(err_count)
    _check(load().qw_kv8_append(
        _dev_ptr(qkv, "qkv"), qkv.shape[0], n_heads, n_kv_heads, head_dim, tp, _dev_ptr(positions, "positions"),
        _dev_ptr(cos_sin, "cos_sin"), cos_sin.shape[0], _dev_ptr(q_gamma, "q_gamma"), _dev_ptr(k_gamma, "k_gamma"), eps,
        _dev_ptr(cu_seqlens_q, "cu_seqlens_q"), _dev_ptr(context_lens, "context_lens"),
        _dev_ptr(block_table, "block_table"), block_table.shape[1], block_size, n_seqs,
        _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), _dev_ptr(k_scale, "k_scale"),
        _dev_ptr(v_scale, "v_scale"), k_cache.shape[0], scale_block, _dev_ptr(q_out, "q_out"),
        _dev_ptr(err_count, "err_count"), dtype_code(qkv.dtype), kv, _stream(stream)))


def kv8_read(k_cache, v_cache, k_scale, v_scale, scale_block, rows, k_out, v_out, err_count=None, stream=None):
    """Values of the 8-bit cache's rows (int64 [n]); k_out or v_out may be None."""
    kv = kv_code(k_cache, v_cache, k_scale, v_scale, scale_block)
    n_slots, nkv, hd = k_cache.shape
    n, out = rows.shape[0], k_out if k_out is not None else v_out
    if rows.dtype is not torch.int64 or (v_out is not None and v_out.dtype is not out.dtype):
        raise QwError(QW_ERR_DTYPE, "rows must be int64, k_out and v_out of one type")
    _kv8_err(err_count)
    need = n * nkv * hd
    if (k_out is not None and k_out.numel() < need) or (v_out is not None and v_out.numel() < need):
        raise QwError(QW_ERR_SHAPE, f"outputs are smaller than {n} rows of {(nkv, hd)}")
    _check(load().qw_kv8_read(
        _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), _dev_ptr(k_scale, "k_scale"),
        _dev_ptr(v_scale, "v_scale"), n_slots, scale_block, nkv, hd, _dev_ptr(rows, "rows"), n, _dev_ptr(k_out, "k_out"),
        _dev_ptr(v_out, "v_out"), _dev_ptr(err_count, "err_count"), dtype_code(out.dtype) if out is not None else QW_BF16, kv,
        _stream(stream)))


def attention_decode_kv8_workspace_size(B, max_context, n_heads, n_kv_heads) -> int:
    return load().qw_attention_decode_kv8_workspace_size(B, max_context, n_heads, n_kv_heads)


def attention_decode_kv8(q, k_cache, v_cache, k_scale, v_scale, scale_block, context_lens, block_table, block_size,
                         max_context, n_heads, n_kv_heads, head_dim, scale, out, workspace, window=0, n_sink=0,
                         stream=None):
    """Decode attention over an 8-bit paged cache; window > 0: the last `window` keys and the first n_sink are seen."""
    kv = kv_code(k_cache, v_cache, k_scale, v_scale, scale_block)
    _kv8_check(k_cache, n_kv_heads, head_dim, q.shape[0], context_lens, block_table, q, out, n_heads, n_heads)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_attention_decode_kv8(
        _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), _dev_ptr(k_scale, "k_scale"),
        _dev_ptr(v_scale, "v_scale"), k_cache.shape[0], scale_block, _dev_ptr(context_lens, "context_lens"),
        _dev_ptr(block_table, "block_table"), block_table.shape[1], block_size, q.shape[0], max_context, n_heads,
        n_kv_heads, head_dim, scale, window, n_sink, _dev_ptr(out, "out"), _dev_ptr(workspace, "workspace"), ws_bytes,
        dtype_code(q.dtype), kv, _stream(stream)))


# the largest workspace that attention_prefill_kv8 asks for
ATTENTION_PREFILL_KV8_WORKSPACE_MAX = 64 * 1024 + 152 * 256 * 130 * 4


def attention_prefill_kv8_workspace_size(n_seqs, total_q, max_seqlen_q, max_context, n_heads, n_kv_heads) -> int:
    return load().qw_attention_prefill_kv8_workspace_size(n_seqs, total_q, max_seqlen_q, max_context, n_heads, n_kv_heads)


def attention_prefill_kv8(q, k_cache, v_cache, k_scale, v_scale, scale_block, cu_seqlens_q, context_lens, block_table,
                          block_size, max_seqlen_q, max_context, n_heads, n_kv_heads, head_dim, scale, out, workspace,
                          window=0, n_sink=0, stream=None):
    """Causal attention of packed new tokens over an 8-bit paged cache that holds their k and v already."""
    kv = kv_code(k_cache, v_cache, k_scale, v_scale, scale_block)
    n_seqs = _kv8_seqs(cu_seqlens_q)
    _kv8_check(k_cache, n_kv_heads, head_dim, n_seqs, context_lens, block_table, q, out, n_heads, n_heads)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_attention_prefill_kv8(
        _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), _dev_ptr(k_scale, "k_scale"),
        _dev_ptr(v_scale, "v_scale"), k_cache.shape[0], scale_block, _dev_ptr(cu_seqlens_q, "cu_seqlens_q"),
        _dev_ptr(context_lens, "context_lens"), _dev_ptr(block_table, "block_table"), block_table.shape[1], block_size,
        n_seqs, q.shape[0], max_seqlen_q, max_context, n_heads, n_kv_heads, head_dim, scale, window,
        n_sink, _dev_ptr(out, "out"), _dev_ptr(workspace, "workspace"), ws_bytes, dtype_code(q.dtype), kv,
        _stream(stream)))


def attention_decode_static(q, k_cache, v_cache, context_lens, seq_base, max_context, n_heads, n_kv_heads,
                            head_dim, scale, out, stream=None):
    """Decode attention whose split-KV scratch is the library's fixed device array (no workspace)."""
    B = q.shape[0]
    _check(load().qw_attention_decode_static(
        _dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"), _dev_ptr(v_cache, "v_cache"), k_cache.shape[0],
        _dev_ptr(context_lens, "context_lens"), _dev_ptr(seq_base, "seq_base"), B, max_context, n_heads, n_kv_heads,
        head_dim, scale, _dev_ptr(out, "out"), dtype_code(q.dtype), _stream(stream)))


def attention_decode_static_scratch_bytes() -> int:
    return load().qw_attention_decode_static_scratch_bytes()


def gemm_workspace_size(M, N, K, tp, mode, epilogue, dtype) -> int:
    return load().qw_gemm_workspace_size(M, N, K, tp, mode, epilogue, dtype_code(dtype))


def gemm(A, W, C_out, N, tp=1, mode=QW_GEMM_COLUMN, epilogue=QW_EPI_NONE, workspace=None, stream=None):
    M, K = A.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_gemm(_dev_ptr(A, "A"), _dev_ptr(W, "W"), _dev_ptr(C_out, "C"), M, N, K, tp, mode, epilogue,
                          _dev_ptr(workspace, "workspace"), ws_bytes, dtype_code(A.dtype), _stream(stream)))


def silu_mul(x, out, tp, stream=None):
    T, I = out.shape
    _check(load().qw_silu_mul(_dev_ptr(x, "x"), _dev_ptr(out, "out"), T, I, tp, dtype_code(x.dtype),
                              _stream(stream)))


def lm_head_workspace_size(n_out, V, H, tp, dtype) -> int:
    return load().qw_lm_head_workspace_size(n_out, V, H, tp, dtype_code(dtype))


def lm_head(hidden, last_idx, n_out, table, tp, logits, next_tokens=None, workspace=None, stream=None):
    T, H = hidden.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().qw_lm_head(_dev_ptr(hidden, "hidden"), T, _dev_ptr(last_idx, "last_idx"), n_out,
                             _dev_ptr(table, "table"), table.shape[0], H, tp, _dev_ptr(logits, "logits"),
                             _dev_ptr(next_tokens, "next_tokens"), _dev_ptr(workspace, "workspace"), ws_bytes,
                             dtype_code(hidden.dtype), _stream(stream)))


def argmax(logits, out, stream=None):
    M, V = logits.shape
    _check(load().qw_argmax(_dev_ptr(logits, "logits"), M, V, _dev_ptr(out, "out"), dtype_code(logits.dtype),
                            _stream(stream)))


def sample_workspace_size(B, V) -> int:
    return load().qw_sample_workspace_size(B, V)


def sample(logits, temperature, top_p, uniforms, out, workspace, stream=None):
    """Temperature / top-p sampling (qw_sample): one token per logits row into out."""
    B, V = logits.shape
    _check(load().qw_sample(_dev_ptr(logits, "logits"), B, V, _dev_ptr(temperature, "temperature"),
                            _dev_ptr(top_p, "top_p"), _dev_ptr(uniforms, "uniforms"), _dev_ptr(out, "out"),
                            _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                            dtype_code(logits.dtype), _stream(stream)))


def selftest_wait_timeout(stream=None):
    """Launches a bounded wait that runs out; the next device_error() raises QW_ERR_TIMEOUT."""
    _check(load().qw_selftest_wait_timeout(_stream(stream)))


class DecodeLayer(C.Structure):
    """qw_decode_layer (include/qw.h): one layer's device pointers."""
    _fields_ = [(f, C.c_void_p) for f in DECODE_LAYER_FIELDS]


def decode_layer_table(layers):
    """Host array of qw_decode_layer records: one dict of CUDA tensors per
    layer (keys DECODE_LAYER_FIELDS).  The tensors must outlive its use."""
    arr = (DecodeLayer * len(layers))()
    for i, lw in enumerate(layers):
        for f in DECODE_LAYER_FIELDS:
            setattr(arr[i], f, _dev_ptr(lw[f], f))
    return arr


def decode_layers_workspace_size(n_layers, B, H, n_heads, n_kv_heads, head_dim, intermediate, tp, max_context) -> int:
    return load().qw_decode_layers_workspace_size(n_layers, B, H, n_heads, n_kv_heads, head_dim, intermediate, tp,
                                                  max_context)


def decode_layers(table, n_layers, x, positions, slot_mapping, context_lens, seq_base, max_context, n_heads,
                  n_kv_heads, head_dim, intermediate, tp, cos_sin, num_slots, eps, scale, final_norm, out,
                  workspace, err_count=None, stream=None):
    B, H = x.shape
    _check(load().qw_decode_layers(
        C.cast(table, C.c_void_p), n_layers, _dev_ptr(x, "x"), _dev_ptr(positions, "positions"),
        _dev_ptr(slot_mapping, "slot_mapping"), _dev_ptr(context_lens, "context_lens"), _dev_ptr(seq_base, "seq_base"),
        B, max_context, H, n_heads, n_kv_heads, head_dim, intermediate, tp, _dev_ptr(cos_sin, "cos_sin"),
        cos_sin.shape[0], num_slots, eps, scale, _dev_ptr(final_norm, "final_norm"), _dev_ptr(out, "out"),
        _dev_ptr(err_count, "err_count"), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def add_rmsnorm_gemm(x, residual_in, residual_out, gamma, eps, W, C, N, tp, epilogue=QW_EPI_NONE, stream=None):
    """C = RMSNorm(x + residual_in) * gamma @ W^T for few tokens; residual_out = x + residual_in."""
    M, K = x.shape
    _check(load().qw_add_rmsnorm_gemm(
        _dev_ptr(x, "x"), _dev_ptr(residual_in, "residual_in"), _dev_ptr(residual_out, "residual_out"),
        _dev_ptr(gamma, "gamma"), eps, _dev_ptr(W, "W"), _dev_ptr(C, "C"), M, N, K, tp, epilogue,
        dtype_code(x.dtype), _stream(stream)))
