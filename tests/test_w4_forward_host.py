"""Host side of the forward pass with 4-bit weights: which calls a layer makes
(no GPU needed)."""
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

import seeded_inputs as si
from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import model as M

CALLS = ("embed_vocab", "w4_embed_vocab", "add_rmsnorm", "add_rmsnorm_gemm", "gemm", "w4_gemm", "attention_decode_rope",
         "qkv_norm_rope_store_kv", "attention_prefill", "lm_head", "w4_lm_head", "gemm_add_rmsnorm", "decode_layers",
         "qkv_gemm_norm_rope_store_kv")


def forward(monkeypatch, w4, table):
    calls = []
    for n in CALLS:
        monkeypatch.setattr(L, n, lambda *a, _n=n, **k: calls.append(_n))
    m = si.QWEN3_0_6B.replace(vocab=512, hidden=256, n_heads=2, n_kv_heads=1, intermediate=256, n_layers=1)
    W = M.W4Weight(None, None, None, 64)
    lin = lambda: W if w4 else None  # noqa: E731
    f = M.Qwen3Forward.__new__(M.Qwen3Forward)
    f.m, f.kv8, f.dtype = m, None, torch.bfloat16
    f.p = M.ModelParams(W if table else None, [M.LayerParams(lin(), lin(), lin(), lin(), None, None, None, None)], None)
    t = torch.zeros(8, 4)
    f.h = f.res = f.res2 = f.y = f.qkv = f.q = f.attn = f.act = f.logits = t
    f.next_tokens, f.err, f.cos_sin, f.workspace = t, None, None, None
    f.k_cache = f.v_cache = [t]
    f.scale, f.max_seqs, f.max_context, f.qkv_width, f._history_ready = 1.0, 8, 16, 512, True
    f.fused_decode = f.fused_qkv = f.fused_prefill = True     # fusions over bf16 weights: not with 4-bit ones
    f._around = lambda *a: nullcontext()
    return f, calls


CTX = SimpleNamespace(ids=torch.zeros(3), n_tokens=3, positions=None, slot_mapping=None, cu_seqlens=None, seq_base=None,
                      max_seqlen=3, context_lens=None, max_context=3, last_idx=torch.zeros(3))


@pytest.mark.parametrize("table", [False, True])
@pytest.mark.parametrize("decode", [False, True])
def test_calls_of_a_4bit_layer(monkeypatch, decode, table):
    f, calls = forward(monkeypatch, True, table)
    (f.decode if decode else f.prefill)(CTX)
    attention = ["attention_decode_rope"] if decode else ["qkv_norm_rope_store_kv", "attention_prefill"]
    assert calls == ["w4_embed_vocab" if table else "embed_vocab", "add_rmsnorm", "w4_gemm"] + attention + [
        "w4_gemm", "add_rmsnorm", "w4_gemm", "w4_gemm", "add_rmsnorm", "w4_lm_head" if table else "lm_head"]


def test_a_bf16_layer_makes_none_of_them(monkeypatch):
    f, calls = forward(monkeypatch, False, False)
    f.fused_decode = False
    f.decode(CTX)
    assert not any(c.startswith("w4") for c in calls) and "add_rmsnorm_gemm" in calls
