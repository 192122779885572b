"""Models that hold some linear weights in 4 bits and the others in bf16: which calls
they make (no GPU needed)."""
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

import seeded_inputs as si
from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import model as M
from test_w4_forward_host import CALLS, CTX

LINEARS = ("qkv", "o", "gate_up", "down")
BF16 = "a bf16 weight"


def forward(monkeypatch, in_4_bits):
    """Two layers; in_4_bits: (layer, weight) pairs.  The calls with their arguments."""
    calls = []
    for n in CALLS:
        monkeypatch.setattr(L, n, lambda *a, _n=n, **k: calls.append((_n, a)))
    monkeypatch.setattr(L, "decode_layers_workspace_size", lambda *a: 256)
    monkeypatch.setattr(L, "decode_layer_table", lambda rows: rows)
    layers = []
    for l in range(2):
        w = [M.W4Weight("codes", None, None, 64) if (l, n) in in_4_bits else BF16 for n in LINEARS]
        layers.append(M.LayerParams(*w, None, None, None, None))
    f = M.Qwen3Forward.__new__(M.Qwen3Forward)
    f.m = si.QWEN3_0_6B.replace(vocab=512, hidden=256, n_heads=2, n_kv_heads=1, intermediate=256, n_layers=2)
    f.p, f.kv8, f.dtype = M.ModelParams(None, layers, None), None, torch.bfloat16
    t = torch.zeros(8, 4)
    f.h = f.res = f.res2 = f.y = f.qkv = f.q = f.attn = f.act = f.logits = t
    f.next_tokens, f.err, f.cos_sin, f.workspace, f.device = t, None, None, None, "cpu"
    f.k_cache = f.v_cache = [t, t]
    f.scale, f.max_seqs, f.max_context, f.qkv_width, f._history_ready = 1.0, 8, 16, 512, True
    f.fused_decode = f.fused_qkv = f.fused_prefill = True
    f._fused = None
    f._around = lambda *a: nullcontext()
    return f, calls


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("in_4_bits", [{(l, n)} for l in range(2) for n in LINEARS]
                         + [{(0, "gate_up"), (0, "down"), (1, "gate_up"), (1, "down")}, {(1, n) for n in LINEARS}])
def test_each_weight_goes_to_its_own_product(monkeypatch, in_4_bits, decode, fused):
    f, calls = forward(monkeypatch, in_4_bits)
    f.fused_decode = f.fused_qkv = f.fused_prefill = fused
    (f.decode if decode else f.prefill)(CTX)
    for name, args in calls:
        assert name == "w4_gemm" or not any(isinstance(a, M.W4Weight) for a in args), name
    products = [name for name, _ in calls if "gemm" in name]
    assert [p == "w4_gemm" for p in products] == [(l, n) in in_4_bits for l in range(2) for n in LINEARS]
    norms = [name for name, _ in calls if "rmsnorm" in name and name != "add_rmsnorm"]
    # a norm is the prologue of the products it feeds in every layer or in none: the residual alternates between buffers
    assert norms == (["add_rmsnorm_gemm"] * 4 if decode and all(n in ("o", "down") for _, n in in_4_bits) else [])


@pytest.mark.parametrize("fused", [True, False])
def test_all_bf16_keeps_its_fused_calls(monkeypatch, fused):
    f, calls = forward(monkeypatch, set())
    f.fused_decode = fused
    f.decode(CTX)
    names = [n for n, _ in calls]
    assert not f.w4 and ("decode_layers" if fused else "add_rmsnorm_gemm") in names
    f, calls = forward(monkeypatch, set())
    f.prefill(CTX)
    assert "gemm_add_rmsnorm" in [n for n, _ in calls] or not f.prefill_fusion_ok()
