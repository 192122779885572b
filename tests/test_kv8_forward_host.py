"""Host side of the forward pass with an 8-bit KV cache: contexts that cannot be
answered are refused before any launch, and the batch descriptions fill in the
fields that such a model reads."""
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

import seeded_inputs as si
from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import model as M


@pytest.fixture
def fwd(monkeypatch):
    """A forward pass whose first library call is noted, not made."""
    calls = []

    def first(*a, **k):
        calls.append("embed_vocab")
        raise StopIteration
    monkeypatch.setattr(L, "embed_vocab", first)
    f = M.Qwen3Forward.__new__(M.Qwen3Forward)
    f.m, f.kv8 = si.QWEN3_0_6B.replace(n_layers=1), M.Kv8Config(torch.int8, 64)
    f.p = SimpleNamespace(layers=[], embed=None)
    f.h, f.err, f.fused_decode, f.dtype = torch.zeros(8, 1), None, False, torch.bfloat16
    f._around = lambda *a: nullcontext()
    f.calls = calls
    return f


def _contexts():
    i32, i64 = (lambda *n: torch.zeros(*n, dtype=torch.int32)), (lambda *n: torch.zeros(*n, dtype=torch.int64))
    pre = M.PrefillContext(i64(5), i64(5), torch.tensor([0, 5], dtype=torch.int32), i64(5), i32(1), i32(1), 5, i32(1, 2),
                           torch.tensor([5], dtype=torch.int32), 5)
    dec = M.DecodeContext(i64(2), i64(2), torch.tensor([6, 9], dtype=torch.int32), i64(2), i32(2), 9, i32(2, 2))
    return pre, dec


@pytest.mark.parametrize("decode", [False, True])
def test_contexts_that_are_refused(fwd, decode):
    """max_context 0 reads no key: a prefill left at that default would answer without its prompt."""
    for bad in ("block_table", "context_lens") + (() if decode else ("max_context=0", "max_context=-1")):
        ctx = _contexts()[decode]
        name, _, value = bad.partition("=")
        setattr(ctx, name, int(value) if value else None)
        with pytest.raises(ValueError, match=name):
            fwd.run_layers(ctx, decode)
    assert not fwd.calls       # refused before the first launch
    with pytest.raises(StopIteration):
        fwd.run_layers(_contexts()[decode], decode)
    assert fwd.calls == ["embed_vocab"]


def test_a_prefill_context_left_at_its_default_is_refused(fwd):
    pre, _ = _contexts()
    pre = M.PrefillContext(pre.ids, pre.positions, pre.cu_seqlens, pre.slot_mapping, pre.seq_base, pre.last_idx, 5,
                           block_table=pre.block_table, context_lens=pre.context_lens)
    with pytest.raises(ValueError, match="max_context"):
        fwd.prefill(pre)
    assert not fwd.calls


def test_batches_with_a_block_table():
    """Whole prompts: the cached keys are the prompts themselves; over a cached prefix the caller says how many."""
    m = si.QWEN3_0_6B
    b = si.prefill_batch(m, [7, 2, 30])
    table = torch.arange(6, dtype=torch.int32).view(3, 2)
    c = M.to_device_prefill(b, "cpu", block_table=table)
    assert c.block_table is table or torch.equal(c.block_table, table)
    assert c.context_lens.dtype == torch.int32 and c.context_lens.tolist() == [7, 2, 30] and c.max_context == 30
    c = M.to_device_prefill(b, "cpu", block_table=table, context_lens=torch.tensor([70, 2, 31], dtype=torch.int32))
    assert c.context_lens.tolist() == [70, 2, 31] and c.max_context == 70
    c = M.to_device_prefill(b, "cpu")
    assert c.block_table is None and c.context_lens is None
    d = M.to_device_decode(si.decode_batch(m, [5, 9, 3]), "cpu", block_table=table)
    assert torch.equal(d.block_table, table) and d.max_context == 9
    assert M.to_device_decode(si.decode_batch(m, [5, 9]), "cpu").block_table is None
