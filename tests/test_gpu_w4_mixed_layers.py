"""The forward pass with some linear weights in 4 bits and the others in bf16, against
the bf16 pass over the weights that the codes stand for; bounds as in
test_gpu_w4_model.py (0.02 of the logits' norm for one layer, 0.03 for two)."""
import dataclasses

import pytest
import torch

import seeded_inputs as si
from test_gpu_kv8_model import _contexts
from test_gpu_w4_model import M, run, values  # noqa: F401

pytestmark = pytest.mark.gpu

LINEARS = ("qkv", "o", "gate_up", "down")


@pytest.mark.parametrize("table", [False, True])
@pytest.mark.parametrize("in_4_bits", [{(0, "gate_up"), (1, "gate_up")}, {(0, "down"), (1, "o")}, {(1, "qkv")},
                                       {(1, n) for n in LINEARS}, {(0, n) for n in LINEARS}, set()])
def test_mixed_layers(M, in_4_bits, table):  # noqa: F811
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=2, tp=2, gamma_sigma=0.1)
    lens, steps = [150, 3, 64], 3
    pre, dec, _, slots = _contexts(M, m, lens, steps)
    p, cfg = M.load_params(m), M.W4Config(group=64)
    q = M.ModelParams(M.w4_weight(p.embed, cfg) if table else p.embed, [
        dataclasses.replace(a, **{n: M.w4_weight(getattr(a, n), cfg) for n in LINEARS if (l, n) in in_4_bits})
        for l, a in enumerate(p.layers)], p.final_norm)
    ref = M.ModelParams(values(M, q.embed, p.embed) if table else p.embed, [
        dataclasses.replace(a, **{n: values(M, getattr(b, n), getattr(a, n)) for n in LINEARS if (l, n) in in_4_bits})
        for l, (a, b) in enumerate(zip(p.layers, q.layers))], p.final_norm)
    args = dict(max_tokens=sum(lens), max_seqs=3, max_context=max(lens) + steps, num_slots=slots)
    f = M.Qwen3Forward(m, q, **args)
    got, want = run(M, f, pre, dec), run(M, M.Qwen3Forward(m, ref, **args), pre, dec)
    for t, (g, r) in enumerate(zip(got, want)):
        rel = float((g.double() - r.double()).norm() / r.double().norm())
        assert rel <= 0.03, (t, rel)

    eager = f.decode(dec[0])[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, _ = f.decode(dec[0])
    logits.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(logits, eager)
