"""The forward pass with 4-bit linear weights: prompts, then decode steps, eager and
replayed, against the same entry points called one by one and against the bf16
forward pass over the weights that the codes stand for.

Distance to that pass: both compute the same function with bf16 tensors between the
steps, about 12 a layer and the logits.  A rounding is off by at most 2^-8 of the
value, 2^-8 / sqrt(3) = 0.0023 rms, and independent ones add in squares:
0.0023 * sqrt(2 * 13) = 0.012 of the logits' norm for one layer if not one of them
agreed.  The bound is 0.02, and 0.03 for two layers.
"""
import dataclasses

import pytest
import torch

import seeded_inputs as si
from test_gpu_kv8_model import BS, _contexts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_transformer_forward_gb300 import build
    build.build()
    from qwen3_transformer_forward_gb300 import model
    return model


def values(M, w, like):
    """The bf16 weight that a W4Weight stands for."""
    from qwen3_transformer_forward_gb300 import _lib as L
    N, K = w.codes.shape[0], w.codes.shape[1] * 2
    out = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    L.w4_embed_vocab(torch.arange(N, device="cuda"), w.codes, w.scales, w.zeros, w.group, 1, out)
    return out.view(like.shape)


def bf16_of(M, q, p):
    """Parameters q (in 4 bits) as bf16 ones of p's shapes."""
    layers = [dataclasses.replace(a, **{n: values(M, getattr(a, n), getattr(b, n)) for n in ("qkv", "o", "gate_up", "down")})
              for a, b in zip(q.layers, p.layers)]
    return M.ModelParams(values(M, q.embed, p.embed) if isinstance(q.embed, M.W4Weight) else q.embed, layers, q.final_norm)


def run(M, f, pre, dec):
    from qwen3_transformer_forward_gb300 import _lib as L
    out = [f.prefill(pre)[0].clone()]
    for c in dec:
        out.append(f.decode(c)[0].clone())
    torch.cuda.synchronize()
    L.device_error()
    assert int(f.err) == 0
    return out


@pytest.mark.parametrize("layers,cfg,bound", [(1, dict(group=128), 0.02), (1, dict(group=32, zeros=True), 0.02),
                                              (2, dict(group=64, table=False), 0.03)])
def test_forward_with_4bit_weights(M, layers, cfg, bound):
    from qwen3_transformer_forward_gb300 import _lib as L
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=layers, tp=2, gamma_sigma=0.1)
    lens, steps = [150, 3, 64], 3
    pre, dec, _, slots = _contexts(M, m, lens, steps)
    p = M.load_params(m)
    q = M.w4_params(p, M.W4Config(**cfg))
    args = dict(max_tokens=sum(lens), max_seqs=3, max_context=max(lens) + steps, num_slots=slots)
    f = M.Qwen3Forward(m, q, **args)
    got, ref = run(M, f, pre, dec), run(M, M.Qwen3Forward(m, bf16_of(M, q, p), **args), pre, dec)
    for t, (g, r) in enumerate(zip(got, ref)):
        rel = float((g.double() - r.double()).norm() / r.double().norm())
        assert rel <= bound, (t, rel)

    if layers == 1:
        # the first steps one by one
        T, w = sum(lens), q.layers[0]
        z = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        h, res, y, qkv = z(T, m.hidden), z(T, m.hidden), z(T, m.hidden), z(T, f.qkv_width)
        f.prefill(pre)
        L.w4_embed_vocab(pre.ids, q.embed.codes, q.embed.scales, q.embed.zeros, q.embed.group, m.tp, h)
        L.add_rmsnorm(h, None, res, w.input_ln, m.eps, y)
        L.w4_gemm(y, w.qkv.codes, w.qkv.scales, w.qkv.zeros, qkv, f.qkv_width, w.qkv.group, m.tp)
        torch.cuda.synchronize()
        assert torch.equal(f.qkv[:T], qkv)

    # a captured decode step, replayed: what the eager step gave
    want = f.decode(dec[0])[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, tokens = f.decode(dec[0])
    for _ in range(2):
        logits.zero_()
        tokens.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        L.device_error()
        assert torch.equal(logits, want)
        assert torch.equal(tokens, want.float().argmax(-1))


def test_load_params_in_4_bits(M):
    """Quantised while loading: the same codes as afterwards; and with the 8-bit KV cache it runs."""
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=2)
    cfg = M.W4Config(group=64)
    a, b = M.load_params(m, w4=cfg), M.w4_params(M.load_params(m), cfg)
    for x, y in [(a.embed, b.embed)] + [(getattr(s, n), getattr(t, n)) for s, t in zip(a.layers, b.layers)
                                        for n in ("qkv", "o", "gate_up", "down")]:
        assert torch.equal(x.codes, y.codes) and torch.equal(x.scales, y.scales) and x.zeros is None
    lens, steps = [70, 200], 2
    pre, dec, slots8, slots = _contexts(M, m, lens, steps)
    args = dict(max_tokens=sum(lens), max_seqs=2, max_context=max(lens) + steps)
    got = run(M, M.Qwen3Forward(m, a, num_slots=slots8, kv8=M.Kv8Config(torch.int8, BS, 32), **args), pre, dec)
    ref = run(M, M.Qwen3Forward(m, a, num_slots=slots, **args), pre, dec)
    for g, r in zip(got, ref):   # the cache's rounding: 0.04 of the norm a layer
        assert float((g.double() - r.double()).norm() / r.double().norm()) <= 0.08


def test_4bit_refusals(M):
    from qwen3_transformer_forward_gb300 import _lib as L
    with pytest.raises(L.QwError) as e:
        M.load_params(si.TINY, w4=M.W4Config(group=32))      # fp32 weights
    assert e.value.code == L.QW_ERR_DTYPE
    m = si.QWEN3_0_6B.replace(vocab=512, n_layers=1, hidden=1024 + 32)
    with pytest.raises(L.QwError) as e:
        M.load_params(m, w4=M.W4Config(group=128))            # rows that are not whole groups
    assert e.value.code == L.QW_ERR_SHAPE
