"""The forward pass with an 8-bit paged KV cache: prompts, then decode steps,
eager and replayed, against the same entry points called one by one and against
the bf16 cache.

Distance to the bf16 cache, one layer: a block's largest of 64 x 128 near-normal
values is about 4.2 sigma, so an int8 step is 4.2 / 127 sigma and its error 0.0095
sigma rms, in k (which moves every score by as much) and in v; e4m3 has 3 bits of
mantissa, 2^-4 / sqrt(3) = 0.036 relative rms.  The attention output moves by at
most the two together, the logits (which the residual stream also feeds) by less:
the bounds are twice that, 0.04 and 0.15 of their norm.
"""
import numpy as np
import pytest
import torch

import seeded_inputs as si

pytestmark = pytest.mark.gpu

BS = 64


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_transformer_forward_gb300 import build
    build.build()
    from qwen3_transformer_forward_gb300 import model
    return model


def _tables(lens, steps):
    need = [-(-(n + steps) // BS) for n in lens]
    perm = torch.randperm(sum(need) + 1, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return table.cuda(), (sum(need) + 1) * BS


def _contexts(M, m, lens, steps):
    """Prefill context and one decode context per step, with both kinds of cache addressing."""
    B = len(lens)
    base = np.concatenate([[0], np.cumsum([n + steps for n in lens])[:-1]]).astype(np.int64)
    table, slots = _tables(lens, steps)
    dev = lambda x, dt: torch.from_numpy(np.asarray(x)).to(dt).cuda()  # noqa: E731
    pos = np.concatenate([np.arange(n) for n in lens])
    cu = np.concatenate([[0], np.cumsum(lens)])
    ids = si.uniform_int(0, "kv8.ids", (len(pos),), 0, m.vocab).cuda()
    pre = M.PrefillContext(ids, dev(pos, torch.int64), dev(cu, torch.int32),
                           dev(np.concatenate([b + np.arange(n) for b, n in zip(base, lens)]), torch.int64),
                           dev(base, torch.int32), dev(cu[1:] - 1, torch.int32), max(lens), table,
                           dev(lens, torch.int32), max(lens) + steps)
    dec = []
    for t in range(steps):
        n = np.asarray(lens) + t
        dec.append(M.DecodeContext(si.uniform_int(0, f"kv8.d{t}", (B,), 0, m.vocab).cuda(), dev(n, torch.int64),
                                   dev(n + 1, torch.int32), dev(base + n, torch.int64), dev(base, torch.int32),
                                   max(lens) + steps, table))
    return pre, dec, slots, int(sum(n + steps for n in lens))


@pytest.mark.parametrize("kv,bound", [(torch.int8, 0.04), (torch.float8_e4m3fn, 0.15)])
def test_forward_with_kv8(M, kv, bound):
    from qwen3_transformer_forward_gb300 import _lib as L
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=1, tp=2, gamma_sigma=0.1)
    lens, steps = [150, 3, 64], 4
    pre, dec, slots8, slots = _contexts(M, m, lens, steps)
    params = M.load_params(m)
    args = dict(max_tokens=sum(lens), max_seqs=3, max_context=max(lens) + steps)
    f8 = M.Qwen3Forward(m, params, num_slots=slots8, kv8=M.Kv8Config(kv, BS, 32), **args)
    f16 = M.Qwen3Forward(m, params, num_slots=slots, **args)
    got, ref = [], []
    for f, out in ((f8, got), (f16, ref)):
        out.append(f.prefill(pre)[0].clone())
        for c in dec:
            out.append(f.decode(c)[0].clone())
        torch.cuda.synchronize()
        L.device_error()
        assert int(f.err) == 0
    for t, (g, r) in enumerate(zip(got, ref)):
        rel = float((g.double() - r.double()).norm() / r.double().norm())
        assert rel <= bound, (t, rel)

    # the layer's steps one by one, on caches of their own
    c = f8.kv8
    k, v = (torch.zeros_like(f8.k_cache[0].view(torch.int8)).view(kv) for _ in range(2))
    ks, vs = torch.zeros_like(f8.k_scale[0]), torch.zeros_like(f8.v_scale[0])
    p, T, H = params.layers[0], sum(lens), m.hidden
    z = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, res, y, qkv, q, attn = z(T, H), z(T, H), z(T, H), z(T, f8.qkv_width), z(T, m.n_heads, 128), z(T, m.n_heads * 128)
    ws = torch.zeros(L.ATTENTION_PREFILL_KV8_WORKSPACE_MAX, dtype=torch.uint8, device="cuda")
    L.embed_vocab(pre.ids, params.embed, m.tp, h)
    L.add_rmsnorm(h, None, res, p.input_ln, m.eps, y)
    L.gemm(y, p.qkv, qkv, f8.qkv_width, m.tp)
    L.kv8_append(qkv, m.n_heads, m.n_kv_heads, 128, m.tp, pre.positions, f8.cos_sin, p.q_norm, p.k_norm, m.eps,
                 pre.cu_seqlens, pre.context_lens, pre.block_table, BS, k, v, ks, vs, 32, q)
    L.attention_prefill_kv8(q, k, v, ks, vs, 32, pre.cu_seqlens, pre.context_lens, pre.block_table, BS, max(lens),
                            pre.max_context, m.n_heads, m.n_kv_heads, 128, 128 ** -0.5, attn, ws)
    f8.prefill(pre)   # again: the blocks hold these tokens already, so codes and scales stay as they are
    torch.cuda.synchronize()
    assert torch.equal(f8.attn[:T].view(-1), attn.view(-1))
    assert torch.equal(f8.q[:T].view(-1), q.view(-1))

    # a captured decode step, replayed: what the eager step gave
    want = f8.decode(dec[0])[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, _ = f8.decode(dec[0])
    logits.zero_()
    graph.replay()
    torch.cuda.synchronize()
    L.device_error()
    assert torch.equal(logits, want)


def test_forward_with_kv8_window(M):
    """A window over every layer: a model whose prompts fit the window answers as without one."""
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=2)
    lens = [40, 90]
    pre, dec, slots, _ = _contexts(M, m, lens, 1)
    params = M.load_params(m)
    out = []
    for window, sink in ((0, 0), (91, 0), (16, 4)):
        f = M.Qwen3Forward(m, params, max_tokens=sum(lens), num_slots=slots, max_seqs=2, max_context=91,
                           kv8=M.Kv8Config(torch.int8, BS, 16, window, sink))
        out.append((f.prefill(pre)[0].clone(), f.decode(dec[0])[0].clone()))
    torch.cuda.synchronize()
    for a, b in zip(out[0], out[1]):
        assert torch.equal(a, b)
    assert not torch.equal(out[0][1], out[2][1])


def test_kv8_refusals(M):
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=1)
    params = M.load_params(m)
    with pytest.raises(ValueError):
        M.Qwen3Forward(si.TINY, M.load_params(si.TINY), max_tokens=8, num_slots=64, max_seqs=1, max_context=8, kv8=M.Kv8Config())
    pre, _, slots, _ = _contexts(M, m, [5], 1)
    f = M.Qwen3Forward(m, params, max_tokens=5, num_slots=slots, max_seqs=1, max_context=8, kv8=M.Kv8Config(torch.int8, BS))
    pre.block_table = None
    with pytest.raises(ValueError):
        f.prefill(pre)
