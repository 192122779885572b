"""Calls on 4-bit weights as they run together: rows of a batch against the rows alone,
a chain with and without the statement that the weights were complete, eager and
replayed, and calls beside other kernels that hold TMEM.  Bounds as in test_gpu_w4.py."""
import pytest
import torch

from test_gpu_w4 import COL, L, NONE, ROW, SILU, gen, matrix, product, run_gemm, sync_ok  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [2, 8, 24, 64, 100, 300])
def test_rows_of_a_batch_and_rows_alone(L, M):  # noqa: F811
    """Other kernels, or other splits of K, may take a row alone: both results lie within the bound of the exact one, so
    they are at most twice the bound apart."""
    c, s, z, w = matrix(512, 2048, 128, True, seed=6)
    x = torch.randn(M, 2048, generator=gen(8)).bfloat16()
    batch = run_gemm(L, x.cuda(), c, s, z, 512, 128, 1, COL, NONE)
    y, e = product(x.double(), w)
    for m in sorted({0, 1, M // 2, M - 1}):
        alone = run_gemm(L, x[m:m + 1].cuda(), c, s, z, 512, 128, 1, COL, NONE)
        sync_ok(L)
        apart = (alone[0].double() - batch[m].double()).abs().cpu()
        assert (apart <= 2 * (2.0 ** -8 * y[m].abs() + e[m])).all(), m


@pytest.mark.parametrize("M", [3, 90, 400])
def test_chain_ready_or_not_eager_or_replayed(L, M):  # noqa: F811
    """Embedding, gate_up with SiluAndMul, down, logits: the same bits each way, for several token ids."""
    H, I, V, tp, G = 256, 384, 600, 2, 32
    g, dev = gen(21), "cuda"
    q = []
    for N, K, zeros in ((V, H, False), (2 * I, H, True), (tp * H, I // tp, True)):
        w = (0.05 * torch.randn(N, K, generator=g)).bfloat16().to(dev)
        q.append((torch.empty(N, K // 2, dtype=torch.uint8, device=dev), torch.empty(N, K // G, dtype=torch.bfloat16, device=dev),
                  torch.empty(N, K // G, dtype=torch.uint8, device=dev) if zeros else None))
        L.w4_quantize(w, G, *q[-1])
    ids = torch.randint(0, V, (M,), generator=g).to(dev)
    x, act, y = (torch.empty(M, k, dtype=torch.bfloat16, device=dev) for k in (H, I, H))
    logits = torch.empty(M, V, dtype=torch.bfloat16, device=dev)
    tok = torch.empty(M, dtype=torch.int64, device=dev)
    ws = torch.zeros(L.w4_lm_head_workspace_size(M, V, H, tp), dtype=torch.uint8, device=dev)

    def step(ready):
        L.w4_embed_vocab(ids, *q[0], G, tp, x)
        L.w4_gemm(x, *q[1], act, 2 * I, G, tp, COL, SILU, weights_ready=ready)
        L.w4_gemm(act, *q[2], y, H, G, tp, ROW, NONE, weights_ready=ready)
        L.w4_lm_head(y, None, M, *q[0], G, tp, logits, tok, ws, weights_ready=ready)

    def results(run):
        for t in (x, act, y, logits):
            t.fill_(float("nan"))
        tok.fill_(-1)
        run()
        sync_ok(L)
        return [t.clone() for t in (x, act, y, logits, tok)]

    step(False)
    torch.cuda.synchronize()
    graphs = []
    for ready in (False, True):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(ready)
    for seed in (None, 1, 2):
        if seed is not None:
            ids.copy_(torch.randint(0, V, (M,), generator=gen(seed)).to(dev))
        first = results(lambda: step(False))
        assert all(torch.isfinite(t.float()).all() for t in first)
        for run in [lambda: step(True)] + [graph.replay for graph in graphs]:
            assert all(torch.equal(a, b) for a, b in zip(first, results(run)))


@pytest.mark.parametrize("M", [40, 200, 1000])
def test_beside_other_kernels_with_tmem(L, M):  # noqa: F811
    """4-bit products on one stream, bf16 products and prefill attention on another."""
    N, K = 2048, 2048
    c, s, z, _ = matrix(N, K, 128, True, seed=3)
    x = torch.randn(M, K, generator=gen(1)).bfloat16().cuda()
    w = (0.02 * torch.randn(N, K, generator=gen(2))).bfloat16().cuda()
    nh, nkv, hd = 16, 8, 128
    q = torch.randn(M, nh, hd, generator=gen(4)).bfloat16().cuda()
    k, v = (torch.randn(M, nkv, hd, generator=gen(i)).bfloat16().cuda() for i in (5, 6))
    cu = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(L.gemm_workspace_size(M, N, K, 1, COL, NONE, torch.bfloat16), 16), dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def outputs(n):
        return [[torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(n)] for _ in range(2)] + [
            [torch.empty(M, nh, hd, dtype=torch.bfloat16, device="cuda") for _ in range(n)]]

    def four(o, st):
        L.w4_gemm(x, c, s, z, o, N, 128, stream=st)

    def others(o, p, st):
        L.gemm(x, w, o, N, 1, COL, NONE, ws, stream=st)
        L.attention_prefill(q, k, v, cu, cu, None, M, nh, nkv, hd, hd ** -0.5, p, stream=st)

    want = outputs(1)
    torch.cuda.synchronize()
    four(want[0][0], a)
    torch.cuda.synchronize()
    others(want[1][0], want[2][0], b)
    torch.cuda.synchronize()
    got = outputs(20)
    torch.cuda.synchronize()
    for o, p, r in zip(*got):
        four(o, a)
        others(p, r, b)
    sync_ok(L)
    for t, ref in zip(got, want):
        assert all(torch.equal(o, ref[0]) for o in t)
