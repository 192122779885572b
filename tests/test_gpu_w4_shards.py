"""Products over 4-bit weights whose shards of K are one step of 128 columns or less,
with many of them for each pair of SMs: every step has a code stage of its own there.
Bounds as in test_gpu_w4.py."""
import pytest
import torch

from test_gpu_w4 import COL, NONE, ROW, SILU, L, check_gemm, gen, matrix, near, product, sync_ok  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,group,tp,mode,epi", [
    (100, 12288, 1024, 128, 8, ROW, NONE), (200, 9600, 512, 64, 8, ROW, NONE), (70, 40000, 160, 32, 5, ROW, NONE),
    (100, 4096, 2560, 128, 20, ROW, NONE), (128, 20000, 384, 128, 3, ROW, NONE), (97, 100000, 96, 32, 1, COL, NONE),
    (120, 120000, 64, 64, 2, COL, SILU), (384, 9001, 672, 32, 7, ROW, NONE), (1000, 12000, 512, 64, 4, ROW, NONE)])
def test_shards_of_one_step(L, M, N, K, group, tp, mode, epi):  # noqa: F811
    first = check_gemm(L, M, N, K, group, M % 3 == 0, tp, mode, epi)
    for _ in range(3):
        assert torch.equal(check_gemm(L, M, N, K, group, M % 3 == 0, tp, mode, epi), first)


@pytest.mark.parametrize("n,V,H,group", [(65, 151936, 128, 128), (40, 151936, 96, 32), (128, 110000, 32, 32)])
def test_lm_head_of_one_step(L, n, V, H, group):  # noqa: F811
    c, s, z, w = matrix(V, H, group, True)
    h = torch.randn(n, H, generator=gen(n)).bfloat16()
    logits = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    tok = torch.empty(n, dtype=torch.int64, device="cuda")
    ws = torch.zeros(L.w4_lm_head_workspace_size(n, V, H, 1), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        logits.fill_(float("nan"))
        L.w4_lm_head(h.cuda(), None, n, c, s, z, group, 1, logits, tok, ws)
        sync_ok(L)
        near(logits, *product(h.double(), w), (n, V, H))
        assert torch.equal(tok.cpu(), logits.float().cpu().argmax(-1))
