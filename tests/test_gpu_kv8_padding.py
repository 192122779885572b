"""Prefill over the 8-bit paged KV cache in a padded batch: more rows of q than the
sequences can have, as a caller with fixed buffer sizes passes them."""
import pytest
import torch

import seeded_inputs as si
from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen, sync_ok  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("lens,lq,pad", [([1500, 1100], [7, 5], 2000), ([9000], [1], 511), ([4000, 3], [2, 30], 300)])
def test_rows_of_padding_ask_for_no_room(L, kv, lens, lq, pad):
    """The same outputs, bit for bit, from the same workspace, whatever the number of padding rows."""
    nh, nkv = 8, 2
    d = Paged(lens, nkv, kv, 32, 128, seed=3).cuda()
    T = sum(lq)
    q = torch.randn(T, nh, HD, generator=gen(4)).bfloat16()
    full = torch.cat([q, torch.full((pad, nh, HD), float("nan"), dtype=torch.bfloat16)])
    ws = torch.zeros(L.ATTENTION_PREFILL_KV8_WORKSPACE_MAX, dtype=torch.uint8, device="cuda")
    want = K._prefill(L, d, q.cuda(), lens, lq, nh, 0, 0, ws=ws)
    got = K._prefill(L, d, full.cuda(), lens, lq, nh, 0, 0, ws=ws)
    sync_ok(L)
    assert torch.equal(got[:T], want) and torch.all(got[T:] == 7.0)


def test_rows_before_the_first_sequence(L):
    """Sequences that begin at a later row, keys split: rows before them stay as they were."""
    nh, nkv, lens, lq = 8, 2, [1500, 1100], [7, 5]
    d = Paged(lens, nkv, I8, 32, 128, seed=3).cuda()
    q = torch.randn(12, nh, HD, generator=gen(4)).bfloat16().cuda()
    want = K._prefill(L, d, q, lens, lq, nh, 0, 0)
    full = torch.cat([torch.zeros(9, nh, HD, dtype=torch.bfloat16, device="cuda"), q])
    out = torch.full_like(full, 7.0)
    ws = torch.zeros(L.attention_prefill_kv8_workspace_size(2, 21, 7, 1500, nh, nkv), dtype=torch.uint8, device="cuda")
    L.attention_prefill_kv8(full, d.k, d.v, d.ks, d.vs, 32, torch.tensor([9, 16, 21], dtype=torch.int32).cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), d.table, 128, 7, 1500, nh, nkv, HD, HD ** -0.5, out, ws)
    sync_ok(L)
    assert torch.equal(out[9:], want) and torch.all(out[:9] == 7.0)


def test_forward_of_a_padded_batch(L):
    """The model takes a prompt of two tokens in a buffer of 2000: the logits of the two tokens alone."""
    from qwen3_transformer_forward_gb300 import model as M
    m = si.QWEN3_0_6B.replace(vocab=4096, n_layers=1)
    params = M.load_params(m)
    max_context, pad = 4096, 1998
    out = []
    for extra in (0, pad):
        b = si.prefill_batch(m, [2])
        ctx = M.to_device_prefill(b)
        ctx.ids = torch.cat([ctx.ids, torch.zeros(extra, dtype=torch.int64, device="cuda")])
        ctx.positions = torch.cat([ctx.positions, torch.zeros(extra, dtype=torch.int64, device="cuda")])
        ctx.block_table = torch.arange(max_context // 256, dtype=torch.int32, device="cuda")[None]
        ctx.context_lens = torch.tensor([2], dtype=torch.int32, device="cuda")
        ctx.max_context = max_context
        f = M.Qwen3Forward(m, params, max_tokens=2 + pad, num_slots=max_context, max_seqs=1, max_context=max_context,
                           kv8=M.Kv8Config())
        out.append(f.prefill(ctx)[0].clone())
        sync_ok(L)
    # (other GEMM tiles for other token counts: bf16 roundings of the hidden rows)
    a, b = (x.double() for x in out)
    assert float((a - b).norm() / b.norm()) <= 0.02
