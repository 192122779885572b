"""What an appended token's codes stand for after its block's scale has grown: half
a step when it was written and half a step of the new scale for each growth
since, counted from the scales themselves."""
import numpy as np
import pytest
import torch

from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen, sync_ok  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("sizes", [[1] * 40, [3, 1, 9, 2, 30, 1, 1], [64, 1, 1]])
def test_each_growth_costs_half_a_step(L, kv, sizes):
    nh, nkv, sb, bs = 2, 2, 32, 64
    total = sum(sizes)
    c = Paged([0, 0], nkv, kv, sb, bs, seed=2, capacity=total)
    d = c.cuda()
    cs = L.rope_cos_sin_table(total + 1, HD, 1e6).cuda()
    gam = torch.ones(HD, dtype=torch.bfloat16, device="cuda")
    v_all = [torch.zeros(0, nkv, HD, dtype=torch.float64) for _ in range(2)]
    lim = [np.zeros((0, nkv, HD)) for _ in range(2)]     # what each value may be off by so far
    grown, n = 0, 0
    for i, m in enumerate(sizes):
        n += m
        lens, lq = [n, n], [m, m]
        qkv, _, _, pos = K._append_case(nh, nkv, 1, lens, lq, 20 + i)
        v = qkv.view(2 * m, -1, HD)[:, nh + nkv:]
        v *= torch.exp(0.7 * torch.randn(2 * m, nkv, 1, generator=gen(60 + i))).bfloat16()     # token sizes that differ
        before = d.vs.cpu().double()
        q = torch.empty(2 * m, nh, HD, dtype=torch.bfloat16, device="cuda")
        L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), cs, gam, gam, 1e-6, torch.tensor([0, m, 2 * m], dtype=torch.int32).cuda(),
                     torch.tensor(lens, dtype=torch.int32).cuda(), d.table, bs, d.k, d.v, d.ks, d.vs, sb, q)
        sync_ok(L)
        after = d.vs.cpu().double()
        codes = K.codes_to_f64(d.v.cpu())
        for s in range(2):
            v_all[s] = torch.cat([v_all[s], v[s * m:(s + 1) * m].double()])
            r = c.rows(s, 0, n)
            sc = after[r // sb].numpy()[..., None]
            y = v_all[s].numpy()
            old = n - m
            grew = np.zeros((n, nkv, 1), bool)
            grew[:old] = (after[r[:old] // sb] > before[r[:old] // sb]).numpy()[..., None]
            grown += int(grew.any(2).any(1).sum())
            new = np.zeros((n, 1, 1), bool)
            new[old:] = True
            prev = np.concatenate([lim[s], np.zeros((m, nkv, HD))])
            # half a step of the code nearest to the value (for an old token: to the value its codes stood for)
            half = K._half_step(np.abs(y) + prev, sc, kv) * (1 + 8 * U) + 8 * U * (np.abs(y) + prev)
            lim[s] = prev + np.where(new | grew, half, 0.0)
            got = codes[r].numpy() * sc
            assert np.all(np.abs(got - y) <= lim[s]), (i, s)
    assert grown > 0
