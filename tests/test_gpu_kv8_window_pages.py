"""Pages behind a sliding window: those that no query of a call sees may be taken
out of the block table, lie outside the cache, or belong to another sequence by
now, with the patterns of NaN in its codes and scales."""
import pytest
import torch

from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen, sync_ok  # noqa: F401  (L: the fixture)
from tests.test_gpu_kv8_finite import check_prefill

pytestmark = pytest.mark.gpu


def _drop(c, lens, first, window, sink):
    """The cache with every page unseen by the queries from key position first[s] on dropped or reused."""
    d = c.cuda()
    d.table, d.k, d.v, d.ks, d.vs = (t.clone() for t in (d.table, d.k, d.v, d.ks, d.vs))
    n = 0
    for s, L_ in enumerate(lens):
        for b in range(-(-L_ // c.bs)):
            a, e = b * c.bs, (b + 1) * c.bs
            if e <= first[s] - window + 1 and a >= sink:
                page = int(c.table[s, b])
                n += 1
                if n % 3 == 0:
                    d.table[s, b] = -1
                elif n % 3 == 1:
                    d.table[s, b] = 10 ** 6
                else:      # still in the table: another owner's tokens
                    rows = slice(page * c.bs, (page + 1) * c.bs)
                    d.k.view(torch.uint8)[rows] = 0x7F
                    d.v.view(torch.uint8)[rows] = 0xFF if c.kv == E4 else 0x7F
                    d.ks[page * c.bs // c.sb:(page + 1) * c.bs // c.sb] = float("nan")
                    d.vs[page * c.bs // c.sb:(page + 1) * c.bs // c.sb] = float("nan")
    assert n >= 6
    return d


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("nh,nkv", [(16, 8), (6, 2), (5, 1)])
@pytest.mark.parametrize("window,sink", [(1, 0), (100, 4), (64, 65), (130, 0)])
def test_pages_behind_the_window(L, kv, nh, nkv, window, sink):
    for lens, lq in (([1500, 700, 64], [40, 1, 1]), ([900, 650], [300, 200])):     # keys split, and not
        c = Paged(lens, nkv, kv, 16, 64, seed=window)
        q = torch.randn(sum(lq), nh, HD, generator=gen(2)).bfloat16()
        d = _drop(c, lens, [n - m for n, m in zip(lens, lq)], window, sink)
        outp = K._prefill(L, d, q.cuda(), lens, lq, nh, window, sink)
        d1 = _drop(c, lens, [n - 1 for n in lens], window, sink)
        qd = torch.randn(len(lens), nh, HD, generator=gen(3)).bfloat16()
        out = K._decode(L, d1, qd.cuda(), lens, nh, window, sink)
        sync_ok(L)
        K._check_decode(out, c, qd, lens, window, sink)
        check_prefill(outp, c, q, lens, lq, window, sink)
