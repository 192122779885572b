"""Queries that are not finite, over the 8-bit paged KV cache: their rows are NaN,
whichever way the keys are cut, and no other row changes."""
import pytest
import torch

from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen, sync_ok  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu


def _poison(q, at, value):
    q = q.clone()
    for i, (t, h) in enumerate(at):
        q[t, h, (37 * i) % HD] = value
    return q


def _check(clean, got, at):
    bad = torch.zeros(got.shape[:2], dtype=torch.bool)
    for t, h in at:
        bad[t, h] = True
    got, clean = got.cpu(), clean.cpu()
    assert torch.isfinite(clean.float()).all()
    assert torch.isnan(got[bad].float()).all()
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("lens,lq,split", [([1500, 1100], [7, 5], True), ([300, 130], [300, 9], False), ([9000], [1], True)])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4)])
def test_prefill(L, kv, lens, lq, split, window, sink):
    nh, nkv = 8, 2
    need = L.attention_prefill_kv8_workspace_size(len(lens), sum(lq), max(lq), max(lens), nh, nkv)
    assert (need > 0) == split
    d = Paged(lens, nkv, kv, 32, 128, seed=3).cuda()
    q = torch.randn(sum(lq), nh, HD, generator=gen(4)).bfloat16()
    clean = K._prefill(L, d, q.cuda(), lens, lq, nh, window, sink)
    at = [(0, 0), (0, 5), (sum(lq) - 1, 7), (sum(lq) // 2, 2)]
    got = K._prefill(L, d, _poison(q, at, float("nan")).cuda(), lens, lq, nh, window, sink)
    sync_ok(L)
    _check(clean, got, at)


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("nh,nkv,lens", [(16, 8, [3000, 40, 777]), (8, 1, [9000, 5]), (32, 2, [130, 2500])])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4)])
def test_decode(L, kv, nh, nkv, lens, window, sink):
    d = Paged(lens, nkv, kv, 32, 128, seed=3).cuda()
    q = torch.randn(len(lens), nh, HD, generator=gen(4)).bfloat16()
    at = [(0, 0), (len(lens) - 1, nh - 1), (1, 2)]
    clean = K._decode(L, d, q.cuda(), lens, nh, window, sink)
    got = K._decode(L, d, _poison(q, at, float("nan")).cuda(), lens, nh, window, sink)
    sync_ok(L)
    _check(clean, got, at)


@pytest.mark.parametrize("lens,lq", [([1500, 40], [6, 3]), ([200], [200])])
@pytest.mark.parametrize("nh,nkv", [(8, 2), (8, 1), (16, 1)])
def test_values_of_zero(L, lens, lq, nh, nkv):
    """NaN times a value of zero is NaN: blocks whose v_scale is zero hide nothing, also where every head has NaN."""
    d = Paged(lens, nkv, I8, 32, 128, seed=3).cuda()
    d.vs.zero_()
    q = torch.randn(sum(lq), nh, HD, generator=gen(4)).bfloat16()
    at = [(0, 1), (sum(lq) - 1, 6)]
    clean = K._prefill(L, d, q.cuda(), lens, lq, nh, 0, 0)
    got = K._prefill(L, d, _poison(q, at, float("nan")).cuda(), lens, lq, nh, 0, 0)
    n = len(lens)
    at_d = [(n - 1, 6)] + [(0, h) for h in range(nh)]
    clean_d = K._decode(L, d, q[:n].cuda(), lens, nh, 0, 0)
    got_d = K._decode(L, d, _poison(q[:n], at_d, float("nan")).cuda(), lens, nh, 0, 0)
    sync_ok(L)
    assert torch.all(clean == 0) and torch.all(clean_d == 0)
    _check(clean, got, at)
    _check(clean_d, got_d, at_d)


@pytest.mark.parametrize("lens,lq", [([3, 0, 2000], [6, 4, 5]), ([3, 40], [6, 40])])
def test_rows_that_see_nothing_stay_zero(L, lens, lq):
    """Queries at negative key positions see no key: zero rows, NaN in them or not."""
    nh, nkv = 4, 2
    d = Paged(lens, nkv, I8, 16, 64, seed=1).cuda()
    q = torch.randn(sum(lq), nh, HD, generator=gen(5)).bfloat16()
    q[0, 0, 3] = float("nan")
    q[2, 3] = float("nan")
    out = K._prefill(L, d, q.cuda(), lens, lq, nh, 0, 0)
    ctx0 = K._decode(L, d, q[:len(lens)].cuda(), [0] * len(lens), nh, 0, 0, max_context=64)
    sync_ok(L)
    assert torch.all(out[:3] == 0) and torch.all(ctx0 == 0)
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("lens,lq", [([1500, 1100], [7, 5]), ([300, 130], [300, 9])])
def test_infinite_queries(L, lens, lq):
    """An infinite element meets codes of both signs: infinity less infinity, a NaN row; other rows within rounding."""
    nh, nkv = 8, 2
    c = Paged(lens, nkv, I8, 32, 128, seed=3)
    d = c.cuda()
    q = torch.randn(sum(lq), nh, HD, generator=gen(4)).bfloat16()
    at = [(0, 3), (sum(lq) - 2, 0)]
    got = K._prefill(L, d, _poison(q, at, float("inf")).cuda(), lens, lq, nh, 0, 0).cpu()
    got_d = K._decode(L, d, _poison(q[:2], [(0, 3)], float("inf")).cuda(), lens, nh, 0, 0).cpu()
    sync_ok(L)
    for t, h in at:
        assert torch.isnan(got[t, h].float()).all()
        got[t, h] = 0
    assert torch.isnan(got_d[0, 3].float()).all()
    got_d[0, 3] = 0
    assert torch.isfinite(got.float()).all() and torch.isfinite(got_d.float()).all()
    for t, h in at:
        q[t, h] = 0          # (a row of zeros: compared nowhere below)
    lo = 0
    for s, (n, m) in enumerate(zip(lens, lq)):
        r = c.rows(s, 0, n)
        o, tol = K.attend64(q[lo:lo + m].double(), c.values("k", r), c.values("v", r), torch.arange(n - m, n), HD ** -0.5, 0, 0)
        ok = (got[lo:lo + m].double() - o).abs() <= tol
        for t, h in at:
            if lo <= t < lo + m:
                ok[t - lo, h] = True
        assert ok.all()
        lo += m
