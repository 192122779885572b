"""Prefill over the 8-bit paged KV cache with a comparison that a NaN fails.

test_gpu_kv8's prefill comparison asks whether an error is above its tolerance,
which a NaN never is.  Its tests, and those of test_gpu_kv8_edges and the served
conversation, run here again with one that asks whether it is at most that."""
import numpy as np
import pytest
import torch

from tests import test_gpu_kv8 as K
from tests import test_gpu_kv8_edges as X
from tests.test_gpu_kv8 import E4, HD, I8, L, gen  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu


def check_prefill(got, c, q, lens, lq, window, sink):
    got = got.cpu().double()
    at = 0
    for s, (n, m) in enumerate(zip(lens, lq)):
        r = c.rows(s, 0, n)
        o, tol = K.attend64(q[at:at + m].double(), c.values("k", r), c.values("v", r), torch.arange(n - m, n), HD ** -0.5,
                            window, sink)
        ok = (got[at:at + m] - o).abs() <= tol
        assert ok.all(), (s, n, m, int((~ok).sum()), [int(i) for i in (~ok).nonzero()[0]])
        at += m


@pytest.fixture(autouse=True)
def nan_fails(monkeypatch):
    monkeypatch.setattr(K, "_check_prefill", check_prefill)


def test_the_comparison_itself():
    """On the CPU's side of it: a NaN and a wrong value fail, the right values pass."""
    c = K.Paged([20], 1, I8, 16, 64, seed=1)
    q = torch.randn(3, 2, HD, generator=gen(1)).bfloat16()
    r = c.rows(0, 0, 20)
    o, _ = K.attend64(q.double(), c.values("k", r), c.values("v", r), torch.arange(17, 20), HD ** -0.5, 0, 0)
    check_prefill(o, c, q, [20], [3], 0, 0)
    for wrong in (float("nan"), 9.0):
        x = o.clone()
        x[1, 1, 7] = wrong
        with pytest.raises(AssertionError):
            check_prefill(x, c, q, [20], [3], 0, 0)


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4), (1, 0)])
def test_prefill(L, kv, window, sink):
    for nh, nkv, sb, bs, lens, lq in (
            (16, 8, 64, 256, [600, 130, 256, 1], [90, 130, 1, 1]), (4, 1, 16, 64, [1024, 300], [1024, 44]),
            (6, 2, 32, 128, [129, 500, 7], [129, 250, 0]), (16, 1, 64, 64, [333], [33]), (2, 2, 32, 64, [700], [513]),
            (16, 8, 64, 256, [6000], [3]), (1, 1, 64, 64, [300, 300, 300], [256, 257, 255])):
        K.test_prefill(L, kv, nh, nkv, sb, bs, lens, lq, window, sink)


@pytest.mark.parametrize("kv", [I8, E4])
def test_scales_and_empty_rows(L, kv):
    K.test_prefill_scales_of_many_sizes(L, kv)
    K.test_prefill_rows_that_see_nothing(L)
    X.test_prefill_few_rows_that_see_nothing(L)
    X.test_sequences_share_a_prefix(L)


@pytest.mark.parametrize("window,sink", [(0, 0), (40, 2)])
def test_nan_patterns_behind_a_sequence(L, window, sink):
    X.test_nan_patterns_behind_a_sequence(L, window, sink)


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("window,sink", [(0, 0), (700, 100)])
def test_few_rows(L, kv, window, sink):
    for lens, lq, nh, nkv in (([1500, 1100, 1024], [7, 3, 1], 8, 2), ([1025], [16], 8, 1), ([5000, 1], [5, 1], 4, 4),
                              ([1300] * 30, [2] * 30, 16, 8), ([9000], [64], 2, 1)):
        X.test_prefill_few_rows(L, kv, lens, lq, nh, nkv, window, sink)


@pytest.mark.parametrize("kv", [I8, E4])
def test_head_layouts(L, kv):
    for nh, nkv in ((7, 1), (15, 1), (26, 2), (21, 7), (108, 9)):
        X.test_head_layouts(L, nh, nkv, kv)


@pytest.mark.parametrize("lens,lq", [([40, 300, 5], [200, 300, 9]), ([2000, 3], [12, 30])])
def test_largest_window_and_sink(L, lens, lq):
    X.test_largest_window_and_sink(L, lens, lq)


@pytest.mark.parametrize("kv", [I8, E4])
def test_serve(L, kv):
    K.test_serve(L, kv, 0, 0)
    K.test_serve(L, kv, 50, 3)
