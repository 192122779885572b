"""Attention over the 8-bit paged KV cache with very large scores whose dot
products are exact: one element of a query is not zero and codes are small whole
numbers, so a score is one product and only the softmax's own roundings count.

Tolerance.  u = 2^-24.  With x_j the exponent in units of log2 and m the row's
largest, the kernels round x_j and m once each (u |x|), the factor log2 e * scale
twice (2u of |x_j - m|: the same factor for both) and x_j - m + shift at most
three times (u (|x_j| + |m|) in the fused form); equal scores have equal
exponents.  So a weight is off by the factor 2^(e_j), e_j = u (4 (|x_j| + |m|) +
2 |x_j - m|) at most and 0 where x_j = m and the difference is formed first, and
by 2^-11 (f16) and a few fp32 roundings; one below f16's normal range (2^-21 of
the largest, which is held times 2^7 or more) by 2^-32 of the largest; the output
by 2^-8 of itself."""
import math

import pytest
import torch

from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen, sync_ok  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _cache(lens, nkv, kv, g):
    """Whole-number codes -15 .. 15 in k and v; scales of 2^-4 and 2^-3 everywhere."""
    c = Paged(lens, nkv, kv, 32, 64, seed=3)
    for n in ("k", "v"):
        x = torch.randint(-15, 16, (c.slots, nkv, HD), generator=g)
        setattr(c, n, x.to(torch.int8) if kv == I8 else x.float().to(E4))
    c.ks = torch.full_like(c.ks, 2.0 ** -4)
    c.vs = torch.full_like(c.vs, 2.0 ** -3)
    return c


def _attend(q, k, v, p, scale):
    """float64: outputs and tolerances; q [n, nh, d] at positions p over k, v [L, nkv, d]."""
    G = q.shape[1] // k.shape[1]
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = torch.einsum("ihd,jhd->hij", q, kk) * (scale / math.log(2.0))
    x = x.masked_fill(~(torch.arange(k.shape[0])[None] <= p[:, None])[None], -float("inf"))
    m = x.amax(-1, keepdim=True)
    w = torch.exp2(x - m)
    w = w / w.sum(-1, keepdim=True)
    e = torch.where(w > 0, math.log(2.0) * U * (4 * (x.abs() + m.abs()) + 2 * (m - x)), torch.zeros_like(x))
    e = torch.where((x == m) & (m.abs() > 600), torch.zeros_like(e), e)      # (no fused form there: exactly zero)
    o = torch.einsum("hij,jhd->ihd", w, vv)
    a = torch.einsum("hij,jhd->ihd", w * (2.0 ** -11 + 16 * U + 2 * e), vv.abs())
    both = (w * 2 * e).sum(-1).T[..., None]
    small = k.shape[0] * 2.0 ** -32 * vv.abs().amax()
    return o, 2.0 ** -8 * o.abs() + a + both * o.abs() + small


def _query(n, nh, tops, g):
    """One element a head, its largest exponent (times code 15) about tops[(row + head) % len]."""
    q = torch.zeros(n, nh, HD)
    for i in range(n):
        for h in range(nh):
            t = tops[(i + h) % len(tops)]
            q[i, h, int(torch.randint(0, HD, (1,), generator=g))] = t
    return q.bfloat16()


# the largest exponent of a row is q * 15 / 16 * scale * log2 e; with scale = ln 2 * 16 / 15 it is q itself
SCALE = float(torch.tensor(math.log(2.0) * 16 / 15, dtype=torch.float32))
TOPS = [1.0, 60.0, 500.0, 510.0, 512.0, 516.0, 520.0, 2.0 ** 12, 2.0 ** 30, -2.0 ** 30, -514.0, 2.0 ** 60, 2.0 ** -40]


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("tops", [TOPS, [510.0], [514.0], [2.0 ** 30], [505.0, 1.0, 519.0]])
def test_large_scores(L, kv, tops):
    g = gen(7)
    nh, nkv = 8, 2
    for lens, lq in (([300, 77], [300, 20]), ([1500, 1030], [7, 9])):     # one CTA walks all keys, and keys split
        c = _cache(lens, nkv, kv, g)
        d = c.cuda()
        q = _query(sum(lq), nh, tops, g)
        cu = torch.tensor([0, lq[0], sum(lq)], dtype=torch.int32).cuda()
        ctx = torch.tensor(lens, dtype=torch.int32).cuda()
        ws = torch.zeros(max(256, L.attention_prefill_kv8_workspace_size(2, sum(lq), max(lq), max(lens), nh, nkv)),
                         dtype=torch.uint8, device="cuda")
        out = torch.full((sum(lq), nh, HD), 7.0, dtype=torch.bfloat16, device="cuda")
        L.attention_prefill_kv8(q.cuda(), d.k, d.v, d.ks, d.vs, 32, cu, ctx, d.table, 64, max(lq), max(lens), nh, nkv, HD, SCALE,
                                out, ws)
        qd = _query(2, nh, tops, g)
        outd = K._decode(L, d, qd.cuda(), lens, nh, 0, 0, scale=SCALE)
        sync_ok(L)
        at = 0
        for s, (n, m) in enumerate(zip(lens, lq)):
            r = c.rows(s, 0, n)
            k, v = c.values("k", r), c.values("v", r)
            for what, got, x, p in (("prefill", out[at:at + m], q[at:at + m], torch.arange(n - m, n)),
                                    ("decode", outd[s:s + 1], qd[s:s + 1], torch.tensor([n - 1]))):
                o, tol = _attend(x.double(), k, v, p, SCALE)
                err = (got.cpu().double() - o).abs()
                ok = err <= tol
                assert ok.all(), (what, s, float((err / tol).max()), [int(i) for i in (~ok).nonzero()[0]])
            at += m


def test_the_largest_score_alone(L):
    """Scores so far apart that one key has all the weight: its value comes out, rounded once."""
    nh, nkv, n = 4, 1, 700
    g = gen(9)
    c = _cache([n], nkv, I8, g)
    at = 5 * torch.arange(nh) + 3
    hot = [11, 333, 650, 699]
    r = c.rows(0, 0, n)
    for h in range(nh):
        c.k[r, 0, at[h]] = torch.randint(-15, 14, (n,), generator=g).to(torch.int8)
        c.k[r[hot[h]], 0, at[h]] = 14
    q = torch.zeros(1, nh, HD)
    for h, top in enumerate((2.0 ** 14, 2.0 ** 30, 2.0 ** 80, 2.0 ** 16)):
        q[0, h, at[h]] = top
    q = q.bfloat16()
    d = c.cuda()
    out = K._decode(L, d, q.cuda(), [n], nh, 0, 0, scale=SCALE)
    outp = K._prefill(L, d, q.cuda(), [n], [1], nh, 0, 0)
    sync_ok(L)
    for h in range(nh):
        want = (c.v[r[hot[h]], 0].double() * 2.0 ** -3).bfloat16()
        assert torch.equal(out.cpu()[0, h], want) and torch.equal(outp.cpu()[0, h], want)
