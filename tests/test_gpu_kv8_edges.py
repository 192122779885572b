"""The 8-bit paged KV cache at its edges: head counts that fill no tile, caches past
2^31 bytes, rows behind a sequence that hold NaN patterns, calls side by side.
The implementations in 64 bits and their tolerances are those of test_gpu_kv8."""
import numpy as np
import pytest
import torch

from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen, sync_ok  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nh,nkv", [(7, 1), (9, 1), (12, 1), (15, 1), (26, 2), (10, 5), (21, 7), (12, 12), (108, 9), (18, 6)])
@pytest.mark.parametrize("kv", [I8, E4])
def test_head_layouts(L, nh, nkv, kv):
    lens, lq = [300, 77], [40, 77]
    c = Paged(lens, nkv, kv, 16, 64, seed=nh)
    d = c.cuda()
    q = torch.randn(2, nh, HD, generator=gen(nh)).bfloat16()
    out = K._decode(L, d, q.cuda(), lens, nh, 0, 0)
    qp = torch.randn(sum(lq), nh, HD, generator=gen(nh)).bfloat16()
    outp = K._prefill(L, d, qp.cuda(), lens, lq, nh, 50, 3)
    sync_ok(L)
    K._check_decode(out, c, q, lens, 0, 0)
    K._check_prefill(outp, c, qp, lens, lq, 50, 3)


@pytest.mark.parametrize("nkv,nh", [(3, 6), (5, 5), (12, 24)])
def test_append_head_layouts(L, nkv, nh):
    for lens, lq in (([70, 20], [70, 20]), ([70, 20], [1, 1])):
        c = Paged(lens, nkv, I8, 16, 64, seed=3)
        qkv, qg, kg, pos = K._append_case(nh, nkv, 1, lens, lq, 8)
        cs = L.rope_cos_sin_table(80, HD, 1e6)
        d = c.cuda()
        q = torch.empty(sum(lq), nh, HD, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lq)]), dtype=torch.int32).cuda()
        L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), cs.cuda(), qg.cuda(), kg.cuda(), 1e-6, cu,
                     torch.tensor(lens, dtype=torch.int32).cuda(), d.table, 64, d.k, d.v, d.ks, d.vs, 16, q)
        sync_ok(L)
        _, k, v = K._split(qkv, nh, nkv, 1)
        y, tol = K._k64(k, kg, cs, pos)
        for a, b, sa, sb, val, vt in ((c.k, d.k, c.ks, d.ks, y, tol), (c.v, d.v, c.vs, d.vs, v, torch.zeros_like(v))):
            K._check_blocks(a.double().numpy(), b.cpu().double().numpy(), c, sa.double().numpy(), sb.cpu().double().numpy(),
                            val.numpy(), vt.numpy(), lens, lq, I8, (nkv, lq))


@pytest.mark.parametrize("window,sink", [(0, 0), (40, 2)])
def test_nan_patterns_behind_a_sequence(L, window, sink):
    """e4m3 rows from a sequence's end to its block's end may hold the patterns of NaN."""
    lens, lq, nh, nkv = [37, 130, 64, 1], [20, 130, 3, 1], 8, 2
    c = Paged(lens, nkv, E4, 64, 64, seed=5)
    for s, n in enumerate(lens):
        r = c.rows(s, n, -(-n // 64) * 64)
        c.k.view(torch.uint8)[r] = 0x7F
        c.v.view(torch.uint8)[r] = 0xFF
    d = c.cuda()
    q = torch.randn(4, nh, HD, generator=gen(1)).bfloat16()
    qp = torch.randn(sum(lq), nh, HD, generator=gen(2)).bfloat16()
    out = K._decode(L, d, q.cuda(), lens, nh, window, sink)
    outp = K._prefill(L, d, qp.cuda(), lens, lq, nh, window, sink)
    sync_ok(L)
    K._check_decode(out, c, q, lens, window, sink)
    K._check_prefill(outp, c, qp, lens, lq, window, sink)


def test_cache_past_two_gib(L):
    """Pages at the far end of a cache of 4.3 GB: append, read, decode and prefill find them."""
    nh, nkv, sb, bs, slots = 8, 8, 32, 128, (1 << 22) + 256
    lens = [200, 50]
    small = Paged(lens, nkv, I8, sb, bs, seed=6)
    shift = (slots - small.slots) // bs                      # the small cache's pages at the end of the large one
    big = Paged.__new__(Paged)
    big.__dict__.update(small.__dict__)
    big.k, big.v = (torch.empty(slots, nkv, HD, dtype=I8, device="cuda") for _ in range(2))
    big.ks, big.vs = (torch.zeros(slots // sb, nkv, device="cuda") for _ in range(2))
    big.k[-small.slots:], big.v[-small.slots:] = small.k.cuda(), small.v.cuda()
    big.ks[-(small.slots // sb):], big.vs[-(small.slots // sb):] = small.ks.cuda(), small.vs.cuda()
    big.table = torch.where(small.table >= 0, small.table + shift, small.table).cuda()
    assert big.k.numel() > 1 << 32
    q = torch.randn(2, nh, HD, generator=gen(1)).bfloat16()
    out = K._decode(L, big, q.cuda(), lens, nh, 0, 0)
    outp = K._prefill(L, big, q.cuda(), lens, [1, 1], nh, 0, 0)
    rows = small.rows(0, 150, 200)
    ko = torch.empty(50, nkv, HD, dtype=torch.float32, device="cuda")
    vo = torch.empty_like(ko)
    L.kv8_read(big.k, big.v, big.ks, big.vs, sb, (rows + shift * bs).cuda(), ko, vo)
    sync_ok(L)
    K._check_decode(out, small, q, lens, 0, 0)
    K._check_decode(outp, small, q, lens, 0, 0)
    assert torch.equal(ko.cpu().double(), (small.k[rows].float() * small.ks[rows // sb][..., None]).double())
    assert torch.equal(vo.cpu().double(), (small.v[rows].float() * small.vs[rows // sb][..., None]).double())
    # the same append on both caches
    qkv, qg, kg, pos = K._append_case(nh, nkv, 1, lens, [7, 1], 8)
    cs = L.rope_cos_sin_table(256, HD, 1e6).cuda()
    cu = torch.tensor([0, 7, 8], dtype=torch.int32).cuda()
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    d = small.cuda()
    for t in (d, big):
        qo = torch.empty(8, nh, HD, dtype=torch.bfloat16, device="cuda")
        L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), cs, qg.cuda(), kg.cuda(), 1e-6, cu, ctx, t.table, bs, t.k, t.v,
                     t.ks, t.vs, sb, qo)
    sync_ok(L)
    assert torch.equal(d.k, big.k[-small.slots:]) and torch.equal(d.v, big.v[-small.slots:])
    assert torch.equal(d.ks.nan_to_num(7), big.ks[-(small.slots // sb):].nan_to_num(7))


def test_cache_that_ends_inside_a_page(L):
    """num_slots is a multiple of scale_block, not of block_size: the blocks that fit are used, the rest counts as missing."""
    nh, nkv, sb, bs = 4, 2, 16, 64
    c = Paged([64], nkv, I8, sb, bs, seed=2, spare=0)
    for keep in (16, 48):
        d = c.cuda()
        d.k, d.v = d.k[:keep].contiguous(), d.v[:keep].contiguous()
        d.ks, d.vs = d.ks[:keep // sb].contiguous(), d.vs[:keep // sb].contiguous()
        q = torch.randn(1, nh, HD, generator=gen(1)).bfloat16()
        qp = torch.randn(64, nh, HD, generator=gen(2)).bfloat16()
        out = K._decode(L, d, q.cuda(), [64], nh, 0, 0)
        outp = K._prefill(L, d, qp.cuda(), [64], [64], nh, 0, 0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        qkv, qg, kg, pos = K._append_case(nh, nkv, 1, [64], [64], 8)
        qo = torch.empty(64, nh, HD, dtype=torch.bfloat16, device="cuda")
        sync_ok(L)
        r = torch.arange(64)
        k, v = c.values("k", r), c.values("v", r)
        k[keep:] = 0
        v[keep:] = 0
        o, tol = K.attend64(q.double(), k, v, torch.tensor([63]), HD ** -0.5, 0, 0)
        assert torch.all((out.cpu().double() - o).abs() <= tol)
        o, tol = K.attend64(qp.double(), k, v, r, HD ** -0.5, 0, 0)
        assert torch.all((outp.cpu().double() - o).abs() <= tol)
        L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), L.rope_cos_sin_table(64, HD, 1e6).cuda(), qg.cuda(), kg.cuda(), 1e-6,
                     torch.tensor([0, 64], dtype=torch.int32).cuda(), torch.tensor([64], dtype=torch.int32).cuda(), d.table, bs,
                     d.k, d.v, d.ks, d.vs, sb, qo, err)
        sync_ok(L)
        assert int(err) == 64 - keep


def test_calls_side_by_side(L):
    """Two decode calls and a prefill call on three streams, each with its workspace, over one cache."""
    lens, lq, nh, nkv = [3000, 500, 900], [30, 20, 1], 16, 8
    c = Paged(lens, nkv, I8, 64, 256, seed=2)
    d = c.cuda()
    qs = [torch.randn(3, nh, HD, generator=gen(i)).bfloat16() for i in range(2)]
    qp = torch.randn(sum(lq), nh, HD, generator=gen(9)).bfloat16()
    dev = [q.cuda() for q in qs] + [qp.cuda()]
    alone = [K._decode(L, d, dev[0], lens, nh, 0, 0), K._decode(L, d, dev[1], lens, nh, 256, 4),
             K._prefill(L, d, dev[2], lens, lq, nh, 0, 0)]
    sync_ok(L)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [None] * 3
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = (K._prefill(L, d, dev[2], lens, lq, nh, 0, 0) if i == 2 else
                          K._decode(L, d, dev[i], lens, nh, 0 if i == 0 else 256, 0 if i == 0 else 4))
        sync_ok(L)
        for a, b in zip(alone, got):
            assert torch.equal(a, b)


def test_negative_softmax_scale(L):
    lens, lq, nh, nkv = [150], [40], 4, 2
    c = Paged(lens, nkv, I8, 16, 64, seed=2)
    q = torch.randn(1, nh, HD, generator=gen(1)).bfloat16()
    out = K._decode(L, c.cuda(), q.cuda(), lens, nh, 0, 0, scale=-0.1)
    sync_ok(L)
    K._check_decode(out, c, q, lens, 0, 0, scale=-0.1)
    qp = torch.randn(40, nh, HD, generator=gen(2)).bfloat16()
    outp = torch.empty_like(qp, device="cuda")
    d = c.cuda()
    ws = torch.zeros(max(L.attention_prefill_kv8_workspace_size(1, 40, 40, 150, nh, nkv), 256), dtype=torch.uint8, device="cuda")
    L.attention_prefill_kv8(qp.cuda(), d.k, d.v, d.ks, d.vs, 16, torch.tensor([0, 40], dtype=torch.int32).cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), d.table, 64, 40, 150, nh, nkv, HD, -0.1, outp, ws)
    sync_ok(L)
    r = c.rows(0, 0, 150)
    o, tol = K.attend64(qp.double(), c.values("k", r), c.values("v", r), torch.arange(110, 150), -0.1, 0, 0)
    assert torch.all((outp.cpu().double() - o).abs() <= tol)


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("lens,lq,nh,nkv", [([1500, 1100, 1024], [7, 3, 1], 8, 2), ([1025], [16], 8, 1), ([5000, 1], [5, 1], 4, 4),
                                            ([1300] * 30, [2] * 30, 16, 8), ([9000], [64], 2, 1), ([1200, 900], [65, 12], 2, 1)])
@pytest.mark.parametrize("window,sink", [(0, 0), (700, 100), (64, 4)])
def test_prefill_few_rows(L, kv, lens, lq, nh, nkv, window, sink):
    """Few rows over many keys: the keys are split, and the parts added."""
    c = Paged(lens, nkv, kv, 32, 128, seed=3)
    q = torch.randn(sum(lq), nh, HD, generator=gen(4)).bfloat16()
    out = K._prefill(L, c.cuda(), q.cuda(), lens, lq, nh, window, sink)
    sync_ok(L)
    K._check_prefill(out, c, q, lens, lq, window, sink)


def test_prefill_few_rows_that_see_nothing(L):
    """As above, with sequences without keys and queries at negative positions."""
    lens, lq, nh, nkv = [3, 0, 2000], [6, 4, 5], 4, 2
    c = Paged(lens, nkv, I8, 16, 64, seed=1)
    q = torch.randn(sum(lq), nh, HD, generator=gen(5)).bfloat16()
    out = K._prefill(L, c.cuda(), q.cuda(), lens, lq, nh, 0, 0)
    sync_ok(L)
    assert torch.all(out[:3] == 0) and torch.all(out[6:10] == 0)
    K._check_prefill(out[3:6], c, q[3:6], [3], [3], 0, 0)
    d = Paged.__new__(Paged)
    d.__dict__.update(c.__dict__)
    d.table = c.table[2:]
    K._check_prefill(out[10:], d, q[10:], [2000], [5], 0, 0)


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("lens,lq", [([40, 300, 5], [200, 300, 9]), ([2000, 3], [12, 30])])
def test_largest_window_and_sink(L, lens, lq):
    """The largest window sees every key, and so does any window whose first tokens are all of them,
    also for queries at negative positions (which see nothing)."""
    nh, nkv = 8, 2
    c = Paged(lens, nkv, I8, 16, 64, seed=8)
    d = c.cuda()
    q = torch.randn(sum(lq), nh, HD, generator=gen(3)).bfloat16().cuda()
    qd = torch.randn(len(lens), nh, HD, generator=gen(4)).bfloat16().cuda()
    want, wantd = K._prefill(L, d, q, lens, lq, nh, 0, 0), K._decode(L, d, qd, lens, nh, 0, 0)
    sync_ok(L)
    K._check_decode(wantd, c, qd.cpu(), lens, 0, 0)
    at = 0
    for n, m in zip(lens, lq):
        assert torch.all(want[at:at + max(m - n, 0)] == 0)
        at += m
    for window, sink in ((BIG, 0), (BIG, BIG), (BIG - 1, 7), (1 << 30, 0)):
        assert torch.equal(K._prefill(L, d, q, lens, lq, nh, window, sink), want)
        assert torch.equal(K._decode(L, d, qd, lens, nh, window, sink), wantd)
    for window in (1, 70):   # (the tiles are dealt out in another order of sums)
        sink = K._decode(L, d, qd, lens, nh, window, BIG)
        K._check_decode(sink, c, qd.cpu(), lens, 0, 0)
        out = K._prefill(L, d, q, lens, lq, nh, window, BIG).cpu()
        at = 0
        for s, (n, m) in enumerate(zip(lens, lq)):
            skip = max(m - n, 0)
            assert torch.all(out[at:at + skip] == 0)
            one = K._only(c, s)
            K._check_prefill(out[at + skip:at + m], one, q[at + skip:at + m].cpu(), [n], [m - skip], 0, 0)
            at += m
    sync_ok(L)


def test_no_context_at_all(L):
    """max_context 0: every sequence is empty, every row zero."""
    nh, nkv, lens = 4, 2, [0, 0, 0]
    d = Paged(lens, nkv, E4, 16, 64, seed=8).cuda()
    q = torch.randn(3, nh, HD, generator=gen(3)).bfloat16().cuda()
    assert torch.all(K._decode(L, d, q, lens, nh, 0, 0) == 0)
    assert torch.all(K._prefill(L, d, q, lens, [1, 1, 1], nh, 0, 0) == 0)
    sync_ok(L)


def test_sequences_share_a_prefix(L):
    """Two sequences whose first pages are the same pages of the cache, each with its own last page."""
    nh, nkv, lens, lq = 8, 2, [200, 170, 190], [72, 42, 62]
    c = Paged(lens, nkv, I8, 16, 64, seed=9)
    c.table[1:, :2] = c.table[0, :2]
    q = torch.randn(3, nh, HD, generator=gen(3)).bfloat16()
    qp = torch.randn(sum(lq), nh, HD, generator=gen(4)).bfloat16()
    d = c.cuda()
    out, outp = K._decode(L, d, q.cuda(), lens, nh, 0, 0), K._prefill(L, d, qp.cuda(), lens, lq, nh, 0, 0)
    sync_ok(L)
    K._check_decode(out, c, q, lens, 0, 0)
    K._check_prefill(outp, c, qp, lens, lq, 0, 0)


def test_append_one_token_with_and_without_offsets(L):
    """Offsets of one token a sequence and none at all are the same call."""
    nh, nkv, lens = 8, 2, [70, 1, 64, 65, 33]
    qkv, qg, kg, pos = K._append_case(nh, nkv, 1, lens, [1] * 5, 8)
    cs = L.rope_cos_sin_table(80, HD, 1e6).cuda()
    got = []
    for cu in (None, torch.arange(6, dtype=torch.int32).cuda()):
        d = Paged(lens, nkv, I8, 32, 64, seed=3).cuda()
        q = torch.empty(5, nh, HD, dtype=torch.bfloat16, device="cuda")
        L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), cs, qg.cuda(), kg.cuda(), 1e-6, cu,
                     torch.tensor(lens, dtype=torch.int32).cuda(), d.table, 64, d.k, d.v, d.ks, d.vs, 32, q)
        sync_ok(L)
        got.append([q] + [t.view(torch.uint8) for t in (d.k, d.v, d.ks, d.vs)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
