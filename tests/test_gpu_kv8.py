"""The 8-bit paged KV cache on the GPU: append, read, decode and prefill
attention against plain float64 implementations.

Tolerances count roundings.  u = 2^-24 is half a step of fp32 relative to the
value, 2^-8 of bf16, 2^-4 of e4m3; an int8 code is off by at most half a scale.
"""
import numpy as np
import pytest
import torch

import seeded_inputs as si

pytestmark = pytest.mark.gpu

HD = 128
U = 2.0 ** -24
CMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
I8, E4 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_transformer_forward_gb300 import build
    build.build()
    from qwen3_transformer_forward_gb300 import _lib
    _lib.load()
    return _lib


def sync_ok(L):
    torch.cuda.synchronize()
    L.device_error()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes_to_f64(c):
    """Values of codes; the e4m3 patterns of NaN stand for +-480."""
    x = c.float().double()
    if c.dtype == E4:
        b = c.view(torch.uint8)
        x = torch.where(b == 0x7F, 480.0, torch.where(b == 0xFF, -480.0, x))
    return x


def pick(codes, rows):
    return codes.view(torch.uint8)[rows].view(codes.dtype)


class Paged:
    """A cache of shuffled pages; pages of no sequence hold garbage codes and NaN scales."""

    def __init__(self, lens, nkv, kv, sb, bs, seed=1, spare=2, capacity=0, wide=0.5):
        g = gen(seed)
        self.lens, self.nkv, self.kv, self.sb, self.bs = list(lens), nkv, kv, sb, bs
        need = [max(-(-(n + capacity) // bs), 0) for n in lens]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        self.max_blocks = max(max(need), 1)
        table = torch.full((len(lens), self.max_blocks), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.table = table
        slots = pages * bs
        raw = torch.randint(0, 256, (2, slots, nkv, HD), generator=g, dtype=torch.int32).to(torch.uint8)
        if kv == I8:
            raw[raw == 128] = 127    # -128 is no code
        scale = torch.exp(wide * torch.randn(2, slots // sb, nkv, generator=g)) / CMAX[kv]
        used = torch.zeros(slots // sb, dtype=torch.bool)
        for s, n in enumerate(lens):
            for p in range(0, n, sb):
                used[self.row(s, p) // sb] = True
        scale[:, ~used] = float("nan")
        if kv == E4:   # NaN patterns only where nothing may look
            live = used.repeat_interleave(sb)
            x = raw[:, live]
            x[(x & 0x7F) == 0x7F] = 0x30
            raw[:, live] = x
        self.k, self.v = (raw[i].view(kv) for i in range(2))
        self.ks, self.vs = scale[0].contiguous(), scale[1].contiguous()
        self.slots = slots

    def row(self, s, p):
        return int(self.table[s, p // self.bs]) * self.bs + p % self.bs

    def rows(self, s, a, b):
        p = torch.arange(a, b)
        return self.table[s, p // self.bs].long() * self.bs + p % self.bs

    def cuda(self):
        d = Paged.__new__(Paged)
        d.__dict__.update(self.__dict__)
        for n in ("k", "v", "ks", "vs", "table"):
            setattr(d, n, getattr(self, n).cuda())
        return d

    def values(self, which, rows):
        codes, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return codes_to_f64(pick(codes, rows)) * scale[rows // self.sb].double()[..., None]


def attend64(q, k, v, p, scale, window, sink):
    """q [n, nh, d] at key positions p [n] over k, v [L, nkv, d]: (out, tolerance), float64.

    Tolerance: the output's rounding, 2^-8 |o|; each weight is rounded to 11 bits
    (2^-11 at most, the sum of the weights is not), and its exponent is off by at
    most the error of a 128-term fp32 dot product with truncated sums, 128 * 2^-23
    of the sum of magnitudes, besides a few fp32 roundings: all relative to
    sum p |v| / l."""
    n, nh, _ = q.shape
    nkv, Lk = k.shape[1], k.shape[0]
    if Lk == 0:
        return torch.zeros(n, nh, HD, dtype=torch.float64), torch.zeros(n, nh, HD, dtype=torch.float64)
    G = nh // nkv
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    x = torch.einsum("ihd,jhd->hij", q, kk) * scale
    j = torch.arange(Lk)
    seen = j[None] <= p[:, None]
    if window:
        seen &= (j[None] > p[:, None] - window) | (j[None] < sink)
    x = x.masked_fill(~seen[None], -float("inf"))
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
    o = torch.einsum("hij,jhd->ihd", w, vv)
    mag = torch.einsum("ihd,jhd->hij", q.abs(), kk.abs()) * abs(scale)
    dx = 128 * 2.0 ** -23 * torch.where(seen[None], mag, torch.zeros_like(mag)).amax(-1)     # [h, i]
    a = torch.einsum("hij,jhd->ihd", w, vv.abs())
    return o, 2.0 ** -8 * o.abs() + a * (2.0 ** -11 + 16 * U + 2 * dx.T[..., None])


# ----------------------------------------------------------------------------
# read
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read(L, kv, dtype):
    c = Paged([70, 1], 3, kv, 16, 64, seed=3)
    rows = torch.cat([c.rows(0, 0, 70), c.rows(1, 0, 1), c.rows(0, 3, 5), torch.tensor([-1, c.slots, -2, 1 << 40])])
    d = c.cuda()
    ko = torch.full((rows.shape[0], 3, HD), 7.0, dtype=dtype, device="cuda")
    vo = torch.full_like(ko, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.kv8_read(d.k, d.v, d.ks, d.vs, 16, rows.cuda(), ko, vo, err)
    only_v = torch.empty_like(vo)
    L.kv8_read(d.k, d.v, d.ks, d.vs, 16, rows.cuda(), None, only_v)
    sync_ok(L)
    assert int(err) == 3                       # -1 asks for zeros, the other three are outside
    assert torch.equal(only_v, vo)
    for got, which in ((ko, "k"), (vo, "v")):
        codes, scale = (c.k, c.ks) if which == "k" else (c.v, c.vs)
        want = torch.zeros(rows.shape[0], 3, HD)
        want[:-4] = codes_to_f64(pick(codes, rows[:-4])).float() * scale[rows[:-4] // 16][..., None]
        assert torch.equal(got.cpu(), want.to(dtype))     # one fp32 product, one rounding


# ----------------------------------------------------------------------------
# append
# ----------------------------------------------------------------------------

def _half_step(y, scale, kv):
    """Half a step of the code nearest to y (the values between two codes are at most this far from one)."""
    return 0.5 * scale if kv == I8 else np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10 * scale)


def _append_case(nh, nkv, tp, lens, lq, seed, gamma=True, dtype=torch.bfloat16):
    g = gen(seed)
    T = sum(lq)
    qkv = torch.randn(T, (nh + 2 * nkv) * HD, generator=g).to(dtype)
    qg = (1 + 0.2 * torch.randn(HD, generator=g)).to(dtype)
    kg = (1 + 0.2 * torch.randn(HD, generator=g)).to(dtype)
    pos = torch.cat([torch.arange(n - q, n) for n, q in zip(lens, lq)] or [torch.zeros(0, dtype=torch.int64)])
    return qkv, qg, kg, pos


def _split(qkv, nh, nkv, tp):
    x = qkv.double().view(qkv.shape[0], tp, -1, HD)
    a, b = nh // tp, nkv // tp
    return (x[:, :, :a].reshape(-1, nh, HD), x[:, :, a:a + b].reshape(-1, nkv, HD), x[:, :, a + b:].reshape(-1, nkv, HD))


def _k64(k, gamma, cs, pos):
    n = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * gamma.double()
    c, s = cs[pos].double()[:, None].chunk(2, -1)
    a, b = n.chunk(2, -1)
    y = torch.cat([a * c - b * s, b * c + a * s], -1)
    # eleven additions of the sum of squares (halved by the square root), rsqrt
    # (two steps), two products, two products and a sum of the rotation: at most
    # 16 roundings of the two terms' magnitudes
    mag = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, 16 * U * torch.cat(mag, -1)


def _check_blocks(c0, c1, cache, scale0, scale1, y, y_tol, lens, lq, kv, what):
    """c0, c1: the cache before and after (numpy values of codes); y [T, nkv, d] the exact new values."""
    C = CMAX[kv]
    touched = np.zeros(c1.shape[0], bool)
    at = 0
    for s, (n, q) in enumerate(zip(lens, lq)):
        first = n - q
        for b in range(max(first, 0) // cache.sb, (n - 1) // cache.sb + 1) if q and n > 0 else ():
            a, e = b * cache.sb, min(n, (b + 1) * cache.sb)
            r = cache.rows(s, a, e).numpy()
            touched[r] = True
            blk = r[0] // cache.sb
            mid = max(a, first)
            new = y[at + mid - first:at + e - first]
            tol = y_tol[at + mid - first:at + e - first]
            top = np.abs(new).max((0, 2))
            want = top / C
            slack = tol.max((0, 2)) / C + 2 * U * want
            if mid > a:
                want = np.maximum(want, scale0[blk])
            assert np.all(np.abs(scale1[blk] - want) <= slack), (what, s, b)
            sc = scale1[blk][None, :, None]
            if mid > a:
                old = c0[r[:mid - a]] * scale0[blk][None, :, None]
                got = c1[r[:mid - a]] * sc
                grew = scale1[blk] > scale0[blk]
                err = np.abs(got - old)
                lim = _half_step(old, sc, kv) * (1 + 8 * U) + 8 * U * np.abs(old)
                assert np.all(err[:, grew] <= lim[:, grew]), (what, "old", s, b)
                assert np.array_equal(c1[r[:mid - a]][:, ~grew], c0[r[:mid - a]][:, ~grew]), (what, "kept", s, b)
            got = c1[r[mid - a:]] * sc
            # the nearest code of a value that is itself off by tol and two more
            # roundings; the largest value may sit past the last code by its own error
            lim = _half_step(new, sc, kv) + tol + 4 * U * np.abs(new) + slack[None, :, None] * C
            assert np.all(np.abs(got - new) <= lim), (what, "new", s, b)
        at += q
    assert np.array_equal(c1[~touched], c0[~touched]), (what, "rows of no new token's block")


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("nh,nkv,tp,sb,bs,lens,lq", [
    (16, 8, 1, 64, 256, [300, 1, 256, 257, 64, 65], [1] * 6),          # decode
    (16, 8, 2, 32, 64, [130, 45, 64], [130, 45, 64]),                  # whole prompts
    (6, 2, 1, 16, 64, [100, 33, 5, 81], [37, 2, 0, 49]),               # chunks inside blocks, one sequence waits
    (4, 4, 4, 64, 64, [200], [199]),
    (3, 1, 1, 16, 128, [16 * 40 + 3] + [17] * 40, [600] + [2] * 40),   # more than 32 sequences
])
def test_append(L, kv, nh, nkv, tp, sb, bs, lens, lq):
    c = Paged(lens, nkv, kv, sb, bs, seed=sum(lens), wide=0.3)
    c.ks = torch.where(torch.isnan(c.ks), c.ks, c.ks * 2.4)     # about a normal row's maximum: some blocks grow, some do not
    c.vs = torch.where(torch.isnan(c.vs), c.vs, c.vs * 2.4)
    qkv, qg, kg, pos = _append_case(nh, nkv, tp, lens, lq, 11)
    T, pad = sum(lq), 3
    full = torch.cat([qkv, torch.full((pad, qkv.shape[1]), float("nan"), dtype=qkv.dtype)])      # padded batch
    pos_full = torch.cat([pos, torch.full((pad,), -5)])
    cs = L.rope_cos_sin_table(max(lens) + 1, HD, 1e6)
    d = c.cuda()
    q = torch.full((T + pad, nh, HD), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    decode = all(x == 1 for x in lq)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lq)]), dtype=torch.int32).cuda()
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    L.kv8_append(full.cuda(), nh, nkv, HD, tp, pos_full.cuda(), cs.cuda(), qg.cuda(), kg.cuda(), 1e-6, None if decode else cu,
                 ctx, d.table, bs, d.k, d.v, d.ks, d.vs, sb, q, err)
    ref_q = torch.empty(T, nh, HD, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(4, nkv, HD, dtype=torch.bfloat16, device="cuda")
    L.qkv_norm_rope_store_kv(qkv.cuda(), nh, nkv, HD, tp, pos.cuda(), cs.cuda(), qg.cuda(), kg.cuda(), 1e-6,
                             torch.full((T,), -1).cuda(), kc, kc.clone(), ref_q)
    sync_ok(L)
    assert int(err) == 0
    assert torch.equal(q[:T], ref_q)                       # the same arithmetic, bit for bit
    assert torch.all(q[T:] == 7.0)                         # padding rows stay as they were
    _, k, v = _split(qkv, nh, nkv, tp)
    y, tol = _k64(k, kg, cs, pos)
    for which, val, val_tol in (("k", y, tol), ("v", v, torch.zeros_like(v))):
        a, b = (c.k, d.k) if which == "k" else (c.v, d.v)
        sa, sb_ = (c.ks, d.ks) if which == "k" else (c.vs, d.vs)
        _check_blocks(codes_to_f64(a).numpy(), codes_to_f64(b.cpu()).numpy(), c, sa.double().numpy(),
                      sb_.cpu().double().numpy(), val.numpy(), val_tol.numpy(), lens, lq, kv, which)


@pytest.mark.parametrize("kv", [I8, E4])
def test_append_is_the_same_twice_and_replayed(L, kv):
    """The same tokens again change nothing; a captured call gives what the call gave."""
    lens, lq, nkv, nh = [90, 40], [30, 40], 2, 4
    c = Paged(lens, nkv, kv, 32, 64, seed=9)
    qkv, qg, kg, pos = _append_case(nh, nkv, 1, lens, lq, 4)
    cs = L.rope_cos_sin_table(100, HD, 1e6).cuda()
    args = [t.cuda() for t in (qkv, pos, qg, kg)]
    cu, ctx = torch.tensor([0, 30, 70], dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()

    def call(d, q):
        L.kv8_append(args[0], nh, nkv, HD, 1, args[1], cs, args[2], args[3], 1e-6, cu, ctx, d.table, 64, d.k, d.v, d.ks, d.vs,
                     32, q)
    a, b = c.cuda(), c.cuda()
    b.k, b.v, b.ks, b.vs = (t.clone() for t in (b.k, b.v, b.ks, b.vs))
    qa = torch.empty(70, nh, HD, dtype=torch.bfloat16, device="cuda")
    qb = torch.empty_like(qa)
    call(a, qa)
    once = [t.clone() for t in (a.k.view(torch.uint8), a.v.view(torch.uint8), a.ks, a.vs, qa)]
    call(a, qa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(b, qb)
    for t, o in ((b.k, c.k), (b.v, c.v)):
        t.view(torch.uint8).copy_(o.view(torch.uint8))
    b.ks.copy_(c.ks)
    b.vs.copy_(c.vs)
    graph.replay()
    sync_ok(L)
    for d, q in ((a, qa), (b, qb)):
        for x, y in zip(once, (d.k.view(torch.uint8), d.v.view(torch.uint8), d.ks, d.vs, q)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))     # (spare blocks' scales are NaN)


def test_append_bad_tokens(L):
    """Positions outside the RoPE table, missing pages, padding sequences, values that are not finite."""
    kv, nh, nkv, sb, bs = I8, 2, 1, 16, 64
    lens = [20, 70, 0, 5]
    lq = [20, 10, 1, 5]
    c = Paged(lens, nkv, kv, sb, bs, seed=2)
    c.table[1, 1] = 99                                   # outside the cache: positions 64 .. 69 of sequence 1
    qkv, qg, kg, pos = _append_case(nh, nkv, 1, [20, 70, 1, 5], lq, 5)
    pos = pos.clone()
    pos[3] = 1000                                        # outside the table
    vcol = (nh + nkv) * HD
    qkv[0, vcol] = float("nan")
    qkv[1, vcol + 1] = float("inf")
    qkv[2, vcol + 2] = -float("inf")
    qkv[31:, vcol:] = 0                                  # sequence 3: v is all zero
    cs = L.rope_cos_sin_table(128, HD, 1e6).cuda()
    d = c.cuda()
    q = torch.full((36, nh, HD), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 30, 31, 36], dtype=torch.int32).cuda()
    L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), cs, qg.cuda(), kg.cuda(), 1e-6, cu,
                 torch.tensor(lens, dtype=torch.int32).cuda(), d.table, bs, d.k, d.v, d.ks, d.vs, sb, q, err)
    sync_ok(L)
    assert int(err) == 1 + 6
    assert torch.all(q[3] == 0) and not torch.isnan(q.float()).any()
    r = c.rows(0, 0, 20)
    vals = d.v.cpu()[r, 0].int()
    assert vals[0, 0] == 0 and vals[1, 1] == 127 and vals[2, 2] == -127
    fin = qkv[:16, vcol:].float()
    fin[3] = 0                                           # the bad position's v is stored as zeros
    fin = fin[torch.isfinite(fin)]
    assert float(d.vs[r[0] // sb, 0]) == float(fin.abs().max() / 127.0)
    assert torch.all(d.k.cpu()[r[3]] == 0) and torch.all(d.v.cpu()[r[3]] == 0)
    r3 = c.rows(3, 0, 5)
    assert torch.all(d.vs.cpu()[r3 // sb] == 0) and torch.all(d.v.cpu()[r3] == 0)
    live = torch.zeros(c.slots, dtype=torch.bool)
    for s, a, b in ((0, 0, 20), (1, 48, 64), (3, 0, 5)):
        live[c.rows(s, a, b)] = True
    assert torch.equal(d.k.cpu()[~live], c.k[~live]) and torch.equal(d.v.cpu()[~live], c.v[~live])


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------

def _decode(L, c, q, lens, nh, window, sink, max_context=None, scale=HD ** -0.5, ws=None, out=None, ctx=None):
    mc = max(lens) if max_context is None else max_context
    if ws is None:
        ws = torch.zeros(L.attention_decode_kv8_workspace_size(len(lens), mc, nh, c.nkv), dtype=torch.uint8, device="cuda")
    out = torch.full((len(lens), nh, HD), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    ctx = torch.tensor(lens, dtype=torch.int32).cuda() if ctx is None else ctx
    L.attention_decode_kv8(q, c.k, c.v, c.ks, c.vs, c.sb, ctx, c.table, c.bs, mc, nh, c.nkv, HD, scale, out, ws,
                           window=window, n_sink=sink)
    return out


def _check_decode(got, c, q, lens, window, sink, scale=HD ** -0.5):
    got = got.cpu().double()
    for s, n in enumerate(lens):
        r = c.rows(s, 0, n)
        o, tol = attend64(q[s:s + 1].double(), c.values("k", r), c.values("v", r), torch.tensor([n - 1]), scale, window, sink)
        if n == 0:
            assert torch.all(got[s] == 0)
            continue
        err = (got[s:s + 1] - o).abs()
        assert torch.all(err <= tol), (s, n, float((err / tol).max()))


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("nh,nkv,sb,bs,lens", [
    (16, 8, 64, 256, [1, 300, 2049, 256, 257, 0, 64, 63, 65]),
    (8, 1, 16, 64, [777, 16, 15, 17]),
    (6, 2, 32, 128, [129, 1000]),
    (5, 1, 16, 64, [40, 3]),
    (16, 1, 64, 64, [513]),
    (3, 3, 32, 64, [9000]),
    (2, 2, 64, 256, [0, 0]),
    (64, 16, 16, 64, [100] * 20),
])
@pytest.mark.parametrize("window,sink", [(0, 0), (1, 0), (100, 4), (64, 70), (33, 0), (5000, 16)])
def test_decode(L, kv, nh, nkv, sb, bs, lens, window, sink):
    c = Paged(lens, nkv, kv, sb, bs, seed=len(lens) + window)
    q = torch.randn(len(lens), nh, HD, generator=gen(5)).bfloat16()
    out = _decode(L, c.cuda(), q.cuda(), lens, nh, window, sink, max_context=c.max_blocks * bs)
    sync_ok(L)
    _check_decode(out, c, q, lens, window, sink)


@pytest.mark.parametrize("kv", [I8, E4])
def test_decode_scales_of_many_sizes(L, kv):
    """Block scales over 2^-90 .. 2^20, zero blocks, queries of extreme sizes: the weights keep their precision."""
    lens, nkv, nh, sb = [700, 333], 2, 8, 16
    c = Paged(lens, nkv, kv, sb, 64, seed=4)
    g = gen(8)
    c.vs = torch.where(torch.isnan(c.vs), c.vs, torch.exp2(torch.randint(-90, 20, c.vs.shape, generator=g).float()))
    c.ks = torch.where(torch.isnan(c.ks), c.ks, c.ks * torch.exp2(torch.randint(-6, 2, c.ks.shape, generator=g).float()))
    for t in (c.ks, c.vs):
        t[(torch.rand(t.shape, generator=g) < 0.2) & ~torch.isnan(t)] = 0.0
    q = torch.randn(2, nh, HD, generator=g).bfloat16()
    q[0, 0] *= 2.0 ** 30
    q[0, 1] *= 2.0 ** -40
    q[1, 2] = 0
    out = _decode(L, c.cuda(), q.cuda(), lens, nh, 0, 0)
    sync_ok(L)
    _check_decode(out, c, q, lens, 0, 0)


def test_decode_all_scales_zero(L):
    c = Paged([100], 2, I8, 32, 64, seed=6)
    c.ks.zero_()
    c.vs.zero_()
    out = _decode(L, c.cuda(), torch.randn(1, 4, HD).bfloat16().cuda(), [100], 4, 0, 0)
    sync_ok(L)
    assert torch.all(out == 0)


def test_missing_pages_read_as_zeros(L):
    """A page outside the cache or below zero counts as zero keys and values, like the bf16 paged cache."""
    lens, nkv, nh = [300, 200], 2, 4
    c = Paged(lens, nkv, I8, 32, 64, seed=6)
    q = torch.randn(2, nh, HD, generator=gen(1)).bfloat16()
    d = c.cuda()
    d.table[0, 1] = -1
    d.table[1, 2] = 10 ** 6
    out = _decode(L, d, q.cuda(), lens, nh, 0, 0).cpu().double()
    sync_ok(L)
    for s, (a, b) in enumerate(((64, 128), (128, 192))):
        r = c.rows(s, 0, lens[s])
        k, v = c.values("k", r), c.values("v", r)
        k[a:b] = 0
        v[a:b] = 0
        o, tol = attend64(q[s:s + 1].double(), k, v, torch.tensor([lens[s] - 1]), HD ** -0.5, 0, 0)
        assert torch.all((out[s:s + 1] - o).abs() <= tol)


def test_decode_overlong_context_is_reported(L):
    """Keys past max_context are not read; qw_device_error says so once."""
    c = Paged([300, 50], 2, I8, 32, 64, seed=6)
    q = torch.randn(2, 4, HD, generator=gen(1)).bfloat16()
    out = _decode(L, c.cuda(), q.cuda(), [300, 50], 4, 0, 0, max_context=128)
    torch.cuda.synchronize()
    with pytest.raises(L.QwError) as e:
        L.device_error()
    assert e.value.code == L.QW_ERR_INVALID_ARG
    L.device_error()
    _check_decode(out[1:], _only(c, 1), q[1:], [50], 0, 0)


def _only(c, s):
    d = Paged.__new__(Paged)
    d.__dict__.update(c.__dict__)
    d.table = c.table[s:s + 1]
    return d


def test_decode_graphs_share_a_workspace(L):
    """Two captured calls on one workspace, replayed in turn with new lengths, queries and another stream."""
    cap, nh, nkv = [2000, 900, 1400, 64], 16, 8
    c = Paged(cap, nkv, I8, 64, 256, seed=3)
    d = c.cuda()
    ws = torch.zeros(L.attention_decode_kv8_workspace_size(4, 2000, nh, nkv), dtype=torch.uint8, device="cuda")
    ctx = torch.tensor(cap, dtype=torch.int32).cuda()
    q = torch.zeros(4, nh, HD, dtype=torch.bfloat16, device="cuda")
    outs, graphs = [], []
    for window, sink in ((0, 0), (130, 4)):
        out = torch.empty_like(q)
        _decode(L, d, q, cap, nh, window, sink, 2000, ws=ws, out=out, ctx=ctx)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            _decode(L, d, q, cap, nh, window, sink, 2000, ws=ws, out=out, ctx=ctx)
        outs.append(out)
        graphs.append(gr)
    side = torch.cuda.Stream()
    for trial, lens in enumerate(([2000, 900, 1400, 64], [1, 0, 777, 64], [1999, 3, 128, 1])):
        qh = torch.randn(4, nh, HD, generator=gen(trial)).bfloat16()
        q.copy_(qh)
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for gr in graphs:
                gr.replay()
        torch.cuda.current_stream().wait_stream(side)
        sync_ok(L)
        for out, (window, sink) in zip(outs, ((0, 0), (130, 4))):
            _check_decode(out, c, qh, lens, window, sink)
        assert int(ws[:64 * 1024].to(torch.int32).sum()) == 0        # counters are back at zero


def test_decode_is_deterministic(L):
    lens, nh, nkv = [5000, 33, 2500], 16, 4
    c = Paged(lens, nkv, E4, 16, 64, seed=3).cuda()
    q = torch.randn(3, nh, HD, generator=gen(2)).bfloat16().cuda()
    first = _decode(L, c, q, lens, nh, 0, 0)
    for _ in range(20):
        assert torch.equal(first, _decode(L, c, q, lens, nh, 0, 0))
    sync_ok(L)


def _prefill(L, c, q, lens, lq, nh, window, sink, max_q=None, max_context=None, out=None, ws=None):
    mq = max(lq) if max_q is None else max_q
    mc = max(max(lens), 0) if max_context is None else max_context
    n = L.attention_prefill_kv8_workspace_size(len(lens), q.shape[0], mq, mc, nh, c.nkv)
    if ws is None:
        ws = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    out = torch.full(tuple(q.shape), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lq)]), dtype=torch.int32).cuda()
    L.attention_prefill_kv8(q, c.k, c.v, c.ks, c.vs, c.sb, cu, torch.tensor(lens, dtype=torch.int32).cuda(), c.table, c.bs, mq,
                            mc, nh, c.nkv, HD, HD ** -0.5, out, ws, window=window, n_sink=sink)
    return out


def _check_prefill(got, c, q, lens, lq, window, sink):
    got = got.cpu().double()
    at = 0
    for s, (n, m) in enumerate(zip(lens, lq)):
        r = c.rows(s, 0, n)
        o, tol = attend64(q[at:at + m].double(), c.values("k", r), c.values("v", r), torch.arange(n - m, n), HD ** -0.5, window,
                          sink)
        err = (got[at:at + m] - o).abs()
        bad = err > tol
        assert not bad.any(), (s, n, m, int(bad.sum()), [int(i) for i in bad.nonzero()[0]], float(err.max()))
        at += m


@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("nh,nkv,sb,bs,lens,lq", [
    (16, 8, 64, 256, [600, 130, 256, 1], [90, 130, 1, 1]),
    (4, 1, 16, 64, [1024, 300], [1024, 44]),
    (6, 2, 32, 128, [129, 500, 7], [129, 250, 0]),
    (5, 1, 16, 64, [200, 64], [77, 64]),
    (16, 1, 64, 64, [333], [33]),
    (2, 2, 32, 64, [700], [513]),
    (16, 8, 64, 256, [6000], [3]),
    (1, 1, 64, 64, [300, 300, 300], [256, 257, 255]),
])
@pytest.mark.parametrize("window,sink", [(0, 0), (1, 0), (100, 4), (64, 200), (300, 0)])
def test_prefill(L, kv, nh, nkv, sb, bs, lens, lq, window, sink):
    c = Paged(lens, nkv, kv, sb, bs, seed=len(lens) + window)
    T, pad = sum(lq), 2
    q = torch.randn(T, nh, HD, generator=gen(5)).bfloat16()
    full = torch.cat([q, torch.full((pad, nh, HD), float("nan"), dtype=torch.bfloat16)])
    out = _prefill(L, c.cuda(), full.cuda(), lens, lq, nh, window, sink)
    sync_ok(L)
    assert torch.all(out[T:] == 7.0)                 # rows of no sequence stay as they were
    _check_prefill(out[:T], c, q, lens, lq, window, sink)


def test_prefill_rows_that_see_nothing(L):
    """More new tokens than keys: the first queries sit at negative key positions and see nothing."""
    lens, lq, nh, nkv = [5, 0, 40], [9, 3, 40], 4, 2
    c = Paged(lens, nkv, I8, 16, 64, seed=1)
    q = torch.randn(sum(lq), nh, HD, generator=gen(5)).bfloat16()
    out = _prefill(L, c.cuda(), q.cuda(), lens, lq, nh, 0, 0)
    sync_ok(L)
    assert torch.all(out[:4] == 0) and torch.all(out[9:12] == 0)
    _check_prefill(out[4:9], c, q[4:9], [5], [5], 0, 0)


@pytest.mark.parametrize("kv", [I8, E4])
def test_prefill_scales_of_many_sizes(L, kv):
    lens, lq, nh, nkv = [900], [300], 8, 2
    c = Paged(lens, nkv, kv, 16, 64, seed=4)
    g = gen(8)
    c.vs = torch.where(torch.isnan(c.vs), c.vs, torch.exp2(torch.randint(-90, 20, c.vs.shape, generator=g).float()))
    c.ks = torch.where(torch.isnan(c.ks), c.ks, c.ks * torch.exp2(torch.randint(-6, 2, c.ks.shape, generator=g).float()))
    for t in (c.ks, c.vs):
        t[(torch.rand(t.shape, generator=g) < 0.2) & ~torch.isnan(t)] = 0.0
    q = torch.randn(300, nh, HD, generator=g).bfloat16()
    q[7, 0] *= 2.0 ** 30
    q[8, 1] *= 2.0 ** -40
    q[9] = 0
    out = _prefill(L, c.cuda(), q.cuda(), lens, lq, nh, 0, 0)
    sync_ok(L)
    _check_prefill(out, c, q, lens, lq, 0, 0)


def test_prefill_one_token_is_decode(L):
    """One query per sequence: prefill and decode agree within both tolerances, windows included."""
    lens, nh, nkv = [1, 500, 64, 2000], 8, 2
    c = Paged(lens, nkv, E4, 32, 128, seed=4)
    q = torch.randn(4, nh, HD, generator=gen(3)).bfloat16()
    for window, sink in ((0, 0), (90, 5)):
        a = _prefill(L, c.cuda(), q.cuda(), lens, [1] * 4, nh, window, sink)
        sync_ok(L)
        _check_decode(a, c, q, lens, window, sink)


# ----------------------------------------------------------------------------
# together: a prompt, a second chunk over the cached prefix, then decode steps
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kv", [I8, E4])
@pytest.mark.parametrize("window,sink", [(0, 0), (50, 3)])
def test_serve(L, kv, window, sink):
    nh, nkv, sb, bs, steps = 8, 2, 32, 64, 20
    prompt, chunk = [100, 33, 64], [40, 1, 77]
    total = [a + b for a, b in zip(prompt, chunk)]
    c = Paged([0, 0, 0], nkv, kv, sb, bs, seed=1, capacity=max(total) + steps)
    d = c.cuda()
    cs = L.rope_cos_sin_table(max(total) + steps, HD, 1e6).cuda()
    gam = torch.ones(HD, dtype=torch.bfloat16, device="cuda")
    mc = max(total) + steps
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(L.attention_decode_kv8_workspace_size(3, mc, nh, nkv), dtype=torch.uint8, device="cuda")
    exact = [torch.zeros(0, nkv, HD, dtype=torch.float64)] * 3     # v as given, for the distance to the bf16 answer

    def step(lens, lq, seed, decode):
        qkv, _, _, pos = _append_case(nh, nkv, 1, lens, lq, seed)
        v = _split(qkv, nh, nkv, 1)[2]
        at = 0
        for s, m in enumerate(lq):
            exact[s] = torch.cat([exact[s], v[at:at + m]])
            at += m
        q = torch.empty(sum(lq), nh, HD, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lq)]), dtype=torch.int32).cuda()
        ctx = torch.tensor(lens, dtype=torch.int32).cuda()
        L.kv8_append(qkv.cuda(), nh, nkv, HD, 1, pos.cuda(), cs, gam, gam, 1e-6, None if decode else cu, ctx, d.table, bs, d.k,
                     d.v, d.ks, d.vs, sb, q, err)
        out = _decode(L, d, q, lens, nh, window, sink, mc, ws=ws, ctx=ctx) if decode else _prefill(
            L, d, q, lens, lq, nh, window, sink, max_context=mc)
        sync_ok(L)
        h = d.cuda()
        for n in ("k", "v", "ks", "vs", "table"):
            setattr(h, n, getattr(d, n).cpu())
        (_check_decode if decode else lambda o, c_, q_, a, w, s_: _check_prefill(o, c_, q_, a, lq, w, s_))(
            out, h, q.cpu(), lens, window, sink)
        # what the cache stands for is near what was appended: a code's half step, and half a step for each time its
        # block's scale grew (tokens come at most 1 + 1 + steps times into a block), of the block's last scale
        for s, n in enumerate(lens):
            r = h.rows(s, 0, n)
            got, sc = h.values("v", r), h.vs[r // sb].double()[..., None]
            step_ = sc * (0.5 if kv == I8 else 16.0)      # e4m3: half a step of the top binade is 16 scales
            assert torch.all((got - exact[s]).abs() <= step_ * (2 + steps))
    step(prompt, prompt, 1, False)
    step(total, chunk, 2, False)
    for t in range(steps):
        step([n + t + 1 for n in total], [1, 1, 1], 10 + t, True)
    assert int(err) == 0
