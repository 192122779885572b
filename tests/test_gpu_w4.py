"""4-bit weights on the GPU: quantiser, embedding, linear layers and lm_head
against plain float64 implementations.

A weight is the bf16 number round((n - z) * s), so the quantiser's codes, the
embedding and every weight that a product uses are exact; only sums and the last
rounding are not.  Sums: bf16 products are exact in fp32, and a sum of K of them in
any order errs by at most K * 2^-23 * sum |x w| (2^-23: matrix instructions may cut
off instead of rounding; u = 2^-24 for the rest is inside it).  The output's rounding
adds 2^-8 relative (bf16, half a step is 2^-9 of the value's upper power of two, at
most 2^-8 of the value).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PLACE = (0, 4, 1, 5, 2, 6, 3, 7)
NONE, SILU = 0, 1
COL, ROW = 0, 1


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_transformer_forward_gb300 import build
    build.build()
    from qwen3_transformer_forward_gb300 import _lib
    _lib.load()
    return _lib


def gen(seed):
    return torch.Generator().manual_seed(seed)


def put(n):
    """Codes [N, K] as bytes [N, K/2], by plain loops over the nibbles."""
    n = n.to(torch.int64).view(n.shape[0], -1, 8)
    w = sum(n[:, :, j] << (4 * p) for j, p in enumerate(PLACE))
    return torch.stack([(w >> (8 * b)) & 255 for b in range(4)], -1).to(torch.uint8).reshape(n.shape[0], -1)


def values(n, s, z, group):
    """The weights in float64."""
    n = n.double().view(n.shape[0], -1, group)
    z = torch.full(s.shape, 8.0).double() if z is None else z.double()
    return ((n - z[..., None]) * s.double()[..., None]).bfloat16().double().view(n.shape[0], -1)


def matrix(N, K, group, zeros, seed=1):
    """Random codes, scales of mixed size (a zero one among them) and zero points; their values."""
    g = gen(seed)
    n = torch.randint(0, 16, (N, K), generator=g)
    s = (0.02 * torch.exp(0.7 * torch.randn(N, K // group, generator=g))).bfloat16()
    s[0, 0] = 0.0
    s[-1, -1] = -s[-1, -1]
    z = torch.randint(0, 16, (N, K // group), generator=g).to(torch.uint8) if zeros else None
    return put(n).cuda(), s.cuda(), None if z is None else z.cuda(), values(n, s, z, group)


def sync_ok(L):
    torch.cuda.synchronize()
    L.device_error()


def near(got, ref, absolute, what):
    """|got - ref| <= 2^-8 |ref| + absolute, NaN and infinities nowhere."""
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() > 2.0 ** -8 * ref.abs() + absolute
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3])


def product(x, w):
    """(x w^T, bound on the error of its fp32 sum)"""
    return x @ w.T, x.shape[1] * 2.0 ** -23 * (x.abs() @ w.abs().T)


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------

def quantize_ref(w, group, zeros):
    x = w.double().view(w.shape[0], -1, group)
    x = torch.where(torch.isnan(x), 0.0, x)
    f = torch.where(torch.isinf(x), 0.0, x)
    lo, hi = f.amin(-1).clamp(max=0.0), f.amax(-1).clamp(min=0.0)
    s = (((hi - lo) / 15.0) if zeros else torch.maximum(hi, -lo) / 7.0).bfloat16()
    d = torch.where(s == 0, 1.0, s.double())[..., None]
    z = torch.round(-lo[..., None] / d).clamp(max=15) if zeros else torch.full_like(d, 8.0)
    n = torch.clamp(torch.round(x / d) + z, 0, 15)
    return n.view(w.shape), s, z[..., 0].to(torch.uint8) if zeros else None


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (3, 64, 64), (5, 128, 128), (37, 96, 32), (129, 1088, 64), (64, 1152, 128)])
def test_quantize(L, N, K, group, zeros):
    g = gen(N + K)
    w = torch.randn(N, K, generator=g).bfloat16()
    w[0, :group] = 0.0                                            # an empty group
    if N > 3:
        w[1, :group] = torch.arange(group).remainder(16).sub(8).bfloat16()   # ties and both ends
        w[1, 0] = 7.0
        w[2, :group] = w[2, :group].abs()                         # one sign
        w[3, :group] = -w[3, :group].abs()
    if N > 30:
        w[4, 3], w[4, 5], w[4, 7] = float("nan"), float("inf"), float("-inf")
        w[5, :group] = float("nan")
        w[6, :group] = float("inf")
        w[7] = (w[7].float() * 2.0 ** -126).bfloat16()            # subnormal weights and scales
        w[8] = (w[8].float() * 2.0 ** -133).bfloat16()
        w[9] = (w[9].float().clamp(-3, 3) * 2.0 ** 126).bfloat16()   # hi - lo past the largest fp32
        w[10] = (w[10].float().round() + 0.5 * torch.randint(0, 2, (K,), generator=g)).bfloat16()
        w[10, ::group] = 7.0                                      # scale 1: many exact halves
    n, s, z = quantize_ref(w, group, zeros)
    codes = torch.full((N, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // group), float("nan"), dtype=torch.bfloat16, device="cuda")
    zs = torch.full((N, K // group), 99, dtype=torch.uint8, device="cuda") if zeros else None
    L.w4_quantize(w.cuda(), group, codes, scales, zs)
    sync_ok(L)
    assert torch.equal(scales.cpu(), s)
    if zeros:
        assert torch.equal(zs.cpu(), z)
    assert torch.equal(codes.cpu(), put(n))


@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_every_quotient(L, zeros):
    """Every pair of 8-bit significands: w = a * 2^i against the scale that a group's largest weight b gives it,
    ties among them.  A group holds one b (its negative too, asymmetric) and 31 of the a."""
    a = torch.arange(128, 256).double()
    w = []
    for i in range(-5, 1):
        x = (a * 2.0 ** i)[None, :].expand(128, 128)
        b = (a * 2.0)[:, None]                                     # the largest of its group
        x = torch.minimum(x, b)
        for part in (x[:, 0:30], x[:, 30:60], x[:, 60:90], x[:, 90:120], x[:, 98:128]):
            sign = torch.where(torch.arange(30) % 2 == 0, 1.0, -1.0) if i % 2 else torch.ones(30)
            for low in ((0.0, 0.25, 1.0) if zeros else (0.0,)):
                w.append(torch.cat([b, -low * b, part * sign], 1))
    w = torch.cat(w).bfloat16()
    n, s, z = quantize_ref(w, 32, zeros)
    N = w.shape[0]
    codes = torch.empty(N, 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, 1, dtype=torch.bfloat16, device="cuda")
    zs = torch.empty(N, 1, dtype=torch.uint8, device="cuda") if zeros else None
    L.w4_quantize(w.cuda(), 32, codes, scales, zs)
    sync_ok(L)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu(), put(n))
    if zeros:
        assert torch.equal(zs.cpu(), z)


def test_quantize_error_is_half_a_step(L):
    """Each weight within half a scale, and the clamp of the rounded scale, of what it was."""
    w = torch.randn(64, 1024, generator=gen(2)).bfloat16()
    for zeros in (False, True):
        c, s = torch.empty(64, 512, dtype=torch.uint8, device="cuda"), torch.empty(64, 8, dtype=torch.bfloat16, device="cuda")
        z = torch.empty(64, 8, dtype=torch.uint8, device="cuda") if zeros else None
        out = torch.empty(64, 1024, dtype=torch.bfloat16, device="cuda")
        L.w4_quantize(w.cuda(), 128, c, s, z)
        L.w4_embed_vocab(torch.arange(64, device="cuda"), c, s, z, 128, 1, out)
        sync_ok(L)
        step = s.double().cpu().repeat_interleave(128, 1)
        # half a step; the zero point's rounding moves both ends by another half; the scale, 2^-9 below what
        # it should be, leaves 15 * 2^-9 of a step at the ends; the value is rounded to bf16
        allowed = (1.0 if zeros else 0.5) + 15 * 2.0 ** -9
        assert ((out.double().cpu() - w.double()).abs() <= allowed * step + 2.0 ** -8 * w.double().abs()).all()


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("V,H,group,tp,T", [(8, 32, 32, 2, 1), (100, 64, 64, 4, 33), (1000, 1152, 128, 1, 257),
                                            (50, 2080, 32, 2, 9), (512, 1024, 64, 1, 1000)])
def test_embed(L, V, H, group, tp, T, zeros):
    c, s, z, w = matrix(V, H, group, zeros)
    ids = torch.randint(0, V, (T,), generator=gen(T))
    ids[0], ids[-1] = V - 1, 0
    if T > 4:
        ids[1], ids[2], ids[3] = -1, V, 2 ** 40
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.w4_embed_vocab(ids.cuda(), c, s, z, group, tp, out, err)
    sync_ok(L)
    ok = (ids >= 0) & (ids < V)
    ref = torch.where(ok[:, None], w[ids.clamp(0, V - 1)], 0.0)
    assert torch.equal(out.double().cpu(), ref)
    assert not torch.signbit(out[~ok.cuda()]).any()
    assert int(err) == int((~ok).sum())


# ---------------------------------------------------------------------------
# linear layers
# ---------------------------------------------------------------------------

def run_gemm(L, x, c, s, z, N, group, tp, mode, epi, stream=None):
    M = x.shape[0]
    out = torch.full((M, N // 2 if epi == SILU else N), float("nan"), dtype=torch.bfloat16, device="cuda")
    size = L.w4_gemm_workspace_size(M, N, x.shape[1], tp, mode, epi)
    ws = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
    L.w4_gemm(x, c, s, z, out, N, group, tp, mode, epi, ws if size else None, stream)
    return out


def check_gemm(L, M, N, K, group, zeros, tp, mode, epi, x=None, seed=1):
    shards = tp if mode == ROW else 1
    c, s, z, w = matrix(shards * N, K // shards, group, zeros, seed)
    if x is None:
        x = torch.randn(M, K, generator=gen(seed + M)).bfloat16()
        x[:, :3] *= 30.0
    out = run_gemm(L, x.cuda(), c, s, z, N, group, tp, mode, epi)
    sync_ok(L)
    x64 = x.double()
    if mode == ROW:
        w = w.view(tp, N, -1).permute(1, 0, 2).reshape(N, K)
    y, e = product(x64, w)
    if epi == SILU:
        (g, u), (eg, eu) = y.view(M, tp, 2, -1).unbind(2), e.view(M, tp, 2, -1).unbind(2)
        a = g * torch.sigmoid(g)
        # |silu'| <= 1.1; exp and the division cost a few fp32 steps of the value
        y, e = (a * u).reshape(M, -1), (1.1 * eg * (u.abs() + eu) + a.abs() * eu + 2.0 ** -20 * (a * u).abs()).reshape(M, -1)
    near(out, y, e, (M, N, K, group, zeros, tp, mode, epi))
    return out


SHAPES = [
    (1, 1, 32, 32, 1, COL, NONE), (1, 16, 64, 64, 1, COL, NONE), (3, 17, 96, 32, 1, COL, NONE),
    (8, 250, 128, 128, 2, COL, NONE), (9, 100, 160, 32, 1, COL, NONE), (16, 4096, 1024, 128, 2, COL, NONE),
    (5, 33, 256, 32, 8, ROW, NONE), (1, 1000, 1536, 128, 3, ROW, NONE), (20, 77, 352, 32, 11, ROW, NONE),
    (2, 16, 64, 32, 1, COL, SILU), (7, 96, 320, 64, 2, COL, SILU), (33, 480, 384, 128, 3, COL, SILU),
    (64, 515, 1024, 64, 1, COL, NONE), (65, 130, 224, 32, 1, COL, NONE), (127, 384, 512, 128, 2, ROW, NONE),
    (130, 272, 640, 64, 1, COL, SILU), (200, 1001, 288, 32, 3, ROW, NONE), (300, 640, 1152, 128, 2, COL, SILU),
    (257, 129, 96, 32, 1, COL, NONE), (513, 768, 2048, 128, 4, COL, NONE), (1000, 1024, 96, 32, 1, COL, SILU),
    # more tiles than pairs of SMs, and K (or its shards) that ends inside 128 columns, or is shorter
    (1999, 3001, 320, 64, 1, COL, NONE), (1500, 2500, 320, 32, 10, ROW, NONE), (1500, 2500, 576, 64, 3, ROW, NONE),
    (2100, 4096, 448, 64, 2, COL, SILU), (1200, 4000, 32, 32, 1, COL, NONE),
    # few tiles over a long K, whose parts end inside and between shards
    (70, 500, 3200, 64, 5, ROW, NONE), (90, 1000, 4096, 128, 1, COL, NONE), (128, 4600, 1664, 128, 1, COL, NONE),
    (190, 256, 5760, 32, 9, ROW, NONE), (100, 2240, 2080, 32, 5, COL, SILU), (180, 7000, 1408, 128, 1, COL, NONE),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group,tp,mode,epi", SHAPES)
def test_gemm(L, M, N, K, group, tp, mode, epi, zeros):
    check_gemm(L, M, N, K, group, zeros, tp, mode, epi)


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 32, 33, 48, 64, 65, 96, 128, 129, 192, 255, 256, 257, 384, 511])
def test_gemm_every_count_of_tokens(L, M):
    check_gemm(L, M, 336, 1024, 64, M % 2 == 0, 1, COL, SILU if M % 3 == 0 else NONE)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_single_weights(L, M):
    """One-hot activations pick single weights out: exact, every column and row."""
    N, K = 48, 256
    c, s, z, w = matrix(N, K, 32, True, seed=9)
    for k0 in range(0, K, M):
        x = torch.zeros(M, K)
        for m in range(M):
            x[m, (k0 + m) % K] = 1.0
        out = run_gemm(L, x.bfloat16().cuda(), c, s, z, N, 32, 1, COL, NONE)
        sync_ok(L)
        assert torch.equal(out.double().cpu(), x.double() @ w.T)


@pytest.mark.parametrize("M", [4, 200])
def test_gemm_rows_do_not_mix(L, M):
    """NaN and infinities stay in their token's row, and a NaN scale in its output column."""
    N, K = 80, 256
    c, s, z, w = matrix(N, K, 64, False, seed=4)
    x = torch.randn(M, K, generator=gen(3)).bfloat16()
    clean = run_gemm(L, x.cuda(), c, s, z, N, 64, 1, COL, NONE)
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    s2 = s.clone()
    s2[11, 1] = float("nan")
    out = run_gemm(L, x.cuda(), c, s2, z, N, 64, 1, COL, NONE)
    sync_ok(L)
    keep_r = torch.tensor([m for m in range(M) if m not in (1, 2)], device="cuda")
    keep_c = torch.tensor([n for n in range(N) if n != 11], device="cuda")
    assert torch.equal(out[keep_r][:, keep_c], clean[keep_r][:, keep_c])
    assert torch.isnan(out[:, 11]).all() and torch.isnan(out[1]).all()
    ref = torch.tensor(float("inf")) * torch.sign(w[:, 7])
    got = out[2].float().cpu()
    assert torch.equal(torch.isnan(got[keep_c.cpu()]), torch.isnan(ref[keep_c.cpu()]))
    fin = ~torch.isnan(ref) & (torch.arange(N) != 11)
    assert torch.equal(got[fin], ref[fin].float())


@pytest.mark.parametrize("M", [1, 8, 24, 64, 100, 300])
def test_gemm_same_results_again_and_as_rows_alone(L, M):
    """No dependence on timing: a call repeated gives the same bits."""
    c, s, z, _ = matrix(512, 2048, 128, True, seed=6)
    x = torch.randn(M, 2048, generator=gen(8)).bfloat16().cuda()
    first = run_gemm(L, x, c, s, z, 512, 128, 1, COL, NONE)
    for _ in range(5):
        assert torch.equal(run_gemm(L, x, c, s, z, 512, 128, 1, COL, NONE), first)
    sync_ok(L)


@pytest.mark.parametrize("M", [1, 30, 150])
def test_gemm_large_and_small_numbers(L, M):
    """Scales and activations near the ends of bf16, subnormal weights among them."""
    N, K = 32, 128
    g = gen(12)
    n = torch.randint(0, 16, (N, K), generator=g)
    s = torch.full((N, K // 32), 1.0)
    s[:8], s[8:16], s[16:24] = 2.0 ** -131, 2.0 ** 100, 2.0 ** -60
    x = torch.randn(M, K, generator=g)
    x[0] *= 2.0 ** 20
    s, x = s.bfloat16(), x.bfloat16()
    out = run_gemm(L, x.cuda(), put(n).cuda(), s.cuda(), None, N, 32, 1, COL, NONE)
    sync_ok(L)
    y, e = product(x.double(), values(n, s, None, 32))
    # sums near 2^-126 are held in steps of 2^-149 (products there too), and bf16 has steps of 2^-133
    near(out, y, e + K * 2.0 ** -149 + 2.0 ** -133, M)


def test_gemm_leaves_its_surroundings(L):
    """Rows before and after the output, and the inputs, stay as they were."""
    N, K = 51, 96
    c, s, z, _ = matrix(N, K, 32, True)
    for M in (1, 13, 70, 260):
        buf = torch.full((M + 16, N), 7.0, dtype=torch.bfloat16, device="cuda")
        x = torch.randn(M, K, generator=gen(M)).bfloat16().cuda()
        keep = [t.clone() for t in (x, c, s, z)]
        L.w4_gemm(x, c, s, z, buf[8:8 + M], N, 32)   # 8 rows of 51: a 16-byte aligned start
        sync_ok(L)
        assert (buf[:8] == 7.0).all() and (buf[8 + M:] == 7.0).all()
        assert all(torch.equal(a, b) for a, b in zip(keep, (x, c, s, z)))


# ---------------------------------------------------------------------------
# lm_head
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,T,V,H,group,tp,last", [(1, 1, 1000, 256, 64, 2, False), (5, 40, 1003, 128, 32, 1, True),
                                                   (8, 8, 4100, 1024, 128, 4, False), (70, 300, 2050, 320, 64, 2, True),
                                                   (130, 131, 515, 96, 32, 1, True)])
def test_lm_head(L, n, T, V, H, group, tp, last):
    c, s, z, w = matrix(V, H, group, n % 2 == 0)
    h = torch.randn(T, H, generator=gen(n)).bfloat16()
    idx = torch.randint(0, T, (n,), generator=gen(T)).int() if last else None
    if last:
        idx[1], idx[2] = -1, T     # outside: zero rows
    logits = torch.full((n, V), float("nan"), dtype=torch.bfloat16, device="cuda")
    tok = torch.full((n,), -5, dtype=torch.int64, device="cuda")
    ws = torch.zeros(L.w4_lm_head_workspace_size(n, V, H, tp), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        L.w4_lm_head(h.cuda(), None if idx is None else idx.cuda(), n, c, s, z, group, tp, logits, tok, ws)
        sync_ok(L)
        x = h.double()[:n]
        if last:
            x = torch.where(((idx >= 0) & (idx < T))[:, None], h.double()[idx.long().clamp(0, T - 1)], 0.0)
        y, e = product(x, w)
        near(logits, y, e, (n, V))
        assert torch.equal(tok.cpu(), logits.float().cpu().argmax(-1))   # of the logits as rounded; first of equals
    only = torch.empty_like(logits)
    if not last:
        L.w4_lm_head(h.cuda(), None, n, c, s, z, group, tp, only)
        sync_ok(L)
        assert torch.equal(only, logits)


@pytest.mark.parametrize("n", [3, 100])
def test_lm_head_ties_and_nan(L, n):
    """Equal logits: the lowest index.  NaN logits are passed over; nothing but NaN gives token 0."""
    V, H = 777, 64
    c, s, z, _ = matrix(V, H, 32, False)
    c[:] = c[5]
    s[:] = s[5]
    h = torch.randn(n, H, generator=gen(5)).bfloat16().cuda()
    h[1] = float("nan")
    s[0, 0] = float("nan")
    logits = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    tok = torch.empty(n, dtype=torch.int64, device="cuda")
    ws = torch.zeros(L.w4_lm_head_workspace_size(n, V, H, 1), dtype=torch.uint8, device="cuda")
    L.w4_lm_head(h, None, n, c, s, z, 32, 1, logits, tok, ws)
    sync_ok(L)
    want = torch.ones(n, dtype=torch.int64)
    want[1] = 0
    assert torch.equal(tok.cpu(), want)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [3, 90, 400])
def test_mlp_from_quantised_weights(L, M):
    """Embedding, gate_up with SiluAndMul, down over two shards, logits: quantised here, run in a row, and again
    from a graph; each step equals the float64 product over the weights that the quantiser stands for."""
    H, I, V, tp, G = 256, 384, 600, 2, 32
    g = gen(21)
    dev = "cuda"
    table = (0.05 * torch.randn(V, H, generator=g)).bfloat16().to(dev)
    gu = (0.05 * torch.randn(2 * I, H, generator=g)).bfloat16().to(dev)
    dn = (0.05 * torch.randn(tp * H, I // tp, generator=g)).bfloat16().to(dev)
    ids = torch.randint(0, V, (M,), generator=g).to(dev)
    q = []
    for w, zeros in ((table, False), (gu, True), (dn, True)):
        N, K = w.shape
        q.append((torch.empty(N, K // 2, dtype=torch.uint8, device=dev),
                  torch.empty(N, K // G, dtype=torch.bfloat16, device=dev),
                  torch.empty(N, K // G, dtype=torch.uint8, device=dev) if zeros else None))
        L.w4_quantize(w, G, *q[-1])
    vals = []
    for (c, s, z) in q:
        v = torch.empty(c.shape[0], c.shape[1] * 2, dtype=torch.bfloat16, device=dev)
        L.w4_embed_vocab(torch.arange(c.shape[0], device=dev), c, s, z, G, 1, v)
        vals.append(v)
    x, act, y = (torch.empty(M, k, dtype=torch.bfloat16, device=dev) for k in (H, I, H))
    logits = torch.empty(M, V, dtype=torch.bfloat16, device=dev)
    tok = torch.empty(M, dtype=torch.int64, device=dev)
    ws = torch.zeros(max(L.w4_lm_head_workspace_size(M, V, H, tp), L.w4_gemm_workspace_size(M, 2 * I, H, tp, COL, SILU),
                         L.w4_gemm_workspace_size(M, H, I, tp, ROW, NONE)), dtype=torch.uint8, device=dev)

    def step(ready=True):
        L.w4_embed_vocab(ids, *q[0], G, tp, x)
        L.w4_gemm(x, *q[1], act, 2 * I, G, tp, COL, SILU, ws, weights_ready=ready)
        L.w4_gemm(act, *q[2], y, H, G, tp, ROW, NONE, ws, weights_ready=ready)
        L.w4_lm_head(y, None, M, *q[0], G, tp, logits, tok, ws, weights_ready=ready)

    step(False)
    sync_ok(L)
    assert torch.equal(x, vals[0][ids])
    y1, e1 = product(x.double().cpu(), vals[1].double().cpu())
    (ga, up), (eg, eu) = y1.view(M, tp, 2, -1).unbind(2), e1.view(M, tp, 2, -1).unbind(2)
    a = ga * torch.sigmoid(ga)
    near(act, (a * up).reshape(M, -1), (1.1 * eg * (up.abs() + eu) + a.abs() * eu + 2.0 ** -20 * (a * up).abs()).reshape(M, -1), "act")
    near(y, *product(act.double().cpu(), vals[2].double().cpu().view(tp, H, -1).permute(1, 0, 2).reshape(H, I)), "down")
    near(logits, *product(y.double().cpu(), vals[0].double().cpu()), "logits")
    assert torch.equal(tok, logits.float().argmax(-1))
    first = [t.clone() for t in (act, y, logits, tok)]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            step()
    for seed in (1, 2):
        ids.copy_(torch.randint(0, V, (M,), generator=gen(seed)).to(dev))
        graph.replay()
        sync_ok(L)
        want = [t.clone() for t in (act, y, logits, tok)]
        step()
        sync_ok(L)
        assert all(torch.equal(a, b) for a, b in zip(want, (act, y, logits, tok)))
    assert len(first) == 4


@pytest.mark.parametrize("M", [1, 12, 100])
def test_weights_written_just_before(L, M):
    """Quantised and multiplied in turn on one stream, without the statement that the weights were there."""
    N, K, G = 512, 1024, 64
    x = torch.randn(M, K, generator=gen(M)).bfloat16().cuda()
    ws = [(0.1 * torch.randn(N, K, generator=gen(i))).bfloat16().cuda() for i in range(6)]
    c, s, z = (torch.empty(N, k, dtype=d, device="cuda") for k, d in ((K // 2, torch.uint8), (K // G, torch.bfloat16),
                                                                     (K // G, torch.uint8)))
    want = []
    for w in ws:
        L.w4_quantize(w, G, c, s, z)
        torch.cuda.synchronize()
        want.append(run_gemm(L, x, c, s, z, N, G, 1, COL, NONE))
        torch.cuda.synchronize()
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in ws]
    for _ in range(20):
        for w, o in zip(ws, outs):
            L.w4_quantize(w, G, c, s, z)
            L.w4_gemm(x, c, s, z, o, N, G)
        sync_ok(L)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("M", [2, 40, 200])
def test_two_streams_and_a_wide_batch_at_once(L, M):
    """Calls side by side on two streams, each into its own output, give what they give alone."""
    N, K = 1024, 2048
    c, s, z, _ = matrix(N, K, 128, True, seed=3)
    xs = [torch.randn(M, K, generator=gen(i)).bfloat16().cuda() for i in range(2)]
    want = [run_gemm(L, x, c, s, z, N, 128, 1, COL, NONE) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(10)] for _ in xs]
    torch.cuda.synchronize()
    for i in range(10):
        for st, x, o in zip(streams, xs, outs):
            L.w4_gemm(x, c, s, z, o[i], N, 128, stream=st)
    sync_ok(L)
    for o, w in zip(outs, want):
        assert all(torch.equal(a, w) for a in o)


@pytest.mark.parametrize("M", [1, 9, 70, 200])
def test_offsets_past_2_to_31(L, M):
    """A matrix of 2.4 GB of codes: its last rows, and its last row as an embedding."""
    N, K, G, tail = 300000, 16384, 128, 40
    c, s, z, w = matrix(tail, K, G, True, seed=2)
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(N, K // G, dtype=torch.bfloat16, device="cuda")
    zeros = torch.full((N, K // G), 3, dtype=torch.uint8, device="cuda")
    codes[-tail:], scales[-tail:], zeros[-tail:] = c, s, z
    x = torch.randn(M, K, generator=gen(M)).bfloat16()
    out = run_gemm(L, x.cuda(), codes, scales, zeros, N, G, 1, COL, NONE)
    row = torch.empty(2, K, dtype=torch.bfloat16, device="cuda")
    L.w4_embed_vocab(torch.tensor([N - 1, 5], device="cuda"), codes, scales, zeros, G, 1, row)
    sync_ok(L)
    near(out[:, -tail:], *product(x.double(), w), M)
    assert (out[:, :-tail] == 0).all()
    assert torch.equal(row[0].double().cpu(), w[-1]) and (row[1] == 0).all()


@pytest.mark.parametrize("M,N,K,group,tp,mode,epi", [(1, 1, 32, 32, 1, COL, NONE), (300, 1, 64, 32, 2, ROW, NONE),
                                                     (16, 3, 128, 128, 1, COL, NONE), (129, 16, 32, 32, 1, COL, SILU),
                                                     (40, 16, 256, 128, 1, COL, SILU), (5000, 32, 128, 64, 2, COL, SILU)])
def test_gemm_smallest(L, M, N, K, group, tp, mode, epi):
    check_gemm(L, M, N, K, group, True, tp, mode, epi)


@pytest.mark.parametrize("M", [1, 6, 13, 33, 64, 140])
def test_gemm_drawn_sizes(L, M):
    """Sizes from all over the range, every kernel choice among them."""
    import random
    rng = random.Random(M)
    for _ in range(6):
        group, tp = rng.choice([32, 64, 128]), rng.choice([1, 2, 3])
        mode, epi = rng.choice([(COL, NONE), (ROW, NONE), (COL, SILU)])
        N = (16 * tp if epi else tp) * rng.randint(1, 120)
        K = group * tp * rng.randint(1, 1500 // group)
        check_gemm(L, M, N, K, group, rng.random() < 0.5, tp, mode, epi, seed=rng.randint(1, 99))


def test_replayed_graphs_side_by_side(L):
    """Two captured graphs over the same weights, replayed in turn and on two streams at once."""
    N, K, V = 768, 512, 1000
    c, s, z, _ = matrix(N, K, 64, True)
    tc, ts, _, _ = matrix(V, N, 64, False)
    runs = []
    for M in (4, 150):
        x = torch.randn(M, K, generator=gen(M)).bfloat16().cuda()
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        logits = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
        tok = torch.empty(M, dtype=torch.int64, device="cuda")
        last = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
        ws = torch.zeros(L.w4_lm_head_workspace_size(M, V, N, 1), dtype=torch.uint8, device="cuda")

        def step():
            L.w4_gemm(x, c, s, z, y, N, 64, weights_ready=True)
            L.w4_lm_head(y, last, M, tc, ts, None, 64, 1, logits, tok, ws, weights_ready=True)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, logits, tok)]
        st = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
            step()
        runs.append((graph, st, (y, logits, tok), want, (x, last, ws, step)))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, st, outs, _, _ in runs:
            with torch.cuda.stream(st):
                for o in outs:
                    o.zero_()
                graph.replay()
        sync_ok(L)
        for _, _, outs, want, _ in runs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("epi", [NONE, SILU])
@pytest.mark.parametrize("M", [3, 8, 11, 16])
def test_gemm_wide_outputs_of_few_tokens(L, M, epi, zeros):
    """More row tiles than warps run at once: each warp walks through all of K, the tokens in shared memory."""
    check_gemm(L, M, 59984, 512, 64, zeros, 1, COL, epi)
    x = torch.randn(M, 512, generator=gen(M)).bfloat16()
    x[1] = float("nan")
    check = run_gemm(L, x.cuda(), *matrix(59984, 512, 64, zeros)[:3], 59984, 64, 1, COL, epi)
    sync_ok(L)
    assert torch.isnan(check[1]).all() and torch.isfinite(torch.cat([check[:1], check[2:]])).all()
