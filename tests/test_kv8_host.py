"""Host-side checks of the 8-bit KV cache entry points (no GPU needed): every
refusal comes before the device is touched, and zero sizes are no-ops."""
import ctypes as C

import pytest
import torch

from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import build as B

FAKE, ODD = C.c_void_p(64), C.c_void_p(72)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _call(lib, name, order, base, **kw):
    a = dict(base, **kw)
    assert set(kw) <= set(base), kw
    return getattr(lib, name)(*[a[k] for k in order])


APPEND = dict(qkv=FAKE, T=4, nh=16, nkv=8, hd=128, tp=1, pos=FAKE, cs=FAKE, maxp=64, qg=FAKE, kg=FAKE, eps=1e-6, cu=FAKE,
              ctx=FAKE, table=FAKE, maxb=4, bs=256, n=2, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, slots=1024, sb=64, q=FAKE,
              err=None, dt=L.QW_BF16, kv=L.QW_I8, st=None)
READ = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, slots=1024, sb=64, nkv=8, hd=128, rows=FAKE, n=3, ko=FAKE, vo=FAKE, err=None,
            dt=L.QW_BF16, kv=L.QW_I8, st=None)
DECODE = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, slots=1024, sb=64, ctx=FAKE, table=FAKE, maxb=4, bs=256, n=2,
              mc=1024, nh=16, nkv=8, hd=128, scale=0.1, window=0, sink=0, out=FAKE, ws=FAKE, wsb=1 << 40, dt=L.QW_BF16,
              kv=L.QW_I8, st=None)
PREFILL = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, slots=1024, sb=64, cu=FAKE, ctx=FAKE, table=FAKE, maxb=4, bs=256,
               n=2, T=8, maxq=4, mc=1024, nh=16, nkv=8, hd=128, scale=0.1, window=0, sink=0, out=FAKE, ws=FAKE,
               wsb=1 << 40, dt=L.QW_BF16, kv=L.QW_E4M3, st=None)
ENTRY = {"append": ("qw_kv8_append", APPEND), "read": ("qw_kv8_read", READ), "decode": ("qw_attention_decode_kv8", DECODE),
         "prefill": ("qw_attention_prefill_kv8", PREFILL)}

SHAPE, ARG, DT, WS, OK = L.QW_ERR_SHAPE, L.QW_ERR_INVALID_ARG, L.QW_ERR_DTYPE, L.QW_ERR_WORKSPACE, L.QW_OK


@pytest.mark.parametrize("op", list(ENTRY))
@pytest.mark.parametrize("kw,want", [
    (dict(dt=7), DT), (dict(kv=L.QW_BF16), DT), (dict(kv=4), DT), (dict(hd=64), SHAPE), (dict(sb=8), SHAPE),
    (dict(sb=128), SHAPE), (dict(sb=48), SHAPE), (dict(slots=1000), SHAPE), (dict(slots=-64), ARG),
    (dict(slots=1 << 31), ARG), (dict(nkv=0), ARG), (dict(n=-1), ARG), (dict(k=None), ARG), (dict(v=None), ARG),
    (dict(ks=None), ARG), (dict(vs=None), ARG), (dict(k=ODD), ARG), (dict(v=ODD), ARG), (dict(ks=C.c_void_p(66)), ARG)])
def test_cache_refusals(lib, op, kw, want):
    name, base = ENTRY[op]
    if op == "read" and "n" in kw:
        kw = dict(n=-1)
    assert _call(lib, name, list(base), base, **kw) == want
    assert lib.qw_last_error_string().decode().startswith(name)


@pytest.mark.parametrize("op", ["append", "decode", "prefill"])
@pytest.mark.parametrize("kw,want", [(dict(table=None), ARG), (dict(bs=100), SHAPE), (dict(bs=0), SHAPE),
                                     (dict(maxb=0), SHAPE), (dict(ctx=None), ARG), (dict(dt=L.QW_F32), DT)])
def test_table_refusals(lib, op, kw, want):
    name, base = ENTRY[op]
    assert _call(lib, name, list(base), base, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(tp=3), SHAPE), (dict(tp=0), ARG), (dict(maxp=0), ARG), (dict(T=-1), ARG), (dict(qkv=None), ARG),
    (dict(q=None), ARG), (dict(q=ODD), ARG), (dict(qkv=ODD), ARG), (dict(cs=ODD), ARG), (dict(pos=None), ARG),
    (dict(kg=None), ARG), (dict(cu=None, T=1), SHAPE), (dict(T=0), OK), (dict(n=0), OK)])
def test_append_refusals(lib, kw, want):
    assert _call(lib, "qw_kv8_append", list(APPEND), APPEND, **kw) == want


@pytest.mark.parametrize("kw,want", [(dict(rows=None), ARG), (dict(ko=ODD), ARG), (dict(vo=ODD), ARG), (dict(n=0), OK),
                                     (dict(ko=None, vo=None), OK), (dict(dt=L.QW_I8), DT)])
def test_read_refusals(lib, kw, want):
    assert _call(lib, "qw_kv8_read", list(READ), READ, **kw) == want


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("kw,want", [
    (dict(nh=12), SHAPE), (dict(nh=17 * 8), SHAPE), (dict(nh=0), ARG), (dict(mc=1025), SHAPE), (dict(mc=-1), ARG),
    (dict(window=-1), ARG), (dict(sink=-1), ARG), (dict(q=None), ARG), (dict(out=None), ARG), (dict(q=ODD), ARG),
    (dict(out=ODD), ARG), (dict(n=0), OK)])
def test_attention_refusals(lib, op, kw, want):
    name, base = ENTRY[op]
    assert _call(lib, name, list(base), base, **kw) == want


def test_workspace_refusals(lib):
    need = lib.qw_attention_decode_kv8_workspace_size(2, 1024, 16, 8)
    assert need >= 64 * 1024
    for kw in (dict(ws=None), dict(wsb=need - 1), dict(wsb=0)):
        assert _call(lib, "qw_attention_decode_kv8", list(DECODE), DECODE, **kw) == WS
    assert _call(lib, "qw_attention_decode_kv8", list(DECODE), DECODE, ws=ODD) == ARG
    # a few rows over many keys: the keys are split, and the parts need room
    need = lib.qw_attention_prefill_kv8_workspace_size(1, 4, 4, 40000, 16, 8)
    args = dict(n=1, T=4, maxq=4, mc=40000, maxb=200)
    if need:
        for kw in (dict(ws=None), dict(wsb=need - 1)):
            assert _call(lib, "qw_attention_prefill_kv8", list(PREFILL), PREFILL, **args, **kw) == WS
    # more (sequence, kv head) pairs than completion counters
    assert _call(lib, "qw_attention_decode_kv8", list(DECODE), DECODE, n=20000) == SHAPE
    # sizes past the 32-bit counts of a call
    assert _call(lib, "qw_attention_decode_kv8", list(DECODE), DECODE, n=2048, maxb=1 << 18, bs=64, mc=1 << 24) == SHAPE
    assert _call(lib, "qw_kv8_append", list(APPEND), APPEND, T=1 << 28) == SHAPE
    assert _call(lib, "qw_attention_prefill_kv8", list(PREFILL), PREFILL, n=70000) == SHAPE
    # sizes that no call takes have no workspace
    for bad in ((-1, 64, 16, 8), (2, -1, 16, 8), (2, 64, 0, 8), (2, 64, 16, 0)):
        assert lib.qw_attention_decode_kv8_workspace_size(*bad) == 0
    assert lib.qw_attention_prefill_kv8_workspace_size(-1, 8, 8, 64, 16, 8) == 0


def test_prefill_sizes(lib):
    for kw, want in ((dict(T=-1), ARG), (dict(maxq=-1), ARG), (dict(T=0), OK), (dict(maxq=0), OK), (dict(cu=None), ARG)):
        assert _call(lib, "qw_attention_prefill_kv8", list(PREFILL), PREFILL, **kw) == want


def test_binding_checks_types_and_sizes(lib):
    k = torch.zeros(128, 2, 128, dtype=torch.int8)
    s = torch.zeros(2, 2)
    assert L.kv_code(k, k, s, s, 64) == L.QW_I8
    e = k.view(torch.float8_e4m3fn)
    assert L.kv_code(e, e, s, s, 64) == L.QW_E4M3
    for args in ((k, e, s, s, 64), (k.to(torch.uint8), k.to(torch.uint8), s, s, 64), (k, k, s.double(), s, 64)):
        with pytest.raises(L.QwError) as err:
            L.kv_code(*args)
        assert err.value.code == DT
    for args in ((k, k, s[:1], s, 64), (k, k, s, s, 32), (k, k[:64], s, s, 64)):
        with pytest.raises(L.QwError) as err:
            L.kv_code(*args)
        assert err.value.code == SHAPE


def test_binding_refuses_what_the_library_cannot_see(lib, monkeypatch):
    """Head counts against the cache's shape, index types, sequence counts, output types and sizes."""
    monkeypatch.setattr(L, "_dev_ptr", lambda t, name: None if t is None else 64)
    monkeypatch.setattr(L, "_stream", lambda s: None)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)
    k, sc = torch.zeros(128, 2, 128, dtype=torch.int8), torch.zeros(2, 2)
    rows = torch.zeros(3, dtype=torch.int64)
    base = dict(qkv=bf(0, 8 * 128), nh=4, nkv=2, pos=rows, cs=torch.zeros(64, 128), qg=bf(128), kg=bf(128), cu=i32(4), ctx=i32(3),
                table=i32(3, 2), q_out=bf(0, 4, 128), q=bf(0, 4, 128), out=bf(0, 4, 128), rows=rows[:0], k_out=None, v_out=None)

    def append(a):
        L.kv8_append(a["qkv"], a["nh"], a["nkv"], 128, 1, a["pos"], a["cs"], a["qg"], a["kg"], 1e-6, a["cu"], a["ctx"], a["table"],
                     64, k, k, sc, sc, 64, a["q_out"])

    def read(a):
        L.kv8_read(k, k, sc, sc, 64, a["rows"], a["k_out"], a["v_out"])

    def decode(a):
        L.attention_decode_kv8(a["q"], k, k, sc, sc, 64, a["ctx"], a["table"], 64, 128, a["nh"], a["nkv"], 128, 0.1, a["out"], None)

    def prefill(a):
        L.attention_prefill_kv8(a["q"], k, k, sc, sc, 64, a["cu"], a["ctx"], a["table"], 64, 4, 128, a["nh"], a["nkv"], 128, 0.1,
                                a["out"], None)

    for f in (append, read, decode, prefill):
        f(base)   # no tokens, no rows: nothing to do
    both = (append, prefill)
    for fs, kw, want in (
            ((append, decode, prefill), dict(nh=2, nkv=1), SHAPE), ((append, decode, prefill), dict(ctx=rows), DT),
            ((append, decode, prefill), dict(table=torch.zeros(3, 2, dtype=torch.int64)), DT), (both, dict(cu=rows), DT),
            (both, dict(table=i32(2, 2)), SHAPE), (both, dict(ctx=i32(2)), SHAPE), ((decode,), dict(q=bf(4, 4, 128)), SHAPE),
            ((decode, prefill), dict(out=torch.zeros(0, 4, 128)), DT),
            ((decode, prefill), dict(q=bf(2, 4, 128), out=bf(1, 4, 128)), SHAPE),
            ((decode, prefill), dict(q=bf(1, 3, 128), out=bf(1, 4, 128)), SHAPE),
            ((append,), dict(qkv=bf(2, 8 * 128)), SHAPE), ((append,), dict(qkv=bf(2, 6 * 128), q_out=bf(2, 4, 128)), SHAPE),
            ((append,), dict(qkv=bf(4, 8 * 128), q_out=bf(4, 4, 128)), SHAPE), ((append,), dict(cs=torch.zeros(64, 64)), SHAPE),
            ((append,), dict(pos=i32(3)), DT), ((append,), dict(cs=bf(64, 128)), DT), ((append,), dict(kg=torch.zeros(128)), DT),
            ((read,), dict(rows=i32(3), k_out=bf(3, 2, 128)), DT), ((read,), dict(rows=rows, k_out=bf(2, 2, 128)), SHAPE),
            ((read,), dict(rows=rows, v_out=bf(2, 2, 128)), SHAPE),
            ((read,), dict(rows=rows, k_out=torch.zeros(3, 2, 128), v_out=bf(3, 2, 128)), DT)):
        for f in fs:
            with pytest.raises(L.QwError) as err:
                f(dict(base, **kw))
            assert err.value.code == want, (f.__name__, kw)


def test_positions_end_at_2_to_30(lib):
    for op in ("decode", "prefill"):
        name, base = ENTRY[op]
        for mc, want in (((1 << 30) + 1, SHAPE), (1 << 30, OK)):
            assert _call(lib, name, list(base), base, n=0, maxb=1 << 25, bs=64, mc=mc) == want
