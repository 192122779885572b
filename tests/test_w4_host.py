"""Host-side checks of the entry points on 4-bit weights (no GPU needed): every
refusal comes before the device is touched, and zero sizes are no-ops."""
import ctypes as C

import pytest
import torch

from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import build as B

FAKE, ODD = C.c_void_p(64), C.c_void_p(72)   # never dereferenced
SHAPE, ARG, DT, WS, OK = L.QW_ERR_SHAPE, L.QW_ERR_INVALID_ARG, L.QW_ERR_DTYPE, L.QW_ERR_WORKSPACE, L.QW_OK
COL, ROW, SILU = L.QW_GEMM_COLUMN, L.QW_GEMM_ROW_REDUCE, L.QW_EPI_SILU_MUL

QUANT = dict(w=FAKE, N=64, K=256, group=64, codes=FAKE, scales=FAKE, zeros=None, dt=L.QW_BF16, st=None)
EMBED = dict(ids=FAKE, T=4, codes=FAKE, scales=FAKE, zeros=None, V=64, H=256, group=64, tp=1, out=FAKE, err=None,
             dt=L.QW_BF16, st=None)
GEMM = dict(A=FAKE, codes=FAKE, scales=FAKE, zeros=None, C=FAKE, M=4, N=64, K=256, group=64, tp=1, mode=COL, epi=0, ws=FAKE,
            wsb=1 << 40, dt=L.QW_BF16, flags=0, st=None)
HEAD = dict(hidden=FAKE, T=8, last=FAKE, n=4, codes=FAKE, scales=FAKE, zeros=None, V=64, H=256, group=64, tp=1, logits=FAKE,
            tok=FAKE, ws=FAKE, wsb=1 << 40, dt=L.QW_BF16, flags=0, st=None)
ENTRY = {"quantize": ("qw_w4_quantize", QUANT), "embed": ("qw_w4_embed_vocab", EMBED), "gemm": ("qw_w4_gemm", GEMM),
         "head": ("qw_w4_lm_head", HEAD)}
WIDTH = {"quantize": "K", "embed": "H", "gemm": "K", "head": "H"}


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def call(lib, op, **kw):
    name, base = ENTRY[op]
    assert set(kw) <= set(base), kw
    return getattr(lib, name)(*dict(base, **kw).values())


@pytest.mark.parametrize("op", list(ENTRY))
@pytest.mark.parametrize("kw,want", [
    (dict(dt=L.QW_F32), DT), (dict(dt=7), DT), (dict(group=16), SHAPE), (dict(group=96), SHAPE), (dict(group=0), SHAPE),
    (dict(width=96), SHAPE), (dict(width=0), ARG), (dict(width=-64), ARG), (dict(width=1 << 31), SHAPE),
    (dict(codes=None), ARG), (dict(codes=ODD), ARG), (dict(scales=None), ARG), (dict(scales=C.c_void_p(65)), ARG)])
def test_weight_refusals(lib, op, kw, want):
    kw = {WIDTH[op] if k == "width" else k: v for k, v in kw.items()}
    assert call(lib, op, **kw) == want
    assert lib.qw_last_error_string().decode().startswith(ENTRY[op][0])


@pytest.mark.parametrize("op,kw,want", [
    ("quantize", dict(N=-1), ARG), ("quantize", dict(N=0), OK), ("quantize", dict(w=None), ARG),
    ("quantize", dict(w=ODD), ARG), ("quantize", dict(N=1 << 31), SHAPE),
    ("embed", dict(T=-1), ARG), ("embed", dict(T=0), OK), ("embed", dict(ids=None), ARG), ("embed", dict(out=None), ARG),
    ("embed", dict(out=ODD), ARG), ("embed", dict(tp=3), SHAPE), ("embed", dict(tp=0), ARG), ("embed", dict(V=0), ARG),
    ("embed", dict(T=1 << 40), SHAPE),
    ("gemm", dict(M=-1), ARG), ("gemm", dict(M=0), OK), ("gemm", dict(M=1 << 21), SHAPE), ("gemm", dict(N=0), ARG),
    ("gemm", dict(A=None), ARG), ("gemm", dict(A=ODD), ARG), ("gemm", dict(C=None), ARG), ("gemm", dict(C=ODD), ARG),
    ("gemm", dict(mode=2), ARG), ("gemm", dict(epi=2), ARG), ("gemm", dict(epi=SILU, mode=ROW), ARG),
    ("gemm", dict(tp=0), ARG), ("gemm", dict(tp=3), SHAPE), ("gemm", dict(tp=3, mode=ROW), SHAPE),
    ("gemm", dict(tp=8, mode=ROW), SHAPE), ("gemm", dict(tp=2, epi=SILU, N=48), SHAPE), ("gemm", dict(epi=SILU, N=24), SHAPE),
    ("gemm", dict(N=1 << 31), SHAPE), ("gemm", dict(flags=2), ARG), ("head", dict(flags=-1), ARG),
    ("head", dict(n=-1), ARG), ("head", dict(n=0), OK), ("head", dict(T=-1), ARG), ("head", dict(last=None, n=9), SHAPE),
    ("head", dict(hidden=None), ARG), ("head", dict(hidden=ODD), ARG), ("head", dict(logits=None), ARG),
    ("head", dict(logits=ODD), ARG), ("head", dict(tp=3), SHAPE), ("head", dict(ws=None), WS), ("head", dict(wsb=1024), WS),
    ("head", dict(ws=None, last=None), WS), ("head", dict(n=1 << 21, T=1 << 22), SHAPE)])
def test_refusals(lib, op, kw, want):
    assert call(lib, op, **kw) == want
    if want != OK:
        assert lib.qw_last_error_string().decode().startswith(ENTRY[op][0])


# ---- the binding's own checks: the tensors lie on the CPU, so a call that passes them is refused as such ----

def mat(N=64, K=256, group=64):
    return (torch.zeros(N, K // 2, dtype=torch.uint8), torch.zeros(N, K // group, dtype=torch.bfloat16),
            torch.zeros(N, K // group, dtype=torch.uint8))


def refused(code, fn, *a, **k):
    with pytest.raises(L.QwError) as e:
        fn(*a, **k)
    assert e.value.code == code, e.value


def test_binding_refusals(lib):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    c, s, z = mat()
    x, y = bf(4, 256), bf(4, 64)
    ids = torch.zeros(4, dtype=torch.int64)
    cuda = ARG   # "must be a CUDA tensor": every check before it passed
    refused(cuda, L.w4_gemm, x, c, s, z, y, 64, 64)
    refused(DT, L.w4_gemm, x, c.to(torch.int32), s, z, y, 64, 64)
    refused(DT, L.w4_gemm, x, c, s.float(), z, y, 64, 64)
    refused(DT, L.w4_gemm, x, c, s, z.int(), y, 64, 64)
    refused(DT, L.w4_gemm, x, c, s, z, y.float(), 64, 64)
    refused(SHAPE, L.w4_gemm, x, c, s, z, y, 64, 32)
    refused(SHAPE, L.w4_gemm, x, c[:63], s, z, y, 64, 64)
    refused(SHAPE, L.w4_gemm, x, c, s, z[:, :3], y, 64, 64)
    refused(SHAPE, L.w4_gemm, x, c, s, z, bf(3, 64), 64, 64)
    refused(SHAPE, L.w4_gemm, x, c, s, z, y, 64, 64, epilogue=SILU)
    refused(SHAPE, L.w4_gemm, x, c, s, None, y, 64, 64, tp=2, mode=ROW)
    refused(SHAPE, L.w4_gemm, x, c, s, None, y, 64, 0)
    refused(cuda, L.w4_embed_vocab, ids, c, s, None, 64, 1, bf(4, 256))
    refused(DT, L.w4_embed_vocab, ids.int(), c, s, None, 64, 1, bf(4, 256))
    refused(SHAPE, L.w4_embed_vocab, ids, c, s, None, 64, 1, bf(3, 256))
    refused(SHAPE, L.w4_embed_vocab, ids, c, s, None, 64, 1, bf(4, 128))
    refused(DT, L.w4_embed_vocab, ids, c, s, None, 64, 1, bf(4, 256), torch.zeros(1))
    refused(cuda, L.w4_quantize, bf(64, 256), 64, c, s, z)
    refused(SHAPE, L.w4_quantize, bf(64, 128), 64, c, s, z)
    refused(cuda, L.w4_lm_head, x, None, 4, c, s, None, 64, 1, y)
    refused(SHAPE, L.w4_lm_head, x, None, 4, c, s, None, 64, 1, bf(3, 64))
    refused(DT, L.w4_lm_head, x, ids, 4, c, s, None, 64, 1, y)
    refused(DT, L.w4_lm_head, x, None, 4, c, s, None, 64, 1, y, ids.int())
    refused(SHAPE, L.w4_lm_head, x, ids.int()[:3], 4, c, s, None, 64, 1, y)
