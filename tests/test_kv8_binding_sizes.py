"""The Python binding of the 8-bit KV cache refuses tensors that the kernels would
read or write past: pointers are replaced, nothing is launched."""
import pytest
import torch

from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import build as B

SHAPE, DT = L.QW_ERR_SHAPE, L.QW_ERR_DTYPE


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    B.build()
    monkeypatch.setattr(L, "_dev_ptr", lambda t, name: None if t is None else 64)
    monkeypatch.setattr(L, "_stream", lambda s: None)


def _append(**kw):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    k, sc = torch.zeros(128, 2, 128, dtype=torch.int8), torch.zeros(2, 2)
    a = dict(q_gamma=bf(128), k_gamma=bf(128), err_count=None)
    a.update(kw)
    L.kv8_append(bf(0, 8 * 128), 4, 2, 128, 1, torch.zeros(0, dtype=torch.int64), torch.zeros(64, 128), a["q_gamma"], a["k_gamma"],
                 1e-6, i32(4), i32(3), i32(3, 2), 64, k, k, sc, sc, 64, bf(0, 4, 128), a["err_count"])


def _read(err_count):
    k, sc = torch.zeros(128, 2, 128, dtype=torch.int8), torch.zeros(2, 2)
    L.kv8_read(k, k, sc, sc, 64, torch.zeros(0, dtype=torch.int64), None, None, err_count)


def test_what_is_right_passes():
    _append()
    _append(err_count=torch.zeros(1, dtype=torch.int32), q_gamma=torch.zeros(1, 128, dtype=torch.bfloat16))
    _read(None)
    _read(torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("which", ["q_gamma", "k_gamma"])
@pytest.mark.parametrize("n", [0, 1, 64, 127])
def test_gammas_have_a_weight_for_each_element_of_a_head(which, n):
    with pytest.raises(L.QwError) as e:
        _append(**{which: torch.zeros(n, dtype=torch.bfloat16)})
    assert e.value.code == SHAPE


@pytest.mark.parametrize("call", [lambda t: _append(err_count=t), _read])
def test_err_count_is_an_int32(call):
    for t, code in ((torch.zeros(1, dtype=torch.int64), DT), (torch.zeros(1, dtype=torch.uint8), DT), (torch.zeros(1), DT),
                    (torch.zeros(0, dtype=torch.int32), SHAPE)):
        with pytest.raises(L.QwError) as e:
            call(t)
        assert e.value.code == code
