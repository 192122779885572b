"""What attention over the 8-bit cache reports through qw_device_error (GPU side)."""
import pytest
import torch

from tests import test_gpu_kv8 as K
from tests.test_gpu_kv8 import E4, HD, I8, L, Paged, gen  # noqa: F401  (L: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,lq,mc", [([1500, 1100], [7, 5], 1200), ([300, 130], [300, 9], 256)])
def test_prefill_reports_an_overlong_context(L, lens, lq, mc):
    """A context beyond max_context: told once, as an argument's mistake; the other sequence is right."""
    nh, nkv = 8, 2
    c = Paged(lens, nkv, I8, 32, 128, seed=3)
    q = torch.randn(sum(lq), nh, HD, generator=gen(4)).bfloat16()
    out = K._prefill(L, c.cuda(), q.cuda(), lens, lq, nh, 0, 0, max_context=mc)
    torch.cuda.synchronize()
    with pytest.raises(L.QwError) as e:
        L.device_error()
    assert e.value.code == L.QW_ERR_INVALID_ARG
    L.device_error()
    assert torch.isfinite(out.float()).all()
    K._check_prefill(out[lq[0]:], K._only(c, 1), q[lq[0]:], lens[1:], lq[1:], 0, 0)
