"""The workspace of prefill attention over the 8-bit KV cache is bounded as stated,
for every batch and whatever its padding (no GPU needed)."""
import random

from qwen3_transformer_forward_gb300 import _lib as L
from qwen3_transformer_forward_gb300 import build as B


def test_padding_does_not_enlarge_the_workspace():
    B.build()
    rng = random.Random(1)
    split = 0
    for _ in range(20000):
        nkv = rng.choice([1, 2, 3, 4, 8, 12])
        nh = nkv * rng.randint(1, 16)
        n, mq, mc = int(2 ** rng.uniform(0, 8)), int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 18))
        total = rng.randint(1, n * mq)
        a = L.attention_prefill_kv8_workspace_size(n, total, mq, mc, nh, nkv)
        b = L.attention_prefill_kv8_workspace_size(n, n * mq + int(2 ** rng.uniform(0, 20)), mq, mc, nh, nkv)
        assert a <= L.ATTENTION_PREFILL_KV8_WORKSPACE_MAX and b <= L.ATTENTION_PREFILL_KV8_WORKSPACE_MAX
        split += b > 0
    assert split > 1000
