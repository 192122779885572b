"""What attention over the 8-bit cache reports through qw_device_error, checked on
the sources (a wait that gives up needs a broken kernel): the word of a wait
never holds the bit that stands for a caller's context length."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "qwen3_transformer_forward_gb300" / "csrc"


def _overflow_bit():
    value = re.search(r"kErrContextOverflow = ([^;]+);", (CSRC / "common.cuh").read_text()).group(1)
    return eval(value.replace("u", ""))   # a literal or a shift of one


def test_no_wait_has_the_bit_of_an_overlong_context():
    bit = _overflow_bit()
    assert bit and bit & (bit - 1) == 0
    # waits that pass the number of their bit
    codes = [int(c) for c in re.findall(r"\bwait\(B_[^;]*?,\s*(\d+)u\);", (CSRC / "attention_kv8_prefill.cu").read_text())]
    assert len(codes) >= 13
    assert all(c < 32 and (1 << c) != bit for c in codes)
    # waits that pass the bit itself, in the files whose words hold the overflow bit too
    for name in ("attention.cu", "attention_kv8.cu"):
        text = (CSRC / name).read_text()
        words = [int(c, 0) for c in re.findall(r"(?:mbar_wait|\bwait)\([^;]*?,\s*(0x[0-9a-f]+|\d+)u\)", text)]
        assert words
        assert all(not w & bit for w in words)
