"""The path of the 8-bit prefill kernel after a wait that gave up, checked on the
source (running it needs a broken kernel): the waits after it are skipped, except
the last, for the MMAs in flight, which TMEM and shared memory must outlive."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "qwen3_transformer_forward_gb300" / "csrc"


def test_the_wait_before_tmem_is_freed_is_never_skipped():
    text = (CSRC / "attention_kv8_prefill.cu").read_text()
    code = re.sub(r"//[^\n]*", "", text)
    assert re.search(r"if \(ok && !tcx::mbar_wait", code)          # a failed wait skips the later ones
    done = re.search(r"commit\(lead, bar\(B_DONE\)\);(.*?)__syncwarp\(\);", code, re.S).group(1)
    # ... so the last one starts afresh, or is not made through that helper
    assert re.search(r"ok = true;\s*wait\(B_DONE, 0u", done) or "tcx::mbar_wait(bar(B_DONE)" in done
    assert code.index("bar(B_DONE));") < code.index("tcx::tmem_dealloc(")
