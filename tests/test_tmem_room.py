"""Shared memory of the kernels that take TMEM, from the sources: beside a CTA of the
tcgen05 kernel on 4-bit weights, whose pair waits for TMEM on two SMs, no CTA that
takes TMEM may fit on an SM."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "qwen3_transformer_forward_gb300" / "csrc"
SM, RESERVED = 228 * 1024, 1024      # shared memory of an SM, and what the system takes of it for each CTA


def code(name):
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def number(text, name):
    return eval(re.search(r"\b%s = ([0-9 *+()]+)[,;]" % name, text).group(1))   # an expression of digits


def w4_smem():
    narrow, wide, unit = re.search(r"size_t SMEM = \(NARROW \? (\d+) : (\d+)\) \* (\d+);", code("w4_gemm_tc.cu")).groups()
    return min(int(narrow), int(wide)) * int(unit)


def others():
    """(kernel, dynamic shared memory, from below)"""
    gemm = code("gemm.cu")
    slab = number(gemm, "BM") * number(gemm, "BK") * 2            # a stage holds more than its activations
    assert "A_BYTES = BM * BK * 2" in gemm
    stages = [int(s) for s in re.findall(r"launch_tc<\w+, (\d+)", gemm)] + [int(s) for s in re.findall(r"gemm_tc_kernel<\d+, (\d+)", gemm)]
    assert stages and "size_t(STAGES) * (TileCfg<BN>::A_BYTES" in gemm
    yield "gemm_tc_kernel", min(stages) * slab
    assert "size_t(M2_STAGES) * (M2_A_BYTES" in gemm and "M2_A_BYTES = M2_ROWS * BK * 2" in gemm
    yield "gemm_tc_m256_kernel", number(gemm, "M2_STAGES") * slab
    assert "size_t(PSTAGES) * (TileCfg<PBN>::A_BYTES" in gemm
    yield "gemm_tc_persist_kernel", number(gemm, "PSTAGES") * slab
    for name in ("attention_prefill.cu", "attention_kv8_prefill.cu"):
        text = code(name)
        assert "TILE = 2 * BOX" in text and "OFF_V = 4 * TILE" in text and "SMEM = 1024 + OFF_BAR + 256" in text
        yield name, 4 * 2 * number(text, "BOX")                   # what lies before OFF_V


def test_no_other_cta_with_tmem_fits_beside_one():
    left = SM - RESERVED - w4_smem()
    for kernel, smem in others():
        assert smem + RESERVED > left, (kernel, smem, left)
    assert w4_smem() + RESERVED > left                            # nor a second one of its own


def test_every_kernel_that_takes_tmem_is_looked_at():
    takes = {p.name for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh") and re.search(r"tmem_alloc\(|tcgen05\.alloc", code(p.name))}
    assert takes == {"tc_common.cuh", "gemm.cu", "attention_prefill.cu", "attention_kv8_prefill.cu", "w4_gemm_tc.cu"}
    assert len(re.findall(r"\btmem_alloc\(smem", code("gemm.cu"))) == 3
