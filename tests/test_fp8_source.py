"""What no run can show of the 8-bit product: that its tensor memory loads are waited for by statements that name the loaded
registers.  A wait that names none (its asm has a memory clobber only) leaves the compiler free to move arithmetic on
registers, plain or in asm that is not volatile, ahead of it."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "patch_tiled_causal_gb300", "csrc")


def test_tensor_memory_loads_are_waited_for_by_name():
    with open(os.path.join(CSRC, "gemm_fp8.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "tmem_ld_wait" not in text
    loads = re.findall(r"\btmem_ld_32x32b_x(?:16|32)\(", text)
    waits = re.findall(r"\btmem_wait_x(?:16|32)\(", text)
    assert loads and waits
    for body in re.findall(r"asm volatile\(\s*\"tcgen05\.wait::ld[^;]*;\"(.*?)\);", text, flags=re.S):
        assert body.count('"+r"') >= 14  # (the rest in a second statement: one takes 30 operands)
