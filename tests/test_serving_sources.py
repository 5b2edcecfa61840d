"""What the serving kernels' sources have to keep, whatever the compiler does."""
import os
import re

import quantized_attention_smoothing_b200 as sage

CSRC = os.path.join(os.path.dirname(sage.__file__), "csrc")


def test_no_tensor_memory_load_in_flight_across_other_code():
    """shared.cu's kernels may spill, so a tcgen05.ld and its wait are one asm
    statement: by the helpers that hold both, or spelt out with the wait."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "shared.cu")).read())
    helpers = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "sage_ptx.cuh")).read())
    used = set(re.findall(r"\b(tmem_ld\w+)\(", text))
    assert used
    bodies = dict(re.findall(r"\bvoid (tmem_ld\w+)\([^)]*\)[^{]*\{\s*asm volatile\((.*?)\);\n\}", helpers + text, flags=re.S))
    for name in used:
        assert "tcgen05.wait::ld" in bodies[name], name
    assert "tmem_wait_ld(" not in text
