"""Column loops of the layer norm kernels at the widest row, 2^31 - 1 columns: the index after the
last step passes the row's end by up to a step, which a 32-bit int does not hold."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_column_loops_end():
    text = open(os.path.join(ROOT, "dense_blas3_gemm_amd", "csrc", "layernorm.hip")).read()
    loops = re.findall(r"for \((\w+) (\w+) = threadIdx\.x; \2 < ([\w.]+); \2 \+= \d+\)", text)
    assert len(loops) >= 5
    for kind, _, end in loops:
        assert kind in ("uint32_t", "int64_t"), (kind, end)
        # compared as the index is: `cols` is the unsigned copy
        assert end != "a.cols" or kind == "int64_t", (kind, end)
