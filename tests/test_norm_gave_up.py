"""What the norm that goes from token to token does after a wait that gave up, by its source (no GPU): its warps wait for one
another's sums of a row, and a row whose sums are not all there is not written."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_quant_gb300", "csrc")


def test_no_row_is_written_from_sums_that_are_not_there():
    with open(os.path.join(CSRC, "residual_norm.cu")) as f:
        src = f.read()
    k = src[src.index("residual_norm_rows_kernel("):src.index("const void* kernel_of")]
    waits = re.findall(r"[^\n]*mbar_wait\([^;]*;", k)
    assert len(waits) == 1
    # All lanes of a warp take the same way, the flag lets the other warps' waits give up at once, and no store follows.
    assert re.search(r"if \(!__all_sync\(0xFFFFFFFFu, mbar_wait\([^;]*&abort_flag,[^;]*\)\)\)\s*return;", waits[0])
    assert k.index("return;", k.index("mbar_wait(")) < k.index("write_residual<1, true>")
    assert k.index("abort_flag = 0;") < k.index("__syncthreads();")
