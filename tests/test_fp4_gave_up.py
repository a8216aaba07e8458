"""What the few-token 4-bit product does after a wait that gave up, by its source (no GPU: no wait gives up there unless a
copy or an MMA never ends). The MMA warp then still commits, so that nobody waits for ever; what lies in tensor memory is
not the sum over K, and must reach neither the output nor, as a partial sum, another CTA's."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_quant_gb300", "csrc")


def few_kernel():
    with open(os.path.join(CSRC, "gemm_fp4.cu")) as f:
        src = f.read()
    return src[src.index("fp4_gemm_kernel("):src.index("struct PairCfg")]


def test_an_early_commit_is_not_taken_for_the_end():
    k = few_kernel()
    # Both sides of the barrier: the flag is in memory before the commit, and read after the wait.
    issuer = k[k.index("} else if (warp == 1) {"):k.index("} else if (warp < 6) {")]
    assert re.search(r"if \(!ok\) __threadfence_block\(\);[^\n]*\n\s*__syncwarp\(\);\n\s*if \(leader\) \{\n\s*if \(!ok\) mma_commit\(done\);",
                     issuer)
    assert re.search(r"finished = mbar_wait\(done,[^;]*&& \*abort_flag == 0;", k)
    # Every wait of the issuer and the producers raises the flag where it gives up.
    for code in ("kDevErrTimeoutMma", "kDevErrTimeoutProducer"):
        waits = re.findall(r"mbar_wait\([^;{]*?" + code, k)
        assert waits and all("abort_flag" in w for w in waits)


def test_a_part_without_its_sum_is_no_number():
    k = few_kernel()
    send = k[k.index("if (c0 >= (ks == 1"):k.index("send_columns<4, kStep>")]
    assert "if (!finished)" in send and "r[i] = 0x7FFFFFFFu;" in send
    assert re.search(r"if \(row < p\.N && finished\) p\.c\[", k)
    assert re.search(r"if \(!mbar_wait_cluster\(parts_full[^;]*finished = false;", k)
