"""Arrivals on another CTA's barrier, by the kernels' sources (no GPU). An arrival without a scope orders nothing between
two CTAs, and a missing order shows in no output until it does: so each names the cluster, shared memory that the other
CTA's MMAs read is released to it, and the thread that issues those acquires from it."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_quant_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_remote_arrivals_name_the_cluster():
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for op in re.findall(r'"(mbarrier\.arrive[\w.:]*)', source(os.path.basename(path))):
            if "shared::cluster" in op:
                assert ".cluster.shared::cluster" in op, (path, op)
                found += 1
    assert found


def test_attention_publishes_what_its_pair_reads():
    src = source("mla_attention.cu")
    kernel = src[src.index("mla_attention_kernel("):src.index("mla_join_kernel")]
    # Stores that the tensor cores read: the weights, and zeros past the end of the keys.
    after = kernel.split("fence_proxy_async_smem();")[1:]
    assert len(after) == 2
    for part in after:
        arrivals = re.findall(r"mbar_(arrive|publish)_cluster\(", part)
        assert arrivals[0] == "publish"
    issuers = kernel[kernel.index("const bool scores = warp == 6"):kernel.index("softmax and stores")]
    waits = dict.fromkeys(("s_empty", "o_empty", "p_full"))
    for name in waits:
        waits[name] = re.findall(r"(wait_\w+)\(&?" + name, issuers)
    assert all(w == ["wait_cluster"] for w in waits.values()), waits
    assert re.findall(r"(wait_\w+)\(&v_full", issuers) == ["wait_one", "wait_cluster"]
