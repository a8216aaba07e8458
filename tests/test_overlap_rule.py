"""The rule on overlap, by the sources (no GPU): which calls let the next one start early, which order, and that the header
and the docstrings state one rule that holds for any number of calls. A weight operand that a call before is still
writing shows in no output until it does."""
import os
import re

import fp8_block_scaled_quant_gb300 as fb

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_quant_gb300", "csrc")
TRIGGER = "griddep_launch_dependents();"

# The files whose kernels let the next one start early, and the calls that issue them last.
EARLY = {
    "gemm.cu": ["gemm", "gemm_noalloc", "linear", "linear_host", "swiglu_gemm", "ffn"],
    "gemm_decode.cu": [],
    "mla.cu": ["mla_absorb_qk", "mla_absorb_v"],
    "mla_append.cu": ["mla_append"],
    "mla_attention.cu": ["mla_attention"],
    "gemm_fp4.cu": ["fp4_gemm", "fp4_linear"],
    "residual_norm.cu": ["residual_norm"],
}
ORDERING = ["act_quant", "weight_quant", "weight_dequant", "moe_gate", "moe_route", "moe_permute", "moe_grouped_gemm",
            "moe_layer", "fp4_quant", "fp4_dequant"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def rule():
    with open(fb.HEADER) as f:
        text = f.read()
    return re.sub(r"\s*\n \*\s*", " ", text[text.index("- Overlap on a stream"):text.index("#ifndef")])


def test_which_files_let_the_next_kernel_start_early():
    always, asked = set(), set()
    for name in sorted(os.listdir(CSRC)):
        for line in source(name).splitlines() if name.endswith(".cu") else []:
            if TRIGGER in line:
                (asked if line.strip().startswith("if (") else always).add(name)
    assert always == set(EARLY)
    # The quantisations do inside a linear layer alone.
    assert asked == {"quant.cu", "fp4_quant.cu"}
    for name, entry in (("quant.cu", "fp8blk_act_quant("), ("fp4_quant.cu", "fp8blk_fp4_quant(")):
        body = source(name)[source(name).index('extern "C" int ' + entry):]
        body = body[:body.index("\n}")]
        assert re.search(r"_launch\([^;]*\bfalse\b", body) and "true" not in body.replace("== 1", "")


def test_the_header_lists_them():
    early, ordering = rule().split("ordering call at least")
    early = early[:early.index("A call that starts so")]
    ordering = ordering[:ordering.index("that launches something")]
    named = lambda t: sorted(re.findall(r"fp8blk_(\w+)", t))  # noqa: E731
    assert named(early) == sorted(sum(EARLY.values(), []))
    assert named(ordering) == sorted(ORDERING)
    known = {n[len("fp8blk_"):] for n in fb.header_functions()}
    assert set(named(early)) | set(named(ordering)) <= known
    # Every call that launches kernels is one or the other.
    rest = {n for n in known - set(named(early)) - set(named(ordering))
            if not n.endswith(("_bytes", "_kernels", "_string")) and n not in ("version", "last_device_error", "capture_id")}
    assert not rest, rest


def test_the_rule_has_no_bound_and_python_says_it():
    assert "any number of early calls" in rule()
    assert "either of the two" not in rule() and "two library calls" not in rule()
    for doc in (fb.__doc__, fb.fp4_quant.__doc__, fb.fp4_gemm.__doc__, fb.fp4_linear.__doc__, fb.residual_norm.__doc__):
        assert "synchronis" in doc or "ordering call" in doc


def test_what_is_read_at_once_is_what_the_rule_names():
    """In the 4-bit product the producer of the weights alone goes ahead of the wait, and it reads w and w_s."""
    src = source("gemm_fp4.cu")
    few = src[src.index("fp4_gemm_kernel("):src.index("struct PairCfg")]
    assert "const bool weights = warp == 0;\n    if (!weights) griddep_wait();" in few
    pair = src[src.index("fp4_gemm_pair_kernel("):src.index("typedef CUresult")]
    ahead = pair[pair.index("const int pre ="):pair.index("griddep_wait();")]
    assert "weights(c);" in ahead and "tokens(" not in ahead
