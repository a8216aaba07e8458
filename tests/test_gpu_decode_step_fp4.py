"""The decode example with 4-bit linears and fused norms: it runs, follows the attention's formula, and replays."""
import pytest
import torch

from test_gpu_decode_step import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,prefix,steps", [(1, 0, 3), (3, 65, 4), (32, 300, 2)])
def test_steps_follow_the_formula(batch, prefix, steps):
    """As for the FP8 layer: the attention's weights and its output are rounded to bf16 once each."""
    seen = example().main(["--batch", str(batch), "--prefix", str(prefix), "--steps", str(steps), "--fp4"])
    assert len(seen) == steps
    for norm, off in seen:
        assert norm == norm and norm < float("inf") and off < 2.0 ** -7


def test_a_captured_step_replays_as_the_calls():
    args = ["--batch", "5", "--prefix", "130", "--steps", "3", "--fp4"]
    torch.manual_seed(7)
    plain = example().main(args)
    torch.manual_seed(7)
    assert example().main(args + ["--graph"]) == plain
