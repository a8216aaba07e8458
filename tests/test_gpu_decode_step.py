"""The decode example: its steps run the cache, attention and MoE layer calls together."""
import importlib.util
import os
import time

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("batch,prefix,steps", [(1, 0, 3), (3, 65, 4), (32, 300, 2)])
def test_steps_follow_the_formula(batch, prefix, steps):
    """The attention's weights and its output are each rounded to bf16 once (2^-9 of their size): together 2^-8 of the
    output's norm at most, and twice that is allowed."""
    seen = example().main(["--batch", str(batch), "--prefix", str(prefix), "--steps", str(steps)])
    assert len(seen) == steps
    for norm, off in seen:
        assert norm == norm and norm < float("inf") and off < 2.0 ** -7


@pytest.mark.gpu
def test_a_captured_step_replays_as_the_calls():
    """One captured step, replayed as the lengths grow on the device, gives the steps' own numbers."""
    args = ["--batch", "5", "--prefix", "130", "--steps", "3"]
    torch.manual_seed(7)
    plain = example().main(args)
    torch.manual_seed(7)
    assert example().main(args + ["--graph"]) == plain


@pytest.mark.gpu
def test_the_side_stream_waits_for_what_it_reads():
    """Weights, page table, lengths and prompt are written on the default stream: nothing runs on the capturing stream
    before they are there. (The default stream is held up behind the prompt; the check comes before the step's work.)"""
    m = example()
    write_prompt, step, seen = m.write_prompt, m.step, []

    def held_up(*args):
        write_prompt(*args)
        torch.cuda._sleep(1 << 30)

    def checked(*args):
        stream = torch.cuda.current_stream()
        if stream != torch.cuda.default_stream() and not torch.cuda.is_current_stream_capturing():
            reached = [torch.cuda.Event() for _ in range(2)]
            reached[0].record(torch.cuda.default_stream())
            reached[1].record(stream)
            time.sleep(0.02)
            seen.append([e.query() for e in reached])
            assert seen[-1] == [False, False]
        return step(*args)

    m.write_prompt, m.step = held_up, checked
    assert len(m.main(["--batch", "2", "--prefix", "70", "--steps", "2", "--graph"])) == 2
    assert len(seen) == 1


def test_batch_is_checked():
    with pytest.raises(SystemExit):
        example().main(["--batch", "33"])
