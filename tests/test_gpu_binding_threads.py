"""Other Python threads run while a call of the compiled binding waits in the library (for room in the launch queue, say).
The waiting is done by a function on the host that stands in for the library's."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

import fp8_block_scaled_quant_gb300 as fb

pytestmark = pytest.mark.gpu
WAIT_S = 0.4


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("slow")
    (d / "slow.cpp").write_text('#include <unistd.h>\nextern "C" int slow() { usleep(%d); return 0; }\n' % int(WAIT_S * 1e6))
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(d / "slow.so"), str(d / "slow.cpp")], check=True)
    return ctypes.CDLL(str(d / "slow.so"))


def setup(replaced):
    names = ["fp8blk_status_string"] + [n for n in fb.header_functions() if "fp4" in n or "residual_norm" in n]
    at = {n: ctypes.cast(getattr(fb.lib(), n), ctypes.c_void_p).value for n in names}
    fb._native().setup({**at, **replaced}, fb.Fp8BlkError, fb._ws_cache, fb._buffer)


@pytest.mark.parametrize("name", ["fp4_quant", "fp4_dequant", "fp4_gemm", "fp4_linear", "residual_norm"])
def test_other_threads_run_while_a_call_waits(slow, name):
    x = torch.randn(4, 256, device="cuda").bfloat16()
    q = fb.fp4_quant(x)
    torch.cuda.synchronize()
    one = torch.ones(256, device="cuda")
    call = {"fp4_quant": lambda: fb.fp4_quant(x), "fp4_dequant": lambda: fb.fp4_dequant(*q),
            "fp4_gemm": lambda: fb.fp4_gemm(*q, *q), "fp4_linear": lambda: fb.fp4_linear(x, *q),
            "residual_norm": lambda: fb.residual_norm(x, None, one)}[name]
    call()
    turns, done = 0, threading.Event()

    def work():
        call()
        done.set()

    setup({"fp8blk_" + name: ctypes.cast(slow.slow, ctypes.c_void_p).value})
    try:
        t = threading.Thread(target=work)
        t.start()
        while not done.is_set():
            turns += 1
            time.sleep(WAIT_S / 100)
        t.join()
    finally:
        setup({})
    assert turns > 20, turns      # (about 100; one or two where the lock is held)


def test_refusals_from_threads():
    """What a call refuses reaches the thread that made it, and the others go on."""
    x = torch.randn(4, 256, device="cuda").bfloat16()
    got = []

    def work(bad):
        for _ in range(200):
            try:
                fb.fp4_quant(torch.randn(4, 264, device="cuda").bfloat16()[:, 1:257] if bad else x)
                got.append((bad, False))
            except fb.Fp8BlkError:
                got.append((bad, True))

    ts = [threading.Thread(target=work, args=(i % 2 == 0,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert len(got) == 800 and all(bad == refused for bad, refused in got)
