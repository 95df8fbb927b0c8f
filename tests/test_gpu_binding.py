"""The module that passes tensors to the library: while the library works,
which may wait for room in a full queue, other Python threads run."""
import sys
import threading
import time

import pytest
import torch

from tests.gpu_common import gpu_available
from tests.test_gpu_experts_float import _calls

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("call", ["quantize", "dispatch", "matmul", "matmul_f8", "layer"])
def test_other_threads_run_during_calls(call):
    """No thread is made to give up the interpreter's lock (the switch interval is longer than the test), so a thread
    that waits for it gets it only from one that gives it up by itself."""
    fn, good = _calls()[call]
    fn(**good)
    torch.cuda.synchronize()
    turns, stop = [0], threading.Event()

    def other():
        while not stop.is_set():
            turns[0] += 1
            time.sleep(1e-4)

    interval = sys.getswitchinterval()
    thread = threading.Thread(target=other, daemon=True)
    thread.start()
    while turns[0] == 0:
        time.sleep(1e-3)
    sys.setswitchinterval(1000)
    try:
        before = turns[0]
        for _ in range(4000):
            fn(**good)
            if turns[0] >= before + 3:
                break
        after = turns[0]
    finally:
        sys.setswitchinterval(interval)
        stop.set()
    thread.join()
    torch.cuda.synchronize()
    assert after >= before + 3
