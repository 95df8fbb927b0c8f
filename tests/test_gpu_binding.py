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


def test_calls_without_it_give_the_same(monkeypatch):
    """Where the module cannot be used every call goes through ctypes: the same bits."""
    import expert_grouping_dispatch_amd as mod
    from expert_grouping_dispatch_amd import experts, experts_float

    g = torch.Generator(device="cuda").manual_seed(1)

    def outputs():
        out = []
        for call, (fn, good) in _calls().items():
            g.manual_seed(2)
            for name in ("x", "input_tokens", "a", "w", "w_gate_up", "w_down"):
                if name in good:
                    good[name].copy_(torch.randn(good[name].shape, generator=g, device="cuda").to(good[name].dtype))
            for name in ("out_q", "out_scales", "out", "output_tokens"):  # some rows are left as they were
                if name in good:
                    good[name].view(torch.uint8).zero_()
            fn(**good)
            out += [good[n].clone() for n in ("out_q", "out_scales", "out", "output_tokens") if n in good]
        return [t.view(torch.uint8) for t in out]

    assert isinstance(experts_float._fast, type(sys))
    with_it = outputs()
    for m in (experts, experts_float):
        monkeypatch.setattr(m, "_fast", mod._CheckInPython())
    for a, b in zip(with_it, outputs()):
        assert torch.equal(a, b)
