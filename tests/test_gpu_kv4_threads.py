"""Calls on the 4-bit cache beside other Python threads."""
import threading
import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dynamic_sparse_attention_head_b200 as msa  # noqa: E402


def _longest_pause(call):
    """Seconds for which another thread stood still at most while `call` ran, and how long that was."""
    pauses, stop, up = [0.0], threading.Event(), threading.Event()

    def beat():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            pauses[0] = max(pauses[0], now - last)
            last = now
            up.set()

    t = threading.Thread(target=beat)
    t.start()
    up.wait()
    pauses[0], t0 = 0.0, time.perf_counter()
    call()
    took = time.perf_counter() - t0
    stop.set()
    t.join()
    return pauses[0], took


def _busy(seconds):
    torch.cuda._sleep(int(seconds * 1.9e9))  # cycles: a bounded wait on the device


@pytest.mark.parametrize("launches", [0, 3000])
def test_other_threads_run_while_a_call_waits(launches):
    """The status call waits for the stream; 3000 launches behind a busy kernel wait for room in its queue."""
    cache = msa.KV4Cache.alloc(2, 1, 16, 64)
    x = torch.ones(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    cache.append(x, x, slot)
    assert cache.device_status() == 0

    def call():
        _busy(0.6)
        for _ in range(launches):
            cache.append(x, x, slot)
        assert cache.device_status() == 0

    pause, took = _longest_pause(call)
    assert took > 0.4 and pause < 0.25, f"a thread stood still for {pause:.2f} of {took:.2f} s"
