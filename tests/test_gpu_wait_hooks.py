"""The hooks that make bounded waits run out, for tests, are their thread's
own: a call of another thread is not touched by them."""
import ctypes
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import Batch, randn, zp  # noqa: E402, F401


@pytest.fixture
def set_elsewhere(zp):  # noqa: F811
    """Sets a hook in a thread of its own, which stays until the test ends."""
    ends, threads = threading.Event(), []

    def start(name, which):
        hook = getattr(zp.lib(), name)
        hook.argtypes, hook.restype = [ctypes.c_int32, ctypes.c_uint64], None
        is_set = threading.Event()

        def run():
            hook(which, 20_000_000)
            is_set.set()
            ends.wait(60)
            hook(-1, 0)
        threads.append(threading.Thread(target=run))
        threads[-1].start()
        assert is_set.wait(60)
    yield start
    ends.set()
    for t in threads:
        t.join()


@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_attention_of_another_thread(zp, set_elsewhere, kernel):  # noqa: F811
    set_elsewhere("zero_test_window_attention_waits", kernel)
    b = Batch([(300, 300), (200, 400)], 4, 2, 64, "f16")
    b.check_forward(zp, 100, 2)  # (asks for stalls too)
    b.check_backward(zp, 100, 2)


@pytest.mark.parametrize("epilogue", [0, 1])
def test_gated_ffn_of_another_thread(zp, set_elsewhere, epilogue):  # noqa: F811
    set_elsewhere("zero_test_gated_ffn_waits", epilogue)
    m, d, f, dt = 200, 128, 256, torch.bfloat16
    x, wg, wu, wd = (randn(s, dt, 20 + k, 0.1) for k, s in enumerate([(m, d), (f, d), (f, d), (d, f)]))
    y, ws = torch.zeros_like(x), zp.new_gated_ffn_workspace(m, d, f)
    zp.zero_gated_ffn(x, wg, wu, wd, y, ws)
    assert zp.zero_workspace_stalls(ws) == 0
    assert bool(torch.isfinite(y).all()) and float(y.abs().max()) > 0
