"""The compiled calls let other Python threads run while an entry point does: a launch into a
full queue waits, perhaps for something that another thread has yet to do.  Here the entry
points are a function that sleeps, and the tensors say what a GPU's would."""
import shutil
import subprocess
import threading
import time

import pytest
import torch

import nvfp4_token_routed_gb300 as M
from nvfp4_token_routed_gb300 import experts

SLEEP = 0.4
STUB = """
#include <stddef.h>
#include <time.h>
int calls = 0;
int stall(void) {
  struct timespec t = {0, 400000000};
  nanosleep(&t, NULL);
  ++calls;
  return 0;
}
size_t bytes(void) { return 256; }
"""


class Fake:
    """A contiguous tensor on device 0 at an address that nobody looks at."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype = tuple(shape), dtype

    def get_device(self):
        return 0

    def stride(self):
        return (self.shape[1], 1) if len(self.shape) == 2 else (1,)

    def data_ptr(self):
        return 4096

    def is_contiguous(self):
        return True


@pytest.fixture
def calls(tmp_path):
    import ctypes as C
    from nvfp4_token_routed_gb300 import build
    build.build()
    L = M.lib()
    calls = pytest.importorskip("nvfp4_token_routed_gb300._calls")
    if not shutil.which("gcc"):
        pytest.skip("no gcc")
    src, so = tmp_path / "stub.c", tmp_path / "stub.so"
    src.write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    stub = C.CDLL(str(so))
    at = [C.cast(stub.stall, C.c_void_p).value] * 10 + [C.cast(stub.bytes, C.c_void_p).value]
    calls.attach((Fake, lambda size, stride, dtype: Fake(size, dtype), lambda: 0, lambda dev: 0),
                 (torch.float32, torch.bfloat16, torch.float16, torch.uint8, torch.int32,
                  torch.int64), (M.MxTensor, M.Checkpoint, M.RoutePlan), tuple(at))
    yield calls, C.c_int.in_dll(stub, "calls")
    experts._attach(L)
    assert experts._fast is calls


def test_other_threads_run_during_a_call(calls):
    calls, entered = calls
    bf, i32 = torch.bfloat16, torch.int32
    x, rows, w = Fake((4, 64), bf), Fake((8, 64), bf), Fake((4, 2), torch.float32)
    ids = Fake((4, 2), i32)
    plan = M.RoutePlan(Fake((9,), i32), Fake((8,), i32), ids)
    stopped, longest = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stopped.is_set():
            time.sleep(0.002)
            now = time.perf_counter()
            longest[0] = max(longest[0], now - last)
            last = now

    quantised, kept = [], []
    todo = [lambda: calls.sort_routes(ids, 8), lambda: calls.dispatch(x, plan, None),
            lambda: calls.combine(rows, plan, w),
            lambda: calls.combine_grad(rows, plan, w, x, None),
            lambda: kept.append(calls.checkpoint(x)) or kept[0],
            lambda: calls.restore(kept[0]),
            lambda: kept.append(calls.expert_act(x, "relu2", 0.0, True)[1]) or kept[1],
            lambda: calls.expert_act_grad(kept[1], x),
            lambda: quantised.append(calls.mx_quantize(x)) or quantised[0],
            lambda: calls.mx_product(quantised[0], quantised[0], None, bf)]
    thread = threading.Thread(target=tick)
    thread.start()
    try:
        for i, f in enumerate(todo):
            time.sleep(0.01)
            longest[0] = 0.0
            assert f() is not None, i
            time.sleep(0.01)
            assert entered.value == i + 1
            # held, the lock would stop the other thread for as long as the entry point sleeps
            assert longest[0] < 0.9 * SLEEP, i
    finally:
        stopped.set()
        thread.join()
