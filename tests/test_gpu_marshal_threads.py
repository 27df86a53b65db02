"""Other Python threads run while a call of the binding's native part launches (a launch waits where
the queue is full): the library's functions are replaced by one that sleeps."""
import ctypes
import os
import shutil
import subprocess
import sys
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def gdn(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    compiler = shutil.which("gcc") or shutil.which("cc") or shutil.which("g++")
    if compiler is None:
        pytest.skip("no C compiler")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    lib = m.load_library()
    source, slow = tmp_path / "slow.c", tmp_path / "slow.so"
    source.write_text("#include <unistd.h>\nint slow(void) { usleep(400000); return 0; }\n")
    subprocess.run([compiler, "-shared", "-fPIC", str(source), "-o", str(slow)], check=True)
    address = ctypes.cast(ctypes.CDLL(str(slow)).slow, ctypes.c_void_p).value
    m._native.bind(*[address] * 4, torch._C._cuda_getCurrentRawStream)
    yield m
    m._bind_marshal(lib)


def test_threads_run_beside_a_launch(gdn):
    i32 = dict(device="cuda", dtype=torch.int32)
    pool = dict(table=torch.zeros(2, 2, **i32), held=torch.zeros(2, **i32),
                free_pages=torch.zeros(4, **i32), free_count=torch.zeros(1, **i32), page_size=16)
    two, q = torch.zeros(2, **i32), torch.zeros(2, 1, 128, device="cuda")
    logits, ws = torch.zeros(2, 1, 30, device="cuda"), torch.zeros(4096, device="cuda", dtype=torch.uint8)
    steps = torch.zeros(8, device="cuda", dtype=torch.int64)
    calls = (lambda: gdn.gdn_qk_norm_rope(q, q, two, steps, q, q),
             lambda: gdn.gdn_page_plan(two, two, **pool),
             lambda: gdn.gdn_page_release(two, **pool),
             lambda: gdn.gdn_verify_tokens(logits, two[:, None], two, clocks=logits[:, 0], workspace=ws))
    turns, over = [0], threading.Event()

    def work():
        while not over.is_set():
            turns[0] += 1
            time.sleep(0.001)

    thread = threading.Thread(target=work)
    thread.start()
    try:
        for call in calls:
            time.sleep(0.05)
            before, t0 = turns[0], time.monotonic()
            call()
            during, took = turns[0] - before, time.monotonic() - t0
            assert took >= 0.35                          # it was the sleeping function
            assert during >= 20                          # (some 300; one where the lock is held)
    finally:
        over.set()
        thread.join()


def test_threads_call_at_once():
    """Two threads with a stream, tensors and a workspace each, calling side by side: the results of
    the same calls one after the other."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_step_streams import Step
    import gated_deltanet_linear_13_gb300 as gdn
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    gdn.load_library()

    def run(step, stream, rounds):
        with torch.cuda.stream(stream):
            for _ in range(rounds):
                step.plan()
                step.rotate()
                step.verify()
                step.release()

    wants, steps = ([Step(gdn, seed) for seed in (3, 4)] for _ in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for step in wants:
        run(step, torch.cuda.current_stream(), 300)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(s, t, 300)) for s, t in zip(steps, streams)]
    for thread in threads:
        thread.start()
    for thread in threads:
        thread.join()
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == 0
    for want, step in zip(wants, steps):
        for a, b in zip(want.state(), step.state()):
            assert torch.equal(a, b)
