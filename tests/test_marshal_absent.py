"""Without the binding's native part, or with one that was built against another torch, the library
is there all the same: calls are checked and marshalled in Python."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

# `how` is what stands in the place of the native part before the library is loaded
START = r'''
import sys, types
sys.path.insert(0, ROOT)
sys.path.insert(0, ROOT + "/tests")
import torch
import gated_deltanet_linear_13_gb300 as gdn
part = None                                              # cannot be imported
if HOW == "other torch":
    def never(*args):
        raise AssertionError("the other torch's native part was used")
    part = types.ModuleType("_marshal")
    part.torch_version = "1.0.0"
    part.bind = part.qk_norm_rope = part.page_plan = part.page_release = part.verify_tokens = never
    gdn._marshal = part
sys.modules["gated_deltanet_linear_13_gb300._marshal"] = part
gdn.load_library()
'''

REFUSALS = r'''
import test_step_abi
assert gdn.load_library().gdn_version() > 0
steps, amplitude = gdn.gdn_rope_phase_steps(64, device="cpu")
assert steps.shape == (32,) and amplitude == 1.0
test_step_abi.test_binding_needs_cuda_tensors()
print("clean")
'''

OPERATORS = r'''
import test_gpu_marshal
torch.save([x.cpu() for x in test_gpu_marshal._run_all()], OUT)
assert gdn.gdn_get_device_error() == 0
print("clean")
'''


def _child(how, script, **names):
    head = "".join(f"{n} = {x!r}\n" for n, x in dict(ROOT=ROOT, HOW=how, **names).items())
    r = subprocess.run([sys.executable, "-c", head + START + script], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "clean" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.parametrize("how", ["missing", "other torch"])
def test_the_library_loads(how):
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    _child(how, REFUSALS)


def test_the_native_part_is_used():
    import gated_deltanet_linear_13_gb300 as gdn
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    gdn.load_library()
    assert gdn._native.torch_version == str(torch.__version__)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["missing", "other torch"])
def test_operators_run(how, tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as gdn
    import test_gpu_marshal
    test_gpu_marshal._native()
    out = str(tmp_path / "out.pt")
    _child(how, OPERATORS, OUT=out)
    for a, b in zip(torch.load(out), test_gpu_marshal._run_all(), strict=True):
        assert torch.equal(a, b.cpu())
    assert gdn.gdn_get_device_error() == 0
