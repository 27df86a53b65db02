"""Page plans and releases of batches around the sizes at which the requests' scan needs more than
the usual 48 KB of shared memory, each as the first call of its process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A plan in one launch (few words of output), one in two, and releases: every request takes two pages
# and gives one back.
SCRIPT = r'''
import sys
sys.path.insert(0, ROOT)
import torch
import gated_deltanet_linear_13_gb300 as gdn
gdn.load_library()

def i32(*x, fill=0):
    return torch.full(x, fill, dtype=torch.int32, device="cuda")

for columns in (2, 40):
    pool = dict(table=i32(B, columns), held=i32(B), free_count=i32(1, fill=2 * B),
                free_pages=torch.arange(2 * B, dtype=torch.int32, device="cuda"))
    slots, positions = i32(17 * B), i32(17 * B)
    gdn.gdn_page_plan(i32(B), i32(B, fill=17), slots, positions, **pool, page_size=16)
    assert gdn.gdn_get_device_error() == 0
    first = 2 * B - 1 - 2 * torch.arange(B, device="cuda")       # each request's first page
    token = torch.arange(17, device="cuda")
    page = first[:, None] - token // 16
    assert torch.equal(slots.view(B, 17).long(), page * 16 + token % 16)
    assert torch.equal(positions.view(B, 17).long(), token.expand(B, 17))
    assert int(pool["free_count"]) == 0 and bool((pool["held"] == 2).all())
    gdn.gdn_page_release(i32(B, fill=16), **pool, page_size=16)
    assert gdn.gdn_get_device_error() == 0
    assert int(pool["free_count"]) == B and bool((pool["held"] == 1).all())
    back = pool["free_pages"][:B].long().flip(0)
    assert torch.equal(back, first - 1)
print("clean")
'''


@pytest.mark.parametrize("b", [2418, 2419, 2440, 2457, 2458])
def test_as_the_first_call(b):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\nB = {b}\n" + SCRIPT],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "clean" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
