"""Where the serving step's operators write and read: their index checks in the
-DGDN_BOUNDS_CHECK build, and what lies around outputs, pools and workspaces of the reported size."""
import os
import subprocess
import sys

import pytest
import torch

from gated_deltanet_linear_13_gb300 import build_lib

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["qk_norm_rope.cuh", "pages.cuh", "verify.cuh"])
def test_kernels_have_index_checks(name):
    with open(os.path.join(build_lib.CSRC, name)) as f:
        assert f.read().count("in_bounds(") >= 4


SCRIPT = r'''
import os, sys
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))
import torch
import gated_deltanet_linear_13_gb300 as gdn
from gated_deltanet_linear_13_gb300 import build_lib
gdn.load_library(build_lib.build(checked=True))
import test_gpu_pages as pages
import test_gpu_qk_norm_rope as rope
import test_gpu_verify as verify

# each of these compares with the definition and asks for a clean error word
for dtype in (torch.bfloat16, torch.float32):
    for inter in (False, True):
        for case in rope.CASES:
            rope.test_tensors(gdn, *case, dtype, inter)
        for fmt in ("bf16", "f8"):
            rope.test_cache(gdn, 77, 24, 4, 256, 250, 128, dtype, fmt, inter)
            rope.test_cache(gdn, 1500, 6, 3, 128, 32, 32, dtype, fmt, inter)
for b, rows, columns, page, most in ((1, 3, 700, 128, 50000), (64, 64, 60, 64, 900),
                                     (513, 700, 9, 32, 60), (8192, 8200, 2, 16, 6)):
    pages.test_steps_of_a_server(gdn, b, rows, columns, page, most)
pages.test_long_prompts(gdn)
pages.test_captured_steps(gdn)
for dtype in (torch.bfloat16, torch.float32):
    for drafts in ("logits", "ids"):
        for case in verify.CASES:
            verify.test_definition(gdn, *case, dtype, drafts)
    verify.test_strides_and_alignment(gdn, dtype)
    for v in (40, 5000, 100003):
        verify.test_masks(gdn, v, dtype)
print("step operators, bounds-checked build: clean")
'''


@pytest.mark.gpu
def test_bounds_checked_build_runs_clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + SCRIPT], capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "bounds-checked build: clean" in r.stdout


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    build_lib.build()
    m.load_library()
    return m


@pytest.fixture
def make():
    from test_gpu_serving_bounds import _Guarded
    return _Guarded()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("to", ["tensors", "bf16", "f8"])
@pytest.mark.parametrize("n,hq,h,d,rot", [(1, 3, 1, 128, 64), (37, 8, 2, 256, 250), (611, 5, 3, 128, 128),
                                          (3000, 2, 1, 256, 64), (259, 3, 2, 88, 40), (5, 2, 1, 8, 2)])
def test_norm_and_rotation_write_their_own(gdn, make, n, hq, h, d, rot, to, dtype):
    if to != "tensors" and d not in (128, 256):
        pytest.skip("a cache's heads have 128 or 256 elements")
    x = torch.randn(n, hq + 2 * h, d, device="cuda").to(dtype)
    positions = torch.arange(n, device="cuda", dtype=torch.int32)
    for interleaved in (False, True):
        steps, _ = gdn.gdn_rope_phase_steps(rot)
        out = dict(q_out=make((n, hq, d), dtype), k_out=make((n, h, d), dtype))
        kw = {}
        if to != "tensors":
            dt = torch.float8_e4m3fn if to == "f8" else torch.bfloat16
            shape = (-(-n // 16), h, 16, d)
            kw = dict(v=x[:, hq + h:], k_cache=make(shape, dt), v_cache=make(shape, dt),
                      slots=torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32))
            if to == "f8":
                kw |= dict(k_exp=make(shape[:3], torch.uint8), v_exp=make(shape[:3], torch.uint8))
        w = torch.ones(d, device="cuda")
        gdn.gdn_qk_norm_rope(x[:, :hq], x[:, hq:hq + h], positions, steps, **out, q_weight=w,
                             k_weight=w, interleaved=interleaved, **kw)
        assert gdn.gdn_get_device_error() == 0
        assert all(bool(t.isfinite().all()) for t in out.values())
    assert make.untouched()


@pytest.mark.gpu
@pytest.mark.parametrize("b,new,page,capacity", [(1, 1, 16, 1), (3, 40, 16, 130), (300, 2, 64, 601),
                                                 (40, 2000, 32, 80001), (8192, 1, 16, 8192)])
def test_plans_write_their_own(gdn, make, b, new, page, capacity):
    i32 = torch.int32
    columns = -(-new // page) + 1
    pool = dict(table=make((b, columns), i32), held=make((b,), i32),
                free_pages=make((b * columns,), i32), free_count=make((1,), i32))
    pool["held"].zero_()
    pool["free_pages"].copy_(torch.randperm(b * columns, device="cuda"))
    pool["free_count"].fill_(b * columns)
    out = dict(slots=make((capacity,), i32), positions=make((capacity,), i32),
               cu_seqlens=make((b + 1,), i32), kv_len_out=make((b,), i32), pages=make((b, columns), i32))
    zero, count = (torch.full((b,), x, device="cuda", dtype=i32) for x in (0, new))
    for capacity_left in (capacity, b * new - 1):           # the second is refused as a whole
        part = {**out, "slots": out["slots"][:capacity_left], "positions": out["positions"][:capacity_left]}
        gdn.gdn_page_plan(zero, count, **part, **pool, page_size=page)
        assert gdn.gdn_get_device_error() == (0 if capacity_left == capacity else 6)
        gdn.gdn_page_release(zero, **pool, page_size=page)
        assert gdn.gdn_get_device_error() == 0
        assert int(pool["free_count"]) == b * columns
    assert make.untouched()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("drafts", ["logits", "ids"])
@pytest.mark.parametrize("b,t,v", [(1, 0, 1), (1, 3, 31), (2, 1, 4097), (1, 2, 248320), (60, 4, 3001),
                                   (700, 0, 513), (3, 64, 700), (5000, 1, 40)])
def test_verification_writes_its_own(gdn, make, b, t, v, drafts, dtype):
    g = torch.Generator(device="cuda").manual_seed(b + v)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    i32, f32 = torch.int32, torch.float32
    out = dict(tokens=make((b, t + 1), i32), accepted=make((b,), i32), logprobs=make((b, t + 1), f32))
    kw = dict(clocks=torch.empty(b, v, device="cuda").exponential_(generator=g))
    if t:
        kw |= dict(draft_ids=torch.randint(0, v, (b, t), generator=g, device="cuda", dtype=i32),
                   accept_u=torch.rand(b, t, generator=g, device="cuda"),
                   draft_logits=rand(b, t, v) if drafts == "logits" else None)
    ws = make((gdn.gdn_verify_tokens_workspace_size(b, t, v, dtype, bool(t) and drafts == "logits"),),
              torch.uint8)
    gdn.gdn_verify_tokens(rand(b, t + 1, v), out.pop("tokens"), out.pop("accepted"),
                          logprobs=out["logprobs"], workspace=ws, **kw)
    assert gdn.gdn_get_device_error() == 0
    assert bool(out["logprobs"].isfinite().all())
    assert make.untouched()
    with pytest.raises(gdn.GDNError):
        gdn.gdn_verify_tokens(rand(b, t + 1, v), torch.zeros(b, t + 1, device="cuda", dtype=i32),
                              torch.zeros(b, device="cuda", dtype=i32), workspace=ws[:-1], **kw)
