"""Where the full-attention layers' operators write and read: their index checks in the
-DGDN_BOUNDS_CHECK build, and what lies around a workspace of the reported size and around the
outputs."""
import os
import subprocess
import sys

import pytest
import torch

from gated_deltanet_linear_13_gb300 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILES = ["kv_cache.cu", "logprobs.cu", "prefix_attention.cu"]


@pytest.mark.parametrize("name", FILES)
def test_kernels_have_index_checks(name):
    """Every kernel source of the library checks its computed indices in the checked build."""
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
import test_gpu_attention_range as far
import test_gpu_logprobs_range as logits
import test_gpu_serving as t

# each of these compares with the definition and asks for a clean error word
for fmt in ("f8", "bf16"):
    t.test_append_and_read(gdn, fmt, 77, 4, 256, 64, torch.bfloat16)
    t.test_append_and_read(gdn, fmt, 333, 3, 128, 16, torch.float32)
    for i in range(len(t.ATTENTION)):
        b, tokens, hq, h, d, prefix, lens, page = t.ATTENTION[i]
        case = t._attention_case(b, tokens, hq, h, d, prefix, lens, page, fmt, seed=100 + i)
        t._check_attention(gdn, case)
        t._check_attention(gdn, case, odt=torch.float32)
    t.test_attention_very_long_prefix(gdn, fmt, 140001 if fmt == "bf16" else 270000)
t.test_attention_many_sequences(gdn)
far.test_scores_of_any_size(gdn, "raw", 40, -1.0, 5000, 200)
far.test_scores_of_any_size(gdn, "nat", 60, 1.0, 0, 1)
for dtype in (torch.bfloat16, torch.float32):
    for n, v, k in ((1, 1, 1), (2, 31, 31), (3, 1000, 5), (1, 4097, 32), (5, 12345, 20),
                    (1, 248320, 20), (40, 70001, 3), (400, 3001, 2), (1300, 1501, 4)):
        t.test_logprobs(gdn, n, v, k, dtype)
    t.test_logprobs_strides_and_alignment(gdn, dtype)
    t.test_logprobs_hard_rows(gdn, 1500, dtype)
    t.test_logprobs_hard_rows(gdn, 100003, dtype)
    logits.test_large_finite_masks(gdn, 10.0, dtype)
print("serving operators, bounds-checked build: clean")
'''


@pytest.mark.gpu
def test_bounds_checked_build_runs_clean():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + SCRIPT], capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "bounds-checked build: clean" in r.stdout


GUARD = 8192                                     # bytes on either side


class _Guarded:
    """Tensors cut out of larger buffers, whose rest has to stay as it is."""

    def __init__(self):
        self.buffers = []

    def __call__(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.buffers.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).reshape(shape)

    def untouched(self):
        return all(bool((b[:GUARD] == 0xA5).all()) and bool((b[GUARD + n:] == 0xA5).all())
                   for b, n in self.buffers)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 3e5])
@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("b,t,hq,h,d,prefix,own,page", [
    (1, 1, 1, 1, 128, 0, 1, 16), (1, 1, 24, 4, 256, 512, 37, 64), (3, 2, 6, 2, 128, 127, 130, 32),
    (5, 1, 3, 1, 128, 0, 513, 16), (2, 130, 6, 1, 256, 300, 257, 64), (1, 33, 32, 4, 128, 77, 400, 16),
    (40, 1, 24, 4, 256, 650, 300, 32), (300, 1, 4, 2, 128, 256, 40, 16),
    (7, 33, 8, 2, 128, 9000, 90, 128), (2, 33, 4, 2, 256, 140001, 200, 128)])
def test_attention_writes_its_own(b, t, hq, h, d, prefix, own, page, fmt, size):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as gdn
    build_lib.build()
    gdn.load_library()
    f8 = fmt == "f8"
    g = torch.Generator(device="cuda").manual_seed(b * prefix + own)
    shared, each = -(-prefix // page), -(-own // page)
    pages = shared + b * each
    cache = [torch.randn(pages, h, page, d, generator=g, device="cuda").to(
        torch.float8_e4m3fn if f8 else torch.bfloat16) for _ in range(2)]
    exps = [torch.full((pages, h, page), 127, dtype=torch.uint8, device="cuda") if f8 else None
            for _ in range(2)]
    i32 = dict(dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    make = _Guarded()
    q = (size * torch.randn(b, t, hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    for odt in (torch.bfloat16, torch.float32):
        out, lse = make(q.shape, odt), make(q.shape[:3], torch.float32)
        ws = make((gdn.gdn_prefix_attention_workspace_size(b, t, hq, h, d),), torch.uint8)
        gdn.gdn_prefix_attention(
            q, *cache, out, prefix_pages=order[:shared], prefix_len=prefix,
            pages=order[shared:].reshape(b, each),
            kv_len=torch.randint(-1, own + 1, (b,), generator=g, device="cuda").to(torch.int32),
            k_exp=exps[0], v_exp=exps[1], lse=lse, workspace=ws)
        assert gdn.gdn_get_device_error() == 0
        assert bool(out.isfinite().all())
    assert make.untouched()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v,k", [(1, 1, 1), (2, 31, 31), (3, 1000, 5), (1, 4097, 32), (1, 248320, 20),
                                   (400, 3001, 2), (1300, 1501, 4), (9000, 700, 0), (64, 50001, 0)])
def test_logprobs_write_their_own(n, v, k, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as gdn
    build_lib.build()
    gdn.load_library()
    g = torch.Generator(device="cuda").manual_seed(n + v)
    make = _Guarded()
    x = torch.randn(n, v, generator=g, device="cuda").to(dtype)
    targets = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = make((n,), torch.float32), make((n,), torch.float32)
    ids, tl = (make((n, k), dt) if k else None for dt in (torch.int32, torch.float32))
    ws = make((gdn.gdn_token_logprobs_workspace_size(n, v, k, dtype),), torch.uint8)
    gdn.gdn_token_logprobs(x, targets, lp, ent, top_ids=ids, top_logprobs=tl, workspace=ws)
    assert gdn.gdn_get_device_error() == 0
    assert bool(lp.isfinite().all() & ent.isfinite().all())
    assert make.untouched()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("n,h,d", [(1, 1, 128), (37, 3, 256), (333, 8, 128)])
def test_cache_calls_write_their_own(n, h, d, fmt):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as gdn
    build_lib.build()
    gdn.load_library()
    f8, page = fmt == "f8", 16
    pages = -(-n // page)
    make = _Guarded()
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    cache = [make((pages, h, page, d), dt) for _ in range(2)]
    exps = [make((pages, h, page), torch.uint8) if f8 else None for _ in range(2)]
    k, v = (torch.randn(n, h, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_append(k, v, *cache, slots, k_exp=exps[0], v_exp=exps[1])
    for odt in (torch.bfloat16, torch.float32):
        ko, vo = make((n, h, d), odt), make((n, h, d), odt)
        gdn.gdn_kv_cache_read(*cache, slots, ko, vo, k_exp=exps[0], v_exp=exps[1])
        assert gdn.gdn_get_device_error() == 0
        if not f8:
            assert torch.equal(ko.bfloat16(), k) and torch.equal(vo.bfloat16(), v)
    assert make.untouched()
