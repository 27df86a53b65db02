"""Shared-prefix attention on a cache without pages: no row has a visible key."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("b,t", [(1, 1), (3, 2), (500, 1)])
def test_cache_without_pages(b, t, d, fmt):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as gdn
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    gdn.load_library()
    f8 = fmt == "f8"
    cache = [torch.empty(0, 2, 32, d, device="cuda",
                         dtype=torch.float8_e4m3fn if f8 else torch.bfloat16) for _ in range(2)]
    exps = [torch.empty(0, 2, 32, dtype=torch.uint8, device="cuda") if f8 else None
            for _ in range(2)]
    q = torch.randn(b, t, 6, d, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    for odt in (torch.bfloat16, torch.float32):
        out = torch.full(q.shape, 7.0, dtype=odt, device="cuda")
        lse = torch.full(q.shape[:3], 7.0, device="cuda")
        gdn.gdn_prefix_attention(q, *cache, out, pages=torch.empty(b, 0, **i32), lse=lse,
                                 kv_len=torch.arange(b, **i32) * 0 - (torch.arange(b, **i32) % 2),
                                 k_exp=exps[0], v_exp=exps[1])
        assert gdn.gdn_get_device_error() == 0
        assert not bool(out.any()) and bool((lse == -math.inf).all())
