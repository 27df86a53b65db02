"""Shared-prefix attention with infinities and NaN in queries and keys, and with a scale of zero:
what include/gdn.h promises of each cache format."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


H, PAGE = 2, 16


def _attend(gdn, fmt, q, k, v, scale):
    """One sequence of the keys and values k, v [n, H, D] (all own tokens, queries q [1, T, Hq, D])."""
    n, _, d = k.shape
    pages = -(-n // PAGE)
    i32 = dict(dtype=torch.int32, device="cuda")
    f8 = fmt == "f8"
    c = [torch.zeros(pages, H, PAGE, d * (1 if f8 else 2), dtype=torch.uint8, device="cuda").view(
        torch.float8_e4m3fn if f8 else torch.bfloat16) for _ in range(2)]
    e = [torch.full((pages, H, PAGE), 127, dtype=torch.uint8, device="cuda") if f8 else None
         for _ in range(2)]
    gdn.gdn_kv_cache_append(k, v, *c, torch.arange(n, **i32), k_exp=e[0], v_exp=e[1])
    out = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    gdn.gdn_prefix_attention(q, *c, out, pages=torch.arange(pages, **i32)[None],
                             kv_len=torch.tensor([n], **i32), k_exp=e[0], v_exp=e[1], lse=lse,
                             scale=scale)
    assert gdn.gdn_get_device_error() == 0
    return out, lse


def _inputs(n, d, t=1, hq=4):
    g = torch.Generator(device="cuda").manual_seed(n + d)
    q, k, v = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
               for s in ((1, t, hq, d), (n, H, d), (n, H, d)))
    return q, k, v


@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_scale_of_zero(gdn, fmt, d, bad):
    """0 * score: every visible key weighs the same, and what is not finite stays so."""
    q, k, v = _inputs(150, d)
    q[0, 0, 1, 3] = bad
    out, lse = _attend(gdn, fmt, q, k, v, 0.0)
    assert bool(out[0, 0, 1].isnan().all()) and bool(lse[0, 0, 1].isnan())
    want = v.double().mean(0)                               # e4m3 holds a value to 2^-4, 150 of them
    for h in (0, 2, 3):
        assert float((out[0, 0, h].double() - want[h // 2]).abs().max()) <= (
            2.0 ** -4 * float(v.abs().double().mean()) if fmt == "f8" else 1e-5)
        assert abs(float(lse[0, 0, h]) - math.log(150)) <= 2e-5


@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_infinite_query_on_keys_of_the_other_sign(gdn, scale):
    """bf16 cache: every score is -inf, so the row has nothing; 8-bit cache: the row is NaN."""
    for n in (1, 140):
        q, k, v = _inputs(n, 128)
        k[..., 7] = -2.0
        q[0, 0, 1, 7] = math.copysign(math.inf, scale)
        for fmt in ("bf16", "f8"):
            out, lse = _attend(gdn, fmt, q, k, v, scale)
            if fmt == "bf16":
                assert not bool(out[0, 0, 1].any()) and float(lse[0, 0, 1]) == -math.inf
            else:
                assert bool(out[0, 0, 1].isnan().all()) and bool(lse[0, 0, 1].isnan())
            others = [0, 2, 3]
            assert bool(out[0, 0, others].isfinite().all() & lse[0, 0, others].isfinite().all())


def test_infinite_key_in_a_bf16_cache(gdn):
    """A score of +inf makes a row NaN, one of -inf is a key without weight."""
    q, k, v = _inputs(200, 128)
    k[50, 0, 9] = math.inf
    q[0, 0, :, 9] = torch.tensor([1.0, -1.0, 1.0, -1.0], device="cuda")
    out, lse = _attend(gdn, "bf16", q, k, v, 0.1)
    assert bool(out[0, 0, 0].isnan().all()) and bool(lse[0, 0, 0].isnan())
    keep = [i for i in range(200) if i != 50]
    s = k[keep, 0].double() @ q[0, 0, 1].double() * 0.1
    want = torch.softmax(s, 0) @ v[keep, 0].double()
    assert float((out[0, 0, 1].double() - want).abs().max()) <= 1e-3
    assert abs(float(lse[0, 0, 1]) - float(torch.logsumexp(s, 0))) <= 1e-4
    assert bool(out[0, 0, 2:].isfinite().all())
