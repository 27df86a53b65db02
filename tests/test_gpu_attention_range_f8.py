"""Shared-prefix attention, 8-bit cache, where the scores are large: against softmax in 64 bits over
what the cache stands for.

The queries are powers of two that lie within 2^10 of each other (which two e4m3 numbers hold), and
the scores of a row lie further apart than fp32 rounds them, or are equal.  Bounds as for the
operator's other tests: (2^-9 + 2^-10) sum_j p_j |v_j| per element, lse 2e-5 (1 + |lse|).
"""
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


H, GROUP, PAGE = 2, 3, 32


def _run(gdn, k, q, prefix, own, scale, seed, one_size=False):
    """Keys k [n, H, D] of prefix + 2 own tokens, random values; q [2, 1, H GROUP, D]."""
    n, d = k.shape[0], k.shape[-1]
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(n, H, d, generator=g, device="cuda").to(torch.bfloat16)
    if one_size:
        v[..., 0] = 5.0
    i32 = dict(dtype=torch.int32, device="cuda")
    shared, each = -(-prefix // PAGE), -(-own // PAGE)
    pages = shared + 2 * each
    at = torch.cat([torch.arange(prefix, device="cuda")] + [
        (shared + b * each) * PAGE + torch.arange(own, device="cuda") for b in range(2)])
    c = [torch.zeros(pages, H, PAGE, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
         for _ in range(2)]
    e = [torch.full((pages, H, PAGE), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = at.to(torch.int32)
    gdn.gdn_kv_cache_append(k, v, *c, slots, k_exp=e[0], v_exp=e[1])
    ks, vs = torch.empty(n, H, d, device="cuda"), torch.empty(n, H, d, device="cuda")
    gdn.gdn_kv_cache_read(*c, slots, ks, vs, k_exp=e[0], v_exp=e[1])
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    gdn.gdn_prefix_attention(
        q, *c, out, lse=lse, scale=scale, prefix_pages=torch.arange(shared, **i32),
        prefix_len=prefix, pages=(shared + torch.arange(2 * each, **i32)).reshape(2, each),
        kv_len=torch.full((2,), own, **i32), k_exp=e[0], v_exp=e[1])
    assert gdn.gdn_get_device_error() == 0
    scale = float(torch.tensor(scale, dtype=torch.float32))
    for b in range(2):
        seen = list(range(prefix)) + list(range(prefix + b * own, prefix + (b + 1) * own))
        for h in range(H):
            keys, vals = ks[seen, h].double(), vs[seen, h].double()
            hs = slice(h * GROUP, (h + 1) * GROUP)
            s = q[b, 0, hs].double() @ keys.T * scale
            z, p = torch.logsumexp(s, -1), torch.softmax(s, -1)
            tol = (2.0 ** -9 + 2.0 ** -10) * (p @ vals.abs()) + 1e-6
            err = (out[b, 0, hs].double() - p @ vals).abs()
            assert bool((err <= tol).all()), (b, h, float(err.max()))
            assert bool(((lse[b, 0, hs].double() - z).abs() <= 2e-5 * (1 + z.abs())).all())


@pytest.mark.parametrize("prefix,own", [(0, 1), (0, 90), (4000, 1), (5000, 200)])
@pytest.mark.parametrize("power", list(range(20, 31)) + [33, 40, 60])
@pytest.mark.parametrize("sign", [1, -1])
def test_equal_and_far_scores(gdn, sign, power, prefix, own):
    """Scores of 2^power, and some lower by a multiple of their 2^-9; values of one size, so that the
    equal ones stay equal with the values' exponents."""
    g = torch.Generator(device="cuda").manual_seed(power + prefix)
    d, n = 128, prefix + 2 * own
    k = torch.zeros(n, H, d, device="cuda")
    k[..., 5] = sign * 2.0 ** (power // 2)
    k[..., 77] = -(2.0 ** (power // 2)) * torch.randint(0, 4, (n, H), generator=g, device="cuda")
    q = torch.zeros(2, 1, H * GROUP, d, device="cuda")
    q[..., 5] = 2.0 ** (power - power // 2)
    q[..., 77] = 2.0 ** (power - power // 2 - 9)
    _run(gdn, k.to(torch.bfloat16), q.to(torch.bfloat16), prefix, own, 1.0, power, one_size=True)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("size", [1e2, 3e3, 1e4, 1e5, 1e6])
def test_random_operands_of_great_size(gdn, size, d):
    """The largest score takes all (further from the next than the products round)."""
    g = torch.Generator(device="cuda").manual_seed(int(size) + d)
    k = torch.randn(700 + 80, H, d, generator=g, device="cuda")
    k[torch.arange(0, 780, 7, device="cuda")] = 0.0
    q = 2.0 ** torch.randint(0, 7, (2, 1, H * GROUP, d), generator=g, device="cuda").float()
    q = q * (2.0 * torch.randint(0, 2, q.shape, generator=g, device="cuda") - 1)
    _run(gdn, (size * k).to(torch.bfloat16), (2.0 ** round(size ** 0.2) * q).to(torch.bfloat16),
         700, 40, 1.0, 9)
