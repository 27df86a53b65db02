"""Shared-prefix attention, bf16 cache, where the scores are large: against softmax in 64 bits.

The queries and keys are such that every score is exact in fp32 (a whole number of units of its
last place), so the definition's differences between scores are what the kernel has to use: a
row's result may not depend on how the scores' size rounds.  Bounds as for the operator's other
tests: (2^-9 + 2^-10) sum_j p_j |v_j| per element, lse 2e-5 (1 + |lse|).
"""
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


D, H, GROUP, PAGE = 128, 2, 3, 32


def _case(rows, prefix, own, seed):
    """keys and values [tokens, H, D] of a prefix and of two sequences, and their cache."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shared, each = -(-prefix // PAGE), -(-max(own, 1) // PAGE)
    pages = shared + 2 * each
    k = rows(g, pages * PAGE)
    v = torch.randn(pages * PAGE, H, D, generator=g, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    pack = lambda x: x.reshape(pages, PAGE, H, D).transpose(1, 2).contiguous()      # noqa: E731
    return dict(k=k, v=v, kc=pack(k), vc=pack(v), prefix=prefix, own=own,
                prefix_pages=torch.arange(shared, **i32),
                pages=(shared + torch.arange(2 * each, **i32)).reshape(2, each),
                own_at=[(shared + i * each) * PAGE for i in range(2)])


def _check(gdn, c, q, scale):
    out = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    gdn.gdn_prefix_attention(
        q, c["kc"], c["vc"], out, lse=lse, scale=scale, prefix_pages=c["prefix_pages"],
        prefix_len=c["prefix"], pages=c["pages"],
        kv_len=torch.full((2,), c["own"], dtype=torch.int32, device="cuda"))
    assert gdn.gdn_get_device_error() == 0
    scale = float(torch.tensor(scale, dtype=torch.float32))
    for b in range(2):
        at = slice(c["own_at"][b], c["own_at"][b] + c["own"])
        for h in range(H):
            keys, vals = (torch.cat([c[n][:c["prefix"], h], c[n][at, h]]).double() for n in "kv")
            hs = slice(h * GROUP, (h + 1) * GROUP)
            s = q[b, 0, hs].double() @ keys.T * scale
            z = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            tol = (2.0 ** -9 + 2.0 ** -10) * (p @ vals.abs()) + 1e-6
            err = (out[b, 0, hs].double() - p @ vals).abs()
            assert bool((err <= tol).all()), (b, h, float(err.max()))
            assert bool(((lse[b, 0, hs].double() - z).abs() <= 2e-5 * (1 + z.abs())).all())


@pytest.mark.parametrize("prefix,own", [(0, 1), (0, 90), (4000, 1), (5000, 200)])
@pytest.mark.parametrize("power,lead", [(20, 1.0), (22, -1.0), (24, 1.0), (27, -1.0), (27, 1.0),
                                        (33, 1.0), (40, -1.0), (60, 1.0), (33, 1.5), (34, -1.5)])
@pytest.mark.parametrize("unit", ["nat", "raw"])
def test_scores_of_any_size(gdn, unit, power, lead, prefix, own):
    """Scores of lead 2^power and a few units of their last place more, at a scale that makes such
    a unit one (nat), or at scale 1 (raw): far past what 2^score, or a rounding of it, could hold.
    (With a lead of 1.5 scores that differ by a unit are the same once scaled by log2 e.)"""
    # at least a unit of the last place of all scores
    last = 2.0 ** (power - (22 if abs(lead) == 1.0 else 23))

    def rows(g, n):
        k = torch.zeros(n, H, D, device="cuda")
        k[..., 5] = lead * 2.0 ** (power // 2)
        k[..., 77] = torch.randint(-3, 4, (n, H), generator=g, device="cuda").float()
        return k.to(torch.bfloat16)

    c = _case(rows, prefix, own, power + prefix)
    q = torch.zeros(2, 1, H * GROUP, D, device="cuda")
    q[..., 5] = 2.0 ** (power - power // 2)
    q[..., 77] = last
    _check(gdn, c, q.to(torch.bfloat16), 1.0 / last if unit == "nat" else 1.0)


@pytest.mark.parametrize("size", [1e4, 1e5, 1e6])
def test_random_operands_of_great_size(gdn, size):
    """Scores of about 1e8 to 1e12 of both signs: the largest takes all (further from the next
    than the products round)."""
    def rows(g, n):
        k = torch.randn(n, H, D, generator=g, device="cuda")
        k[torch.arange(0, n, 7, device="cuda")] = 0.0
        return (size * k).to(torch.bfloat16)

    c = _case(rows, 700, 40, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    q = (size * torch.randn(2, 1, H * GROUP, D, generator=g, device="cuda")).to(torch.bfloat16)
    _check(gdn, c, q, 1.0)
