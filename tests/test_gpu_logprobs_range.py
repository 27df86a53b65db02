"""Token log probabilities where the logits (or the scale) are large: against the definition in 64
bits, centred on the row's largest logit so that the reference itself loses nothing.

Bounds, with spread = sum_v p_v (m - x_v) in nats, m the row's largest x = scale * logit:
  * ln z: exponentials of 2^-22, their sums over a thread's few dozen terms and 32 x 5 joins 2e-6,
    the scale's and the exponents' rounding at 2^-23 of each term's own m - x (2^-23 spread):
    4e-6 + 2^-22 spread in all, whatever the size of m.
  * a log probability adds the rounding of its own (x - m): 2^-22 (m - x).
  * the entropy log z - w / z: 4e-6 (2 + spread).
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _same(got, want, tol, what):
    """got within tol of want (as fp32 holds it); infinities equal, no NaN."""
    want = want.float().double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    err = (got - want).abs()[~inf]
    bad = ~(err <= tol[~inf])                               # (a NaN is bad)
    assert not bool(bad.any()), (what, float(err[bad].max()), float(tol[~inf][bad].max()))


def _check(gdn, logits, scale=1.0, k=3, targets=None):
    """All outputs of finite or -inf logits with at least one finite in each row."""
    n, v = logits.shape
    if targets is None:
        targets = torch.randint(0, v, (n,), generator=_gen(n + v), device="cuda", dtype=torch.int32)
    lp, ent = (torch.full((n,), 77.0, device="cuda") for _ in range(2))
    ids = torch.full((n, k), -5, dtype=torch.int32, device="cuda")
    tl = torch.full((n, k), 77.0, device="cuda")
    gdn.gdn_token_logprobs(logits, targets, lp, ent, top_ids=ids, top_logprobs=tl, scale=scale)
    assert gdn.gdn_get_device_error() == 0
    scale = float(torch.tensor(scale, dtype=torch.float32))
    for r in range(n):                                      # (row by row: 64 bits of a whole row)
        raw = logits[r].double()
        y = (raw - raw.max()) * scale                       # x - m
        e = torch.exp(y)
        z = e.sum()
        ey = torch.where(e > 0, e * y, torch.zeros_like(e))
        spread = float(-ey.sum() / z)
        want = y - torch.log(z)
        tol = 4e-6 + 2.0 ** -22 * (spread + y.abs())
        t = int(targets[r])
        _same(lp[r:r + 1].double(), want[t:t + 1], tol[t:t + 1], ("logprob", r))
        h = torch.log(z) - ey.sum() / z
        _same(ent[r].double()[None], h[None], torch.full_like(h, 4e-6 * (2 + spread))[None],
              ("entropy", r))
        order = torch.sort(raw, descending=True, stable=True).indices[:k]
        assert torch.equal(ids[r].long(), order), r
        _same(tl[r].double(), want[order], tol[order], ("top", r))


@pytest.mark.parametrize("base", [0.0, 1e3, 1e4, 5e4, 1e6, -1e6])
def test_rising_rows_far_from_zero(gdn, base):
    """A common offset and logits that rise all along, so that a thread's largest logit changes
    time and again (each warp has about eight granules): the sums so far keep their weight."""
    n, v = 40, 248320
    x = base + torch.arange(v, device="cuda") * (0.75 / 256) - 0.75 * v / 256
    x = x + torch.randn(n, v, generator=_gen(1), device="cuda")
    _check(gdn, x)


@pytest.mark.parametrize("scale", [30.0, 1e3, 1e4])
def test_rising_rows_at_low_temperature(gdn, scale):
    n, v = 40, 248320
    x = torch.arange(v, device="cuda") * (0.75 / 256) - 0.75 * v / 256
    x = (x + torch.randn(n, v, generator=_gen(2), device="cuda")) / scale + 100.0
    _check(gdn, x, scale=scale)


MASKS = [-1e9, -1e10, -1e12, -1e20, -1e29, -3e38]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [0.5, 1.0, 1 / 0.3, 10.0, 100.0])
def test_large_finite_masks(gdn, scale, dtype):
    """Tokens masked with a large finite number, whole stretches of the vocabulary and single ones,
    -inf among them; rows that hold nothing else; rows of one or many huge logits."""
    v, g = 100003, _gen(3)
    rows = []
    for mask in MASKS:
        x = 2 * torch.randn(v, generator=g, device="cuda")
        x[1000:] = mask                                     # a stretch
        rows.append(x)
        x = torch.full((v,), mask, device="cuda")           # a few live ones
        x[[17, 50000, v - 1]] = torch.tensor([1.0, -2.0, 0.5], device="cuda")
        rows.append(x)
        x = 2 * torch.randn(v, generator=g, device="cuda")
        x[torch.rand(v, generator=g, device="cuda") < 0.5] = mask
        x[v // 2:v // 2 + 5000] = -math.inf
        rows.append(x)
        rows.append(torch.full((v,), mask, device="cuda"))  # nothing live
        x = torch.full((v,), mask, device="cuda")
        x[::3] = -math.inf
        rows.append(x)
    for top in (1e10, 1e20, 3e38):
        x = 2 * torch.randn(v, generator=g, device="cuda")
        x[40000] = top                                      # one huge logit
        rows.append(x)
        rows.append(torch.full((v,), top, device="cuda"))
    _check(gdn, torch.stack(rows).to(dtype), scale=scale)


@pytest.mark.parametrize("base", [2.9e6, 2.91e6, 1e7, 1e8])
@pytest.mark.parametrize("v", [7001, 248320])
def test_both_sides_of_the_centred_sums(gdn, base, v):
    """Logits around and past the size from which a thread centres each logit before scaling it."""
    x = base * (1 + 2e-6 * torch.rand(40, v, generator=_gen(4), device="cuda"))
    x[:, ::7] = 2.5e6
    _check(gdn, x)


@pytest.mark.parametrize("scale,size", [(1e-38, 3e38), (1e-20, 1e21), (1e20, 1e-19), (1e20, 1e15),
                                        (2e37, 1e-36), (1e-45, 1.0)])
def test_scales_of_any_size(gdn, scale, size):
    x = size * (2 * torch.rand(40, 30011, generator=_gen(5), device="cuda") - 1)
    x[:10, 100:] = torch.finfo(torch.float32).min
    x[5:15, ::5] = -math.inf
    _check(gdn, x, scale=scale)
