"""gdn_verify_tokens where its numbers are far apart or very close: log probabilities of accepted
drafts whose logits lie further below the row's largest than fp32 reaches, and the token behind a
refusal where the draft's probabilities are nearly the target's."""
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


def _run(gdn, target, **kw):
    b, t1, _ = target.shape
    tokens = torch.full((b, t1), -9, device="cuda", dtype=torch.int32)
    accepted = torch.full((b,), -9, device="cuda", dtype=torch.int32)
    logprobs = torch.full((b, t1), 9.0, device="cuda")
    gdn.gdn_verify_tokens(target, tokens, accepted, logprobs=logprobs, **kw)
    assert gdn.gdn_get_device_error() == 0
    return tokens, accepted, logprobs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -40, 2.0 ** -2])
def test_log_probabilities_of_far_drafts(gdn, scale, dtype):
    """p / q = 1 for a draft 6e38 below its row's largest logit: accepted, with its log probability."""
    v = 50
    x = torch.zeros(1, 2, v, device="cuda", dtype=dtype)
    x[..., 0], x[..., 1] = 3e38, -3e38
    tokens, accepted, logprobs = _run(
        gdn, x, clocks=torch.ones(1, v, device="cuda"), draft_logits=x[:, :1].contiguous(),
        draft_ids=torch.ones(1, 1, device="cuda", dtype=torch.int32),
        accept_u=torch.full((1, 1), 0.25, device="cuda"), scale=torch.full((1,), scale, device="cuda"))
    assert int(accepted) == 1 and tokens.tolist() == [[1, 0]]
    want = (float(x[0, 0, 1]) - float(x[0, 0, 0])) * scale   # (z is 1)
    assert abs(float(logprobs[0, 0]) - want) <= 2.0 ** -22 * abs(want)
    assert abs(float(logprobs[0, 1])) <= 4e-6


@pytest.mark.parametrize("dtype,close", [(torch.float32, 1e-2), (torch.float32, 1e-4),
                                         (torch.bfloat16, 1e-2), (torch.bfloat16, 1e-4)])
@pytest.mark.parametrize("v", [3000, 50021])
def test_draft_probabilities_close_to_the_targets(gdn, v, dtype, close):
    """A probability is off by 2^-20 of itself (its row's sum, the exponential) and 2^-22 more for every
    binary order below its row's largest (the exponent's rounding: 2^-24 each of the difference, the
    scale and their product, times ln 2), whatever p - q leaves of it: the token given is within that
    of the first."""
    b = 48
    g = torch.Generator(device="cuda").manual_seed(v)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = (3 * randn(b, 2, v)).to(dtype)
    y = (x[:, :1].float() + close * randn(b, 1, v)).to(dtype)
    scale = torch.tensor([1.0, 1.25, 0.7], device="cuda").repeat(b // 3)
    clocks = torch.empty(b, v, device="cuda").exponential_(generator=g)
    logs = [torch.log_softmax(z[:, 0].double() * scale.double()[:, None], 1) for z in (x, y)]
    (p, q), below = [z.exp() for z in logs], [(z.amax(1, keepdim=True) - z) / 0.6931471805599453 for z in logs]
    ids = (q - p).argmax(1, keepdim=True).to(torch.int32)
    if not bool((p != q).any(1).all()):
        pytest.skip("rounded to the same rows")
    ratio = (p / q).gather(1, ids.long())[:, 0]
    tokens, accepted, _ = _run(gdn, x, clocks=clocks, draft_logits=y, draft_ids=ids, scale=scale,
                               accept_u=torch.full((b, 1), 1 - 2.0 ** -24, device="cuda"))
    refused = ratio < 1 - 2.0 ** -17
    assert int(refused.sum()) >= b // 2 and not bool(accepted[refused].any())
    race = (p - q) / clocks.double()
    slack = (2.0 ** -20 + 2.0 ** -22 * torch.maximum(*below)) * (p + q) / clocks.double()
    got = tokens[:, :1].long()
    assert bool((got[refused] >= 0).all())
    good = (race + slack).gather(1, got.clamp(min=0))[:, 0] >= (race - slack).amax(1)
    assert bool(good[refused].all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [70, 9001])
def test_rows_that_do_not_count(gdn, v, dtype):
    """NaN in the draft's rows of greedy sequences, behind the last draft and in rows of sequences
    that are left out change nothing."""
    b, t = 9, 3
    g = torch.Generator(device="cuda").manual_seed(v)
    x = (3 * torch.randn(b, t + 1, v, generator=g, device="cuda")).to(dtype)
    y = (x[:, :t].float() + 0.5 * torch.randn(b, t, v, generator=g, device="cuda")).to(dtype)
    ids = x[:, :t].float().argmax(-1).to(torch.int32)
    ids[3:6, 1] = -1                                     # one draft each
    kw = dict(clocks=torch.empty(b, v, device="cuda").exponential_(generator=g), draft_ids=ids,
              accept_u=torch.rand(b, t, generator=g, device="cuda"),
              scale=torch.tensor([float("inf"), 1.0, -1.0] * 3, device="cuda"))
    want = _run(gdn, x, draft_logits=y, **kw)
    spoilt_x, spoilt_y = x.clone(), y.clone()
    spoilt_y[0::3] = float("nan")
    spoilt_x[2::3], spoilt_y[2::3] = float("nan"), float("nan")
    spoilt_x[3:6, 2:], spoilt_y[3:6, 1:] = float("nan"), float("nan")
    for a, z in zip(want, _run(gdn, spoilt_x, draft_logits=spoilt_y, **kw)):
        assert torch.equal(a, z)
    assert bool((want[1][0::3] == torch.tensor([3, 1, 3], device="cuda")).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", ["lowest", -1e30, -3e4])
def test_drafts_far_below_in_both_rows(gdn, low, dtype):
    """A draft at the same far logit in the target's row and the draft's: p / q is what the rows'
    largest logits (4 above 1, or 1 above 4, beside zeros) and sums leave."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    v, us = 300, [0.0, 0.01, 0.04, 0.06, 0.9, 0.999]
    x = torch.zeros(2 * len(us), 2, v, device="cuda", dtype=dtype)
    y = torch.zeros(2 * len(us), 1, v, device="cuda", dtype=dtype)
    x[:len(us), :, 7], y[:len(us), :, 7] = 4.0, 1.0
    x[len(us):, :, 7], y[len(us):, :, 7] = 1.0, 4.0
    x[..., 3], y[..., 3] = low, low
    u = torch.tensor(us + us, device="cuda")[:, None]
    tokens, accepted, _ = _run(
        gdn, x, clocks=torch.ones(len(u), v, device="cuda"), draft_logits=y, accept_u=u,
        draft_ids=torch.full((len(u), 1), 3, device="cuda", dtype=torch.int32))
    # the same logit in both: p / q = sum e^y / sum e^x, 298 zeros in each
    one, four = 298 + 2.718281828459045, 298 + 54.598150033144236
    ratio = torch.tensor([one / four] * len(us) + [four / one] * len(us), dtype=torch.float64)
    assert accepted.tolist() == (u[:, 0].cpu().double() < ratio).int().tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 3.0, 2.0 ** -3])
def test_lowest_values_with_far_maxima(gdn, scale, dtype):
    """The same where the largest logits alone decide: one logit of hundreds, the rest masked."""
    low, v = torch.finfo(dtype).min, 40
    cases = [(300.0, 299.0), (299.0, 300.0), (0.0, 2.0), (2.0, 0.0), (-5.0, 5.0), (640.0, 0.0)]
    x = torch.full((len(cases), 2, v), low, device="cuda", dtype=dtype)
    y = torch.full((len(cases), 1, v), low, device="cuda", dtype=dtype)
    for i, (a, b) in enumerate(cases):
        x[i, :, 5], y[i, :, 5] = a, b
    u = torch.full((len(cases), 1), 0.5, device="cuda")
    _, accepted, _ = _run(
        gdn, x, clocks=torch.ones(len(cases), v, device="cuda"), draft_logits=y, accept_u=u,
        draft_ids=torch.full((len(cases), 1), 3, device="cuda", dtype=torch.int32),
        scale=torch.full((len(cases),), scale, device="cuda"))
    # p / q = e^(scale (b - a)), a and b as the type holds them (299 is 300 in bf16)
    held = zip(x[:, 0, 5].tolist(), y[:, 0, 5].tolist())
    want = [int(0.5 < 2.718281828459045 ** (scale * (b - a))) for a, b in held]
    assert accepted.tolist() == want
