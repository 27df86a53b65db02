"""gdn_verify_tokens with clocks at the ends of their range, against the definition in 64 bits: a
clock between 0 and 2^-126 rings as one of 2^-126; zero, negative, NaN and infinite ones never.
The weights are chosen so that the first clock is ahead of every other by a tenth or more (the
kernel's weights are right to 2^-16 and better), so tokens are equal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
INF, LEAST = math.inf, 2.0 ** -126


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def _first(w, clocks):
    """The index whose clock rings first (-1: none does): weights below 2^-126 of one count as 0."""
    w, e = w.double(), clocks.double()
    rings = (e > 0) & (e < INF) & (w > 0)
    race = torch.where(rings, w / e.clamp(min=LEAST), torch.zeros_like(w))
    if float(race.max()) == 0.0:
        return -1
    two = race.topk(min(2, race.numel())).values
    assert race.numel() == 1 or float(two[1]) <= 0.9 * float(two[0])      # (the test's own cases)
    return int(race.argmax())


def _weights(x):
    """p over its largest, and what counts as 0."""
    w = torch.exp(x.double() - x.double().max())
    return torch.where(w < LEAST, torch.zeros_like(w), w)


def _run(gdn, target, clocks, **kw):
    b, t1, _ = target.shape
    tokens = torch.full((b, t1), -9, device="cuda", dtype=torch.int32)
    accepted = torch.full((b,), -9, device="cuda", dtype=torch.int32)
    logprobs = torch.full((b, t1), 9.0, device="cuda")
    gdn.gdn_verify_tokens(target, tokens, accepted, clocks=clocks, logprobs=logprobs, **kw)
    assert gdn.gdn_get_device_error() == 0
    return tokens, accepted, logprobs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [700, 2048, 60001])
def test_tiny_clocks_without_drafts(gdn, v, dtype):
    """Rows of -rise with a 0 behind the tiny clock, in the same granule and in later ones."""
    rows, clocks = [], []
    for rise in (0.0, 3.0, 50.0, 86.0, 100.0, 5000.0):
        for tiny in (1e-40, 2.0 ** -149, 1.1e-38, 2.0 ** -126, 3e-38):
            for at, peak in ((0, 600), (0, 1), (699, 3), (5, v - 1), (v - 1, 0)):
                x, e = torch.full((v,), -rise), torch.ones(v)
                x[peak], e[at] = 0.0, tiny
                # at a rise of 86 or so the tiny clock and the peak are close: kept apart
                e[peak] = 0.5 if at != peak else tiny
                rows.append(x)
                clocks.append(e)
    x, e = torch.stack(rows).to(dtype).cuda(), torch.stack(clocks).cuda()
    tokens, accepted, logprobs = _run(gdn, x[:, None], e)
    assert tokens[:, 0].tolist() == [_first(_weights(a), k) for a, k in zip(x, e)]
    assert accepted.tolist() == [0] * len(rows) and bool(logprobs.isfinite().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_tiny_clocks(gdn, dtype):
    """Both ring as one of 2^-126, so the larger weight is first, wherever they lie."""
    v, rows, clocks = 9000, [], []
    for first, second in ((1e-45, 1e-40), (1e-40, 1e-45), (1e-38, 1e-45)):
        for i, j in ((0, 1), (3, 300), (10, 8990), (8000, 40)):
            for high, low in ((i, j), (j, i)):
                x, e = torch.full((v,), -4.0), torch.ones(v)
                x[high], x[low], e[i], e[j] = 1.0, -1.0, first, second
                rows.append(x)
                clocks.append(e)
    x, e = torch.stack(rows).to(dtype).cuda(), torch.stack(clocks).cuda()
    tokens, _, _ = _run(gdn, x[:, None], e)
    assert tokens[:, 0].tolist() == [_first(_weights(a), k) for a, k in zip(x, e)]


@pytest.mark.parametrize("drafts", ["logits", "ids"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [40, 5000, 30001])
def test_tiny_clocks_behind_drafts(gdn, v, dtype, drafts):
    """Draft 0 is 3, refused (u = 2) or accepted (u = 0)."""
    rows, clocks, us = [], [], []
    for u in (0.0, 2.0):
        for tiny in (1e-40, 2.0 ** -149, 1.1e-38):
            for at, peak in ((0, v - 2), (v - 1, 1), (7, 6)):
                for rise in (2.0, 100.0):
                    x, e = torch.full((2, v), -rise), torch.ones(v)
                    x[:, peak], x[:, 3], e[at], e[peak] = 1.0, 0.5, tiny, 0.5
                    rows.append(x)
                    clocks.append(e)
                    us.append([u])
    x, e = torch.stack(rows).to(dtype).cuda(), torch.stack(clocks).cuda()
    b = x.shape[0]
    y = torch.zeros(b, 1, v, device="cuda", dtype=dtype)
    y[:, :, 3] = 40.0                                     # q is all on the draft, but for e^-40
    ids = torch.full((b, 1), 3, device="cuda", dtype=torch.int32)
    tokens, accepted, _ = _run(gdn, x, e, draft_ids=ids, accept_u=torch.tensor(us, device="cuda"),
                               draft_logits=y if drafts == "logits" else None)
    for i in range(b):
        refused = us[i][0] > 0
        assert int(accepted[i]) == (0 if refused else 1)
        w = _weights(x[i, 0 if refused else 1])
        if refused:
            q = torch.zeros_like(w)
            q[3] = 1.0
            if drafts == "logits":
                q = torch.softmax(y[i, 0].double(), 0)
            w = (w - q * float(w.sum())).clamp(min=0)
        want = _first(w, e[i])
        assert tokens[i].tolist() == ([want, -1] if refused else [3, want]), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [600, 20001])
@pytest.mark.parametrize("clock", [0.0, -1.0, math.nan, INF])
def test_clocks_that_never_ring(gdn, clock, v, dtype):
    """Rows in which nothing rings: without drafts and behind accepted ones no token (and a log
    probability of 0); a refused draft is the token itself.  One clock among them decides."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn(4, 2, v, generator=g, device="cuda").to(dtype)
    e = torch.full((4, v), clock, device="cuda")
    e[2:, v // 3] = 3.0
    tokens, _, logprobs = _run(gdn, x[:, :1].contiguous(), e)
    assert tokens[:, 0].tolist() == [-1, -1, v // 3, v // 3]
    assert logprobs[:2, 0].tolist() == [0.0, 0.0] and bool((logprobs[2:] < 0).all())
    ids = torch.full((4, 1), 5, device="cuda", dtype=torch.int32)
    u = torch.tensor([[0.0], [1.0], [0.0], [1.0]], device="cuda")
    y = torch.full((4, 1, v), -20.0, device="cuda", dtype=dtype)
    y[:, :, 5] = 20.0                                     # p / q is below 1
    for draft in (None, y):
        tokens, accepted, logprobs = _run(gdn, x, e, draft_ids=ids, draft_logits=draft, accept_u=u)
        assert accepted.tolist() == [1, 0, 1, 0]
        assert tokens.tolist() == [[5, -1], [5, -1], [5, v // 3], [v // 3, -1]]
        assert float(logprobs[0, 1]) == 0.0 and bool((logprobs[:, 0] < 0).all())
        want = torch.log_softmax(x[1, 0].double(), 0)[5]
        # 4e-6 + 2^-22 (|lse| + |x|), lse at most 10.5 and |x| below 6
        assert abs(float(logprobs[1, 0]) - float(want)) <= 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [1, 9, 513, 4097, 30001])
@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
def test_ties_go_to_the_lower_id(gdn, order, v, dtype):
    """Whole logits and clocks that are powers of two: w / E of two tokens is the same number or
    apart by 7% and more (e^2 and 8 are the closest of e^k and a power of two, k = 1 .. 5)."""
    b, t = 12, 1
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randint(-3, 3, (b, t + 1, v), generator=g, device="cuda").to(dtype)
    if order != "mixed":
        x = x.sort(-1, descending=order == "falling").values
    e = 2.0 ** torch.randint(-2, 3, (b, v), generator=g, device="cuda").float()
    ids = torch.randint(0, v, (b, 1), generator=g, device="cuda", dtype=torch.int32)
    u = torch.tensor([0.0, 2.0] * (b // 2), device="cuda")[:, None]

    def first(row, i, never=-1):
        w = torch.exp(x[i, row].double() - x[i, row].double().max())
        if never >= 0:
            w[never] = 0.0
        race = w / e[i].double()
        return int((race == race.max()).nonzero()[0, 0]) if float(race.max()) > 0 else never

    tokens, _, _ = _run(gdn, x[:, :1].contiguous(), e)
    assert tokens[:, 0].tolist() == [first(0, i) for i in range(b)]
    tokens, accepted, _ = _run(gdn, x, e, draft_ids=ids, accept_u=u)
    assert accepted.tolist() == [1, 0] * (b // 2)
    for i in range(b):
        drafted = int(ids[i, 0])
        want = [drafted, first(1, i)] if i % 2 == 0 else [first(0, i, drafted), -1]
        assert tokens[i].tolist() == want, i
