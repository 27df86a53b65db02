"""gdn_verify_tokens against its definition in 64 bits.

Decisions are whole numbers: equal, but where the definition's own two sides are within 2^-18 of
each other (the kernel's probabilities are ratios of sums in 32 bits: a few 2^-22), where either
is right; such cases are counted and few.  A race over max(p - q, 0) is compared by its values, each
with an error of 2^-20 (p + q): the token given has to be within that of the largest.
Log probabilities: as gdn_token_logprobs: 4e-6 + 2^-22 (|lse| + |x|), of scaled logits.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
INF = math.inf


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


def _clean(gdn):
    st = gdn.gdn_get_device_error()
    assert st == 0, gdn.gdn_status_string(st)


def _call(gdn, c, **kw):
    b, t1, _ = c["target"].shape
    out = dict(tokens=torch.full((b, t1), -9, device="cuda", dtype=torch.int32),
               accepted=torch.full((b,), -9, device="cuda", dtype=torch.int32),
               logprobs=torch.full((b, t1), 9.0, device="cuda"))
    gdn.gdn_verify_tokens(c["target"], out["tokens"], out["accepted"], clocks=c["clocks"],
                          draft_ids=c.get("ids"), draft_logits=c.get("draft"),
                          accept_u=c.get("u"), scale=c.get("scale"), logprobs=out["logprobs"], **kw)
    return out


def _no_distribution(x):
    return bool(torch.isnan(x).any()) or float(x.max()) == INF or float(x.max()) == -INF


def _check(c, out, close=0):
    """Every sequence against the definition; returns how many decisions were too close to tell."""
    target, draft, ids = c["target"], c.get("draft"), c.get("ids")
    b, t1, v = target.shape
    t = t1 - 1
    told = 0
    for i in range(b):
        scale = 1.0 if c.get("scale") is None else float(c["scale"][i])
        tokens, accepted = out["tokens"][i].tolist(), int(out["accepted"][i])
        logprobs = out["logprobs"][i].tolist()
        if not (scale == INF or 2.0 ** -64 <= scale <= 2.0 ** 64):
            assert tokens == [-9] * t1 and accepted == -9 and logprobs == [9.0] * t1
            continue
        greedy, s = scale == INF, (1.0 if scale == INF else scale)
        n = 0
        while n < t and 0 <= int(ids[i, n]) < v:
            n += 1
        assert 0 <= accepted <= n

        def logp(x):
            x = x.double()
            x = (x - x.max()) * s
            return x - torch.logsumexp(x, 0)

        def first_of(x):                       # the lowest index of the largest
            return int((x == x.max()).nonzero()[0, 0])

        for j in range(accepted + 1):
            x = target[i, j]
            drafted = int(ids[i, j]) if j < n else -1
            taken = j < accepted
            if _no_distribution(x):
                assert not taken and tokens[j] == -1 and logprobs[j] == 0.0
                continue
            lp = logp(x)
            lq = None
            if drafted >= 0 and draft is not None and not greedy:
                lq = "none" if _no_distribution(draft[i, j]) else logp(draft[i, j])
            if drafted >= 0:
                if greedy:
                    assert taken == (drafted == first_of(x)), (i, j)
                elif isinstance(lq, str):
                    assert not taken
                elif float(lp[drafted]) == -INF:
                    assert not taken
                else:
                    u = float(c["u"][i, j])
                    ratio = math.exp(min(700.0, float(lp[drafted]) - (0.0 if lq is None else
                                                                     float(lq[drafted]))))
                    if abs(u - ratio) <= 2.0 ** -18 * ratio:
                        told += 1
                    else:
                        assert taken == (u < ratio), (i, j, u, ratio)
            if taken:
                assert tokens[j] == drafted
            elif greedy:
                assert tokens[j] == first_of(x)
            elif isinstance(lq, str):
                assert tokens[j] == -1 and logprobs[j] == 0.0
                continue
            else:
                p = lp.exp()
                q = torch.zeros_like(p) if lq is None else lq.exp()
                if drafted >= 0 and lq is None:
                    p = p.clone()
                    p[drafted] = 0.0
                clocks = c["clocks"][i].double()
                rings = clocks > 0
                e = torch.where(rings, clocks, torch.ones_like(clocks))
                slack = torch.where(rings, 2.0 ** -20 * (p + q) / e, torch.zeros_like(p))
                race = torch.where(rings, (p - q).clamp(min=0) / e, torch.zeros_like(p))
                most = float((race - slack).max())
                token = tokens[j]
                if token == drafted and drafted >= 0 or token == -1:
                    # (no token with any weight left)
                    assert most <= 0.0 and token == drafted
                else:
                    if most <= 0.0:
                        told += 1
                    assert float(race[token] + slack[token]) >= most, (i, j, token)
                    if int(((race + slack) >= most).sum()) > 1:
                        told += 1
                    elif float(race.max()) > 0:
                        assert token == int(race.argmax())
            token = tokens[j]
            if token >= 0:
                x64 = x.double() * s
                lse = torch.logsumexp(x64, 0)
                tol = 4e-6 + 2.0 ** -22 * (abs(float(lse)) + abs(float(x64[token])))
                if math.isfinite(tol):
                    want = float((x.double()[token] - x.double().max()) * s
                                 - torch.logsumexp((x.double() - x.double().max()) * s, 0))
                    assert abs(logprobs[j] - want) <= tol, (i, j, logprobs[j], want)
        assert tokens[accepted + 1:] == [-1] * (t - accepted)
        assert logprobs[accepted + 1:] == [0.0] * (t - accepted)
    assert told <= close, told


def _case(b, t, v, dtype, drafts, seed, spread=3.0, off=0.7):
    g = _gen(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = spread * randn(b, t + 1, v)
    c = dict(target=x.to(dtype), clocks=torch.empty(b, v, device="cuda").exponential_(generator=g))
    scales = torch.tensor([1.0, 0.7, INF, 1.6, -1.0, 1.0, math.nan, 0.0], device="cuda")
    c["scale"] = scales[torch.arange(b, device="cuda") % 8].contiguous() if b > 1 else None
    if t:
        y = (x[:, :t] + off * randn(b, t, v)).to(dtype)
        clock = torch.empty(b, t, v, device="cuda").exponential_(generator=g)
        c["ids"] = (y.float() - clock.log()).argmax(-1).to(torch.int32)
        if b > 2:
            c["ids"][2] = c["target"][2, :t].float().argmax(-1)     # greedy, all good
            c["ids"][1, t // 2:] = -1
            c["ids"][min(5, b - 1), 0] = -2 ** 31
        c["u"] = torch.rand(b, t, generator=g, device="cuda")
        c["draft"] = y if drafts == "logits" else None
    return c


CASES = [(1, 0, 1), (1, 1, 1), (2, 1, 2), (1, 3, 17), (3, 2, 511), (8, 4, 512), (9, 5, 1000),
         (17, 7, 4097), (5, 3, 30011), (1, 4, 248320), (4, 2, 151936), (33, 1, 2053),
         (200, 0, 3001), (2, 64, 1001), (3, 33, 64), (700, 3, 129)]


@pytest.mark.parametrize("drafts", ["logits", "ids"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,t,v", CASES)
def test_definition(gdn, b, t, v, dtype, drafts):
    c = _case(b, t, v, dtype, drafts, seed=b * 1000 + t * 10 + v)
    out = _call(gdn, c)
    _clean(gdn)
    _check(c, out, close=2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(gdn, dtype):
    """Rows that are slices of wider ones, starting at any element."""
    for v, pad, first in ((1000, 24, 8), (1000, 7, 3), (4099, 1, 1), (2048, 16, 5)):
        c = _case(6, 3, v, dtype, "logits", seed=v + first)
        for name in ("target", "draft"):
            x = c[name]
            wide = torch.full((x.shape[0], x.shape[1], v + pad), 1e4, device="cuda", dtype=dtype)
            wide[..., first:first + v] = x if first + v <= v + pad else 0
            if first + v <= v + pad:
                c[name] = wide[..., first:first + v]
        out = _call(gdn, c)
        _clean(gdn)
        _check(c, out, close=1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [range(1, 42), (4089, 4096, 4097, 4103, 6145, 8200)])
def test_every_alignment(gdn, sizes, dtype):
    """Rows of the target and of the draft that begin at any element, each at its own, around the
    sizes of a vector and of a slice; most drafts are refused, so that the race runs."""
    for v in sizes:
        for off, more in ((0, 0), (1, 0), (0, 1), (3, 6), (5, 2), (7, 7)):
            c = _case(3, 2, v, dtype, "logits", seed=v)
            c["scale"], c["u"] = None, 0.5 + c["u"] / 2
            c["ids"] = c["ids"].clamp(min=0)
            c["ids"][1] = c["draft"][1].float().argmax(-1)
            for name, first in (("target", off), ("draft", more)):
                x = c[name]
                wide = torch.full((*x.shape[:2], v + 9), math.nan, dtype=dtype, device="cuda")
                wide[..., first:first + v] = x
                c[name] = wide[..., first:first + v]
            out = _call(gdn, c)
            _check(c, out, close=3)
    _clean(gdn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [40, 5000, 100003])
def test_masks(gdn, v, dtype):
    """Masks of -inf and of the type's lowest value, rows with one logit left or none, NaN and
    infinities, in the target's rows and in the draft's."""
    low = torch.finfo(dtype).min
    b, t = 14, 2
    c = _case(b, t, v, dtype, "logits", seed=v)
    c["scale"] = torch.tensor([1.0, 0.5] * 7, device="cuda")
    c["ids"] = c["ids"].clamp(0, v // 2 - 1)
    x, y = c["target"], c["draft"]
    x[0, :, v // 2:] = -INF
    x[1, :, v // 2:] = low
    y[2, :, v // 2:] = -INF
    y[3, :, v // 2:] = low
    x[4], x[4, :, 7] = -INF, 3.0                           # one logit left
    x[5, 0] = -INF                                         # none
    x[6, 1, 3] = math.nan
    x[7, 0, 5] = INF
    y[8, 0] = -INF
    y[9, 0, v - 1] = math.nan
    y[10, 0, 0] = INF
    x[11, 2] = math.nan                                    # the row behind the drafts
    c["u"][11] = 0.0
    y[12, 0, int(c["ids"][12, 0])] = -INF                  # a draft that q gives nothing
    x[13, 0, int(c["ids"][13, 0])] = -INF                  # one that p gives nothing
    c["u"][13] = 0.0
    out = _call(gdn, c)
    _clean(gdn)
    _check(c, out, close=2)
    assert int(out["tokens"][5, 0]) == -1 and int(out["accepted"][5]) == 0
    assert int(out["accepted"][13]) == 0
    # behind the last draft nothing is read
    c["ids"][:, 1] = -1
    x[:, 2], y[:, 1] = math.nan, math.nan
    out = _call(gdn, c)
    _clean(gdn)
    _check(c, out, close=2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scales_and_sizes(gdn, dtype):
    """Inverse temperatures over their whole range with logits of any size."""
    for size, scale in ((3e38, 2.0 ** -64), (3e38, 1.0), (1e-30, 2.0 ** 64), (3e4, 1e-4),
                        (1e6, 1.0), (1e12, 1e-12), (100.0, 30.0), (1e-6, 1.0)):
        for drafts in ("logits", "ids"):
            c = _case(6, 2, 3001, dtype, drafts, seed=11)
            for name in ("target", "draft"):
                if c.get(name) is not None:
                    c[name] = (c[name].double() / 20 * size).clamp(-3.3e38, 3.3e38).to(dtype)
            c["scale"] = torch.full((6,), scale, device="cuda")
            c["ids"] = (c["target"][:, :2].float().argmax(-1) if size * scale > 50
                        else c["ids"].clamp(min=0)).to(torch.int32)
            out = _call(gdn, c)
            _clean(gdn)
            _check(c, out, close=2)


def test_greedy(gdn):
    """Equal largest logits go to the lowest id, as drafts and as the token behind them."""
    for dtype in (torch.bfloat16, torch.float32):
        for v in (9, 1030, 20011):
            b, t = 6, 3
            x = torch.randn(b, t + 1, v, generator=_gen(v), device="cuda").to(dtype)
            top = float(x.float().max()) + 1
            for i in range(b):
                for j in range(t + 1):
                    for k in ((i * 131 + j * 17) % v, (i * 7 + j * 1009) % v, v - 1):
                        x[i, j, k] = top
            x[5] = 0.0
            x[5, :, ::2] = -0.0
            c = dict(target=x, clocks=torch.zeros(b, v, device="cuda"),
                     scale=torch.full((b,), INF, device="cuda"), u=torch.ones(b, t, device="cuda"))
            first = (x.float() == x.float().amax(-1, keepdim=True)).int().argmax(-1)
            c["ids"] = first[:, :t].to(torch.int32).contiguous()
            c["ids"][1, 1] = v - 1                          # equal, not the first
            c["ids"][2, 0] = (int(first[2, 0]) + 1) % v
            out = _call(gdn, c)
            _clean(gdn)
            _check(c, out)
            assert out["accepted"].tolist()[0] == 3 and out["accepted"].tolist()[1] == 1
            assert out["tokens"][0].tolist() == first[0].tolist()


def test_random_numbers_at_their_ends(gdn):
    """Clocks that never ring (0, negative, NaN, inf), uniform numbers of 0 and 1, p = q."""
    c = _case(8, 2, 600, torch.float32, "logits", seed=2)
    c["scale"] = None
    c["ids"] = c["ids"].clamp(min=0)
    k = c["clocks"]
    k[0, ::2], k[1, 1::2], k[2, :300], k[3] = 0.0, -1.0, math.nan, INF
    k[4] = 0.0
    c["u"][0], c["u"][1] = 0.0, 1.0
    c["u"][4], c["u"][5] = 1.0, math.nan
    c["draft"][6] = c["target"][6, :2]                      # p = q: every u below 1 accepts
    c["draft"][7], c["u"][7] = c["target"][7, :2], 1.0      # refused without a residual
    out = _call(gdn, c)
    _clean(gdn)
    assert int(out["accepted"][6]) == 2
    assert int(out["accepted"][7]) == 0 and int(out["tokens"][7, 0]) == int(c["ids"][7, 0])
    assert int(out["accepted"][5]) == 0
    keep = [0, 1, 2, 6]
    part = {n: (x if x is None else x[keep]) for n, x in c.items()}
    _check(part, {n: x[keep] for n, x in out.items()}, close=2)


def test_ids_out_of_range(gdn):
    c = _case(4, 3, 100, torch.bfloat16, "logits", seed=5)
    c["scale"] = None
    c["u"].zero_()
    c["ids"] = torch.tensor([[1, 100, 2], [3, 4, 5], [2 ** 31 - 1, 1, 1], [1, -1, 200]],
                            device="cuda", dtype=torch.int32)
    out = _call(gdn, c)
    assert gdn.gdn_get_device_error() == 6
    _check(c, out, close=1)
    assert out["accepted"].tolist()[0] <= 1 and int(out["accepted"][2]) == 0
    c["ids"][0, 1], c["ids"][2, 0] = -1, -1
    _call(gdn, c)
    _clean(gdn)                                             # ids behind a negative one: ignored


@pytest.mark.parametrize("drafts", ["logits", "ids"])
def test_tokens_are_the_targets(gdn, drafts):
    """The first token of 60000 verifications of a draft from q (or of a fixed draft) is
    distributed as p: chi squared over nine tokens (8 degrees of freedom), its 1 - 1e-6 quantile
    42.7; the second token, where there is one, likewise."""
    n, v = 60000, 9
    g = _gen(77)
    p = torch.randn(2, v, generator=g, device="cuda")
    q = torch.randn(1, v, generator=g, device="cuda")
    c = dict(target=p.expand(n, 2, v).contiguous(),
             clocks=torch.empty(n, v, device="cuda").exponential_(generator=g),
             u=torch.rand(n, 1, generator=g, device="cuda"))
    if drafts == "logits":
        c["draft"] = q.expand(n, 1, v).contiguous()
        clock = torch.empty(n, v, device="cuda").exponential_(generator=g)
        c["ids"] = (q - clock.log()).argmax(-1, keepdim=True).to(torch.int32)
    else:
        c["ids"] = torch.full((n, 1), 4, device="cuda", dtype=torch.int32)
    out = _call(gdn, c)
    _clean(gdn)
    for j, rows in ((0, slice(None)), (1, out["accepted"] == 1)):
        got = torch.bincount(out["tokens"][rows, j].long(), minlength=v).double()
        want = torch.softmax(p[j].double(), 0) * got.sum()
        assert float(((got - want) ** 2 / want).sum()) <= 42.7


def test_repeats_graphs_and_streams(gdn):
    """The same call gives the same bits; two captured calls with a workspace each replay on two
    streams at once, with new numbers."""
    cases = [_case(12, 3, 5003, torch.bfloat16, "logits", seed=s) for s in (1, 2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for c, side in zip(cases, streams):
        ws = torch.full((gdn.gdn_verify_tokens_workspace_size(12, 3, 5003),), 255,
                        dtype=torch.uint8, device="cuda")
        out = dict(tokens=torch.zeros(12, 4, device="cuda", dtype=torch.int32),
                   accepted=torch.zeros(12, device="cuda", dtype=torch.int32),
                   logprobs=torch.zeros(12, 4, device="cuda"))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            gdn.gdn_verify_tokens(c["target"], out["tokens"], out["accepted"], clocks=c["clocks"],
                                  draft_ids=c["ids"], draft_logits=c["draft"], accept_u=c["u"],
                                  scale=c["scale"], logprobs=out["logprobs"], workspace=ws)
        graphs.append(graph)
        outs.append(out)
    for turn in range(4):
        for c in cases:
            c["u"].uniform_(generator=_gen(turn))
            c["clocks"].exponential_(generator=_gen(turn + 9))
        torch.cuda.synchronize()
        for graph, side in zip(graphs, streams):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            active = torch.isinf(c["scale"]) | (c["scale"] > 0)
            for again in (_call(gdn, c), _call(gdn, c, stream=streams[0])):
                torch.cuda.synchronize()
                for name in out:
                    assert torch.equal(out[name][active], again[name][active])
    _clean(gdn)


def test_refusals(gdn):
    c = _case(3, 2, 50, torch.float32, "logits", seed=1)
    b = torch.zeros(3, device="cuda", dtype=torch.int32)
    base = dict(target_logits=c["target"], tokens=torch.zeros(3, 3, device="cuda", dtype=torch.int32),
                accepted=b, clocks=c["clocks"], draft_ids=c["ids"], draft_logits=c["draft"],
                accept_u=c["u"], scale=c["scale"])
    for bad in (dict(target_logits=c["target"][0]), dict(target_logits=c["target"].half()),
                dict(target_logits=c["target"].transpose(0, 1)), dict(tokens=b),
                dict(accepted=b[:2]), dict(clocks=c["clocks"].double()), dict(clocks=c["clocks"][:2]),
                dict(draft_ids=None), dict(draft_ids=c["ids"].long()), dict(accept_u=None),
                dict(draft_logits=c["draft"].bfloat16()), dict(draft_logits=c["target"]),
                dict(scale=c["scale"].double()), dict(scale=c["scale"].cpu()),
                dict(logprobs=c["u"]), dict(workspace=torch.zeros(8, device="cuda")),
                dict(target_logits=c["target"].expand(3, 3, 50)[..., ::2]),
                dict(target_logits=c["target"][:, :1], tokens=b[:, None])):
        with pytest.raises((ValueError, TypeError, gdn.GDNError)):
            gdn.gdn_verify_tokens(**{**base, **bad})
    gdn.gdn_verify_tokens(**base)
    _clean(gdn)
