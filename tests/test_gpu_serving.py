"""The full-attention layers' operators on the GPU against their definitions in 64 bits: the
paged key/value cache, shared-prefix attention, token log probabilities.

Tolerances.
  * Cache: the codes and exponents are whole numbers that the definition fixes: equal.  A value
    read back is the stored one: equal.
  * Attention, per element, with A = sum_j p_j |v_j| of its row: the probabilities are rounded to
    nine significant bits at least (relative 2^-9 each, so 2^-9 A in all), the scores are fp32
    sums whose relative effect on the p_j is below 2^-10 (another 2^-10 A allowed), the output
    rounds once more (2^-9 |out| for bf16).  Probabilities below 2^-27 of the row's largest may
    be rounded absolutely: 1e-6 max|v|.
    lse: fp32 sums of scores and of exponentials: 2e-5 (1 + |lse|).
  * Log probabilities: z = sum e^(x-m) in fp32 over at most 2^18 terms, pairwise across threads:
    4e-6 relative; log z, m + log z and x - lse round at 2^-23 of their size.
    |logprob error| <= 4e-6 + 2^-22 (|lse| + |x|); the entropy log z - w / z likewise:
    4e-6 (2 + |w / z|).
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


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _clean(gdn):
    st = gdn.gdn_get_device_error()
    assert st == 0, gdn.gdn_status_string(st)


# ------------------------------------------------------------------------------- the cache

def _pow2(e):
    """2^e in float64, exactly, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _codes(x):
    """The definition: exponent by exponent search, codes by the nearest of the table."""
    x = x.double()
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    top = fin.amax(-1)
    e = torch.full(top.shape, -60, dtype=torch.int64, device=x.device)
    for cand in range(60, -60, -1):       # the least e that fits: go down while it does
        e = torch.where(top * 2.0 ** -(cand - 1) > 448, torch.maximum(
            e, torch.full_like(e, cand)), e)
    y = x * _pow2(-e)[..., None]
    # four significant bits, down to 2^-9
    binade = torch.frexp(torch.nan_to_num(y, nan=1.0, posinf=1.0, neginf=1.0))[1] - 1
    unit = _pow2(binade.clamp(min=-6) - 3)
    y = torch.round(y / unit) * unit
    y = torch.where(torch.isnan(x), x, y.clamp(-448, 448))
    y = torch.where(torch.isinf(x), torch.sign(x) * 448, y)
    return y, (e + 127).to(torch.uint8)


def _empty_cache(pages, h, p, d, fmt, fill=0x7f):
    dt = torch.float8_e4m3fn if fmt == "f8" else torch.bfloat16
    c = {}
    for n in ("k", "v"):
        c[n] = torch.full((pages, h, p, d * (1 if fmt == "f8" else 2)), fill, dtype=torch.uint8,
                          device="cuda").view(dt)
        c[n + "_exp"] = (torch.full((pages, h, p), 255, dtype=torch.uint8, device="cuda")
                         if fmt == "f8" else None)
    return c


@pytest.mark.parametrize("fmt", ["f8", "bf16"])
@pytest.mark.parametrize("n,h,d,p,dtype", [
    (1, 1, 128, 16, torch.bfloat16), (3, 1, 128, 16, torch.float32), (33, 3, 128, 32, torch.bfloat16),
    (77, 4, 256, 64, torch.bfloat16), (500, 2, 256, 128, torch.float32),
    (4001, 8, 128, 64, torch.bfloat16)])
def test_append_and_read(gdn, fmt, n, h, d, p, dtype):
    g = _gen(n)
    pages = -(-n // p) + 2
    wide = torch.exp(3 * _randn(g, n, 2 * h + 1, 1)) * _randn(g, n, 2 * h + 1, d)
    wide[0, 0] = 0.0                                        # a zero vector
    if n > 2:
        wide[1, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.0])
        wide[2, 0] = 1e-38                                  # below the least scale
        wide[2, 1] = 3e38 * torch.sign(wide[2, 1])          # above the largest one
        wide[1, 1, :2] = torch.tensor([448.0 * 4, 449.0 * 4])   # both sides of a scale's edge
    wide = wide.to(dtype)
    k, v = wide[:, :h], wide[:, h:2 * h]                    # strided slices
    slots = torch.randperm(pages * p, generator=g, device="cuda")[:n].to(torch.int32)
    skip = torch.zeros(n, dtype=torch.bool, device="cuda")
    if n > 5:
        skip[5] = True
        slots[5] = -1
    c = _empty_cache(pages, h, p, d, fmt)
    before = {x: (None if y is None else y.view(torch.uint8).clone()) for x, y in c.items()}
    gdn.gdn_kv_cache_append(k, v, c["k"], c["v"], slots, k_exp=c["k_exp"], v_exp=c["v_exp"])
    _clean(gdn)
    at = (slots.long()[~skip] // p, slice(None), slots.long()[~skip] % p)
    want = {}
    for name, x in (("k", k), ("v", v)):
        got = c[name][at[0], :, at[2]] if fmt == "bf16" else (
            c[name].view(torch.uint8)[at].view(torch.float8_e4m3fn))
        if fmt == "f8":
            codes, exps = _codes(x[~skip])
            assert torch.equal(c[name + "_exp"][at], exps)
            assert torch.equal(torch.nan_to_num(got.double(), nan=1e9),
                               torch.nan_to_num(codes, nan=1e9))
            want[name] = codes * _pow2(exps.long() - 127)[..., None]
        else:
            want[name] = x[~skip].to(torch.bfloat16).double()
            assert torch.equal(torch.nan_to_num(got.double(), nan=1e9),
                               torch.nan_to_num(want[name], nan=1e9))
        # nothing else is touched
        mask = torch.ones(pages, h, p, dtype=torch.bool, device="cuda")
        mask[at] = False
        assert torch.equal(c[name].view(torch.uint8)[mask], before[name][mask])
    for odt in (torch.bfloat16, torch.float32):
        ko = torch.full((n, h, d), 7.0, dtype=odt, device="cuda")
        vo = ko.clone()
        gdn.gdn_kv_cache_read(c["k"], c["v"], slots, ko, vo, k_exp=c["k_exp"], v_exp=c["v_exp"])
        _clean(gdn)
        for name, o in (("k", ko), ("v", vo)):
            assert torch.equal(torch.nan_to_num(o[~skip].double(), nan=1e9),
                               torch.nan_to_num(want[name], nan=1e9))
            assert not o[skip].any()


def test_cache_slots_out_of_range(gdn):
    c = _empty_cache(2, 2, 16, 128, "bf16", fill=0)
    x = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([32, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_cache_append(x, x, c["k"], c["v"], slots)
    assert gdn.gdn_get_device_error() == 6
    assert float(c["k"].float().sum()) == 2 * 128 and bool((c["k"][0, :, 5] == 1).all())
    out = torch.full_like(x, 9.0)
    gdn.gdn_kv_cache_read(c["k"], c["v"], slots, out, out.clone())
    assert gdn.gdn_get_device_error() == 6
    assert bool((out[1] == 1).all()) and not out[0].any() and not out[2].any()
    _clean(gdn)


def test_cache_past_32_bits(gdn):
    """Vectors whose element offsets pass 2^31, written, read back and attended to."""
    p, d, pages = 128, 256, (1 << 16) + 40
    c = {n: torch.zeros(pages, 1, p, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
         for n in ("k", "v")}
    c |= {n + "_exp": torch.full((pages, 1, p), 127, dtype=torch.uint8, device="cuda")
          for n in ("k", "v")}
    g = _gen(3)
    n = 200
    k, v = (_randn(g, n, 1, d).to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(n, device="cuda") + (pages - 3) * p
    gdn.gdn_kv_cache_append(k, v, c["k"], c["v"], slots.to(torch.int32), k_exp=c["k_exp"],
                            v_exp=c["v_exp"])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    gdn.gdn_kv_cache_read(c["k"], c["v"], slots.to(torch.int32), ko, vo, k_exp=c["k_exp"],
                          v_exp=c["v_exp"])
    _clean(gdn)
    codes, exps = _codes(k)
    assert torch.equal(ko.double(), codes * _pow2(exps.long() - 127)[..., None])
    case = dict(q=_randn(g, 1, 1, 4, d).to(torch.bfloat16), cache=c, prefix=130,
                prefix_pages=[pages - 3, pages - 2], pages=[[pages - 2]], lens=[70])
    _check_attention(gdn, case)


# ------------------------------------------------------------------------------- attention

def _attention_case(b, t, hq, h, d, prefix, lens, p, fmt, seed, sink=False, junk=True):
    g = _gen(seed)
    shared, each = -(-prefix // p), max(1, -(-max(max(lens), 1) // p))
    pages = shared + b * each + 1
    c = _empty_cache(pages, h, p, d, fmt, fill=0x7f if junk else 0)  # NaN wherever nothing is written
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    case = dict(cache=c, prefix=prefix, prefix_pages=order[:shared],
                pages=[order[shared + i * each:shared + (i + 1) * each] for i in range(b)],
                lens=lens, q=(1.5 * _randn(g, b, t, hq, d)).to(torch.bfloat16))

    def put(n, page_list):
        for name in ("k", "v"):
            x = (_randn(g, n, h, d) * torch.exp(0.7 * _randn(g, n, h, 1))).to(torch.bfloat16)
            if sink and name == "k":
                x[0] *= 6                                   # one key that outweighs the others
            i = torch.arange(n, device="cuda")
            at = (torch.tensor(page_list, device="cuda", dtype=torch.int64)[i // p], slice(None),
                  i % p)
            if fmt == "f8":
                codes, exps = _codes(x)
                c[name].view(torch.uint8)[at] = codes.float().to(torch.float8_e4m3fn).view(
                    torch.uint8)
                c[name + "_exp"][at] = exps
            else:
                c[name][at] = x

    if prefix:
        put(prefix, case["prefix_pages"])
    for i, n in enumerate(lens):
        if n > 0:
            put(n, case["pages"][i])
    return case


def _dense(c, name, page_list, n, head, p):
    x = c[name].view(torch.uint8)[torch.tensor(page_list, dtype=torch.int64, device="cuda"), head]
    x = x.view(c[name].dtype).double()
    if c[name + "_exp"] is not None:
        e = c[name + "_exp"][torch.tensor(page_list, dtype=torch.int64, device="cuda"), head]
        x = x * _pow2(e.long() - 127)[..., None]
    return x.reshape(-1, x.shape[-1])[:n]


def _reference(case, scale):
    """out, lse and A = sum p |v| in 64 bits, row by row of the definition; max |v|."""
    q, c = case["q"].double(), case["cache"]
    b, t, hq, d = q.shape
    h, p = c["k"].shape[1], c["k"].shape[2]
    g = hq // h
    out = torch.zeros_like(q)
    size = torch.zeros_like(q)
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64, device="cuda")
    vmax = 0.0
    for head in range(h):
        pk, pv = (_dense(c, n, case["prefix_pages"], case["prefix"], head, p) for n in ("k", "v"))
        for i, n in enumerate(case["lens"]):
            if n < 0:
                continue
            sk, sv = (_dense(c, x, case["pages"][i], n, head, p) for x in ("k", "v"))
            for r in range(t):
                own = max(0, n - t + 1 + r)
                keys, vals = torch.cat([pk, sk[:own]]), torch.cat([pv, sv[:own]])
                if keys.shape[0] == 0:
                    continue
                s = q[i, r, head * g:(head + 1) * g] @ keys.T * scale
                z = torch.logsumexp(s, -1)
                pr = torch.exp(s - z[:, None])
                hs = slice(head * g, (head + 1) * g)
                out[i, r, hs], size[i, r, hs], lse[i, r, hs] = pr @ vals, pr @ vals.abs(), z
                vmax = max(vmax, float(vals.abs().max()))
    return out, lse, size, vmax


def _attend(gdn, case, odt=torch.bfloat16, scale=None, q=None, **kw):
    c = case["cache"]
    q = case["q"] if q is None else q
    out = torch.full(q.shape, float("nan"), dtype=odt, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    gdn.gdn_prefix_attention(
        q, c["k"], c["v"], out, k_exp=c["k_exp"], v_exp=c["v_exp"], lse=lse, scale=scale,
        prefix_pages=torch.tensor(case["prefix_pages"], dtype=torch.int32, device="cuda"),
        prefix_len=case["prefix"],
        pages=torch.tensor(case["pages"], dtype=torch.int32, device="cuda"),
        kv_len=torch.tensor(case["lens"], dtype=torch.int32, device="cuda"), **kw)
    return out, lse


def _check_attention(gdn, case, odt=torch.bfloat16, scale=None, **kw):
    out, lse = _attend(gdn, case, odt, scale, **kw)
    _clean(gdn)
    ref, rlse, size, vmax = _reference(case, case["q"].shape[-1] ** -0.5 if scale is None else scale)
    tol = (2.0 ** -9 + 2.0 ** -10) * size + 1e-6 * vmax
    if odt == torch.bfloat16:
        tol = tol + 2.0 ** -9 * ref.abs()
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp(min=1e-30)).max())} of its bound"
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    worst = ((lse.double() - rlse).abs() / (1 + rlse.abs()))[~empty]
    assert worst.numel() == 0 or float(worst.max()) <= 2e-5, float(worst.max())
    return out, lse


ATTENTION = [
    # b, t, hq, h, d, prefix, lens, page
    (1, 1, 1, 1, 128, 0, [1], 16),
    (1, 1, 8, 1, 128, 1, [1], 16),
    (1, 1, 24, 4, 256, 512, [37], 64),
    (3, 1, 24, 4, 256, 127, [0, 1, 130], 32),
    (3, 2, 6, 2, 128, 128, [5, -1, 129], 128),
    (4, 1, 8, 8, 256, 129, [0, 128, 127, 300], 16),
    (4, 4, 24, 4, 256, 1000, [4, 3, 0, 260], 64),
    (2, 7, 16, 2, 128, 0, [7, 200], 32),
    (5, 1, 3, 1, 128, 0, [0, -1, 0, 2, 513], 16),
    (2, 130, 6, 1, 256, 300, [130, 257], 64),
    (1, 33, 32, 4, 128, 77, [400], 16),
    (40, 1, 24, 4, 256, 650, [(i * 37) % 300 for i in range(40)], 32),
    (70, 2, 16, 2, 128, 2000, [2 + (i * 13) % 90 for i in range(70)], 64),
    (300, 1, 4, 2, 128, 256, [(i * 7) % 40 for i in range(300)], 16),
]


@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("i", range(len(ATTENTION)))
def test_attention(gdn, i, fmt):
    b, t, hq, h, d, prefix, lens, p = ATTENTION[i]
    _check_attention(gdn, _attention_case(b, t, hq, h, d, prefix, lens, p, fmt, seed=100 + i))


@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("d", [128, 256])
def test_attention_forms(gdn, fmt, d):
    """fp32 output, a scale of its own, strided queries, a key that outweighs all others."""
    case = _attention_case(3, 4, 8, 2, d, 700, [4, 90, 300], 32, fmt, seed=7, sink=True)
    _check_attention(gdn, case, odt=torch.float32)
    _check_attention(gdn, case, scale=0.02)
    _check_attention(gdn, case, scale=-0.1)
    wide = torch.randn(3, 4, 12, d, device="cuda").to(torch.bfloat16)
    wide[:, :, 2:10] = case["q"]
    plain, _ = _attend(gdn, case)
    strided, _ = _attend(gdn, case, q=wide[:, :, 2:10])
    assert torch.equal(plain, strided)


@pytest.mark.parametrize("fmt", ["bf16", "f8"])
def test_attention_scores_grow(gdn, fmt):
    """Keys whose scores rise from tile to tile (the running maximum moves all the time), fall,
    and spread over hundreds."""
    for sign in (1.0, -1.0):
        case = _attention_case(2, 1, 4, 2, 128, 1500, [40, 300], 64, fmt, seed=11)
        c = case["cache"]
        case["q"].fill_(1.0)
        ramp = sign * torch.linspace(-1.0, 1.0, 1500, device="cuda")
        i = torch.arange(1500, device="cuda")
        at = (torch.tensor(case["prefix_pages"], device="cuda")[i // 64], slice(None), i % 64)
        x = (ramp[:, None, None] + 0.01 * torch.randn(1500, 2, 128, device="cuda")).to(torch.bfloat16)
        if fmt == "f8":
            codes, exps = _codes(x)
            c["k"].view(torch.uint8)[at] = codes.float().to(torch.float8_e4m3fn).view(torch.uint8)
            c["k_exp"][at] = exps
        else:
            c["k"][at] = x
        _check_attention(gdn, case, scale=1.0)


def test_attention_value_sizes(gdn):
    """8-bit values whose scales lie far apart: tiny and zero vectors among large ones."""
    case = _attention_case(2, 2, 8, 2, 256, 600, [2, 200], 32, "f8", seed=12)
    e = case["cache"]["v_exp"]
    g = _gen(13)
    live = e != 255
    shift = torch.randint(-18, 19, e.shape, generator=g, device="cuda")
    case["cache"]["v_exp"].copy_(torch.where(live, (e.long() + shift).to(torch.uint8), e))
    zero = live & (torch.rand(e.shape, generator=g, device="cuda") < 0.2)
    case["cache"]["v"].view(torch.uint8)[zero] = 0
    case["cache"]["v_exp"][zero] = 127 - 60
    _check_attention(gdn, case)


def test_attention_only_tiny_values(gdn):
    case = _attention_case(1, 1, 4, 1, 128, 300, [3], 16, "f8", seed=14)
    e = case["cache"]["v_exp"]
    case["cache"]["v_exp"].copy_(torch.where(e != 255, torch.full_like(e, 127 - 60), e))
    _check_attention(gdn, case)


def test_attention_on_another_stream_and_in_a_graph(gdn):
    """Replayed from a graph as the sequences grow: the lengths are read on the device."""
    case = _attention_case(4, 1, 24, 4, 256, 400, [300, 300, 300, 300], 64, "bf16", seed=21)
    c, q = case["cache"], case["q"]
    i32 = dict(dtype=torch.int32, device="cuda")
    pp, pages = torch.tensor(case["prefix_pages"], **i32), torch.tensor(case["pages"], **i32)
    lens = torch.tensor([300, 300, 300, 300], **i32)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = torch.empty(gdn.gdn_prefix_attention_workspace_size(4, 1, 24, 4, 256) or 16,
                     dtype=torch.uint8, device="cuda")

    def call():
        gdn.gdn_prefix_attention(q, c["k"], c["v"], out, pages=pages, kv_len=lens,
                                 prefix_pages=pp, prefix_len=400, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    want, _ = _attend(gdn, case)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([0, 1, 299, 300], [17, 64, 65, -1], [300, 2, 0, 128]):
        lens.copy_(torch.tensor(now, **i32))
        graph.replay()
        torch.cuda.synchronize()
        want, wlse = _attend(gdn, dict(case, lens=now))
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    _clean(gdn)


def test_attention_repeats_bit_for_bit(gdn):
    case = _attention_case(9, 3, 24, 4, 256, 5000, [3 + 31 * i for i in range(9)], 64, "f8", seed=31)
    first, _ = _attend(gdn, case)
    for _ in range(3):
        again, _ = _attend(gdn, case)
        assert torch.equal(first, again)


def test_attention_records_bad_lengths_and_pages(gdn):
    case = _attention_case(2, 1, 8, 2, 128, 64, [10, 20], 32, "bf16", seed=41)
    good, _ = _attend(gdn, case)
    _clean(gdn)
    _attend(gdn, dict(case, lens=[10, 2000]))
    assert gdn.gdn_get_device_error() == 6
    for bad in (-1, case["cache"]["k"].shape[0], 2 ** 31 - 1):
        out, _ = _attend(gdn, dict(case, pages=[case["pages"][0], [bad]]))
        assert gdn.gdn_get_device_error() == 6
        assert torch.equal(out[0], good[0])
        _attend(gdn, dict(case, prefix_pages=[case["prefix_pages"][0], bad]))
        assert gdn.gdn_get_device_error() == 6
    again, _ = _attend(gdn, case)
    _clean(gdn)
    assert torch.equal(good, again)


@pytest.mark.parametrize("fmt", ["bf16", "f8"])
def test_attention_nan_stays_in_its_rows(gdn, fmt):
    """A query with a NaN or an infinity makes its own rows NaN, and a NaN key the rows that see
    it; the other rows keep their bits."""
    case = _attention_case(2, 3, 8, 2, 128, 300, [3, 200], 32, fmt, seed=61)
    good, glse = _attend(gdn, case)
    q = case["q"].clone()
    q[0, 1, 3, 5] = math.nan
    q[1, 2, 6, 0] = math.inf
    out, lse = _attend(gdn, case, q=q)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    bad[0, 1, 3] = bad[1, 2, 6] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], glse[~bad])
    # the last own token of sequence 1: seen by its last query alone
    page, off = case["pages"][1][199 // 32], 199 % 32
    case["cache"]["k"].view(torch.uint8)[page, 0, off] = 0x7f if fmt == "f8" else 0xff
    out, lse = _attend(gdn, case)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    bad[1, 2, :4] = True
    assert bool(lse[bad].isnan().all()) and bool(out[bad].isnan().all())
    assert torch.equal(out[~bad], good[~bad])


def test_attention_many_sequences(gdn):
    """More sequences than the kernel's threads lay out at a time, with and without a prefix."""
    for prefix in (0, 200):
        case = _attention_case(500, 1, 4, 2, 128, prefix, [(i * 11) % 150 - (i % 7 == 3) * 200
                                                           for i in range(500)], 16, "f8", seed=71)
        case["lens"] = [max(n, -1) for n in case["lens"]]
        _check_attention(gdn, case)


@pytest.mark.parametrize("fmt,prefix", [("bf16", 140001), ("f8", 270000)])
def test_attention_very_long_prefix(gdn, fmt, prefix):
    """Several row tiles on a prefix so long that its keys are worked on in blocks."""
    _check_attention(gdn, _attention_case(2, 33, 4, 2, 256, prefix, [33, 200], 128, fmt, seed=72))


def test_attention_no_tokens(gdn):
    case = _attention_case(1, 1, 4, 1, 128, 16, [1], 16, "bf16", seed=51)
    q = case["q"][:, :0]
    assert _attend(gdn, case, q=q)[0].numel() == 0


# ---------------------------------------------------------------------------- log probabilities

def _check_logprobs(gdn, logits, targets, k, scale=1.0, workspace=None):
    n, v = logits.shape
    lp, ent = (torch.full((n,), 77.0, device="cuda") for _ in range(2))
    ids = torch.full((n, k), -5, dtype=torch.int32, device="cuda") if k else None
    tl = torch.full((n, k), 77.0, device="cuda") if k else None
    gdn.gdn_token_logprobs(logits, targets, lp, ent, top_ids=ids, top_logprobs=tl, scale=scale,
                           workspace=workspace)
    st = gdn.gdn_get_device_error()
    assert st == (6 if bool((targets >= v).any()) else 0)
    for r in range(n):
        raw = logits[r].double()
        x = raw * float(torch.tensor(scale, dtype=torch.float32))
        if bool((raw == -math.inf).all()):
            assert float(ent[r]) == 0.0
            want, lse, dead = torch.full_like(x, -math.inf), 0.0, True
        else:
            # centred on the maximum: exact even where the logits dwarf their differences
            m = float(x.max())
            z = torch.logsumexp(x - m, 0)
            lse, dead = m + float(z), False
            want = (x - m) - z
        t = int(targets[r])
        if t < 0:
            assert float(lp[r]) == 0.0
        elif t >= v:
            assert math.isnan(float(lp[r]))
        else:
            _near(float(lp[r]), float(want[t]), 4e-6 + 2.0 ** -22 * (abs(lse) + abs(float(x[t]))))
        if not dead:
            p = torch.exp(want)
            plogp = torch.where(p > 0, p * want, torch.where(torch.isnan(p), p, torch.zeros_like(p)))
            h = -float(plogp.sum())
            spread = float(torch.where(p > 0, p * (m - x), torch.zeros_like(p)).sum())
            _near(float(ent[r]), h, 4e-6 * (2 + abs(spread)))
        if k:
            key = torch.where(torch.isnan(raw), torch.full_like(raw, math.inf), raw)
            order = sorted(range(v), key=lambda i: (not math.isnan(raw_list[i]), -key_list[i], i)) \
                if v <= 2000 and (raw_list := raw.tolist()) is not None and \
                (key_list := key.tolist()) is not None else \
                torch.sort(raw, descending=True, stable=True).indices[:k].tolist()
            assert ids[r].tolist() == order[:k]
            for j in range(k):
                xv = float(x[order[j]])
                _near(float(tl[r, j]), float(want[order[j]]), 4e-6 + 2.0 ** -22 * (
                    abs(lse) + (abs(xv) if math.isfinite(xv) else 0)))


def _near(got, want, tol):
    if math.isnan(want):
        assert math.isnan(got)
    elif math.isinf(want):
        assert got == want
    else:
        assert abs(got - want) <= tol, (got, want, tol)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v,k", [(1, 1, 1), (1, 2, 0), (2, 31, 31), (3, 1000, 5), (1, 4097, 32),
                                   (5, 12345, 20), (1, 248320, 20), (2, 151669, 1),
                                   (40, 70001, 3), (400, 3001, 2)])
def test_logprobs(gdn, n, v, k, dtype):
    g = _gen(n * v + k)
    x = (3 * _randn(g, n, v)).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    if n > 2:
        t[1] = -1
    _check_logprobs(gdn, x, t, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_strides_and_alignment(gdn, dtype):
    g = _gen(5)
    for cut in (1, 3, 8):
        wide = (2 * _randn(g, 6, 5003 + cut)).to(dtype)
        x = wide[:, cut:]
        assert x.stride(0) == 5003 + cut
        t = torch.randint(0, 5003, (6,), generator=g, device="cuda", dtype=torch.int32)
        _check_logprobs(gdn, x, t, 7, scale=0.7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [40, 1500, 100003])
def test_logprobs_hard_rows(gdn, v, dtype):
    """Ties, masked logits (-inf and the type's lowest value), rows with one or no live logit,
    infinities, NaN, signed zeros, rows that rise or fall all along, a far outlier."""
    g = _gen(v)
    low = torch.finfo(dtype).min
    r = lambda: 2 * _randn(g, v)                                            # noqa: E731
    rows = [torch.zeros(v, device="cuda"), torch.full((v,), -math.inf, device="cuda"),
            torch.full((v,), float(low), device="cuda")]
    one = torch.full((v,), -math.inf, device="cuda")
    one[v // 3] = -2.5
    half = r()
    half[torch.rand(v, generator=g, device="cuda") < 0.5] = -math.inf
    lows = r()
    lows[::2] = low
    nan = r()
    nan[v // 2] = math.nan
    pinf = r()
    pinf[v - 1] = math.inf
    zeros = torch.zeros(v, device="cuda")
    zeros[::3] = -0.0
    up = torch.linspace(-9, 9, v, device="cuda")
    outlier = r()
    outlier[v - 2] = 60.0
    ties = (torch.randint(0, 3, (v,), generator=g, device="cuda")).float()
    rows += [one, half, lows, nan, pinf, zeros, up, -up, outlier, ties]
    x = torch.stack(rows).to(dtype)
    n = len(rows)
    t = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    t[3] = v // 3
    t[0] = v
    _check_logprobs(gdn, x, t, min(v, 32))
    _check_logprobs(gdn, x, t, 1)
    _check_logprobs(gdn, x, t, 0)


def test_own_workspace_belongs_to_the_stream(gdn, monkeypatch):
    """A workspace that a call allocates comes from the stream it runs on (a Stream, a raw one)."""
    x = torch.zeros(2, 5000, dtype=torch.bfloat16, device="cuda")
    ent = torch.empty(2, device="cuda")
    q = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen, empty = [], torch.empty

    def recorded(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", recorded)
    for stream in (side, side.cuda_stream):
        gdn.gdn_token_logprobs(x, None, None, ent, stream=stream)
        gdn.gdn_prefix_attention(q, kv, kv, out, pages=one, kv_len=one[0], stream=stream)
    monkeypatch.undo()
    side.synchronize()
    _clean(gdn)
    assert seen == [side.cuda_stream] * 4


def test_logprobs_parts_and_streams(gdn):
    """Without targets or without entropy; on another stream; bit for bit the same again."""
    g = _gen(9)
    x = (3 * _randn(g, 4, 50000)).to(torch.bfloat16)
    t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    a = [torch.empty(4, device="cuda") for _ in range(2)]
    ids = torch.empty(4, 8, dtype=torch.int32, device="cuda")
    tl = torch.empty(4, 8, device="cuda")
    gdn.gdn_token_logprobs(x, t, *a, top_ids=ids, top_logprobs=tl)
    ent = torch.empty(4, device="cuda")
    gdn.gdn_token_logprobs(x, None, None, ent)
    lp = torch.empty(4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gdn.gdn_token_logprobs(x, t, lp, stream=side)
    side.synchronize()
    ids2, tl2 = torch.empty_like(ids), torch.empty_like(tl)
    gdn.gdn_token_logprobs(x, None, None, top_ids=ids2, top_logprobs=tl2)
    _clean(gdn)
    assert torch.equal(lp, a[0]) and torch.equal(ent, a[1])
    assert torch.equal(ids, ids2) and torch.equal(tl, tl2)
