"""gdn_qk_norm_rope against its definition in 64 bits.

Tolerance, per element, with (a, b) the pair's normalised elements: the sum of squares has at most
13 roundings in a row (eight elements a lane, then five levels), half of which reach 1 / sqrt, whose
function is good to 2^-22; with the two products the norm is within 13 2^-24 + 2^-22 < 2^-20.  cos
and sin come from an angle rounded to 2^-24 of half a turn (2^-22.3) by a function good to 2^-23:
2^-21.5 each.  Two products and a sum more: |error| <= A (|a| + |b|) 2^-19, A the amplitude.  An
element that is not turned has |a| 2^-20.  A stored value is rounded once more, by half a step: bf16
2^-8 (fp32 2^-24) of its size.  An 8-bit code is off by 2^-4 of its value or 2^-10 of its scale, and
the scale's exponent is the least that holds the vector's largest size, itself within 2^-19.
Without norm and rotation (values) nothing is rounded but the result.
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


def _angles(positions, steps):
    """Exactly reduced: the phase as a 64-bit whole number, in turns of [-1/2, 1/2)."""
    return (positions.long()[:, None] * steps).double() * 2.0 ** -64 * (2 * math.pi)


def _definition(x, weight, eps, positions, steps, amplitude, interleaved):
    """(value, bound on the error before the last rounding) in 64 bits."""
    x = x.double()
    bound = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
        bound = x.abs() * 2.0 ** -20
    r = 0 if steps is None else 2 * steps.numel()
    if r:
        i = torch.arange(r // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        a, b = x[..., first], x[..., second]
        w = _angles(positions, steps)[:, None]
        y, bound = x.clone(), bound.clone()
        y[..., first] = amplitude * (a * torch.cos(w) - b * torch.sin(w))
        y[..., second] = amplitude * (a * torch.sin(w) + b * torch.cos(w))
        size = abs(amplitude) * (a.abs() + b.abs()) * 2.0 ** -19
        bound[..., first], bound[..., second] = size, size
        x = y
    return x, bound


def _half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def _compare(got, want, bound, dtype):
    err = (got.double() - want).abs()
    limit = bound + _half_step(dtype) * (want.abs() + bound) + 1e-44
    assert bool((err <= limit).all()), float((err / limit).max())


def _compare_f8(codes, exps, want, bound):
    """codes (float8), exps (biased) of vectors `want`."""
    e = exps.double() - 127
    top = want.abs().amax(-1)
    slack = bound.amax(-1)
    scale = torch.exp2(e)
    assert bool((scale * 448 >= (top - slack) * (e < 60)).all())
    assert bool(((scale / 2 * 448 < top + slack) | (e == -60)).all())
    err = (codes.double() * scale[..., None] - want).abs()
    limit = bound + 2.0 ** -4 * (want.abs() + bound) + scale[..., None] * 2.0 ** -10
    assert bool((err <= limit).all()), float((err / limit).max())


def _steps(gdn, rot, base=10000.0, **kw):
    return gdn.gdn_rope_phase_steps(rot, base, **kw) if rot else (None, 1.0)


FAR = [0, 1, 2 ** 31 - 1, -(2 ** 31), -1, 123456789]


def _inputs(n, hq, h, d, dtype, gated, seed):
    """Queries, keys and values of one projection's rows; gates may lie between the queries."""
    g = _gen(seed)
    width = hq * (2 if gated else 1) + 2 * h
    rows = (_randn(g, n, width, d) * torch.exp(_randn(g, n, width, 1))).to(dtype)
    q = rows[:, :2 * hq:2] if gated else rows[:, :hq]
    positions = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    for i, x in enumerate(FAR[:n]):
        positions[i] = x
    weights = [1 + 0.3 * _randn(g, d) for _ in range(2)]
    return q, rows[:, -2 * h:-h], rows[:, -h:], positions, weights


CASES = [  # n, hq, h, d, rot
    (1, 24, 4, 256, 64), (1, 1, 1, 8, 8), (2, 3, 1, 64, 64), (3, 8, 2, 128, 128), (7, 5, 5, 96, 96),
    (33, 6, 2, 96, 48), (65, 16, 2, 128, 20), (5, 24, 4, 256, 250), (129, 4, 1, 24, 2),
    (300, 24, 4, 256, 64), (1000, 16, 2, 128, 128), (2501, 3, 1, 192, 90), (700, 12, 3, 248, 0),
    (4097, 2, 1, 64, 16),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,h,d,rot", CASES)
def test_tensors(gdn, n, hq, h, d, rot, dtype, interleaved):
    q, k, _, positions, (wq, wk) = _inputs(n, hq, h, d, dtype, n % 2 == 1, seed=n + d)
    steps, _ = _steps(gdn, rot)
    q_out = torch.full((n, hq, d), 9.0, device="cuda", dtype=dtype)
    k_out = torch.full((n, h, d), 9.0, device="cuda", dtype=dtype)
    gdn.gdn_qk_norm_rope(q, k, positions, steps, q_out, k_out, q_weight=wq, k_weight=wk, eps=1e-5,
                         interleaved=interleaved, amplitude=1.25)
    _clean(gdn)
    for x, w, out in ((q, wq, q_out), (k, wk, k_out)):
        want, bound = _definition(x, w, 1e-5, positions, steps, 1.25, interleaved)
        _compare(out, want, bound, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("n,hq,h,d,rot,page,dtype", [
    (1, 24, 4, 256, 64, 64, torch.bfloat16), (3, 2, 1, 128, 128, 16, torch.float32),
    (77, 24, 4, 256, 250, 128, torch.bfloat16), (1500, 6, 3, 128, 32, 32, torch.bfloat16),
    (900, 8, 1, 256, 256, 64, torch.float32)])
def test_cache(gdn, n, hq, h, d, rot, page, dtype, fmt, interleaved):
    q, k, v, positions, (wq, wk) = _inputs(n, hq, h, d, dtype, n % 2 == 0, seed=n)
    steps, amplitude = _steps(gdn, rot, 1e6, scaling="yarn", factor=4.0, original_context=8192)
    g = _gen(n + 1)
    pages = -(-n // page) + 2
    cache = {}
    for name in ("k", "v"):
        fill = torch.randint(0, 120, (pages, h, page, d * (1 if fmt == "f8" else 2)), generator=g,
                             device="cuda", dtype=torch.uint8)
        cache[name] = fill.view(torch.float8_e4m3fn if fmt == "f8" else torch.bfloat16)
        cache[name + "_exp"] = (torch.full((pages, h, page), 99, device="cuda", dtype=torch.uint8)
                                if fmt == "f8" else None)
    before = {x: None if y is None else y.view(torch.uint8).clone() for x, y in cache.items()}
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    if n > 5:
        slots[4], live[4] = -1, False
        slots[n - 1], live[n - 1] = -2 ** 31, False
    q_out = torch.full((n, hq, d), 9.0, device="cuda", dtype=dtype)
    k_out = torch.full((n, h, d), 9.0, device="cuda", dtype=dtype) if n % 3 == 0 else None
    gdn.gdn_qk_norm_rope(q, k, positions, steps, q_out, k_out, q_weight=wq, k_weight=wk,
                         interleaved=interleaved, amplitude=amplitude, v=v, k_cache=cache["k"],
                         v_cache=cache["v"], slots=slots, k_exp=cache["k_exp"],
                         v_exp=cache["v_exp"])
    _clean(gdn)
    want, bound = _definition(q, wq, 1e-6, positions, steps, amplitude, interleaved)
    _compare(q_out, want, bound, dtype)
    key = _definition(k, wk, 1e-6, positions, steps, amplitude, interleaved)
    if k_out is not None:
        _compare(k_out, *key, dtype)
    at = (slots.long()[live] // page, slice(None), slots.long()[live] % page)
    for name, (want, bound) in (("k", key), ("v", (v.double(), torch.zeros(n, h, d, device="cuda")))):
        got = cache[name].view(torch.uint8)[at].view(cache[name].dtype)
        if fmt == "f8":
            _compare_f8(got, cache[name + "_exp"][at], want[live], bound[live].double())
        else:
            _compare(got, want[live], bound[live].double(), torch.bfloat16)
        rest = torch.ones(pages, h, page, dtype=torch.bool, device="cuda")
        rest[at] = False                                   # nothing else is touched
        assert torch.equal(cache[name].view(torch.uint8)[rest], before[name][rest])
        if fmt == "f8":
            assert torch.equal(cache[name + "_exp"][rest], before[name + "_exp"][rest])


def test_values_are_appended_as_by_the_cache_write(gdn):
    """Values (and keys without norm or rotation) go to the cache exactly as gdn_kv_cache_append
    writes them, special values among them."""
    n, h, d, page = 40, 2, 128, 16
    g = _gen(5)
    x = _randn(g, n, 4 * h, d) * torch.exp(8 * _randn(g, n, 4 * h, 1))
    x[0] = 0.0
    x[1, :, :3] = torch.tensor([math.nan, math.inf, -math.inf], device="cuda")
    x[2], x[3] = 1e-38, 3e38
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        q, k, v = y[:, :2 * h], y[:, 2 * h:3 * h], y[:, 3 * h:]
        slots = torch.randperm(48, generator=g, device="cuda")[:n].to(torch.int32)
        for f8 in (True, False):
            made = []
            for _ in range(2):
                c = [torch.zeros(3, h, page, d, device="cuda",
                                 dtype=torch.uint8 if f8 else torch.bfloat16) for _ in range(2)]
                c = [t.view(torch.float8_e4m3fn) if f8 else t for t in c]
                e = [torch.zeros(3, h, page, device="cuda", dtype=torch.uint8) if f8 else None
                     for _ in range(2)]
                made.append(c + e)
            gdn.gdn_kv_cache_append(k, v, made[0][0], made[0][1], slots, k_exp=made[0][2],
                                    v_exp=made[0][3])
            q_out = torch.empty(n, 2 * h, d, device="cuda", dtype=dtype)
            gdn.gdn_qk_norm_rope(q, k, None, None, q_out, v=v, k_cache=made[1][0],
                                 v_cache=made[1][1], slots=slots, k_exp=made[1][2],
                                 v_exp=made[1][3])
            _clean(gdn)
            for a, b in zip(*made):
                if a is not None:
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            assert torch.equal(q_out.view(torch.uint8), q.contiguous().view(torch.uint8))


def test_slots_out_of_range(gdn):
    n, h, d = 4, 1, 128
    x = torch.ones(n, 3, d, device="cuda", dtype=torch.bfloat16)
    c = torch.zeros(2, h, 16, d, device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([31, 32, 2 ** 31 - 1, 3], device="cuda", dtype=torch.int32)
    out = torch.empty(n, 1, d, device="cuda", dtype=torch.bfloat16)
    gdn.gdn_qk_norm_rope(x[:, :1], x[:, 1:2], None, None, out, v=x[:, 2:], k_cache=c,
                         v_cache=c.clone(), slots=slots)
    assert gdn.gdn_get_device_error() == 6
    assert float(c.float().sum()) == 2 * d and bool((out == 1).all())
    _clean(gdn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_and_one_weight(gdn, dtype):
    """q_out is q, k_out is k; a missing weight leaves its heads without a norm."""
    for n in (3, 3001):
        g = _gen(n)
        q = _randn(g, n, 6, 128).to(dtype)
        k = _randn(g, n, 2, 128).to(dtype)
        positions = torch.arange(n, device="cuda", dtype=torch.int32)
        steps, _ = _steps(gdn, 64)
        w = 1 + 0.1 * _randn(g, 128)
        q0, k0 = q.clone(), k.clone()
        gdn.gdn_qk_norm_rope(q, k, positions, steps, q, k, k_weight=w)
        _clean(gdn)
        _compare(q, *_definition(q0, None, 0, positions, steps, 1.0, False), dtype)
        _compare(k, *_definition(k0, w, 1e-6, positions, steps, 1.0, False), dtype)


def test_turning_back(gdn):
    """The rotation by -p undoes the one by p: the angles of both are exact."""
    n, d = 64, 256
    g = _gen(8)
    q = _randn(g, n, 3, d)
    p = torch.randint(0, 2 ** 31 - 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    steps, _ = _steps(gdn, d)
    out, k = torch.empty_like(q), torch.empty(n, 1, d, device="cuda")
    gdn.gdn_qk_norm_rope(q, q[:, :1], p, steps, out, k)
    gdn.gdn_qk_norm_rope(out, k, -p, steps, out, k)
    _clean(gdn)
    pair = q[..., :d // 2].abs() + q[..., d // 2:].abs()
    assert bool(((out - q).abs() <= 2.0 ** -17 * torch.cat([pair, pair], -1)).all())


def test_special_values_stay_in_their_vector(gdn):
    n, hq, d = 9, 4, 128
    g = _gen(3)
    q = _randn(g, n, hq, d).to(torch.bfloat16)
    k = _randn(g, n, 2, d).to(torch.bfloat16)
    p = torch.arange(n, device="cuda", dtype=torch.int32)
    steps, _ = _steps(gdn, 32)
    w = torch.ones(d, device="cuda")
    clean = [torch.empty_like(q), torch.empty_like(k)]
    gdn.gdn_qk_norm_rope(q, k, p, steps, *clean, q_weight=w, k_weight=w)
    q[2, 1, 5], q[4, 3, 100], k[6, 0, 7], q[0, 0] = math.nan, math.inf, math.nan, 0.0
    out = [torch.empty_like(q), torch.empty_like(k)]
    gdn.gdn_qk_norm_rope(q, k, p, steps, *out, q_weight=w, k_weight=w)
    _clean(gdn)
    assert bool(out[0][2, 1].isnan().all()) and bool(out[1][6, 0].isnan().all())
    assert bool(out[0][4, 3, 100].isnan()) and not out[0][0, 0].any()
    for a, b, touched in ((out[0], clean[0], [(2, 1), (4, 3), (0, 0)]), (out[1], clean[1], [(6, 0)])):
        same = torch.ones(a.shape[:2], dtype=torch.bool, device="cuda")
        for t in touched:
            same[t] = False
        assert torch.equal(a[same], b[same])


def test_graph_and_streams(gdn):
    """Captured with its positions and slots on the device, replayed as they move on, on a stream
    of its own; bit for bit what a plain call gives."""
    n, hq, h, d, page = 12, 4, 2, 256, 16
    g = _gen(1)
    x = _randn(g, n, hq + 2 * h, d).to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
    steps, _ = _steps(gdn, 64)
    w = 1 + 0.1 * _randn(g, d)
    p = torch.arange(n, device="cuda", dtype=torch.int32)
    slots = p.clone()

    def call(c, out, stream=None):
        gdn.gdn_qk_norm_rope(q, k, p, steps, out, q_weight=w, k_weight=w, v=v, k_cache=c[0],
                             v_cache=c[1], slots=slots, stream=stream)

    def fresh():
        return [torch.zeros(4, h, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]

    one, two = fresh(), fresh()
    out, out2 = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(one, out)
    for i in range(3):
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        call(two, out2, stream=side)
        side.synchronize()
        assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(one, two))
        p += 1000003
        slots += n
        torch.cuda.synchronize()
    _clean(gdn)


def test_refusals(gdn):
    q = torch.zeros(2, 4, 128, device="cuda", dtype=torch.bfloat16)
    k = q[:, :2].contiguous()
    p = torch.zeros(2, device="cuda", dtype=torch.int32)
    steps, _ = _steps(gdn, 64)
    c = torch.zeros(1, 2, 16, 128, device="cuda", dtype=torch.bfloat16)
    call = gdn.gdn_qk_norm_rope
    for bad in (dict(q_out=q[:, :2]), dict(q_out=q.float()), dict(k_out=None), dict(k=k.float()),
                dict(positions=p.long()), dict(positions=p[:1]), dict(steps=steps.int()),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=q.half()),
                dict(q_weight=torch.ones(128, device="cuda", dtype=torch.bfloat16)),
                dict(k_weight=torch.ones(64, device="cuda")), dict(q=q.cpu()), dict(v=k),
                dict(k_cache=c, v_cache=c, slots=p), dict(k_cache=c, v_cache=c, v=k),
                dict(k_cache=c, v_cache=c[:, :1], v=k, slots=p)):
        a = {**dict(q=q, k=k, positions=p, steps=steps, q_out=q, k_out=k), **bad}
        with pytest.raises((ValueError, TypeError, AttributeError, gdn.GDNError)):
            call(a.pop("q"), a.pop("k"), a.pop("positions"), a.pop("steps"), a.pop("q_out"),
                 a.pop("k_out"), **a)
    empty = q[:0]
    call(empty, k[:0], p[:0], steps, empty.clone(), k[:0].clone())
    _clean(gdn)
