"""The serving step's entry points without a GPU (query/key norm with rotation, page plans and
releases, verification of drafted tokens): bad arguments are refused on the host before any CUDA
call, empty calls are no-ops; the rotation's phase steps against 50-digit arithmetic.  No call
here reaches a launch.
"""
import ctypes
import decimal
import math
from decimal import Decimal

import pytest
import torch

import gated_deltanet_linear_13_gb300 as gdn
from gated_deltanet_linear_13_gb300 import build_lib

A = 0x10000   # a fake, 16-byte aligned address


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return gdn.load_library()


def _cache(**kw):
    base = dict(num_pages=8, page_size=64, num_kv_heads=4, head_dim=256, format=gdn.GDN_KV_BF16,
                k=A, v=A, k_exp=None, v_exp=None)
    base.update(kw)
    return gdn.GdnKvCache(*[base[f] for f, _ in gdn.GdnKvCache._fields_])


ROPE = dict(n=4, hq=24, h=4, d=256, dt=gdn.GDN_BF16, q=A, qt=24 * 512, qh=512, k=A, kt=1024, qw=A,
            kw=A, eps=1e-6, pos=A, rot=64, layout=0, amp=1.0, steps=A, qo=A, qot=24 * 256, ko=A,
            cache=None, v=A, vt=1024, slots=A)


def _rope(L, **kw):
    a = {**ROPE, **kw}
    rope = gdn.GdnRope(a["rot"], a["layout"], a["amp"], a["steps"])
    cache = None if a["cache"] is None else ctypes.byref(a["cache"])
    return L.gdn_qk_norm_rope(a["n"], a["hq"], a["h"], a["d"], a["dt"], a["q"], a["qt"], a["qh"],
                              a["k"], a["kt"], a["qw"], a["kw"], a["eps"], a["pos"],
                              None if kw.get("no_rope") else ctypes.byref(rope), a["qo"],
                              a["qot"], a["ko"], cache, a["v"], a["vt"], a["slots"], None)


BAD_ROPE = [
    (dict(n=-1), 1), (dict(hq=0), 1), (dict(h=0), 1), (dict(d=0), 1), (dict(dt=7), 1),
    (dict(no_rope=True), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(n=(1 << 30) + 1), 2), (dict(d=260), 2), (dict(d=264), 2), (dict(d=100), 2), (dict(hq=65535), 2),
    (dict(rot=-2), 1), (dict(rot=63), 1), (dict(rot=258), 1), (dict(layout=2), 1),
    (dict(amp=math.nan), 1), (dict(steps=None), 1), (dict(steps=A + 4), 1), (dict(pos=None), 1),
    (dict(pos=A + 2), 1), (dict(q=None), 1), (dict(q=A + 8), 1), (dict(k=None), 1),
    (dict(k=A + 2), 1), (dict(qo=None), 1), (dict(qo=A + 4), 1), (dict(qw=A + 4), 1),
    (dict(kw=A + 8), 1), (dict(ko=A + 8), 1), (dict(ko=None), 1),
    (dict(qh=248), 1), (dict(qh=516), 1), (dict(qt=24 * 512 + 4), 1), (dict(qt=24 * 512 - 512), 1),
    (dict(kt=1016), 1), (dict(kt=1028), 1), (dict(qot=24 * 256 - 8), 1), (dict(qot=24 * 256 + 4), 1),
    (dict(cache=_cache(num_pages=-1)), 1), (dict(cache=_cache(page_size=48)), 2),
    (dict(cache=_cache(num_kv_heads=2)), 1), (dict(cache=_cache(head_dim=128)), 1),
    (dict(cache=_cache(format=1)), 1), (dict(cache=_cache(), v=None), 1),
    (dict(cache=_cache(), v=A + 8), 1), (dict(cache=_cache(), vt=1000), 1),
    (dict(cache=_cache(), vt=1028), 1), (dict(cache=_cache(), slots=None), 1),
    (dict(cache=_cache(), slots=A + 1), 1),
    (dict(dt=gdn.GDN_F32, qt=24 * 512 + 2), 1),
]


@pytest.mark.parametrize("bad,status", BAD_ROPE)
def test_rope_refusals(L, bad, status):
    assert _rope(L, **bad) == status


def test_rope_empty(L):
    assert _rope(L, n=0, q=None, k=None, qo=None, ko=None, pos=None, steps=None) == 0


POOL = dict(num_pages=100, page_size=16, num_rows=8, max_pages=50, table=A, held=A, free_pages=A,
            free_count=A)


def _pool(**kw):
    return gdn.GdnPagePool(*[{**POOL, **kw}[f] for f, _ in gdn.GdnPagePool._fields_])


BAD_POOL = [
    (dict(num_pages=-1), 1), (dict(num_rows=-1), 1), (dict(max_pages=-1), 1),
    (dict(page_size=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=256), 2), (dict(num_pages=1 << 27), 2), (dict(max_pages=1 << 27), 2),
    (dict(table=None), 1), (dict(held=None), 1), (dict(free_pages=None), 1),
    (dict(free_count=None), 1), (dict(table=A + 1), 1), (dict(held=A + 2), 1),
    (dict(free_pages=A + 3), 1), (dict(free_count=A + 2), 1),
]


@pytest.mark.parametrize("bad,status", BAD_POOL)
def test_bad_pools_are_refused(L, bad, status):
    p = ctypes.byref(_pool(**bad))
    assert L.gdn_page_plan(p, 2, None, A, A, 64, 0, A, A, A, A, A, None) == status
    assert L.gdn_page_release(p, 2, None, A, None) == status


def test_page_arguments(L):
    def plan(p=_pool(), b=2, rows=A, kv=A, new=A, cap=64, off=0, slots=A, pos=A, cu=A, out=A, pg=A):
        return L.gdn_page_plan(ctypes.byref(p), b, rows, kv, new, cap, off, slots, pos, cu, out, pg,
                               None)

    assert L.gdn_page_plan(None, 2, None, A, A, 64, 0, A, A, A, A, A, None) == 1
    assert plan(b=-1) == 1 and plan(b=8193) == 2
    assert plan(cap=-1) == 1 and plan(off=-1) == 1 and plan(off=0x7fffffff) == 2
    assert plan(kv=None) == 1 and plan(new=None) == 1
    for name in ("rows", "kv", "new", "slots", "pos", "cu", "out", "pg"):
        assert plan(**{name: A + 2}) == 1
    assert L.gdn_page_release(None, 2, None, A, None) == 1
    p = ctypes.byref(_pool())
    assert L.gdn_page_release(p, -1, None, A, None) == 1
    assert L.gdn_page_release(p, 8193, None, A, None) == 2
    assert L.gdn_page_release(p, 2, None, None, None) == 1
    assert L.gdn_page_release(p, 2, A + 1, A, None) == 1
    assert L.gdn_page_release(p, 2, None, A + 2, None) == 1
    assert L.gdn_page_release(p, 0, None, None, None) == 0


def test_verify_arguments(L):
    need = L.gdn_verify_tokens_workspace_size(3, 4, 1000, gdn.GDN_BF16, 1)
    assert need > 0

    def verify(b=3, t=4, v=1000, dt=gdn.GDN_BF16, x=A, xs=1000, ids=A, y=A, ys=1000, u=A, clocks=A,
               scale=A, tokens=A, accepted=A, lp=A, ws=A, wsb=need):
        return L.gdn_verify_tokens(b, t, v, dt, x, xs, ids, y, ys, u, clocks, scale, tokens,
                                   accepted, lp, ws, wsb, None)

    assert verify(b=-1) == 1 and verify(t=-1) == 1 and verify(v=0) == 1 and verify(dt=3) == 1
    assert verify(t=65) == 2 and verify(v=(1 << 30) + 1) == 2 and verify(b=(1 << 24) + 1) == 2
    assert verify(x=None) == 1 and verify(x=A + 1) == 1 and verify(xs=999) == 1
    assert verify(dt=gdn.GDN_F32, x=A + 2) == 1
    assert verify(ids=None) == 1 and verify(ids=A + 2) == 1
    assert verify(y=A + 1) == 1 and verify(ys=999) == 1
    assert verify(u=None) == 1 and verify(u=A + 2) == 1
    assert verify(clocks=None) == 1 and verify(clocks=A + 3) == 1
    assert verify(scale=A + 1) == 1 and verify(tokens=None) == 1 and verify(tokens=A + 2) == 1
    assert verify(accepted=None) == 1 and verify(accepted=A + 1) == 1 and verify(lp=A + 2) == 1
    assert verify(ws=None) == 3 and verify(ws=A + 8) == 3 and verify(wsb=need - 1) == 3
    assert verify(b=0, x=None, ws=None) == 0
    size = L.gdn_verify_tokens_workspace_size
    assert size(0, 4, 1000, gdn.GDN_BF16, 1) == 0 and size(3, 65, 1000, gdn.GDN_BF16, 1) == 0
    assert size(3, 4, 0, gdn.GDN_BF16, 1) == 0 and size(3, 4, 1000, 9, 1) == 0
    assert size(3, 0, 1000, gdn.GDN_F32, 1) == size(3, 0, 1000, gdn.GDN_F32, 0) > 0


# ------------------------------------------------------------------------- phase steps

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def _steps(r, base, scaling, factor, original, fast, slow):
    """The definition in 50 digits: steps and amplitude."""
    with decimal.localcontext() as c:
        c.prec = 50
        base, factor = Decimal(base), Decimal(factor)
        if scaling == "ntk" and r > 2:
            base *= factor ** (Decimal(r) / Decimal(r - 2))
        f = [base ** (Decimal(-2 * p) / Decimal(r)) for p in range(r // 2)]
        if scaling == "linear":
            f = [x / factor for x in f]
        amplitude = Decimal(1)
        if scaling == "yarn":
            amplitude = factor.ln() / 10 + 1

            def pair(turns):
                return r * (Decimal(original) / (Decimal(turns) * 2 * PI)).ln() / (2 * base.ln())

            lo = max(Decimal(0), pair(fast).to_integral_value(decimal.ROUND_FLOOR))
            hi = min(Decimal(r - 1), pair(slow).to_integral_value(decimal.ROUND_CEILING))
            span = max(hi - lo, Decimal("0.001"))
            w = [min(Decimal(1), max(Decimal(0), (p - lo) / span)) for p in range(r // 2)]
            f = [x / factor * y + x * (1 - y) for x, y in zip(f, w)]
        return [x / (2 * PI) * 2 ** 64 for x in f], float(amplitude)


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
@pytest.mark.parametrize("r,base,factor", [(64, 1e7, 4.0), (2, 10000.0, 1.0), (128, 5e5, 8.0),
                                           (96, 10000.0, 40.0), (250, 1.5, 2.5)])
def test_phase_steps(L, r, base, factor, scaling):
    """pow, log and their arguments in double: relative 2^-46 of a step is a generous count of
    their roundings (an exponent of up to 24 doublings loses five bits)."""
    args = dict(factor=factor, original_context=32768.0)
    steps, amplitude = gdn.gdn_rope_phase_steps(r, base, scaling=scaling, device="cpu", **args)
    want, amp = _steps(r, base, scaling, factor, 32768, 32, 1)
    assert steps.shape == (r // 2,) and steps.dtype is torch.int64
    for got, x in zip(steps.tolist(), want):
        assert abs(Decimal(got % 2 ** 64) - x) <= x * Decimal(2) ** -46 + 1
    assert abs(amplitude - amp) <= 2.0 ** -23 * amp


def test_phase_step_refusals(L):
    steps = (ctypes.c_uint64 * 64)()
    amp = ctypes.c_float()

    def make(r=64, base=1e4, scaling=0, factor=1.0, original=4096.0, fast=32.0, slow=1.0,
             out=steps, a=ctypes.byref(amp)):
        return L.gdn_rope_phase_steps(r, base, scaling, factor, original, fast, slow, out, a)

    assert make() == 0 and make(r=0, out=None) == 0
    assert make(r=-2) == 1 and make(r=7) == 1 and make(out=None) == 1 and make(a=None) == 1
    for base in (1.0, 0.5, -3.0, math.inf, math.nan):
        assert make(base=base) == 1
    assert make(scaling=4) == 1 and make(scaling=-1) == 1
    for s in (1, 2, 3):
        for factor in (0.5, -1.0, math.nan, math.inf):
            assert make(scaling=s, factor=factor) == 1
    assert make(scaling=2, base=1e300, factor=1e300) == 1
    assert make(scaling=3, original=0.0) == 1 and make(scaling=3, fast=1.0) == 1
    assert make(scaling=3, slow=0.0) == 1 and make(scaling=3, fast=math.inf) == 1
    with pytest.raises(ValueError):
        gdn.gdn_rope_phase_steps(64, scaling="other", device="cpu")


def test_binding_needs_cuda_tensors():
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_qk_norm_rope(q, k, None, None, q, k)
    i = torch.zeros(4, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_page_plan(i[0], i[0], table=i, held=i[0], free_pages=i[0], free_count=i[0, :1],
                          page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_page_release(i[0], table=i, held=i[0], free_pages=i[0], free_count=i[0, :1],
                             page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_verify_tokens(torch.zeros(1, 1, 8), i[:1, :1], i[0, :1], clocks=torch.zeros(1, 8))
