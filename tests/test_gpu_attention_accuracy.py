"""How exact shared-prefix attention is with fp32 outputs: the bits that include/gdn.h promises.

Bound of a row's element, all sums over its visible keys j, p_j the softmax in 64 bits:

  * Scores: fp32 sums of exact products; with D / 16 <= 16 steps of an addition and its operands'
    alignment each, 2^-19 sum_i |q_i k_ji| scale (in nats) =: eps_j.  8-bit cache: a query is the
    sum of two e4m3 numbers; what that leaves out of it is computed here, its product with k_j is
    added to eps_j.  An error eps_j of a score moves p_j by a factor of e^eps_j:
    sum p_j eps_j |v_j| + (sum p_j |v_j|) sum p_j eps_j.
  * Probabilities: 2^-21 for the exponential and the sums' reference, and the rounding of P for the
    second product: bf16 cache 2^-16 (the leading eight bits by truncation, the rest to eight);
    8-bit cache 2^-11 (eleven bits, half a unit), and no finer than half of e5m2's least number,
    2^-17, against a largest one of at least 2^8 in which the values' scales are:
    2^-25 max_i(p_i 2^e_i) |code_j|.
  * fp32 sums of the second product and of l: 2^-24 an addition, n / 8 + 64 of them for n keys.
"""
import pytest
import torch


def split_query(q):
    """What the two e4m3 terms of a query row hold of it (64 bits)."""
    top = q.double().abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    frac, e = torch.frexp(top)                              # top = frac 2^e, frac of [1/2, 1)
    e = e - 9 + (frac > 0.875).to(e.dtype)                  # top 2^-e of (224, 448]
    x = torch.ldexp(q.double(), -e)
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 4)
    hi = torch.round(x / step) * step                       # four significant bits
    lo = (x - hi).float().to(torch.float8_e4m3fn).double()
    return torch.ldexp(hi + lo, e)


def softmax_and_bound(q, k, v, codes, exps, scale, f8):
    """Rows q [r, D] over keys k and values v [n, D] in 64 bits: out, its bound, lse, its bound."""
    q, k, v = q.double(), k.double(), v.double()
    s = q @ k.T * scale
    z = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - z)
    eps = 2.0 ** -19 * abs(scale) * (q.abs() @ k.abs().T)
    if f8:
        eps = eps + abs(scale) * ((q - split_query(q)) @ k.T).abs()
    size, peps = p @ v.abs(), (p * eps).sum(-1, keepdim=True)
    sums = 2.0 ** -24 * (k.shape[0] / 8 + 64)
    bound = (p * eps) @ v.abs() + size * peps + size * (
        2 * sums + 2.0 ** -21 + (2.0 ** -11 if f8 else 2.0 ** -16))
    if f8:
        largest = (p * torch.exp2(exps.double())).amax(-1, keepdim=True)
        bound = bound + 2.0 ** -25 * largest * codes.double().abs().sum(0)
    return p @ v, bound, z[:, 0], peps[:, 0] + sums + 2.0 ** -21 + 2.0 ** -22 * z[:, 0].abs()


def _quantise(x):
    top = x.double().abs().amax(-1)
    frac, e = torch.frexp(top)
    e = e - 9 + (frac > 0.875).to(e.dtype)
    codes = torch.ldexp(x.double(), -e[..., None]).float().to(torch.float8_e4m3fn)
    return codes, e


def _rows(n, d, seed, f8):
    g = torch.Generator().manual_seed(seed)
    q = (1.5 * torch.randn(6, d, generator=g)).to(torch.bfloat16)
    k, v = (torch.randn(n, d, generator=g).to(torch.bfloat16) for _ in range(2))
    codes = exps = None
    if f8:
        kc, ke = _quantise(k)
        codes, exps = _quantise(v)
        k = torch.ldexp(kc.double(), ke[:, None])
        v = torch.ldexp(codes.double(), exps[:, None])
    return q, k, v, codes, exps


@pytest.mark.parametrize("n", [3, 40, 700])
@pytest.mark.parametrize("f8", [False, True])
def test_the_bound_sees_a_lost_term(n, f8):
    """(On the CPU.)  The rounding that the header promises stays within the bound, one term less
    does not."""
    q, k, v, codes, exps = _rows(n, 128, n, f8)
    scale = 128 ** -0.5
    out, bound, _, _ = softmax_and_bound(q, k, v, codes, exps, scale, f8)
    s = q.double() @ k.double().T * scale
    p = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
    if f8:
        p2 = p * torch.exp2(exps.double())
        p2 = p2 / p2.amax(-1, keepdim=True) * 256           # as the kernel's first tile has it
        back = (p * torch.exp2(exps.double())).amax(-1, keepdim=True) / 256
        rounded = {11: p2.half().double()}
        one = p2.half()
        first = one.to(torch.float8_e5m2).double()
        second = (one.double() - first).half().to(torch.float8_e5m2).double()
        rounded[6] = first + second
        got = {b: (x * back) @ codes.double() for b, x in rounded.items()}
        kept, lost = got[11], got[6]
    else:
        def cut(x, bits):                                   # truncated to so many significant bits
            step = torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - bits)
            return torch.floor(x / step) * step
        kept, lost = cut(p, 8) + (p - cut(p, 8)).to(torch.bfloat16).double(), cut(p, 8)
        kept, lost = kept @ v.double(), lost @ v.double()
    assert bool(((kept - out).abs() <= bound).all())
    assert not bool(((lost - out).abs() <= bound).all())


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def _dense(c, name, pages, n, head):
    """A sequence's stored vectors of one head, their codes and exponents."""
    at = torch.tensor(pages, dtype=torch.int64, device="cuda")
    raw = c[name].view(torch.uint8)[at, head].view(c[name].dtype).double()
    d = raw.shape[-1]
    if c[name + "_exp"] is None:
        return raw.reshape(-1, d)[:n], None, None
    e = c[name + "_exp"][at, head].long() - 127
    x = torch.ldexp(raw, e[..., None])
    return x.reshape(-1, d)[:n], raw.reshape(-1, d)[:n], e.reshape(-1)[:n]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "f8"])
@pytest.mark.parametrize("b,t,hq,h,d,prefix,lens,page", [
    (1, 1, 8, 1, 128, 1, [1], 16), (3, 1, 8, 2, 128, 0, [2, 5, 9], 16), (2, 2, 12, 2, 256, 3, [2, 30], 32),
    (1, 1, 24, 4, 256, 512, [37], 64), (3, 2, 6, 2, 128, 128, [5, 40, 129], 128),
    (4, 4, 24, 4, 256, 1000, [4, 30, 90, 260], 64), (2, 130, 6, 1, 256, 300, [130, 257], 64),
    (1, 33, 32, 4, 128, 77, [400], 16), (70, 2, 16, 2, 128, 2000, [2 + (i * 13) % 90 for i in range(70)], 64),
    (3, 1, 24, 4, 256, 9000, [40, 7, 300], 32)])
def test_fp32_outputs(gdn, b, t, hq, h, d, prefix, lens, page, fmt):
    from test_gpu_serving import _attend, _attention_case
    case = _attention_case(b, t, hq, h, d, prefix, lens, page, fmt, seed=300 + prefix)
    out, lse = _attend(gdn, case, odt=torch.float32)
    assert gdn.gdn_get_device_error() == 0
    c, f8, group, scale = case["cache"], fmt == "f8", hq // h, d ** -0.5
    worst = 0.0
    for head in range(h):
        hs = slice(head * group, (head + 1) * group)
        pk, pv = (_dense(c, n, case["prefix_pages"], prefix, head) for n in "kv") if prefix else (
            None, None)
        for i, n in enumerate(lens):
            sk, sv = (_dense(c, x, case["pages"][i], n, head) for x in "kv")
            k, v, codes, exps = (
                x if y is None or x is None else torch.cat([y, x]) for x, y in (
                    (sk[0], pk and pk[0]), (sv[0], pv and pv[0]), (sv[1], pv and pv[1]),
                    (sv[2], pv and pv[2])))
            for r in range(t):
                seen = prefix + n - t + 1 + r
                ref, bound, z, zbound = softmax_and_bound(
                    case["q"][i, r, hs], k[:seen], v[:seen], codes[:seen] if f8 else None,
                    exps[:seen] if f8 else None, scale, f8)
                err = (out[i, r, hs].double() - ref).abs()
                assert bool((err <= bound).all()), float((err / bound).max())
                worst = max(worst, float((err / bound).max()))
                assert bool(((lse[i, r, hs].double() - z).abs() <= zbound).all())
    print("worst", worst)
