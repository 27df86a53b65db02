"""The full-attention layers' entry points without a GPU: bad arguments are refused on the host
before any CUDA call (the C ABI by status, the binding by exception), empty calls are no-ops.
No call here reaches a launch.
"""
import ctypes

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


BAD_CACHES = [
    (dict(num_pages=-1), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=0), 1),
    (dict(page_size=0), 1), (dict(format=2), 1), (dict(head_dim=64), 2), (dict(page_size=8), 2),
    (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(num_kv_heads=1025), 2), (dict(num_pages=1 << 24, page_size=128), 2),
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=A + 8), 1), (dict(v=A + 2), 1),
    (dict(format=1), 1), (dict(format=1, k_exp=A), 1),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused(L, bad, status):
    c = ctypes.byref(_cache(**bad))
    assert L.gdn_kv_cache_append(c, 4, gdn.GDN_BF16, A, 1024, A, 1024, A, None) == status
    assert L.gdn_kv_cache_read(c, 4, A, gdn.GDN_BF16, A, A, None) == status
    assert L.gdn_prefix_attention(c, 1, 1, 24, A, 24 * 256, A, 64, A, 1, A, 1.0, gdn.GDN_BF16, A,
                                  None, A, 1 << 40, None) == status


@pytest.mark.parametrize("bad", [dict(k_exp=A + 1), dict(v_exp=A + 2), dict(k_exp=A + 3, v_exp=A + 3)])
def test_unaligned_exponents_are_refused(L, bad):
    """The attention reads four exponents at a time."""
    c = ctypes.byref(_cache(**{**dict(format=1, k_exp=A, v_exp=A), **bad}))
    assert L.gdn_kv_cache_append(c, 4, gdn.GDN_BF16, A, 1024, A, 1024, A, None) == 1
    assert L.gdn_kv_cache_read(c, 4, A, gdn.GDN_BF16, A, A, None) == 1
    assert L.gdn_prefix_attention(c, 1, 1, 24, A, 24 * 256, A, 64, A, 1, A, 1.0, gdn.GDN_BF16, A,
                                  None, A, 1 << 40, None) == 1


def test_kv_cache_arguments(L):
    c = ctypes.byref(_cache())

    def append(n=4, dt=gdn.GDN_BF16, k=A, ks=1024, v=A, vs=1024, slots=A, cache=c):
        return L.gdn_kv_cache_append(cache, n, dt, k, ks, v, vs, slots, None)

    assert append(cache=None) == 1
    assert append(n=-1) == 1 and append(dt=5) == 1
    assert append(k=None) == 1 and append(v=A + 8) == 1
    assert append(slots=None) == 1 and append(slots=A + 2) == 1
    assert append(ks=1023) == 1                    # shorter than a token
    assert append(vs=1028) == 1                    # not a multiple of 16 bytes
    assert append(dt=gdn.GDN_F32, ks=1026) == 1
    assert append(n=0, k=None, v=None, slots=None) == 0

    def read(n=4, slots=A, dt=gdn.GDN_BF16, k=A, v=A):
        return L.gdn_kv_cache_read(c, n, slots, dt, k, v, None)

    assert read(n=-2) == 1 and read(dt=-1) == 1
    assert read(k=None) == 1 and read(v=A + 4) == 1 and read(slots=None) == 1
    assert read(n=0, k=None, v=None, slots=None) == 0


def test_attention_arguments(L):
    need = L.gdn_prefix_attention_workspace_size(2, 4, 24, 4, 256)

    def att(b=2, t=4, hq=24, q=A, qs=24 * 256, pp=A, plen=100, pages=A, mp=2, lens=A, scale=1.0,
            dt=gdn.GDN_BF16, out=A, lse=None, ws=A, wsb=need, cache=_cache()):
        return L.gdn_prefix_attention(ctypes.byref(cache), b, t, hq, q, qs, pp, plen, pages, mp,
                                      lens, scale, dt, out, lse, ws, wsb, None)

    assert att(b=-1) == 1 and att(t=-1) == 1 and att(hq=0) == 1
    assert att(hq=23) == 1                         # not a multiple of the key/value heads
    assert att(hq=2048, qs=2048 * 256) == 2
    assert att(b=1 << 15, t=1 << 10) == 2
    assert att(plen=-1) == 1 and att(mp=-1) == 1 and att(scale=float("nan")) == 1
    assert att(dt=9) == 1
    assert att(q=None) == 1 and att(q=A + 8) == 1 and att(out=None) == 1 and att(out=A + 8) == 1
    assert att(qs=24 * 256 - 8) == 1 and att(qs=24 * 256 + 4) == 1
    assert att(pp=None) == 1 and att(pages=None) == 1 and att(lens=None) == 1
    assert att(lens=A + 1) == 1 and att(lse=A + 2) == 1
    assert att(cache=_cache(num_pages=0, k=None, v=None)) == 1     # pages of an empty cache
    assert att(mp=1 << 26) == 2                    # token counts past 32 bits
    if need:
        assert att(ws=None) == 3 and att(wsb=need - 1) == 3 and att(ws=A + 4) == 3
    assert att(b=0, q=None, out=None) == 0 and att(t=0, q=None, out=None) == 0
    # sizes without a workspace
    assert L.gdn_prefix_attention_workspace_size(0, 4, 24, 4, 256) == 0
    assert L.gdn_prefix_attention_workspace_size(2, 4, 23, 4, 256) == 0
    assert L.gdn_prefix_attention_workspace_size(2, 4, 24, 4, 64) == 0


def test_logprobs_arguments(L):
    def lp(n=3, v=1000, dt=gdn.GDN_BF16, x=A, stride=1000, tg=A, scale=1.0, lp_=A, ent=A, k=5,
           ids=A, tl=A, ws=A, wsb=1 << 40):
        return L.gdn_token_logprobs(n, v, dt, x, stride, tg, scale, lp_, ent, k, ids, tl, ws, wsb,
                                    None)

    assert lp(n=-1) == 1 and lp(v=0) == 1 and lp(dt=3) == 1 and lp(k=-1) == 1
    assert lp(v=4, k=5) == 1 and lp(k=33) == 2
    assert lp(scale=0.0) == 1 and lp(scale=-1.0) == 1 and lp(scale=float("inf")) == 1
    assert lp(stride=999) == 1
    assert lp(x=None) == 1 and lp(x=A + 1) == 1 and lp(dt=gdn.GDN_F32, x=A + 2) == 1
    assert lp(tg=None) == 1 and lp(lp_=None) == 1
    assert lp(ids=None) == 1 and lp(tl=None) == 1
    assert lp(ent=A + 2) == 1 and lp(ids=A + 1) == 1
    need = L.gdn_token_logprobs_workspace_size(3, 1000, gdn.GDN_BF16, 5)
    if need:
        assert lp(ws=None) == 3 and lp(wsb=need - 1) == 3
    assert lp(n=0, x=None, tg=None, lp_=None) == 0
    assert L.gdn_token_logprobs_workspace_size(3, 1000, gdn.GDN_BF16, 33) == 0


def test_binding_refuses_host_tensors_and_bad_types(L):
    k = torch.zeros(2, 4, 16, 128, dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_kv_cache_append(x, x, k, k, slots)
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_kv_cache_read(k, k, slots, x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_prefix_attention(x[None], k, k, x[None], pages=slots[None], kv_len=slots[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_token_logprobs(torch.zeros(2, 9), slots, torch.zeros(2))


def test_token_strides(L):
    """One token stride for slices of wider rows; anything else is refused."""
    dev, bf = torch.device("cpu"), torch.bfloat16
    wide = torch.zeros(2, 3, 40, 128, dtype=bf)
    f = lambda t, shape: gdn._token_stride(t, "q", shape, bf, dev)  # noqa: E731
    assert f(wide[:, :, 8:32], (2, 3, 24, 128)) == 40 * 128
    assert f(wide[:1, :, 8:32], (1, 3, 24, 128)) == 40 * 128
    assert f(wide[:, :1, :24], (2, 1, 24, 128)) == 3 * 40 * 128
    assert f(wide[0, 0][None, None], (1, 1, 40, 128)) == 40 * 128
    for bad in (wide[:, :2], wide.transpose(0, 1), wide.transpose(2, 3), wide[..., ::2],
                wide[:, :, ::2]):
        with pytest.raises(ValueError):
            f(bad, tuple(bad.shape))
    with pytest.raises(TypeError):
        f(wide.float(), tuple(wide.shape))
