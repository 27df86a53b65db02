"""The binding's native part: usual calls go through it, everything else through the checks in
Python, with the same results."""
import pytest
import torch

import gated_deltanet_linear_13_gb300 as gdn
from gated_deltanet_linear_13_gb300 import build_lib


def _native():
    build_lib.build()
    gdn.load_library()
    return gdn._native


def test_what_is_unusual_is_left_to_the_binding():
    m = _native()
    q = torch.zeros(2, 4, 128)
    for args in ((), (1, 2), (q,) * 18, (None,) * 18, ("q",) * 18):
        assert m.qk_norm_rope(*args) is None
    for args in ((), (None,) * 15, (q,) * 15):
        assert m.page_plan(*args) is None
    for args in ((), (None,) * 8, (q,) * 8):
        assert m.page_release(*args) is None
    for args in ((), (None,) * 11, (q,) * 11):
        assert m.verify_tokens(*args) is None
    with pytest.raises(TypeError):
        m.bind(1, 2)
    with pytest.raises(TypeError):
        m.bind("a", "b", "c", "d", None)


class _Counted:
    """A function of the native part that counts its answers, or (off) always answers None."""

    def __init__(self, f, off):
        self.f, self.off, self.answers = f, off, 0

    def __call__(self, *args):
        st = None if self.off else self.f(*args)
        self.answers += st is not None
        return st


class _Part:
    def __init__(self, native, off):
        self.calls = {n: _Counted(getattr(native, n), off)
                      for n in ("qk_norm_rope", "page_plan", "page_release", "verify_tokens")}
        self.__dict__.update(self.calls)


@pytest.mark.gpu
def test_both_ways_give_the_same(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    native = _native()
    results = []
    for off in (False, True):
        part = _Part(native, off)
        monkeypatch.setattr(gdn, "_native", part)
        results.append(_run_all())
        if not off:
            assert {n: c.answers for n, c in part.calls.items()} == dict(
                qk_norm_rope=16, page_plan=2, page_release=1, verify_tokens=4)
    assert gdn.gdn_get_device_error() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)


def _run_all():
    g = torch.Generator(device="cuda").manual_seed(3)
    out = []

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def i32(x):
        return torch.tensor(x, device="cuda", dtype=torch.int32)

    side = torch.cuda.Stream()
    # norm and rotation: strided and dense, one token, with and without each part
    steps, _ = gdn.gdn_rope_phase_steps(64)
    w = randn(128)
    for n in (1, 5):
        for dtype in (torch.bfloat16, torch.float32):
            rows = randn(n, 10, 128).to(dtype)
            p = torch.arange(n, device="cuda", dtype=torch.int32)
            for fmt in (None, torch.bfloat16, torch.float8_e4m3fn, "plain"):
                c = {}
                if isinstance(fmt, torch.dtype):
                    def cache(shape, dt):
                        return torch.zeros(shape, device="cuda", dtype=torch.uint8).view(dt)
                    width = 128 * (2 if fmt is torch.bfloat16 else 1)
                    c = dict(v=rows[:, 8:], slots=p,
                             k_cache=cache((1, 2, 16, width), fmt), v_cache=cache((1, 2, 16, width), fmt))
                    if fmt is torch.float8_e4m3fn:
                        c |= dict(k_exp=cache((1, 2, 16), torch.uint8), v_exp=cache((1, 2, 16), torch.uint8))
                q_out = torch.zeros(n, 3, 128, device="cuda", dtype=dtype)
                k_out = torch.zeros(n, 2, 128, device="cuda", dtype=dtype)
                torch.cuda.synchronize()
                gdn.gdn_qk_norm_rope(rows[:, :6:2], rows[:, 6:8], None if fmt == "plain" else p,
                                     None if fmt == "plain" else steps, q_out,
                                     k_out if fmt in (None, "plain") else None,
                                     q_weight=w, k_weight=None if fmt == "plain" else w,
                                     interleaved=n == 1, amplitude=1.5,
                                     stream=side if n == 1 else side.cuda_stream, **c)
                torch.cuda.synchronize()
                out += [q_out, k_out] + [c[x].view(torch.uint8) for x in ("k_cache", "v_cache", "k_exp",
                                                                         "v_exp") if x in c]
    # pages
    pool = dict(table=i32([[0] * 4] * 3), held=i32([0] * 3), free_pages=i32(list(range(12))),
                free_count=i32([12]), page_size=16)
    slots, positions, cu = i32([0] * 60), i32([0] * 60), i32([0] * 4)
    after, pages = i32([0] * 3), i32([[0] * 4] * 3)
    gdn.gdn_page_plan(i32([0, 0, 0]), i32([20, 5, 33]), slots, positions, cu, after, pages,
                      rows=i32([2, -1, 0]), position_offset=7, **pool)
    gdn.gdn_page_plan(i32([0]), i32([3]), **pool)
    gdn.gdn_page_release(i32([2, 3, 17]), **pool, stream=torch.cuda.current_stream())
    out += [slots, positions, cu, after, pages, *(x for x in pool.values() if torch.is_tensor(x))]
    # verification: with drafts, strided rows, without drafts, one sequence
    for b, t, wide in ((3, 2, 0), (3, 2, 5), (1, 1, 3), (4, 0, 0)):
        x, y = (randn(b, t + k, 700 + wide)[..., :700] for k in (1, 0))
        tokens = torch.zeros(b, t + 1, device="cuda", dtype=torch.int32)
        accepted, lp = torch.zeros(b, device="cuda", dtype=torch.int32), torch.zeros(b, t + 1, device="cuda")
        kw = {}
        if t:
            kw = dict(draft_ids=torch.randint(0, 700, (b, t), generator=g, device="cuda", dtype=torch.int32),
                      draft_logits=y, accept_u=torch.rand(b, t, generator=g, device="cuda"))
        ws = torch.empty(gdn.gdn_verify_tokens_workspace_size(b, t, 700, torch.float32, bool(t)),
                         dtype=torch.uint8, device="cuda")
        gdn.gdn_verify_tokens(x, tokens, accepted, logprobs=lp, workspace=ws,
                              clocks=torch.empty(b, 700, device="cuda").exponential_(generator=g), **kw)
        out += [tokens, accepted, lp]
    torch.cuda.synchronize()
    return out
