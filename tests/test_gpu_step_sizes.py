"""The serving step's operators where offsets pass 32 bits, and where a dimension is nothing.
Definitions and tolerances as in test_gpu_qk_norm_rope and test_gpu_verify."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def test_rotation_past_32_bits(gdn):
    """Tokens more than 2^30 elements apart, and a cache of more than 2^31 elements."""
    import test_gpu_qk_norm_rope as t
    n, hq, h, d, page = 4, 6, 2, 256, 64
    apart = (1 << 30) + 1024
    big = torch.empty(3 * apart + 10 * d, dtype=torch.bfloat16, device="cuda")
    rows = big.as_strided((n, hq + 2 * h, d), (apart, d, 1))
    g = t._gen(3)
    for i in range(n):
        rows[i] = t._randn(g, hq + 2 * h, d).to(torch.bfloat16)
    pages = (1 << 31) // (h * page * d) + 40
    cache = [torch.zeros(pages, h, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.tensor([pages * page - 1, 5, (pages - 3) * page, pages * page - 70], device="cuda",
                         dtype=torch.int32)
    positions = torch.tensor([7, 2 ** 31 - 1, 0, 123456], device="cuda", dtype=torch.int32)
    steps, _ = gdn.gdn_rope_phase_steps(64)
    w = 1 + 0.1 * t._randn(g, d)
    q, k, v = rows[:, :hq], rows[:, hq:hq + h], rows[:, hq + h:]
    want_q = t._definition(q, w, 1e-6, positions, steps, 1.0, False)
    want_k = t._definition(k, w, 1e-6, positions, steps, 1.0, False)
    gdn.gdn_qk_norm_rope(q, k, positions, steps, q, q_weight=w, k_weight=w, v=v, k_cache=cache[0],
                         v_cache=cache[1], slots=slots)          # (queries in place)
    t._clean(gdn)
    t._compare(q, *want_q, torch.bfloat16)
    at = (slots.long() // page, slice(None), slots.long() % page)
    t._compare(cache[0][at], *want_k, torch.bfloat16)
    assert torch.equal(cache[1][at], v)
    assert int((cache[0] != 0).any(-1).sum()) == n * h


@pytest.mark.parametrize("drafts", ["logits", "ids"])
def test_verification_past_32_bits(gdn, drafts):
    """Rows and clocks behind more than 2^31 elements: the sequences at the end are as if alone."""
    import test_gpu_verify as t
    b, tokens, v = 90, 2, 8_100_000
    g = t._gen(9)
    last = [0, b - 2, b - 1]
    x = torch.empty(b, tokens + 1, v, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(b, tokens, v, dtype=torch.bfloat16, device="cuda") if drafts == "logits" else None
    clocks = torch.empty(b, v, device="cuda")
    scale = torch.full((b,), -1.0, device="cuda")                # the others are left out
    ids = torch.zeros(b, tokens, dtype=torch.int32, device="cuda")
    for i in last:
        part = 3 * torch.randn(tokens + 1, v, generator=g, device="cuda")
        x[i] = part.to(torch.bfloat16)
        other = part[:tokens] + 0.5 * torch.randn(tokens, v, generator=g, device="cuda")
        if y is not None:
            y[i] = other.to(torch.bfloat16)
        clocks[i].exponential_(generator=g)
        ids[i] = other.argmax(-1).to(torch.int32)
        scale[i] = 1.0
    scale[last[1]] = float("inf")
    u = torch.rand(b, tokens, generator=g, device="cuda")
    c = dict(target=x, draft=y, clocks=clocks, ids=ids, u=u, scale=scale)
    out = t._call(gdn, c)
    t._clean(gdn)
    t._check({n: None if z is None else z[last] for n, z in c.items()},
             {n: z[last] for n, z in out.items()}, close=2)
    assert int((out["accepted"] != -9).sum()) == len(last)


def test_nothing(gdn):
    """No requests, no rows, no columns, no pages; a batch without sequences; tokens without any."""
    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")

    for rows, columns, pages in ((0, 0, 0), (3, 0, 0), (0, 5, 7), (3, 4, 0)):
        pool = dict(table=i32(rows, columns), held=i32(rows), free_pages=i32(pages), free_count=i32(1),
                    page_size=16)
        slots, cu = i32(4), i32(rows + 1)
        gdn.gdn_page_plan(i32(rows), i32(rows), slots, cu_seqlens=cu, **pool)
        gdn.gdn_page_release(i32(rows), **pool)
        assert gdn.gdn_get_device_error() == 0 and slots.tolist() == [-1] * 4
        if rows:                                                # a token, but no page for it
            gdn.gdn_page_plan(i32(rows), i32(rows) + 1, slots, **pool)
            assert gdn.gdn_get_device_error() == 6 and slots.tolist() == [-1] * 4
    empty = torch.empty(0, 3, 50, device="cuda")
    gdn.gdn_verify_tokens(empty, i32(0, 3), i32(0), clocks=torch.empty(0, 50, device="cuda"),
                          draft_ids=i32(0, 2), accept_u=torch.empty(0, 2, device="cuda"))
    q = torch.empty(0, 2, 128, device="cuda")
    gdn.gdn_qk_norm_rope(q, q, i32(0), gdn.gdn_rope_phase_steps(64)[0], q.clone(), q.clone())
    assert gdn.gdn_get_device_error() == 0
