"""The speculative decoding example end to end: its steps against plain torch on the tensors that
they leave, the captured step against the plain one, and the cache after many steps.

Tolerances: keys in the cache as in test_gpu_qk_norm_rope; the attention against a 64-bit softmax
over what the cache stands for, 2^-7 of the row's sum of p |v| (test_gpu_serving); decisions and log
probabilities as in test_gpu_verify; pages, slots and states are equal.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.join(os.path.dirname(HERE), "examples"))


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_deltanet_linear_13_gb300 as m
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    m.load_library()
    return m


def _stored(s, name, pages):
    """What pages of the cache stand for, in 64 bits: [heads, tokens, elements]."""
    cache, exps = (s.k_cache, s.exps["k_exp"]) if name == "k" else (s.v_cache, s.exps["v_exp"])
    x = cache.view(torch.uint8)[pages.long()].view(torch.float8_e4m3fn).double()
    x = x * torch.exp2(exps[pages.long()].double() - 127)[..., None]
    return x.movedim(1, 0).reshape(x.shape[1], -1, x.shape[-1])


@pytest.mark.parametrize("batch,drafts,prefix", [(5, 3, 700), (1, 1, 16), (9, 6, 33)])
def test_steps(gdn, batch, drafts, prefix):
    import hybrid_serve as ex
    import test_gpu_qk_norm_rope as rope
    import test_gpu_verify as verify
    n, steps = drafts + 1, 6
    s = ex.Server(batch, drafts, prefix, vocab=1000, longest=n * (steps + 1))
    history = [[] for _ in range(batch)]                  # keys and values of each kept token
    for _ in range(steps):
        kv = s.kv_len.tolist()
        state = s.state.clone()
        s.random_numbers()
        s.step()
        assert gdn.gdn_get_device_error() == 0
        assert not torch.equal(s.state, state)
        # ---- slots and positions: the block tables' pages, one token after the other
        pages, after = s.pages.long(), s.kv_after.tolist()
        assert after == [k + n for k in kv]
        at = torch.tensor(kv, device="cuda")[:, None] + torch.arange(n, device="cuda")
        page = pages.gather(1, at // ex.PAGE)
        assert torch.equal(s.slots.long().reshape(batch, n), page * ex.PAGE + at % ex.PAGE)
        assert torch.equal(s.positions.long().reshape(batch, n), prefix + at)
        used = [p for i in range(batch) for p in pages[i, :-(-after[i] // ex.PAGE)].tolist()]
        assert len(set(used)) == len(used)
        # ---- queries, and keys and values in the cache
        qkv = s.qkv
        want, bound = rope._definition(qkv[:, :ex.HQ], s.q_weight, 1e-6, s.positions, s.phase_steps,
                                       s.amplitude, False)
        rope._compare(s.q.reshape(want.shape), want, bound, torch.bfloat16)
        key = rope._definition(qkv[:, ex.HQ:ex.HQ + ex.HKV], s.k_weight, 1e-6, s.positions,
                               s.phase_steps, s.amplitude, False)
        where = (s.slots.long() // ex.PAGE, slice(None), s.slots.long() % ex.PAGE)
        rope._compare_f8(s.k_cache.view(torch.uint8)[where].view(torch.float8_e4m3fn),
                         s.exps["k_exp"][where], *key)
        # ---- attention
        group = ex.HQ // ex.HKV
        for i in range(batch):
            k, v = (torch.cat([_stored(s, x, s.prefix_pages)[:, :prefix],
                               _stored(s, x, pages[i])[:, :after[i]]], 1) for x in ("k", "v"))
            q = s.q[i].double().reshape(n, ex.HKV, group, ex.D_ATT)
            score = torch.einsum("thgd,hnd->thgn", q, k) * ex.D_ATT ** -0.5
            last = prefix + kv[i] + torch.arange(n, device="cuda")
            hidden = torch.arange(k.shape[1], device="cuda") > last[:, None]
            p = torch.softmax(score.masked_fill(hidden[:, None, None], -float("inf")), -1)
            ref = torch.einsum("thgn,hnd->thgd", p, v).reshape(n, ex.HQ, ex.D_ATT)
            size = torch.einsum("thgn,hnd->thgd", p, v.abs()).reshape(n, ex.HQ, ex.D_ATT)
            assert bool(((s.att[i].double() - ref).abs() <= 2.0 ** -7 * size + 1e-6).all())
        # ---- decisions
        verify._check(dict(target=s.logits, draft=s.draft_logits, ids=s.draft_ids, u=s.accept_u,
                           clocks=s.clocks[:, 0], scale=s.scale),
                      dict(tokens=s.tokens, accepted=s.accepted, logprobs=s.logprobs), close=1)
        # ---- back to the last accepted token
        taken = s.accepted.tolist()
        assert s.kv_len.tolist() == [k + 1 + a for k, a in zip(kv, taken)]
        row = torch.arange(batch, device="cuda") * n + s.accepted.long()
        assert torch.equal(s.state, s.snaps[row]) and torch.equal(s.conv_state, s.conv_snaps[row])
        assert s.last.tolist() == [int(s.tokens[i, a]) for i, a in enumerate(taken)]
        held = [-(-k // ex.PAGE) for k in s.kv_len.tolist()]
        assert s.pool["held"].tolist() == held
        assert int(s.pool["free_count"]) == s.pool["free_pages"].numel() - sum(held)
        free = s.pool["free_pages"][:int(s.pool["free_count"])].tolist()
        mine = [p for i in range(batch) for p in s.pool["table"][i, :held[i]].tolist()]
        assert sorted(free + mine) == list(range(s.pool["free_pages"].numel()))
        for i, a in enumerate(taken):
            history[i] += [[_stored(s, x, pages[i])[:, kv[i] + j].clone() for x in ("k", "v")]
                           for j in range(1 + a)]
    # every kept token's key and value are where the tables say
    for i in range(batch):
        for name, at in (("k", 0), ("v", 1)):
            now = _stored(s, name, s.pool["table"][i])
            for t, kept in enumerate(history[i]):
                assert torch.equal(now[:, t], kept[at])


def test_captured_steps(gdn):
    """Replays of one captured step give what plain steps give, bit for bit."""
    import hybrid_serve as ex
    plain, captured = (ex.Server(6, 3, 100, vocab=2000, longest=60, seed=4) for _ in range(2))
    graph = captured.capture()
    plain.random_numbers()                                # (as the capture did)
    for _ in range(8):
        for s in (plain, captured):
            s.random_numbers()
        plain.step()
        graph.replay()
        for name in ("tokens", "accepted", "kv_len", "last", "slots", "state"):
            assert torch.equal(getattr(plain, name), getattr(captured, name)), name
    for name in ("table", "held", "free_pages", "free_count"):
        assert torch.equal(plain.pool[name], captured.pool[name])
    assert gdn.gdn_get_device_error() == 0
