"""The hybrid verification example end to end: its parts against plain torch on the tensors that
it returns.  Tolerances: as the operators' own tests (the attention against a 64-bit softmax over
what the cache stands for, 2^-7 of the row's sum of p |v|; log probabilities 1e-4)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("batch,tokens,prefix,own", [(5, 4, 700, 50), (1, 1, 65, 0), (3, 7, 1, 130)])
def test_hybrid_verify(batch, tokens, prefix, own):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_13_gb300 import build_lib
    build_lib.build()
    import gated_deltanet_linear_13_gb300 as gdn
    import hybrid_verify as ex
    o = ex.run(batch=batch, tokens=tokens, prefix=prefix, own=own, vocab=5000)
    assert gdn.gdn_get_device_error() == 0

    def stored(n, pages, count):             # what the cache stands for, in 64 bits
        x = o["cache"][n].view(torch.uint8)[pages.long()].view(torch.float8_e4m3fn).double()
        x = x * torch.exp2(o["exps"][n + "_exp"][pages.long()].double() - 127)[..., None]
        return x.movedim(1, 0).reshape(x.shape[1], -1, x.shape[-1])[:, :count]

    group = ex.HQ // ex.HKV
    for i in range(batch):
        k, v = (torch.cat([stored(n, o["prefix_pages"], prefix),
                           stored(n, o["own_pages"][i], own + tokens)], 1) for n in ("k", "v"))
        q = o["q"][i].double().reshape(tokens, ex.HKV, group, ex.D_ATT)
        s = torch.einsum("thgd,hnd->thgn", q, k) * ex.D_ATT ** -0.5
        last = prefix + own + torch.arange(tokens, device="cuda")
        s = s.masked_fill((torch.arange(k.shape[1], device="cuda") > last[:, None])[:, None, None],
                          -float("inf"))
        p = torch.softmax(s, -1)
        ref = torch.einsum("thgn,hnd->thgd", p, v).reshape(tokens, ex.HQ, ex.D_ATT)
        size = torch.einsum("thgn,hnd->thgd", p, v.abs()).reshape(tokens, ex.HQ, ex.D_ATT)
        assert bool(((o["attention"][i].double() - ref).abs() <= 2.0 ** -7 * size + 1e-6).all())
    logp = torch.log_softmax(o["logits"].double(), -1)
    want = logp.gather(1, o["draft"].long()[:, None])[:, 0]
    assert float((o["logprobs"].double() - want).abs().max()) <= 1e-4
    assert float((o["entropy"].double() + (logp.exp() * logp).sum(-1)).abs().max()) <= 1e-4
    order = torch.sort(o["logits"], dim=-1, descending=True, stable=True).indices
    assert torch.equal(o["top_ids"].long(), order[:, :5])
    # the recurrent state is the snapshot after the last accepted token
    kept = torch.arange(batch, device="cuda") * tokens + o["accepted"] - 1
    assert torch.equal(o["state"], o["snaps"][kept])
    assert torch.equal(o["kv_len"].long(), own + o["accepted"])
