"""One verification step of a hybrid model's layers for a batch that shares a prompt prefix.

A batch of requests has drafted T tokens each on top of a common prefix.  The step runs what the
two kinds of layer of a hybrid Gated DeltaNet model need, each through the library:

  * recurrent layer: ``gdn_decode_multi`` over the T tokens, keeping the state after every token;
  * full-attention layer: ``gdn_kv_cache_append`` writes the new keys and values (8-bit codes),
    ``gdn_prefix_attention`` attends to the shared prefix and to the sequences' own tokens;
  * the head: ``gdn_token_logprobs`` scores the drafted tokens under the step's logits and gives
    the alternatives; the accepted tokens decide which recurrent snapshot
    ``gdn_state_checkpoint`` restores and how far the cache's lengths go.

Weights and activations are random: the projections around the layers are plain matrix products.

    python examples/hybrid_verify.py [--batch 8] [--tokens 4] [--prefix 2000] [--vocab 32000]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_13_gb300 as gdn  # noqa: E402

D_REC, HK, HV, WIDTH = 128, 4, 8, 4          # recurrent layer
D_ATT, HQ, HKV, PAGE = 256, 12, 2, 64        # attention layer: 12 query heads on 2 key/value heads


def _rand(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def run(batch=8, tokens=4, prefix=2000, own=50, vocab=32000, top_k=5, seed=0):
    """Returns the step's tensors by name (see main for their use)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, i32 = "cuda", torch.int32
    channels = (2 * HK + HV) * D_REC
    # ---- the state of the batch before the step
    state = 0.1 * torch.randn(batch, HV, D_REC, D_REC, generator=g, device=dev)
    conv_state = _rand(g, batch, WIDTH - 1, channels)
    snaps = torch.zeros(batch * tokens, HV, D_REC, D_REC, device=dev)
    conv_snaps = torch.zeros(batch * tokens, WIDTH - 1, channels, dtype=torch.bfloat16, device=dev)
    shared, each = -(-prefix // PAGE), -(-(own + tokens) // PAGE)
    pages = shared + batch * each
    cache = {n: torch.zeros(pages, HKV, PAGE, D_ATT, dtype=torch.uint8, device=dev).view(
        torch.float8_e4m3fn) for n in ("k", "v")}
    exps = {n + "_exp": torch.full((pages, HKV, PAGE), 127, dtype=torch.uint8, device=dev)
            for n in ("k", "v")}
    prefix_pages = torch.arange(shared, dtype=i32, device=dev)
    own_pages = (shared + torch.arange(batch * each, dtype=i32, device=dev)).reshape(batch, each)

    def slots(first, count):                 # of tokens first .. of every sequence's own
        t = first + torch.arange(count, device=dev)
        return (own_pages[:, t // PAGE] * PAGE + t % PAGE).to(i32).reshape(-1)

    # the shared prefix's keys and values once, the sequences' own tokens so far
    gdn.gdn_kv_cache_append(_rand(g, prefix, HKV, D_ATT), _rand(g, prefix, HKV, D_ATT),
                            cache["k"], cache["v"], torch.arange(prefix, dtype=i32, device=dev),
                            **exps)
    gdn.gdn_kv_cache_append(_rand(g, batch * own, HKV, D_ATT), _rand(g, batch * own, HKV, D_ATT),
                            cache["k"], cache["v"], slots(0, own), **exps)

    # ---- recurrent layer over the drafted tokens, the state kept after each
    x = _rand(g, batch, tokens, channels)
    a, b = _rand(g, batch, tokens, HV), _rand(g, batch, tokens, HV)
    A_log = torch.rand(HV, generator=g, device=dev)
    conv_weight = _rand(g, channels, WIDTH, scale=0.5)
    rec = torch.empty(batch, tokens, HV, D_REC, dtype=torch.bfloat16, device=dev)
    gdn.gdn_decode_multi(
        x, None, None, a, b, A_log, None, state, rec, num_k_heads=HK, conv_weight=conv_weight,
        conv_state=conv_state, snap_state=snaps, snap_conv_state=conv_snaps,
        snap_slots=torch.arange(batch * tokens, dtype=i32, device=dev).reshape(batch, tokens))

    # ---- attention layer: one projection's rows hold queries, keys and values side by side
    w_qkv = _rand(g, HV * D_REC, (HQ + 2 * HKV) * D_ATT, scale=0.02)
    qkv = (rec.reshape(batch * tokens, -1) @ w_qkv).reshape(batch, tokens, -1, D_ATT)
    q, k, v = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HKV], qkv[:, :, HQ + HKV:]
    flat = qkv.reshape(batch * tokens, -1, D_ATT)
    gdn.gdn_kv_cache_append(flat[:, HQ:HQ + HKV], flat[:, HQ + HKV:], cache["k"], cache["v"],
                            slots(own, tokens), **exps)
    kv_len = torch.full((batch,), own + tokens, dtype=i32, device=dev)
    att = torch.empty(batch, tokens, HQ, D_ATT, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(batch, tokens, HQ, device=dev)
    gdn.gdn_prefix_attention(q, cache["k"], cache["v"], att, prefix_pages=prefix_pages,
                             prefix_len=prefix, pages=own_pages, kv_len=kv_len, lse=lse, **exps)

    # ---- the head: scores of the drafted tokens, their alternatives
    logits = att.reshape(batch * tokens, -1) @ _rand(g, HQ * D_ATT, vocab, scale=0.3)
    draft = torch.randint(0, vocab, (batch * tokens,), generator=g, device=dev, dtype=i32)
    draft[::2] = logits.float().argmax(-1).to(i32)[::2]          # some good drafts
    logp, entropy = (torch.empty(batch * tokens, device=dev) for _ in range(2))
    top_ids = torch.empty(batch * tokens, top_k, dtype=i32, device=dev)
    top_logp = torch.empty(batch * tokens, top_k, device=dev)
    gdn.gdn_token_logprobs(logits, draft, logp, entropy, top_ids=top_ids, top_logprobs=top_logp)

    # ---- accept each sequence's leading drafts that are the most likely token; the recurrent
    # state goes back to the last accepted one (at least one token is kept), the lengths too
    good = (draft == top_ids[:, 0]).reshape(batch, tokens).long().cumprod(1).sum(1).clamp(min=1)
    rows = torch.arange(batch, dtype=i32, device=dev)
    gdn.gdn_state_checkpoint("restore", state, conv_state, snaps, conv_snaps, rows,
                             (rows * tokens + good.to(i32) - 1).to(i32), num_k_heads=HK)
    kv_len = (kv_len - tokens + good).to(i32)
    return dict(q=q, k=k, v=v, cache=cache, exps=exps, prefix_pages=prefix_pages,
                own_pages=own_pages, prefix=prefix, attention=att, lse=lse, logits=logits,
                draft=draft, logprobs=logp, entropy=entropy, top_ids=top_ids, accepted=good,
                state=state, snaps=snaps, kv_len=kv_len, own=own)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 8), ("tokens", 4), ("prefix", 2000), ("vocab", 32000)):
        p.add_argument("--" + name, type=int, default=value)
    o = run(**vars(p.parse_args()))
    status = gdn.gdn_get_device_error()
    if status:
        sys.exit(gdn.gdn_status_string(status))
    print("accepted tokens:", o["accepted"].tolist())
    print("mean log probability of the drafts: %.3f, mean entropy %.3f nats"
          % (float(o["logprobs"].mean()), float(o["entropy"].mean())))


if __name__ == "__main__":
    main()
