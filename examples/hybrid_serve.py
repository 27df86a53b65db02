"""Speculative decoding with a hybrid model's layers: steps that need nothing from the host.

A batch of requests continues a shared prompt prefix.  Every step drafts T tokens, runs the target
model's layers over the last token and the drafts, accepts what the target's probabilities allow,
draws the next token, and takes back what was refused.  The parts that are not plain matrix
products go through the library:

  * ``gdn_page_plan``: pages, slots, positions and block tables of the step's tokens;
  * recurrent layer: ``gdn_decode_multi``, keeping the state after every token;
  * full-attention layer: ``gdn_qk_norm_rope`` normalises and rotates queries and keys and writes
    keys and values to their slots, ``gdn_prefix_attention`` attends to prefix and own tokens;
  * the head: ``gdn_verify_tokens`` accepts drafts and draws the next token;
  * taking back: ``gdn_state_checkpoint`` restores the recurrent state after the last accepted
    token, ``gdn_page_release`` gives back the pages behind it.

Lengths, pages, tokens and random numbers stay on the device, so one captured step is replayed for
all of them.  Weights are random, and so is the drafting model.

    python examples/hybrid_serve.py [--batch 8] [--drafts 3] [--prefix 2000] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_13_gb300 as gdn  # noqa: E402

D_REC, HK, HV, WIDTH = 128, 2, 4, 4          # recurrent layer
D_ATT, HQ, HKV, PAGE = 128, 8, 2, 16         # attention layer: 8 query heads on 2 key/value heads
ROTARY, BASE = 64, 1e6                       # half of each head is rotated
HIDDEN = 256
I32, BF16 = torch.int32, torch.bfloat16


class Server:
    """The weights, the device state and one step of the batch."""

    def __init__(self, batch=8, drafts=3, prefix=2000, vocab=4096, longest=400, seed=0):
        self.batch, self.drafts, self.prefix, self.vocab = batch, drafts, prefix, vocab
        g = self.generator = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, scale=1.0, dtype=BF16):
            return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)

        channels, n = (2 * HK + HV) * D_REC, drafts + 1
        # ---- weights
        self.embedding = rand(vocab, HIDDEN)
        self.w_in = rand(HIDDEN, channels + 2 * HV, scale=HIDDEN ** -0.5)
        self.a_log = torch.rand(HV, generator=g, device="cuda")
        self.conv_weight = rand(channels, WIDTH, scale=0.5)
        self.w_qkv = rand(HV * D_REC, (HQ + 2 * HKV) * D_ATT, scale=0.05)
        self.q_weight, self.k_weight = (1 + rand(D_ATT, scale=0.1, dtype=torch.float32)
                                        for _ in range(2))
        self.w_out = rand(HQ * D_ATT, vocab, scale=0.2)
        self.w_draft = rand(HIDDEN, vocab, scale=0.1)
        self.phase_steps, self.amplitude = gdn.gdn_rope_phase_steps(ROTARY, BASE)
        # ---- recurrent state, and a slot for the state after every token of a step
        self.state = rand(batch, HV, D_REC, D_REC, scale=0.1, dtype=torch.float32)
        self.conv_state = rand(batch, WIDTH - 1, channels)
        self.snaps = torch.zeros(batch * n, HV, D_REC, D_REC, device="cuda")
        self.conv_snaps = torch.zeros(batch * n, WIDTH - 1, channels, dtype=BF16, device="cuda")
        self.rows = torch.arange(batch, dtype=I32, device="cuda")
        self.snap_slots = torch.arange(batch * n, dtype=I32, device="cuda").reshape(batch, n)
        # ---- the paged cache: the prefix's pages, then a pool for the requests' own tokens
        shared, columns = -(-prefix // PAGE), -(-longest // PAGE)
        own = batch * columns
        shape = (shared + own, HKV, PAGE, D_ATT)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(
            torch.float8_e4m3fn) for _ in range(2))
        self.exps = {x: torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda")
                     for x in ("k_exp", "v_exp")}
        self.prefix_pages = own + torch.arange(shared, dtype=I32, device="cuda")
        self.pool = dict(table=torch.zeros(batch, columns, dtype=I32, device="cuda"),
                         held=torch.zeros(batch, dtype=I32, device="cuda"),
                         free_pages=torch.randperm(own, generator=g, device="cuda").to(I32),
                         free_count=torch.tensor([own], dtype=I32, device="cuda"), page_size=PAGE)
        x = rand(prefix, HQ + 2 * HKV, D_ATT)
        at = torch.arange(prefix, dtype=I32, device="cuda")
        gdn.gdn_qk_norm_rope(
            x[:, :HQ], x[:, HQ:HQ + HKV], at, self.phase_steps, torch.empty_like(x[:, :HQ].contiguous()),
            q_weight=self.q_weight, k_weight=self.k_weight, amplitude=self.amplitude,
            v=x[:, HQ + HKV:], k_cache=self.k_cache, v_cache=self.v_cache, slots=at + own * PAGE,
            **self.exps)
        # ---- what a step reads and writes
        self.kv_len = torch.zeros(batch, dtype=I32, device="cuda")
        self.kv_after, self.accepted = torch.empty_like(self.kv_len), torch.empty_like(self.kv_len)
        self.new_len = torch.full((batch,), n, dtype=I32, device="cuda")
        self.last = torch.randint(0, vocab, (batch,), generator=g, device="cuda", dtype=I32)
        self.slots, self.positions = (torch.empty(batch * n, dtype=I32, device="cuda")
                                      for _ in range(2))
        self.pages = torch.zeros(batch, columns, dtype=I32, device="cuda")
        self.draft_ids = torch.empty(batch, drafts, dtype=I32, device="cuda")
        self.draft_logits = torch.empty(batch, drafts, vocab, dtype=BF16, device="cuda")
        self.rec = torch.empty(batch, n, HV, D_REC, dtype=BF16, device="cuda")
        self.q = torch.empty(batch, n, HQ, D_ATT, dtype=BF16, device="cuda")
        self.att, self.lse = torch.empty_like(self.q), torch.empty(batch, n, HQ, device="cuda")
        self.tokens = torch.empty(batch, n, dtype=I32, device="cuda")
        self.logprobs = torch.empty(batch, n, device="cuda")
        self.scale = torch.full((batch,), 1.25, device="cuda")
        self.scale[::4] = float("inf")                    # every fourth request is greedy
        self.clocks, self.draft_clocks = (torch.empty(batch, k, vocab, device="cuda")
                                          for k in (1, drafts))
        self.accept_u = torch.empty(batch, drafts, device="cuda")

    def random_numbers(self):
        """The next step's."""
        self.clocks.exponential_(generator=self.generator)
        self.draft_clocks.exponential_(generator=self.generator)
        self.accept_u.uniform_(generator=self.generator)

    def step(self):
        b, n = self.batch, self.drafts + 1
        # ---- the drafting model: each token's logits from the one before
        token = self.last
        for i in range(self.drafts):
            logits = self.embedding[token.long()] @ self.w_draft
            self.draft_logits[:, i] = logits
            scaled = logits.float() * self.scale.clamp(max=100.0)[:, None]
            token = (scaled - self.draft_clocks[:, i].log()).argmax(-1).to(I32)
            self.draft_ids[:, i] = token
        # ---- pages, slots and positions of the last token and the drafts
        gdn.gdn_page_plan(self.kv_len, self.new_len, self.slots, self.positions,
                          kv_len_out=self.kv_after, pages=self.pages,
                          position_offset=self.prefix, **self.pool)
        # ---- recurrent layer
        inputs = torch.cat([self.last[:, None], self.draft_ids], 1).long()
        x = self.embedding[inputs] @ self.w_in
        channels = x.shape[-1] - 2 * HV
        gdn.gdn_decode_multi(
            x[..., :channels].contiguous(), None, None, x[..., channels:channels + HV].contiguous(),
            x[..., channels + HV:].contiguous(), self.a_log, None, self.state, self.rec,
            num_k_heads=HK, conv_weight=self.conv_weight, conv_state=self.conv_state,
            snap_state=self.snaps, snap_conv_state=self.conv_snaps, snap_slots=self.snap_slots)
        # ---- attention layer: one projection's rows hold queries, keys and values
        qkv = self.qkv = (self.rec.reshape(b * n, -1) @ self.w_qkv).reshape(b * n, -1, D_ATT)
        gdn.gdn_qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], self.positions, self.phase_steps,
                             self.q.view(b * n, HQ, D_ATT), q_weight=self.q_weight,
                             k_weight=self.k_weight, amplitude=self.amplitude,
                             v=qkv[:, HQ + HKV:], k_cache=self.k_cache, v_cache=self.v_cache,
                             slots=self.slots, **self.exps)
        gdn.gdn_prefix_attention(self.q, self.k_cache, self.v_cache, self.att,
                                 prefix_pages=self.prefix_pages, prefix_len=self.prefix,
                                 pages=self.pages, kv_len=self.kv_after, lse=self.lse, **self.exps)
        # ---- the head: accept drafts, draw the next token
        self.logits = (self.att.reshape(b * n, -1) @ self.w_out).reshape(b, n, -1)
        gdn.gdn_verify_tokens(self.logits, self.tokens, self.accepted, clocks=self.clocks[:, 0],
                              draft_ids=self.draft_ids, draft_logits=self.draft_logits,
                              accept_u=self.accept_u, scale=self.scale, logprobs=self.logprobs)
        # ---- back to the last accepted token: recurrent state, length, pages
        gdn.gdn_state_checkpoint("restore", self.state, self.conv_state, self.snaps,
                                 self.conv_snaps, self.rows, self.rows * n + self.accepted,
                                 num_k_heads=HK)
        self.kv_len += 1 + self.accepted
        gdn.gdn_page_release(self.kv_len, **self.pool)
        self.last.copy_(self.tokens.gather(1, self.accepted.long()[:, None])[:, 0])

    def capture(self):
        """One step as a graph; what it changes is put back as it was."""
        held = [self.state, self.conv_state, self.kv_len, self.last, self.k_cache.view(torch.uint8),
                self.v_cache.view(torch.uint8), *self.exps.values(),
                *(x for x in self.pool.values() if isinstance(x, torch.Tensor))]
        before = [x.clone() for x in held]
        self.random_numbers()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()                                   # (library handles are made outside)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        for x, y in zip(held, before):
            x.copy_(y)
        return graph


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 8), ("drafts", 3), ("prefix", 2000), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    o = p.parse_args()
    server = Server(o.batch, o.drafts, o.prefix, longest=(o.drafts + 1) * (o.steps + 1))
    graph = server.capture()
    given = torch.zeros(o.batch, dtype=torch.int64, device="cuda")
    for _ in range(o.steps):
        server.random_numbers()
        graph.replay()
        given += 1 + server.accepted
    status = gdn.gdn_get_device_error()
    if status:
        sys.exit(gdn.gdn_status_string(status))
    print("tokens of each request after %d steps:" % o.steps, given.tolist())
    print("pages held: %d, free: %d" % (int(server.pool["held"].sum()),
                                        int(server.pool["free_count"])))


if __name__ == "__main__":
    main()
