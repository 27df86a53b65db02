"""Timed cases of what a hybrid model's serving step does around its attention layers and behind
its logits: the norm of queries and keys with their rotation by position, written on into the
paged cache; the step's block tables and slots, built on the GPU from the requests' lengths; and
the verification of drafted tokens from given random numbers.

Every case is a plain dict; ``op`` names the operator:

  rope     queries and keys are normalised by head, rotated by their positions, and go to tensors
           or (keys, with the values) to their slots of the paged cache
  pages    a step's new tokens get pages, slots and positions, then what was rejected of them (or
           the requests that end) gives its pages back
  verify   drafted tokens are accepted or refused under the target's probabilities, and one more
           token is drawn behind the last accepted one (without drafts: plain sampling)

``run`` computes the plain form with elementary torch operations, or, where ``own`` is true, calls
the framework.
"""
import math
import random

import torch

own = False

E_MIN, E_MAX, E_BIAS = -60, 60, 127     # stored scale exponents of the 8-bit cache
F8_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the next token of a single request: latency
        dict(name="rope one token", op="rope", n=1, hq=24, hkv=4, d=256, rot=64, pairs="half",
             dtype="bf16", to="bf16", page=64, scaling="none", far=4000, gated=True),
        # a decode step of 64 requests; the query projection's rows hold a gate beside each head
        dict(name="rope decode", op="rope", n=64, hq=24, hkv=4, d=256, rot=64, pairs="half",
             dtype="bf16", to="bf16", page=64, scaling="none", far=32000, gated=True),
        # four drafted tokens of 32 requests into the 8-bit cache, context extended fourfold
        dict(name="rope verify f8", op="rope", n=128, hq=24, hkv=4, d=256, rot=64, pairs="half",
             dtype="bf16", to="f8", page=64, scaling="yarn", far=131072, gated=False),
        # a prompt's chunk
        dict(name="rope prompt", op="rope", n=16384, hq=24, hkv=4, d=256, rot=64, pairs="half",
             dtype="bf16", to="bf16", page=64, scaling="none", far=131072, gated=False),
        # fp32 activations, the whole head rotated, neighbouring pairs, no cache
        dict(name="rope f32", op="rope", n=2501, hq=16, hkv=2, d=128, rot=128, pairs="neighbours",
             dtype="f32", to="tensors", page=16, scaling="ntk", far=1000000, gated=False),
        # a verification step of 64 requests, five tokens each
        dict(name="pages verify", op="pages", b=64, new=5, kv=3000, page=64, ragged=False),
        # decode and short prefills in one batch, small pages
        dict(name="pages mixed", op="pages", b=7, new=513, kv=700, page=16, ragged=True),
        # the prompts of 300 requests begin
        dict(name="pages prompts", op="pages", b=300, new=800, kv=0, page=32, ragged=True),
        # one request's three drafts over the model's vocabulary: latency
        dict(name="verify one", op="verify", b=1, t=3, v=248320, dtype="bf16", drafts="logits"),
        # a batch's four drafts each
        dict(name="verify batch", op="verify", b=64, t=4, v=248320, dtype="bf16", drafts="logits"),
        # drafts looked up in the text (no probabilities of their own), fp32 logits, odd vocabulary
        dict(name="verify lookup f32", op="verify", b=16, t=7, v=151669, dtype="f32", drafts="ids"),
        # the next token of 128 requests without drafts
        dict(name="verify sample", op="verify", b=128, t=0, v=151936, dtype="bf16", drafts="ids"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "pages", "verify", "verify"])
    if op == "pages":
        new = rng.choice([1, 1, 2, 5, 9, _spread(rng, 10, 4000)])
        return dict(op=op, b=_spread(rng, 1, max(1, min(400, 240000 // new))), new=new,
                    kv=rng.choice([0, _spread(rng, 1, 4000), _spread(rng, 1, 4000)]),
                    page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.6)
    if op == "verify":
        v, t = _spread(rng, 1000, 248320), rng.choice([0, 1, 2, 3, 4, 5, 7, 15])
        drafts = rng.choice(["logits", "ids"]) if t else "ids"
        dtype = rng.choice(["bf16", "f32"])
        most = 140_000_000 // (v * (2 * t + 1 if drafts == "logits" else t + 3))
        most = most if dtype == "bf16" else most // 2
        return dict(op=op, b=_spread(rng, 1, max(1, min(256, most))), t=t, v=v, dtype=dtype,
                    drafts=drafts)
    to = rng.choice(["tensors", "bf16", "bf16", "f8"])
    d = rng.choice([64, 96, 128, 192, 256]) if to == "tensors" else rng.choice([128, 256])
    hkv, g = rng.choice([(1, 8), (2, 8), (4, 6), (4, 1), (8, 4), (2, 3), (3, 5)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 16384 * 32 * 256 // ((hkv * (g + 2)) * d * (2 if dtype == "f32" else 1))
    return dict(op=op, n=_spread(rng, 1, 300 if to == "f8" else min(60000, most)), hq=hkv * g,
                hkv=hkv, d=d, rot=rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                pairs=rng.choice(["half", "neighbours"]), dtype=dtype, to=to,
                page=rng.choice([16, 32, 64, 128]),
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                far=_spread(rng, 100, 2000000), gated=rng.random() < 0.3)


def work(case):
    if case["op"] == "pages":
        tokens = case["b"] * case["new"]                 # the capacity of slots and positions
        each = _columns(case) * 4
        return {"bytes": tokens * 8 + case["b"] * (2 * each + 40), "flops": 0}
    if case["op"] == "verify":
        b, t, v = case["b"], case["t"], case["v"]
        e = 2 if case["dtype"] == "bf16" else 4
        rows = b * (2 * t + 1 if case["drafts"] == "logits" else t + 1)
        return {"bytes": rows * v * e + b * v * 4 + b * (t + 1) * 16, "flops": 4 * rows * v}
    n, d = case["n"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["to"] == "tensors":
        size = n * (case["hq"] + case["hkv"]) * d * 2 * e
    else:
        kept = 2 * d if case["to"] == "bf16" else d + 1
        size = n * (case["hq"] * d * 2 * e + 2 * case["hkv"] * (d * e + kept))
    return {"bytes": size + 8 * n, "flops": 8 * n * (case["hq"] + case["hkv"]) * d}


# ---------------------------------------------------------------------------- their inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _frequencies(case):
    """Radians a token of each pair, and the amplitude, for a context `factor` times as long."""
    r, base, factor, trained = case["rot"], 10000.0, 4.0, 32768
    scaling = case["scaling"]
    if scaling == "ntk" and r > 2:
        base *= factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "yarn":
        return f, 1.0

    def pair_of(turns):                     # the pair that makes so many turns over the context
        return r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(0, math.floor(pair_of(32.0))), min(r - 1, math.ceil(pair_of(1.0)))
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(r // 2)]
    return [x / factor * w + x * (1 - w) for x, w in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def _prepare_rope(case, g):
    n, hq, hkv, d, p = (case[x] for x in ("n", "hq", "hkv", "d", "page"))
    s = {}
    width = hq * (2 if case["gated"] else 1) + 2 * hkv
    # one projection's rows: queries (each with its gate, where there are gates), keys, values
    rows = (_randn(g, n, width, d) * torch.exp(0.4 * _randn(g, n, width, 1))).to(_dtype(case))
    s["q"] = rows[:, :2 * hq:2] if case["gated"] else rows[:, :hq]
    s["k"], s["v"] = rows[:, -2 * hkv:-hkv], rows[:, -hkv:]
    s["q_weight"], s["k_weight"] = 1.0 + 0.2 * _randn(g, d), 1.0 + 0.2 * _randn(g, d)
    f, s["amplitude"] = _frequencies(case)
    s["frequencies"] = torch.tensor(f, device="cuda", dtype=torch.float64)
    # the same as steps of phase, 2^64 to the turn
    steps = [round(x / (2 * math.pi) * 2 ** 64) % 2 ** 64 for x in f]
    s["phase_steps"] = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in steps],
                                    device="cuda", dtype=torch.int64)
    if n > 1000:                                         # a prompt's chunk, behind others
        first = int(torch.randint(0, max(1, case["far"] - n), (1,), generator=g, device="cuda"))
        s["positions"] = first + torch.arange(n, device="cuda", dtype=torch.int32)
    else:
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda",
                                       dtype=torch.int32)
    s["q_out"] = torch.empty(n, hq, d, device="cuda", dtype=_dtype(case))
    if case["to"] == "tensors":
        s["k_out"] = torch.empty(n, hkv, d, device="cuda", dtype=_dtype(case))
        return s
    pages = -(-n // p) + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(n, device="cuda") + p // 2          # the first token in the midst of a page
    s["slots"] = (order[i // p] * p + i % p).to(torch.int32)
    for name in ("k", "v"):                              # a cache in use
        x = _randn(g, pages, hkv, p, d)
        s[name + "_cache"], s[name + "_exp"] = (
            _quantise(x) if case["to"] == "f8" else (x.to(torch.bfloat16), None))
    return s


def _lengths(case, seed):
    """Own tokens before the step, new tokens, and tokens kept after it, of each request; a batch
    of more than eight is padded with some that it leaves out."""
    r = random.Random(int(seed) * 31 + 5)
    b, new = case["b"], case["new"]
    kv = [r.randint(case["kv"] // 3, case["kv"]) for _ in range(b)]
    fresh = [r.randint(0 if b > 1 else 1, new) if case["ragged"] else new for _ in range(b)]
    kept = [k + r.choice([0, r.randint(0, n), n]) for k, n in zip(kv, fresh)]
    return kv, fresh, kept, b // 9


def _columns(case):
    """Columns of the block tables: room for the longest request and a quarter more."""
    return -(-(case["kv"] + case["new"]) * 5 // (4 * case["page"])) + 1


def _prepare_pages(case, seed):
    p, b, columns = case["page"], case["b"], _columns(case)
    kv, fresh, kept, out = _lengths(case, seed)
    r = random.Random(int(seed) * 17 + 3)
    rows = b + b // 4 + 1                                # requests that the tables have room for
    mine = r.sample(range(rows), b)
    held = [-(-k // p) for k in kv]
    total = b * (-(-case["kv"] // p) + -(-case["new"] // p) + 1) + rows
    order = list(range(total))
    r.shuffle(order)
    table = [[0] * columns for _ in range(rows)]
    of_row = [0] * rows
    for row, n in zip(mine, held):
        table[row][:n] = order[:n]
        order = order[n:]
        of_row[row] = n
    i32 = dict(device="cuda", dtype=torch.int32)
    s = {"table": torch.tensor(table, **i32), "held": torch.tensor(of_row, **i32),
         "free_pages": torch.tensor(order + [0] * (total - len(order)), **i32),
         "free_count": torch.tensor([len(order)], **i32)}
    s["rows"] = torch.tensor(mine[:b - out] + [-1] * out, **i32)
    s["kv_len"], s["new_len"], s["keep_len"] = (torch.tensor(x, **i32) for x in (kv, fresh, kept))
    n = b * case["new"]
    s["slots"], s["positions"] = torch.zeros(n, **i32), torch.zeros(n, **i32)
    s["cu_seqlens"], s["kv_len_out"] = torch.zeros(b + 1, **i32), torch.zeros(b, **i32)
    s["pages"] = torch.zeros(b, columns, **i32)
    s["offset"] = 1000                                   # tokens of a shared prefix
    return s


def _prepare_verify(case, seed):
    g = _gen(seed)
    r = random.Random(int(seed) * 7 + 1)
    b, t, v = case["b"], case["t"], case["v"]
    s = {}
    # rows of different sharpness, as a model's are
    x = 3.0 * _randn(g, b, t + 1, v) * torch.exp(0.3 * _randn(g, b, t + 1, 1))
    s["target"] = x.to(_dtype(case))
    s["draft"] = s["draft_ids"] = s["accept_u"] = None
    # temperatures, some greedy requests, some padding at the end of larger batches
    scale = [r.choice([1.0, 1.0, 1.25, 1 / 0.7, 0.8, math.inf]) for _ in range(b)]
    scale[b - b // 9:] = [-1.0] * (b // 9)
    s["scale"] = torch.tensor(scale, device="cuda")
    if t:
        # the draft model's logits are the target's with an error; its tokens come from them
        y = x[:, :t] + 0.7 * _randn(g, b, t, v)
        y = y.to(_dtype(case)) if case["drafts"] == "logits" else y
        ids = []
        for i in range(t):
            z = y[:, i].float() * s["scale"].clamp(0.1, 50.0)[:, None]
            clock = torch.empty(b, v, device="cuda").exponential_(generator=g)
            ids.append((z - torch.log(clock)).argmax(-1))
        s["draft_ids"] = torch.stack(ids, 1).to(torch.int32)
        for i in range(1, b, 5):                         # fewer drafts than the others
            s["draft_ids"][i, r.randint(0, t):] = -1
        s["draft"] = y if case["drafts"] == "logits" else None
        s["accept_u"] = torch.rand(b, t, generator=g, device="cuda")
    s["clocks"] = torch.empty(b, v, device="cuda").exponential_(generator=g)
    s["tokens"] = torch.full((b, t + 1), -7, device="cuda", dtype=torch.int32)
    s["accepted"] = torch.full((b,), -7, device="cuda", dtype=torch.int32)
    s["logprobs"] = torch.full((b, t + 1), 7.0, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "rope":
        s = _prepare_rope(case, _gen(seed))
    elif case["op"] == "pages":
        s = _prepare_pages(case, seed)
    else:
        s = _prepare_verify(case, seed)
    s["case"] = case
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _outputs(s):
    op = s["case"]["op"]
    if op == "rope":
        names = ("q_out", "k_out", "k_cache", "v_cache", "k_exp", "v_exp")
    elif op == "pages":
        names = ("slots", "positions", "cu_seqlens", "kv_len_out", "pages", "table", "held",
                 "free_pages", "free_count")
    else:
        names = ("tokens", "accepted", "logprobs")
    return {x: s[x] for x in names if s.get(x) is not None}


def _run_own(s):
    import gated_deltanet_linear_13_gb300 as gdn
    case = s["case"]
    if case["op"] == "rope":
        kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                  interleaved=case["pairs"] == "neighbours", amplitude=s["amplitude"])
        if case["to"] == "tensors":
            gdn.gdn_qk_norm_rope(s["q"], s["k"], s["positions"], s["phase_steps"], s["q_out"],
                                 s["k_out"], **kw)
        else:
            gdn.gdn_qk_norm_rope(s["q"], s["k"], s["positions"], s["phase_steps"], s["q_out"],
                                 v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                                 slots=s["slots"], k_exp=s["k_exp"], v_exp=s["v_exp"], **kw)
    elif case["op"] == "pages":
        pool = dict(table=s["table"], held=s["held"], free_pages=s["free_pages"],
                    free_count=s["free_count"], page_size=case["page"])
        gdn.gdn_page_plan(s["kv_len"], s["new_len"], s["slots"], s["positions"], s["cu_seqlens"],
                          s["kv_len_out"], s["pages"], rows=s["rows"],
                          position_offset=s["offset"], **pool)
        gdn.gdn_page_release(s["keep_len"], rows=s["rows"], **pool)
    else:
        if "workspace" not in s:
            b, t1, v = s["target"].shape
            s["workspace"] = torch.empty(gdn.gdn_verify_tokens_workspace_size(
                b, t1 - 1, v, dtype=s["target"].dtype, draft_logits=s["draft"] is not None),
                dtype=torch.uint8, device="cuda")
        gdn.gdn_verify_tokens(s["target"], s["tokens"], s["accepted"], clocks=s["clocks"],
                              draft_ids=s["draft_ids"], draft_logits=s["draft"],
                              accept_u=s["accept_u"], scale=s["scale"], logprobs=s["logprobs"],
                              workspace=s["workspace"])
    return _outputs(s)


def _run_plain(s):
    {"rope": _plain_rope, "pages": _plain_pages, "verify": _plain_verify}[s["case"]["op"]](s)
    return _outputs(s)


# ------------------------------------------------------------------------ plain: rotation

def _quantise(x):
    """Codes and biased exponents of the vectors of x: the least whole e of [E_MIN, E_MAX] with
    max|x| 2^-e <= 448; codes x 2^-e in e4m3, saturating."""
    top = x.abs().amax(-1)
    frac, e = torch.frexp(top)                           # top = frac 2^e, frac in [0.5, 1)
    e = torch.where(frac > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    scaled = x * torch.exp2(-e.float()).unsqueeze(-1)
    return scaled.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn), (e + E_BIAS).to(torch.uint8)


def _plain_norm_rope(s, x, weight):
    case, r = s["case"], s["case"]["rot"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    angle = s["positions"].double()[:, None] * s["frequencies"]      # far positions: 64 bits
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    if case["pairs"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rope(s):
    case = s["case"]
    s["q_out"].copy_(_plain_norm_rope(s, s["q"], s["q_weight"]))
    k = _plain_norm_rope(s, s["k"], s["k_weight"])
    if case["to"] == "tensors":
        s["k_out"].copy_(k)
        return
    slots, p = s["slots"].long(), case["page"]
    for name, x in (("k", k), ("v", s["v"].float())):
        cache = s[name + "_cache"]
        if case["to"] == "f8":
            codes, exps = _quantise(x)
            cache.view(torch.uint8)[slots // p, :, slots % p] = codes.view(torch.uint8)
            s[name + "_exp"][slots // p, :, slots % p] = exps
        else:
            cache[slots // p, :, slots % p] = x.to(torch.bfloat16)


# --------------------------------------------------------------------------- plain: pages

def _before(x):
    """Sums of the entries before each."""
    return torch.cumsum(x, 0) - x


def _plain_pages(s):
    case, p = s["case"], s["case"]["page"]
    b, columns = s["pages"].shape
    rows = s["rows"].long()
    inside = rows >= 0
    rows = rows.clamp(min=0)
    kv, new = s["kv_len"].long(), torch.where(inside, s["new_len"].long(), 0)
    held = s["held"].long()[rows]
    need = torch.where(inside, ((kv + new + p - 1) // p - held).clamp(min=0), 0)
    first_token, first_page = _before(new), _before(need)
    count = s["free_count"].long()
    s["cu_seqlens"][:1] = 0
    s["cu_seqlens"][1:] = torch.cumsum(new, 0).to(torch.int32)
    s["kv_len_out"].copy_(torch.where(inside, kv + new, -1))
    # the block tables: pages held, then pages from the end of the free ones
    col = torch.arange(columns, device="cuda")
    taken = count - 1 - (first_page[:, None] + col - held[:, None])
    fresh = s["free_pages"][taken.clamp(0, s["free_pages"].numel() - 1)]
    is_new = (col >= held[:, None]) & (col < (held + need)[:, None])
    block = torch.where(is_new, fresh, s["table"][rows])
    written = inside[:, None] & (col < (held + need)[:, None])
    s["pages"].copy_(torch.where(written, block, s["pages"]))
    # (entries left out write to a row behind the last)
    to = torch.where(inside, rows, s["table"].shape[0])
    wide = torch.cat([s["table"], s["table"][:1]])
    wide[to] = block
    s["table"].copy_(wide[:-1])
    wide = torch.cat([s["held"], s["held"][:1]])
    wide[to] = (held + need).to(torch.int32)
    s["held"].copy_(wide[:-1])
    # the tokens
    i = torch.arange(s["slots"].numel(), device="cuda")
    seq = torch.searchsorted(torch.cumsum(new, 0), i, right=True).clamp(max=b - 1)
    at = kv[seq] + i - first_token[seq]
    live = i < new.sum()
    page = block[seq, (at // p).clamp(0, columns - 1)].long()
    s["slots"].copy_(torch.where(live, page * p + at % p, -1))
    s["positions"].copy_(torch.where(live, at + s["offset"], 0))
    s["free_count"].sub_(need.sum().to(torch.int32))
    # what is not kept goes back, the last page of the last request first
    held = s["held"].long()[rows]
    keep = (s["keep_len"].long() + p - 1) // p
    gone = torch.where(inside, (held - keep).clamp(min=0), 0)
    to_free = s["free_count"].long() + gone.sum() - 1 - (_before(gone)[:, None] + col
                                                       - keep[:, None])
    back = inside[:, None] & (col >= keep[:, None]) & (col < held[:, None])
    wide = torch.cat([s["free_pages"], s["free_pages"][:1]])
    wide[torch.where(back, to_free, s["free_pages"].numel())] = s["table"][rows]
    s["free_pages"].copy_(wide[:-1])
    wide = torch.cat([s["held"], s["held"][:1]])
    wide[to] = (held - gone).to(torch.int32)
    s["held"].copy_(wide[:-1])
    s["free_count"].add_(gone.sum().to(torch.int32))


# --------------------------------------------------------------------- plain: verification

def _normaliser(x, scale):
    """Largest logit and sum of exp(scale (x - largest)) of the rows."""
    x = x.float()
    m = x.amax(-1, keepdim=True)
    return m[..., 0], torch.exp((x - m) * scale[:, None, None]).sum(-1)


def _plain_verify(s):
    target, draft, ids = s["target"], s["draft"], s["draft_ids"]
    b, t1, v = target.shape
    t = t1 - 1
    greedy, active = torch.isinf(s["scale"]), s["scale"] > 0
    scale = torch.where(greedy | ~active, torch.ones_like(s["scale"]), s["scale"])
    m, z = _normaliser(target, scale)
    best = target.float().argmax(-1)
    seq = torch.arange(b, device="cuda")
    accepted = torch.zeros(b, device="cuda", dtype=torch.int64)
    wide = scale.double()
    if t:
        n = (ids >= 0).long().cumprod(1)                 # drafts of each sequence, then none
        at = ids.long().clamp(min=0)[..., None]
        # next to a border: 64 bits
        ratio = (target[:, :t].gather(2, at)[..., 0].double() - m[:, :t].double()) * wide[:, None]
        ratio = ratio - torch.log(z[:, :t].double())
        if draft is not None:
            md, zd = _normaliser(draft, scale)
            ratio = ratio - (draft.gather(2, at)[..., 0].double() - md.double()) * wide[:, None]
            ratio = ratio + torch.log(zd.double())
        good = torch.where(greedy[:, None], ids == best[:, :t],
                           s["accept_u"].double() < torch.exp(ratio))
        accepted = (good & (n > 0)).long().cumprod(1).sum(1)
    # one more token from the row behind the last accepted one
    row = target[seq, accepted].double()
    weight = torch.exp((row - m[seq, accepted].double()[:, None]) * wide[:, None])
    weight = weight / z[seq, accepted].double()[:, None]
    last = torch.full_like(accepted, -1)
    if t:
        refused = accepted < n.sum(1)
        i = accepted.clamp(max=t - 1)
        last = torch.where(refused, ids[seq, i].long(), -1)
        if draft is not None:
            other = torch.exp((draft[seq, i].double() - md[seq, i].double()[:, None])
                              * wide[:, None]) / zd[seq, i].double()[:, None]
        else:
            other = (torch.arange(v, device="cuda") == last[:, None]).double()
        weight = torch.where(refused[:, None], (weight - other).clamp(min=0), weight)
    race, token = (weight / s["clocks"].double()).max(-1)
    token = torch.where(race > 0, token, last)
    token = torch.where(greedy, best[seq, accepted], token)
    col = torch.arange(t1, device="cuda")
    out = torch.where(col == accepted[:, None], token[:, None], -1)
    if t:
        drafts = torch.cat([ids.long(), ids[:, :1].long()], 1)
        out = torch.where(col < accepted[:, None], drafts, out)
    logp = target.gather(2, out.clamp(min=0)[..., None])[..., 0].float() - m
    logp = logp * scale[:, None] - torch.log(z)
    logp = torch.where(out >= 0, logp, 0.0)
    s["tokens"].copy_(torch.where(active[:, None], out.to(torch.int32), s["tokens"]))
    s["accepted"].copy_(torch.where(active, accepted.to(torch.int32), s["accepted"]))
    s["logprobs"].copy_(torch.where(active[:, None], logp, s["logprobs"]))


# ------------------------------------------------------------------- the answer in 64 bits

def exact(case, seed):
    """The definitions in 64 bits; whole numbers have none."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    return (_exact_rope if case["op"] == "rope" else _exact_verify)(case, s)


def _exact_rope(case, s):
    r, d = case["rot"], case["d"]
    pair = torch.arange(r // 2, device="cuda")
    first = pair if case["pairs"] == "half" else 2 * pair
    second = pair + r // 2 if case["pairs"] == "half" else 2 * pair + 1
    turn = torch.polar(torch.full((case["n"], r // 2), float(s["amplitude"]), device="cuda",
                                  dtype=torch.float64),
                       torch.outer(s["positions"].double(), s["frequencies"]))
    done = {}
    for name in ("q", "k"):
        x = s[name].double()
        x = s[name + "_weight"].double() * x / (x.norm(dim=-1, keepdim=True) ** 2 / d
                                                + EPS).sqrt()
        y = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = y.real, y.imag
        done[name] = x
    out = {"q_out": done["q"]}
    if case["to"] == "tensors":
        return out | {"k_out": done["k"]}
    done["v"] = s["v"].double()
    slots = s["slots"].long()
    page, off = slots // case["page"], slots % case["page"]
    for name in ("k", "v"):
        x, cache = done[name], s[name + "_cache"].float().double()
        if case["to"] == "f8":
            e = torch.ceil(torch.log2(x.abs().amax(-1) / F8_MAX)).clamp(E_MIN, E_MAX)
            x = x * torch.pow(2.0, -e)[..., None]
            # four significant bits, down to 2^-9
            unit = torch.pow(2.0, torch.floor(torch.log2(x.abs())).clamp(min=-6) - 3)
            x = (torch.round(x / unit) * unit).clamp(-F8_MAX, F8_MAX)
            out[name + "_exp"] = None
        cache[page, :, off] = x
        out[name + "_cache"] = cache
    return out


def _exact_verify(case, s):
    b, t = case["b"], case["t"]
    logprobs = s["logprobs"].double()
    for i in range(b):
        scale = float(s["scale"][i])
        if scale < 0:
            continue
        greedy = math.isinf(scale)
        logprobs[i] = 0.0
        for j in range(t + 1):
            x = s["target"][i, j].double() * (1.0 if greedy else scale)
            logp = x - torch.logsumexp(x, 0)
            drafted = int(s["draft_ids"][i, j]) if j < t else -1
            p, q = logp.exp(), torch.zeros_like(x)
            if drafted >= 0 and case["drafts"] == "logits":
                y = s["draft"][i, j].double() * (1.0 if greedy else scale)
                q = (y - torch.logsumexp(y, 0)).exp()
            elif drafted >= 0:
                q[drafted] = 1.0
            if drafted >= 0:
                taken = (drafted == int(x.argmax()) if greedy else
                         float(s["accept_u"][i, j]) * float(q[drafted]) < float(p[drafted]))
                if taken:
                    logprobs[i, j] = logp[drafted]
                    continue
            token = int(x.argmax()) if greedy else int(
                ((p - q).clamp(min=0) / s["clocks"][i].double()).argmax())
            logprobs[i, j] = logp[token]
            break
    return {"tokens": None, "accepted": None, "logprobs": logprobs}
