"""Timed cases of the hybrid model's serving operators: the paged key/value cache (written and
read back), attention of a batch that shares a long prefix, and the log probabilities of given
tokens.

A hybrid Gated DeltaNet model interleaves its recurrent layers with full-attention layers and
reuses long prompt prefixes.  Next to the recurrent state such a layer keeps a paged key/value
cache; a batch of requests that start with the same prompt attends to one copy of it; and a
multi-token verification step scores the drafted tokens.

Every case is a plain dict; ``op`` names the operator:

  append     new tokens' keys and values go to their cache slots (bf16, or 8-bit codes with a
             power-of-two scale per token and head)
  read       cached tokens are gathered and read back as bf16
  attention  T new tokens of each of B sequences attend to the shared prefix and to their own
             tokens, causally
  logprobs   log probability of a token per row, the row's entropy, the top alternatives

``run`` computes the plain form with elementary torch operations in 32 bits, or, where ``own``
is true, calls the framework.
"""
import math

import torch

own = False

E_MIN, E_MAX, E_BIAS = -60, 60, 127     # stored scale exponents of the 8-bit format
F8_MAX = 448.0


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the attention layers' cache write of a decode step: one token of each of 64 sequences
        dict(name="append f8 decode", op="append", n=64, hkv=4, d=256, page=64, fmt="f8"),
        # a prompt's cache write: keys and values are slices of the fused projection's rows
        dict(name="append f8 prompt", op="append", n=16384, hkv=4, d=256, page=64, fmt="f8"),
        # cached blocks handed on as bf16 (another cache, a transfer): odd count, short head
        dict(name="read f8 blocks", op="read", n=40001, hkv=8, d=128, page=16, fmt="f8"),
        # the read-back of one request's recent tokens
        dict(name="read bf16 request", op="read", n=777, hkv=4, d=256, page=32, fmt="bf16"),
        # a single request on a short cached prompt: latency
        dict(name="attention one request", op="attention", b=1, t=1, hq=24, hkv=4, d=256,
             prefix=512, kv=37, page=64, fmt="bf16"),
        # a decode step of 32 requests on a 16k-token document, 8-bit cache, ragged tails
        dict(name="attention f8 decode", op="attention", b=32, t=1, hq=24, hkv=4, d=256,
             prefix=16384, kv=900, page=64, fmt="f8"),
        # verification of four drafted tokens of 16 requests on a long context
        dict(name="attention bf16 verify", op="attention", b=16, t=4, hq=24, hkv=4, d=256,
             prefix=32771, kv=333, page=16, fmt="bf16"),
        # a large decode batch with a shared system prompt and long tails of its own
        dict(name="attention bf16 batch", op="attention", b=128, t=1, hq=24, hkv=4, d=256,
             prefix=4096, kv=2048, page=128, fmt="bf16"),
        # two requests prefill a few hundred tokens each behind a cached document
        dict(name="attention bf16 prompt", op="attention", b=2, t=333, hq=16, hkv=2, d=128,
             prefix=20000, kv=700, page=32, fmt="bf16"),
        # one token's log probability with its alternatives: latency
        dict(name="logprobs one row", op="logprobs", n=1, v=248320, k=5, dtype="bf16"),
        # a verification step's rows over the model's vocabulary
        dict(name="logprobs verify", op="logprobs", n=64, v=248320, k=20, dtype="bf16"),
        # scoring a prompt from fp32 logits, odd vocabulary, no alternatives
        dict(name="logprobs prompt f32", op="logprobs", n=1000, v=151669, k=0, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "logprobs"])
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([128, 256])
    fmt = rng.choice(["bf16", "f8"])
    if op in ("append", "read"):
        hkv = rng.choice([1, 2, 4, 8])
        most = 16384 * 4 * 256 // (hkv * d)
        return dict(op=op, n=_spread(rng, 1, most), hkv=hkv, d=d, page=page, fmt=fmt)
    if op == "logprobs":
        v = _spread(rng, 1000, 248320)
        return dict(op=op, n=_spread(rng, 1, max(1, 150_000_000 // v)), v=v,
                    k=rng.choice([0, 1, 5, 20, 32]), dtype=rng.choice(["bf16", "f32"]))
    hkv, g = rng.choice([(1, 8), (2, 8), (4, 6), (4, 1), (8, 2), (2, 3), (4, 4)])
    t = rng.choice([1, 1, 1, 2, 4, 7, 16, _spread(rng, 17, 300)])
    b = _spread(rng, 1, max(1, min(128, 600 // t)))
    kv = t + _spread(rng, 1, 1500)
    rows = b * t * g
    # no dearer than the largest listed cases: the products' size, and the sequences' own tokens
    most = max(200, min(32768, 6_000_000_000 // (4 * rows * hkv * d)))
    prefix = rng.choice([0, _spread(rng, 100, most), _spread(rng, 100, most),
                         _spread(rng, 100, most)])
    return dict(op=op, b=b, t=t, hq=hkv * g, hkv=hkv, d=d, prefix=prefix, kv=kv, page=page,
                fmt=fmt)


def _lens(case):
    """The sequences' own token counts, the call's T new tokens included: ragged up to kv."""
    b, t, kv = case["b"], case["t"], case["kv"]
    return [t + (i * 7919 + 13) % max(1, kv - t + 1) if b > 1 else kv for i in range(b)]


def work(case):
    op = case["op"]
    if op in ("append", "read"):
        vectors = 2 * case["n"] * case["hkv"]
        cached = case["d"] + 1 if case["fmt"] == "f8" else 2 * case["d"]
        return {"bytes": vectors * (2 * case["d"] + cached) + 4 * case["n"],
                "flops": 4 * vectors * case["d"] if case["fmt"] == "f8" else 0}
    if op == "logprobs":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["n"]
        return {"bytes": n * case["v"] * e + n * (12 + 8 * case["k"]), "flops": 5 * n * case["v"]}
    b, t, hq, hkv, d = (case[x] for x in ("b", "t", "hq", "hkv", "d"))
    lens = _lens(case)
    vec = 2 * (d + 1 if case["fmt"] == "f8" else 2 * d) * hkv
    pairs = b * t * case["prefix"] + sum(n - t + 1 + i for n in lens for i in range(t))
    return {"bytes": (case["prefix"] + sum(lens)) * vec + b * t * hq * (4 * d + 4),
            "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------- their inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _tokens(g, n, h, d):
    """Keys or values of n tokens: normal, their size varying from token to token."""
    x = _randn(g, n, h, d)
    return (x * torch.exp(0.4 * _randn(g, n, h, 1))).to(torch.bfloat16)


def _quantise(x):
    """Codes and biased exponents of the vectors of x: the least whole e of [E_MIN, E_MAX] with
    max|x| 2^-e <= 448 over the vector's finite values; codes x 2^-e in e4m3, saturating."""
    x = x.float()
    mag = x.abs()
    top = torch.where(torch.isfinite(mag), mag, torch.zeros_like(mag)).amax(-1)
    frac, e = torch.frexp(top)                        # top = frac 2^e, frac in [0.5, 1)
    e = torch.where(frac > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    scaled = x * torch.exp2(-e.float()).unsqueeze(-1)
    return scaled.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn), (e + E_BIAS).to(torch.uint8)


def _dequantise(codes, exps):
    return codes.float() * torch.exp2(exps.float() - E_BIAS).unsqueeze(-1)


def _cache(g, pages, case):
    """A cache in use: every slot holds some token's keys and values."""
    n, h, d, p = pages, case["hkv"], case["d"], case["page"]
    out = {}
    for name in ("k", "v"):
        x = _tokens(g, n, h, p * d).reshape(n, h, p, d)
        if case["fmt"] == "f8":
            out[name], out[name + "_exp"] = _quantise(x)
        else:
            out[name], out[name + "_exp"] = x, None
    return out


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "logprobs":
        n, v, k = case["n"], case["v"], case["k"]
        # rows of different sharpness, as a model's are
        x = 3.0 * _randn(g, n, v) * torch.exp(0.3 * _randn(g, n, 1))
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["targets"] = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["logprobs"] = torch.empty(n, device="cuda")
        s["entropy"] = torch.empty(n, device="cuda")
        s["top_ids"] = torch.empty(n, k, device="cuda", dtype=torch.int32) if k else None
        s["top_logprobs"] = torch.empty(n, k, device="cuda") if k else None
        return s
    p, h, d = case["page"], case["hkv"], case["d"]
    if op in ("append", "read"):
        n = case["n"]
        pages = -(-n // p) + 3
        s["cache"] = _cache(g, pages, case)
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(n, device="cuda") + p // 2   # the first token in the midst of a page
        s["slots"] = (order[i // p] * p + i % p).to(torch.int32)
        if op == "append":
            # keys and values side by side in a projection's output rows
            kv = torch.cat([_tokens(g, n, h, d), _tokens(g, n, h, d)], dim=1)
            s["k"], s["v"] = kv[:, :h], kv[:, h:]
        else:
            s["k_out"] = torch.empty(n, h, d, device="cuda", dtype=torch.bfloat16)
            s["v_out"] = torch.empty_like(s["k_out"])
        return s
    b, t, hq = case["b"], case["t"], case["hq"]
    lens = _lens(case)
    shared = -(-case["prefix"] // p)
    each = -(-max(lens) // p)
    s["cache"] = _cache(g, shared + b * each, case)
    order = torch.randperm(shared + b * each, generator=g, device="cuda").to(torch.int32)
    s["prefix_pages"] = order[:shared].contiguous()
    s["pages"] = order[shared:].reshape(b, each).contiguous()
    s["kv_len"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["q"] = (1.5 * _randn(g, b, t, hq, d)).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(b, t, hq, device="cuda")
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import gated_deltanet_linear_13_gb300 as gdn
    op = s["case"]["op"]
    if op == "logprobs":
        if "workspace" not in s:
            n, v = s["logits"].shape
            s["workspace"] = torch.empty(
                gdn.gdn_token_logprobs_workspace_size(n, v, s["case"]["k"],
                                                      dtype=s["logits"].dtype),
                dtype=torch.uint8, device="cuda")
        gdn.gdn_token_logprobs(s["logits"], s["targets"], s["logprobs"], s["entropy"],
                               top_ids=s["top_ids"], top_logprobs=s["top_logprobs"],
                               workspace=s["workspace"])
        return {x: s[x] for x in ("logprobs", "entropy", "top_ids", "top_logprobs")}
    c = s["cache"]
    if op == "append":
        gdn.gdn_kv_cache_append(s["k"], s["v"], c["k"], c["v"], s["slots"], k_exp=c["k_exp"],
                                v_exp=c["v_exp"])
        return dict(c)
    if op == "read":
        gdn.gdn_kv_cache_read(c["k"], c["v"], s["slots"], s["k_out"], s["v_out"],
                              k_exp=c["k_exp"], v_exp=c["v_exp"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if "workspace" not in s:
        b, t, hq, d = s["q"].shape
        s["workspace"] = torch.empty(
            gdn.gdn_prefix_attention_workspace_size(b, t, hq, s["case"]["hkv"], d),
            dtype=torch.uint8, device="cuda")
    gdn.gdn_prefix_attention(s["q"], c["k"], c["v"], s["out"], prefix_pages=s["prefix_pages"],
                             prefix_len=s["case"]["prefix"], pages=s["pages"],
                             kv_len=s["kv_len"], k_exp=c["k_exp"], v_exp=c["v_exp"],
                             lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _put(cache, slots, x):
    """Vectors x[n] into the cache [pages, heads, page, ...] at their slots."""
    page = cache.shape[2]
    cache[slots // page, :, slots % page] = x


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "logprobs":
        x = s["logits"].float()
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1)
        entropy = torch.log(z) - (e * (x - m)).sum(-1) / z
        lse = m[:, 0] + torch.log(z)
        out = {"logprobs": x.gather(1, s["targets"].long()[:, None])[:, 0] - lse,
               "entropy": entropy, "top_ids": None, "top_logprobs": None}
        if case["k"]:
            del e
            top, ids = torch.sort(x, dim=-1, descending=True, stable=True)
            out["top_ids"] = ids[:, :case["k"]].to(torch.int32)
            out["top_logprobs"] = top[:, :case["k"]] - lse[:, None]
        return out
    c = s["cache"]
    if op == "append":
        slots = s["slots"].long()
        for name in ("k", "v"):
            if case["fmt"] == "f8":
                codes, exps = _quantise(s[name])
                _put(c[name].view(torch.uint8), slots, codes.view(torch.uint8))
                _put(c[name + "_exp"], slots, exps)
            else:
                _put(c[name], slots, s[name])
        return dict(c)
    if op == "read":
        at = (s["slots"].long() // case["page"], slice(None), s["slots"].long() % case["page"])
        out = {}
        for name in ("k", "v"):
            if case["fmt"] == "f8":
                codes = c[name].view(torch.uint8)[at].view(torch.float8_e4m3fn)
                out[name] = _dequantise(codes, c[name + "_exp"][at]).to(torch.bfloat16)
            else:
                out[name] = c[name][at]
        return out
    return _plain_attention(s)


def _pages_of(c, name, pages):
    """The tokens of `pages` [..., n] as fp32 [..., heads, n * page, d]."""
    x = c[name].view(torch.uint8)[pages].view(c[name].dtype)
    x = x.float() if c[name + "_exp"] is None else _dequantise(x, c[name + "_exp"][pages])
    x = x.movedim(-3, -4)                               # [..., heads, n, page, d]
    return x.reshape(*x.shape[:-3], x.shape[-3] * x.shape[-2], x.shape[-1])


def _plain_attention(s):
    case, c, q = s["case"], s["cache"], s["q"]
    b, t, hq, d = q.shape
    h, length = case["hkv"], case["prefix"]
    g = hq // h
    q = q.float().reshape(b, t, h, g, d) / math.sqrt(d)
    # the shared prefix: one product over all rows of the batch
    flat = q.permute(2, 0, 1, 3, 4).reshape(h, b * t * g, d)
    pages = s["prefix_pages"].long()
    kp, vp = (_pages_of(c, x, pages)[:, :length] for x in ("k", "v"))
    sp = torch.matmul(flat, kp.transpose(1, 2))          # [h, b t g, length]
    # the sequences' own tokens, causal over the last t
    rows = q.permute(0, 2, 1, 3, 4).reshape(b, h, t * g, d)
    ks, vs = (_pages_of(c, x, s["pages"].long()) for x in ("k", "v"))
    ss = torch.matmul(rows, ks.transpose(2, 3)).reshape(b, h, t, g, -1)
    j = torch.arange(ss.shape[-1], device=q.device)
    seen = s["kv_len"].long()[:, None] - t + 1 + torch.arange(t, device=q.device)
    ss = ss.masked_fill((j >= seen[..., None])[:, None, :, None, :], -math.inf)
    ss = ss.reshape(b, h, t * g, -1)
    # softmax over both, each row's maximum and sum
    m = ss.amax(-1)
    if length:
        m = torch.maximum(m, sp.amax(-1).reshape(h, b, t * g).transpose(0, 1))
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    ps = torch.exp(ss - m[..., None])
    z, o = ps.sum(-1), torch.matmul(ps, vs)
    if length:
        pp = torch.exp(sp - m.transpose(0, 1).reshape(h, b * t * g)[..., None])
        z = z + pp.sum(-1).reshape(h, b, t * g).transpose(0, 1)
        o = o + torch.matmul(pp, vp).reshape(h, b, t * g, d).transpose(0, 1)
    o = o / torch.where(z > 0, z, torch.ones_like(z))[..., None]
    lse = m + torch.log(z)
    out = o.reshape(b, h, t, g, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d)
    return {"out": out.to(torch.bfloat16),
            "lse": lse.reshape(b, h, t, g).permute(0, 2, 1, 3).reshape(b, t, hq)}


# ------------------------------------------------------------------- the answer in 64 bits

def _value(c, name, page, head):
    """One page of one head in 64 bits: [page, d]."""
    x = c[name][page, head].to(torch.float64 if c[name + "_exp"] is None else torch.float32)
    x = x.double()
    if c[name + "_exp"] is not None:
        x = x * torch.pow(2.0, c[name + "_exp"][page, head].double() - 127)[..., None]
    return x


def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        out = {"logprobs": [], "entropy": [], "top_ids": None, "top_logprobs": []}
        for r in range(case["n"]):
            x = s["logits"][r].double()
            logp = x - torch.logsumexp(x, 0)
            out["logprobs"].append(logp[int(s["targets"][r])])
            out["entropy"].append(-(logp.exp() * logp).sum())
            if case["k"]:
                out["top_logprobs"].append(torch.topk(logp, case["k"]).values)
        return {"logprobs": torch.stack(out["logprobs"]), "entropy": torch.stack(out["entropy"]),
                "top_ids": None,
                "top_logprobs": torch.stack(out["top_logprobs"]) if case["k"] else None}
    if op == "append":
        page, off = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
        out = {}
        for name in ("k", "v"):
            x, cache = s[name].double(), s["cache"][name].float().double()
            out[name + "_exp"] = s["cache"][name + "_exp"]
            if case["fmt"] == "f8":
                e = torch.ceil(torch.log2(x.abs().amax(-1) / F8_MAX)).clamp(E_MIN, E_MAX)
                x = x * torch.pow(2.0, -e)[..., None]
                # four significant bits, down to 2^-9
                unit = torch.pow(2.0, torch.floor(torch.log2(x.abs())).clamp(min=-6) - 3)
                x = (torch.round(x / unit) * unit).clamp(-F8_MAX, F8_MAX)
                out[name + "_exp"][page, :, off] = (e + 127).to(torch.uint8)
            cache[page, :, off] = x
            out[name] = cache
        return out
    if op == "read":
        page, off = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
        out = {}
        for name in ("k", "v"):
            x = s["cache"][name].float().double()[page, :, off]
            if s["cache"][name + "_exp"] is not None:
                e = s["cache"][name + "_exp"][page, :, off].double() - 127
                x = x * torch.pow(2.0, e)[..., None]
            out[name] = x
        return out
    b, t, hq, d = s["q"].shape
    group = hq // case["hkv"]
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["kv_len"].tolist()
    for head in range(case["hkv"]):
        gathered = {}
        for name in ("k", "v"):
            x = _value(s["cache"], name, s["prefix_pages"].long(), head)
            gathered[name] = x.reshape(-1, d)[:case["prefix"]]
        for i in range(b):
            keys, values = (torch.cat([gathered[name], _value(
                s["cache"], name, s["pages"][i].long(), head).reshape(-1, d)[:lens[i]]])
                for name in ("k", "v"))
            rows = s["q"][i, :, head * group:(head + 1) * group].double()     # [t, group, d]
            score = torch.einsum("tgd,nd->tgn", rows, keys) * d ** -0.5
            last = case["prefix"] + lens[i] - t + torch.arange(t, device="cuda")
            hidden = torch.arange(keys.shape[0], device="cuda") > last[:, None]
            score = score.masked_fill(hidden[:, None], -math.inf)
            norm = torch.logsumexp(score, -1)
            prob = torch.exp(score - norm[..., None])
            out[i, :, head * group:(head + 1) * group] = torch.einsum("tgn,nd->tgd", prob, values)
            lse[i, :, head * group:(head + 1) * group] = norm
    return {"out": out, "lse": lse}
