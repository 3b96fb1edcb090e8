"""The operators of a decode step between its weight products: cases, inputs,
plain forms and references, for measuring the library's kernels.

Three operators, told apart by a case's "op":
  rope    rotary positions on q and k, with k and v written to a paged cache;
  attn    attention of a batch of sequences that share a prefix;
  logits  penalties, biases and grammar masks on logits, with the argmax.

`run` computes them in their plain form (elementary torch operations in 32
bits) or, with `own` set, through the package's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
NEG_INF = float("-inf")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decode step of one sequence (3B heads): the smallest call, latency only.
        dict(name="rope_decode1", op="rope", n=1, hq=16, hkv=2, d=128, rot=128, layout="half", scaling="plain",
             base=1e6, factor=1.0, orig=0, type="f32", cache="bf16", page=16, top=32768),
        # A prompt chunk of odd length, small heads of which half rotate, pairs interleaved, 16-bit inputs.
        dict(name="rope_chunk_interleaved", op="rope", n=1021, hq=14, hkv=2, d=64, rot=32, layout="interleaved",
             scaling="linear", base=1e4, factor=4.0, orig=8192, type="f16", cache="f16", page=16, top=32768),
        # A long prompt at once, positions beyond the trained length, scaled by frequency.
        dict(name="rope_prompt16k", op="rope", n=16384, hq=32, hkv=8, d=128, rot=128, layout="half", scaling="yarn",
             base=1e6, factor=4.0, orig=32768, type="f32", cache="bf16", page=64, top=131072),
        # Two samples of a short prompt (1.5B heads): latency only.
        dict(name="attn_short", op="attn", b=2, nq=1, hq=12, hkv=2, d=128, prefix=160, suffix=33, page=16,
             cache="bf16", fused=False),
        # Eight samples of one prompt (1.5B heads), one token each: the ordinary parallel-sampling step.
        dict(name="attn_samples8", op="attn", b=8, nq=1, hq=12, hkv=2, d=128, prefix=4096, suffix=512, page=16,
             cache="bf16", fused=True),
        # Eight sequences verifying four drafts each over a long document of odd length (3B heads); q is a part
        # of the QKV output.
        dict(name="attn_verify", op="attn", b=8, nq=5, hq=16, hkv=2, d=128, prefix=32749, suffix=777, page=64,
             cache="f16", fused=True),
        # No shared part, small heads, ragged lengths that reach down to nothing.
        dict(name="attn_noprefix", op="attn", b=16, nq=1, hq=14, hkv=2, d=64, prefix=0, suffix=1500, page=16,
             cache="f16", fused=False),
        # Many sequences on one system prompt: memory-bound, most of it the sequences' own keys.
        dict(name="attn_users64", op="attn", b=64, nq=1, hq=32, hkv=8, d=128, prefix=16384, suffix=2048, page=128,
             cache="bf16", fused=False),
        # The largest: many sequences verifying drafts over a long shared document; matrix-product-bound.
        dict(name="attn_users64_verify", op="attn", b=64, nq=4, hq=32, hkv=8, d=128, prefix=65536, suffix=1024,
             page=256, cache="bf16", fused=False),
        # Greedy step of one sequence with all rules; only the token comes back.
        dict(name="logits_greedy1", op="logits", rows=1, v=151936, type="f32", hist=700, bias=20, mask=0.3,
             write=False),
        # Sampled rows with an odd vocabulary in 16 bits, logits written for the sampler.
        dict(name="logits_odd16", op="logits", rows=5, v=50257, type="bf16", hist=2000, bias=300, mask=0.05,
             write=True),
        # A large batch, logits written.
        dict(name="logits_batch192", op="logits", rows=192, v=151936, type="f32", hist=2048, bias=64, mask=0.5,
             write=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


HEADS = [(12, 2, 128), (16, 2, 128), (14, 2, 64), (32, 8, 128), (8, 8, 64), (16, 1, 128), (24, 4, 96)]


def draw(rng):
    limit = {}
    for c in listed():
        w = work(c)
        limit[c["op"]] = (max(limit.get(c["op"], (0, 0))[0], w["bytes"]), max(limit.get(c["op"], (0, 0))[1], w["flops"]))
    op = rng.choice(["rope", "attn", "attn", "logits"])
    while True:
        if op == "rope":
            hq, hkv, d = rng.choice(HEADS)
            t = rng.choice(["f32", "f32", "f16", "bf16"])
            scaling = rng.choice(["plain", "linear", "bands", "yarn"])
            case = dict(op="rope", n=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                        layout=rng.choice(["half", "interleaved"]), scaling=scaling, base=rng.choice([1e4, 5e5, 1e6]),
                        factor=1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0]), orig=rng.choice([8192, 32768]),
                        type=t, cache=rng.choice(["f16", "bf16"]) if t == "f32" else t,
                        page=rng.choice([16, 32, 64, 128]), top=rng.choice([32768, 131072]))
        elif op == "attn":
            hq, hkv, d = rng.choice(HEADS)
            case = dict(op="attn", b=_log(rng, 1, 64), nq=rng.choice([1, 1, 1, 2, 4, 5, 8]), hq=hq, hkv=hkv, d=d,
                        prefix=_log(rng, 1, 65536) if rng.random() < 0.9 else 0, suffix=_log(rng, 8, 2048),
                        page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["f16", "bf16"]),
                        fused=rng.random() < 0.5)
        else:
            case = dict(op="logits", rows=_log(rng, 1, 192), v=rng.choice([rng.randint(16000, 152000), 151936, 128256]),
                        type=rng.choice(["f32", "f32", "f16", "bf16"]), hist=_log(rng, 16, 8192),
                        bias=_log(rng, 1, 512), mask=rng.choice([0.01, 0.3, 0.95]), write=rng.random() < 0.6)
        w = work(case)
        if w["bytes"] <= limit[op][0] and w["flops"] <= limit[op][1]:
            return case


def _spread(count, lo, hi):
    """`count` lengths evenly spread over lo..hi (the same for every seed; their order is not)."""
    return [lo + (hi - lo) * i // max(1, count - 1) for i in range(count)] if count > 1 else [(lo + hi + 1) // 2]


def _suffixes(c):
    # a sequence's suffix holds its own queries, except where there is no prefix: there one starts with nothing
    return _spread(c["b"], c["nq"] if c["prefix"] else 0, max(c["suffix"], c["nq"]))


def work(c):
    if c["op"] == "rope":
        h = c["hq"] + 2 * c["hkv"]
        return {"bytes": c["n"] * (h * c["d"] * (SIZE[c["type"]] + SIZE[c["cache"]]) + 8),
                "flops": 3 * c["n"] * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "attn":
        rows, own_keys, e = c["b"] * c["nq"], sum(_suffixes(c)), SIZE[c["cache"]]
        return {"bytes": 2 * e * c["d"] * (c["hkv"] * (c["prefix"] + own_keys) + c["hq"] * rows),
                "flops": 4 * c["d"] * c["hq"] * (rows * c["prefix"] + c["nq"] * own_keys)}
    n = c["rows"] * c["v"]
    return {"bytes": n * SIZE[c["type"]] * (2 if c["write"] else 1) + n // 8 + 8 * sum(_spread(c["rows"], 0, c["hist"]))
            + 12 * c["rows"] * c["bias"] + 24 * c["rows"], "flops": 2 * n}


# ------------------------------------------------------------------ the inputs

def _inverse_frequencies(c):
    """theta_i in 64 bits: base^(-2i/rot), scaled for long contexts."""
    i = np.arange(c["rot"] // 2, dtype=np.float64)
    t = c["base"] ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        return t / c["factor"], 1.0
    if c["scaling"] == "bands":       # by wavelength against the trained length: short ones keep, long ones stretch
        lo, hi = 1.0, 4.0
        s = np.clip((c["orig"] * t / (2 * np.pi) - lo) / (hi - lo), 0.0, 1.0)
        return t * ((1 - s) / c["factor"] + s), 1.0
    if c["scaling"] == "yarn":        # by pair index, a ramp between the pairs that turn 32 times and once
        def pair(turns):
            return c["rot"] * math.log(c["orig"] / (turns * 2 * math.pi)) / (2 * math.log(c["base"]))
        lo, hi = max(0, math.floor(pair(32.0))), min(c["rot"] - 1, math.ceil(pair(1.0)))
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return t * (1 - ramp) + t / c["factor"] * ramp, 0.1 * math.log(c["factor"]) + 1.0
    return t, 1.0


def _prepare_rope(c, g, rng):
    n, hq, hkv, d, page = c["n"], c["hq"], c["hkv"], c["d"], c["page"]
    # the QKV product's output: q, k and v are parts of one row
    qkv = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device=DEV).to(DT[c["type"]])
    pages = (n + 2 * page - 1) // page + 3
    shape = (pages, page, hkv, d)
    cache = [torch.randn(shape, generator=g, device=DEV).to(DT[c["cache"]]) for _ in range(2)]
    first = rng.randint(0, c["top"] - n)
    pos = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(n, device=DEV) + first % page
    slots = (order[at // page] * page + at % page).to(torch.int32)
    theta, mscale = _inverse_frequencies(c)
    # the cosines and sines that a program without the kernels keeps: a table over all positions
    a = torch.arange(c["top"], dtype=torch.float64, device=DEV)[:, None] * torch.from_numpy(theta).to(DEV)
    s = dict(c=c, q=qkv[:, :hq * d].view(n, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d),
             v=qkv[:, (hq + hkv) * d:].view(n, hkv, d), pos=pos, slots=slots, cache=cache,
             cos=(torch.cos(a) * mscale).float(), sin=(torch.sin(a) * mscale).float())
    if own:
        import quantized_q4_weight_gb300 as q
        s["plan"] = q.rope_plan(c["rot"], c["base"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                                orig_len=c["orig"])
        s["kv"] = q.KvCache(*cache)
    return s


def _prepare_attn(c, g, rng):
    b, nq, hq, hkv, d, page, p = c["b"], c["nq"], c["hq"], c["hkv"], c["d"], c["page"], c["prefix"]
    dt = DT[c["cache"]]
    lens = _suffixes(c)
    rng.shuffle(lens)
    top = max(c["suffix"], nq)
    own_pages, pre_pages = (top + page - 1) // page, (p + page - 1) // page
    pages = pre_pages + sum((n + page - 1) // page for n in lens) + 2
    k = torch.randn((pages, page, hkv, d), generator=g, device=DEV).to(dt)
    v = torch.randn((pages, page, hkv, d), generator=g, device=DEV).to(dt)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    prefix_pages = order[:pre_pages].clone()
    # a table row names the pages that a sequence has; the entries after them name none that it reads
    suffix_pages = torch.zeros((b, own_pages), dtype=torch.int32)
    at, host = pre_pages, order.cpu()
    for i, n in enumerate(lens):
        m = (n + page - 1) // page
        suffix_pages[i, :m] = host[at:at + m]
        at += m
    width = (hq + 2 * hkv if c["fused"] else hq) * d
    # scores with a spread of two, as sharper heads have
    q = (2.0 * torch.randn((b * nq, width), generator=g, device=DEV)).to(dt)[:, :hq * d].view(b, nq, hq, d)
    s = dict(c=c, q=q, k=k, v=v, prefix_pages=prefix_pages, suffix_pages=suffix_pages.to(DEV),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV), top=top)
    if own:
        import quantized_q4_weight_gb300 as qg
        s["batch"] = qg.AttnBatch(b, nq, hq, qg.KvCache(k, v), p, s["prefix_pages"], s["lens"], s["suffix_pages"], top)
        s["ws"] = qg.new_workspace(s["batch"].workspace_bytes())
    return s


def _prepare_logits(c, g, rng):
    r, v, h = c["rows"], c["v"], c["hist"]
    x = (4.0 * torch.randn((r, v), generator=g, device=DEV)).to(DT[c["type"]])
    lens = _spread(r, 0, h)
    rng.shuffle(lens)
    # token ids as text has them: few are frequent (a density that falls off as 1 / id)
    u = torch.rand((r, h), generator=g, device=DEV, dtype=torch.float64)
    hist = (torch.exp(u * math.log(v)).long() - 1).clamp_(0, v - 1)
    order = torch.rand((r, v), generator=g, device=DEV)
    bias_ids = order[:, :].topk(c["bias"], dim=1).indices.contiguous()
    bias = 5.0 * torch.randn((r, c["bias"]), generator=g, device=DEV)
    words = (v + 31) // 32
    bits = torch.rand((r, words, 32), generator=g, device=DEV) < c["mask"]
    mask = (bits.long() << torch.arange(32, device=DEV)).sum(2)
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)
    rows = torch.rand((3, r), generator=g, device=DEV)
    s = dict(c=c, x=x, hist=hist, hist_len=torch.tensor(lens, dtype=torch.int32, device=DEV), bias_ids=bias_ids, bias=bias,
             bias_len=torch.full((r,), c["bias"], dtype=torch.int32, device=DEV), mask=mask,
             rep=1.0 + 0.5 * rows[0], freq=0.5 * rows[1], pres=rows[2].clone())
    if own:
        import quantized_q4_weight_gb300 as q
        s["rules"] = q.LogitsRules(r, v, history=s["hist"], history_len=s["hist_len"], repetition=s["rep"],
                                   frequency=s["freq"], presence=s["pres"], bias_ids=s["bias_ids"], bias=s["bias"],
                                   bias_len=s["bias_len"], mask=s["mask"])
        s["ws"] = q.new_workspace(s["rules"].workspace_bytes())
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    return {"rope": _prepare_rope, "attn": _prepare_attn, "logits": _prepare_logits}[case["op"]](case, g, rng)


# ------------------------------------------------------------------ the plain forms

def _pairs(x, rot, layout):
    """The rotated part's pairs as two tensors."""
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])


def _rotated(x, cos, sin, rot, layout):
    out = x.clone()
    a, b = _pairs(x, rot, layout)
    oa, ob = _pairs(out, rot, layout)
    oa.copy_(a * cos - b * sin)
    ob.copy_(a * sin + b * cos)
    return out


def _plain_rope(s):
    c = s["c"]
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, None, :], s["sin"][at][:, None, :]
    q = _rotated(s["q"].float(), cos, sin, c["rot"], c["layout"]).to(DT[c["cache"]])
    k = _rotated(s["k"].float(), cos, sin, c["rot"], c["layout"]).to(DT[c["cache"]])
    rows = s["slots"].long()
    ck, cv = s["cache"]
    ck.view(-1, c["hkv"], c["d"])[rows] = k
    cv.view(-1, c["hkv"], c["d"])[rows] = s["v"].float().to(DT[c["cache"]])
    return [q, ck, cv]


def _plain_attn(s, dt=torch.float32):
    """Both parts' scores, one softmax over them, both products with V."""
    c = s["c"]
    b, nq, hq, hkv, d, p, top = c["b"], c["nq"], c["hq"], c["hkv"], c["d"], c["prefix"], s["top"]
    grp = hq // hkv
    q = s["q"].to(dt).view(b, nq, hkv, grp, d) / math.sqrt(d)
    at = s["prefix_pages"].long()
    pk, pv = (x[at].reshape(-1, hkv, d)[:p].to(dt) for x in (s["k"], s["v"]))          # [p, hkv, d]
    at = s["suffix_pages"].long()
    sk, sv = (x[at].reshape(b, -1, hkv, d)[:, :top].to(dt) for x in (s["k"], s["v"]))  # [b, top, hkv, d]
    rows = q.permute(2, 0, 1, 3, 4).reshape(hkv, b * nq * grp, d)
    shared = torch.matmul(rows, pk.permute(1, 2, 0)).view(hkv, b, nq * grp, p)
    mine = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(hkv, b, nq * grp, d), sk.permute(2, 0, 3, 1))
    last = s["lens"].view(b, 1) - nq + torch.arange(nq, device=DEV)                     # [b, nq]: the last key each query sees
    seen = (torch.arange(top, device=DEV) <= last[:, :, None]).view(b, nq, 1, top).expand(b, nq, grp, top)
    # what a sequence does not have is not there, whatever its pages hold
    there = (torch.arange(top, device=DEV) < s["lens"][:, None])[:, :, None, None]
    sv = torch.where(there, sv, torch.zeros((), dtype=dt, device=DEV))
    mine = torch.where(seen.reshape(1, b, nq * grp, top), mine, torch.full((), NEG_INF, dtype=dt, device=DEV))
    m = mine.amax(3, keepdim=True)
    if p:
        m = torch.maximum(m, shared.amax(3, keepdim=True))
    m = torch.where(m == NEG_INF, torch.zeros((), dtype=dt, device=DEV), m)
    e_mine = torch.exp(mine - m)
    total = e_mine.sum(3, keepdim=True)
    o = torch.matmul(e_mine, sv.permute(2, 0, 1, 3))
    if p:
        e_shared = torch.exp(shared - m)
        total = total + e_shared.sum(3, keepdim=True)
        o = o + torch.matmul(e_shared.view(hkv, b * nq * grp, p), pv.permute(1, 0, 2)).view(o.shape)
    o = torch.where(total > 0, o / total, torch.zeros((), dtype=dt, device=DEV))
    return o.view(hkv, b, nq, grp, d).permute(1, 2, 0, 3, 4).reshape(b, nq, hq, d)


def _plain_logits(s):
    c = s["c"]
    r, v = c["rows"], c["v"]
    x = s["x"].float()
    # one place more than there are tokens: what lies after a row's length is counted there
    there = torch.arange(c["hist"], device=DEV) < s["hist_len"][:, None]
    ids = torch.where(there, s["hist"], v)
    count = torch.zeros((r, v + 1), device=DEV).scatter_add_(1, ids, torch.ones((), device=DEV).expand(r, c["hist"]))[:, :v]
    hit = count > 0
    rep = s["rep"][:, None]
    x = torch.where(hit, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][:, None] * count
    x = x - s["pres"][:, None] * hit.float()
    bias = torch.zeros((r, v), device=DEV).scatter_(1, s["bias_ids"], s["bias"])
    x = x + bias
    bit = torch.arange(v, device=DEV)
    allowed = (s["mask"][:, bit // 32] >> (bit % 32).to(torch.int32)) & 1
    x = torch.where(allowed.bool(), x, torch.full((), NEG_INF, device=DEV))
    best = x.amax(1)
    first = torch.where(x == best[:, None], bit, v).amin(1)
    idx = torch.where(best == NEG_INF, -1, first)
    return [idx, best] + ([x.to(DT[c["type"]])] if c["write"] else [])


def run(s):
    c = s["c"]
    if own:
        import quantized_q4_weight_gb300 as q
        if c["op"] == "rope":
            return [q.rope_kv(s["plan"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kv"])] + s["cache"]
        if c["op"] == "attn":
            return q.attn_prefix(s["q"], s["batch"], s["ws"])
        out = torch.empty_like(s["x"]) if c["write"] else None
        idx, val = q.logits_rules(s["x"], s["rules"], s["ws"], out=out)
        return [idx, val] + ([out] if c["write"] else [])
    if c["op"] == "rope":
        return _plain_rope(s)
    if c["op"] == "attn":
        return _plain_attn(s).to(DT[c["cache"]])
    return _plain_logits(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(c, s):
    """Each pair as a complex number, times mscale * exp(i pos theta)."""
    theta, mscale = _inverse_frequencies(c)
    a = s["pos"].double()[:, None] * torch.from_numpy(theta).to(DEV)
    turn = torch.polar(torch.full_like(a, mscale), a)[:, None, :]

    def rot(x):
        x, r = x.double(), c["rot"]
        pairs = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["layout"] == "half" else \
            x[..., :r].unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2) if c["layout"] == "half" else z
        return torch.cat([z.flatten(-2), x[..., r:]], -1)

    out = [rot(s["q"])]
    for cache, x in zip(s["cache"], (rot(s["k"]), s["v"].double())):
        full = cache.double().flatten(0, 1)
        full[s["slots"].long()] = x
        out.append(full.view(cache.shape))
    return out


def _exact_attn(c, s):
    """Sequence by sequence over its whole context, a softmax in 64 bits."""
    b, nq, hq, hkv, d, p = c["b"], c["nq"], c["hq"], c["hkv"], c["d"], c["prefix"]
    grp, out = hq // hkv, torch.zeros((b, nq, hq, d), dtype=torch.float64, device=DEV)
    pre = [x[s["prefix_pages"].long()].flatten(0, 1)[:p].double() for x in (s["k"], s["v"])]
    for i, n in enumerate(s["lens"].tolist()):
        mine = [x[s["suffix_pages"][i].long()].flatten(0, 1)[:n].double() for x in (s["k"], s["v"])]
        for h in range(hkv):
            keys, vals = (torch.cat([u[:, h], w[:, h]]) for u, w in zip(pre, mine))
            q = s["q"][i, :, h * grp:(h + 1) * grp].double()                     # [nq, grp, d]
            score = torch.einsum("qgd,kd->qgk", q, keys) * d ** -0.5
            hidden = torch.arange(p + n, device=DEV)[None, :] > (p + n - nq + torch.arange(nq, device=DEV))[:, None]
            score = score.masked_fill(hidden[:, None, :], NEG_INF)
            w = torch.softmax(score, -1).nan_to_num(0.0) if p + n else score     # a row that sees nothing gives nothing
            out[i, :, h * grp:(h + 1) * grp] = torch.einsum("qgk,kd->qgd", w, vals)
    return out


def _exact_logits(c, s):
    """Row by row, touched tokens one group at a time; the index has no value here (in 32 bits near ties may fall elsewhere)."""
    out = s["x"].double()
    for i, n in enumerate(s["hist_len"].tolist()):
        ids, times = torch.unique(s["hist"][i, :n], return_counts=True)
        x, r = out[i, ids], s["rep"][i].double()
        x = torch.where(x > 0, x / r, x * r)
        out[i, ids] = x - s["freq"][i].double() * times - s["pres"][i].double()
        out[i, s["bias_ids"][i]] += s["bias"][i].double()
    words = torch.from_numpy(np.unpackbits(s["mask"].cpu().numpy().view(np.uint8), axis=1, bitorder="little")).to(DEV)
    out.masked_fill_(words[:, :c["v"]] == 0, NEG_INF)
    return [None, out.max(1).values] + ([out] if c["write"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "logits": _exact_logits}[case["op"]](case, s)
