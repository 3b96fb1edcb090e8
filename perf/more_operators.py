"""Operators of a decode step over an 8-bit cache and of beam search: cases,
inputs, plain forms and references, for measuring the library's kernels.

Five operators, told apart by a case's "op":
  norm    norms of q and k for each head with rotary positions, k and v written to a paged cache;
  append  rows written to an 8-bit cache with a scale for each block of tokens and head;
  attn8   attention over such a cache, with a sliding window and first tokens that stay visible;
  beam    the best continuations over a group's beams and the vocabulary;
  fork    page tables reordered by parent, with each row's partly filled page copied.

`run` computes them in their plain form (elementary torch operations in 32
bits) or, with `own` set, through the package's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}
TOP = {"int8": 127.0, "e4m3": 448.0}
DEV = "cuda"
NEG_INF = float("-inf")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decode step of eight sequences (3B heads): latency only.
        dict(name="norm_decode8", op="norm", n=8, hq=16, hkv=2, d=128, rot=128, layout="half", base=1e6, type="f32",
             cache="bf16", page=16, top=32768),
        # A long prompt of odd length at once.
        dict(name="norm_prompt16k", op="norm", n=16381, hq=32, hkv=8, d=128, rot=128, layout="half", base=1e6,
             type="f32", cache="f16", page=64, top=131072),
        # One new token of each of 64 sequences: latency.
        dict(name="append_decode64", op="append", b=64, new=1, old=1000, ragged=False, hkv=8, d=128, type="f32",
             cache="e4m3", page=64, block=64),
        # Chunks of eight prompts of different lengths, behind what each has already.
        dict(name="append_prompts8", op="append", b=8, new=6000, old=500, ragged=True, hkv=8, d=128, type="bf16",
             cache="e4m3", page=64, block=32),
        # Two short sequences (1.5B heads): latency only.
        dict(name="attn8_short", op="attn8", b=2, nq=1, hq=12, hkv=2, d=128, top=200, window=0, sinks=0, page=16,
             block=16, cache="int8", type="f16"),
        # Eight long sequences, one token each (3B heads): the keys of few heads over all multiprocessors.
        dict(name="attn8_long8", op="attn8", b=8, nq=1, hq=16, hkv=2, d=128, top=32749, window=0, sinks=0, page=64,
             block=64, cache="int8", type="bf16"),
        # Drafts of four tokens under a sliding window with four first tokens visible, heads of 96.
        dict(name="attn8_window", op="attn8", b=32, nq=4, hq=24, hkv=4, d=96, top=20011, window=4096, sinks=4, page=128,
             block=64, cache="e4m3", type="f16"),
        # Many users of different lengths, down to nothing: bound by the cache's bytes.
        dict(name="attn8_users64", op="attn8", b=64, nq=1, hq=32, hkv=8, d=128, top=16384, window=0, sinks=0, page=64,
             block=32, cache="e4m3", type="bf16"),
        # One search of four beams, twice as many candidates: latency.
        dict(name="beam_one4", op="beam", groups=1, beams=4, v=151936, n=8, type="f32"),
        # A batch of searches of eight beams on 16-bit logits: bound by their bytes.
        dict(name="beam_batch64", op="beam", groups=64, beams=8, v=128257, n=16, type="bf16"),
        # Eight beams of one search, 28 layers of a 16-bit cache (1.5B heads): short pages, latency.
        dict(name="fork_beams8", op="fork", b=8, group=8, layers=28, hkv=2, d=128, page=16, block=0, cache="bf16", top=1500),
        # Many searches over 36 layers of an 8-bit cache (3B heads): bound by the pages' bytes.
        dict(name="fork_batch256", op="fork", b=256, group=4, layers=36, hkv=2, d=128, page=64, block=32, cache="e4m3",
             top=4000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


HEADS = [(12, 2, 128), (16, 2, 128), (14, 2, 64), (32, 8, 128), (8, 8, 64), (16, 1, 128), (24, 4, 96)]


def draw(rng):
    limit = {}
    for c in listed():
        w = work(c)
        limit[c["op"]] = [max(a, b) for a, b in zip(limit.get(c["op"], (0, 0)), (w["bytes"], w["flops"]))]
    op = rng.choice(["norm", "append", "attn8", "attn8", "beam", "fork"])
    while True:
        hq, hkv, d = rng.choice(HEADS)
        page = rng.choice([16, 32, 64, 128])
        block = rng.choice([x for x in (16, 32, 64) if x <= page])
        if op == "norm":
            t = rng.choice(["f32", "f32", "f16", "bf16"])
            case = dict(op="norm", n=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                        layout=rng.choice(["half", "interleaved"]), base=rng.choice([1e4, 5e5, 1e6]), type=t,
                        cache=rng.choice(["f16", "bf16"]) if t == "f32" else t, page=page,
                        top=rng.choice([32768, 131072]))
        elif op == "append":
            ragged = rng.random() < 0.5
            case = dict(op="append", b=_log(rng, 1, 16 if ragged else 64), new=_log(rng, 1, 6000) if ragged else rng.choice([1, 1, 4]),
                        old=_log(rng, 1, 1000), ragged=ragged, hkv=hkv, d=d, type=rng.choice(["f32", "f16", "bf16"]),
                        cache="e4m3", page=page, block=block)
        elif op == "attn8":
            nq = rng.choice([1, 1, 1, 2, 4, 5, 8])
            window = _log(rng, 16, 8192) if rng.random() < 0.4 else 0
            case = dict(op="attn8", b=_log(rng, 1, 64), nq=nq, hq=hq, hkv=hkv, d=d, top=_log(rng, 8, 32768),
                        window=window, sinks=rng.choice([0, 1, 4, 16]) if window else 0, page=page, block=block,
                        cache=rng.choice(["int8", "e4m3"]), type=rng.choice(["f16", "bf16"]))
        elif op == "beam":
            beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
            case = dict(op="beam", groups=_log(rng, 1, 64), beams=beams, v=rng.choice([rng.randint(16000, 152000), 151936, 128256]),
                        n=rng.choice([beams, 2 * beams]), type=rng.choice(["f32", "f16", "bf16"]))
        else:
            group = rng.choice([1, 2, 4, 5, 8])
            cache = rng.choice(["f16", "bf16", "int8", "e4m3"])
            case = dict(op="fork", b=group * _log(rng, 1, 64), group=group, layers=rng.choice([1, 24, 28, 32, 36]), hkv=hkv, d=d,
                        page=page, block=block if SIZE[cache] == 1 else 0, cache=cache, top=_log(rng, 64, 4000))
        w = work(case)
        if w["bytes"] <= limit[op][0] and w["flops"] <= limit[op][1]:
            return case


def _spread(count, lo, hi):
    """`count` lengths evenly spread over lo..hi (the same for every seed; their order is not)."""
    return [lo + (hi - lo) * i // max(1, count - 1) for i in range(count)] if count > 1 else [(lo + hi + 1) // 2]


def _seen(n, nq, window, sinks):
    """Keys that the queries of a sequence of n rows see together."""
    if not window:
        return n
    first = max(0, n - nq + 1 - window)
    return n - first + min(first, sinks)


def work(c):
    if c["op"] == "norm":
        h = c["hq"] + 2 * c["hkv"]
        return {"bytes": c["n"] * (h * c["d"] * (SIZE[c["type"]] + SIZE[c["cache"]]) + 8),
                "flops": c["n"] * (c["hq"] + c["hkv"]) * (4 * c["d"] + 3 * c["rot"])}
    if c["op"] == "append":
        n = sum(_new(c))
        return {"bytes": 2 * c["hkv"] * n * (c["d"] * (SIZE[c["type"]] + 1) + 8 / c["block"]), "flops": 6 * n * c["hkv"] * c["d"]}
    if c["op"] == "attn8":
        lens = _spread(c["b"], 0, max(c["top"], c["nq"]))
        keys = sum(_seen(n, c["nq"], c["window"], c["sinks"]) for n in lens)
        return {"bytes": 2 * c["hkv"] * keys * (c["d"] + 4 / c["block"]) + 2 * SIZE[c["type"]] * c["b"] * c["nq"] * c["hq"] * c["d"],
                "flops": 4 * c["d"] * c["hq"] * c["nq"] * keys}
    if c["op"] == "beam":
        n = c["groups"] * c["beams"] * c["v"]
        return {"bytes": n * SIZE[c["type"]] + 16 * c["groups"] * c["n"], "flops": 4 * n}
    rows = sum(n % c["page"] for n in _spread(c["b"], 0, c["top"]))
    return {"bytes": 4 * c["layers"] * rows * c["hkv"] * (c["d"] * SIZE[c["cache"]] + (4 / c["block"] if c["block"] else 0))
            + 8 * sum(-(-n // c["page"]) for n in _spread(c["b"], 0, c["top"])), "flops": 0}


# ------------------------------------------------------------------ the inputs

def _new(c):
    """New rows of each sequence."""
    return _spread(c["b"], 0, c["new"]) if c["ragged"] else [c["new"]] * c["b"]


def _prepare_norm(c, g, rng):
    n, hq, hkv, d, page = c["n"], c["hq"], c["hkv"], c["d"], c["page"]
    # the QKV product's output: q, k and v are parts of one row
    qkv = (3.0 * torch.randn((n, (hq + 2 * hkv) * d), generator=g, device=DEV)).to(DT[c["type"]])
    pages = (n + 2 * page - 1) // page + 3
    cache = [torch.randn((pages, page, hkv, d), generator=g, device=DEV).to(DT[c["cache"]]) for _ in range(2)]
    first = rng.randint(0, c["top"] - n)
    pos = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(n, device=DEV) + first % page
    slots = (order[at // page] * page + at % page).to(torch.int32)
    weights = [1.0 + 0.25 * torch.randn((d,), generator=g, device=DEV) for _ in range(2)]
    # the cosines and sines that a program without the kernels keeps: a table over all positions
    theta = c["base"] ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV) / c["rot"])
    a = torch.arange(c["top"], dtype=torch.float64, device=DEV)[:, None] * theta
    s = dict(c=c, q=qkv[:, :hq * d].view(n, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d),
             v=qkv[:, (hq + hkv) * d:].view(n, hkv, d), pos=pos, slots=slots, cache=cache, weights=weights, eps=1e-6,
             cos=torch.cos(a).float(), sin=torch.sin(a).float())
    if own:
        import quantized_q4_weight_gb300 as q
        s["plan"] = q.rope_plan(c["rot"], c["base"], layout=c["layout"])
        s["norm"] = q.QkNorm(weights[0], weights[1], s["eps"])
        s["kv"] = q.KvCache(*cache)
    return s


def _codes(x, kind):
    """Values already divided by their scale as codes."""
    x = x.clamp(-TOP[kind], TOP[kind])
    return torch.round(x).to(torch.int8) if kind == "int8" else x.to(torch.float8_e4m3fn)


def _cache8(c, pages, g):
    """Codes [pages][page][heads][d] and scales [pages][blocks][heads] of a cache full of values."""
    page, block, hkv, d = c["page"], c["block"], c["hkv"], c["d"]
    out = []
    for _ in range(2):
        scale = (0.5 + torch.rand((pages, page // block, hkv), generator=g, device=DEV)) * 3.0 / TOP[c["cache"]]
        codes = torch.empty((pages, page, hkv, d), dtype=DT[c["cache"]], device=DEV)
        step = max(1, (1 << 26) // (page * hkv * d))
        for i in range(0, pages, step):
            x = torch.randn((min(step, pages - i), page, hkv, d), generator=g, device=DEV) * (TOP[c["cache"]] / 3.0)
            codes[i:i + step] = _codes(x, c["cache"])
        out += [codes, scale]
    return out


def _tables(lens, page, columns, pages, g, spare=0):
    """A table row names the pages that a sequence has; the entries after them name none that it reads."""
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    host, table, at = order.cpu(), torch.zeros((len(lens), max(1, columns)), dtype=torch.int32), 0
    for i, n in enumerate(lens):
        m = -(-n // page)
        table[i, :m] = host[at:at + m]
        at += m
    return table.to(DEV), order[at:at + spare].clone()


def _prepare_append(c, g, rng):
    b, hkv, d, page = c["b"], c["hkv"], c["d"], c["page"]
    new, old = _new(c), _spread(b, 0, c["old"])
    rng.shuffle(new)
    rng.shuffle(old)
    lens = [x + y for x, y in zip(new, old)]
    columns = -(-(max(new) + max(old)) // page)
    # as many pages for every order of the lengths
    pages = sum(-(-n // page) for n in new + old) + 2
    k, ks, v, vs = _cache8(c, pages, g)
    table, _ = _tables(lens, page, columns, pages, g)
    n = sum(new)
    # k and v are parts of the QKV product's rows
    qkv = (2.0 * torch.randn((max(1, n), 4 * hkv * d), generator=g, device=DEV)).to(DT[c["type"]])[:n]
    first = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    s = dict(c=c, k=qkv[:, 2 * hkv * d:3 * hkv * d].view(n, hkv, d), v=qkv[:, 3 * hkv * d:].view(n, hkv, d), first=first,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV), table=table, most=max(new), cache=[k, ks, v, vs])
    if own:
        import quantized_q4_weight_gb300 as q
        s["batch"] = q.Kv8Batch(b, 1 if c["ragged"] else c["new"], hkv, q.Kv8Cache(k, v, ks, vs), s["lens"], table, columns * page)
    return s


def _prepare_attn8(c, g, rng):
    b, nq, hq, d, page = c["b"], c["nq"], c["hq"], c["d"], c["page"]
    top = max(c["top"], nq)
    lens = _spread(b, 0, top)
    rng.shuffle(lens)
    columns, pages = -(-top // page), sum(-(-n // page) for n in lens) + 2
    k, ks, v, vs = _cache8(c, pages, g)
    table, _ = _tables(lens, page, columns, pages, g)
    # scores with a spread of two, as sharper heads have
    q = (2.0 * torch.randn((b, nq, hq, d), generator=g, device=DEV)).to(DT[c["type"]])
    s = dict(c=c, q=q, cache=[k, ks, v, vs], table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), top=top)
    if own:
        import quantized_q4_weight_gb300 as qg
        s["batch"] = qg.Kv8Batch(b, nq, hq, qg.Kv8Cache(k, v, ks, vs), s["lens"], table, top, window=c["window"], sinks=c["sinks"])
        s["ws"] = qg.new_workspace(s["batch"].workspace_bytes())
    return s


def _prepare_beam(c, g, rng):
    rows = c["groups"] * c["beams"]
    x = (3.0 * torch.randn((rows, c["v"]), generator=g, device=DEV)).to(DT[c["type"]])
    # running scores: sums of logarithms of probabilities, the beams of a search near one another
    scores = -20.0 * torch.rand((c["groups"], 1), generator=g, device=DEV) - 2.0 * torch.rand((c["groups"], c["beams"]), generator=g, device=DEV)
    s = dict(c=c, x=x, scores=scores.contiguous())
    if own:
        import quantized_q4_weight_gb300 as q
        s["step"] = q.BeamStep(c["groups"], c["beams"], c["v"], c["n"], s["scores"])
        s["ws"] = q.new_workspace(s["step"].workspace_bytes())
    return s


def _prepare_fork(c, g, rng):
    b, layers, page, hkv, d = c["b"], c["layers"], c["page"], c["hkv"], c["d"]
    # rows of a group may end anywhere: the tails, which are what is copied, run over all lengths of a page
    lens = _spread(b, 0, c["top"])
    rng.shuffle(lens)
    columns = -(-c["top"] // page) + 1
    # only a row's last page is its own: the others are shared by the searches that began with them
    shared = 64
    pages = shared + 2 * b + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = order[torch.randint(0, shared, (b, columns), generator=g, device=DEV)].contiguous()
    table[torch.arange(b, device=DEV), torch.tensor([n // page for n in lens], device=DEV)] = order[shared:shared + b]
    # a group's children: of parents of their own group, as a permutation would have each length once
    parents = torch.tensor([i - i % c["group"] + j for i, j in zip(range(b), (rng.randrange(c["group"]) for _ in range(b)))],
                           dtype=torch.int32, device=DEV)
    parents = torch.tensor(rng.sample(range(b), b), dtype=torch.int32, device=DEV) if c["group"] == 1 else parents
    if c["block"]:
        many = dict(c, hkv=hkv)
        k, ks, v, vs = (x.view(layers, pages, *x.shape[1:]) for x in _cache8(many, layers * pages, g))
        cache = [k, v, ks, vs]
    else:
        cache = [torch.randn((layers, pages, page, hkv, d), generator=g, device=DEV).to(DT[c["cache"]]) for _ in range(2)]
    s = dict(c=c, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), parents=parents,
             fresh=order[shared + b:shared + 2 * b].clone(), table_out=torch.zeros_like(table),
             lens_out=torch.zeros((b,), dtype=torch.int32, device=DEV))
    if own:
        import quantized_q4_weight_gb300 as q
        made = [q.Kv8Cache(*x) if c["block"] else q.KvCache(*x) for x in zip(*cache)]
        s["pool"] = q.PagePool(made)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    return {"norm": _prepare_norm, "append": _prepare_append, "attn8": _prepare_attn8, "beam": _prepare_beam,
            "fork": _prepare_fork}[case["op"]](case, g, rng)


# ------------------------------------------------------------------ the plain forms

def _pairs(x, rot, layout):
    """The rotated part's pairs as two tensors."""
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])


def _normed_rotated(x, w, s, cos, sin):
    c = s["c"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
    out = x.clone()
    a, b = _pairs(x, c["rot"], c["layout"])
    oa, ob = _pairs(out, c["rot"], c["layout"])
    oa.copy_(a * cos - b * sin)
    ob.copy_(a * sin + b * cos)
    return out


def _plain_norm(s):
    c, pos = s["c"], s["pos"].long()
    cos, sin = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]
    q = _normed_rotated(s["q"], s["weights"][0], s, cos, sin).to(DT[c["cache"]])
    at = s["slots"].long()
    s["cache"][0].view(-1, c["hkv"], c["d"])[at] = _normed_rotated(s["k"], s["weights"][1], s, cos, sin).to(DT[c["cache"]])
    s["cache"][1].view(-1, c["hkv"], c["d"])[at] = s["v"].to(DT[c["cache"]])
    return [q] + s["cache"]


def _write_blocks(s, x, codes, scale):
    """The touched blocks of all sequences as one padded tensor [sequences][blocks][rows][heads][d], formed anew and put back."""
    c = s["c"]
    b, page, block, hkv, d = c["b"], c["page"], c["block"], c["hkv"], c["d"]
    first = s["first"].long()
    new, lens = first[1:] - first[:-1], s["lens"].long()
    old = lens - new
    most = (s["most"] + 2 * block - 2) // block                         # blocks that so many rows can touch
    at = old[:, None] // block + torch.arange(most, device=DEV)         # block number in the sequence
    there = (at * block < lens[:, None]) & (new > 0)[:, None]
    per = page // block
    pages = torch.gather(s["table"].long(), 1, (at // per).clamp(max=s["table"].shape[1] - 1))
    # blocks that are not there go to one place behind the others
    flat = torch.where(there, pages * per + at % per, codes.shape[0] * per)
    rows = at[:, :, None] * block + torch.arange(block, device=DEV)     # row number in the sequence
    fresh = (rows >= old[:, None, None]) & (rows < lens[:, None, None]) & there[:, :, None]
    token = torch.where(fresh, first[:-1, None, None] + rows - old[:, None, None], 0)
    xs = torch.where(fresh[..., None, None], x[token].float(), torch.zeros((), device=DEV))
    had = (at * block < old[:, None]) & there
    spare = lambda t: torch.cat([t, t[:1]])  # noqa: E731
    was = spare(codes.view(torch.uint8).view(-1, block, hkv, d))
    was_scale = spare(scale.view(-1, hkv))
    c0 = was[flat].view(codes.dtype)
    s0 = torch.where(had[..., None], was_scale[flat], torch.zeros((), device=DEV))
    top = torch.full((), TOP[c["cache"]], device=DEV)
    s1 = torch.maximum(s0, xs.abs().amax((2, 4)) / top)
    by, was_by = 1.0 / s1[:, :, None, :, None], s0[:, :, None, :, None]
    held = torch.where(s1[:, :, None, :, None] > was_by, c0.float() * (was_by * by), c0.float())
    value = torch.where(fresh[..., None, None], xs * by, held)
    value = torch.where(s1[:, :, None, :, None] > 0, value, torch.zeros((), device=DEV))
    made = _codes(value, c["cache"]).view(torch.uint8)
    keep = (rows < lens[:, None, None])[..., None, None]
    was[flat] = torch.where(keep, made, c0.view(torch.uint8))
    was_scale[flat] = s1
    codes.view(torch.uint8).view(-1, block, hkv, d).copy_(was[:-1])
    scale.view(-1, hkv).copy_(was_scale[:-1])


def _plain_append(s):
    k, ks, v, vs = s["cache"]
    if s["k"].shape[0]:
        _write_blocks(s, s["k"], k, ks)
        _write_blocks(s, s["v"], v, vs)
    return s["cache"]


def _plain_attn8(s):
    c = s["c"]
    b, nq, hq, hkv, d, page, block = c["b"], c["nq"], c["hq"], c["hkv"], c["d"], c["page"], c["block"]
    grp, cols = hq // hkv, s["table"].shape[1]
    n = cols * page
    at = s["table"].long()

    def values(codes, scale):
        x = codes.view(torch.uint8)[at].view(codes.dtype).float().view(b, cols, page // block, block, hkv, d)
        return (x * scale[at][:, :, :, None, :, None]).view(b, n, hkv, d).permute(0, 2, 1, 3)

    k, ks, v, vs = s["cache"]
    pos = torch.arange(n, device=DEV)
    last = s["lens"][:, None] - nq + torch.arange(nq, device=DEV)         # a query's own position
    seen = pos <= last[..., None]
    if c["window"]:
        seen = seen & ((pos > last[..., None] - c["window"]) | (pos < c["sinks"]))
    seen = seen[:, None, :, None, :]
    q = s["q"].float().view(b, nq, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, nq * grp, d)
    x = torch.matmul(q, values(k, ks).transpose(2, 3)).mul_(d ** -0.5).view(b, hkv, nq, grp, n)
    x = torch.where(seen, x, torch.full((), NEG_INF, device=DEV))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG_INF, torch.zeros((), device=DEV), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(b, hkv, nq * grp, n), values(v, vs)).view(b, hkv, nq, grp, d)
    o = torch.where(total > 0, o / total, torch.zeros((), device=DEV))
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(b * nq, hq)
    return [o.permute(0, 2, 1, 3, 4).reshape(b, nq, hq, d).to(DT[c["type"]]), lse]


def _plain_beam(s):
    c = s["c"]
    x = s["x"].float()
    m = x.amax(1, keepdim=True)
    # sums over the vocabulary and the order of near scores need more than 32 bits
    lse = m.double() + torch.log(torch.exp(x - m).sum(1, keepdim=True, dtype=torch.float64))
    score = (x.double() - lse + s["scores"].double().view(-1, 1)).view(c["groups"], c["beams"] * c["v"])
    best, at = torch.sort(score, dim=1, descending=True, stable=True)
    best, at = best[:, :c["n"]], at[:, :c["n"]]
    row = at // c["v"] + c["beams"] * torch.arange(c["groups"], device=DEV)[:, None]
    return [best.float(), at % c["v"], row.to(torch.int32)]


def _plain_fork(s):
    c = s["c"]
    b, page = c["b"], c["page"]
    parents = s["parents"].long()
    lens = s["lens"][parents]
    full = (lens // page).long()
    cols = torch.arange(s["table"].shape[1], device=DEV)
    table = s["table"][parents]
    last = torch.gather(table, 1, full[:, None])[:, 0].long()
    # up to the page of the next row
    table = torch.where(cols < full[:, None], table, torch.where(cols == full[:, None], s["fresh"][:, None], s["table_out"]))
    rows = torch.arange(page, device=DEV) < (lens % page)[:, None]
    to = s["fresh"].long()
    for x in s["cache"][:2]:
        x = x.view(torch.uint8)
        x[:, to] = torch.where(rows[None, :, :, None, None], x[:, last], x[:, to])
    if c["block"]:
        had = (torch.arange(page // c["block"], device=DEV) * c["block"] < (lens % page)[:, None])[None, :, :, None]
        for x in s["cache"][2:]:
            x[:, to] = torch.where(had, x[:, last], x[:, to])
    s["table_out"].copy_(table)
    s["lens_out"].copy_(lens)
    return [s["table_out"], s["lens_out"]] + s["cache"]


def run(s):
    c = s["c"]
    if own:
        import quantized_q4_weight_gb300 as q
        if c["op"] == "norm":
            return [q.norm_rope_kv(s["plan"], s["norm"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kv"])] + s["cache"]
        if c["op"] == "append":
            q.kv8_append(s["k"], s["v"], s["batch"], first=s["first"] if c["ragged"] else None, max_new=s["most"])
            return s["cache"]
        if c["op"] == "attn8":
            lse = torch.empty((c["b"] * c["nq"], c["hq"]), device=DEV)
            return [q.attn_kv8(s["q"], s["batch"], s["ws"], lse=lse), lse]
        if c["op"] == "beam":
            return list(q.beam_select(s["x"], s["step"], s["ws"]))
        q.fork_pages(s["pool"], s["parents"], s["lens"], s["table"], s["fresh"], s["table_out"], s["lens_out"])
        return [s["table_out"], s["lens_out"]] + s["cache"]
    return {"norm": _plain_norm, "append": _plain_append, "attn8": _plain_attn8, "beam": _plain_beam,
            "fork": _plain_fork}[c["op"]](s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(c, s):
    """Each pair of the normed head as a complex number, times exp(i pos theta)."""
    theta = torch.tensor([c["base"] ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)], dtype=torch.float64, device=DEV)
    a = s["pos"].double()[:, None] * theta
    turn = torch.polar(torch.ones_like(a), a)[:, None, :]

    def rot(x, w):
        x, r = x.double(), c["rot"]
        x = x / (x.square().sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt() * w.double()
        pairs = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["layout"] == "half" else \
            x[..., :r].unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2) if c["layout"] == "half" else z
        return torch.cat([z.flatten(-2), x[..., r:]], -1)

    out = [rot(s["q"], s["weights"][0])]
    for cache, x in zip(s["cache"], (rot(s["k"], s["weights"][1]), s["v"].double())):
        full = cache.double().flatten(0, 1)
        full[s["slots"].long()] = x
        out.append(full.view(cache.shape))
    return out


def _nearest_e4m3(x):
    """The nearest value of four exponent and three fraction bits (1 / 512 the smallest), ties to even."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(x / step) * step


def _exact_append(c, s):
    """Sequence by sequence and block by block."""
    out, first = [], s["first"].tolist()
    for x, codes, scale in ((s["k"], s["cache"][0], s["cache"][1]), (s["v"], s["cache"][2], s["cache"][3])):
        codes, scale = codes.float().double(), scale.double()
        for i, n in enumerate(s["lens"].tolist()):
            old = n - (first[i + 1] - first[i])
            for j in range(old // c["block"], -(-n // c["block"])):
                lo, hi, at = j * c["block"], min(n, (j + 1) * c["block"]), int(s["table"][i, j * c["block"] // c["page"]])
                if max(lo, old) >= hi:
                    continue
                part = x[first[i] + max(lo, old) - old:first[i] + hi - old].double()
                u, r = lo % c["page"] // c["block"], lo % c["page"]
                was = scale[at, u] if old > lo else torch.zeros_like(scale[at, u])
                now = torch.maximum(was, part.abs().amax((0, 2)) / TOP[c["cache"]])
                if old > lo:
                    held = codes[at, r:r + old - lo]
                    codes[at, r:r + old - lo] = torch.where((now > was)[:, None], _nearest_e4m3(held * (was / now)[:, None]), held)
                codes[at, r + max(lo, old) - lo:r + hi - lo] = _nearest_e4m3(part / now[:, None])
                scale[at, u] = now
        out += [codes, scale]
    return out


def _exact_attn8(c, s):
    """Sequence by sequence over the rows that its queries see, a softmax in 64 bits."""
    b, nq, hq, hkv, d = c["b"], c["nq"], c["hq"], c["hkv"], c["d"]
    grp = hq // hkv
    out = torch.zeros((b, nq, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, nq, hq), NEG_INF, dtype=torch.float64, device=DEV)
    k, ks, v, vs = s["cache"]
    for i, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        at = s["table"][i, :-(-n // c["page"])].long()
        keys, vals = ((x.view(torch.uint8)[at].view(x.dtype).float().double().unflatten(1, (-1, c["block"])) * y[at].double()[:, :, None, :, None])
                      .flatten(0, 2)[:n] for x, y in ((k, ks), (v, vs)))
        for j in range(nq):
            p = n - nq + j
            rows = torch.arange(p + 1, device=DEV)
            if c["window"]:
                rows = rows[(rows > p - c["window"]) | (rows < c["sinks"])]
            if p < 0 or not rows.numel():
                continue
            q = s["q"][i, j].double().view(hkv, grp, d)
            score = torch.einsum("hgd,khd->hgk", q, keys[rows]) / math.sqrt(d)
            lse[i, j] = torch.logsumexp(score, -1).view(hq)
            out[i, j] = torch.einsum("hgk,khd->hgd", torch.softmax(score, -1), vals[rows]).reshape(hq, d)
    return [out, lse.view(b * nq, hq)]


def _exact_beam(c, s):
    """Group by group."""
    best = []
    for i in range(c["groups"]):
        x = torch.log_softmax(s["x"][i * c["beams"]:(i + 1) * c["beams"]].double(), 1) + s["scores"][i].double()[:, None]
        best.append(torch.topk(x.flatten(), c["n"]).values)
    return [torch.stack(best), None, None]


def _exact_fork(c, s):
    """Row by row; the tables and lengths are whole numbers, copies as they are."""
    table, lens, page = s["table"].tolist(), s["lens"].tolist(), c["page"]
    out = [x.float() for x in s["cache"]]
    for to, parent in zip(s["fresh"].tolist(), s["parents"].tolist()):
        n = lens[parent] % page
        last = table[parent][lens[parent] // page]
        for x in out[:2]:
            x[:, to, :n] = x[:, last, :n]
        for x in out[2:]:
            m = -(-n // c["block"])
            x[:, to, :m] = x[:, last, :m]
    # whole numbers in an int8 cache have no value here
    return [None, None] + [None if y.dtype == torch.int8 else x for x, y in zip(out, s["cache"])]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attn8": _exact_attn8, "beam": _exact_beam,
            "fork": _exact_fork}[case["op"]](case, s)
