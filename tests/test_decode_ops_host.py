"""The argument checks of the operators between the GEMVs: a refused call
returns its status before any CUDA call, so these run without a GPU.  Pointers
are numbers that nothing follows."""
import copy
import ctypes
import gc
import pickle

import pytest

import quantized_q4_weight_gb300 as q

OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from quantized_q4_weight_gb300 import _build
    _build.build()
    return q.lib()


def cache(**kw):
    f = dict(k=BIG, v=2 * BIG, type=q.BF16, n_pages=100, page_size=16, n_heads=2, head_dim=128, page_stride=4096,
             row_stride=256, head_stride=128)
    f.update(kw)
    return q.KvCacheStruct(**f)


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(type=q.F32), INVALID), (dict(type=9), INVALID),
              (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), INVALID),
              (dict(n_heads=0), INVALID), (dict(head_dim=12), INVALID), (dict(head_dim=264), INVALID),
              (dict(head_dim=0), INVALID), (dict(page_stride=-8), INVALID), (dict(row_stride=1 << 62), INVALID),
              (dict(k=BIG + 8), MISALIGNED), (dict(row_stride=260), MISALIGNED), (dict(head_stride=129), MISALIGNED)]


def test_rope_init(L):
    def init(**kw):
        f = dict(rot_dim=128, layout=0, scaling=0, base=1e4, factor=2.0, orig_len=4096.0, low=1.0, high=4.0, mscale=0.0)
        f.update(kw)
        plan = q.RopePlan()
        return L.qgemv_rope_init(ctypes.byref(q.RopeConfig(**f)), ctypes.byref(plan)), plan

    nan, inf = float("nan"), float("inf")
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(layout=2), dict(scaling=4), dict(scaling=-1),
                dict(base=1.0), dict(base=nan), dict(base=inf), dict(mscale=nan), dict(scaling=1, factor=0.5),
                dict(scaling=1, factor=inf), dict(scaling=2, orig_len=0.0), dict(scaling=2, low=4.0),
                dict(scaling=3, low=0.0), dict(scaling=3, high=inf), dict(scaling=3, orig_len=nan)):
        assert init(**bad)[0] == INVALID, bad
    assert L.qgemv_rope_init(None, ctypes.byref(q.RopePlan())) == INVALID
    s, p = init()
    assert s == OK and p.mscale == 1.0 and p.rot_dim == 128
    # the frequencies in whole units of 2^-64 turns, to the 53 bits of a double
    import math
    for i in range(64):
        want = 1e4 ** (-2 * i / 128) / (2 * math.pi) * 2 ** 64
        assert abs(p.turns[i] - want) <= 2.0 ** -50 * want + 0.5
    assert all(p.turns[i] == 0 for i in range(64, 128))
    assert abs(init(scaling=3, factor=4.0, high=32.0)[1].mscale - (0.1 * math.log(4) + 1)) < 1e-6
    assert init(scaling=3, factor=4.0, high=32.0, mscale=1.5)[1].mscale == 1.5
    lin, plain = init(scaling=1, factor=4.0)[1], init()[1]
    assert all(abs(lin.turns[i] * 4 - plain.turns[i]) <= 2.0 ** -50 * plain.turns[i] + 4 for i in range(64))
    # the ramps' ends: short wavelengths keep their frequency, long ones are divided
    for sc, hi in ((2, 4.0), (3, 32.0)):
        p = init(scaling=sc, factor=8.0, high=hi)[1]
        assert p.turns[0] == plain.turns[0] and abs(p.turns[63] * 8 - plain.turns[63]) <= 2.0 ** -50 * plain.turns[63] + 8
        assert all(p.turns[i] >= p.turns[i + 1] for i in range(63))


def rope(L, c=None, **kw):
    plan = q.rope_plan(kw.pop("rot", 128), 1e4)
    f = dict(plan=plan.address, q=4096, k=BIG // 2, v=BIG // 2 + (1 << 30), t=q.F32, qs=1536, ks=256, vs=256, pos=1 << 34,
             slots=1 << 35, n=10, hq=12, d=128, o=1 << 36, ot=q.BF16, os=1536)
    f.update(kw)
    c = cache() if c is None else c
    return L.qgemv_rope_kv(f["plan"], f["q"], f["k"], f["v"], f["t"], f["qs"], f["ks"], f["vs"], f["pos"], f["slots"],
                           f["n"], f["hq"], f["d"], f["o"], f["ot"], f["os"], ctypes.addressof(c) if c else None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(plan=None), INVALID), (dict(q=None, k=None, v=None), INVALID), (dict(v=None), INVALID),
    (dict(k=None), INVALID), (dict(pos=None), INVALID), (dict(slots=None), INVALID), (dict(t=3), INVALID),
    (dict(ot=-1), INVALID), (dict(o=None), INVALID), (dict(n=0), INVALID), (dict(n=1 << 32), INVALID),
    (dict(hq=0), INVALID), (dict(d=127), INVALID), (dict(d=64), INVALID), (dict(rot=256), INVALID),
    (dict(qs=1535), INVALID), (dict(os=100), INVALID), (dict(qs=-1536), INVALID), (dict(ks=1 << 60), INVALID),
    (dict(q=4098), MISALIGNED), (dict(o=(1 << 36) + 1), MISALIGNED), (dict(k=BIG // 2 + 2), MISALIGNED),
    (dict(pos=(1 << 34) + 2), MISALIGNED), (dict(slots=(1 << 35) + 1), MISALIGNED),
    (dict(o=4096, ot=q.BF16), INVALID),                 # over q with another type
    (dict(o=4096 + 4, ot=q.F32), INVALID),              # shifted over q
    (dict(o=BIG), INVALID), (dict(q=2 * BIG), INVALID), (dict(k=BIG), INVALID),      # over the cache
    (dict(o=BIG // 2), INVALID), (dict(o=1 << 34), INVALID), (dict(o=1 << 35), INVALID)])
def test_rope_refusals(L, bad, status):
    assert rope(L, **bad) == status


@pytest.mark.parametrize("bad,status", BAD_CACHES + [(dict(n_pages=1 << 28, page_size=16, page_stride=0), INVALID)])
def test_rope_refuses_caches(L, bad, status):
    assert rope(L, cache(**bad)) == status


def attn(L, c=None, b=None, ws_bytes=BIG // 4, **kw):
    f = dict(q=1 << 30, qt=1536, qh=128, o=1 << 31, ot=q.BF16, os=1536, oh=128, lse=1 << 32, ws=1 << 38)
    f.update(kw)
    c = cache() if c is None else c
    b = batch() if b is None else b
    return L.qgemv_attn_prefix(f["q"], f["qt"], f["qh"], ctypes.addressof(c), ctypes.addressof(b), f["o"], f["ot"],
                               f["os"], f["oh"], f["lse"], f["ws"], ws_bytes, None)


def batch(**kw):
    f = dict(n_seqs=4, n_q=2, n_q_heads=12, prefix_len=100, prefix_pages=4096, suffix_len=8192, suffix_pages=1 << 16,
             suffix_pages_stride=10, max_suffix=150, scale=0.0)
    f.update(kw)
    return q.AttnBatchStruct(**f)


def attn_ws(L, b, c):
    return L.qgemv_attn_workspace_bytes(ctypes.addressof(b), ctypes.addressof(c))


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_attn_refuses_caches(L, bad, status):
    assert attn(L, c=cache(**bad)) == status
    assert attn_ws(L, batch(), cache(**bad)) == 0


@pytest.mark.parametrize("bad", [dict(n_seqs=0), dict(n_q=0), dict(n_q=9), dict(n_q_heads=0), dict(n_q_heads=13),
                                 dict(prefix_len=-1), dict(prefix_len=2 ** 31 - 1), dict(max_suffix=-1),
                                 dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                 dict(n_seqs=1 << 20, n_q=8, n_q_heads=4096)])
def test_attn_refuses_batches(L, bad):
    assert attn(L, b=batch(**bad)) == INVALID
    assert attn_ws(L, batch(**bad), cache()) == 0


@pytest.mark.parametrize("bad", [dict(prefix_pages=None), dict(suffix_len=None), dict(suffix_pages=None),
                                 dict(suffix_pages_stride=-1)])
def test_attn_refuses_tables(L, bad):
    assert attn(L, b=batch(**bad)) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(ot=q.F16), INVALID), (dict(ot=7), INVALID),
    (dict(qt=-8), INVALID), (dict(os=1 << 60), INVALID), (dict(q=(1 << 30) + 8), MISALIGNED), (dict(qt=1540), MISALIGNED),
    (dict(qh=100), MISALIGNED), (dict(o=(1 << 31) + 1), MISALIGNED), (dict(lse=(1 << 32) + 2), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=20000), WORKSPACE), (dict(ws=(1 << 38) + 8), MISALIGNED),
    (dict(o=1 << 30), INVALID), (dict(o=1 << 38), INVALID), (dict(o=BIG), INVALID), (dict(lse=1 << 31), INVALID),
    (dict(lse=1 << 38), INVALID), (dict(ws=1 << 30), INVALID), (dict(o=8192), INVALID)])
def test_attn_refusals(L, bad, status):
    assert attn(L, **bad) == status


def test_attn_workspace_grows_with_the_batch(L):
    def need(**kw):
        return attn_ws(L, batch(**kw), cache())
    assert need() > 16384
    assert need(prefix_len=0, max_suffix=0) == 16384 and need(n_seqs=8, prefix_len=100000) > need(prefix_len=100000) / 2


def logits(L, ws_bytes=16384, s=None, **kw):
    f = dict(x=1 << 30, t=q.F32, xs=1000, o=1 << 31, os=1000, idx=1 << 32, val=1 << 33, ws=1 << 38)
    f.update(kw)
    s = spec() if s is None else s
    return L.qgemv_logits_rules(f["x"], f["t"], f["xs"], ctypes.addressof(s), f["o"], f["os"], f["idx"], f["val"],
                                f["ws"], ws_bytes, None)


def spec(**kw):
    f = dict(rows=3, vocab=1000, history=4096, history_stride=50, history_len=8192, max_history=50, repetition=16384,
             frequency=16640, presence=16896, bias_ids=20480, bias=24576, bias_stride=4, bias_len=28672, max_bias=4,
             mask=32768, mask_stride=32)
    f.update(kw)
    return q.LogitsSpec(**f)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=0), INVALID), (dict(vocab=0), INVALID), (dict(vocab=1 << 31), INVALID), (dict(history=None), INVALID),
    (dict(history_len=None), INVALID), (dict(max_history=-1), INVALID), (dict(max_history=1 << 20), INVALID),
    (dict(history_stride=-1), INVALID), (dict(bias=None), INVALID), (dict(bias_ids=None), INVALID),
    (dict(bias_len=None), INVALID), (dict(max_bias=4096), INVALID), (dict(mask_stride=31), INVALID),
    (dict(history=4100), MISALIGNED), (dict(bias_ids=20484), MISALIGNED), (dict(mask=32769), MISALIGNED),
    (dict(repetition=16385), MISALIGNED), (dict(history_len=8193), MISALIGNED), (dict(bias_len=28673), MISALIGNED),
    (dict(bias=24577), MISALIGNED), (dict(mask=1 << 31), INVALID), (dict(history=1 << 32), INVALID)])
def test_logits_refuses_specs(L, bad, status):
    assert logits(L, s=spec(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), INVALID), (dict(t=5), INVALID), (dict(idx=None), INVALID), (dict(val=None), INVALID),
    (dict(o=None, idx=None, val=None), INVALID), (dict(xs=999), INVALID), (dict(os=999), INVALID),
    (dict(x=(1 << 30) + 2), MISALIGNED), (dict(o=(1 << 31) + 1), MISALIGNED), (dict(idx=(1 << 32) + 4), MISALIGNED),
    (dict(val=(1 << 33) + 2), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16383), WORKSPACE),
    (dict(ws=(1 << 38) + 4), MISALIGNED), (dict(o=(1 << 30) + 4), INVALID), (dict(o=1 << 30, os=1004), INVALID),
    (dict(val=1 << 32), INVALID), (dict(idx=1 << 31), INVALID), (dict(ws=1 << 30), INVALID)])
def test_logits_refusals(L, bad, status):
    assert logits(L, **bad) == status


def test_logits_workspace(L):
    for s, want in ((spec(), 16384), (spec(rows=0), 0)):
        assert L.qgemv_logits_workspace_bytes(ctypes.addressof(s)) == want


# Tall batches on short prefixes: rows enough for the tcgen05 kernel, prefixes below,
# at and above its tile of 128 keys, and row tiles just below and above the
# rule's 1824 (6 * 304) per 64 keys.
TALL = [(n_seqs, n_q, heads, kv) for kv, heads, n_q in ((8, 64, 8), (8, 64, 4), (8, 32, 8), (32, 32, 8), (1, 64, 8))
        for n_seqs in (1824 // kv * 64 // (n_q * heads // kv) + d for d in (-1, 0, 1, 8))]


@pytest.mark.parametrize("n_seqs,n_q,heads,kv", TALL)
def test_tall_batches_on_short_prefixes_have_a_plan(L, n_seqs, n_q, heads, kv):
    c = cache(n_heads=kv, page_stride=2048 * kv, row_stride=128 * kv)
    for prefix in (0, 1, 63, 64, 65, 100, 127, 128, 129, 191, 192, 255, 256, 257):
        b = batch(n_seqs=n_seqs, n_q=n_q, n_q_heads=heads, prefix_len=prefix)
        rows = n_seqs * n_q * heads                 # a partial row: head_dim sums, maximum and sum in fp32
        parts = (attn_ws(L, b, c) - 16384) / (rows * (4 * 128 + 8))
        # at least one part a row for the suffix and one for a prefix, at most one per 64 keys each
        assert parts == int(parts)
        assert 1 + (prefix > 0) <= parts <= -(-prefix // 64) + -(-149 // 64), (prefix, parts)


def plan_copies(p):
    yield copy.copy(p)
    yield copy.deepcopy(p)
    yield pickle.loads(pickle.dumps(p))
    yield copy.deepcopy({"model": [p]})["model"][0]


def test_copies_of_a_rope_plan_are_plans_of_their_own():
    p = q.rope_plan(96, 1e5, layout="interleaved", scaling="yarn", factor=4.0, orig_len=8192)
    want = bytes(p)
    copies = list(plan_copies(p))
    assert len({x.address for x in [p, *copies]}) == 5
    del p
    gc.collect()
    others = [q.rope_plan(8, 10.0 + i) for i in range(200)]     # would take the freed memory
    for x in copies:
        assert x.address == ctypes.addressof(x) and ctypes.string_at(x.address, ctypes.sizeof(x)) == want
    assert all(o.rot_dim == 8 for o in others)


def test_a_plan_filled_through_the_c_call_is_a_plan(L):
    plan = q.RopePlan()
    cfg = q.RopeConfig(rot_dim=64, layout=0, scaling=0, base=1e4)
    assert L.qgemv_rope_init(ctypes.byref(cfg), ctypes.byref(plan)) == OK
    assert plan.address == ctypes.addressof(plan) and bytes(plan) == bytes(q.rope_plan(64, 1e4))


def test_the_binding_takes_the_structures_themselves():
    """A plan is read where it lies at the call; something else is refused by its size."""
    ext = q._load_binding()
    none = [None] * 8
    for x in (q.rope_plan(64, 1e4), *plan_copies(q.rope_plan(64, 1e4))):
        with pytest.raises(ValueError, match="q, or k and v"):
            ext.rope_kv(x, *none)
    for bad in (q.KvCacheStruct(), b"1234", 4096, "x"):
        with pytest.raises(ValueError, match="plan"):
            ext.rope_kv(bad, *none)
    plan = q.rope_plan(64, 1e4)
    for bad in (plan, b"", 4096):
        with pytest.raises(ValueError, match="cache"):
            ext.rope_kv(plan, *none[:5], bad, None, None)
        with pytest.raises(ValueError, match="cache"):
            ext.attn_prefix(None, bad, None, None, None, None, None)
        with pytest.raises(ValueError, match="batch"):
            ext.attn_prefix(None, q.KvCacheStruct(), bad, None, None, None, None)
        with pytest.raises(ValueError, match="rules"):
            ext.logits_rules(None, bad, None, None, None, None, None)


ACCEPTED = "past the checks"


def outcome(status):
    """A refusal's status; whatever the device says, or its absence, is past the checks."""
    return status if status in (INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE) else ACCEPTED


@pytest.mark.parametrize("over", ["o", "lse", "ws"])
def test_attn_refuses_outputs_over_its_page_tables(L, over):
    # q, o, suffix lengths and tables far apart; 4 sequences, 7 pages of prefix, 10 of suffix each
    at = dict(o=1 << 31, lse=1 << 32, ws=1 << 38)[over]
    assert outcome(attn(L)) == ACCEPTED
    assert attn(L, b=batch(prefix_pages=at)) == INVALID
    assert attn(L, b=batch(prefix_pages=at - 7 * 4 + 4)) == INVALID
    assert outcome(attn(L, b=batch(prefix_pages=at - 7 * 4))) == ACCEPTED
    assert attn(L, b=batch(suffix_pages=at)) == INVALID
    assert attn(L, b=batch(suffix_pages=at - 4 * 40 + 4)) == INVALID
    assert outcome(attn(L, b=batch(suffix_pages=at - 4 * 40))) == ACCEPTED
    # tables that are not read may lie anywhere
    assert outcome(attn(L, b=batch(prefix_len=0, prefix_pages=at))) == ACCEPTED
    assert outcome(attn(L, b=batch(max_suffix=0, suffix_pages=at))) == ACCEPTED


def test_attn_refuses_outputs_that_overlap_themselves(L):
    # 8 tokens of 12 heads of 128: any order of tokens and heads with distinct pieces
    for os, oh in ((1536, 128), (128, 1024), (2000, 160), (136, 1200), (3072 // 2, 128), (128 * 12 + 8, 128),
                   (256, 8 * 256 + 128), (320, 8 * 320 - 160)):
        assert outcome(attn(L, os=os, oh=oh)) == ACCEPTED, (os, oh)
    # pieces of two lattices between one another: 12 heads 128 * 16 apart, tokens 128 apart, and interleaved pairs
    assert outcome(attn(L, os=128, oh=2048)) == ACCEPTED
    assert outcome(attn(L, b=batch(n_seqs=1, n_q=2, n_q_heads=4), os=384, oh=256 * 3)) == ACCEPTED
    assert outcome(attn(L, b=batch(n_seqs=1, n_q=2, n_q_heads=4), os=384, oh=256)) == ACCEPTED
    for os, oh in ((0, 128), (1536, 0), (1535, 128), (1536, 127), (127, 1024), (128, 1023), (1024, 128), (128, 128),
                   (256, 256), (384, 256), (3 * 128, 2 * 128)):
        assert attn(L, os=os, oh=oh, ot=q.BF16) == INVALID, (os, oh)
    # a stride that nothing is reached with does not count
    assert outcome(attn(L, b=batch(n_seqs=1, n_q=1), os=0)) == ACCEPTED
    assert outcome(attn(L, c=cache(n_heads=1), b=batch(n_q_heads=1), os=128, oh=0)) == ACCEPTED


def test_attn_overlap_rule_against_counting(L):
    """The rule against a count of the elements, over small lattices."""
    import random
    rng = random.Random(4)
    seen = [0, 0]
    for _ in range(400):
        n, heads = rng.randint(1, 6), rng.choice([2, 4, 6])
        os, oh = rng.randint(0, 40), rng.randint(0, 40)
        places = [t * os + h * oh for t in range(n) for h in range(heads)]
        distinct = all(abs(a - b) >= 8 for i, a in enumerate(places) for b in places[:i])
        got = outcome(attn(L, c=cache(head_dim=8), b=batch(n_seqs=n, n_q=1, n_q_heads=heads), os=os, oh=oh))
        assert got == (ACCEPTED if distinct else INVALID), (n, heads, os, oh)
        seen[distinct] += 1
    assert min(seen) > 50


def fused(L, n=10, **kw):
    """rope on the parts of one fp32 QKV buffer of 12 + 2 + 2 heads of 128, rows 2048 elements apart."""
    at = 1 << 30
    f = dict(q=at, k=at + 4 * 1536, v=at + 4 * 1792, qs=2048, ks=2048, vs=2048, n=n, ot=q.F32, o=1 << 36, os=1536)
    f.update(kw)
    return rope(L, **f)


def test_rope_in_a_fused_buffer(L):
    at = 1 << 30
    assert outcome(fused(L)) == ACCEPTED
    assert outcome(fused(L, o=at, os=2048)) == ACCEPTED                      # in place
    # in place over k or v: the write of a q head and the read of a k head would race
    assert fused(L, o=at, os=2048, k=at) == INVALID
    assert fused(L, o=at, os=2048, v=at) == INVALID
    assert fused(L, o=at, os=2048, k=at + 4 * 1535) == INVALID
    assert fused(L, o=at, os=2048, k=at + 4 * (2048 * 3 + 1400)) == INVALID     # another token's q
    assert fused(L, o=at, os=2048, v=at - 4 * 255) == INVALID
    assert outcome(fused(L, o=at, os=2048, v=at - 4 * 256)) == ACCEPTED
    # one token, in place over k
    assert fused(L, n=1, o=at, os=0, k=at + 4 * 1280) == INVALID
    # a result between the rows of its inputs touches none of them
    assert outcome(fused(L, qs=4096, ks=4096, vs=4096, o=at + 4 * 2048, os=4096)) == ACCEPTED
    assert outcome(fused(L, qs=4096, ks=4096, vs=4096, o=at + 4 * 2048 + 2 * 1024, os=8192, ot=q.BF16)) == ACCEPTED
    assert fused(L, qs=4096, ks=4096, vs=4096, o=at + 4 * 2047, os=4096) == INVALID
    assert fused(L, qs=4096, ks=4096, vs=4096, o=at + 4 * 2561, os=4096) == INVALID


def test_rope_overlap_rule_against_counting(L):
    """Rows of k against rows of the result, each of any stride, against a count of the bytes."""
    import random
    rng = random.Random(5)
    seen = [0, 0]
    c = cache(head_dim=8, n_heads=1, row_stride=8, page_stride=128)
    for _ in range(600):
        n, hq = rng.randint(1, 5), rng.randint(1, 3)
        os, ks = rng.randint(8 * hq, 60), rng.randint(0, 60)
        if rng.random() < 0.5:
            ks = os = max(os, ks)
        ot = rng.choice([q.F32, q.F16])
        ob = 4 if ot == q.F32 else 2
        off = 4 * rng.randint(-100, 100)
        written = {t * os * ob + i for t in range(n) for i in range(8 * hq * ob)}
        read = {off + t * ks * 4 + i for t in range(n) for i in range(8 * 4)}
        got = outcome(rope(L, c, rot=8, d=8, hq=hq, n=n, qs=8 * hq, o=1 << 36, os=os, ot=ot, k=(1 << 36) + off, ks=ks,
                           v=1 << 33, vs=8))
        assert got == (INVALID if written & read else ACCEPTED), (n, hq, os, ks, ot, off)
        seen[bool(written & read)] += 1
    assert min(seen) > 100


def test_attn_workspace_against_bounds(L):
    """Over sizes on both sides of every threshold: a whole number of partial rows a row,
    at least one for each kind of keys there is and at most one per 64 keys (per
    stream of 128 rows where two streams share the key tiles), and no less for more
    sequences, more rows to a head or longer contexts than a small part of them needs."""
    import random
    rng = random.Random(6)
    kinds = set()
    for _ in range(4000):
        kv, group, nq, d = rng.choice([1, 2, 8, 32]), rng.choice([1, 4, 7, 16]), rng.randint(1, 8), rng.choice([64, 128, 192, 256])
        n = int(2 ** rng.uniform(0, 9))
        prefix = rng.choice([0, 1, 63, 64, 100, 127, 128, 129, int(2 ** rng.uniform(0, 18))])
        own = rng.choice([0, 1, nq - 1, nq, 64, 100, int(2 ** rng.uniform(0, 16))])
        c = cache(n_heads=kv, head_dim=d, row_stride=kv * d, page_stride=16 * kv * d, head_stride=d)
        b = batch(n_seqs=n, n_q=nq, n_q_heads=kv * group, prefix_len=prefix, max_suffix=own)
        rows = n * nq * kv * group
        bytes_ = attn_ws(L, b, c)
        assert bytes_ >= 16384
        parts, rest = divmod(bytes_ - 16384, rows * (4 * d + 8))
        assert rest == 0
        shared = max(0, own - nq + 1)
        assert (prefix > 0) + (shared > 0) <= parts <= -(-prefix // 64) + -(-shared // 64) + 1, (n, nq, kv, group, prefix, own)
        # attn_prefix asks for exactly this much
        at = dict(q=1 << 40, o=1 << 41, lse=1 << 42, ws=1 << 43, qt=kv * group * d, qh=d, os=kv * group * d, oh=d)
        c.k, c.v = 1 << 44, 1 << 45
        assert attn(L, c=c, b=b, ws_bytes=bytes_ - 1, **at) == WORKSPACE
        assert outcome(attn(L, c=c, b=b, ws_bytes=bytes_, **at)) == ACCEPTED
        kinds.add((prefix > 0, shared > 0, n * nq * group > 64, parts > 2))
    assert len(kinds) >= 12
    # more of anything never needs less than the keys and rows themselves ask for
    sizes = [attn_ws(L, batch(n_seqs=n, prefix_len=100000), cache()) for n in (1, 2, 4, 8, 16, 32)]
    assert sizes == sorted(sizes) and sizes[-1] > sizes[0]
