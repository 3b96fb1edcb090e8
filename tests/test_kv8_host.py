"""The argument checks of the operators over an 8-bit cache and of beam search: a
refused call returns its status before any CUDA call, so these run without a GPU.
Pointers are numbers that nothing follows."""
import ctypes

import pytest

import quantized_q4_weight_gb300 as q
from tests.test_decode_ops_host import BAD_CACHES, BIG, INVALID, MISALIGNED, OK, UNSUPPORTED, WORKSPACE, cache

ACCEPTED = "past the checks"


def outcome(status):
    return status if status in (INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE) else ACCEPTED


@pytest.fixture(scope="module")
def L():
    from quantized_q4_weight_gb300 import _build
    _build.build()
    return q.lib()


def cache8(**kw):
    f = dict(k=BIG, v=2 * BIG, k_scale=3 * BIG, v_scale=4 * BIG, type=q.CODE_INT8, n_pages=100, page_size=64, block_size=16,
             n_heads=2, head_dim=128, page_stride=64 * 256, row_stride=256, head_stride=128, scale_page_stride=8,
             scale_block_stride=2, scale_head_stride=1)
    f.update(kw)
    return q.Kv8CacheStruct(**f)


BAD_CACHES8 = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID),
               (dict(type=2), INVALID), (dict(type=-1), INVALID), (dict(n_pages=0), INVALID), (dict(n_pages=1 << 31), INVALID),
               (dict(page_size=8, block_size=8), INVALID), (dict(page_size=48), INVALID), (dict(page_size=1 << 17), INVALID),
               (dict(block_size=8), INVALID), (dict(block_size=24), INVALID), (dict(block_size=128), INVALID),
               (dict(n_heads=0), INVALID), (dict(n_heads=4097), INVALID), (dict(head_dim=8), INVALID),
               (dict(head_dim=120), INVALID), (dict(head_dim=272), INVALID), (dict(page_stride=-16), INVALID),
               (dict(row_stride=1 << 62), INVALID), (dict(head_stride=0), INVALID), (dict(page_stride=0), INVALID),
               (dict(row_stride=0), INVALID), (dict(scale_page_stride=-1), INVALID), (dict(scale_block_stride=1 << 60), INVALID),
               (dict(scale_head_stride=-1), INVALID), (dict(k=BIG + 8), MISALIGNED), (dict(v=2 * BIG + 4), MISALIGNED),
               (dict(row_stride=264), MISALIGNED), (dict(head_stride=136), MISALIGNED), (dict(k_scale=3 * BIG + 2), MISALIGNED)]


def batch8(**kw):
    f = dict(n_seqs=4, n_q=2, n_q_heads=12, max_len=1000, lens=4096, pages=8192, pages_stride=16, window=0, sinks=0, scale=0.0)
    f.update(kw)
    return q.Kv8BatchStruct(**f)


BAD_BATCHES = [dict(n_seqs=0), dict(n_seqs=(1 << 20) + 1), dict(n_q=0), dict(n_q=9), dict(max_len=-1), dict(max_len=2 ** 31 - 1)]
BAD_ATTN = [dict(n_q_heads=0), dict(n_q_heads=13), dict(n_q_heads=4098), dict(window=-1), dict(sinks=-1), dict(scale=-1.0),
            dict(scale=float("nan")), dict(scale=float("inf")), dict(window=(1 << 30) + 1),
            dict(n_seqs=1 << 20, n_q=8, n_q_heads=4096)]


# ------------------------------------------------------------------ append

def append(L, c=None, b=None, **kw):
    f = dict(k=1 << 30, v=1 << 31, t=q.F32, ks=256, vs=256, n=8, first=None, most=2)
    f.update(kw)
    c = cache8() if c is None else c
    b = batch8() if b is None else b
    return L.qgemv_kv8_append(f["k"], f["v"], f["t"], f["ks"], f["vs"], f["n"], ctypes.addressof(c), ctypes.addressof(b),
                              f["first"], f["most"], None)


@pytest.mark.parametrize("bad,status", BAD_CACHES8)
def test_caches(L, bad, status):
    assert append(L, cache8(**bad)) == status
    assert attn(L, cache8(**bad)) == status and attn_ws(L, batch8(), cache8(**bad)) == 0


@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_batches(L, bad):
    assert append(L, b=batch8(**bad)) == INVALID and attn(L, b=batch8(**bad)) == INVALID
    assert attn_ws(L, batch8(**bad), cache8()) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(t=3), INVALID), (dict(n=-1), INVALID), (dict(n=7), INVALID),
    (dict(most=1), INVALID), (dict(most=-1), INVALID), (dict(ks=-256), INVALID), (dict(vs=1 << 60), INVALID),
    (dict(k=(1 << 30) + 2), MISALIGNED), (dict(v=(1 << 31) + 1), MISALIGNED), (dict(first=4098), MISALIGNED),
    (dict(k=BIG), INVALID), (dict(v=2 * BIG + 64), INVALID), (dict(k=3 * BIG - 4), INVALID), (dict(first=4 * BIG), INVALID),
    (dict(ks=1 << 31), UNSUPPORTED)])
def test_append_refusals(L, bad, status):
    assert outcome(append(L)) == ACCEPTED
    assert append(L, **bad) == status


def test_append_batches_and_lists(L):
    assert append(L, b=batch8(lens=None)) == INVALID and append(L, b=batch8(pages=None)) == INVALID
    assert append(L, b=batch8(pages_stride=-1)) == INVALID and append(L, b=batch8(lens=4098)) == MISALIGNED
    assert append(L, b=batch8(pages=BIG)) == INVALID            # the tables over the cache
    assert append(L, cache8(v_scale=3 * BIG + 16)) == INVALID    # its arrays over one another
    assert append(L, cache8(row_stride=1 << 32, page_stride=1 << 38)) in (UNSUPPORTED, INVALID)
    # with a list any number of tokens; none of them is no launch
    assert outcome(append(L, first=1 << 20, n=100, most=60)) == ACCEPTED
    assert append(L, first=1 << 20, n=0, most=60, k=None, v=None) == OK
    assert append(L, first=1 << 20, n=10, most=0) == OK
    far = cache8(k=1 << 60, v=2 << 60, k_scale=3 << 60, v_scale=4 << 60)
    many = batch8(n_seqs=1 << 20, max_len=1 << 30, pages=1 << 58, pages_stride=1 << 24)
    assert append(L, far, many, first=1 << 20, n=1 << 30, most=1 << 30, v=1 << 55) == UNSUPPORTED   # too many blocks


# --------------------------------------------------------------- attention

def attn(L, c=None, b=None, ws_bytes=BIG // 4, **kw):
    f = dict(q=1 << 30, t=q.BF16, qt=1536, qh=128, o=1 << 31, ot=q.BF16, os=1536, oh=128, lse=1 << 32, ws=1 << 38)
    f.update(kw)
    c = cache8() if c is None else c
    b = batch8() if b is None else b
    return L.qgemv_attn_kv8(f["q"], f["t"], f["qt"], f["qh"], ctypes.addressof(c), ctypes.addressof(b), f["o"], f["ot"], f["os"],
                            f["oh"], f["lse"], f["ws"], ws_bytes, None)


def attn_ws(L, b, c):
    return L.qgemv_attn_kv8_workspace_bytes(ctypes.addressof(b), ctypes.addressof(c))


@pytest.mark.parametrize("bad", BAD_ATTN)
def test_attn_batches(L, bad):
    assert attn(L, b=batch8(**bad)) == INVALID and attn_ws(L, batch8(**bad), cache8()) == 0
    if "n_seqs" not in bad:  # the append takes no part in these
        assert outcome(append(L, b=batch8(**bad))) == ACCEPTED


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(t=q.F32), INVALID), (dict(ot=q.F16), INVALID), (dict(ot=7), INVALID),
    (dict(qt=-8), INVALID), (dict(os=1 << 60), INVALID), (dict(os=1535), INVALID), (dict(oh=0), INVALID),
    (dict(q=(1 << 30) + 8), MISALIGNED), (dict(qt=1540), MISALIGNED), (dict(qh=100), MISALIGNED), (dict(o=(1 << 31) + 1), MISALIGNED),
    (dict(lse=(1 << 32) + 2), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16383), WORKSPACE),
    (dict(ws=(1 << 38) + 8), MISALIGNED), (dict(o=1 << 30), INVALID), (dict(o=1 << 38), INVALID), (dict(o=BIG), INVALID),
    (dict(o=3 * BIG), INVALID), (dict(lse=1 << 31), INVALID), (dict(lse=4 * BIG), INVALID), (dict(ws=1 << 30), INVALID),
    (dict(o=8192), INVALID), (dict(o=4096), INVALID)])
def test_attn_refusals(L, bad, status):
    assert outcome(attn(L)) == ACCEPTED
    assert attn(L, **bad) == status


def test_attn_other_refusals(L):
    assert attn(L, b=batch8(lens=None)) == INVALID and attn(L, b=batch8(pages=None)) == INVALID
    assert outcome(attn(L, b=batch8(pages=None, max_len=0))) == ACCEPTED
    assert attn(L, cache8(page_stride=1 << 40, n_pages=10)) == UNSUPPORTED       # more than a tensor map's stride
    assert outcome(attn(L, cache8(n_heads=1, head_stride=0), batch8(n_q_heads=6), qt=768, os=768)) == ACCEPTED


def test_attn_workspace_is_asked_for_exactly(L):
    import random
    rng = random.Random(7)
    for _ in range(2000):
        kv, group, d = rng.choice([1, 2, 8, 32]), rng.choice([1, 4, 7, 16]), rng.choice([16, 64, 80, 128, 256])
        b = batch8(n_seqs=int(2 ** rng.uniform(0, 11)), n_q=rng.randint(1, 8), n_q_heads=kv * group,
                   max_len=rng.choice([0, 1, 767, 768, 769, int(2 ** rng.uniform(0, 20))]), pages=1 << 50, pages_stride=1 << 16,
                   window=rng.choice([0, 0, 100, 5000]), sinks=rng.choice([0, 4]))
        c = cache8(n_heads=kv, head_dim=d, row_stride=kv * d, page_stride=64 * kv * d, head_stride=d, scale_page_stride=4 * kv,
                   scale_block_stride=kv, k=1 << 44, v=1 << 45, k_scale=1 << 46, v_scale=1 << 47)
        n = attn_ws(L, b, c)
        assert n >= 16384 and n < 64 << 20
        at = dict(q=1 << 40, o=1 << 41, lse=1 << 42, ws=1 << 43, qt=kv * group * d, qh=d, os=kv * group * d, oh=d)
        assert attn(L, c, b, ws_bytes=n - 1, **at) == WORKSPACE
        assert outcome(attn(L, c, b, ws_bytes=n, **at)) == ACCEPTED


# ---------------------------------------------------- norms with rotation

def norm_rope(L, c="cache", eps=1e-6, qw=1 << 20, kw=1 << 21, **kw2):
    plan = q.rope_plan(kw2.pop("rot", 128), 1e4)
    norm = q.QkNormStruct(qw, kw, eps)
    f = dict(plan=plan.address, norm=ctypes.addressof(norm), q=4096, k=BIG // 2, v=BIG // 2 + (1 << 30), t=q.F32, qs=1536,
             ks=256, vs=256, pos=1 << 34, slots=1 << 35, n=10, hq=12, hk=2, d=128, o=1 << 36, ot=q.BF16, os=1536, ko=1 << 37,
             kt=q.F32, kos=256)
    f.update(kw2)
    c = cache() if c == "cache" else c
    return L.qgemv_norm_rope_kv(f["plan"], f["norm"], f["q"], f["k"], f["v"], f["t"], f["qs"], f["ks"], f["vs"], f["pos"],
                                f["slots"], f["n"], f["hq"], f["hk"], f["d"], f["o"], f["ot"], f["os"], f["ko"], f["kt"], f["kos"],
                                ctypes.addressof(c) if c else None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(plan=None), INVALID), (dict(norm=None), INVALID), (dict(q=None, k=None), INVALID), (dict(v=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(qw=None), INVALID), (dict(kw=None), INVALID), (dict(qw=(1 << 20) + 2), MISALIGNED),
    (dict(t=3), INVALID), (dict(ot=-1), INVALID), (dict(o=None), INVALID), (dict(n=0), INVALID), (dict(n=1 << 32), INVALID),
    (dict(hq=0), INVALID), (dict(hk=3), INVALID), (dict(hk=0), INVALID), (dict(d=127), INVALID), (dict(d=64), INVALID),
    (dict(d=258), INVALID), (dict(rot=256), INVALID), (dict(qs=1535), INVALID), (dict(os=100), INVALID), (dict(ks=1 << 60), INVALID),
    (dict(q=4098), MISALIGNED), (dict(o=(1 << 36) + 1), MISALIGNED), (dict(k=BIG // 2 + 2), MISALIGNED),
    (dict(pos=(1 << 34) + 2), MISALIGNED), (dict(slots=(1 << 35) + 1), MISALIGNED), (dict(o=4096, ot=q.BF16), INVALID),
    (dict(o=4100, ot=q.F32), INVALID), (dict(o=BIG), INVALID), (dict(q=2 * BIG), INVALID), (dict(k=BIG), INVALID),
    (dict(o=BIG // 2), INVALID), (dict(o=1 << 34), INVALID), (dict(o=1 << 35), INVALID), (dict(o=1 << 20), INVALID),
    (dict(o=1 << 21), INVALID), (dict(kw=BIG), INVALID)])
def test_norm_rope_refusals(L, bad, status):
    assert outcome(norm_rope(L)) == ACCEPTED
    assert norm_rope(L, **bad) == status


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_norm_rope_caches(L, bad, status):
    assert norm_rope(L, cache(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(ko=None), INVALID), (dict(kt=3), INVALID), (dict(kos=255), INVALID), (dict(ko=(1 << 37) + 1), MISALIGNED), (dict(ko=1 << 36), INVALID),
    (dict(ko=4096), INVALID), (dict(ko=BIG // 2), INVALID), (dict(ko=1 << 34), INVALID), (dict(ko=1 << 20), INVALID)])
def test_norm_rope_without_a_cache(L, bad, status):
    assert outcome(norm_rope(L, None, v=None, slots=None)) == ACCEPTED
    assert norm_rope(L, None, v=None, slots=None, **bad) == status


def test_norm_rope_parts(L):
    assert outcome(norm_rope(L, q=None, qw=None)) == ACCEPTED
    assert outcome(norm_rope(L, k=None, kw=None, v=None, slots=None)) == ACCEPTED
    assert outcome(norm_rope(L, o=4096, ot=q.F32)) == ACCEPTED              # q in place
    # in place over k: a q head's write and a k head's read would race
    assert norm_rope(L, q=BIG // 2 - 4 * 1280, o=BIG // 2 - 4 * 1280, ot=q.F32) == INVALID


# ------------------------------------------------------------------- beams

def spec(**kw):
    f = dict(n_groups=3, n_beams=4, n_best=8, vocab=1000, scores=4096, done=8192)
    f.update(kw)
    return q.BeamSpec(**f)


def beam(L, s=None, ws_bytes=BIG, **kw):
    f = dict(x=1 << 30, t=q.F32, xs=1000, score=1 << 31, token=1 << 32, parent=1 << 33, ws=1 << 38)
    f.update(kw)
    s = spec() if s is None else s
    return L.qgemv_beam_select(f["x"], f["t"], f["xs"], ctypes.addressof(s), f["score"], f["token"], f["parent"], f["ws"],
                               ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n_groups=0), INVALID), (dict(n_groups=(1 << 20) + 1), INVALID), (dict(n_beams=0), INVALID), (dict(n_beams=17), INVALID),
    (dict(n_best=0), INVALID), (dict(n_best=33), INVALID), (dict(vocab=0), INVALID), (dict(vocab=(1 << 26) + 1), INVALID),
    (dict(scores=None), INVALID), (dict(scores=4098), MISALIGNED), (dict(done=8193), MISALIGNED), (dict(scores=1 << 31), INVALID),
    (dict(done=1 << 32), INVALID)])
def test_beam_specs(L, bad, status):
    assert beam(L, spec(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), INVALID), (dict(t=4), INVALID), (dict(xs=999), INVALID), (dict(xs=1 << 60), INVALID), (dict(score=None), INVALID),
    (dict(token=None), INVALID), (dict(parent=None), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16384), WORKSPACE),
    (dict(x=(1 << 30) + 2), MISALIGNED), (dict(score=(1 << 31) + 2), MISALIGNED), (dict(token=(1 << 32) + 4), MISALIGNED),
    (dict(parent=(1 << 33) + 1), MISALIGNED), (dict(ws=(1 << 38) + 4), MISALIGNED), (dict(score=1 << 30), INVALID),
    (dict(token=1 << 31), INVALID), (dict(parent=4096), INVALID), (dict(ws=1 << 30), INVALID)])
def test_beam_refusals(L, bad, status):
    assert outcome(beam(L)) == ACCEPTED
    assert beam(L, **bad) == status


def test_beam_workspace(L):
    import random
    rng = random.Random(8)
    for _ in range(500):
        s = spec(n_groups=int(2 ** rng.uniform(0, 14)), n_beams=rng.randint(1, 16), n_best=rng.randint(1, 32),
                 vocab=int(2 ** rng.uniform(0, 26)), scores=1 << 50, done=None)
        n = L.qgemv_beam_workspace_bytes(ctypes.addressof(s))
        # rows of a launch, at most 64 slices each with their n_best keys, maximum and sum
        assert 16384 < n <= 16384 + 16 + min(s.n_groups, 4080) * s.n_beams * 64 * 8 * (s.n_best + 1)
        at = dict(x=1 << 54, xs=s.vocab, score=1 << 51, token=1 << 52, parent=1 << 53, ws=1 << 55)
        assert beam(L, s, ws_bytes=n - 1, **at) == WORKSPACE and outcome(beam(L, s, ws_bytes=n, **at)) == ACCEPTED
    assert L.qgemv_beam_workspace_bytes(ctypes.addressof(spec(n_beams=17))) == 0


# ------------------------------------------------------------------- pages

def fork(L, caches=None, eight=True, n=None, **kw):
    f = dict(n_in=4, n_out=6, n_columns=10, parents=4096, lens=8192, pages=16384, pages_stride=10, fresh=32768,
             pages_out=65536, out_stride=10, lens_out=1 << 17)
    f.update(kw)
    caches = [cache8(), cache8(k=5 * BIG, v=6 * BIG, k_scale=7 * BIG, v_scale=8 * BIG)] if caches is None else caches
    arr = ((q.Kv8CacheStruct if eight else q.KvCacheStruct) * len(caches))(*caches)
    s = q.ForkStruct(**f)
    at = ctypes.addressof(arr)
    return L.qgemv_fork_pages(ctypes.addressof(s), None if eight else at, at if eight else None, len(caches) if n is None else n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n_in=0), INVALID), (dict(n_out=0), INVALID), (dict(n_columns=0), INVALID), (dict(n_in=(1 << 20) + 1), INVALID),
    (dict(parents=None), INVALID), (dict(lens=None), INVALID), (dict(pages=None), INVALID), (dict(fresh=None), INVALID),
    (dict(pages_out=None), INVALID), (dict(lens_out=None), INVALID), (dict(pages_stride=9), INVALID), (dict(out_stride=9), INVALID),
    (dict(pages_stride=-10), INVALID), (dict(parents=4098), MISALIGNED), (dict(lens=8193), MISALIGNED), (dict(pages=16386), MISALIGNED),
    (dict(fresh=32769), MISALIGNED), (dict(pages_out=65538), MISALIGNED), (dict(lens_out=(1 << 17) + 1), MISALIGNED),
    (dict(pages_out=16384), INVALID), (dict(pages_out=16384 + 4 * 39), INVALID), (dict(lens_out=8192), INVALID),
    (dict(lens_out=65536), INVALID), (dict(pages_out=BIG), INVALID), (dict(fresh=3 * BIG), INVALID), (dict(n=0), INVALID)])
def test_fork_refusals(L, bad, status):
    assert outcome(fork(L)) == ACCEPTED
    assert fork(L, **bad) == status


def test_fork_caches(L):
    for bad, status in BAD_CACHES8:
        assert fork(L, [cache8(), cache8(**bad)]) == status
    for bad, status in BAD_CACHES:
        assert fork(L, [cache(), cache(**bad)], eight=False) == status
    assert outcome(fork(L, [cache(), cache(k=3 * BIG, v=4 * BIG)], eight=False)) == ACCEPTED
    other = dict(k=5 * BIG, v=6 * BIG, k_scale=7 * BIG, v_scale=8 * BIG)
    for bad in (dict(n_pages=101), dict(block_size=32, scale_page_stride=4), dict(head_dim=64), dict(type=q.CODE_E4M3)):
        assert fork(L, [cache8(), cache8(**{**other, **bad})]) == INVALID
    arr = (q.Kv8CacheStruct * 1)(cache8())
    s = q.ForkStruct(n_in=1, n_out=1, n_columns=1, parents=4096, lens=8192, pages=16384, pages_stride=1, fresh=32768,
                     pages_out=65536, out_stride=1, lens_out=1 << 17)
    both = ctypes.addressof(arr)
    assert L.qgemv_fork_pages(ctypes.addressof(s), None, None, 1, None) == INVALID
    assert L.qgemv_fork_pages(ctypes.addressof(s), both, both, 1, None) == INVALID


def test_the_binding_takes_the_structures_themselves():
    ext = q._load_binding()
    plan = q.rope_plan(64, 1e4)
    with pytest.raises(ValueError, match="plan"):
        ext.norm_rope_kv(b"1", *[None] * 10)
    with pytest.raises(ValueError, match="norm"):
        ext.norm_rope_kv(plan, plan, *[None] * 9)
    with pytest.raises(ValueError, match="q or k"):
        ext.norm_rope_kv(plan, q.QkNormStruct(), *[None] * 9)
    with pytest.raises(ValueError, match="cache"):
        ext.kv8_append(None, None, plan, *[None] * 4)
    with pytest.raises(ValueError, match="batch"):
        ext.attn_kv8(None, q.Kv8CacheStruct(), plan, *[None] * 4)
    with pytest.raises(ValueError, match="step"):
        ext.beam_select(None, plan, *[None] * 5)
    with pytest.raises(ValueError, match="fork_pages"):
        ext.fork_pages(b"", True, *[None] * 7)
    with pytest.raises(TypeError):
        ext.attn_kv8(None)


def test_constructors_refuse_what_does_not_fit():
    import torch
    k, s = torch.zeros((4, 32, 2, 64), dtype=torch.int8), torch.zeros((4, 2, 2))
    for bad in ((k, k.float(), s, s), (k, k[:3], s, s), (k[0], k[0], s, s), (k, k, s[:3], s[:3]), (k, k, s.double(), s.double()),
                (k, k, s[:, :, :1], s[:, :, :1]), (k, k, s, s)):           # the last: not on a GPU
        with pytest.raises(ValueError, match="Kv8Cache"):
            q.Kv8Cache(*bad)
    with pytest.raises(ValueError, match="QkNorm"):
        q.QkNorm(torch.ones(64), torch.ones(64))
    with pytest.raises(ValueError, match="BeamStep"):
        q.BeamStep(1, 4, 100, 4, torch.zeros(4))
    with pytest.raises(ValueError, match="PagePool"):
        q.PagePool([])


@pytest.mark.parametrize("shared", ["scale_page_stride", "scale_block_stride", "scale_head_stride"])
def test_scales_of_several_blocks_are_for_reading(L, shared):
    """A stride of 0 between scales: two blocks would write one float.  The attention only reads them."""
    c = cache8(**{shared: 0})
    assert append(L, c) == INVALID and append(L, c, first=1 << 20, n=0, most=60, k=None, v=None) == INVALID
    assert fork(L, [c]) == INVALID and fork(L, [cache8(k=5 * BIG, v=6 * BIG, k_scale=7 * BIG, v_scale=8 * BIG), c]) == INVALID
    assert outcome(attn(L, c)) == ACCEPTED and attn_ws(L, batch8(), c) > 0
    # strides that nothing is reached by may be 0
    one = dict(scale_page_stride=dict(n_pages=1), scale_block_stride=dict(block_size=64), scale_head_stride=dict(n_heads=1))
    c = cache8(**{shared: 0}, **one[shared])
    assert outcome(append(L, c)) == ACCEPTED and outcome(fork(L, [c])) == ACCEPTED


def test_codes_of_k_and_v_may_interleave(L):
    """k and v as halves of one buffer's pages, rows or heads; and what lies over one another by a byte is refused."""
    d, heads, page = 128, 2, 64
    row = heads * d
    for kw, step in ((dict(page_stride=2 * page * row, row_stride=row, head_stride=d), page * row),      # [pages][2][rows][heads]
                     (dict(page_stride=2 * page * row, row_stride=2 * row, head_stride=d), row),          # [pages][rows][2][heads]
                     (dict(page_stride=2 * page * row, row_stride=2 * row, head_stride=2 * d), d),         # [pages][rows][heads][2]
                     (dict(page_stride=2 * page * row, row_stride=d, head_stride=2 * page * d), page * d),  # [pages][heads][2][rows]
                     (dict(page_stride=page * d, row_stride=d, head_stride=200 * page * d), 100 * page * d)):  # [heads][2][pages]
        for way in (1, -1):
            assert outcome(append(L, cache8(v=BIG + way * step, **kw))) == ACCEPTED, (kw, way)
            assert append(L, cache8(v=BIG + way * (step - 16), **kw)) == INVALID, (kw, way)
    assert append(L, cache8(v=BIG)) == INVALID and append(L, cache8(v=BIG + 99 * page * row + 63 * row + 128 + 112)) == INVALID


def test_scales_may_interleave_with_one_another_and_with_the_codes(L):
    for kw, step in ((dict(scale_page_stride=16, scale_block_stride=2, scale_head_stride=1), 8),
                     (dict(scale_page_stride=16, scale_block_stride=4, scale_head_stride=1), 2),
                     (dict(scale_page_stride=16, scale_block_stride=4, scale_head_stride=2), 1)):
        assert outcome(append(L, cache8(v_scale=3 * BIG + 4 * step, **kw))) == ACCEPTED
        assert append(L, cache8(v_scale=3 * BIG + (4 * step - 4 if step > 1 else 0), **kw)) == INVALID
    # pages that end in their scales
    codes = 64 * 256
    kw = dict(page_stride=codes + 64, scale_page_stride=(codes + 64) // 4)
    assert outcome(append(L, cache8(k_scale=BIG + codes, **kw))) == ACCEPTED
    assert append(L, cache8(k_scale=BIG + codes - 4, **kw)) == INVALID
    assert append(L, cache8(k_scale=BIG + codes + 36, **kw)) == INVALID      # the last ones in the next page's codes


def test_places_against_a_plain_count(L):
    """Small caches at every distance of k from v: accepted where a list of all bytes has none twice."""
    import random
    rng = random.Random(9)
    for _ in range(300):
        n = [rng.randint(1, 3), 16, rng.randint(1, 3)]
        order = rng.sample(range(3), 3)
        s, at = [0, 0, 0], 16
        for i in order:
            s[i] = at * rng.choice([1, 1, 2])
            at = s[i] * n[i]
        places = sorted(a * s[0] + b * s[1] + c * s[2] for a in range(n[0]) for b in range(n[1]) for c in range(n[2]))
        for delta in rng.sample(range(0, 2 * at + 32, 16), min(8, (2 * at + 32) // 16)):
            meets = bool(set(places) & {x + delta for x in places})
            c = cache8(n_pages=n[0], page_size=16, block_size=16, n_heads=n[2], head_dim=16, page_stride=s[0], row_stride=s[1],
                       head_stride=s[2], v=BIG + delta, scale_page_stride=n[2])
            got = append(L, c, ks=16 * n[2], vs=16 * n[2])
            assert got == INVALID if meets else outcome(got) == ACCEPTED, (n, s, delta)


def test_norm_rope_of_nothing_is_refused():
    with pytest.raises(ValueError, match="q or k"):
        q.norm_rope_kv(q.rope_plan(64, 1e4), q.QkNorm(None, None), None, None)


class Elsewhere:
    """A tensor as far as its description goes, said to lie on a device; nothing follows its address."""

    def __init__(self, device, shape, dtype):
        import torch
        self._t, self.device, self.is_cuda = torch.empty(shape, dtype=dtype, device="meta"), torch.device(device), True

    def data_ptr(self):
        return 4096

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_what_lies_on_two_devices_is_refused():
    """A kernel runs on the device of its first tensor: descriptions of another's memory do not reach it."""
    import torch

    def at(device, dtype, *shape):
        return Elsewhere(device, shape, dtype)

    def cache_on(device):
        return q.Kv8Cache(*(at(device, torch.int8, 4, 32, 2, 64) for _ in range(2)), *(at(device, torch.float32, 4, 2, 2) for _ in range(2)))

    def kv_on(device):
        c = q.KvCache.__new__(q.KvCache)
        c.k, c.struct = at(device, torch.float16, 4, 16, 2, 64), cache()
        return c

    f, i = torch.float32, torch.int32
    here, there = "cuda:0", "cuda:1"
    with pytest.raises(ValueError, match="QkNorm.*cuda:0"):
        q.QkNorm(at(here, f, 64), at(there, f, 64))
    norm, plan = q.QkNorm(at(there, f, 64), at(there, f, 64)), q.rope_plan(64, 1e4)
    with pytest.raises(ValueError, match="norm_rope_kv.*weights.*cuda:1"):
        q.norm_rope_kv(plan, norm, at(here, f, 3, 4, 64), None, pos=at(here, i, 3))
    with pytest.raises(ValueError, match="norm_rope_kv.*cache.*cuda:0"):
        q.norm_rope_kv(plan, norm, at(there, f, 3, 4, 64), at(there, f, 3, 2, 64), cache=kv_on(here))
    for lens, pages in ((there, here), (here, there)):
        with pytest.raises(ValueError, match="Kv8Batch.*cuda:0"):
            q.Kv8Batch(2, 1, 4, cache_on(here), at(lens, i, 2), at(pages, i, 2, 3), 96)
    batch = q.Kv8Batch(2, 1, 4, cache_on(there), at(there, i, 2), at(there, i, 2, 3), 96)
    assert q.Kv8Batch(2, 1, 4, cache_on(there), at(there, i, 2), None, 0).n_seqs == 2
    with pytest.raises(ValueError, match="kv8_append.*cuda:1"):
        q.kv8_append(at(here, f, 2, 2, 64), at(here, f, 2, 2, 64), batch)
    with pytest.raises(ValueError, match="attn_kv8.*cuda:1"):
        q.attn_kv8(at(here, torch.float16, 2, 4, 64), batch, at(here, torch.uint8, 1 << 20))
    with pytest.raises(ValueError, match="BeamStep.*cuda:0"):
        q.BeamStep(1, 4, 100, 4, at(here, f, 1, 4), at(there, i, 1, 4))
    with pytest.raises(ValueError, match="beam_select.*cuda:1"):
        q.beam_select(at(here, f, 4, 100), q.BeamStep(1, 4, 100, 4, at(there, f, 1, 4)), at(here, torch.uint8, 1 << 20))
    with pytest.raises(ValueError, match="PagePool.*cuda:0"):
        q.PagePool([cache_on(here), cache_on(there)])
    with pytest.raises(ValueError, match="fork_pages.*cuda:1"):
        q.fork_pages(q.PagePool([cache_on(there)]), *(at(here, i, 2) for _ in range(2)), at(here, i, 2, 3), at(here, i, 2),
                     at(here, i, 2, 3), at(here, i, 2))
