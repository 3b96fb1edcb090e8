"""Attention over a shared prefix and own suffixes (qgemv_attn_prefix)
against the softmax in 64 bits, sequence by sequence.

Tolerance, from the arithmetic, with u half a unit of the cache's type at 1,
w the exact weights and A = sum w |v|:
  - a score is off by at most e = (d + 8) 2^-24 scale sum |q k| (fp32 sums of
    exact products) and 2^-21 from the base-2 exponential and its argument;
  - each weight enters the product with v rounded: u relative, and for fp16
    2^-25 absolute below its normal range, relative to the part's maximum;
  - sums of n terms in fp32: n 2^-24, here below 2^-12 A even at 10000 keys
    since partial sums are short (tiles of 64, parts, then parts together).
So |o - o64| <= (u + 2 (e + 2^-21) + 2^-12) A + n 2^-25 max |v| [fp16] and half a
unit of the output; lse is off by e + 2^-20 + 2^-12.
"""
import math

import pytest
import torch

import quantized_q4_weight_gb300 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_q4_weight_gb300 import _build
    _build.build()


class Case:
    def __init__(self, b, nq, hq, hkv, d, prefix, lens, page=16, dtype=torch.bfloat16, seed=0, spread=1.5, poison=True,
                 heads_first=False, max_suffix=None, q_pad=0, scale=None):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.b, self.nq, self.hq, self.hkv, self.d, self.prefix, self.lens, self.page = b, nq, hq, hkv, d, prefix, lens, page
        self.scale = d ** -0.5 if scale is None else scale
        top = max(lens) if max_suffix is None else max_suffix
        per = -(-max(top, 1) // page)
        pre = -(-prefix // page)
        pages = pre + b * per + 3
        shape = (pages, hkv, page, d) if heads_first else (pages, page, hkv, d)
        kv = [torch.randn(shape, generator=g, device=DEV).to(dtype) for _ in range(2)]
        if heads_first:
            kv = [x.transpose(1, 2) for x in kv]
        self.k, self.v = kv
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        self.prefix_pages, self.suffix_pages = order[:pre].clone(), order[pre:pre + b * per].view(b, per).clone()
        self.len_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        x = spread * torch.randn((b * nq, hq * d + q_pad), generator=g, device=DEV)
        self.q = x.to(dtype)[:, :hq * d].unflatten(1, (hq, d))
        if poison:  # rows that nobody has: the pages' ends and the pages left over
            used = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
            for table, n in [(self.prefix_pages, prefix)] + [(self.suffix_pages[i], n) for i, n in enumerate(lens)]:
                j = torch.arange(n, device=DEV)
                used[table.long()[j // page], j % page] = True
            self.k[~used] = float("nan")
            self.v[~used] = float("inf")
        self.cache = q.KvCache(self.k, self.v)
        self.batch = q.AttnBatch(b, nq, hq, self.cache, prefix, self.prefix_pages if pre else None, self.len_t,
                                 self.suffix_pages, top, scale=scale)
        self.ws = q.new_workspace(self.batch.workspace_bytes())

    def rows(self, i):
        """Keys and values of sequence i's context, float64 [rows][hkv][d]."""
        out = []
        for x in (self.k, self.v):
            parts = []
            for table, n in ((self.prefix_pages, self.prefix), (self.suffix_pages[i], self.lens[i])):
                j = torch.arange(n, device=DEV)
                parts.append(x[table.long()[j // self.page], j % self.page] if n else x[:0, 0])
            out.append(torch.cat(parts).double())
        return out

    def exact(self):
        """(o, A, lse, e): float64 outputs, sum w |v|, log of the sum, bound of a score's error."""
        b, nq, hq, hkv, d = self.b, self.nq, self.hq, self.hkv, self.d
        o = torch.zeros((b, nq, hq, d), dtype=torch.float64, device=DEV)
        A, lse, worst = torch.zeros_like(o), torch.full((b, nq, hq), float("-inf"), dtype=torch.float64, device=DEV), 0.0
        for i in range(b):
            k, v = self.rows(i)
            for t in range(nq):
                n = self.prefix + max(0, self.lens[i] - nq + t + 1)
                if n <= 0:
                    continue
                for h in range(hq):
                    x = self.q[i * nq + t, h].double()
                    kk, vv = k[:n, h // (hq // hkv)], v[:n, h // (hq // hkv)]
                    s = self.scale * (kk * x).sum(1)
                    worst = max(worst, float((self.scale * (kk * x).abs().sum(1)).max()))
                    w = torch.softmax(s, 0)
                    o[i, t, h] = w @ vv
                    A[i, t, h] = w @ vv.abs()
                    lse[i, t, h] = torch.logsumexp(s, 0)
        return o, A, lse, (d + 8) * 2.0 ** -24 * worst

    def run(self, **kw):
        return q.attn_prefix(self.q, self.batch, self.ws, **kw)

    def check(self, out_type=None, o=None):
        lse = torch.full((self.b * self.nq, self.hq), 5.0, device=DEV)
        out = torch.full(self.q.shape, 3.0, dtype=out_type or self.k.dtype, device=DEV) if o is None else o
        self.run(out=out, lse=lse)
        torch.cuda.synchronize()
        assert q.device_status() == 0
        ref, A, l64, e = self.exact()
        u, uo = HALF_UNIT[self.k.dtype], HALF_UNIT[out.dtype]
        keys = self.prefix + max(self.lens)
        vmax = 6.0
        tol = (u + 2 * (e + 2.0 ** -21) + 2.0 ** -12) * A + uo * ref.abs() + 1e-30
        if self.k.dtype == torch.float16:
            tol = tol + keys * 2.0 ** -25 * vmax * (A > 0)
        got = out.double().view(ref.shape)
        assert bool(torch.isfinite(got).all())
        assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() - tol).max())
        gl = lse.double().view(l64.shape)
        none = torch.isinf(l64)
        assert bool((gl[none] == float("-inf")).all()) and bool((got[none] == 0).all())
        assert bool(((gl - l64)[~none].abs() <= e + 2.0 ** -20 + 2.0 ** -12 + 2.0 ** -22 * l64[~none].abs()).all())
        return out, lse


@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 130, 1000])
@pytest.mark.parametrize("lens", [[0, 1, 2], [64, 63, 65], [200, 0, 37]])
def test_lengths(prefix, lens):
    Case(3, 1, 6, 2, 64, prefix, lens, seed=prefix + lens[0]).check()


@pytest.mark.parametrize("nq", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("hq,hkv", [(12, 2), (16, 2), (8, 8), (16, 1), (5, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_and_heads(nq, hq, hkv, d):
    Case(3, nq, hq, hkv, d, 150, [0, nq, 90], seed=nq * hq + d).check()


@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_head_sizes(d, dtype):
    for nq, hq in ((1, 4), (3, 16), (8, 12)):        # 2, 24 and 48 rows a sequence and cache head
        Case(2, nq, hq, 2, d, 100, [40, 77], dtype=dtype, seed=d + nq).check()


@pytest.mark.parametrize("page", [1, 2, 16, 64, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(page, heads_first):
    Case(3, 2, 6, 2, 64, 333, [5, 100, 257], page=page, heads_first=heads_first, seed=page).check()


@pytest.mark.parametrize("b,nq,hq,hkv,prefix,top", [(1, 1, 2, 2, 5000, 30), (1, 1, 12, 2, 0, 9000), (2, 1, 32, 8, 700, 40),
                                                    (40, 1, 8, 1, 300, 50), (24, 4, 16, 2, 513, 20),
                                                    (64, 2, 4, 2, 129, 300)])
def test_shapes_of_batches(b, nq, hq, hkv, prefix, top):
    lens = [(i * 7919) % (top + 1) for i in range(b)]
    lens[0] = top
    Case(b, nq, hq, hkv, 64, prefix, lens, seed=b).check()


# More (key, row) pairs of the rows that only later queries see than a warp has
# lanes: narrow heads, many queries a sequence, blocks of one warp.
@pytest.mark.parametrize("d", [8, 16])
def test_many_queries_of_narrow_heads(d):
    Case(80, 8, 4, 1, d, 70, [(i * 7919) % 41 for i in range(80)], seed=d).check()


# Few parts for the warps that combine them, one and more waves of rows.
@pytest.mark.parametrize("b,nq,hq,hkv,d,prefix,top", [(15, 4, 14, 2, 64, 193, 584), (60, 1, 16, 1, 128, 2000, 200),
                                                      (19, 2, 14, 2, 64, 873, 79), (30, 1, 16, 2, 128, 5000, 200),
                                                      (6, 8, 8, 8, 256, 300, 100), (50, 3, 16, 2, 32, 10, 90)])
def test_rows_of_few_parts(b, nq, hq, hkv, d, prefix, top):
    lens = [(i * 7919) % (top + 1) for i in range(b)]
    lens[0] = top
    Case(b, nq, hq, hkv, d, prefix, lens, seed=b).check()


def test_tall_row_tiles_over_a_long_prefix():
    # many rows per cache head: several tiles of rows share the prefix, the last one part full
    for b, nq, hq, hkv, d, prefix in ((35, 4, 16, 2, 128, 1500), (33, 8, 8, 1, 64, 2049), (70, 1, 32, 8, 128, 777),
                                      (9, 8, 32, 2, 128, 640)):
        Case(b, nq, hq, hkv, d, prefix, [nq + i % 5 for i in range(b)], page=64, seed=b).check()
    Case(40, 4, 8, 2, 96, 1000, [4] * 40, page=32, dtype=torch.float16, seed=5).check()


def test_fp32_outputs_strides_and_scale():
    c = Case(3, 3, 6, 2, 128, 90, [3, 50, 9], dtype=torch.float16, q_pad=64, seed=3)
    wide = torch.full((9, 6 * 128 + 8), 4.0, device=DEV)
    o, _ = c.check(o=wide[:, :768].unflatten(1, (6, 128)))
    assert bool((wide[:, 768:] == 4).all())
    heads = torch.zeros((6, 9, 128), dtype=torch.float16, device=DEV).transpose(0, 1)   # [tokens][heads] by strides
    c.check(o=heads)
    Case(2, 1, 4, 2, 64, 70, [9, 30], scale=0.4, seed=4).check(out_type=torch.float32)


def test_sharp_scores_and_a_dominating_key():
    c = Case(2, 2, 4, 2, 64, 500, [10, 30], spread=12.0, seed=6)
    c.check()
    c = Case(2, 1, 4, 2, 64, 500, [10, 30], seed=7)
    c.k[c.prefix_pages.long()[3], 5] = 30.0 * c.q[0, 0]  # one key far above the others for some rows
    c.check()


def test_no_key_at_all():
    for lens, nq in (([0, 0], 1), ([0, 2], 5)):
        c = Case(2, nq, 4, 2, 64, 0, lens, max_suffix=16, seed=8)
        out, lse = c.check()
        assert bool((out.view(2, nq, 4, 64)[0] == 0).all()) and bool((lse.view(2, nq, 4)[0] == float("-inf")).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_query_does_not_see_does_not_reach_it(bad):
    c = Case(2, 4, 6, 2, 64, 70, [30, 66], seed=9)
    clean = c.run().clone()
    for i in range(2):       # each sequence's last token: only its last query sees it
        j = c.lens[i] - 1
        c.v[c.suffix_pages[i, j // 16].long(), j % 16] = bad
        c.k[c.suffix_pages[i, j // 16].long(), j % 16] = bad
    out = c.run()
    torch.cuda.synchronize()
    a, b = out.view(2, 4, 6, 64), clean.view(2, 4, 6, 64)
    assert torch.equal(a[:, :3], b[:, :3])
    assert not bool(torch.isfinite(a[:, 3]).all())


def test_the_same_bits_again_and_with_other_sequences_beside():
    c = Case(5, 2, 8, 2, 64, 2000, [600, 3, 0, 64, 250], seed=10)
    first = c.run().clone()
    for _ in range(5):
        assert torch.equal(c.run(), first)


def test_lengths_and_tables_change_in_place():
    """A decode loop counts its device lengths up and calls again."""
    c = Case(2, 1, 6, 2, 64, 40, [60, 64], max_suffix=100, poison=False, seed=11)
    for lens in ([1, 30], [100, 0], [65, 99]):
        c.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        c.lens = lens
        c.check()


def test_pages_and_lengths_outside_are_recorded_and_unseen():
    c = Case(2, 1, 4, 2, 64, 64, [40, 20], page=16, seed=12)
    keep = c.prefix_pages.clone()
    for bad in (-1, c.cache.struct.n_pages, 2 ** 31 - 1):
        c.prefix_pages.copy_(keep)
        c.prefix_pages[3] = bad
        out = c.run()
        assert q.device_status() == 7
        # as if the prefix ended before its last page
        c.prefix_pages.copy_(keep)
        short = q.AttnBatch(2, 1, 4, c.cache, 48, c.prefix_pages, c.len_t, c.suffix_pages, 40)
        want = q.attn_prefix(c.q, short, c.ws)
        assert q.device_status() == 0
        assert float((out.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())
    c.len_t[0] = 41          # above max_suffix: counts as 40
    want = c.exact()[0]
    out = c.run()
    assert q.device_status() == 7
    assert float((out.double().view(want.shape) - want).abs().max()) < 2.0 ** -6
    c.len_t[0] = -3          # counts as 0
    out = c.run()
    assert q.device_status() == 7
    c.len_t[0], c.lens = 0, [0, 20]
    assert torch.equal(out, c.run()) and q.device_status() == 0


def test_another_stream_and_two_workspaces():
    a, b = Case(4, 1, 8, 2, 128, 3000, [50] * 4, seed=13), Case(4, 1, 8, 2, 128, 3000, [70] * 4, seed=14)
    wa, wb = a.run().clone(), b.run().clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    for _ in range(10):
        a.run(out=oa, stream=s1)
        b.run(out=ob, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, its rows at the far end."""
    page, hkv, d = 256, 8, 128
    pages = 2 ** 32 // (page * hkv * d) + 40
    if torch.cuda.mem_get_info()[0] < 4 * pages * page * hkv * d * 2:
        pytest.skip("needs 40 GB of device memory")
    k = torch.zeros((pages, page, hkv, d), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    small = Case(2, 2, 16, hkv, d, 500, [300, 77], page=page, dtype=torch.float16, poison=False, seed=15)
    n = small.k.shape[0]
    k[-n:], v[-n:] = small.k, small.v
    cache = q.KvCache(k, v)
    shift = pages - n
    batch = q.AttnBatch(2, 2, 16, cache, 500, small.prefix_pages + shift, small.len_t, small.suffix_pages + shift, 300)
    got = q.attn_prefix(small.q, batch, small.ws)
    assert torch.equal(got, small.run()) and q.device_status() == 0
    # and the cache write there
    plan = q.rope_plan(d, 1e4)
    x = torch.randn((3, hkv, d), device=DEV)
    slots = torch.tensor([pages * page - 1, 5, (pages - 1) * page], dtype=torch.int32, device=DEV)
    q.rope_kv(plan, None, x, x, torch.zeros(3, dtype=torch.int32, device=DEV), slots, cache)
    assert torch.equal(v.view(-1, hkv, d)[slots.long()], x.half()) and q.device_status() == 0


def test_four_dimensional_views():
    for b, nq in ((4, 1), (1, 4), (3, 2)):
        c = Case(b, nq, 6, 2, 64, 50, [nq + 3] * b, q_pad=256, seed=b)
        want, _ = c.check()
        got = q.attn_prefix(c.q.unflatten(0, (b, nq)), c.batch, c.ws)
        assert torch.equal(got.view(want.shape), want)


def test_a_captured_step_follows_its_lengths():
    """Rotary positions with the cache write and the attention in a CUDA graph,
    replayed as the device's lengths, slots and positions move on."""
    c = Case(3, 1, 6, 2, 64, 200, [1, 2, 3], max_suffix=40, poison=False, seed=20)
    plan = q.rope_plan(64, 1e4)
    x = torch.randn((3, (6 + 4) * 64), device=DEV)
    parts = (x[:, :384].unflatten(1, (6, 64)), x[:, 384:512].unflatten(1, (2, 64)), x[:, 512:].unflatten(1, (2, 64)))
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    rq, out = torch.empty((3, 6, 64), dtype=torch.bfloat16, device=DEV), torch.empty((3, 6, 64), dtype=torch.bfloat16, device=DEV)

    def step():
        q.rope_kv(plan, *parts, pos, slots, c.cache, out=rq)
        q.attn_prefix(rq, c.batch, c.ws, out=out)

    def place():
        j = (c.len_t - 1).long()
        slots.copy_(c.suffix_pages[torch.arange(3, device=DEV), j // 16] * 16 + (j % 16).int())
        pos.copy_(200 + j.int())

    place()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(4):
        c.len_t += 1
        x.normal_()
        place()
        g.replay()
        got = out.clone()
        step()
        assert torch.equal(out, got)
        c.lens = c.len_t.tolist()
        c.q = rq
        ref, A, _, e = c.exact()
        assert bool(((got.double().view(ref.shape) - ref).abs() <= (2.0 ** -8 + 2 * e + 2.0 ** -11) * A + 2.0 ** -8 * ref.abs()).all())
    assert q.device_status() == 0


# Many rows over a long prefix: six tiles of 64 rows and keys per slot of 304, the tcgen05 kernel.
@pytest.mark.parametrize("b,nq,hq,hkv,d,prefix,page,heads_first,dtype", [
    (12, 4, 16, 2, 128, 13000, 16, False, torch.bfloat16),     # 384 rows a head: a pair of tiles, and one and its absent half
    (9, 4, 16, 2, 128, 24064, 64, True, torch.float16),        # 288: the second tile of a pair part full; whole tiles of keys
    (10, 1, 56, 8, 128, 7700, 8, False, torch.bfloat16),       # 70: one row tile, its streams over alternate keys
    (16, 1, 64, 8, 64, 7425, 32, False, torch.float16),        # 128: the same, full, heads of 64
    (20, 2, 10, 2, 96, 15001, 256, False, torch.bfloat16),     # 200 rows, heads of 96
    (33, 8, 4, 1, 40, 23700, 128, True, torch.float16),        # 1056 rows, heads of 40
])
def test_tall_batches_over_long_prefixes(b, nq, hq, hkv, d, prefix, page, heads_first, dtype):
    c = Case(b, nq, hq, hkv, d, prefix, [nq + (7 * i) % 90 for i in range(b)], page=page, dtype=dtype,
             heads_first=heads_first, seed=b + d)
    c.check()
    first = c.run().clone()
    for _ in range(3):
        assert torch.equal(c.run(), first)


def test_tall_batches_with_sharp_scores():
    """Maxima that rise by far more than 2^8 from tile to tile: the sums are rescaled."""
    c = Case(12, 4, 16, 2, 128, 13000, [4] * 12, page=64, dtype=torch.bfloat16, spread=20.0, seed=31)
    c.check()
    c = Case(12, 4, 16, 2, 128, 13000, [4] * 12, page=64, dtype=torch.float16, seed=32)
    for j in (5000, 9999, 12900):
        c.k[c.prefix_pages.long()[j // 64], j % 64] *= 1 + j / 3000
    c.check()


def test_tall_batches_with_absent_pages():
    b, prefix, page = 12, 13000, 16
    c = Case(b, 4, 16, 2, 128, prefix, [4] * b, page=page, seed=33)
    keep = c.prefix_pages.clone()
    gone = [0, 17, 400, 811]
    c.prefix_pages[gone] = torch.tensor([-1, c.cache.struct.n_pages, 2 ** 31 - 1, -7], dtype=torch.int32, device=DEV)
    out = c.run()
    torch.cuda.synchronize()
    assert q.device_status() == 7
    rest = torch.cat([keep[[i for i in range(prefix // page) if i not in gone]], keep[-1:]])
    c.prefix_pages.copy_(keep)
    c.prefix_pages, c.prefix = rest, prefix - page * len(gone)
    ref, A, _, e = c.exact()
    got = out.double().view(ref.shape)
    assert bool(((got - ref).abs() <= (2.0 ** -8 + 2 * e + 2.0 ** -11) * A + 2.0 ** -8 * ref.abs()).all())


def test_tall_batches_without_suffixes_and_after_other_work():
    """No suffix part precedes the prefix kernel, and what it reads was written just before."""
    c = Case(40, 1, 64, 8, 128, 8000, [0] * 40, page=32, max_suffix=0, seed=34)
    c.check()
    src = [x.clone() for x in (c.k, c.v)]
    for i in range(5):
        c.k.zero_()
        c.v.zero_()
        big = torch.empty(1 << 28, device=DEV).zero_()
        c.k.copy_(src[0])
        c.v.copy_(src[1])
        out = c.run()
    assert torch.equal(out, c.run())
    c.check()
    del big


def test_a_long_prefix_written_by_the_launch_before():
    """The prefix kernel does not wait for the suffix parts, and must still see
    what the launch before those wrote: here the whole prefix, by rope_kv."""
    b, prefix, page, hkv, d = 12, 13000, 64, 2, 128
    c = Case(b, 4, 16, hkv, d, prefix, [60 + i for i in range(b)], page=page, poison=False, seed=40)
    want = c.run().clone()
    j = torch.arange(prefix, device=DEV)
    rows = (c.prefix_pages.long()[j // page] * page + j % page)
    k, v = (x.view(-1, hkv, d)[rows].clone() for x in (c.k, c.v))
    slots, zero = rows.to(torch.int32), torch.zeros(prefix, dtype=torch.int32, device=DEV)
    plan = q.rope_plan(d, 1e4)            # position 0 everywhere: copied as they are
    junk = torch.full_like(k, 50.0)
    for _ in range(20):
        q.rope_kv(plan, None, junk, junk, zero, slots, c.cache)
        c.run()
        q.rope_kv(plan, None, k, v, zero, slots, c.cache)
        out = c.run()
        assert torch.equal(out, want)
    assert q.device_status() == 0


class Wide(Case):
    """A case of many sequences: the same reference, all sequences and heads at once."""

    def exact(self):
        b, nq, hkv, d, top = self.b, self.nq, self.hkv, self.d, max(max(self.lens), 1)
        grp = self.hq // hkv
        x = self.q.double().view(b, nq, hkv, grp, d)
        j = torch.arange(self.prefix, device=DEV)
        shared = [t[self.prefix_pages.long()[j // self.page], j % self.page].double() for t in (self.k, self.v)]
        j = torch.arange(top, device=DEV).expand(b, top)
        there = j < torch.tensor(self.lens, device=DEV)[:, None]
        own = [torch.where(there[:, :, None, None], t[self.suffix_pages.long().gather(1, j // self.page), j % self.page].double(), 0.0)
               for t in (self.k, self.v)]
        last = torch.tensor(self.lens, device=DEV)[:, None] - nq + torch.arange(nq, device=DEV)     # [b, nq]
        hidden = (torch.arange(top, device=DEV) > last[:, :, None])[:, :, None, None, :]

        def scores(q_, ks, ko):
            s = torch.cat([torch.einsum("bqhgd,khd->bqhgk", q_, ks), torch.einsum("bqhgd,bkhd->bqhgk", q_, ko)], -1)
            return self.scale * s

        s = scores(x, shared[0], own[0])
        s[..., self.prefix:] = s[..., self.prefix:].masked_fill(hidden, float("-inf"))
        mag = scores(x.abs(), shared[0].abs(), own[0].abs())
        none = torch.isinf(s).all(-1, keepdim=True)
        w = torch.softmax(s, -1).masked_fill(none, 0.0)

        def weighted(vs, vo):
            return torch.einsum("bqhgk,khd->bqhgd", w[..., :self.prefix], vs) + torch.einsum("bqhgk,bkhd->bqhgd", w[..., self.prefix:], vo)

        shape = (b, nq, self.hq)
        return weighted(*(t for t in (shared[1], own[1]))).reshape(*shape, d), \
            weighted(shared[1].abs(), own[1].abs()).reshape(*shape, d), torch.logsumexp(s, -1).view(shape), \
            (d + 8) * 2.0 ** -24 * float(mag.max())


# So many rows that the tcgen05 kernel's share of work is met by one tile of 64
# keys: prefixes below, at and above the tile of 128 that it takes.
@pytest.mark.parametrize("prefix", [64, 100, 127, 128, 129, 200])
def test_very_tall_batches_on_short_prefixes(prefix):
    for b, nq, hq, hkv in ((228, 8, 64, 8), (227, 8, 64, 8), (456, 4, 64, 8)):
        Wide(b, nq, hq, hkv, 64, prefix, [(5 * i) % 12 for i in range(b)], seed=prefix + b).check()


# One key far above all others, whose values are all that there is to see.  The
# weights of the others are 2^-27 of the largest: below f16's exponents when the
# largest is 1, and a sum of a thousand of them is what the result consists of.
# Tolerance: that of the module without its n 2^-25, instead of which a weight is
# off by at most 2^-31 of the row's largest, w_max; so n 2^-31 w_max max |v|.
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,nq,hq,hkv,d,prefix,own,every", [
    (40, 1, 16, 8, 64, 0, 1024, 1 << 20),        # ranges of 1024 own keys, the first key far above
    (40, 1, 16, 8, 128, 0, 1024, 1 << 20),
    (3, 8, 8, 8, 256, 0, 1024, 64),
    (2, 1, 64, 2, 64, 4000, 2, 64),              # 64 rows: tiles of 16 rows a warp
    (12, 4, 16, 2, 128, 13000, 4, 128),          # the tcgen05 kernel, one such key in every tile
    (16, 1, 64, 8, 64, 7425, 8, 128),
])
def test_weights_far_below_the_largest_count(b, nq, hq, hkv, d, prefix, own, every, dtype):
    c = Wide(b, nq, hq, hkv, d, prefix, [own] * b, page=64, dtype=dtype, poison=False, seed=b, scale=math.log(2.0))
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k.zero_()
    c.v.copy_(50 + 50 * torch.rand(c.v.shape, device=DEV))
    for table, n in [(c.prefix_pages, prefix)] + [(t, own) for t in c.suffix_pages]:
        j = torch.arange(0, n if prefix == 0 or table is c.prefix_pages else 0, every, device=DEV)
        c.k[table.long()[j // 64], j % 64, :, 0] = 27.0
        c.v[table.long()[j // 64], j % 64] = 0.0
    out = torch.empty(c.q.shape, device=DEV)
    c.run(out=out)
    ref, A, lse, e = c.exact()
    assert q.device_status() == 0
    u, n = HALF_UNIT[dtype], prefix + own
    w_max = torch.exp(27.0 * math.log(2.0) - lse)[..., None]
    tol = (u + 2 * (e + 2.0 ** -21) + 2.0 ** -12 + 2.0 ** -24) * A
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -31 * w_max * 100.0
    got = out.double().view(ref.shape)
    assert bool((tol < ref / 4).all())               # so zeros would not do
    assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() / ref).max())


@pytest.mark.parametrize("b,nq,hq,hkv,d,prefix", [(5, 2, 8, 2, 64, 2000), (3, 1, 12, 2, 128, 160), (12, 4, 16, 2, 128, 13000),
                                                  (10, 1, 56, 8, 128, 7700), (40, 3, 8, 2, 96, 300)])
def test_other_sequences_beside(b, nq, hq, hkv, d, prefix):
    """A sequence's result is its own: the same bits whatever the others of its batch
    hold, and within both errors' bounds of its result in a batch of another size."""
    top = 150
    c = Case(b, nq, hq, hkv, d, prefix, [(i * 37) % (top + 1) for i in range(b)], max_suffix=top, poison=False, seed=b + d)
    o, lse = (t.clone() for t in c.check())
    mine = 1
    keep = c.q.view(b, nq, hq, d)[mine].clone()
    # other queries, lengths, own keys and values in all but one sequence
    c.q.normal_()
    c.q.view(b, nq, hq, d)[mine] = keep
    for i in range(b):
        if i != mine:
            rows = c.suffix_pages[i].long()
            c.k[rows], c.v[rows] = torch.randn_like(c.k[rows]), float("nan")
            c.v[rows[:2]] = 5.0
            c.len_t[i] = (11 * i + 3) % (2 * c.page)
    lse2 = torch.empty_like(lse)
    o2 = c.run(lse=lse2)
    assert torch.equal(o2.view(b, nq, hq, d)[mine], o.view(b, nq, hq, d)[mine])
    assert torch.equal(lse2.view(b, nq, hq)[mine], lse.view(b, nq, hq)[mine])
    # alone: another split of its keys
    alone = q.AttnBatch(1, nq, hq, c.cache, prefix, c.prefix_pages, c.len_t[mine:mine + 1].clone(),
                        c.suffix_pages[mine:mine + 1].clone(), top)
    a = q.attn_prefix(keep, alone, q.new_workspace(alone.workspace_bytes()))
    assert q.device_status() == 0
    c.b, c.lens, c.q = 1, [c.lens[mine]], keep
    c.suffix_pages = c.suffix_pages[mine:mine + 1]
    ref, A, _, e = c.exact()
    tol = (2.0 ** -8 + 2 * (e + 2.0 ** -21) + 2.0 ** -12) * A + 2.0 ** -8 * ref.abs() + 1e-30
    for got in (a, o2.view(b, nq, hq, d)[mine]):
        assert bool(((got.double().view(ref.shape) - ref).abs() <= tol).all())


@pytest.mark.parametrize("b", [16, 17])      # 128 rows a head: streams over alternate keys; 136: pairs of row tiles
def test_offsets_past_32_bits_through_tensor_maps(b):
    """A cache of more than 2^32 elements, a tall batch's long prefix at its far end."""
    page, hkv, d, prefix = 256, 8, 128, 7700
    pages = 2 ** 32 // (page * hkv * d) + 60
    if torch.cuda.mem_get_info()[0] < 4 * pages * page * hkv * d * 2:
        pytest.skip("needs 40 GB of device memory")
    small = Case(b, 4, 16, hkv, d, prefix, [4 + i for i in range(b)], page=page, dtype=torch.float16, poison=False, seed=b)
    n = small.k.shape[0]
    k = torch.zeros((pages, page, hkv, d), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    k[-n:], v[-n:] = small.k, small.v
    shift = pages - n
    batch = q.AttnBatch(b, 4, 16, q.KvCache(k, v), prefix, small.prefix_pages + shift, small.len_t, small.suffix_pages + shift,
                        max(small.lens))
    got = q.attn_prefix(small.q, batch, small.ws)
    assert torch.equal(got, small.run()) and q.device_status() == 0
    small.check()


# Scores so large that rounding the largest one's product with the scale moves it
# by whole units: tied keys must still share the weight, and nothing may overflow.
# The scores are exact in fp32 (one product each), the others lie 2^20 below, so
# the result is the mean of the tied keys' values: of 16-bit values times one
# weight, half a unit of it (u A) and the sums' roundings apart.
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,nq,hq,hkv,d,prefix,own", [(3, 2, 4, 2, 64, 300, 40), (2, 1, 64, 2, 128, 500, 10),
                                                      (12, 4, 16, 2, 128, 13000, 4), (16, 1, 64, 8, 64, 7425, 8)])
def test_tied_scores_of_any_size(b, nq, hq, hkv, d, prefix, own, dtype):
    for size in (2.0 ** 20, 2.0 ** 24, 2.0 ** 26, 2.0 ** 27):
        c = Wide(b, nq, hq, hkv, d, prefix, [own] * b, page=64, dtype=dtype, poison=False, seed=b, scale=0.3)
        kk = 2.0 ** 14                               # q stays within f16 at every size
        # q k scale log2(e) from size / 2 to size, in as many steps as there are rows
        steps = torch.linspace(0.5, 1.0, c.q.shape[0] * hq, device=DEV).view(c.q.shape[0], hq)
        c.q.zero_()
        c.q[..., 0] = (size / (kk * 0.3 * 1.4427) * steps).to(dtype)
        c.k.zero_()
        j = torch.arange(0, prefix, 7, device=DEV)
        c.k[c.prefix_pages.long()[j // 64], j % 64, :, 0] = kk
        out = torch.empty(c.q.shape, device=DEV)
        lse = torch.empty((b * nq, hq), device=DEV)
        c.run(out=out, lse=lse)
        assert q.device_status() == 0
        tied = c.v[c.prefix_pages.long()[j // 64], j % 64].double()
        want = tied.mean(0).repeat_interleave(hq // hkv, 0).expand(b * nq, hq, d)
        mag = tied.abs().mean(0).repeat_interleave(hq // hkv, 0)
        assert bool(((out.double() - want).abs() <= (HALF_UNIT[dtype] + 2.0 ** -12) * mag).all()), size
        l64 = 0.3 * kk * c.q[..., 0].double() + math.log(j.numel())
        assert bool(((lse.double() - l64).abs() <= 2.0 ** -22 * l64).all()), size


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_maximum_that_rises_little_at_large_scores(dtype):
    """Scores near 2^26.1 in powers of two, a later one 6.9 above the first tile's: less
    than the rise that moves the tcgen05 kernel's reference, but with the roundings of
    both products with the scale (up to 4 each) more.  Both scores are exact in fp32;
    the result is (v2 + w v1) / (1 + w) with w = exp(-0.3 * 16), to half a unit of the
    weights and the sums' 2^-12."""
    c = Wide(12, 4, 16, 2, 128, 13000, [4] * 12, page=64, dtype=dtype, poison=False, seed=50, scale=0.3)
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = 16384.0, 1.0
    c.k.zero_()
    place = [(c.prefix_pages.long()[j // 64], j % 64) for j in (5, 300)]
    for at, low in zip(place, (0.0, 16.0)):
        c.k[at][:, 0], c.k[at][:, 1] = 10240.0, low
    out, lse = torch.empty(c.q.shape, device=DEV), torch.empty((48, 16), device=DEV)
    c.run(out=out, lse=lse)
    assert q.device_status() == 0
    v1, v2 = (c.v[at].double() for at in place)
    w = math.exp(-4.8)
    want, mag = (v2 + w * v1) / (1 + w), (v2.abs() + w * v1.abs()) / (1 + w)
    want, mag = (t.repeat_interleave(8, 0).expand(48, 16, 128) for t in (want, mag))
    assert bool(((out.double() - want).abs() <= (HALF_UNIT[dtype] + 2.0 ** -12) * mag).all())
    l64 = 0.3 * (16384.0 * 10240.0 + 16.0) + math.log1p(w)
    assert bool(((lse.double() - l64).abs() <= 2.0 ** -22 * l64).all())
