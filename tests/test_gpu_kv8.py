"""An 8-bit cache: qgemv_kv8_append against its definition (bit for bit: each step
is one fp32 operation) and qgemv_attn_kv8 against the softmax in 64 bits.

The attention's tolerance, from the arithmetic.  A weight enters its product in
f16, off by half a unit (2^-11 of it).  Its exponent is off by the d products'
fp32 sums (at most d 2^-23 of sum |q c| each) and by a few fp32 roundings of
numbers up to |score| + |log2 of the scale|, and so, relatively, is the weight;
the sum of the weights likewise.  So o is off by at most
(2^-11 + 2 e) sum p |v|, e = d 2^-23 S + 2^-20 (1 + T), with S the largest sum
|q k| scale and T the largest exponent, then half a unit of the output's type; lse by
2 e.  bf16 queries are exact operands but for elements below 2^-14 of their row's largest,
which are off by 2^-25 of it: d 2^-25 S more at most, within e.
"""
import math

import numpy as np
import pytest
import torch

import quantized_q4_weight_gb300 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
CODES = [torch.int8, torch.float8_e4m3fn]


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_q4_weight_gb300 import _build
    _build.build()


def gen(seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def encode(x, code):
    x = x.clamp(-TOP[code], TOP[code])
    return torch.round(x).to(torch.int8) if code == torch.int8 else x.to(code)


def make_cache(pages, page, block, heads, d, code, g, order="rows"):
    """A cache full of values; order: how pages lie in memory."""
    out = []
    for _ in range(2):
        shape = (pages, page, heads, d) if order == "rows" else (pages, heads, page, d)
        x = encode(torch.randn(shape, generator=g, device=DEV) * TOP[code] / 3, code)
        sshape = (pages, page // block, heads) if order == "rows" else (pages, heads, page // block)
        s = (0.3 + torch.rand(sshape, generator=g, device=DEV)) * 3 / TOP[code]
        out += [x, s] if order == "rows" else [x.transpose(1, 2), s.transpose(1, 2)]
    return q.Kv8Cache(out[0], out[2], out[1], out[3])


def make_table(lens, page, columns, pages, g):
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table, at = torch.full((len(lens), max(1, columns)), -7, dtype=torch.int32), 0
    for i, n in enumerate(lens):
        m = -(-n // page)
        table[i, :m] = order[at:at + m]
        at += m
    return table.to(DEV)


# ------------------------------------------------------------------ append

def append_ref(c, x, lens, table, first, codes, scale, page, block):
    """The definition, on the CPU: fp32 steps by numpy."""
    top = np.float32(TOP[codes.dtype])
    raw = codes.cpu().contiguous()
    val, sc = raw.float().numpy().copy(), scale.cpu().numpy().copy()
    x = x.float().cpu().numpy()

    def enc(v):
        v = np.nan_to_num(v, nan=0.0, posinf=float(top), neginf=-float(top))
        return encode(torch.from_numpy(v.astype(np.float32)), codes.dtype).float().numpy()

    for b, n in enumerate(lens):
        new = first[b + 1] - first[b]
        old = n - new
        for start in range(old // block * block, n if new else 0, block):
            lo, hi = max(start, old), min(start + block, n)
            pg, r, u = int(table[b, start // page]), start % page, start % page // block
            for h in range(val.shape[2]):
                part = x[first[b] + lo - old:first[b] + hi - old, h]
                was = sc[pg, u, h] if old > start else np.float32(0)
                now = np.fmax(was, np.float32(np.nanmax(np.append(np.abs(part), 0)) / top))
                with np.errstate(all="ignore"):
                    inv = np.float32(1) / now if now > 0 else np.float32(0)
                    if old > start and now > was:
                        val[pg, r:r + old - start, h] = enc(val[pg, r:r + old - start, h] * (was * inv))
                    val[pg, r + lo - start:r + hi - start, h] = enc(part * inv)
                sc[pg, u, h] = now
    return val, sc


def check_append(b, new, old, page, block, heads, d, tin, code, order="rows", ragged=False, seed=0, misalign=False, edit=None):
    g = gen(seed)
    rng = np.random.RandomState(seed)
    news = [int(rng.randint(0, new + 1)) for _ in range(b)] if ragged else [new] * b
    lens = [int(rng.randint(0, old + 1)) + n for n in news]
    columns = -(-max(max(lens), 1) // page)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(pages, page, block, heads, d, code, g, order)
    table = make_table(lens, page, columns, pages, g)
    first = np.concatenate([[0], np.cumsum(news)])
    n = int(first[-1])
    pad = 1 if misalign else 0
    buf = (2 * torch.randn((n, 2 * heads * d + pad), generator=g, device=DEV)).to(tin)
    if edit:
        edit(buf)
    xk, xv = (buf[:, pad + i * heads * d:pad + (i + 1) * heads * d].unflatten(1, (heads, d)) for i in range(2))
    batch = q.Kv8Batch(b, 1 if ragged else new, heads, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), table,
                       columns * page)
    t = table.cpu().numpy()
    want = [append_ref(cache, x, lens, t, first, c, s, page, block)
            for x, c, s in ((xk, cache.k, cache.k_scale), (xv, cache.v, cache.v_scale))]
    f = torch.tensor(first, dtype=torch.int32, device=DEV) if ragged else None
    for _ in range(2):  # a second time changes nothing
        q.kv8_append(xk, xv, batch, first=f, max_new=max(news) if ragged else None)
        torch.cuda.synchronize()
        assert q.device_status() == 0
        for (val, sc), c, s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
            assert np.array_equal(s.cpu().numpy(), sc)
            assert np.array_equal(c.float().cpu().numpy(), val)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("tin", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,new,old,page,block,heads,d", [(1, 1, 0, 16, 16, 1, 16), (3, 1, 70, 16, 16, 2, 128),
                                                          (5, 4, 200, 64, 32, 2, 96), (2, 8, 100, 64, 64, 3, 256),
                                                          (4, 1, 15, 128, 128, 8, 64)])
def test_append_tokens(b, new, old, page, block, heads, d, tin, code):
    check_append(b, new, old, page, block, heads, d, tin, code)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("b,new,old,page,block,heads,d", [(1, 300, 0, 16, 16, 1, 128), (6, 150, 90, 64, 32, 2, 64),
                                                          (3, 400, 30, 128, 128, 2, 256), (9, 3, 3, 16, 16, 2, 80)])
def test_append_ragged(b, new, old, page, block, heads, d, code):
    check_append(b, new, old, page, block, heads, d, torch.float32, code, ragged=True)
    check_append(b, new, old, page, block, heads, d, torch.bfloat16, code, order="heads", ragged=True, seed=3)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("tin", [torch.float32, torch.float16])
def test_append_unaligned(tin, code):
    check_append(2, 40, 20, 32, 16, 2, 48, tin, code, ragged=True, misalign=True)


@pytest.mark.parametrize("code", CODES)
def test_append_odd_values(code):
    def zeros(buf):
        buf[::2] = 0
    def nans(buf):
        buf[:, 5] = float("nan")
        buf[3] = float("nan")
    def tiny(buf):
        buf *= 1e-36
    def infinite(buf):
        buf[2, 7] = float("inf")
        buf[2, 300] = float("-inf")
    def growing(buf):
        buf *= torch.logspace(-3, 3, buf.shape[0], device=DEV)[:, None]
    for edit in (zeros, nans, tiny, growing):
        check_append(3, 8, 60, 32, 32, 2, 128, torch.float32, code, edit=edit)
    check_append(2, 3, 20, 64, 16, 2, 128, torch.float32, code, edit=infinite)
    check_append(1, 5, 0, 16, 16, 2, 128, torch.float32, code, edit=lambda buf: buf.zero_())


def test_append_scale_grows_over_calls():
    """Token after token, each larger than those before: old codes move to the new scale each time."""
    g = gen(5)
    cache = make_cache(2, 32, 32, 1, 64, torch.int8, g)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    batch = q.Kv8Batch(1, 1, 1, cache, lens, torch.tensor([[1]], dtype=torch.int32, device=DEV), 32)
    x = torch.randn((32, 1, 64), generator=g, device=DEV) * torch.linspace(0.1, 5.0, 32, device=DEV)[:, None, None]
    for i in range(32):
        lens.fill_(i + 1)
        q.kv8_append(x[i:i + 1], x[i:i + 1], batch)
    got = cache.k[1].float() * cache.k_scale[1, 0][None, :, None]
    # a value is rounded once when written and once for each growth after it; the scales add up to at most
    # sum_i s_i / 2, of which each is below the last one's
    assert float((got - x).abs().max()) <= 0.5 * 32 * float(cache.k_scale[1, 0, 0])
    assert float((got[-1] - x[-1]).abs().max()) <= 0.5 * float(cache.k_scale[1, 0, 0]) * (1 + 2.0 ** -20)
    assert torch.equal(cache.k, cache.k) and q.device_status() == 0


def test_append_bad_pages_and_lengths():
    """What does not lie in the cache is recorded and written nowhere."""
    g = gen(1)
    for case in ("page", "short", "long", "token"):
        cache = make_cache(4, 16, 16, 2, 64, torch.int8, g)
        lens = torch.tensor([5, 20], dtype=torch.int32, device=DEV)
        table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
        first = torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)
        x = torch.randn((6, 2, 64), generator=g, device=DEV)
        if case == "page":
            table[0, 0] = 4
        elif case == "short":
            lens[0] = 1         # fewer rows than tokens
        elif case == "long":
            lens[0] = 100       # counts as 32, whose last two rows are page 1's
            table[0, 1] = -1
        else:
            first[0] = -1
        k0, s0 = cache.k.clone(), cache.k_scale.clone()
        q.kv8_append(x, x, q.Kv8Batch(2, 1, 2, cache, lens, table, 32), first=first)
        assert q.device_status() == 7
        assert torch.equal(cache.k[:2], k0[:2]) and torch.equal(cache.k_scale[:2], s0[:2])
        # the other sequence has its rows 16 .. 19 on page 3
        val, sc = append_ref(None, x[2:], [20], np.array([[2, 3]]), [0, 4], k0, s0, 16, 16)
        assert np.array_equal(cache.k[2:].float().cpu().numpy(), val[2:])
        assert np.array_equal(cache.k_scale[2:].cpu().numpy(), sc[2:])


def test_padded_places_are_passed_over():
    """Sequences of length 0 write nothing and see nothing, with no error, whatever their tables name."""
    g = gen(23)
    cache = make_cache(6, 16, 16, 2, 64, torch.int8, g)
    lens = torch.tensor([0, 18, 0, 5], dtype=torch.int32, device=DEV)
    table = torch.tensor([[1, 2], [1, 2], [99, -4], [3, -1]], dtype=torch.int32, device=DEV)
    x = torch.randn((4, 2, 64), generator=g, device=DEV)
    batch = q.Kv8Batch(4, 1, 4, cache, lens, table, 32)
    k0, s0 = cache.k.clone(), cache.k_scale.clone()
    q.kv8_append(x, x, batch)
    val, sc = append_ref(None, x[[1, 3]], [18, 5], np.array([[1, 2], [3, -1]]), [0, 1, 2], k0, s0, 16, 16)
    assert np.array_equal(cache.k.float().cpu().numpy(), val) and np.array_equal(cache.k_scale.cpu().numpy(), sc)
    xq = torch.randn((4, 1, 4, 64), generator=g, device=DEV).to(torch.float16)
    out = q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes()))
    assert not bool(out[[0, 2]].any()) and bool(out[[1, 3]].any()) and q.device_status() == 0


# --------------------------------------------------------------- attention

def attn_ref(xq, cache, lens, table, nq, window, sinks, scale=None):
    """float64 o, lse [tokens][heads], the bound's sum p |v| and exponents' errors e."""
    codes = [c.float().cpu().double().numpy() for c in (cache.k, cache.v)]
    sc = [s.cpu().double().numpy() for s in (cache.k_scale, cache.v_scale)]
    pages, page, hkv, d = codes[0].shape
    block = page // sc[0].shape[1]
    k, v = (c * np.repeat(s, block, axis=1)[..., None] for c, s in zip(codes, sc))
    x = xq.double().cpu().numpy().reshape(len(lens), nq, -1, d)
    hq = x.shape[2]
    grp = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    o, mag, err = np.zeros_like(x), np.zeros_like(x), np.zeros(x.shape[:3])
    lse = np.full(x.shape[:3], -np.inf)
    t = table.cpu().numpy()
    tv = np.log2(np.maximum(sc[1], 2.0 ** -60))
    for b, n in enumerate(lens):
        for i in range(nq):
            p = n - nq + i
            rows = [j for j in range(p + 1) if (not window or j > p - window or j < sinks) and 0 <= t[b, j // page] < pages]
            if not rows:
                continue
            at = (t[b, np.array(rows) // page], np.array(rows) % page)
            for h in range(hq):
                kk, vv = k[at[0], at[1], h // grp], v[at[0], at[1], h // grp]
                s = kk @ x[b, i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                o[b, i, h], mag[b, i, h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum()
                lse[b, i, h] = m + np.log(w.sum())
                big = (np.abs(kk) @ np.abs(x[b, i, h])).max() * scale
                exps = np.abs(s).max() * 1.4427 + np.abs(tv).max()
                err[b, i, h] = d * 2.0 ** -23 * big + 2.0 ** -20 * (1 + exps)
    return o, lse.reshape(-1, hq), mag, err


def check_attn(lens, nq, hq, hkv, d, page, block, code, tq=torch.float16, window=0, sinks=0, to=None, order="rows", seed=0,
               scale=None, strided=False, max_len=None, edit=None, table_edit=None, spread=2.0, want=None):
    g = gen(seed)
    b, top = len(lens), max(max(lens), 1)
    columns = -(-top // page)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(pages, page, block, hkv, d, code, g, order)
    table = make_table(lens, page, columns, pages, g)
    if edit:
        edit(cache, table)
    if table_edit:
        table_edit(table)
    width = (hq + 2) * d if strided else hq * d
    xq = (spread * torch.randn((b * nq, width), generator=g, device=DEV)).to(tq)[:, :hq * d].view(b, nq, hq, d)
    batch = q.Kv8Batch(b, nq, hq, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), table,
                       columns * page if max_len is None else max_len, window=window, sinks=sinks, scale=scale)
    ws = q.new_workspace(batch.workspace_bytes())
    ws[16384:] = 0xFF  # what lies there before does not matter
    out = torch.full((b, nq, hq, d), 9.0, dtype=to or tq, device=DEV)
    lse = torch.full((b * nq, hq), 9.0, device=DEV)
    q.attn_kv8(xq, batch, ws, out=out, lse=lse)
    torch.cuda.synchronize()
    assert q.device_status() == (7 if want else 0)
    ref, ref_lse, mag, e = attn_ref(xq, cache, lens, table, nq, window, sinks, scale)
    got = out.double().cpu().numpy()
    tol = (2.0 ** -11 + 2 * e[..., None]) * mag * 1.01 + HALF_UNIT[to or tq] * np.abs(ref) * 1.01 + \
        (2.0 ** -25 if (to or tq) == torch.float16 else 1e-37)
    bad = np.abs(got - ref) - tol
    assert np.all(bad <= 0), (float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))
    gl = lse.double().cpu().numpy()
    seen = np.isfinite(ref_lse)
    assert np.array_equal(seen, np.isfinite(gl)) and np.all(gl[~seen] == -np.inf)
    el = 2 * e.reshape(gl.shape)[seen] + 2.0 ** -22 * np.abs(ref_lse[seen])
    assert np.all(np.abs(gl[seen] - ref_lse[seen]) <= el)
    return out, lse, batch, xq, ws


SHAPES = [(12, 2, 128), (14, 2, 64), (24, 4, 96), (3, 3, 16), (16, 1, 128), (4, 2, 256), (5, 1, 80), (8, 8, 64)]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("nq", [1, 3])
def test_attn_short(nq, hq, hkv, d, code):
    check_attn([1, 17, 0, 200, 16, 33, 2], nq, hq, hkv, d, 16, 16, code)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_attn_long(hq, hkv, d, code):
    """Ranges that cut units, one sequence much longer than the others."""
    check_attn([5, 3000, 0, 700, 1], 1, hq, hkv, d, 64, 32, code, tq=torch.bfloat16, seed=1)


@pytest.mark.parametrize("nq,hq,hkv,d", [(8, 16, 2, 128), (5, 16, 2, 64), (8, 8, 1, 256), (4, 24, 4, 96), (8, 64, 1, 128),
                                         (2, 40, 4, 128), (3, 8, 1, 128), (7, 4, 1, 64)])
@pytest.mark.parametrize("lens", [[9, 40, 300], [1200, 2, 0, 8]])
def test_attn_many_rows(nq, hq, hkv, d, lens):
    """Query rows in one to several tiles of 8 to 32."""
    check_attn(lens, nq, hq, hkv, d, 32, 16, torch.int8, seed=2)
    check_attn(lens, nq, hq, hkv, d, 32, 32, torch.float8_e4m3fn, tq=torch.bfloat16, to=torch.float32, seed=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (16, 4), (33, 40), (100, 16), (256, 0), (1000, 3), (5000, 2)])
@pytest.mark.parametrize("nq", [1, 4])
def test_attn_window(nq, window, sinks):
    check_attn([1, 3, 20, 64, 200, 777, 0], nq, 8, 2, 64, 16, 16, torch.int8, window=window, sinks=sinks, seed=4)
    check_attn([2100, 40], nq, 6, 2, 128, 64, 32, torch.float8_e4m3fn, window=window, sinks=sinks, seed=5)


@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (64, 64), (128, 32), (256, 256), (1024, 16)])
@pytest.mark.parametrize("order", ["rows", "heads"])
def test_attn_pages(page, block, order):
    check_attn([1500, 70, 129], 2, 8, 2, 128, page, block, torch.int8, order=order, seed=6)


@pytest.mark.parametrize("to", [torch.float32, torch.float16])
def test_attn_strided_q_scale_and_types(to):
    check_attn([100, 800], 2, 12, 2, 128, 16, 16, torch.int8, to=to, strided=True, scale=0.3, seed=7)
    check_attn([100, 800], 1, 12, 2, 128, 16, 16, torch.float8_e4m3fn, to=to, strided=True, spread=40.0, seed=8)


def test_attn_scales_far_apart():
    """Blocks whose scales differ by many powers of two, blocks of zeros among them."""
    def edit(cache, table):
        s = cache.v_scale
        s.copy_(torch.exp2(torch.randint(-30, 12, s.shape, generator=gen(9), device=DEV).float()))
        cache.v.view(torch.uint8)[::3] = 0
        s[::3] = 0
        cache.k.view(torch.uint8)[1::3] = 0
        cache.k_scale[1::3] = 0
    for code in CODES:
        check_attn([600, 90, 2000], 2, 8, 2, 128, 32, 16, code, edit=edit, seed=10, to=torch.float32)


def test_attn_bf16_query_range():
    """Rows of queries of any size: the largest power of two is divided out."""
    g = gen(11)
    cache = make_cache(8, 32, 16, 2, 128, torch.int8, g)
    lens, table = [100, 64], make_table([100, 64], 32, 4, 8, g)
    batch = q.Kv8Batch(2, 1, 4, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), table, 128, scale=1.0)
    base = torch.randn((2, 1, 4, 128), generator=g, device=DEV)
    ws = q.new_workspace(batch.workspace_bytes())
    plain = q.Kv8Batch(2, 1, 4, cache, batch.tables[0], table, 128, scale=2.0 ** 18)
    for e in (0, 60, -60, 100, -100):
        x = ((base * 2.0 ** -20).to(torch.bfloat16).float() * 2.0 ** e).to(torch.bfloat16)
        b2 = q.Kv8Batch(2, 1, 4, cache, batch.tables[0], table, 128, scale=2.0 ** (18 - e))
        # the same values times 2^-e, which is exact (x itself, at e = -100, has subnormal elements, already rounded)
        want = q.attn_kv8((x.double() * 2.0 ** -e).to(torch.bfloat16), plain, ws)
        assert torch.equal(q.attn_kv8(x, b2, ws), want), e
    assert bool(torch.isfinite(want).all()) and q.device_status() == 0


def test_attn_hidden_rows_hold_anything():
    """NaN codes and NaN scales in rows that are not seen: beyond a length, outside a window, in pages of no one."""
    lens, window, sinks, page, block = [50, 333, 7], 40, 4, 32, 16

    def poison(cache, table):
        t = table.cpu().numpy()
        seen = np.zeros((cache.k.shape[0], page), bool)
        blocks = np.zeros((cache.k.shape[0], page // block), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                if any(j <= p and (j > p - window or j < sinks) for p in (n - 2, n - 1)):
                    seen[t[b, j // page], j % page] = blocks[t[b, j // page], j % page // block] = True
        hide, hide_b = torch.from_numpy(~seen).to(DEV), torch.from_numpy(~blocks).to(DEV)
        for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            c.view(torch.uint8)[hide] = 0x7F
            s[hide_b] = float("nan")

    for code in CODES:
        g = gen(12)
        make_cache(30, page, block, 2, 128, code, g)
        clean = {}

        def run(edit):
            return check_attn_raw(lens, 2, 8, 2, 128, page, block, code, window, sinks, edit)
        a, la = run(None)
        b, lb = run(poison)
        assert torch.equal(a, b) and torch.equal(la, lb) and bool(torch.isfinite(b).all()), clean


def check_attn_raw(lens, nq, hq, hkv, d, page, block, code, window, sinks, edit, seed=13):
    g = gen(seed)
    columns = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(pages, page, block, hkv, d, code, g)
    table = make_table(lens, page, columns, pages, g)
    if edit:
        edit(cache, table)
    xq = torch.randn((len(lens), nq, hq, d), generator=g, device=DEV).to(torch.float16)
    batch = q.Kv8Batch(len(lens), nq, hq, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), table, columns * page,
                       window=window, sinks=sinks)
    lse = torch.empty((len(lens) * nq, hq), device=DEV)
    out = q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes()), lse=lse)
    assert q.device_status() == 0
    return out, lse


def test_attn_later_row_not_seen_by_earlier_query():
    """The last rows are seen by the last query only: an infinite scale there leaves the others whole."""
    g = gen(14)
    cache = make_cache(4, 32, 16, 2, 64, torch.int8, g)
    lens = torch.tensor([35], dtype=torch.int32, device=DEV)
    table = torch.tensor([[1, 2, 0]], dtype=torch.int32, device=DEV)
    xq = torch.randn((1, 4, 4, 64), generator=g, device=DEV).to(torch.float16)
    batch = q.Kv8Batch(1, 4, 4, cache, lens, table, 96)
    ws = q.new_workspace(batch.workspace_bytes())
    good = q.attn_kv8(xq, batch, ws)
    cache.v_scale[2, 0] = float("inf")   # rows 32 .. 34: query 0, at row 31, sees none of them
    bad = q.attn_kv8(xq, batch, ws)
    assert torch.equal(good[:, 0], bad[:, 0]) and not bool(torch.isfinite(bad[:, 1:]).any())


def test_attn_absent_pages_and_lengths():
    def drop(table):
        table[0, 1] = -1
        table[1, 3] = 1 << 20
    check_attn([300, 900, 40], 1, 8, 2, 128, 64, 16, torch.int8, table_edit=drop, want=True)
    check_attn([100, 90, 40], 2, 8, 2, 64, 32, 16, torch.float8_e4m3fn, table_edit=drop, want=True)
    g = gen(15)
    cache = make_cache(20, 16, 16, 2, 64, torch.int8, g)
    for top in (48, 1024):  # a block for each unit, ranges
        table = torch.arange(20, dtype=torch.int32, device=DEV)[:3].repeat(2, 1) if top == 48 else \
            (torch.arange(64, dtype=torch.int32, device=DEV) % 20).repeat(2, 1)
        xq = torch.randn((2, 1, 4, 64), generator=g, device=DEV).to(torch.bfloat16)

        def run(lens):
            batch = q.Kv8Batch(2, 1, 4, cache, torch.tensor(lens, dtype=torch.int32, device=DEV), table, top)
            return q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes()))
        a = run([-3, top + 9])
        assert q.device_status() == 7
        b = run([0, top])
        assert q.device_status() == 0 and torch.equal(a, b) and not bool(a[0].any())


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d", [80, 96])
@pytest.mark.parametrize("nq,hq,hkv", [(1, 8, 2), (3, 12, 3), (4, 24, 4), (5, 24, 4)])
def test_attn_heads_up_to_96(nq, hq, hkv, d, code):
    """One to four tiles of rows, whole and cut units."""
    check_attn([1, 17, 0, 200, 33, 600], nq, hq, hkv, d, 16, 16, code, seed=45)
    check_attn([1, 2300, 500], nq, hq, hkv, d, 64, 32, code, tq=torch.bfloat16, to=torch.float32, seed=46)


@pytest.mark.parametrize("nq,hq,hkv,d", [(8, 16, 2, 128), (5, 16, 2, 64), (8, 8, 1, 256), (4, 24, 4, 96), (1, 12, 2, 128)])
def test_attn_ranges(nq, hq, hkv, d):
    """Cut units of each kind of tile: with and without a window, pages of 16 and of 256 rows, pages of no one."""
    def drop(table):
        table[0, 3] = -1
        table[1, 1] = 1 << 20
    check_attn([2600, 40, 0, 1900], nq, hq, hkv, d, 16, 16, torch.int8, seed=41)
    check_attn([2600, 40, 0, 1900], nq, hq, hkv, d, 256, 128, torch.float8_e4m3fn, tq=torch.bfloat16, window=1700, sinks=70,
               seed=42)
    check_attn([2100, 900, 5000], nq, hq, hkv, d, 64, 32, torch.int8, window=2048, table_edit=drop, want=True, seed=43)


@pytest.mark.parametrize("seqs,nq,hq,hkv,d", [(76, 1, 8, 2, 128), (40, 4, 24, 4, 96), (100, 1, 12, 2, 64), (160, 2, 4, 2, 128)])
def test_attn_windows_that_fill_the_machine(seqs, nq, hq, hkv, d):
    """Units of a full window, a block each, and some of less."""
    lens = [int(x) for x in np.random.RandomState(seqs).randint(1200, 1400, seqs)]
    lens[3], lens[5], lens[-1] = 0, 17, 1025
    check_attn(lens, nq, hq, hkv, d, 64, 64, torch.float8_e4m3fn, window=1000, sinks=5, seed=44)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0, 5000, 0]])
def test_attn_empty(lens):
    for top in (None, 8192):
        check_attn(lens, 2, 8, 2, 128, 64, 64, torch.int8, max_len=max(max(lens), 64) if top is None else 5056 if max(lens) else 64)
    g = gen(16)
    cache = make_cache(2, 16, 16, 1, 32, torch.int8, g)
    batch = q.Kv8Batch(2, 1, 1, cache, torch.zeros(2, dtype=torch.int32, device=DEV), None, 0)
    xq = torch.ones((2, 1, 1, 32), dtype=torch.float16, device=DEV)
    assert not bool(q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes())).any()) and q.device_status() == 0


def test_attn_many_sequences():
    """More sequences than the ranges' walk takes: a block for each unit, whatever its length."""
    rng = np.random.RandomState(3)
    lens = [int(x) for x in rng.randint(0, 60, 1100)]
    lens[700] = 1500
    check_attn(lens, 1, 2, 1, 32, 32, 16, torch.int8, seed=17)


def test_attn_offsets_beyond_32_bits():
    """A cache of 5 GB a side: pages whose byte offsets pass 2^32."""
    g = gen(18)
    page, hkv, d = 64, 8, 128
    pages = 5 * (1 << 30) // (page * hkv * d)
    k = torch.zeros((pages, page, hkv, d), dtype=torch.int8, device=DEV)
    v = torch.zeros((pages, page, hkv, d), dtype=torch.int8, device=DEV)
    ks = torch.full((pages, 2, hkv), 0.01, device=DEV)
    vs = torch.full((pages, 2, hkv), 0.01, device=DEV)
    use = [pages - 1, 3, pages - 2, pages // 2]
    for c in (k, v):
        for p in use:
            c[p] = torch.randint(-127, 128, (page, hkv, d), generator=g, device=DEV, dtype=torch.int8)
    table = torch.tensor([use], dtype=torch.int32, device=DEV)
    xq = torch.randn((1, 1, 32, d), generator=g, device=DEV).to(torch.float16)
    lens = torch.tensor([250], dtype=torch.int32, device=DEV)
    batch = q.Kv8Batch(1, 1, 32, q.Kv8Cache(k, v, ks, vs), lens, table, 256)
    got = q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes()))
    small = q.Kv8Cache(k[use], v[use], ks[use], vs[use])
    batch = q.Kv8Batch(1, 1, 32, small, lens, torch.arange(4, dtype=torch.int32, device=DEV)[None], 256)
    assert torch.equal(got, q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes())))
    # a written row far behind
    x = torch.randn((1, hkv, d), generator=g, device=DEV)
    far = q.Kv8Batch(1, 1, 32, q.Kv8Cache(k, v, ks, vs), torch.tensor([1], dtype=torch.int32, device=DEV), table, 256)
    q.kv8_append(x, x, far)
    err = (k[pages - 1, 0].float() * ks[pages - 1, 0][:, None] - x[0]).abs().max()
    assert float(err) <= float(x.abs().max()) / 127 * 0.51


def test_attn_repeats_bit_for_bit_and_shares_a_workspace():
    out, lse, batch, xq, ws = check_attn([3000, 10, 700, 1900], 2, 16, 2, 128, 64, 32, torch.int8, seed=19)
    for _ in range(5):
        again = torch.empty_like(lse)
        assert torch.equal(out, q.attn_kv8(xq, batch, ws, lse=again)) and torch.equal(lse, again)
    assert not bool(ws[:16384].any())


def test_step_captured_and_replayed():
    """Append and attention in a graph, lengths and tokens updated between replays; an eager pass between them."""
    g = gen(20)
    b, hq, hkv, d, page = 3, 8, 2, 128, 32
    cache = make_cache(64, page, 16, hkv, d, torch.float8_e4m3fn, g)
    lens = torch.tensor([40, 700, 1], dtype=torch.int32, device=DEV)
    table = torch.randperm(64, generator=g, device=DEV).to(torch.int32)[:60].view(3, 20)
    table = torch.cat([table, table[:, :4]], 1).contiguous()
    batch = q.Kv8Batch(b, 1, hq, cache, lens, table, 640 + 64)
    ws = q.new_workspace(batch.workspace_bytes())
    xk, xv = (torch.randn((b, hkv, d), generator=g, device=DEV) for _ in range(2))
    xq = torch.randn((b, 1, hq, d), generator=g, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(xq)

    def step():
        q.kv8_append(xk, xv, batch)
        q.attn_kv8(xq, batch, ws, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    for i in range(4):
        lens.add_(torch.tensor([1, -100 if i == 2 else 1, 1], dtype=torch.int32, device=DEV))
        xk.normal_(generator=g)
        xv.normal_(generator=g)
        xq.copy_(torch.randn(xq.shape, generator=g, device=DEV))
        before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        after = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        for t, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
            t.copy_(s)
        step()
        assert torch.equal(got, out)
        for t, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), after):
            assert torch.equal(t.view(torch.uint8) if t.dtype != torch.float32 else t,
                               s.view(torch.uint8) if s.dtype != torch.float32 else s)
    assert q.device_status() == 0 and len(state) == 4


def test_other_stream():
    out, lse, batch, xq, ws = check_attn([1000, 77], 1, 8, 2, 128, 64, 32, torch.int8, seed=21)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = q.attn_kv8(xq, batch, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("nq,hq,hkv,d", [(1, 12, 2, 128), (1, 14, 2, 64), (4, 24, 4, 96), (2, 4, 2, 256)])
def test_attn_every_half_of_a_tile_has_its_own_scales(nq, hq, hkv, d, code):
    """Four lanes copy a tile's scales and all lanes use them: blocks of 16 rows whose scales of k and v are other
    powers of two from one half of a tile to the next, in units of their own and in ranges, the same bits each time."""
    def edit(cache, table):
        for k, s in enumerate((cache.k_scale, cache.v_scale)):
            s.copy_(torch.exp2(torch.randint(-9, -2, s.shape, generator=gen(60 + k), device=DEV).float()))
    for lens in ([5, 333, 700], [4000, 31]):
        out, lse, batch, xq, ws = check_attn(lens, nq, hq, hkv, d, 16, 16, code, edit=edit, seed=61)
        for _ in range(10):
            again = torch.empty_like(lse)
            assert torch.equal(out, q.attn_kv8(xq, batch, ws, out=torch.empty_like(out), lse=again)) and torch.equal(lse, again)


def test_attn_reads_one_scale_for_a_whole_cache():
    """Expanded scales, strides of 0: the same bits as with a scale for each; what writes them refuses."""
    g = gen(62)
    cache = make_cache(20, 32, 16, 2, 64, torch.int8, g)
    one = [torch.tensor([[[s]]], device=DEV) for s in (0.02, 0.03)]
    shared = q.Kv8Cache(cache.k, cache.v, *(x.expand(20, 2, 2) for x in one))
    each = q.Kv8Cache(cache.k, cache.v, *(x.expand(20, 2, 2).contiguous() for x in one))
    lens, table = torch.tensor([300, 70], dtype=torch.int32, device=DEV), make_table([300, 70], 32, 10, 20, g)
    xq = torch.randn((2, 1, 8, 64), generator=g, device=DEV).to(torch.float16)
    outs = []
    for c in (shared, each):
        batch = q.Kv8Batch(2, 1, 8, c, lens, table, 320)
        outs.append(q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes())))
    assert torch.equal(*outs)
    x = torch.randn((2, 2, 64), generator=g, device=DEV)
    with pytest.raises(Exception, match="qgemv_kv8_append"):
        q.kv8_append(x, x, q.Kv8Batch(2, 1, 8, shared, lens, table, 320))
    with pytest.raises(Exception, match="qgemv_fork_pages"):
        q.fork_pages(q.PagePool([shared]), lens * 0, lens, table, lens * 0 - 1, torch.zeros_like(table), torch.zeros_like(lens))


@pytest.mark.parametrize("code", CODES)
def test_k_and_v_in_one_buffer(code):
    """[pages][2][rows][heads][d] and scales beside it: what caches of their own give, step by step."""
    g = gen(63)
    cache = make_cache(12, 32, 16, 2, 64, code, g)
    both = torch.stack([cache.k.view(torch.uint8), cache.v.view(torch.uint8)], 1).view(code)
    scales = torch.stack([cache.k_scale, cache.v_scale], 1)
    one = q.Kv8Cache(both[:, 0], both[:, 1], scales[:, 0], scales[:, 1])
    lens, table = torch.tensor([70, 200], dtype=torch.int32, device=DEV), make_table([70, 200], 32, 7, 12, g)
    x = [3 * torch.randn((6, 2, 64), generator=g, device=DEV) for _ in range(2)]
    xq = torch.randn((2, 3, 8, 64), generator=g, device=DEV).to(torch.float16)
    outs = []
    for c in (cache, one):
        batch = q.Kv8Batch(2, 3, 8, c, lens, table, 224)
        q.kv8_append(*x, batch)
        outs.append(q.attn_kv8(xq, batch, q.new_workspace(batch.workspace_bytes())))
    assert torch.equal(*outs) and q.device_status() == 0
    for a, b in ((cache.k, one.k), (cache.v, one.v), (cache.k_scale, one.k_scale), (cache.v_scale, one.v_scale)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("code", CODES)
def test_append_row_after_row_is_the_definition(code):
    """Forty rows, one a call, each larger than those before: the codes and scales of every step bit for bit, the
    rounding of old codes to each new scale among them; pages of no one stay as they were."""
    g = gen(64)
    cache = make_cache(5, 16, 16, 2, 64, code, g)
    lens, table = torch.zeros(1, dtype=torch.int32, device=DEV), torch.tensor([[3, 0, 4]], dtype=torch.int32, device=DEV)
    batch = q.Kv8Batch(1, 1, 2, cache, lens, table, 48)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    x = torch.randn((2, 40, 2, 64), generator=g, device=DEV) * torch.linspace(0.1, 5.0, 40, device=DEV)[:, None, None]
    for i in range(40):
        want = [append_ref(cache, x[j, i:i + 1], [i + 1], table.cpu().numpy(), [0, 1], c, s, 16, 16)
                for j, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale)))]
        lens.fill_(i + 1)
        q.kv8_append(x[0, i:i + 1], x[1, i:i + 1], batch)
        for (val, sc), c, s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
            assert np.array_equal(c.float().cpu().numpy(), val) and np.array_equal(s.cpu().numpy(), sc), i
    for t, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        assert torch.equal(t[1:3].contiguous().view(torch.uint8), was[1:3].contiguous().view(torch.uint8))
    assert torch.equal(cache.k[4, 8:].view(torch.uint8), before[0][4, 8:].view(torch.uint8)) and q.device_status() == 0
