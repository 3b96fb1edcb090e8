"""Rotary positions with the cache write (qgemv_rope_kv) against the formula
in 64 bits.

Tolerance, from the arithmetic: the angle is off by at most 2^-24 pi (its
conversion to fp32) plus sincospif's error (two units of 2^-24), the products
and their sum by three fp32 roundings: below 1e-6 mscale (|x| + |y|) in all,
then half a unit of the output's type.
"""
import math

import numpy as np
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


def theta(rot, base, scaling="plain", factor=1.0, orig=0.0, low=1.0, high=None):
    out = []
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        if scaling == "linear":
            t /= factor
        elif scaling == "bands":
            s = (orig * t / (2 * math.pi) - low) / ((high or 4.0) - low)
            s = min(1.0, max(0.0, s))
            t = t * ((1 - s) / factor + s)
        elif scaling == "yarn":
            def pair(n):
                return rot * math.log(orig / (2 * math.pi * n)) / (2 * math.log(base))
            a, b = max(0, math.floor(pair(high or 32.0))), min(rot - 1, math.ceil(pair(low)))
            w = min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
            t = t * (1 - w) + t / factor * w
        out.append(t)
    return np.array(out)


def rotated(x, pos, th, rot, layout, mscale=1.0):
    """float64 [n][heads][d] and the bound's |x| + |y| per element."""
    x = x.astype(np.float64)
    a = pos.astype(np.float64)[:, None] * th
    c, s = (mscale * np.cos(a))[:, None, :], (mscale * np.sin(a))[:, None, :]
    i = np.arange(rot // 2)
    ix, iy = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    out, mag = x.copy(), np.abs(x)
    out[..., ix] = x[..., ix] * c - x[..., iy] * s
    out[..., iy] = x[..., ix] * s + x[..., iy] * c
    mag[..., ix] = mag[..., iy] = mscale * (np.abs(x[..., ix]) + np.abs(x[..., iy]))
    return out, mag


def close(got, ref, mag, dtype):
    u = HALF_UNIT[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-38
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = 1e-6 * mag + u * (np.abs(ref) + 1e-6 * mag) + tiny
    assert np.all(err <= tol), float(np.max(err - tol))


def run(n, hq, hkv, d, rot, layout, tin, tq, tc, plan_args, top=4096, strided=False, page=16, seed=0, misalign=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    base = plan_args.pop("base", 1e4)
    plan = q.rope_plan(rot, base, layout=layout, **plan_args)
    width = (hq + 2 * hkv) * d
    pad = 3 if misalign else 16 if strided else 0
    buf = torch.randn((n, width + pad), generator=g, device=DEV).to(tin)
    off = 1 if misalign else 0
    row = buf[:, off:off + width]
    xq, xk, xv = row[:, :hq * d].view(n, hq, d) if not misalign else row[:, :hq * d].unflatten(1, (hq, d)), \
        row[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), row[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    pages = (n + page - 1) // page + 2
    ck = torch.full((pages, page, hkv, d), 7.0, device=DEV, dtype=tc)
    cv = torch.full((pages, page, hkv, d), 9.0, device=DEV, dtype=tc)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32)
    pos = torch.randint(0, top, (n,), generator=g, device=DEV).to(torch.int32)
    out = torch.empty((n, hq, d), dtype=tq, device=DEV)
    want_k, want_v = ck.double().cpu().numpy().reshape(-1, hkv, d), cv.double().cpu().numpy().reshape(-1, hkv, d)
    q.rope_kv(plan, xq, xk, xv, pos, slots, q.KvCache(ck, cv), out=out)
    torch.cuda.synchronize()
    assert q.device_status() == 0
    th = theta(rot, base, **{{"orig_len": "orig"}.get(k, k): v for k, v in plan_args.items()})
    ms = 0.1 * math.log(plan_args["factor"]) + 1 if plan_args.get("scaling") == "yarn" else 1.0
    p = pos.cpu().numpy()
    ref, mag = rotated(xq.float().cpu().numpy(), p, th, rot, layout, ms)
    close(out, ref, mag, tq)
    refk, magk = rotated(xk.float().cpu().numpy(), p, th, rot, layout, ms)
    s = slots.long().cpu().numpy()
    mags = np.zeros_like(want_k)
    want_k[s], mags[s] = refk, magk
    close(ck.view(-1, hkv, d), want_k, mags, tc)
    want_v[s] = xv.double().cpu().numpy()
    assert np.array_equal(cv.view(-1, hkv, d).double().cpu().numpy(),
                          torch.from_numpy(want_v).to(torch.float32).to(tc).double().numpy())


@pytest.mark.parametrize("n", [1, 2, 7, 333])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hkv,d,rot", [(12, 2, 128, 128), (14, 2, 64, 32), (3, 1, 96, 96), (4, 4, 256, 64),
                                          (2, 1, 8, 8), (5, 1, 128, 40)])
def test_layouts_and_heads(n, layout, hq, hkv, d, rot):
    run(n, hq, hkv, d, rot, layout, torch.float32, torch.bfloat16, torch.bfloat16, {}, seed=n + d)


# Enough tokens for blocks as narrow as their heads fill, with heads that leave
# a last turn short, in each layout and width of input.
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tin", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,d,rot", [(14, 2, 64, 16), (13, 3, 96, 96), (1, 1, 8, 8), (5, 2, 256, 64), (41, 5, 128, 64)])
def test_many_tokens(layout, tin, hq, hkv, d, rot):
    run(1723, hq, hkv, d, rot, layout, tin, torch.bfloat16, torch.float16, {}, top=30000, page=32, seed=hq + d)


@pytest.mark.parametrize("tin", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tq", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tc", [torch.float16, torch.bfloat16])
def test_types(tin, tq, tc):
    run(9, 6, 2, 64, 64, "half", tin, tq, tc, {}, seed=3)
    run(9, 6, 2, 64, 32, "interleaved", tin, tq, tc, {}, seed=4)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [2, 6, 22])
def test_sizes_without_wide_accesses(layout, rot):
    run(5, 3, 2, 24, rot, layout, torch.float32, torch.float32, torch.float16, {}, seed=rot)
    run(5, 3, 2, 24, 24, layout, torch.bfloat16, torch.float32, torch.bfloat16, {}, seed=rot, misalign=True)


def test_strided_rows():
    run(19, 12, 2, 128, 128, "half", torch.float16, torch.float16, torch.float16, {}, strided=True)


@pytest.mark.parametrize("args", [dict(scaling="linear", factor=4.0), dict(scaling="bands", factor=8.0, orig_len=8192),
                                  dict(scaling="yarn", factor=4.0, orig_len=32768),
                                  dict(scaling="yarn", factor=16.0, orig_len=64)])
@pytest.mark.parametrize("top", [4096, 1 << 20])
def test_scalings_and_long_positions(args, top):
    for base in (1e4, 1e6):
        run(257, 4, 2, 128, 128, "half", torch.float32, torch.float32, torch.bfloat16, dict(args, base=base), top=top,
            seed=top % 7)


def test_positions_at_the_ends_of_32_bits():
    """The angle's error stays that of its 53-bit frequency: 2^31 * 2^-54 turns."""
    plan = q.rope_plan(64, 1e4)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    x = torch.randn((5, 2, 64), device=DEV)
    out = torch.empty_like(x)
    q.rope_kv(plan, x, None, None, pos, out=out)
    th = theta(64, 1e4)
    # the reference's own product in extended precision
    a = pos.cpu().numpy().astype(np.longdouble)[:, None] * th.astype(np.longdouble)
    two_pi = np.longdouble("6.283185307179586476925286766559")
    frac = (a / two_pi) - np.rint(a / two_pi)
    c, s = np.cos((frac * two_pi).astype(np.float64)), np.sin((frac * two_pi).astype(np.float64))
    xs = x.double().cpu().numpy()
    ref = np.concatenate([xs[..., :32] * c[:, None] - xs[..., 32:] * s[:, None],
                          xs[..., :32] * s[:, None] + xs[..., 32:] * c[:, None]], -1)
    mag = np.abs(xs[..., :32]) + np.abs(xs[..., 32:])
    tol = (1e-6 + 2 * math.pi * 2.0 ** -22) * np.concatenate([mag, mag], -1)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


def test_tokens_without_a_row_and_rows_outside():
    n, hq, hkv, d = 6, 2, 2, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device=DEV)
    xq, xk, xv = x[:, :hq * d].view(n, hq, d), x[:, hq * d:(hq + hkv) * d].view(n, hkv, d), x[:, -hkv * d:].view(n, hkv, d)
    ck = torch.full((2, 4, hkv, d), 7.0, device=DEV, dtype=torch.float16)
    cv = torch.full((2, 4, hkv, d), 9.0, device=DEV, dtype=torch.float16)
    plan, pos = q.rope_plan(d, 1e4), torch.arange(n, dtype=torch.int32, device=DEV)
    slots = torch.tensor([-1, 3, -1, 0, 7, -1], dtype=torch.int32, device=DEV)
    out = q.rope_kv(plan, xq, xk, xv, pos, slots, q.KvCache(ck, cv))
    assert q.device_status() == 0
    th = theta(d, 1e4)
    ref, mag = rotated(xq.cpu().numpy(), pos.cpu().numpy(), th, d, "half")
    close(out, ref, mag, torch.float16)
    untouched = [1, 2, 4, 5, 6]
    assert torch.all(ck.view(8, hkv, d)[untouched] == 7) and torch.all(cv.view(8, hkv, d)[untouched] == 9)
    assert torch.equal(cv.view(8, hkv, d)[[3, 0, 7]], xv[[1, 3, 4]].half())
    # rows outside the cache: not written, recorded
    before = ck.clone()
    for bad in (8, -2, 2 ** 31 - 1):
        slots.fill_(bad)
        q.rope_kv(plan, xq, xk, xv, pos, slots, q.KvCache(ck, cv))
        assert q.device_status() == 7 and torch.equal(ck, before)


def test_in_place_and_parts_alone():
    n, hq, hkv, d = 11, 4, 2, 128
    x = torch.randn((n, (hq + 2 * hkv) * d), device=DEV).bfloat16()
    plan, pos = q.rope_plan(d, 1e6), torch.arange(100, 100 + n, dtype=torch.int32, device=DEV)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    caches = [[torch.zeros((1, 16, hkv, d), device=DEV, dtype=torch.bfloat16) for _ in range(2)] for _ in range(3)]

    def parts(b):
        return b[:, :hq * d].unflatten(1, (hq, d)), b[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), \
            b[:, (hq + hkv) * d:].unflatten(1, (hkv, d))

    want = q.rope_kv(plan, *parts(x), pos, slots, q.KvCache(*caches[0]))
    only_q = q.rope_kv(plan, parts(x)[0], None, None, pos)
    assert q.rope_kv(plan, None, *parts(x)[1:], pos, slots, q.KvCache(*caches[1])) is None
    y = x.clone()
    a = parts(y)
    q.rope_kv(plan, *a, pos, slots, q.KvCache(*caches[2]), out=a[0])
    torch.cuda.synchronize()
    assert torch.equal(want, only_q) and torch.equal(a[0], want) and torch.equal(y[:, hq * d:], x[:, hq * d:])
    for c in caches[1:]:
        assert torch.equal(c[0], caches[0][0]) and torch.equal(c[1], caches[0][1])


def test_heads_before_rows_and_another_stream():
    n, hkv, d, page = 40, 3, 64, 16
    k = torch.zeros((4, hkv, page, d), device=DEV, dtype=torch.float16)
    v = torch.zeros_like(k)
    x = torch.randn((n, hkv, d), device=DEV)
    plan, pos = q.rope_plan(d, 1e4), torch.zeros(n, dtype=torch.int32, device=DEV)
    slots = torch.randperm(4 * page, device=DEV)[:n].to(torch.int32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q.rope_kv(plan, None, x, x, pos, slots, q.KvCache(k.transpose(1, 2), v.transpose(1, 2)), stream=s)
    s.synchronize()
    want = torch.zeros((4 * page, hkv, d), device=DEV, dtype=torch.float16)
    want[slots.long()] = x.half()       # position 0: no rotation
    assert torch.equal(k.transpose(1, 2).reshape(-1, hkv, d), want)
    assert torch.equal(v.transpose(1, 2).reshape(-1, hkv, d), want)


def test_a_result_that_does_not_fit_is_out_of_memory():
    """As torch raises it: a caller that frees something and tries again catches that type."""
    x = torch.zeros((1, 4, 256), device=DEV).expand(1 << 30, 4, 256)      # 4 TB of results
    pos = torch.zeros((1,), dtype=torch.int32, device=DEV)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        q.rope_kv(q.rope_plan(64, 1e4), x, None, None, pos)
    y = torch.randn((1, 4, 256), device=DEV)
    assert torch.equal(q.rope_kv(q.rope_plan(64, 1e4), y, None, None, pos), y) and q.device_status() == 0
