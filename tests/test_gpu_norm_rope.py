"""Norms of q and k with rotary positions and the cache write
(qgemv_norm_rope_kv) against the formula in 64 bits.

Tolerance, from the arithmetic: the sum of d <= 256 squares in fp32 by fused steps and
shuffles is off by less than 40 roundings of 2^-24, of which the root takes half;
rsqrtf adds two units of 2^-23, the products with it and the weight 2^-24 each: the
normed element is off by less than 2^-19 of itself.  The rotation adds 1e-6
(|x| + |y|) (as rope_kv's), then half a unit of the output's type.
"""
import numpy as np
import pytest
import torch

import quantized_q4_weight_gb300 as q
from tests.test_gpu_rope import HALF_UNIT, rotated, theta

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_q4_weight_gb300 import _build
    _build.build()


def normed(x, w, eps):
    x = x.astype(np.float64)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w.astype(np.float64)


def close(got, ref, mag, dtype):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = (2.0 ** -19 + 1e-6) * mag
    tol = tol + HALF_UNIT[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == torch.float16 else 1e-38)
    assert np.all(err <= tol), float(np.max(err - tol))


def run(n, hq, hkv, d, rot, layout, tin, tq, tc, to_cache=True, misalign=False, strided=False, seed=0, scale=3.0, eps=1e-6,
        page=16, in_place=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    plan = q.rope_plan(rot, 1e4, layout=layout)
    width = (hq + 2 * hkv) * d
    pad = 3 if misalign else 16 if strided else 0
    off = 1 if misalign else 0
    buf = (scale * torch.randn((n, width + pad), generator=g, device=DEV)).to(tin)
    row = buf[:, off:off + width]
    xq, xk, xv = row[:, :hq * d].unflatten(1, (hq, d)), row[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), \
        row[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    wq, wk = (1 + 0.3 * torch.randn((d,), generator=g, device=DEV) for _ in range(2))
    pos = torch.randint(0, 4096, (n,), generator=g, device=DEV).to(torch.int32)
    norm = q.QkNorm(wq, wk, eps)
    hold = [x.float().cpu().numpy() for x in (xq, xk, xv)]
    out = xq if in_place else torch.empty((n, hq, d), dtype=tq, device=DEV)
    th, p = theta(rot, 1e4), pos.cpu().numpy()
    refq, magq = rotated(normed(hold[0], wq.cpu().numpy(), eps), p, th, rot, layout)
    refk, magk = rotated(normed(hold[1], wk.cpu().numpy(), eps), p, th, rot, layout)
    if not to_cache:
        k_out = torch.empty((n, hkv, d), dtype=tc, device=DEV)
        assert q.norm_rope_kv(plan, norm, xq, xk, None, pos, out=out, k_out=k_out) is out
        torch.cuda.synchronize()
        close(out, refq, magq, out.dtype)
        close(k_out, refk, magk, tc)
        assert q.device_status() == 0
        return
    pages = (n + page - 1) // page + 2
    ck = torch.full((pages, page, hkv, d), 7.0, device=DEV, dtype=tc)
    cv = torch.full((pages, page, hkv, d), 9.0, device=DEV, dtype=tc)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32)
    q.norm_rope_kv(plan, norm, xq, xk, xv, pos, slots, q.KvCache(ck, cv), out=out)
    torch.cuda.synchronize()
    assert q.device_status() == 0
    close(out, refq, magq, out.dtype)
    want = np.full((pages * page, hkv, d), 7.0)
    mags = np.zeros_like(want)
    s = slots.long().cpu().numpy()
    want[s], mags[s] = refk, magk
    close(ck.view(-1, hkv, d), want, mags, tc)
    want = torch.full((pages * page, hkv, d), 9.0)
    want[s] = torch.from_numpy(hold[2])
    assert torch.equal(cv.view(-1, hkv, d).cpu(), want.to(tc))


@pytest.mark.parametrize("n", [1, 2, 7, 400])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hkv,d,rot", [(12, 2, 128, 128), (14, 2, 64, 32), (3, 1, 96, 96), (4, 4, 256, 64),
                                          (2, 1, 8, 8), (5, 1, 128, 40), (40, 8, 128, 128)])
def test_norm_rope(n, layout, hq, hkv, d, rot):
    run(n, hq, hkv, d, rot, layout, torch.float32, torch.bfloat16, torch.bfloat16)
    run(n, hq, hkv, d, rot, layout, torch.bfloat16, torch.bfloat16, torch.float16, strided=True, seed=1)
    run(n, hq, hkv, d, rot, layout, torch.float16, torch.float32, torch.float16, to_cache=False, seed=2)


@pytest.mark.parametrize("tin", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tq", [torch.float32, torch.float16, torch.bfloat16])
def test_types(tin, tq):
    for tc in (torch.float16, torch.bfloat16):
        run(33, 6, 2, 64, 64, "half", tin, tq, tc)
    for tk in (torch.float32, torch.float16, torch.bfloat16):
        run(33, 6, 2, 64, 64, "interleaved", tin, tq, tk, to_cache=False)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 20), (256, 256), (10, 6), (2, 2)])
def test_unaligned(layout, d, rot):
    if d % 8 == 0:
        run(9, 3, 2, d, rot, layout, torch.float32, torch.float16, torch.float16, misalign=True)
    run(9, 3, 2, d, rot, layout, torch.float16, torch.float32, torch.float16, to_cache=False, misalign=True)


def test_in_place_and_extremes():
    run(50, 4, 2, 128, 128, "half", torch.bfloat16, torch.bfloat16, torch.bfloat16, in_place=True)
    run(50, 4, 2, 128, 128, "half", torch.float32, torch.float32, torch.bfloat16, scale=1e-9)
    run(50, 4, 2, 128, 128, "half", torch.float32, torch.float32, torch.bfloat16, scale=1e15, eps=1e-12)


def test_a_head_of_zeros_and_parts_left_out():
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    plan, w = q.rope_plan(64, 1e4), torch.ones(64, device=DEV)
    x = torch.randn((5, 4, 64), generator=g, device=DEV)
    x[2] = 0
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    both = q.norm_rope_kv(plan, q.QkNorm(w, w), x, x, None, pos, k_out=torch.empty_like(x))
    assert not bool(both[2].any()) and bool(torch.isfinite(both).all())
    only_q = q.norm_rope_kv(plan, q.QkNorm(w, None), x, None, None, pos)
    assert torch.equal(only_q, both)
    k_out = torch.empty_like(x)
    assert q.norm_rope_kv(plan, q.QkNorm(None, w), None, x, None, pos, k_out=k_out) is None
    assert torch.equal(k_out, both)
    # one token gives the bits that it has among others
    for i in range(5):
        assert torch.equal(q.norm_rope_kv(plan, q.QkNorm(w, None), x[i:i + 1], None, None, pos[i:i + 1]), both[i:i + 1])


def test_slots():
    """-1 writes no row; another slot outside the cache none either, and is recorded."""
    plan, w = q.rope_plan(32, 1e4), torch.ones(32, device=DEV)
    x = torch.ones((3, 2, 32), device=DEV)
    ck, cv = (torch.zeros((2, 16, 2, 32), dtype=torch.float16, device=DEV) for _ in range(2))
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad, status in ((-1, 0), (32, 7), (-5, 7)):
        slots = torch.tensor([4, bad, 9], dtype=torch.int32, device=DEV)
        ck.zero_()
        q.norm_rope_kv(plan, q.QkNorm(w, w), x, x, x, pos, slots, q.KvCache(ck, cv))
        assert q.device_status() == status
        assert sorted(set(ck.view(32, -1).any(1).nonzero().flatten().tolist())) == [4, 9]
