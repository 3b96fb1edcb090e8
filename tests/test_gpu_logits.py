"""Rules on logits (qgemv_logits_rules) against a loop in numpy.

The rules are single fp32 operations in a stated order, so the reference
takes them in float32 one by one (numpy rounds each to nearest) and the
results must be equal bit for bit (-0 and +0 alike); against 64 bits each row is
within the roundings' bound.
"""
import numpy as np
import pytest
import torch

import quantized_q4_weight_gb300 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_q4_weight_gb300 import _build
    _build.build()


def reference(x, hist, hist_len, rep, freq, pres, bias_ids, bias, bias_len, mask, f=np.float32):
    out = x.astype(f)
    R, V = x.shape
    for r in range(R):
        if hist is not None:
            ids = hist[r, :hist_len[r]]
            ids = ids[(ids >= 0) & (ids < V)]
            tok, c = np.unique(ids, return_counts=True)
            v = out[r, tok]
            re, fr, pr = (f(a[r]) if a is not None else f(d) for a, d in ((rep, 1), (freq, 0), (pres, 0)))
            v = np.where(v > 0, v / re, v * re).astype(f)
            v = (v - (fr * c.astype(f)).astype(f)).astype(f)
            out[r, tok] = (v - pr).astype(f)
        if bias is not None:
            for t, b in {int(t): b for t, b in zip(bias_ids[r, :bias_len[r]], bias[r, :bias_len[r]])}.items():
                if 0 <= t < V:
                    out[r, t] = f(out[r, t] + f(b))
        if mask is not None:
            m = mask[r if mask.shape[0] > 1 else 0]
            bits = np.unpackbits(m.view(np.uint8), bitorder="little")[:V].astype(bool)
            out[r, ~bits] = -np.inf
    idx = np.full(R, -1, np.int64)
    val = np.full(R, -np.inf, f)
    for r in range(R):
        row = np.where(np.isnan(out[r]), -np.inf, out[r])
        if row.max() > -np.inf:
            idx[r] = int(np.flatnonzero(row == row.max())[0])
            val[r] = row.max()
    return out, idx, val


def make(R, V, hist, bias, dtype, seed, p_mask=0.4):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((4 * rng.standard_normal((R, V))).astype(np.float32)).to(dtype)
    d = dict(hist=None, hist_len=None, rep=None, freq=None, pres=None, bias_ids=None, bias=None, bias_len=None, mask=None)
    if hist:
        d["hist"] = np.minimum((V ** rng.random((R, hist))).astype(np.int64), V + 2) - 1
        d["hist_len"] = rng.integers(0, hist + 1, R).astype(np.int32)
        d["hist_len"][0] = hist
        for n, lo, hi in (("rep", 0.8, 1.8), ("freq", -0.2, 0.8), ("pres", 0, 1)):
            d[n] = rng.uniform(lo, hi, R).astype(np.float32)
    if bias:
        d["bias_ids"] = rng.integers(-1, V + 1, (R, bias)).astype(np.int64)
        d["bias"] = (3 * rng.standard_normal((R, bias))).astype(np.float32)
        d["bias_len"] = rng.integers(0, bias + 1, R).astype(np.int32)
    if p_mask is not None:
        d["mask"] = np.packbits(rng.random((R, (V + 31) // 32 * 32)) < p_mask, axis=1, bitorder="little").view(np.int32)
    return x, d


def call(x, d, out=None, ws=None, xd=None):
    R, V = x.shape
    t = {k: (None if v is None else torch.from_numpy(v).to(DEV)) for k, v in d.items()}
    rules = q.LogitsRules(R, V, history=t["hist"], history_len=t["hist_len"], repetition=t["rep"], frequency=t["freq"],
                          presence=t["pres"], bias_ids=t["bias_ids"], bias=t["bias"], bias_len=t["bias_len"],
                          mask=t["mask"])
    xd = x.to(DEV) if xd is None else xd
    ws = q.new_workspace(rules.workspace_bytes()) if ws is None else ws
    return q.logits_rules(xd, rules, ws, out=out)


def check(x, d, **kw):
    want, idx, val = reference(x.float().numpy(), **d)
    out = torch.full(x.shape, 77.0, dtype=x.dtype, device=DEV)
    gi, gv = call(x, d, out=out, **kw)
    torch.cuda.synchronize()
    assert q.device_status() == 0
    stored = torch.from_numpy(want).to(x.dtype)
    assert torch.equal(torch.nan_to_num(out.cpu().float(), nan=123.0), torch.nan_to_num(stored.float(), nan=123.0))
    assert np.array_equal(gi.cpu().numpy(), idx) and np.array_equal(gv.cpu().numpy(), val)
    # and against the rules in 64 bits: five roundings of values below the row's largest step
    w64, _, v64 = reference(x.float().numpy(), **{k: (v.astype(np.float64) if v is not None and v.dtype == np.float32 else v)
                                                 for k, v in d.items()}, f=np.float64)
    fin = np.isfinite(w64)
    c = 0 if d["hist"] is None else d["hist"].shape[1]
    assert np.all(np.abs(want[fin] - w64[fin]) <= 5 * 2.0 ** -24 * (2 * np.abs(x.float().numpy()[fin]) + c + 16))
    return gi, gv


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(1, 1), (2, 31), (3, 33), (1, 2048), (4, 5001), (2, 50257), (70, 777), (1, 151936)])
def test_sizes_and_types(R, V, dtype):
    x, d = make(R, V, 60, 9, dtype, R * 31 + V)
    check(x, d)


@pytest.mark.parametrize("hist,bias,p_mask", [(0, 0, None), (0, 0, 0.2), (40, 0, None), (0, 12, None), (3000, 0, 0.9),
                                             (1, 1, 0.5), (500, 4095, 0.5)])
def test_each_rule_alone_and_together(hist, bias, p_mask):
    x, d = make(5, 4099, hist, bias, torch.float32, 7 + hist + bias, p_mask)
    check(x, d)


def test_one_rule_of_the_three_penalties():
    for keep in ("rep", "freq", "pres"):
        x, d = make(3, 900, 50, 0, torch.float32, 11, None)
        check(x, {k: (None if k in ("rep", "freq", "pres") and k != keep else v) for k, v in d.items()})


def test_many_rows_share_one_launch_and_more_take_two():
    x, d = make(1100, 515, 20, 3, torch.bfloat16, 3)
    check(x, d)
    x, d = make(700, 9000, 16, 2, torch.float32, 4)
    check(x, d)


def test_many_slices_of_one_row():
    # one row in slices, 32 rows in fewer and longer ones, every slice up to its bound
    for R in (1, 3, 32):
        x, d = make(R, 140001, 4000, 50, torch.float32, R)
        check(x, d)


def test_ties_empty_rows_infinities_and_nan():
    V = 5000
    x = torch.zeros((9, V))
    x[0, 100:] = -0.0                                # -0 == +0: token 0
    x[1] = -5.0
    x[1, [4444, 17]] = 2.5                           # tie across slices
    x[2] = float("-inf")                             # nothing to choose
    x[3] = float("nan")
    x[3, 4000] = -3.0                                # NaN is passed over
    x[4] = float("nan")                              # everywhere masked, below
    x[5] = float("nan")
    x[5, 9] = float("-inf")
    x[6, 77] = float("inf")
    x[7] = torch.finfo(torch.float32).min            # the type's lowest value is above -infinity
    x[8, 3] = float("inf")                           # masked
    mask = np.full((9, (V + 31) // 32), -1, np.int32)
    mask[4] = 0
    mask[8, 0] = ~(1 << 3)
    d = dict(hist=None, hist_len=None, rep=None, freq=None, pres=None, bias_ids=None, bias=None, bias_len=None, mask=mask)
    gi, gv = check(x, d)
    assert gi.tolist() == [0, 17, -1, 4000, -1, -1, 77, 0, 0]
    assert gv[2] == float("-inf") and gv[4] == float("-inf")
    out = torch.empty((9, V), device=DEV)
    call(x, d, out=out)
    assert torch.all(out[4] == float("-inf")) and out[8, 3] == float("-inf")


def test_in_place_strided_and_without_outputs():
    x, d = make(4, 3001, 30, 5, torch.float16, 21)
    want, idx, val = reference(x.float().numpy(), **d)
    xd = x.to(DEV)
    gi, gv = call(x, d, out=xd, xd=xd)               # in place
    assert torch.equal(xd.cpu(), torch.from_numpy(want).half())
    wide = torch.full((4, 3100), 5.0, dtype=torch.float16, device=DEV)
    wide[:, 3:3004] = x.to(DEV)
    outw = torch.full((4, 4000), 6.0, dtype=torch.float16, device=DEV)
    o = outw[:, 2:3003]
    gi2, _ = call(x, d, out=o, xd=wide[:, 3:3004])   # other alignment on both sides
    assert torch.equal(o.cpu(), torch.from_numpy(want).half())
    assert torch.all(outw[:, :2] == 6) and torch.all(outw[:, 3003:] == 6)
    gi3, gv3 = call(x, d)                            # the token only
    for g in (gi, gi2, gi3):
        assert np.array_equal(g.cpu().numpy(), idx)
    assert np.array_equal(gv3.cpu().numpy(), val)


def test_one_mask_for_all_rows_and_a_shared_workspace():
    x, d = make(6, 2500, 10, 2, torch.float32, 8)
    d["mask"] = d["mask"][:1].copy()
    ws = q.new_workspace(1 << 16)
    for _ in range(3):
        check(x, d, ws=ws)
    assert int(ws[:16384].int().sum()) == 0          # the counter area is zero again


def test_lengths_outside_their_bounds_are_recorded():
    x, d = make(3, 1000, 20, 4, torch.float32, 5)
    for name, bad, used in (("hist_len", 21, 20), ("hist_len", -1, 0), ("bias_len", 5, 4), ("bias_len", -7, 0)):
        e = dict(d)
        e[name] = d[name].copy()
        e[name][1] = used
        _, idx, val = reference(x.float().numpy(), **e)
        e[name] = e[name].copy()
        e[name][1] = bad
        gi, gv = call(x, e)
        assert q.device_status() == 7
        assert np.array_equal(gi.cpu().numpy(), idx) and np.array_equal(gv.cpu().numpy(), val)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,hist,bias", [(64, 120007, 600, 30), (300, 50257, 3000, 200), (40, 151936, 0, 0),
                                           (90, 70001, 9000, 64), (60, 99999, 20000, 4000), (1024, 8191, 33, 5)])
def test_many_rows_in_ranges(R, V, hist, bias, dtype):
    """Enough tokens for the blocks to take ranges that cross rows, lists of every size class."""
    x, d = make(R, V, hist, bias, dtype, R + V)
    check(x, d)


def test_many_rows_in_place_and_strided():
    x, d = make(100, 60001, 100, 9, torch.float16, 77)
    want, idx, _ = reference(x.float().numpy(), **d)
    xd = x.to(DEV)
    gi, _ = call(x, d, out=xd, xd=xd)
    assert torch.equal(xd.cpu(), torch.from_numpy(want).half()) and np.array_equal(gi.cpu().numpy(), idx)
    wide = torch.full((100, 60021), 5.0, dtype=torch.float16, device=DEV)
    wide[:, 5:60006] = x.to(DEV)
    outw = torch.full((100, 60100), 6.0, dtype=torch.float16, device=DEV)
    gi, _ = call(x, d, out=outw[:, 6:60007], xd=wide[:, 5:60006])
    assert torch.equal(outw[:, 6:60007].cpu(), torch.from_numpy(want).half()) and np.array_equal(gi.cpu().numpy(), idx)
    assert torch.all(outw[:, :6] == 6) and torch.all(outw[:, 60007:] == 6)


def test_results_made_by_the_call_are_tensors_of_their_own_kind():
    x, d = make(3, 500, 10, 2, torch.float32, 9)
    gi, gv = call(x, d)
    idx, val = torch.empty(3, dtype=torch.int64, device=DEV), torch.empty(3, device=DEV)
    t = {k: (None if v is None else torch.from_numpy(v).to(DEV)) for k, v in d.items()}
    rules = q.LogitsRules(3, 500, history=t["hist"], history_len=t["hist_len"], repetition=t["rep"], frequency=t["freq"],
                          presence=t["pres"], bias_ids=t["bias_ids"], bias=t["bias"], bias_len=t["bias_len"], mask=t["mask"])
    ws = q.new_workspace(rules.workspace_bytes())
    for kw in (dict(idx=idx), dict(val=val), dict(idx=idx, val=val)):
        a, b = q.logits_rules(x.to(DEV), rules, ws, **kw)
        assert torch.equal(a, gi) and torch.equal(b, gv)
        assert ("idx" not in kw or a is idx) and ("val" not in kw or b is val)
    assert gi.dtype == torch.int64 and gv.dtype == torch.float32 and gi.shape == gv.shape == (3,) and gi.is_contiguous()
    assert torch.equal(gi + 1 - 1, gi) and (gv * 2).shape == (3,) and gi.cpu().tolist() == gi.tolist()
    assert gi.device == x.to(DEV).device and not gv.requires_grad


def test_results_made_by_the_call_are_saved_together():
    """Index and value have storages of their own: one type a storage, as a file of tensors wants it."""
    import io
    x, d = make(3, 500, 10, 2, torch.float32, 12)
    gi, gv = call(x, d)
    assert gi.untyped_storage().data_ptr() != gv.untyped_storage().data_ptr()
    assert gi.untyped_storage().nbytes() == 24 and gv.untyped_storage().nbytes() == 12
    f = io.BytesIO()
    torch.save((gi, gv), f)
    f.seek(0)
    a, b = torch.load(f)
    assert torch.equal(a, gi) and torch.equal(b, gv)


@pytest.mark.parametrize("which", ["hist", "bias", "both"])
def test_lists_without_columns(which):
    """The first step of a loop: a history or bias list with room for nothing touches nothing."""
    x, d = make(3, 700, 4, 3, torch.float32, 13)
    for name in ("hist", "bias_ids", "bias"):
        if which == "both" or name.startswith(which):
            d[name] = np.ascontiguousarray(d[name][:, :0])
    for name, kind in (("hist_len", "hist"), ("bias_len", "bias")):
        if which in (kind, "both"):
            d[name][:] = 0
    check(x, d)
    # a length past the bound counts as the bound, and is recorded
    e = dict(d)
    name = "bias_len" if which == "bias" else "hist_len"
    e[name] = d[name].copy()
    e[name][1] = 1
    _, idx, val = reference(x.float().numpy(), **d)
    gi, gv = call(x, e)
    assert q.device_status() == 7
    assert np.array_equal(gi.cpu().numpy(), idx) and np.array_equal(gv.cpu().numpy(), val)
