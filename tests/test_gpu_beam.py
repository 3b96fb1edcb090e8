"""Beam search's selection (qgemv_beam_select) and the reordering of pages
(qgemv_fork_pages) against plain implementations.

The selection is compared as whole numbers with a sort of the scores in 64 bits;
where two neighbours of that order lie closer than 1e-5 (the fp32 sums of
exponentials may be off by that: 2^-22 for each term and 2^-24 of a logit times
log2 e for its exponent, below 1e-5 for logits up to 64) the inputs are changed
beforehand, on the CPU, until none do.  Scores are off by at most that and half a
unit of fp32.
"""
import numpy as np
import pytest
import torch

import quantized_q4_weight_gb300 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
NEAR = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_q4_weight_gb300 import _build
    _build.build()


def select_ref(x, scores, n, done=None):
    """x float64 [groups][beams][vocab] -> score, token, row and the smallest gap between rows of neighbours."""
    groups, beams, vocab = x.shape
    out = (np.full((groups, n), -np.inf), np.full((groups, n), -1), np.full((groups, n), -1))
    gap = np.inf
    for g in range(groups):
        c = []
        for b in range(beams):
            run = float(scores[g, b])
            if not run > -np.inf:
                continue
            if done is not None and done[g, b] >= 0:
                c.append((-run, b, 0.0, int(done[g, b])))
                continue
            v = np.where(np.isnan(x[g, b]), -np.inf, x[g, b])
            m = v.max()
            if not np.isfinite(m):
                continue
            lse = m + np.log(np.exp(v - m).sum())
            at = np.lexsort((np.arange(vocab), -v))[:n]
            c += [(-(v[t] - lse + run), b, -v[t], int(t)) for t in at if v[t] > -np.inf]
        c.sort()
        for k, (s, b, _, t) in enumerate(c[:n]):
            out[0][g, k], out[1][g, k], out[2][g, k] = -s, t, g * beams + b
        for u, w in zip(c[:n], c[1:n + 1]):
            if u[1] != w[1]:
                gap = min(gap, w[0] - u[0])
    return out, gap


def check(groups, beams, vocab, n, dtype, seed=0, make=None, done=None, stride=0, offset=0, scores=None):
    for attempt in range(50):
        rng = np.random.RandomState(1000 * seed + attempt)
        x = torch.from_numpy(rng.randn(groups, beams, vocab).astype(np.float32) * 3).to(dtype)
        if make:
            make(x)
        s = (-rng.rand(groups, beams) * 5).astype(np.float32) if scores is None else scores
        want, gap = select_ref(x.double().numpy(), s, n, done)
        if gap > NEAR:
            break
    assert gap > NEAR
    rows = groups * beams
    buf = torch.zeros((rows * (vocab + stride) + offset,), dtype=dtype, device=DEV)
    xd = buf[offset:].view(rows, vocab + stride)[:, :vocab]
    xd.copy_(x.view(rows, vocab))
    st = torch.from_numpy(s).to(DEV)
    dn = None if done is None else torch.from_numpy(done.astype(np.int32)).to(DEV)
    step = q.BeamStep(groups, beams, vocab, n, st, dn)
    ws = q.new_workspace(step.workspace_bytes())
    ws[16384:] = 0xFF
    for _ in range(2):
        score, token, parent = q.beam_select(xd, step, ws)
        torch.cuda.synchronize()
        assert np.array_equal(token.cpu().numpy(), want[1]) and np.array_equal(parent.cpu().numpy(), want[2])
        got = score.cpu().numpy()
        live = np.isfinite(want[0])
        assert np.array_equal(live, np.isfinite(got)) and np.all(got[~live] == -np.inf)
        assert np.all(np.abs(got[live] - want[0][live]) <= NEAR + 2.0 ** -24 * np.abs(want[0][live]))
    assert not bool(ws[:16384].any()) and q.device_status() == 0
    return xd, step, ws, (score, token, parent)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("groups,beams,vocab,n", [(1, 1, 1, 1), (1, 1, 7, 8), (2, 3, 100, 6), (1, 4, 2048, 8), (3, 2, 8193, 4),
                                                  (1, 16, 30011, 32), (5, 5, 16384, 5), (1, 2, 151936, 4), (20, 8, 9001, 16)])
def test_select(groups, beams, vocab, n, dtype):
    check(groups, beams, vocab, n, dtype)


@pytest.mark.parametrize("dtype,stride,offset", [(torch.float32, 1, 1), (torch.float32, 2, 3), (torch.float16, 3, 5),
                                                 (torch.bfloat16, 1, 7), (torch.float32, 0, 1)])
def test_unaligned_rows(dtype, stride, offset):
    check(2, 4, 10007, 8, dtype, stride=stride, offset=offset, seed=1)
    check(1, 2, 5, 4, dtype, stride=stride, offset=offset, seed=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_values(dtype):
    """More equal values than any list holds: the lowest tokens, row after row."""
    def flat(x):
        x.fill_(1.0)
    def steps(x):
        x.copy_(torch.floor(x * 0.5))
    same = np.zeros((2, 3), np.float32)
    # rows alike to the bit have equal scores: the lower row comes first, and the gap of 0 is meant
    x = torch.ones((6, 20000), dtype=dtype, device=DEV)
    step = q.BeamStep(2, 3, 20000, 8, torch.from_numpy(same).to(DEV))
    score, token, parent = q.beam_select(x, step, q.new_workspace(step.workspace_bytes()))
    assert token.tolist() == [list(range(8))] * 2 and parent.tolist() == [[0] * 8, [3] * 8]
    assert float((score + np.log(20000)).abs().max()) <= NEAR
    check(2, 3, 20000, 8, dtype, make=flat, scores=np.array([[0, -1, -2], [-3, -2.5, 0]], np.float32))
    check(2, 3, 30000, 32, dtype, make=steps, seed=3)


def test_masked_and_odd_values():
    def some(x):
        x[0, 0, :] = float("-inf")
        x[0, 1, 5:] = float("-inf")
        x[1, 0, ::2] = float("nan")
        x[1, 2, 77] = float("inf")
        x[1, 1, :] = float("nan")
    check(2, 3, 5000, 16, torch.float32, make=some)
    def none(x):
        x.fill_(float("-inf"))
    check(2, 2, 300, 4, torch.float16, make=none)
    def big(x):
        x *= 1e4
    check(1, 3, 3000, 6, torch.float32, make=lambda x: x.mul_(5.0), seed=4)
    def few(x):
        x[:, :, 3:] = float("-inf")
    check(3, 2, 40000, 8, torch.float32, make=few, seed=5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("beams,vocab,n", [(1, 128257, 1), (1, 128257, 32), (2, 63489, 4), (1, 8193, 32), (1, 2049, 32), (1, 300, 32)])
def test_thin_last_slices_and_many_best(beams, vocab, n, dtype):
    check(1, beams, vocab, n, dtype, seed=21)


@pytest.mark.parametrize("every", [50, 997])
@pytest.mark.parametrize("vocab,n", [(20000, 16), (128257, 32), (9000, 5)])
def test_grammars_that_leave_few(vocab, n, every):
    """Most logits -infinity: warps without a value, and rows with fewer continuations than wanted."""
    def make(x):
        keep = x[:, :, 3::every].clone()
        x.fill_(-float("inf"))
        x[:, :, 3::every] = keep
        x[-1, -1, 100:] = -float("inf")
    check(2, 2, vocab, n, torch.float32, seed=22, make=make)


def test_scores_of_beams_not_alive():
    s = np.array([[0.0, -np.inf, -np.inf], [-np.inf] * 3, [np.nan, -1.0, -2.0]], np.float32)
    check(3, 3, 4000, 6, torch.float32, scores=s)


def test_done_beams():
    done = np.array([[-1, 7, -1], [3, 3, 3], [-1, -1, 2 ** 31 - 2]])
    check(3, 3, 9000, 6, torch.float16, done=done, seed=6)
    s = np.array([[-50.0, -1.0, -2.0]] * 3, np.float32)
    check(3, 3, 9000, 6, torch.float16, done=done, scores=s, seed=7)


def test_more_groups_than_a_launch_takes():
    groups, vocab = 4100, 40
    x = torch.randn((groups, vocab), device=DEV)
    step = q.BeamStep(groups, 1, vocab, 2, torch.zeros((groups, 1), device=DEV))
    ws = q.new_workspace(step.workspace_bytes())
    score, token, parent = q.beam_select(x, step, ws)
    best = torch.topk(torch.log_softmax(x.double(), 1), 2)
    assert torch.equal(token, best.indices) and float((score - best.values).abs().max()) < NEAR
    assert parent.tolist() == [[i, i] for i in range(groups)] and not bool(ws[:16384].any())


def test_captured_and_on_another_stream():
    xd, step, ws, want = check(4, 4, 20011, 8, torch.float32, seed=8)
    side = torch.cuda.Stream()
    got = q.beam_select(xd, step, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.beam_select(xd, step, ws, *out)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# ------------------------------------------------------------------- pages

def fork_ref(caches, parents, lens, table, fresh, out, lens_out, page, block):
    """On the CPU, in place; caches: lists of arrays [pages][rows or blocks][...] with their rows per entry."""
    n_pages, cols = caches[0][0].shape[0], table.shape[1]
    src = [[a.copy() for a in c] for c in caches]
    for i, p in enumerate(parents):
        if p < 0 or p >= len(lens):
            continue
        n = min(max(lens[p], 0), cols * page)
        full, rows = n // page, n % page
        lens_out[i] = n
        out[i, :full] = table[p, :full]
        f = fresh[i] if 0 <= fresh[i] < n_pages else -1
        if full < cols:
            if f >= 0:
                out[i, full] = f
            elif rows:
                out[i, full] = table[p, full]
        if f < 0 or not rows or not 0 <= table[p, full] < n_pages or table[p, full] == f:
            continue
        for c, s in zip(caches, src):
            for a, b in zip(c, s):
                m = rows if a.shape[1] == page and a.ndim == 4 else -(-rows // block)
                a[f, :m] = b[table[p, full], :m]


def check_fork(n_in, n_out, layers, page, heads, d, dtype, block=16, columns=6, seed=0, order="rows", edit=None, status=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.RandomState(seed)
    eight = dtype in (torch.int8, torch.float8_e4m3fn)
    pages = n_in * columns + n_out + 3
    caches = []
    for _ in range(layers):
        shape = (pages, page, heads, d) if order == "rows" else (pages, heads, page, d)
        x = [torch.randint(0, 120, shape, generator=g, device=DEV).to(torch.uint8).view(dtype) if eight else
             torch.randn(shape, generator=g, device=DEV).to(dtype) for _ in range(2)]
        if order == "heads":
            x = [t.transpose(1, 2) for t in x]
        if eight:
            x += [torch.rand((pages, page // block, heads), generator=g, device=DEV) for _ in range(2)]
        caches.append(x)
    order_ = rng.permutation(pages)
    table = order_[:n_in * columns].reshape(n_in, columns).astype(np.int32)
    fresh = order_[n_in * columns:n_in * columns + n_out].astype(np.int32)
    lens = rng.randint(0, columns * page + 1, n_in).astype(np.int32)
    if n_in > 2:
        lens[0], lens[1], lens[2] = 0, columns * page, page
    parents = rng.randint(0, n_in, n_out).astype(np.int32)
    if edit:
        edit(parents, lens, table, fresh, pages)
    out, lens_out = np.full((n_out, columns), -9, np.int32), np.full((n_out,), -9, np.int32)
    host = [[t.contiguous().view(torch.uint8 if eight and t.dtype == dtype else t.dtype).cpu() for t in c] for c in caches]
    host = [[(t.view(torch.int16) if t.dtype in (torch.float16, torch.bfloat16) else t).numpy().copy() for t in c] for c in host]
    dev = [torch.from_numpy(t).to(DEV) for t in (parents, lens, table, fresh, out, lens_out)]
    fork_ref(host, parents, lens, table, fresh, out, lens_out, page, block)
    pool = q.PagePool([q.Kv8Cache(*c) if eight else q.KvCache(*c) for c in caches])
    for _ in range(2):
        q.fork_pages(pool, *dev)
        torch.cuda.synchronize()
        assert q.device_status() == status
        assert np.array_equal(dev[4].cpu().numpy(), out) and np.array_equal(dev[5].cpu().numpy(), lens_out)
        for c, h in zip(caches, host):
            for t, a in zip(c, h):
                t = t.contiguous()
                t = t.view(torch.uint8) if eight and t.dtype == dtype else t.view(torch.int16) if not eight else t
                assert np.array_equal(t.cpu().numpy(), a)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("n_in,n_out,layers,page,heads,d", [(1, 1, 1, 16, 1, 16), (4, 8, 3, 16, 2, 128), (8, 8, 28, 32, 2, 64),
                                                            (1, 5, 2, 64, 8, 96), (7, 3, 70, 16, 1, 32)])
def test_fork(n_in, n_out, layers, page, heads, d, dtype):
    check_fork(n_in, n_out, layers, page, heads, d, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_fork_other_orders(dtype):
    check_fork(3, 6, 2, 32, 4, 128, dtype, order="heads", block=32)
    check_fork(300, 500, 1, 16, 1, 16, dtype, seed=1, columns=2)


def test_fork_small_pages():
    for page in (1, 2, 8):
        check_fork(4, 6, 2, page, 2, 64, torch.float16, seed=2)


def test_fork_keeps_and_bad_numbers():
    def keep(parents, lens, table, fresh, pages):
        fresh[::2] = -1
        parents[1] = -1
        lens[3] = 37
        parents[3] = 3
        fresh[3] = table[3, 37 // 16]   # the child goes on in its parent's page
    check_fork(5, 7, 2, 16, 2, 64, torch.int8, edit=keep, seed=3)
    for k in range(5):
        def bad(parents, lens, table, fresh, pages):
            lens[:] = 21
            if k == 0:
                parents[2] = 5
            elif k == 1:
                parents[2] = -2
            elif k == 2:
                lens[parents[2]] = -4
            elif k == 3:
                fresh[2] = pages
            else:
                table[parents[2], 1] = pages
        check_fork(5, 7, 2, 16, 2, 64, torch.bfloat16, edit=bad, seed=4, status=7)


def test_fork_long_length_counts_as_the_end():
    def long(parents, lens, table, fresh, pages):
        lens[3] = 10 ** 6
        parents[:] = 3
    check_fork(5, 2, 2, 16, 2, 64, torch.float16, edit=long, seed=5, status=7)
