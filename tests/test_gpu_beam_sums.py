"""Beam selection's sums over the vocabulary where a logit's size, or a mask's, could
cost them: masks of a type's lowest value, offsets that all logits of a row
share, maxima that come late.

A score is s = (x - M) - log(sum exp(x - M)) + run, here in 64 bits.  The kernel's
sum is off, relatively, by a weighted mean of its terms' errors, 2^-22 of ex2 and, of the exponent,
|x - m| (2^-23 + 2^-26) for the difference, the product and log2 e, m the reference, and by
2^-24 for each addition, of which some hundreds follow one another: below 1e-5 for
every offset, as the exponents of the terms that count are below 64.
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


def scores_of(x, run):
    """x float64 [beams][vocab] -> scores in 64 bits, -infinity where nothing continues."""
    v = np.where(np.isnan(x), -np.inf, x)
    m = v.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = v - m
        return d - np.log(np.exp(d).sum(1, keepdims=True)) + run[:, None]


def best_of(x, run, n):
    """The n best of one search and the smallest gap between neighbours of different rows."""
    s = scores_of(x, run)
    beams, vocab = x.shape
    top = [(b, t) for b in range(beams) for t in np.lexsort((np.arange(vocab), -x[b]))[:n + 1] if s[b, t] > -np.inf]
    top.sort(key=lambda c: (-s[c], c[0], -x[c], c[1]))
    gap = min([s[u] - s[w] for u, w in zip(top[:n], top[1:n + 1]) if u[0] != w[0]], default=np.inf)
    return [(s[c], c[1], c[0]) for c in top[:n]], gap


def check(beams, vocab, n, dtype, make, seed=0):
    for attempt in range(50):
        rng = np.random.RandomState(100 * seed + attempt)
        x = torch.from_numpy(rng.randn(beams, vocab).astype(np.float32) * 3).to(dtype)
        make(x)
        run = (-rng.rand(beams) * 5).astype(np.float32)
        want, gap = best_of(x.double().numpy(), run.astype(np.float64), n)
        if gap > 2 * NEAR:
            break
    assert gap > 2 * NEAR
    step = q.BeamStep(1, beams, vocab, n, torch.from_numpy(run).to(DEV).view(1, beams))
    score, token, parent = (t[0].tolist() for t in q.beam_select(x.to(DEV), step, q.new_workspace(step.workspace_bytes())))
    assert q.device_status() == 0
    assert token == [c[1] for c in want] + [-1] * (n - len(want))
    assert parent == [c[2] for c in want] + [-1] * (n - len(want))
    worst = max(abs(a - c[0]) - 2.0 ** -24 * abs(c[0]) for a, c in zip(score, want))
    assert worst <= NEAR, worst


def lowest(dtype):
    return torch.finfo(dtype).min


def keep(x, at):
    """All but `at` of every row at the type's lowest value."""
    held = x[:, at].clone()
    x.fill_(lowest(x.dtype))
    x[:, at] = held


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [300, 20011, 128257])
def test_masks_of_the_lowest_value(vocab, dtype):
    v = vocab
    for k, at in enumerate((slice(0, 3), slice(v - 100, v), slice(v // 2, v // 2 + v // 8), slice(5, v, 997), slice(1, v, 50),
                            slice(0, v - v // 3))):
        check(3, vocab, 4, dtype, lambda x: keep(x, at), seed=k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [77, 30011])
def test_rows_of_nothing_but_the_lowest_value(vocab, dtype):
    """Such a row's tokens are alike, at -log of their number each, and lose to what other rows hold."""
    def one(x):
        x[1] = lowest(x.dtype)
    check(3, vocab, 8, dtype, one, seed=11)

    def some(x):  # half of the row's tokens masked by -infinity beside
        keep(x, slice(7, None, 20))
        x[:, ::2] = -float("inf")
        x[0] = lowest(x.dtype)
        x[0, 1::2] = -float("inf")
    check(2, vocab, 6, dtype, some, seed=12)


@pytest.mark.parametrize("dtype,size", [(torch.float32, 3e38), (torch.float32, -3e38), (torch.bfloat16, 3e38), (torch.float32, 1e30)])
def test_logits_of_any_finite_size(dtype, size):
    """One value far above all: its probability is 1."""
    def far(x):
        x[:, 1234] = size
        x[0] = torch.where(torch.arange(x.shape[1]) == 1234, torch.tensor(size, dtype=dtype), torch.tensor(-3e38, dtype=dtype))
    check(2, 9000, 1, dtype, far, seed=13)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("offset", [13.0, 60.0, 1e3, -1e3, 3e4, 1e5, -1e6, 1e8])
def test_an_offset_of_all_logits(offset, dtype):
    if dtype == torch.float16 and abs(offset) > 6e4:
        offset = offset / abs(offset) * 6e4

    def shift(x):
        x.copy_((x.float() + offset).to(x.dtype))
        # rows of different offsets: what a row's own costs it does not cancel
        x[1] = (x[1].float() + 0.37 * offset).to(x.dtype) if dtype != torch.float16 else x[1] * 0.5
    check(3, 9001, 8, dtype, shift, seed=14)


def test_large_logits():
    """Spread over tens of thousands: the largest's probability is 1."""
    check(3, 3000, 6, torch.float32, lambda x: x.mul_(1e4), seed=15)
    check(2, 50021, 4, torch.bfloat16, lambda x: x.mul_(300.0), seed=16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_maxima_that_come_late(dtype):
    """A row's largest value in its last batch, up to 39 above all before it.

    The reference follows within 8, so a term's exponent, below 11.55, is off by 2^-21 at most (3.3e-7 of the term),
    log2 e by 2^-26 of it (1.1e-7), ex2 by 2^-22, and ten or so additions, in order of size, by 2^-24 each: 1.3e-6."""
    rows, vocab = 1024, 20011
    rng = np.random.RandomState(17)
    x = rng.uniform(-1, 1, (rows, vocab)).astype(np.float32)
    at = rng.randint(vocab - 500, vocab, rows)
    x[np.arange(rows), at] = rng.uniform(5, 39, rows)
    x = torch.from_numpy(x).to(dtype)
    step = q.BeamStep(rows, 1, vocab, 1, torch.zeros((rows, 1), device=DEV))
    score, token, _ = q.beam_select(x.to(DEV), step, q.new_workspace(step.workspace_bytes()))
    best = torch.log_softmax(x.double(), 1)[torch.arange(rows), torch.from_numpy(at)]
    assert token[:, 0].tolist() == at.tolist() and q.device_status() == 0
    off = (score[:, 0].cpu().double() - best).abs() - 2.0 ** -24 * best.abs()
    assert float(off.max()) <= 1.3e-6, float(off.max())
