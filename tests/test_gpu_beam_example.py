"""examples/beam_search.py against the same search whose norms, rotation, cache
write, attention and reordering are plain torch operations in 64 bits.

Both run the library's GEMVs, fed with the same tokens and parents.  What differs
is the attention's 16-bit weights (2^-11 relative) and roundings of q and k; each may
move a Q8_0 activation code of a later GEMV by one, 1/127 of its block's largest
value, and so may a code of the cache.  With two layers of three such GEMVs behind
an attention, each change at most 1/127 in the 2-norm, the logits differ by less
than 6/127 (codes of the cache that move are few: those whose value lies within an fp32
rounding of a border).
"""
import importlib.util
import math
import os

import pytest
import torch

import quantized_q4_weight_gb300 as q

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMALL = dict(d_model=256, d_ff=512, heads=4, kv_heads=2, head_dim=64, vocab=2000, layers=2, pages=96, rope_base=1e4)


@pytest.fixture(scope="module")
def ex():
    from quantized_q4_weight_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_norm_rope(base):
    def f(plan, norm, xq, xk, xv=None, pos=None, slots=None, cache=None, out=None, k_out=None, stream=None):
        d = xq.shape[-1]
        a = pos.double()[:, None] * base ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]

        def turned(x, w):
            x = x.double()
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + norm.struct.eps) * w.double()
            u, v = x[..., :d // 2], x[..., d // 2:]
            return torch.cat([u * c - v * s, u * s + v * c], -1)
        k_out.copy_(turned(xk, norm.weights[1]))
        return out.copy_(turned(xq, norm.weights[0]))
    return f


def plain_append(xk, xv, batch, first=None, max_new=None, stream=None):
    lens, pages = (t.tolist() for t in batch.tables)
    nq, page, block = batch.n_q, batch.cache.struct.page_size, batch.cache.struct.block_size
    for x, codes, scale in ((xk, batch.cache.k, batch.cache.k_scale), (xv, batch.cache.v, batch.cache.v_scale)):
        for b, n in enumerate(lens):
            for j in range(n - nq, n):
                p, r, u = pages[b][j // page], j % page, j % page // block
                part = x[b * nq + j - n + nq].float()
                was = scale[p, u] if r % block else torch.zeros_like(scale[p, u])
                now = torch.maximum(was, part.abs().amax(-1) / torch.full_like(was, 127.0))
                old = codes[p, r - r % block:r].float()
                codes[p, r - r % block:r] = torch.where((now > was)[:, None], torch.round(old * (was / now)[:, None]), old).to(torch.int8)
                codes[p, r] = torch.round(part / now[:, None]).to(torch.int8)
                scale[p, u] = now


def plain_attn(xq, batch, ws, out=None, lse=None, stream=None):
    c, s = batch.cache, batch.struct
    lens, pages = batch.tables
    page, block = s_page(c), c.struct.block_size
    x = xq.double().view(s.n_seqs, s.n_q, s.n_q_heads, -1)
    grp = s.n_q_heads // c.k.shape[2]
    for b in range(s.n_seqs):
        n = int(lens[b])
        j = torch.arange(n, device="cuda")
        p, r = pages[b].long()[j // page], j % page
        k, v = (t[p, r].double() * sc[p, r // block].double()[..., None]
                for t, sc in ((c.k, c.k_scale), (c.v, c.v_scale)))
        for t in range(s.n_q):
            at = n - s.n_q + t
            sees = (j <= at) & ((j > at - s.window) | (j < s.sinks)) if s.window else j <= at
            w = torch.einsum("hd,khd->hk", x[b, t], k[sees].repeat_interleave(grp, 1)) / math.sqrt(k.shape[-1])
            o = torch.einsum("hk,khd->hd", torch.softmax(w, 1), v[sees].repeat_interleave(grp, 1))
            out.view(s.n_seqs, s.n_q, s.n_q_heads, -1)[b, t] = o.float()
    return out


def s_page(c):
    return c.struct.page_size


def plain_fork(pool, parents, lens, pages, fresh, pages_out, lens_out, stream=None):
    page, block = pool.caches[0].struct.page_size, pool.caches[0].struct.block_size
    for i, p in enumerate(parents.tolist()):
        n = int(lens[p])
        full, rows = n // page, n % page
        pages_out[i, :full] = pages[p, :full]
        pages_out[i, full] = fresh[i]
        lens_out[i] = n
        a, b, m = int(pages[p, full]), int(fresh[i]), -(-rows // block)
        for c in pool.caches:
            for t in (c.k, c.v):
                t[b, :rows] = t[a, :rows]
            for t in (c.k_scale, c.v_scale):
                t[b, :m] = t[a, :m]


@pytest.mark.parametrize("window,sinks,end", [(0, 0, -1), (24, 3, -1), (0, 0, 7)])
def test_search_matches_the_plain_forms(ex, monkeypatch, window, sinks, end):
    beams, steps = 4, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompt = torch.randint(0, 2000, (45,), generator=g, device="cuda")
    ours = ex.BeamSearch(ex.Model(**SMALL), prompt, beams, steps, end=end, window=window, sinks=sinks)
    got = []
    for _ in range(steps):
        run, done = ours.scores.clone(), ours.done.clone()
        ours.step()
        got.append((ours.last_logits.clone(), ours.last_choice))
        # the choice against a sort in 64 bits, where its neighbours are further apart than the sums' rounding
        x = torch.log_softmax(ours.last_logits.double(), 1) + run.double()[:, None]
        for r in range(beams):
            if int(done[r]) >= 0:
                x[r] = float("-inf")
                x[r, int(done[r])] = run[r].double()
        best = torch.sort(x.flatten(), descending=True, stable=True)
        gaps = best.values[:beams] - best.values[1:beams + 1]
        if float(gaps.min()) > 1e-5:
            alive = best.values[:beams] > float("-inf")
            want = torch.where(alive, best.indices[:beams], -1)
            score, token, parent = ours.last_choice
            assert torch.equal(token[0], torch.where(alive, want % 2000, -1))
            assert torch.equal(parent[0].long(), torch.where(alive, want // 2000, -1))
            assert float((score[0].double() - best.values[:beams])[alive].abs().max()) < 1e-4
    assert q.device_status() == 0
    assert len({tuple(t) for t in ours.text.tolist()}) == beams          # the beams are different texts

    monkeypatch.setattr(q, "norm_rope_kv", plain_norm_rope(1e4))
    monkeypatch.setattr(q, "kv8_append", plain_append)
    monkeypatch.setattr(q, "attn_kv8", plain_attn)
    monkeypatch.setattr(q, "fork_pages", plain_fork)
    it = iter(got)
    chosen = {}

    def replay(x, step, ws, *a, **k):
        logits, choice = next(it)
        chosen["err"] = (logits - x).norm(dim=1) / x.norm(dim=1)
        return choice
    monkeypatch.setattr(q, "beam_select", replay)
    ref = ex.BeamSearch(ex.Model(**SMALL), prompt, beams, steps, end=end, window=window, sinks=sinks)
    for i in range(steps):
        ref.step()
        live = got[i][1][0][0] > float("-inf")
        assert float(chosen["err"][live].max()) < 6 / 127, (i, chosen["err"])
    assert torch.equal(ref.text, ours.text)


def test_limits(ex):
    m = ex.Model(**SMALL)
    prompt = torch.arange(20, device="cuda")
    for args in ((prompt, 9, 4), (prompt, 0, 4), (prompt, 2, 0), (prompt[:0], 2, 4), (prompt, 8, 400)):
        with pytest.raises(ValueError):
            ex.BeamSearch(m, *args)
    s = ex.BeamSearch(m, prompt[:1], 1, 2)          # a prompt of one token, one beam
    s.step()
    s.step()
    with pytest.raises(RuntimeError, match="full"):
        s.step()
    assert q.device_status() == 0
