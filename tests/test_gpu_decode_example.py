"""examples/shared_prompt_decode.py against the same decoder whose rotary
positions, attention and logits rules are plain torch operations in 64 bits.

Both run the library's GEMVs, fed with the same tokens.  What differs is the
attention's 16-bit weights (2^-8 relative) and the rounding of q and k; each
may move a Q8_0 activation code of a later GEMV by one, 1/127 of its block's
largest value.  With two layers of three such GEMVs behind an attention, each
change at most 1/127 in the 2-norm, the logits differ by less than 6/127.
"""
import importlib.util
import math
import os

import pytest
import torch

import quantized_q4_weight_gb300 as q

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from quantized_q4_weight_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("shared_prompt_decode", os.path.join(ROOT, "examples", "shared_prompt_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_rope_kv(base):
    def f(plan, xq, xk, xv, pos, slots, cache, out=None, stream=None):
        d = xq.shape[-1]
        th = base ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        a = pos.double()[:, None] * th
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]

        def rot(x):
            x = x.double()
            u, w = x[..., :d // 2], x[..., d // 2:]
            return torch.cat([u * c - w * s, u * s + w * c], -1)
        flat = [t.view(-1, *t.shape[2:]) for t in (cache.k, cache.v)]
        flat[0][slots.long()] = rot(xk).to(cache.k.dtype)
        flat[1][slots.long()] = xv.to(cache.v.dtype)
        return rot(xq).to(cache.k.dtype)
    return f


def plain_attn(xq, batch, ws, out=None, lse=None, stream=None):
    c, b = batch.cache, batch.struct
    prefix, lens, own = batch.tables
    page = c.k.shape[1]
    x = xq.double().view(b.n_seqs, b.n_q, b.n_q_heads, -1)
    for i in range(b.n_seqs):
        n = int(lens[i])
        rows = [prefix.long()[torch.arange(b.prefix_len, device="cuda") // page] * page +
                torch.arange(b.prefix_len, device="cuda") % page if b.prefix_len else torch.zeros(0, dtype=torch.long, device="cuda"),
                own[i].long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page]
        k, v = (t.view(-1, *t.shape[2:])[torch.cat(rows)].double() for t in (c.k, c.v))
        grp = b.n_q_heads // k.shape[1]
        for t in range(b.n_q):
            seen = b.prefix_len + n - b.n_q + t + 1
            s = torch.einsum("hd,khd->hk", x[i, t], k[:seen].repeat_interleave(grp, 1)) / math.sqrt(k.shape[-1])
            o = torch.einsum("hk,khd->hd", torch.softmax(s, 1), v[:seen].repeat_interleave(grp, 1))
            out.view(b.n_seqs, b.n_q, b.n_q_heads, -1)[i, t] = o.float()
    return out


def plain_logits(history, lens, rules):
    """The rules in 64 bits on the last step's logits, from the histories as they were."""
    def f(x):
        y = x.double()
        rep, freq, pres = (t.double() for t in rules.tensors[2:5])
        for r in range(x.shape[0]):
            ids, c = torch.unique(history[r, :int(lens[r])], return_counts=True)
            v = y[r, ids]
            y[r, ids] = torch.where(v > 0, v / rep[r], v * rep[r]) - freq[r] * c - pres[r]
        return y
    return f


def test_decode_matches_the_plain_forms(ex, monkeypatch):
    args = dict(d_model=256, d_ff=512, heads=4, kv_heads=2, head_dim=64, vocab=2000, layers=2, pages=64, rope_base=1e4)
    samples, steps = 8, 20
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompt = torch.randint(0, 2000, (75,), generator=g, device="cuda")
    ours = ex.SharedPrompt(ex.Model(**args), prompt, samples, steps + 1)
    got, tokens, hist = [], [], []
    for _ in range(steps):
        before = ours.history.clone(), ours.history_len.clone()
        ours.step()
        got.append(ours.last_logits.clone())
        tokens.append(ours.tokens.clone())
        hist.append(before)
        # the token is the best one under the rules, by a margin that rounding does not reach
        y = plain_logits(*before, ours.rules)(ours.last_logits)
        top = y.topk(2, 1)
        clear = top.values[:, 0] - top.values[:, 1] > 1e-4 * top.values[:, 0].abs()
        assert torch.equal(ours.tokens[clear], top.indices[clear, 0])
    assert q.device_status() == 0
    assert len({tuple(int(t[i]) for t in tokens) for i in range(samples)}) > 1   # the rules set the samples apart

    monkeypatch.setattr(q, "rope_kv", plain_rope_kv(1e4))
    monkeypatch.setattr(q, "attn_prefix", plain_attn)
    ref = ex.SharedPrompt(ex.Model(**args), prompt, samples, steps + 1)
    for i in range(steps):
        ref.step()
        ref.tokens = tokens[i]
        err = (got[i] - ref.last_logits).norm(dim=1) / ref.last_logits.norm(dim=1)
        assert float(err.max()) < 6 / 127, (i, float(err.max()))


SMALL = dict(d_model=256, d_ff=512, heads=4, kv_heads=2, head_dim=64, vocab=2000, layers=1, rope_base=1e4)


@pytest.mark.parametrize("most", [1, 16, 17])
def test_a_step_past_the_samples_pages_is_refused(ex, most):
    """Before anything is launched: the page and history of a further token do not exist."""
    s = ex.SharedPrompt(ex.Model(pages=16, **SMALL), torch.arange(20, device="cuda"), 2, most)
    for _ in range(most):
        s.step()
    lens = s.lens.clone()
    with pytest.raises(RuntimeError, match="full"):
        s.step()
    assert torch.equal(s.lens, lens) and q.device_status() == 0


def test_prompts_and_pages_that_do_not_fit_are_refused(ex):
    m = ex.Model(pages=16, **SMALL)
    prompt = torch.arange(20, device="cuda")
    for args in ((prompt, 9, 4), (prompt, 0, 4), (prompt, 2, 0), (prompt[:0], 2, 4), (prompt, 8, 40)):
        with pytest.raises(ValueError):
            ex.SharedPrompt(m, *args)
    with pytest.raises(ValueError, match="one page"):
        ex.SharedPrompt(ex.Model(pages=64, page_size=4, **SMALL), prompt, 2, 4)
    s = ex.SharedPrompt(m, prompt[:1], 2, 4)          # a prompt of one token: nothing is shared
    s.step()
    assert q.device_status() == 0
