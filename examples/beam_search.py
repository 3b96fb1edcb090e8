"""Beam search over a paged 8-bit cache: the library's GEMVs with the operators of
such a step between them.

A decoder with norms on the heads of q and k and seeded synthetic Q4_0 weights.  A
step is, per layer: the QKV product (gemv_seq_ep), norms and rotary positions
(norm_rope_kv), the write of k and v as 8-bit codes (kv8_append), attention over
them under a sliding window with first tokens that stay visible (attn_kv8), the
output product with the residual (gemv_seq_ep) and the FFN (ffn_residual); then
the lm_head product (gemv_f32), the best continuations over all beams
(beam_select) and their sequences (fork_pages): a beam shares its parent's whole
pages and gets a page of its own for its next rows.  The norms of the hidden state,
the embedding and the choice of free pages are torch operations; nothing in a step
waits for the device.

    python examples/beam_search.py [--layers 4] [--prompt 300] [--tokens 64] [--beams 4]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_q4_weight_gb300 as q  # noqa: E402
import synth  # noqa: E402

DEV = "cuda"
T_MAX = 8  # tokens of a step: what the GEMVs take


class Model:
    """Weights, cache and buffers of a decoder; `heads` query heads share `kv_heads` cache heads."""

    def __init__(self, d_model=1536, d_ff=8960, heads=12, kv_heads=2, head_dim=128, vocab=151936, layers=4, seed=1,
                 pages=512, page_size=32, block_size=16, code=torch.int8, rope_base=1e6):
        self.d, self.ff, self.h, self.g, self.hd, self.vocab, self.page, self.pages = \
            d_model, d_ff, heads, kv_heads, head_dim, vocab, page_size, pages
        self.qkv = (heads + 2 * kv_heads) * head_dim
        rng = torch.Generator(device=DEV)
        rng.manual_seed(seed)

        def weights(n, N, K):
            return q.pack_q4_0(torch.from_numpy(synth.q4_0_weights(seed + n, N, K).reshape(-1)).to(DEV), N, K)

        def scale(n):
            return 1 + 0.1 * torch.randn(n, generator=rng, device=DEV)

        def cache():
            kv = [torch.zeros((pages, page_size, kv_heads, head_dim), dtype=code, device=DEV) for _ in range(2)]
            scales = [torch.zeros((pages, page_size // block_size, kv_heads), device=DEV) for _ in range(2)]
            return q.Kv8Cache(*kv, *scales)

        self.layers = [dict(
            norm1=scale(d_model), norm2=scale(d_model), heads=q.QkNorm(scale(head_dim), scale(head_dim)),
            wqkv=weights(10 * i, self.qkv, d_model), wo=weights(10 * i + 1, d_model, heads * head_dim),
            gate=weights(10 * i + 2, d_ff, d_model), up=weights(10 * i + 3, d_ff, d_model),
            down=weights(10 * i + 4, d_model, d_ff), cache=cache()) for i in range(layers)]
        self.pool = q.PagePool([L["cache"] for L in self.layers])
        self.norm = scale(d_model)
        self.head = weights(9999, vocab, d_model)
        self.embed = 0.5 * torch.randn((vocab, d_model), generator=rng, device=DEV)
        self.rope = q.rope_plan(head_dim, rope_base)
        # one workspace for every call: they run one after the other on one stream
        self.ws = q.new_workspace(max(q.ffn_workspace_bytes(d_model, d_ff, T_MAX),
                                      q.workspace_bytes(vocab, d_model, T_MAX), 32 << 20))
        self.buf = {n: torch.empty((T_MAX, w), device=DEV) for n, w in
                    (("qkv", self.qkv), ("attn", heads * head_dim), ("x", d_model), ("logits", vocab))}
        self.q = torch.empty((T_MAX, heads, head_dim), dtype=torch.float16, device=DEV)
        self.k = torch.empty((T_MAX, kv_heads, head_dim), device=DEV)

    @staticmethod
    def _norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    def _product(self, W, x, y, residual=None):
        T, N = y.shape
        q.gemv_seq_ep(q.seq_ep_items([(W, x, y, N, x.shape[1], None, residual)]), q.W_PACKED, T, self.ws, x_f32=True)

    def hidden(self, tokens, pos, batch):
        """The last norm's output for the step's tokens; `batch(layer)` is that layer's Kv8Batch, whose
        lengths count the tokens already."""
        T = tokens.numel()
        x, qkv, attn = (self.buf[n][:T] for n in ("x", "qkv", "attn"))
        x.copy_(self.embed[tokens])
        hq, hk = self.h * self.hd, (self.h + self.g) * self.hd
        for i, L in enumerate(self.layers):
            self._product(L["wqkv"], self._norm(x, L["norm1"]), qkv)
            xq, xk = qkv[:, :hq].unflatten(1, (self.h, self.hd)), qkv[:, hq:hk].unflatten(1, (self.g, self.hd))
            xv = qkv[:, hk:].unflatten(1, (self.g, self.hd))
            xq = q.norm_rope_kv(self.rope, L["heads"], xq, xk, None, pos, out=self.q[:T], k_out=self.k[:T])
            q.kv8_append(self.k[:T], xv, batch(i))
            q.attn_kv8(xq, batch(i), self.ws, out=attn.unflatten(1, (self.h, self.hd)))
            self._product(L["wo"], attn, x, residual=x)
            q.ffn_residual(L["gate"], L["up"], L["down"], q.W_PACKED, self._norm(x, L["norm2"]), x, self.d, self.ff, T,
                           self.ws, y=x)
        return self._norm(x, self.norm)

    def logits(self, h):
        T = h.shape[0]
        return q.gemv_f32(self.head, q.W_PACKED, h, self.vocab, self.d, T, self.ws, y=self.buf["logits"][:T])


class BeamSearch:
    """State of a search of `beams` beams behind a prompt (int64 tokens on the device) for at most `most` tokens."""

    def __init__(self, model: Model, prompt, beams: int, most: int, end: int = -1, window: int = 0, sinks: int = 0):
        m, page, n = model, model.page, prompt.numel()
        if not (1 <= beams <= T_MAX and most >= 1 and n >= 1):
            raise ValueError(f"1..{T_MAX} beams of at least one token each, after a prompt of at least one")
        self.m, self.beams, self.end, self.left, self.length = m, beams, end, most, n + most
        columns = -(-(n + most) // page) + 1
        # the beams' pages, those of their children before the parents let go, and the prompt's
        if 2 * beams * columns + columns > m.pages:
            raise ValueError("the model's cache has too few pages for the prompt and the beams")
        self.columns = torch.arange(columns, device=DEV)
        self.tables = [torch.zeros((beams, columns), dtype=torch.int32, device=DEV) for _ in range(2)]
        self.lens = [torch.zeros(beams, dtype=torch.int32, device=DEV) for _ in range(2)]
        self.at = 0
        self.batches = [[q.Kv8Batch(beams, 1, m.h, L["cache"], lens, table, n + most, window=window, sinks=sinks)
                         for L in m.layers] for lens, table in zip(self.lens, self.tables)]
        assert self.batches[0][0].workspace_bytes() <= m.ws.numel()
        self._prefill(prompt, columns, window, sinks)
        # one beam is alive at first: the others would be copies of it
        self.scores = torch.full((beams,), float("-inf"), device=DEV)
        self.scores[0] = 0.0
        self.done = torch.full((beams,), -1, dtype=torch.int32, device=DEV)
        self.select = q.BeamStep(1, beams, m.vocab, beams, self.scores, self.done)
        self.tokens = prompt[-1].expand(beams).clone()
        self.text = torch.full((beams, most), -1, dtype=torch.int64, device=DEV)
        self.steps = 0

    def _prefill(self, prompt, columns, window, sinks):
        """All but the prompt's last token, as one sequence in chunks of eight; then every beam begins from it."""
        m, n = self.m, prompt.numel() - 1
        table = torch.arange(columns, dtype=torch.int32, device=DEV).view(1, columns)
        length = torch.zeros(1, dtype=torch.int32, device=DEV)
        for a in range(0, n, T_MAX):
            T = min(T_MAX, n - a)
            length.fill_(a + T)
            batches = [q.Kv8Batch(1, T, m.h, L["cache"], length, table, self.length, window=window, sinks=sinks)
                       for L in m.layers]
            m.hidden(prompt[a:a + T], torch.arange(a, a + T, dtype=torch.int32, device=DEV), lambda i: batches[i])
        parents = torch.zeros(self.beams, dtype=torch.int32, device=DEV)
        fresh = columns + torch.arange(self.beams, dtype=torch.int32, device=DEV)
        q.fork_pages(m.pool, parents, length, table, fresh, self.tables[0], self.lens[0])

    def _free_pages(self):
        """Pages that no beam reads, one for each."""
        held = self.columns[None, :] <= (self.lens[self.at] // self.m.page)[:, None]
        used = torch.zeros(self.m.pages + 1, dtype=torch.int32, device=DEV)
        used[torch.where(held, self.tables[self.at], self.m.pages).flatten().long()] = 1
        return torch.argsort(used[:-1], stable=True)[:self.beams].to(torch.int32)

    def step(self):
        """One token more for every beam; returns the beams' scores."""
        if self.left == 0:
            raise RuntimeError("the beams' pages are full")
        self.left -= 1
        m, lens, table = self.m, self.lens[self.at], self.tables[self.at]
        pos = lens.clone()
        lens += 1
        self.last_logits = m.logits(m.hidden(self.tokens, pos, lambda i: self.batches[self.at][i]))
        scores, token, parent = q.beam_select(self.last_logits, self.select, m.ws)
        self.last_choice = scores, token, parent
        # places without a continuation stay as they are, with a score that keeps them out
        alive = parent[0] >= 0
        rows = torch.where(alive, parent[0], 0).long()
        q.fork_pages(m.pool, rows.to(torch.int32), lens, table, self._free_pages(), self.tables[1 - self.at], self.lens[1 - self.at])
        self.at = 1 - self.at
        self.scores.copy_(scores[0])
        self.tokens = torch.where(alive, token[0], self.tokens)
        self.done.copy_(torch.where(self.tokens == self.end, self.end, -1))
        self.text = self.text[rows]
        self.text[:, self.steps] = self.tokens
        self.steps += 1
        return self.scores


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--beams", type=int, default=4)
    a = ap.parse_args()
    m = Model(layers=a.layers)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    prompt = torch.randint(0, m.vocab, (a.prompt,), generator=g, device=DEV)
    s = BeamSearch(m, prompt, a.beams, a.tokens + 1, window=256, sinks=4)
    s.step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens):
        s.step()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert q.device_status() == 0
    print(f"{a.layers} layers, prompt {a.prompt}, {a.beams} beams: {1e3 * t / a.tokens:.3f} ms a step")
    for score, text in zip(s.scores.tolist(), s.text.tolist()):
        print(f"{score:9.3f}", text[:10])


if __name__ == "__main__":
    main()
