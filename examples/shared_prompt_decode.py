"""Eight samples of one prompt, decoded together: the library's GEMVs with the
operators between them.

A Qwen2.5-shaped decoder with seeded synthetic Q4_0 weights.  The prompt goes
through the model eight tokens at a time, into cache pages that all samples
then share; each sample has pages of its own for what it writes.  A step is,
per layer: the QKV product with its bias (gemv_seq_ep), rotary positions and
the cache write (rope_kv), attention over the shared prompt and the own suffix
(attn_prefix), the output product with the residual (gemv_seq_ep) and the FFN
with the residual (ffn_residual); then the lm_head product (gemv_f32) and the
rules on its logits with the argmax (logits_rules), whose token joins the
sample's history.  The norms are torch operations.

    python examples/shared_prompt_decode.py [--layers 4] [--prompt 512] [--tokens 64]
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
                 pages=512, page_size=16, rope_base=1e6):
        self.d, self.ff, self.h, self.g, self.hd, self.vocab, self.page = \
            d_model, d_ff, heads, kv_heads, head_dim, vocab, page_size
        self.qkv = (heads + 2 * kv_heads) * head_dim
        rng = torch.Generator(device=DEV)
        rng.manual_seed(seed)

        def weights(n, N, K):
            w = torch.from_numpy(synth.q4_0_weights(seed + n, N, K).reshape(-1)).to(DEV)
            return q.pack_q4_0(w, N, K)

        def vector(n):
            return 0.1 * torch.randn(n, generator=rng, device=DEV)

        self.layers = []
        for i in range(layers):
            kv = [torch.zeros((pages, page_size, kv_heads, head_dim), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            self.layers.append(dict(
                norm1=1 + vector(d_model), norm2=1 + vector(d_model), bias=vector(self.qkv),
                wqkv=weights(10 * i, self.qkv, d_model), wo=weights(10 * i + 1, d_model, heads * head_dim),
                gate=weights(10 * i + 2, d_ff, d_model), up=weights(10 * i + 3, d_ff, d_model),
                down=weights(10 * i + 4, d_model, d_ff), cache=q.KvCache(*kv)))
        self.norm = 1 + vector(d_model)
        self.head = weights(9999, vocab, d_model)
        self.embed = 0.5 * torch.randn((vocab, d_model), generator=rng, device=DEV)
        self.rope = q.rope_plan(head_dim, rope_base)
        # one workspace for every call: they run one after the other on one stream
        self.ws = q.new_workspace(max(q.ffn_workspace_bytes(d_model, d_ff, T_MAX),
                                      q.workspace_bytes(vocab, d_model, T_MAX), 32 << 20))
        self.buf = {n: torch.empty((T_MAX, w), device=DEV) for n, w in
                    (("qkv", self.qkv), ("attn", heads * head_dim), ("x", d_model), ("logits", vocab))}

    @staticmethod
    def _norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

    def _product(self, W, x, y, bias=None, residual=None):
        T, N = y.shape
        items = q.seq_ep_items([(W, x, y, N, x.shape[1], bias, residual)])
        q.gemv_seq_ep(items, q.W_PACKED, T, self.ws, x_f32=True)

    def hidden(self, tokens, pos, slots, batch):
        """The last norm's output for the step's tokens; `batch(layer)` is that layer's AttnBatch."""
        T = tokens.numel()
        x, qkv, attn = (self.buf[n][:T] for n in ("x", "qkv", "attn"))
        x.copy_(self.embed[tokens])
        hq, hk = self.h * self.hd, (self.h + self.g) * self.hd
        for i, L in enumerate(self.layers):
            self._product(L["wqkv"], self._norm(x, L["norm1"]), qkv, bias=L["bias"])
            xq = q.rope_kv(self.rope, qkv[:, :hq].unflatten(1, (self.h, self.hd)),
                           qkv[:, hq:hk].unflatten(1, (self.g, self.hd)), qkv[:, hk:].unflatten(1, (self.g, self.hd)),
                           pos, slots, L["cache"])
            q.attn_prefix(xq, batch(i), self.ws, out=attn.unflatten(1, (self.h, self.hd)))
            self._product(L["wo"], attn, x, residual=x)
            q.ffn_residual(L["gate"], L["up"], L["down"], q.W_PACKED, self._norm(x, L["norm2"]), x, self.d, self.ff, T,
                           self.ws, y=x)
        return self._norm(x, self.norm)

    def logits(self, h):
        T = h.shape[0]
        return q.gemv_f32(self.head, q.W_PACKED, h, self.vocab, self.d, T, self.ws, y=self.buf["logits"][:T])


class SharedPrompt:
    """Decoding state of `samples` samples of one prompt (int64 tokens on the device)."""

    def __init__(self, model: Model, prompt, samples: int, most: int, rules=True):
        m, page = model, model.page
        # the prompt's last token is the first step's input, so it opens every sample's own suffix
        self.m, self.shared = model, prompt.numel() - 1
        pre, own = -(-self.shared // page), -(-most // page)
        if not (1 <= samples <= T_MAX and most >= 1 and prompt.numel() >= 1):
            raise ValueError(f"1..{T_MAX} samples of at least one token each, after a prompt of at least one")
        if page % T_MAX:
            raise ValueError(f"pages of {page} rows: a chunk of {T_MAX} tokens must lie in one page")
        if pre + samples * own > m.layers[0]["cache"].k.shape[0]:
            raise ValueError("the model's cache has too few pages for the prompt and the samples")
        self.left = most  # steps that the samples' pages and histories have room for
        self.prefix_pages = torch.arange(pre, dtype=torch.int32, device=DEV)
        self.own_pages = pre + torch.arange(samples * own, dtype=torch.int32, device=DEV).view(samples, own)
        self.lens = torch.zeros(samples, dtype=torch.int32, device=DEV)
        self._prefill(prompt)
        self.batches = [q.AttnBatch(samples, 1, m.h, L["cache"], self.shared, self.prefix_pages, self.lens, self.own_pages, most)
                        for L in m.layers]
        assert self.batches[0].workspace_bytes() <= m.ws.numel()
        # the rules: histories that grow with the samples, penalties that differ between them
        n = prompt.numel()
        self.history = torch.zeros((samples, n + most), dtype=torch.int64, device=DEV)
        self.history[:, :n] = prompt
        self.history_len = torch.full((samples,), n, dtype=torch.int32, device=DEV)
        spread = torch.linspace(0, 1, samples, device=DEV)
        self.rules = q.LogitsRules(samples, m.vocab, history=self.history, history_len=self.history_len,
                                   repetition=1.05 + 0.3 * spread, frequency=0.2 * spread,
                                   presence=spread.clone()) if rules else q.LogitsRules(samples, m.vocab)
        self.rows = torch.arange(samples, device=DEV)
        self.tokens = prompt[-1].expand(samples).clone()

    def _prefill(self, prompt):
        """The prompt in chunks of eight tokens: a chunk is the suffix, with its
        own page table, of the part of the prompt that is in the cache."""
        m, page = self.m, self.m.page
        for a in range(0, self.shared, T_MAX):
            T = min(T_MAX, self.shared - a)
            pos = torch.arange(a, a + T, dtype=torch.int32, device=DEV)
            # chunks are aligned to eight rows, so one lies in one page: the suffix's page
            # table names it, and the prefix ends inside it or before
            length = torch.tensor([a % page + T], dtype=torch.int32, device=DEV)
            first = a - a % page
            table = self.prefix_pages[first // page:first // page + 1].view(1, 1)
            batches = [q.AttnBatch(1, T, m.h, L["cache"], first, self.prefix_pages, length, table, page) for L in m.layers]
            m.hidden(prompt[a:a + T], pos, pos, lambda i: batches[i])

    def step(self):
        """One token for every sample; returns them (int64 [samples])."""
        if self.left == 0:
            raise RuntimeError("the samples' pages are full")
        self.left -= 1
        m, page = self.m, self.m.page
        pos = self.shared + self.lens
        own = self.own_pages[self.rows, (self.lens // page).long()]
        slots = own * page + self.lens % page
        self.lens += 1
        h = m.hidden(self.tokens, pos, slots, lambda i: self.batches[i])
        self.last_logits = m.logits(h)
        self.tokens, _ = q.logits_rules(self.last_logits, self.rules, m.ws)
        self.history[self.rows, self.history_len.long()] = self.tokens
        self.history_len += 1
        return self.tokens


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    m = Model(layers=a.layers)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    prompt = torch.randint(0, m.vocab, (a.prompt,), generator=g, device=DEV)
    s = SharedPrompt(m, prompt, samples=8, most=a.tokens + 1)
    s.step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    out = [s.step().clone() for _ in range(a.tokens)]
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert q.device_status() == 0
    print(f"{a.layers} layers, prompt {a.prompt}, 8 samples: {8 * len(out) / t:.0f} tokens/s, {1e3 * t / len(out):.3f} ms a step")
    for i in range(8):
        print(i, [int(x[i]) for x in out[:8]])


if __name__ == "__main__":
    main()
