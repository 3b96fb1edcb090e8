"""Results that a call makes for itself when it runs on a stream of its own.

The current stream is kept busy, and then writes blocks of every size that the
call may ask for and that have already been given back: those blocks must not
become the call's results, which the other stream writes at once.
"""
import pytest
import torch

import quantized_q4_weight_gb300 as q
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_q4_weight_gb300 import _build
    _build.build()


def on_a_busy_device(call, n=16):
    """call(stream), with the current stream busy for about 0.1 s and behind that the
    last writes of blocks that are free again, of the sizes of the call's results."""
    want = [x.clone() for x in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for w in want:
        for size in (w.numel() * w.element_size(), 8 * w.numel() + 4 * w.numel()):
            blocks = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(n)]
            for b in blocks:
                b.fill_(0x55)
            del b, blocks
    got = call(s)
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def cache(pages=8, page=16, heads=2, d=64):
    return q.KvCache(*(torch.randn((pages, page, heads, d), device=DEV).half() for _ in range(2)))


def test_rotated_queries():
    plan, pos = q.rope_plan(64, 1e4), torch.arange(9, dtype=torch.int32, device=DEV)
    x = torch.randn((9, 4, 64), device=DEV)
    on_a_busy_device(lambda s: [q.rope_kv(plan, x, None, None, pos, stream=s)])
    kv, slots = cache(), torch.arange(9, dtype=torch.int32, device=DEV)
    on_a_busy_device(lambda s: [q.rope_kv(plan, x, x[:, :2].contiguous(), x[:, 2:].contiguous(), pos, slots, kv, stream=s)])


def test_attention():
    kv = cache()
    pages = torch.arange(8, dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 20], dtype=torch.int32, device=DEV)
    b = q.AttnBatch(2, 1, 4, kv, 60, pages[:4].clone(), lens, pages[4:].view(2, 2).clone(), 32)
    ws, x = q.new_workspace(b.workspace_bytes()), torch.randn((2, 4, 64), device=DEV).half()
    on_a_busy_device(lambda s: [q.attn_prefix(x, b, ws, stream=s)])


def test_logits():
    rules, x = q.LogitsRules(5, 3000), torch.randn((5, 3000), device=DEV)
    ws = q.new_workspace(rules.workspace_bytes())
    idx, val = torch.empty(5, dtype=torch.int64, device=DEV), torch.empty(5, device=DEV)
    on_a_busy_device(lambda s: list(q.logits_rules(x, rules, ws, stream=s)))
    on_a_busy_device(lambda s: list(q.logits_rules(x, rules, ws, idx=idx.clone() if s is None else idx, stream=s)))
    on_a_busy_device(lambda s: list(q.logits_rules(x, rules, ws, val=val.clone() if s is None else val, stream=s)))


def test_results_on_the_default_stream_by_name():
    x, plan, pos = torch.randn((9, 4, 64), device=DEV), q.rope_plan(64, 1e4), torch.arange(9, dtype=torch.int32, device=DEV)
    want = q.rope_kv(plan, x, None, None, pos)
    torch.cuda.synchronize()
    before = torch.cuda.current_stream()
    got = q.rope_kv(plan, x, None, None, pos, stream=torch.cuda.default_stream())
    side = torch.cuda.Stream()
    again = q.rope_kv(plan, x, None, None, pos, stream=side)
    assert torch.cuda.current_stream() == before      # the call leaves the current stream as it was
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def test_products_on_a_stream_of_their_own():
    N, K, T = 512, 256, 3
    w = q.pack_q4_0(torch.from_numpy(synth.q4_0_weights(1, N, K).reshape(-1)).to(DEV), N, K)
    x, ws = torch.randn((T, K), device=DEV), q.new_workspace(q.workspace_bytes(N, K, T))
    xq = q.quantize_q8_0(x, T, K)
    for call in (lambda s: [q.gemv_f32(w, q.W_PACKED, x, N, K, T, ws, stream=s)],
                 lambda s: [q.gemv(w, q.W_PACKED, xq, N, K, T, ws, stream=s)],
                 lambda s: [q.gemv_argmax_f32(w, q.W_PACKED, x, N, K, T, ws, stream=s)],
                 lambda s: list(q.gemv_top2_f32(w, q.W_PACKED, x, N, K, T, ws, stream=s)),
                 lambda s: [q.unpack_q4_0(w, N, K, stream=s)],
                 lambda s: list(q.quantize_vec_i8(x, T, K, stream=s))):
        on_a_busy_device(call)
