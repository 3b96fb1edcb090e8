"""A call with stream= takes the memory of the results it makes with that stream
current.  The library and the device are stood in for, so this runs without a GPU."""
import contextlib

import pytest
import torch

import quantized_q4_weight_gb300 as q

W = torch.zeros(64, dtype=torch.uint8)
X = torch.zeros((2, 32), dtype=torch.float32)
TOK = torch.zeros(2, dtype=torch.int64)
SHAPE = (64, 64, 2)   # N, K, T
CALLS = {
    "pack_q4_0": lambda s: q.pack_q4_0(W, 64, 64, stream=s),
    "unpack_q4_0": lambda s: q.unpack_q4_0(W, 64, 64, stream=s),
    "quantize_q8_0": lambda s: q.quantize_q8_0(X, 2, 32, stream=s),
    "gemv": lambda s: q.gemv(W, 0, W, *SHAPE, W, stream=s),
    "gemv_f32": lambda s: q.gemv_f32(W, 0, X, *SHAPE, W, stream=s),
    "gemv_argmax": lambda s: q.gemv_argmax(W, 0, W, *SHAPE, W, stream=s),
    "gemv_argmax_f32": lambda s: q.gemv_argmax_f32(W, 0, X, *SHAPE, W, stream=s),
    "gemv_top2": lambda s: q.gemv_top2(W, 0, W, *SHAPE, W, stream=s),
    "gemv_top2_f32": lambda s: q.gemv_top2_f32(W, 0, X, *SHAPE, W, stream=s),
    "verify_f32": lambda s: q.verify_f32(W, 0, X, TOK, *SHAPE, W, stream=s),
    "verify_commit": lambda s: q.verify_commit(TOK, TOK, stream=s),
    "ffn": lambda s: q.ffn(W, W, W, 0, X, 64, 64, 2, W, stream=s),
    "ffn_residual": lambda s: q.ffn_residual(W, W, W, 0, X, X, 64, 64, 2, W, stream=s),
    "silu_mul_q8": lambda s: q.silu_mul_q8(X, X, 2, 32, stream=s),
    "pack_q8_0": lambda s: q.pack_q8_0(W, 64, 64, stream=s),
    "unpack_q8_0": lambda s: q.unpack_q8_0(W, 64, 64, stream=s),
    "requant_f32_q4_0": lambda s: q.requant_f32_q4_0(X, 64, 64, stream=s),
    "requant_q8_0_q4_0": lambda s: q.requant_q8_0_q4_0(W, 64, 64, stream=s),
    "gemv_q8_0": lambda s: q.gemv_q8_0(W, W, *SHAPE, W, stream=s),
    "block_isums": lambda s: q.block_isums(W, 0, W, *SHAPE, stream=s),
    "block_isums_tc": lambda s: q.block_isums_tc(W, 0, W, *SHAPE, True, stream=s),
    "pack_gs64": lambda s: q.pack_gs64(W, X, 64, 64, stream=s),
    "unpack_gs64": lambda s: q.unpack_gs64(W, 64, 64, stream=s),
    "quantize_vec_i8": lambda s: q.quantize_vec_i8(X, 2, 32, stream=s),
    "gemv_gs64": lambda s: q.gemv_gs64(W, W, X, *SHAPE, W, stream=s),
    "gemv_gs64_f32": lambda s: q.gemv_gs64_f32(W, X, *SHAPE, W, stream=s),
}


class FakeStream:
    cuda_stream = 4096


class FakeLibrary:
    def __getattr__(self, name):
        return lambda *a: 0 if not name.endswith("bytes") else 64


@pytest.mark.parametrize("name", sorted(CALLS))
def test_results_are_made_on_the_calls_stream(name, monkeypatch):
    current, made = [], []
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def recorded(*a, **kw):
        made.append(current[-1] if current else None)
        return empty(*a, **kw)

    monkeypatch.setattr(q, "lib", FakeLibrary)
    monkeypatch.setattr(q, "_ptr", lambda t: None)
    monkeypatch.setattr(q, "_stream", lambda s=None: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    s = FakeStream()
    CALLS[name](s)
    assert made and all(m is s for m in made)
    made.clear()
    CALLS[name](None)
    assert made and all(m is None for m in made)
