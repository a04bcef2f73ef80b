"""CPU tests of where the binding takes a call's workspace from when the caller passes none: the pool
of the stream the call runs on.  (A block of another stream's pool can be one that kernels queued on
that stream still use.)"""
import contextlib
import types

import pytest
import torch

import pagedattention_paged_kv_gb300 as pkv


class Buffer:
    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        pass


@pytest.fixture
def made(monkeypatch):
    """(bytes, stream that was current) of every torch.empty, with streams that are only names."""
    current, out = ["the current stream"], []

    @contextlib.contextmanager
    def on(stream):
        current.append(current[-1] if stream is None else stream)
        yield
        current.pop()

    def empty(nbytes, dtype=None, device=None):
        out.append((nbytes, current[-1]))
        return Buffer()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    return out


@pytest.mark.parametrize("stream", [None, types.SimpleNamespace(cuda_stream=7)])
def test_a_latent_call_s_fresh_workspace_belongs_to_its_stream(made, stream):
    at, have, keep = pkv._call_workspace(None, 0, stream, lambda a, b: a + b, 100, 28)
    assert (at, have) == (4096, 128) and isinstance(keep, Buffer)
    assert made == [(128, "the current stream" if stream is None else stream)]


class Tensor:
    """What a paged call reads of a tensor before it launches."""
    dtype, device = torch.bfloat16, "cuda:0"

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def __getitem__(self, i):
        return self

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("stream", [types.SimpleNamespace(cuda_stream=7)])
@pytest.mark.parametrize("call", ["decode", "decode_fp8", "varlen", "decode_kvwrite"])
def test_a_paged_call_s_fresh_workspace_belongs_to_its_stream(made, monkeypatch, call, stream):
    monkeypatch.setattr(pkv, "_require", lambda *a, **kw: None)
    monkeypatch.setattr(pkv, "workspace_size", lambda *a: 512)
    monkeypatch.setattr(Buffer, "numel", lambda self: 512, raising=False)
    monkeypatch.setattr(Buffer, "element_size", lambda self: 1, raising=False)
    launched = []
    monkeypatch.setattr(pkv, "lib", lambda: type("L", (), {"__getattr__": lambda s, n: lambda *a: launched.append(n) or 0})())
    q, cache, tables, lens = Tensor(4, 8, 128), Tensor(9, 16, 2, 128), Tensor(4, 3), Tensor(4)
    rows = Tensor(4, 2, 128)
    {"decode": lambda: pkv.paged_attention_decode(q, q, cache, cache, tables, lens, 0.1, stream=stream),
     "decode_fp8": lambda: pkv.paged_attention_decode_fp8(q, q, cache, cache, tables, lens, 0.1, 1.0, 1.0, stream=stream),
     "varlen": lambda: pkv.paged_attention_varlen(q, q, Tensor(5), cache, cache, tables, lens, 0.1, max_q_len=1,
                                                  stream=stream),
     "decode_kvwrite": lambda: pkv.paged_attention_decode_kvwrite(q, q, rows, rows, cache, cache, tables, lens, 0.1,
                                                                  stream=stream)}[call]()
    assert len(launched) == 1 and made == [(512, stream)]
