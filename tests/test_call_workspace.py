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
