"""The Python binding with fakes in CUDA's place (CPU): mostly the key/value cache."""
import contextlib

import pytest
import torch

from gated_rank_subspace_gsi_gb300 import lib


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.fixture
def cuda(monkeypatch):
    """What the binding sees of CUDA: streams, the allocator, the library."""
    seen = {"current": 11, "allocated": [], "launched": []}

    @contextlib.contextmanager
    def stream(s):
        was, seen["current"] = seen["current"], s.cuda_stream
        yield
        seen["current"] = was

    def empty(shape, dtype=None, device=None):
        seen["allocated"].append(seen["current"])
        return torch.zeros(shape, dtype=dtype)

    def attention(kv, q, row_start, length, max_rows, scale, out, lse=None, accumulate=False, stream=None):
        seen["launched"].append(lib._raw(stream))

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(lib, "_current_stream", lambda: seen["current"])
    monkeypatch.setattr(lib, "gsi_kv_attention", attention)
    monkeypatch.setattr(lib.KVCache, "_ints", lambda *a: None)
    return seen


def cache():
    c = object.__new__(lib.KVCache)
    c.kv, c.seqs, c.heads, c.q_heads, c.head_dim = None, 1, 1, 2, 64
    return c


@pytest.mark.parametrize("stream", [None, 11, 22, FakeStream(11), FakeStream(33)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_tensors_made_for_a_call_are_of_its_stream(cuda, stream, accumulate):
    """The allocator orders a block's next use after its last one on the stream that
    it was allocated under, and on no other: out and lse belong to the call's."""
    q = torch.zeros((3, 128), dtype=torch.bfloat16)
    cache().attention(q, None, None, 3, accumulate=accumulate, stream=stream)
    want = 11 if stream is None else lib._raw(stream)
    assert cuda["launched"] == [want]
    assert cuda["allocated"] == [want] * (2 if accumulate else 1)
    assert cuda["current"] == 11


@pytest.mark.parametrize("stream", [None, 11, 22, FakeStream(33)])
def test_an_output_of_a_gated_linear_is_of_its_stream(cuda, monkeypatch, stream):
    monkeypatch.setattr(lib, "gsi_forward", lambda h, x, y, gate, rho, s: cuda["launched"].append(lib._raw(s)))
    layer = object.__new__(lib.GatedLinear)
    layer.h, layer.d_out = None, 8
    layer(torch.zeros((2, 4)), stream=stream)
    assert cuda["allocated"] == cuda["launched"] == [11 if stream is None else lib._raw(stream)]
