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
    monkeypatch.setattr(lib, "_current_device", lambda: -1, raising=False)
    monkeypatch.setattr(lib, "gsi_kv_attention", attention)
    monkeypatch.setattr(lib.KVCache, "_ints", lambda *a: None)
    return seen


def cache():
    c = object.__new__(lib.KVCache)
    c.kv, c.seqs, c.heads, c.q_heads, c.head_dim = None, 1, 1, 2, 64
    c._device = -1  # the fakes' tensors are the CPU's
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


class FakeTensor:
    """A contiguous CUDA tensor, as far as the binding looks at it."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device

    def is_contiguous(self):
        return True

    def stride(self):
        return (self.shape[-1], 1)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000


def fake_buffers(device, **other):
    shapes = {"k_pages": ((4, 2, 64, 64), torch.int8), "k_scale": ((4, 2), torch.float32),
              "k_tail": ((1, 2, 64, 64), torch.bfloat16), "page_table": ((1, 3), torch.int32)}
    shapes.update({"v" + n[1:]: s for n, s in list(shapes.items()) if n[0] == "k"})
    return {n: FakeTensor(s, d, other.get(n, device)) for n, (s, d) in shapes.items()}


def test_a_cache_is_of_the_current_device(monkeypatch):
    """Kernels are queued on the current device: a cache, and a call's tensors, of another
    one are refused before the library sees them."""
    made = []
    monkeypatch.setattr(lib, "gsi_kv_create", lambda b: made.append(b))
    monkeypatch.setattr(lib, "_current_device", lambda: 0, raising=False)
    for bad in (fake_buffers(1), fake_buffers(0, v_tail=1), fake_buffers(1, k_pages=0)):
        with pytest.raises(ValueError):
            lib.KVCache(1, 2, 64, 4, 3, buffers=bad)
    assert not made
    c = lib.KVCache(1, 2, 64, 4, 3, buffers=fake_buffers(0))
    assert len(made) == 1

    def tensors(**other):
        shapes = {"row_start": ((2,), torch.int32), "length": ((1,), torch.int32), "spare": ((1, 3), torch.int32),
                  "x": ((1, 128), torch.float32), "out": ((1, 128), torch.bfloat16), "lse": ((1, 2), torch.float32)}
        return {n: FakeTensor(s, d, other.get(n, 0)) for n, (s, d) in shapes.items()}

    calls = {"append": lambda t: c.append(t["x"], t["x"], t["row_start"], t["length"], 1),
             "attention": lambda t: c.attention(t["x"], t["row_start"], t["length"], 1, out=t["out"], lse=t["lse"]),
             "evict": lambda t: c.evict(t["length"], 64, 8, t["spare"])}
    called = []
    for name in ("append", "attention", "evict"):
        monkeypatch.setattr(lib, "gsi_kv_" + name, lambda *a: called.append(a))
    uses = {"append": ("x", "row_start", "length"), "attention": ("x", "row_start", "length", "out", "lse"),
            "evict": ("length", "spare")}
    for name, call in calls.items():
        for n in uses[name]:
            with pytest.raises(TypeError):
                call(tensors(**{n: 1}))
    assert not called
    for call in calls.values():
        call(tensors())
    assert len(called) == 3
    monkeypatch.setattr(lib, "_current_device", lambda: 1)
    for call in calls.values():
        with pytest.raises(ValueError):
            call(tensors())
    assert len(called) == 3
