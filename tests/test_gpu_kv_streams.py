"""Calls of the 8-bit key/value cache on another stream than torch's current one,
with the tensors that the binding allocates for them.
"""
import pytest
import torch

from test_gpu_kv import Pair

pytestmark = pytest.mark.gpu

BUSY = 40_000_000  # cycles: about 20 ms, far longer than a call's host side


def held(gsi):
    """A cache, and the queries of one more row for each sequence."""
    p = Pair(gsi, 3, 2, 2, 64, "int8", seed=17)
    p.step([200, 70, 1])
    (q, k, v), start = p.rows([1, 1, 1])
    p.c.append(k[1], v[1], start, p.len, 1)
    p.c.score.zero_()
    torch.cuda.synchronize()
    return p, q[1], start


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_memory_of_a_call_is_not_given_out_while_it_runs(gsi, kind):
    """The call waits on a busy stream; tensors made meanwhile on the current one
    keep what they were filled with, and the weights are those of a plain call."""
    p, q, start = held(gsi)
    out = p.c.attention(q, start, p.len, 1, accumulate=True)
    torch.cuda.synchronize()
    want = p.c.score.clone()
    p.c.score.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    p.c.attention(q, start, p.len, 1, accumulate=True, stream=side if kind == "stream" else side.cuda_stream)
    made = [torch.full_like(x, 7.0) for x in (out, torch.empty((3, 4), device="cuda")) for _ in range(6)]
    torch.cuda.synchronize()
    for x in made:
        assert (x == 7.0).all()
    assert torch.equal(p.c.score, want)
    assert p.c.status() == 0
    p.c.close()


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_a_call_does_not_get_memory_in_use(gsi, kind):
    """Blocks that the current stream has freed and still writes to are not the call's."""
    p, q, start = held(gsi)
    want = p.c.attention(q, start, p.len, 1, accumulate=True).clone()
    weights = p.c.score.clone()
    p.c.score.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(x) for x in (want, torch.empty((3, 4), device="cuda")) for _ in range(6)]
    torch.cuda._sleep(BUSY)
    for x in freed:
        x.fill_(float("nan"))
    del freed, x
    out = p.c.attention(q, start, p.len, 1, accumulate=True, stream=side if kind == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(p.c.score, weights)
    assert p.c.status() == 0
    p.c.close()
