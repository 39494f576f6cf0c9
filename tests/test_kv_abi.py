"""Refusals of the key/value cache's entry points (CPU: each case is answered
before any CUDA call; the pointer values are never followed)."""
import ctypes
import math

import pytest

A = 0x10000


@pytest.fixture(scope="module")
def gsi():
    from gated_rank_subspace_gsi_gb300 import build, lib
    build.build()
    return lib


def _buffers(lib, **kw):
    b = dict(format=0, seqs=2, heads=4, q_heads=8, head_dim=128, max_pages=16, pages=32,
             k_pages=A, v_pages=A, k_scale=A, v_scale=A, k_tail=A, v_tail=A, page_table=A, score=A)
    b.update(kw)
    s = lib.KvBuffers()
    for n, v in b.items():
        setattr(s, n, v)
    return s


@pytest.mark.parametrize("change,status", [
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
    (dict(k_tail=None), 1), (dict(v_tail=None), 1), (dict(page_table=None), 1),
    (dict(k_pages=A + 8), 1), (dict(v_tail=A + 4), 1), (dict(score=A + 4), 1),
    (dict(format=2), 1), (dict(format=-1), 1),
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(head_dim=512), 2),
    (dict(q_heads=6), 2), (dict(q_heads=0), 2), (dict(q_heads=4 * 65), 2), (dict(heads=0), 2),
    (dict(heads=8192, q_heads=8192), 2), (dict(seqs=0), 2), (dict(seqs=65536), 2),
    (dict(max_pages=0), 2), (dict(pages=0), 2), (dict(pages=2 ** 31 // 256), 2), (dict(pages=2 ** 40), 2),
])
def test_create_refuses(gsi, change, status):
    cl = gsi.library()
    out = ctypes.c_void_p(123)
    assert cl.gsi_kv_create(ctypes.byref(_buffers(gsi, **change)), ctypes.byref(out)) == status
    assert not out.value


def test_null_handles(gsi):
    cl = gsi.library()
    out = ctypes.c_void_p()
    assert cl.gsi_kv_create(None, ctypes.byref(out)) == 1
    assert cl.gsi_kv_create(ctypes.byref(_buffers(gsi)), None) == 1
    assert cl.gsi_kv_append(None, A, 512, A, 512, 0, A, 1, 1, A, None) == 1
    assert cl.gsi_kv_attention(None, A, 1024, 0, A, 1, 1, A, ctypes.c_float(1), A, 1024, None, 0, None) == 1
    assert cl.gsi_kv_evict(None, A, 64, 8, A, A, None) == 1
    assert cl.gsi_kv_status(None, None) == 1
    cl.gsi_kv_destroy(None)


def test_status_strings(gsi):
    cl = gsi.library()
    assert b"NONFINITE" in cl.gsi_status_string(9)
    assert b"PAGE" in cl.gsi_status_string(10)
    assert b"unknown" in cl.gsi_status_string(11)


@pytest.mark.gpu
def test_calls_refuse(gsi):
    """Argument checks of a live handle (host only: nothing is launched)."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = gsi.KVCache(2, 4, 128, 32, 16, q_heads=8, score=True)
    cl, f = gsi.library(), ctypes.c_float
    ok = [c.kv, A, 512, A, 512, 0, A, 4, 2, A, None]

    def append(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return cl.gsi_kv_append(*a)

    assert append(_7=0, _8=0) == 0                       # no rows: nothing to do
    for bad in (dict(_1=None), dict(_1=A + 4), dict(_2=511), dict(_2=514), dict(_3=None), dict(_4=508),
                dict(_5=2), dict(_6=None), dict(_6=A + 2), dict(_7=-1), dict(_7=2 ** 31), dict(_8=5),
                dict(_8=-1), dict(_9=None), dict(_9=A + 1)):
        assert append(**bad) == 1, bad
    assert append(_2=516, _5=1) == 1                     # bf16: the row stride is not 16-byte aligned
    ok = [c.kv, A, 1024, 0, A, 4, 2, A, f(0.1), A, 1024, A, 0, None]

    def attend(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return cl.gsi_kv_attention(*a)

    assert attend(_5=0, _6=0) == 0
    for bad in (dict(_1=None), dict(_2=1020), dict(_3=7), dict(_4=None), dict(_5=-1), dict(_6=5),
                dict(_7=None), dict(_8=f(math.nan)), dict(_8=f(math.inf)), dict(_9=None), dict(_9=A + 8),
                dict(_10=1023), dict(_11=A + 2), dict(_11=None, _12=1)):
        assert attend(**bad) == 1, bad
    for bad in ((None, 64, 8, A, A), (A, 0, 0, A, A), (A, 64, 65, A, A), (A, 64, -1, A, A),
                (A, 64, 8, None, A), (A, 64, 8, A, None), (A + 2, 64, 8, A, A)):
        assert cl.gsi_kv_evict(c.kv, *bad, None) == 1, bad
    plain = gsi.KVCache(2, 4, 128, 32, 16, q_heads=8)    # no score buffer
    assert cl.gsi_kv_evict(plain.kv, A, 64, 8, A, A, None) == 1
    assert cl.gsi_kv_attention(plain.kv, A, 1024, 0, A, 4, 2, A, f(0.1), A, 1024, A, 1, None) == 1
    x = torch.zeros((4, 512), device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        c.append(x.half(), x.half(), i, i[:2], 1)
    with pytest.raises(TypeError):
        c.append(x, x, i.long(), i[:2], 1)
    with pytest.raises(ValueError):
        c.append(x[:, :256], x[:, :256], i, i[:2], 1)
    with pytest.raises(ValueError):
        c.append(x.t().contiguous().t(), x, i, i[:2], 1)
    with pytest.raises(TypeError):
        gsi.KVCache(2, 4, 128, 32, 16, buffers={**c.buffers, "k_tail": c.k_tail.float()})
    plain.close()
    c.close()


@pytest.mark.gpu
def test_host_tensors_are_refused(gsi):
    """The binding takes no address of host memory."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = gsi.KVCache(2, 4, 128, 32, 16, q_heads=8, score=True)
    x, q = torch.zeros((4, 512), device="cuda"), torch.zeros((4, 1024), device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    spare = torch.zeros((2, 16), dtype=torch.int32, device="cuda")
    for call in (lambda: c.append(x.cpu(), x, i, i[:2], 1), lambda: c.append(x, x.cpu(), i, i[:2], 1),
                 lambda: c.append(x, x, i.cpu(), i[:2], 1), lambda: c.append(x, x, i, i[:2].cpu(), 1),
                 lambda: c.attention(q.cpu(), i, i[:2], 1), lambda: c.attention(q, i.cpu(), i[:2], 1),
                 lambda: c.attention(q, i, i[:2], 1, out=q.bfloat16().cpu()),
                 lambda: c.attention(q, i, i[:2], 1, lse=torch.zeros((4, 8))),
                 lambda: c.evict(i[:2].cpu(), 64, 8, spare), lambda: c.evict(i[:2], 64, 8, spare.cpu()),
                 lambda: c.evict(i[:2], 64, 8, spare, i[:2].cpu())):
        with pytest.raises(TypeError):
            call()
    c.close()


def test_kernels_read_no_buffer_as_constant():
    """Under programmatic dependent launch a kernel of the cache may start while earlier
    ones of the stream still write the pages: none reads through the read-only path
    (ld.global.nc, __ldg, what __restrict__ lets the compiler use), whose lines must not
    change while the kernel lives."""
    import os
    import re
    from gated_rank_subspace_gsi_gb300 import build
    names = [n for n in os.listdir(build.CSRC) if n.startswith("gsi_kv")]
    assert len(names) >= 8
    for n in names:
        with open(os.path.join(build.CSRC, n)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"ld_stream_v4|__ldg\b|__restrict__|global\.nc", code), n
