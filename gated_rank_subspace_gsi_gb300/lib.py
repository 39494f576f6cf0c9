"""ctypes binding of libgsi.so, the C ABI in include/gsi.h.

Argument marshalling only: every step of the gated map runs in the library's
CUDA kernels.  Functions keep the C names.  Tensors are torch tensors (device
memory for everything except the *_host variant); PyTorch supplies memory and
streams and nothing else.  If libgsi.so is missing it is built with nvcc; if
that is impossible the import fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

GSI_OK = 0
GSI_ERR_INVALID_ARG = 1
GSI_ERR_UNSUPPORTED_SHAPE = 2
GSI_ERR_NOMEM = 3
GSI_ERR_CUDA = 4
GSI_ERR_WORKSPACE = 5
GSI_ERR_TIMEOUT = 6
GSI_ERR_LAUNCH = 7
GSI_ERR_RANK = 8
GSI_ERR_NONFINITE = 9
GSI_ERR_PAGE = 10

# every function declared in include/gsi.h
EXPORTS = ("gsi_create", "gsi_forward", "gsi_forward_host", "gsi_precompute_M",
           "gsi_reserve", "gsi_device_status", "gsi_destroy", "gsi_status_string",
           "gsi_forward_launch_count", "gsi_forward_noalloc", "gsi_set_prefetch",
           "gsi_set_prefetch_group", "gsi_group_create", "gsi_group_forward",
           "gsi_group_forward_host",
           "gsi_group_set_prefetch", "gsi_group_destroy", "gsi_calibrate_workspace_size",
           "gsi_calibrate", "gsi_calibrate_status", "gsi_calibrate_launch_count",
           "gsi_calibrate_timed", "gsi_calibrate_cascade", "gsi_refine_rank1_workspace_size",
           "gsi_refine_rank1", "gsi_calibrate_cascade_rank1", "gsi_refine_rank1_launch_count",
           "gsi_kv_create", "gsi_kv_append", "gsi_kv_attention", "gsi_kv_evict", "gsi_kv_status",
           "gsi_kv_destroy")

GSI_KV_INT8 = 0
GSI_KV_E4M3 = 1
GSI_F32 = 0
GSI_BF16 = 1

_lock = threading.Lock()
_lib = None


class KvBuffers(ctypes.Structure):
    """gsi_kv_buffers_t: the device buffers of a key/value cache and their sizes."""
    _fields_ = [("format", ctypes.c_int32), ("seqs", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("pages", ctypes.c_int64),
                ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("score", ctypes.c_void_p)]


class GsiError(RuntimeError):
    """A call into libgsi returned a status other than GSI_OK."""

    def __init__(self, status: int, what: str):
        self.status = int(status)
        msg = _load().gsi_status_string(self.status).decode()
        super().__init__(f"{what}: {msg}")


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            _build.build()
        lib = ctypes.CDLL(path)
        P, I64 = ctypes.c_void_p, ctypes.c_int64
        lib.gsi_create.argtypes = [P, P, P, I64, I64, I64, ctypes.c_float, ctypes.POINTER(P)]
        lib.gsi_create.restype = ctypes.c_int
        lib.gsi_forward.argtypes = [P, P, I64, P, P, P, P]
        lib.gsi_forward.restype = ctypes.c_int
        lib.gsi_forward_host.argtypes = [P, P, I64, P, P, P, P]
        lib.gsi_forward_host.restype = ctypes.c_int
        lib.gsi_precompute_M.argtypes = [P, P, P, I64, I64, I64, P]
        lib.gsi_precompute_M.restype = ctypes.c_int
        lib.gsi_reserve.argtypes = [P, I64]
        lib.gsi_reserve.restype = ctypes.c_int
        lib.gsi_device_status.argtypes = [P, P]
        lib.gsi_device_status.restype = ctypes.c_int
        lib.gsi_destroy.argtypes = [P]
        lib.gsi_destroy.restype = None
        lib.gsi_status_string.argtypes = [ctypes.c_int]
        lib.gsi_status_string.restype = ctypes.c_char_p
        lib.gsi_forward_launch_count.argtypes = [P, I64]
        lib.gsi_forward_launch_count.restype = ctypes.c_int
        lib.gsi_forward_noalloc.argtypes = [P, P, P, I64, I64, I64, ctypes.c_float, P, P, P, P, P]
        lib.gsi_forward_noalloc.restype = ctypes.c_int
        lib.gsi_set_prefetch.argtypes = [P, P]
        lib.gsi_set_prefetch.restype = ctypes.c_int
        lib.gsi_set_prefetch_group.argtypes = [P, P]
        lib.gsi_set_prefetch_group.restype = ctypes.c_int
        lib.gsi_group_create.argtypes = [ctypes.c_int, P, ctypes.POINTER(P)]
        lib.gsi_group_create.restype = ctypes.c_int
        lib.gsi_group_forward.argtypes = [P, P, P, P, P, P]
        lib.gsi_group_forward.restype = ctypes.c_int
        lib.gsi_group_forward_host.argtypes = [P, P, P, P, P, P]
        lib.gsi_group_forward_host.restype = ctypes.c_int
        lib.gsi_group_set_prefetch.argtypes = [P, P]
        lib.gsi_group_set_prefetch.restype = ctypes.c_int
        lib.gsi_group_destroy.argtypes = [P]
        lib.gsi_group_destroy.restype = None
        lib.gsi_calibrate_workspace_size.argtypes = [I64, I64, I64, ctypes.POINTER(ctypes.c_size_t)]
        lib.gsi_calibrate_workspace_size.restype = ctypes.c_int
        lib.gsi_calibrate.argtypes = [P, I64, I64, I64, P, ctypes.c_int, P, P, ctypes.c_size_t, P]
        lib.gsi_calibrate.restype = ctypes.c_int
        lib.gsi_calibrate_timed.argtypes = [P, I64, I64, I64, P, ctypes.c_int, P, P, ctypes.c_size_t,
                                            P, P, P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        lib.gsi_calibrate_timed.restype = ctypes.c_int
        lib.gsi_calibrate_cascade.argtypes = [P, ctypes.c_int, I64, I64, I64, P, ctypes.c_int,
                                              ctypes.c_int, P, P, ctypes.c_size_t, P]
        lib.gsi_calibrate_cascade.restype = ctypes.c_int
        lib.gsi_calibrate_status.argtypes = [P, P]
        lib.gsi_calibrate_status.restype = ctypes.c_int
        lib.gsi_calibrate_launch_count.argtypes = [I64, I64, I64, ctypes.c_int]
        lib.gsi_calibrate_launch_count.restype = ctypes.c_int
        lib.gsi_refine_rank1_workspace_size.argtypes = [I64, I64, I64,
                                                        ctypes.POINTER(ctypes.c_size_t)]
        lib.gsi_refine_rank1_workspace_size.restype = ctypes.c_int
        lib.gsi_refine_rank1.argtypes = [P, I64, I64, I64, P, ctypes.c_int, P, P, P,
                                         ctypes.c_size_t, P]
        lib.gsi_refine_rank1.restype = ctypes.c_int
        lib.gsi_calibrate_cascade_rank1.argtypes = [P, ctypes.c_int, I64, I64, I64, P,
                                                    ctypes.c_int, ctypes.c_int, P, P, P,
                                                    ctypes.c_size_t, P]
        lib.gsi_calibrate_cascade_rank1.restype = ctypes.c_int
        lib.gsi_refine_rank1_launch_count.argtypes = [I64, I64, I64, ctypes.c_int]
        lib.gsi_refine_rank1_launch_count.restype = ctypes.c_int
        lib.gsi_kv_create.argtypes = [ctypes.POINTER(KvBuffers), ctypes.POINTER(P)]
        lib.gsi_kv_create.restype = ctypes.c_int
        lib.gsi_kv_append.argtypes = [P, P, I64, P, I64, ctypes.c_int, P, I64, I64, P, P]
        lib.gsi_kv_append.restype = ctypes.c_int
        lib.gsi_kv_attention.argtypes = [P, P, I64, ctypes.c_int, P, I64, I64, P, ctypes.c_float,
                                         P, I64, P, ctypes.c_int, P]
        lib.gsi_kv_attention.restype = ctypes.c_int
        lib.gsi_kv_evict.argtypes = [P, P, I64, I64, P, P, P]
        lib.gsi_kv_evict.restype = ctypes.c_int
        lib.gsi_kv_status.argtypes = [P, P]
        lib.gsi_kv_status.restype = ctypes.c_int
        lib.gsi_kv_destroy.argtypes = [P]
        lib.gsi_kv_destroy.restype = None
        _lib = lib
        return lib


def library():
    """The loaded ctypes library (built on first use if missing)."""
    return _load()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


_raw_stream = None


def _current_stream() -> int:
    """The current stream's handle.  torch.cuda.current_stream() builds a Python
    object (about 5 us); torch's own fast path, where it has one, a number."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        try:
            get, dev = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            torch.cuda.init()
            get(dev())
            _raw_stream = lambda: get(dev())  # noqa: E731
        except AttributeError:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


_device_index = None


def _current_device() -> int:
    """The current CUDA device's number."""
    global _device_index
    if _device_index is None:
        import torch
        torch.cuda.init()
        _device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _device_index()


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(_current_stream())
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _raw(stream) -> int:
    if stream is None:
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """torch.empty of the stream that a call is queued on.  The caching allocator
    gives a block out again in the order of the stream that it was allocated
    under; under another one the block could still be in use by earlier work of
    that stream, or serve later work of it while the call runs."""
    import torch
    if stream is None or _raw(stream) == _current_stream():
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_raw(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(st: int, what: str):
    if st != GSI_OK:
        raise GsiError(st, what)


def gsi_status_string(status: int) -> str:
    return _load().gsi_status_string(int(status)).decode()


def gsi_create(W, V_k, M, eps: float) -> ctypes.c_void_p:
    """Handle for one gated linear.  W (d_out x d), V_k (d x k), M (d_out x k):
    bf16 CUDA tensors, borrowed (keep them alive and unchanged)."""
    d_out, d = W.shape
    d2, k = V_k.shape
    if d2 != d or tuple(M.shape) != (d_out, k):
        raise ValueError("W, V_k and M shapes disagree")
    h = ctypes.c_void_p()
    _check(_load().gsi_create(_ptr(W), _ptr(V_k), _ptr(M), d_out, d, k, float(eps),
                              ctypes.byref(h)), "gsi_create")
    return h


def gsi_forward(h, x, y, gate=None, rho=None, stream=None, T=None):
    """y (T x d_out fp32), gate (T uint8) and rho (T fp32) of the gated map on
    x (T x d bf16), all CUDA tensors; asynchronous on `stream`."""
    T = x.shape[0] if T is None else T
    _check(_load().gsi_forward(h, _ptr(x), T, _ptr(y), _ptr(gate), _ptr(rho), _stream(stream)),
           "gsi_forward")


def gsi_forward_host(h, x_host, y_host, gate_host=None, rho_host=None, stream=None, T=None):
    """gsi_forward on host (CPU, ideally pinned) tensors; copies are queued on
    `stream`, which the caller synchronises before reading the outputs."""
    T = x_host.shape[0] if T is None else T
    _check(_load().gsi_forward_host(h, _ptr(x_host), T, _ptr(y_host), _ptr(gate_host),
                                    _ptr(rho_host), _stream(stream)), "gsi_forward_host")


def gsi_precompute_M(W, V_k, M, stream=None):
    """M = bf16(W V_k) on the GPU (fp32 accumulation)."""
    d_out, d = W.shape
    _, k = V_k.shape
    _check(_load().gsi_precompute_M(_ptr(W), _ptr(V_k), _ptr(M), d_out, d, k, _stream(stream)),
           "gsi_precompute_M")


def gsi_reserve(h, max_T: int):
    _check(_load().gsi_reserve(h, int(max_T)), "gsi_reserve")


def gsi_device_status(h, stream=None) -> int:
    """Synchronise the stream, return (and clear) the handle's device status."""
    return int(_load().gsi_device_status(h, _stream(stream)))


def gsi_destroy(h):
    if h is not None:
        _load().gsi_destroy(h)


def gsi_set_prefetch(h, next_h):
    """Make each one-token call on h prefetch next_h's operands into L2
    (next_h None removes the link)."""
    _check(_load().gsi_set_prefetch(h, next_h), "gsi_set_prefetch")


def gsi_set_prefetch_group(h, group):
    """Make each one-token call on h prefetch every member of `group` into L2
    (None removes the link)."""
    _check(_load().gsi_set_prefetch_group(h, group), "gsi_set_prefetch_group")


def _ptr_array(items):
    arr = (ctypes.c_void_p * len(items))()
    for i, t in enumerate(items):
        arr[i] = _ptr(t)
    return arr


def gsi_group_create(handles) -> ctypes.c_void_p:
    """One launch for several independent one-token calls (a group of handles)."""
    arr = (ctypes.c_void_p * len(handles))(*[h.value if isinstance(h, ctypes.c_void_p) else h
                                             for h in handles])
    g = ctypes.c_void_p()
    _check(_load().gsi_group_create(len(handles), arr, ctypes.byref(g)), "gsi_group_create")
    return g


def gsi_group_forward(g, xs, ys, gates=None, rhos=None, stream=None):
    """One token through every member of group g (lists of device tensors)."""
    _check(_load().gsi_group_forward(g, _ptr_array(xs), _ptr_array(ys),
                                     _ptr_array(gates) if gates is not None else None,
                                     _ptr_array(rhos) if rhos is not None else None,
                                     _stream(stream)), "gsi_group_forward")


def gsi_group_forward_host(g, xs, ys, gates=None, rhos=None, stream=None):
    """gsi_group_forward on host buffers (lists of CPU tensors, page-locked
    for the copy-free path)."""
    _check(_load().gsi_group_forward_host(g, _ptr_array(xs), _ptr_array(ys),
                                          _ptr_array(gates) if gates is not None else None,
                                          _ptr_array(rhos) if rhos is not None else None,
                                          _stream(stream)), "gsi_group_forward_host")


def gsi_group_set_prefetch(g, next_h):
    _check(_load().gsi_group_set_prefetch(g, next_h), "gsi_group_set_prefetch")


def gsi_group_destroy(g):
    if g is not None:
        _load().gsi_group_destroy(g)


def gsi_forward_launch_count(h, T: int) -> int:
    return int(_load().gsi_forward_launch_count(h, int(T)))


def gsi_forward_noalloc(W, V_k, M, eps: float, x, y, gate=None, rho=None, stream=None):
    """One token of the gated map with no handle and no allocation (for
    callers whose device memory is owned by another allocator); its scratch is
    a fixed array inside the library, shared by all calls on a device."""
    d_out, d = W.shape
    _, k = V_k.shape
    _check(_load().gsi_forward_noalloc(_ptr(W), _ptr(V_k), _ptr(M), d_out, d, k, float(eps),
                                       _ptr(x), _ptr(y), _ptr(gate), _ptr(rho), _stream(stream)),
           "gsi_forward_noalloc")


class GatedLinear:
    """One gated linear (W, V_k, M, eps) bound to a libgsi handle.

    Holds references to the borrowed tensors so they outlive the handle.
    """

    def __init__(self, W, V_k, M, eps: float, max_T: int = 0):
        import torch
        for name, t in (("W", W), ("V_k", V_k), ("M", M)):
            if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
                raise TypeError(f"{name} must be a contiguous bf16 CUDA tensor")
        self.W, self.V_k, self.M, self.eps = W, V_k, M, float(eps)
        self.d_out, self.d = W.shape
        self.k = V_k.shape[1]
        self.h = gsi_create(W, V_k, M, eps)
        if max_T > 0:
            gsi_reserve(self.h, max_T)

    def forward(self, x, y=None, gate=None, rho=None, stream=None):
        T = x.shape[0]
        if y is None:
            import torch
            y = _empty((T, self.d_out), torch.float32, x.device, stream)
        gsi_forward(self.h, x, y, gate, rho, stream)
        return y

    __call__ = forward

    def status(self, stream=None) -> int:
        return gsi_device_status(self.h, stream)

    def close(self):
        if self.h is not None:
            gsi_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- calibration of V_k ---------------------------------------------------


def gsi_calibrate_workspace_size(n: int, d: int, k: int) -> int:
    """Device scratch bytes gsi_calibrate needs for n tokens of width d, rank k."""
    out = ctypes.c_size_t()
    _check(_load().gsi_calibrate_workspace_size(int(n), int(d), int(k), ctypes.byref(out)),
           "gsi_calibrate_workspace_size")
    return int(out.value)


def gsi_calibrate(X, Q0, iters: int, V_k, workspace, stream=None):
    """V_k (d x k bf16) = orthonormal basis of span((X^T X)^iters Q0), by block
    power iteration on the GPU.  X (n x d), Q0 (d x k): bf16 CUDA tensors;
    workspace: a CUDA tensor of at least gsi_calibrate_workspace_size bytes."""
    n, d = X.shape
    d2, k = Q0.shape
    if d2 != d or tuple(V_k.shape) != (d, k):
        raise ValueError("X, Q0 and V_k shapes disagree")
    nbytes = workspace.numel() * workspace.element_size()
    _check(_load().gsi_calibrate(_ptr(X), n, d, k, _ptr(Q0), int(iters), _ptr(V_k),
                                 _ptr(workspace), nbytes, _stream(stream)), "gsi_calibrate")


def gsi_calibrate_status(workspace, stream=None) -> int:
    """Synchronise the stream; the device-side status of the last gsi_calibrate."""
    return int(_load().gsi_calibrate_status(_ptr(workspace), _stream(stream)))


def gsi_calibrate_launch_count(n: int, d: int, k: int, iters: int) -> int:
    return int(_load().gsi_calibrate_launch_count(int(n), int(d), int(k), int(iters)))


CAL_KINDS = ("transpose", "tensor-core GEMM", "split-K sum", "Gram matrix", "Cholesky",
             "forward substitution")


def gsi_calibrate_timed(X, Q0, iters: int, V_k, workspace, stream=None, max_launches: int = 4096):
    """gsi_calibrate with an event pair around every launch; returns a list of
    (kind name, ms) in launch order (synchronises the stream)."""
    n, d = X.shape
    _, k = Q0.shape
    ms = (ctypes.c_float * max_launches)()
    kinds = (ctypes.c_int * max_launches)()
    cnt = ctypes.c_int()
    nbytes = workspace.numel() * workspace.element_size()
    _check(_load().gsi_calibrate_timed(_ptr(X), n, d, k, _ptr(Q0), int(iters), _ptr(V_k),
                                       _ptr(workspace), nbytes, _stream(stream), ms, kinds,
                                       max_launches, ctypes.byref(cnt)), "gsi_calibrate_timed")
    return [(CAL_KINDS[kinds[i]], float(ms[i])) for i in range(cnt.value)]


def gsi_calibrate_cascade(Xs, Q0, iters_first: int, iters_next: int, Vs, workspace, stream=None):
    """Depth cascade: V_0 from Q0 with iters_first iterations on Xs[0]; V_l
    from V_{l-1} with iters_next iterations on Xs[l].  Xs: list of n x d bf16
    CUDA tensors; Vs: list of d x k bf16 CUDA tensors (outputs)."""
    if len(Xs) != len(Vs) or not Xs:
        raise ValueError("one output basis per layer")
    n, d = Xs[0].shape
    _, k = Q0.shape
    xa = _ptr_array(Xs)
    va = _ptr_array(Vs)
    nbytes = workspace.numel() * workspace.element_size()
    _check(_load().gsi_calibrate_cascade(xa, len(Xs), n, d, k, _ptr(Q0), int(iters_first),
                                         int(iters_next), va, _ptr(workspace), nbytes,
                                         _stream(stream)), "gsi_calibrate_cascade")


def gsi_refine_rank1_workspace_size(n: int, d: int, k: int) -> int:
    """Device scratch bytes gsi_refine_rank1 (and the rank-1 cascade) need."""
    out = ctypes.c_size_t()
    _check(_load().gsi_refine_rank1_workspace_size(int(n), int(d), int(k), ctypes.byref(out)),
           "gsi_refine_rank1_workspace_size")
    return int(out.value)


def gsi_refine_rank1(X, V_in, corrections: int, V_out, workspace, order=None, stream=None):
    """`corrections` rank-1 DGKS corrections of the start basis V_in (d x k
    bf16) for the tokens X (n x d bf16), into V_out; order (int32 CUDA tensor
    of `corrections` entries, optional) receives the corrected columns."""
    n, d = X.shape
    _, k = V_in.shape
    nbytes = workspace.numel() * workspace.element_size()
    _check(_load().gsi_refine_rank1(_ptr(X), n, d, k, _ptr(V_in), int(corrections), _ptr(V_out),
                                    _ptr(order), _ptr(workspace), nbytes, _stream(stream)),
           "gsi_refine_rank1")


def gsi_calibrate_cascade_rank1(Xs, Q0, iters_first: int, corrections: int, Vs, workspace,
                                order=None, stream=None):
    """Depth cascade in rank-1 form: V_0 = gsi_calibrate(Xs[0], Q0,
    iters_first); V_l = gsi_refine_rank1(Xs[l], V_{l-1}, corrections).  order:
    optional int32 CUDA tensor of (layers - 1) * corrections entries."""
    if len(Xs) != len(Vs) or not Xs:
        raise ValueError("one output basis per layer")
    n, d = Xs[0].shape
    _, k = Q0.shape
    xa = _ptr_array(Xs)
    va = _ptr_array(Vs)
    nbytes = workspace.numel() * workspace.element_size()
    _check(_load().gsi_calibrate_cascade_rank1(xa, len(Xs), n, d, k, _ptr(Q0), int(iters_first),
                                               int(corrections), va, _ptr(order),
                                               _ptr(workspace), nbytes, _stream(stream)),
           "gsi_calibrate_cascade_rank1")


def gsi_refine_rank1_launch_count(n: int, d: int, k: int, corrections: int) -> int:
    return int(_load().gsi_refine_rank1_launch_count(int(n), int(d), int(k), int(corrections)))


# ---- the key/value cache in 8 bits ------------------------------------------


def gsi_kv_create(buffers: KvBuffers) -> ctypes.c_void_p:
    """Handle on the device buffers of a key/value cache (borrowed)."""
    kv = ctypes.c_void_p()
    _check(_load().gsi_kv_create(ctypes.byref(buffers), ctypes.byref(kv)), "gsi_kv_create")
    return kv


_kv_types = None


def _kv_rows(t, what: str):
    """(address, row stride, dtype) of a rows x width fp32 or bf16 tensor."""
    global _kv_types
    if _kv_types is None:
        import torch
        _kv_types = {torch.float32: GSI_F32, torch.bfloat16: GSI_BF16}
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"{what} must be rows x width with contiguous rows")
    dt = _kv_types.get(t.dtype)
    if dt is None or not t.is_cuda:
        raise TypeError(f"{what} must be an fp32 or bf16 CUDA tensor")
    return t.data_ptr(), (stride[0] if shape[0] > 1 else shape[1]), dt


def gsi_kv_append(kv, k, v, row_start, length, max_rows: int, stream=None):
    """Append the packed new rows k, v (rows x heads * D, fp32 or bf16, row
    slices allowed) to the cache; row_start (seqs + 1) and length (seqs: tokens
    held before the call): int32 CUDA tensors.  max_rows: a bound of the new rows
    of a sequence; one above the rows of the call will do."""
    kp, ldk, dt = _kv_rows(k, "k")
    vp, ldv, dtv = _kv_rows(v, "v")
    if dtv != dt or k.shape != v.shape:
        raise ValueError("k and v differ in shape or type")
    rows = k.shape[0]
    _check(_load().gsi_kv_append(kv, kp, ldk, vp, ldv, dt, row_start.data_ptr(), rows,
                                 min(max_rows, rows), length.data_ptr(), _raw(stream)),
           "gsi_kv_append")


def gsi_kv_attention(kv, q, row_start, length, max_rows: int, scale: float, out, lse=None,
                     accumulate: bool = False, stream=None):
    """Attention of the new rows q (rows x q_heads * D, fp32 or bf16) over the
    cache, after gsi_kv_append of the same rows with the same length; out: bf16.
    accumulate adds each token's weight to the cache's score (needs lse).
    max_rows as for gsi_kv_append; rows of a sequence beyond it are not computed.
    fp32 queries count with 11 bits, and with 21 where an lse is given."""
    qp, ldq, dt = _kv_rows(q, "q")
    op, ldo, dto = _kv_rows(out, "out")
    if dto != GSI_BF16 or out.shape != q.shape:
        raise ValueError("out must be bf16 of q's shape")
    if lse is not None:
        import torch
        if not (lse.dtype == torch.float32 and lse.is_cuda and lse.is_contiguous()):
            raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    rows = q.shape[0]
    _check(_load().gsi_kv_attention(kv, qp, ldq, dt, row_start.data_ptr(), rows,
                                    min(max_rows, rows), length.data_ptr(), scale, op, ldo,
                                    None if lse is None else lse.data_ptr(), 1 if accumulate else 0,
                                    _raw(stream)), "gsi_kv_attention")


def gsi_kv_evict(kv, length, budget: int, recent: int, spare_table, length_out, stream=None):
    """Cut every sequence longer than budget to its last `recent` tokens and the
    budget - recent others of largest score, into the pages of spare_table."""
    _check(_load().gsi_kv_evict(kv, _ptr(length), int(budget), int(recent), _ptr(spare_table),
                                _ptr(length_out), _stream(stream)), "gsi_kv_evict")


def gsi_kv_status(kv, stream=None) -> int:
    """Synchronise the stream, return (and clear) the cache's device status."""
    return int(_load().gsi_kv_status(kv, _stream(stream)))


def gsi_kv_destroy(kv):
    if kv is not None:
        _load().gsi_kv_destroy(kv)


class KVCache:
    """A key/value cache in 8 bits: its device buffers and a libgsi handle.

    seqs sequences of `heads` key/value heads of `head_dim`, in a pool of
    `pages` pages of 64 tokens, at most max_pages to a sequence.  fmt: "int8" or
    "e4m3".  buffers: a dict of the tensors below, or None to allocate them
    (page_table then starts as -1: no page).  score=True allocates the
    accumulated weights that eviction goes by.  Lengths are the caller's: int32
    CUDA tensors of seqs entries.  The cache is of the current device, which has
    to be current in its calls as well, and so are their tensors.
    """

    PAGE = 64

    def __init__(self, seqs: int, heads: int, head_dim: int, pages: int, max_pages: int,
                 q_heads=None, fmt: str = "int8", score: bool = False, buffers=None,
                 device="cuda"):
        import torch
        q_heads = heads if q_heads is None else q_heads
        if fmt not in ("int8", "e4m3"):
            raise ValueError("fmt must be 'int8' or 'e4m3'")
        code = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
        shapes = {"k_pages": ((pages, heads, 64, head_dim), code),
                  "k_scale": ((pages, heads), torch.float32),
                  "k_tail": ((seqs, heads, 64, head_dim), torch.bfloat16)}
        shapes.update({"v" + n[1:]: s for n, s in list(shapes.items())})
        shapes["page_table"] = ((seqs, max_pages), torch.int32)
        if buffers is None:
            buffers = {n: torch.zeros(s, dtype=dt, device=device) for n, (s, dt) in shapes.items()}
            buffers["page_table"].fill_(-1)
            if score:
                buffers["score"] = torch.zeros((pages, heads, 64), dtype=torch.float32,
                                               device=device)
        shapes["score"] = ((pages, heads, 64), torch.float32)
        for n, (shape, dt) in shapes.items():
            t = buffers.get(n)
            if t is None and n == "score":
                continue
            if t is None or tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous() \
                    or not t.is_cuda:
                raise TypeError(f"{n} must be a contiguous CUDA tensor {shape} of {dt}")
        self._device = _current_device()
        for n in shapes:
            if buffers.get(n) is not None and buffers[n].get_device() != self._device:
                raise ValueError(f"{n} is not of the current device, cuda:{self._device}")
        self.buffers = dict(buffers)
        for n in shapes:
            setattr(self, n, buffers.get(n))
        self.seqs, self.heads, self.q_heads, self.head_dim = seqs, heads, q_heads, head_dim
        self.kv, self._int = None, torch.int32
        b = KvBuffers(GSI_KV_INT8 if fmt == "int8" else GSI_KV_E4M3, seqs, heads, q_heads,
                      head_dim, max_pages, pages)
        for n in shapes:
            if buffers.get(n) is not None:
                setattr(b, n, buffers[n].data_ptr())
        self.kv = gsi_kv_create(b)

    def _ints(self, t, n: int, what: str):
        if not (t.dtype == self._int and t.get_device() == self._device and t.numel() == n
                and t.is_contiguous()):
            raise TypeError(f"{what} must be a contiguous int32 tensor of {n} entries on "
                            f"cuda:{self._device}")

    def _elsewhere(self):
        """What is raised where the current device or a tensor is not the cache's."""
        if _current_device() != self._device:
            raise ValueError(f"cuda:{self._device}, the cache's device, is not the current one")
        raise TypeError(f"a tensor of the call is not on cuda:{self._device}")

    def append(self, k, v, row_start, length, max_rows: int, stream=None):
        dev = self._device
        if _current_device() != dev or k.get_device() != dev or v.get_device() != dev:
            self._elsewhere()
        self._ints(row_start, self.seqs + 1, "row_start")
        self._ints(length, self.seqs, "length")
        if k.shape[1] != self.heads * self.head_dim:
            raise ValueError("k must be rows x heads * head_dim")
        gsi_kv_append(self.kv, k, v, row_start, length, max_rows, stream)

    def attention(self, q, row_start, length, max_rows: int, scale=None, out=None, lse=None,
                  accumulate: bool = False, stream=None):
        """An out that is not given is allocated under the call's stream, as torch
        would there: work of other streams waits for the call before it reads it."""
        dev = self._device
        if _current_device() != dev or q.get_device() != dev or \
                (out is not None and out.get_device() != dev) or \
                (lse is not None and lse.get_device() != dev):
            self._elsewhere()
        self._ints(row_start, self.seqs + 1, "row_start")
        self._ints(length, self.seqs, "length")
        if q.shape[1] != self.q_heads * self.head_dim:
            raise ValueError("q must be rows x q_heads * head_dim")
        if out is None:
            import torch
            out = _empty(q.shape, torch.bfloat16, q.device, stream)
        if accumulate and lse is None:
            import torch
            lse = _empty((q.shape[0], self.q_heads), torch.float32, q.device, stream)
        if lse is not None and lse.numel() != q.shape[0] * self.q_heads:
            raise ValueError("lse must be rows x q_heads")
        scale = self.head_dim ** -0.5 if scale is None else scale
        gsi_kv_attention(self.kv, q, row_start, length, max_rows, scale, out, lse, accumulate,
                         stream)
        return out

    def evict(self, length, budget: int, recent: int, spare_table, length_out=None, stream=None):
        length_out = length if length_out is None else length_out
        if _current_device() != self._device:
            self._elsewhere()
        self._ints(length, self.seqs, "length")
        self._ints(length_out, self.seqs, "length_out")
        self._ints(spare_table, self.page_table.numel(), "spare_table")
        gsi_kv_evict(self.kv, length, budget, recent, spare_table, length_out, stream)
        return length_out

    def status(self, stream=None) -> int:
        return gsi_kv_status(self.kv, stream)

    def close(self):
        if self.kv is not None:
            gsi_kv_destroy(self.kv)
            self.kv = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
