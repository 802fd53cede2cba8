"""Same-device collective primitives for MI355X: Python binding of include/dt.h.

Every function here only marshals torch tensors into the C ABI of
libdtcoll.so (device pointers, element counts, dtype and op codes, the HIP
stream handle) and raises ``DtError`` on a non-OK status.  All data movement
runs in the library's HIP kernels; PyTorch supplies device memory and
streams.  There is no fallback path: if the library is missing, import fails.

Names follow the C ABI (``dt_allreduce`` ...).  Rank r's buffer is element r
of a list of tensors on the same GPU.  Calls are queued on ``stream``
(default: torch's current stream) and return before the GPU runs them.
With ``async_op=True`` the call follows the async mode of the c10d page
(arganzheng.life, "PyTorch communication stack", sec. 4.3-4.4): it is queued
on a side stream that first waits for the current stream, and the returned
``Work`` keeps the tensors alive until ``wait()`` makes the consumer stream
wait for the end event.
"""
from __future__ import annotations

import atexit
import ctypes
import threading
import types
import weakref
from typing import Dict, List, Optional, Sequence

import torch

from . import _lib

_L = _lib.load()


def _load_marshal():
    """The host helper of the model-step operators' binding, or a stand-in that
    says why they cannot be called: the collectives do without it."""
    try:
        from . import _marshal as helper
        if helper.torch_version == str(torch.__version__):
            return helper
        why = f"it was built for torch {helper.torch_version}, this is {torch.__version__}"
    except ImportError as e:
        why = str(e)

    def missing(*_):
        raise ImportError(f"the binding's helper _marshal is missing ({why}); run `python collective_communication_primitives_amd/build.py`")

    return types.SimpleNamespace(buffers=missing, counts=missing)


_marshal = _load_marshal()

DT_FLOAT32, DT_BFLOAT16, DT_INT32 = 0, 1, 2
DT_SUM, DT_MAX, DT_MIN, DT_AVG = 0, 1, 2, 3
DT_OK, DT_ERR_ARG, DT_ERR_UNSUPPORTED, DT_ERR_HIP, DT_ERR_TIMEOUT = 0, 1, 2, 3, 4
DT_MAX_RANKS = 16
DEFAULT_BUCKET_BYTES = 25 << 20
SCRATCH_BYTES = 256 << 20  # DT_SCRATCH_BYTES: the static staging buffer of dt_bucket_allreduce_noalloc

_DTYPES = {torch.float32: DT_FLOAT32, torch.bfloat16: DT_BFLOAT16, torch.int32: DT_INT32}
_OPS = {"sum": DT_SUM, "max": DT_MAX, "min": DT_MIN, "avg": DT_AVG}

LIBRARY_PATH = _lib.LIBRARY


class DtError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} ({status})")
        self.status = status


def _check(status: int) -> None:
    if status != DT_OK:
        detail = _L.dt_last_error().decode() or _L.dt_status_string(status).decode()
        raise DtError(status, detail)


def status_string(status: int) -> str:
    return _L.dt_status_string(int(status)).decode()


def version() -> str:
    return _L.dt_version().decode()


def _ptr_array(tensors: Sequence[torch.Tensor]):
    return (ctypes.c_void_p * max(1, len(tensors)))(*[t.data_ptr() for t in tensors])


def _size_array(values: Sequence[int]):
    return (ctypes.c_size_t * max(1, len(values)))(*[int(v) for v in values])


def _dtype_code(tensors: Sequence[torch.Tensor]) -> int:
    """The tensors' common dtype code, after checking that every tensor is a
    contiguous tensor of that dtype on the current GPU (a host or
    other-device pointer must never reach a kernel)."""
    t0 = tensors[0]
    dt = t0.dtype
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.dtype != dt:
            raise TypeError("all rank tensors must share one dtype")
        if t.get_device() != dev:
            raise ValueError(f"rank tensors must live on the current GPU (cuda:{dev}), got {t.device}")
        if not t.is_contiguous():
            raise ValueError("rank tensors must be contiguous")
    return _DTYPES[dt]


def _on_gpu(tensors: Sequence[torch.Tensor], what: str) -> None:
    """Every tensor must be a contiguous tensor on the current GPU."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous tensors on the current GPU (cuda:{dev}), got {t.device}")


def _check_windows(windows: Sequence[torch.Tensor], status: torch.Tensor, p: int) -> None:
    for w in windows:
        if w.dtype != torch.int32 or w.numel() < p:
            raise ValueError("each window must be an int32 tensor of at least nranks cells")
    if status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 device tensor")
    _on_gpu(list(windows) + [status], "windows and status")


def _op_code(op) -> int:
    return _OPS[op] if isinstance(op, str) else int(op)


if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
    def _current_stream_handle() -> int:
        # the raw handle without building a torch Stream object (about 2 us less per call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
else:  # other torch builds: the public accessor
    def _current_stream_handle() -> int:
        return torch.cuda.current_stream().cuda_stream


def _stream_handle(stream) -> int:
    if stream is None:
        return _current_stream_handle()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _as_stream(handle: int, dev: int) -> torch.cuda.Stream:
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


_side_streams: Dict[int, torch.cuda.Stream] = {}


def side_stream(device: Optional[int] = None) -> torch.cuda.Stream:
    """The library's default communication stream for a device (default priority)."""
    dev = torch.cuda.current_device() if device is None else device
    if dev not in _side_streams:
        _side_streams[dev] = torch.cuda.Stream(device=dev)
    return _side_streams[dev]


def join_streams(producers: Sequence[torch.cuda.Stream], stream=None) -> None:
    """User rule 4 of the c10d page (sec. 5): inputs computed on streams other
    than the current one must be joined into it before the collective is
    issued, because an async collective orders itself after the current
    stream only.  Makes ``stream`` (default: current) wait for everything
    queued so far on each producer stream; the host does not block."""
    target = torch.cuda.current_stream() if stream is None else stream
    for p in producers:
        if p is not None and p != target:
            target.wait_stream(p)


class Work:
    """Handle of an async collective: the start/end event pair plus the stash
    of tensors that must outlive the GPU work (released by ``wait``)."""

    def __init__(self, handle: ctypes.c_void_p, stash: List[torch.Tensor]):
        self._h = handle
        self._stash = stash
        self._lib = _L
        _live_works.add(self)

    def wait(self, stream=None) -> None:
        """Make ``stream`` (default: current) wait for the end event; the host does not block."""
        _check(self._lib.dt_work_wait(self._h, _stream_handle(stream)))
        self._stash = []

    def is_completed(self) -> bool:
        rc = self._lib.dt_work_query(self._h)
        if rc < 0:
            raise DtError(DT_ERR_HIP, _L.dt_last_error().decode())
        return rc == 1

    def _release(self) -> None:
        """Free the handle now (at exit): wait for the work first if its
        tensors are still held, so they are not released under it."""
        h = getattr(self, "_h", None)
        if h:
            if getattr(self, "_stash", None):
                torch.cuda.synchronize()
            self._lib.dt_work_free(h)
            self._h = None
            self._stash = []

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            if getattr(self, "_stash", None) and _shelf is not None:
                # dropped without wait(): shelve the tensors until the GPU is done
                _shelf.append((h, self._stash))
            else:
                self._lib.dt_work_free(h)
            self._h = None
            self._stash = []


# Works dropped without wait(): (handle, tensors).  As in the c10d page
# (sec. 4.4), a forgotten wait() leaks nothing but may not free the tensors
# while the collective can still touch them: they stay here until the work's
# end event has completed, and are released by the next collective call.
_shelf: List = []

# Every object of this module that owns HIP handles, so that _release_all
# can free them before the interpreter (and with it the HIP runtime and any
# profiler attached to it) shuts down.
_live_works: "weakref.WeakSet[Work]" = weakref.WeakSet()
_live_pipelines: "weakref.WeakSet[HSDPPipeline]" = weakref.WeakSet()


def _release_all() -> None:
    """Free every HIP event the binding still owns, deterministically, while
    the runtime is whole: live HSDP pipelines (their destroy waits for the
    work they queued), live and shelved works.  Registered with atexit at
    import; afterwards no destructor of this module calls into HIP.  The
    tensors a work or pipeline kept alive are dropped only after its handle
    has been released (the c10d page, sec. 5: a stash outlives its GPU work)."""
    for pipe in list(_live_pipelines):
        pipe.close()
    for work in list(_live_works):
        work._release()
    if _shelf:
        torch.cuda.synchronize()  # the shelved tensors may still be in use on the GPU
        for h, _stash in _shelf:
            _L.dt_work_free(h)
        _shelf.clear()


atexit.register(_release_all)


def _unshelve() -> None:
    keep = []
    for h, stash in _shelf:
        if _L.dt_work_query(h) == 0:
            keep.append((h, stash))
        else:
            _L.dt_work_free(h)
    _shelf[:] = keep


# prepare() runs a collective's validation and marshalling once and keeps the
# resulting launch instead of enqueuing it.
_preparing = threading.local()


class Prepared:
    """One collective bound to fixed buffers, counts, dtype and op (made by
    ``prepare``).  Each call enqueues it again on ``stream`` (default: the
    current stream) at the host cost of the C call alone: the pointer arrays
    and checks were done once.  The buffers stay referenced while this object
    lives; their contents may change between calls.  A graph that captured a
    call needs this object for as long as it is replayed, and calls on several
    streams at once need a prepared call each: they share its buffers."""

    def __init__(self, fn, stash: List[torch.Tensor], space: Optional["_Space"] = None):
        self._fn = fn
        self._stash = stash
        self._space = space

    def __call__(self, stream=None) -> None:
        handle = _stream_handle(stream)
        if self._space is not None:
            self._space.used_on(handle)
        _check(self._fn(handle))


class _Space:
    """The workspace that prepare() made for a call: torch's allocator hands it
    out in the order of one stream, so another stream that runs the call first
    waits for that order and is recorded as a user of the memory."""

    def __init__(self, tensor: torch.Tensor, home: int):
        self._tensor = tensor
        self._seen = {home}
        self._ready = torch.cuda.Event()
        self._ready.record(_as_stream(home, tensor.device.index))

    def used_on(self, handle: int) -> None:
        if handle in self._seen or torch.cuda.is_current_stream_capturing():
            return  # a capture begins behind all work of the device
        stream = _as_stream(handle, self._tensor.device.index)
        stream.wait_event(self._ready)
        self._tensor.record_stream(stream)
        self._seen.add(handle)


def prepare(collective, *args, **kwargs) -> Prepared:
    """Validate and marshal one call of ``collective`` (``dt_allreduce``,
    ``dt_reduce_scatter``, ...; same arguments, without ``async_op``) once,
    for loops that repeat the same collective on the same buffers."""
    if kwargs.get("async_op"):
        raise ValueError("prepare() binds a synchronous call; order it with streams and events")
    _preparing.active = True
    _preparing.result = None
    _preparing.space = None
    try:
        collective(*args, **kwargs)
        if _preparing.result is None:
            raise TypeError(f"{collective!r} does not enqueue a collective")
        fn, stash = _preparing.result
        space = _preparing.space
    finally:
        _preparing.active = False
        _preparing.result = None
        _preparing.space = None
    return Prepared(fn, stash, space)


def _launch(fn, stash, async_op: bool, stream, comm_stream):
    """Queue ``fn(stream_handle)`` either on ``stream`` or, for async_op, on a
    side stream ordered after the current stream."""
    if getattr(_preparing, "active", False):
        _preparing.result = (fn, list(stash))
        return None
    if _shelf:
        _unshelve()
    if not async_op:
        _check(fn(_stream_handle(stream)))
        return None
    producer = _stream_handle(stream)
    comm = _stream_handle(comm_stream if comm_stream is not None else side_stream())
    h = ctypes.c_void_p()
    _check(_L.dt_work_begin(producer, comm, ctypes.byref(h)))
    work = Work(h, list(stash))
    _check(fn(comm))
    _check(_L.dt_work_end(h, comm))
    return work


# ----------------------------------------------------------- collectives --
def dt_allreduce(send: Sequence[torch.Tensor], recv: Optional[Sequence[torch.Tensor]] = None, op="sum",
                 stream=None, async_op: bool = False, comm_stream=None):
    """AllReduce: recv[q] = fold over ranks of send[r] (in place when recv is None)."""
    recv = list(send) if recv is None else list(recv)
    n = send[0].numel()
    if any(t.numel() != n for t in list(send) + recv) or len(recv) != len(send):
        raise ValueError("every rank's send and recv must have the same number of elements")
    code = _dtype_code(list(send) + recv)
    s, r = _ptr_array(send), _ptr_array(recv)
    w = _launch(lambda st: _L.dt_allreduce(s, r, len(send), n, code, _op_code(op), st), list(send) + recv,
                async_op, stream, comm_stream)
    return w if async_op else recv


def dt_reduce_scatter(send: Sequence[torch.Tensor], recv: Sequence[torch.Tensor], op="sum", stream=None,
                      async_op: bool = False, comm_stream=None):
    """ReduceScatter: recv[r] = chunk r of the fold; send[r] holds P * recv[r].numel() elements."""
    p = len(send)
    m = recv[0].numel()
    if len(recv) != p or any(t.numel() != p * m for t in send) or any(t.numel() != m for t in recv):
        raise ValueError("send[r] must hold nranks * recvcount elements and recv[r] recvcount")
    code = _dtype_code(list(send) + list(recv))
    s, r = _ptr_array(send), _ptr_array(recv)
    w = _launch(lambda st: _L.dt_reduce_scatter(s, r, p, m, code, _op_code(op), st), list(send) + list(recv),
                async_op, stream, comm_stream)
    return w if async_op else list(recv)


def dt_all_gather(send: Sequence[torch.Tensor], recv: Sequence[torch.Tensor], stream=None,
                  async_op: bool = False, comm_stream=None):
    """AllGather (equal or uneven Shard(0)): recv[q] = concat(send[0], ..., send[P-1])."""
    p = len(send)
    counts = [t.numel() for t in send]
    total = sum(counts)
    if len(recv) != p or any(t.numel() != total for t in recv):
        raise ValueError("every recv must hold the sum of the send counts")
    code = _dtype_code(list(send) + list(recv))
    s, r = _ptr_array(send), _ptr_array(recv)
    equal = all(c == counts[0] for c in counts)
    c_arr = None if equal else _size_array(counts)
    w = _launch(lambda st: _L.dt_all_gather(s, r, p, c_arr, counts[0] if equal else 0, code, st),
                list(send) + list(recv), async_op, stream, comm_stream)
    return w if async_op else list(recv)


def dt_all_to_all(send: Sequence[torch.Tensor], recv: Sequence[torch.Tensor], splits, stream=None,
                  async_op: bool = False, comm_stream=None):
    """AllToAll with splits[i][j] elements from rank i to rank j (row-major P x P)."""
    p = len(send)
    flat = [int(v) for row in splits for v in row] if hasattr(splits[0], "__len__") else [int(v) for v in splits]
    if len(flat) != p * p:
        raise ValueError("splits must be P x P")
    for i in range(p):
        if send[i].numel() != sum(flat[i * p:(i + 1) * p]):
            raise ValueError(f"send[{i}] must hold the sum of row {i} of splits")
        if recv[i].numel() != sum(flat[j * p + i] for j in range(p)):
            raise ValueError(f"recv[{i}] must hold the sum of column {i} of splits")
    code = _dtype_code(list(send) + list(recv))
    s, r, sp = _ptr_array(send), _ptr_array(recv), _size_array(flat)
    w = _launch(lambda st: _L.dt_all_to_all(s, r, p, sp, code, st), list(send) + list(recv), async_op, stream,
                comm_stream)
    return w if async_op else list(recv)


def dt_all_gather_into_vec(send: Sequence[torch.Tensor], recv: Sequence[Sequence[torch.Tensor]], stream=None,
                           async_op: bool = False, comm_stream=None):
    """AllGatherIntoVec: recv[q][r] receives a copy of send[r] for every rank q."""
    p = len(send)
    if len(recv) != p or any(len(row) != p for row in recv):
        raise ValueError("recv must be P lists of P tensors")
    for q in range(p):
        for r in range(p):
            if recv[q][r].numel() != send[r].numel():
                raise ValueError(f"recv[{q}][{r}] must hold send[{r}].numel() elements")
    flat = [t for row in recv for t in row]
    code = _dtype_code(list(send) + flat)
    counts = [t.numel() for t in send]
    s, r, c = _ptr_array(send), _ptr_array(flat), _size_array(counts)
    w = _launch(lambda st: _L.dt_all_gather_into_vec(s, r, p, c, 0, code, st), list(send) + flat, async_op,
                stream, comm_stream)
    return w if async_op else recv


def dt_broadcast(root_send: torch.Tensor, recv: Sequence[torch.Tensor], stream=None, async_op: bool = False,
                 comm_stream=None):
    """Broadcast: every recv[q] receives a copy of root_send."""
    n = root_send.numel()
    if any(t.numel() != n for t in recv):
        raise ValueError("every recv must hold root_send.numel() elements")
    code = _dtype_code([root_send] + list(recv))
    r = _ptr_array(recv)
    w = _launch(lambda st: _L.dt_broadcast(root_send.data_ptr(), r, len(recv), n, code, st),
                [root_send] + list(recv), async_op, stream, comm_stream)
    return w if async_op else list(recv)


def dt_replicate_to_shard(send: Sequence[torch.Tensor], recv: Sequence[torch.Tensor], stream=None,
                          async_op: bool = False, comm_stream=None):
    """ReplicateToShard: recv[r] = slice r of send[r] (send[r] holds P * recv[r].numel())."""
    p = len(send)
    m = recv[0].numel()
    if len(recv) != p or any(t.numel() != p * m for t in send) or any(t.numel() != m for t in recv):
        raise ValueError("send[r] must hold nranks * recvcount elements and recv[r] recvcount")
    code = _dtype_code(list(send) + list(recv))
    s, r = _ptr_array(send), _ptr_array(recv)
    w = _launch(lambda st: _L.dt_replicate_to_shard(s, r, p, m, code, st), list(send) + list(recv), async_op,
                stream, comm_stream)
    return w if async_op else list(recv)


def dt_all_to_all_dims(send: Sequence[torch.Tensor], recv: Sequence[torch.Tensor], rows: int, cols: int,
                       src_dim: int, dst_dim: int, stream=None, async_op: bool = False, comm_stream=None):
    """AllToAll between shard dimensions of a [rows, cols] tensor: send[r] is
    rank r's block under Shard(src_dim), recv[r] its block under Shard(dst_dim)."""
    p = len(send)
    blk = {0: (rows // p) * cols, 1: rows * (cols // p)}
    if len(recv) != p or any(t.numel() != blk[src_dim] for t in send) or any(t.numel() != blk[dst_dim] for t in recv):
        raise ValueError("send/recv blocks do not match the [rows, cols] shard shapes")
    code = _dtype_code(list(send) + list(recv))
    s, r = _ptr_array(send), _ptr_array(recv)
    w = _launch(lambda st: _L.dt_all_to_all_dims(s, r, p, rows, cols, src_dim, dst_dim, code, st),
                list(send) + list(recv), async_op, stream, comm_stream)
    return w if async_op else list(recv)


def dt_bucket_allreduce(grads: Sequence[Sequence[torch.Tensor]], bucket_bytes: int = DEFAULT_BUCKET_BYTES,
                        bucket_ws: Optional[Sequence[torch.Tensor]] = None, op="sum", stream=None,
                        async_op: bool = False, comm_stream=None):
    """Fused-bucket AllReduce in place over grads[r][t] (rank r, tensor t).

    With ``bucket_ws`` (one device buffer of >= bucket_bytes per rank) each
    bucket is staged through it; without, buckets are reduced in place."""
    p, nt = len(grads), len(grads[0])
    numels = [g.numel() for g in grads[0]]
    for rank in grads:
        if len(rank) != nt or [g.numel() for g in rank] != numels:
            raise ValueError("every rank must list tensors of the same sizes")
    flat = [g for rank in grads for g in rank]
    code = _dtype_code(flat)
    if bucket_ws is not None:
        if len(bucket_ws) != p or any(w.numel() * w.element_size() < bucket_bytes for w in bucket_ws):
            raise ValueError("bucket_ws needs one buffer of at least bucket_bytes per rank")
        _on_gpu(bucket_ws, "bucket_ws")
    g_arr, n_arr = _ptr_array(flat), _size_array(numels)
    ws_arr = _ptr_array(bucket_ws) if bucket_ws is not None else None
    stash = flat + (list(bucket_ws) if bucket_ws is not None else [])
    w = _launch(lambda st: _L.dt_bucket_allreduce(g_arr, n_arr, nt, p, bucket_bytes, ws_arr, code, _op_code(op), st),
                stash, async_op, stream, comm_stream)
    return w if async_op else grads


def dt_bucket_allreduce_noalloc(grads: Sequence[Sequence[torch.Tensor]], bucket_bytes: int = DEFAULT_BUCKET_BYTES,
                                op="sum", stream=None, async_op: bool = False, comm_stream=None):
    """Staged fused-bucket AllReduce in place over grads[r][t], with the
    buckets staged in the library's static device buffer (SCRATCH_BYTES)
    instead of caller workspaces: nothing is allocated.  nranks *
    bucket_bytes must fit that buffer.  Calls that may overlap in time on one
    GPU share the buffer and must be ordered by the caller."""
    p, nt = len(grads), len(grads[0])
    numels = [g.numel() for g in grads[0]]
    for rank in grads:
        if len(rank) != nt or [g.numel() for g in rank] != numels:
            raise ValueError("every rank must list tensors of the same sizes")
    flat = [g for rank in grads for g in rank]
    code = _dtype_code(flat)
    g_arr, n_arr = _ptr_array(flat), _size_array(numels)
    w = _launch(lambda st: _L.dt_bucket_allreduce_noalloc(g_arr, n_arr, nt, p, bucket_bytes, code, _op_code(op), st),
                flat, async_op, stream, comm_stream)
    return w if async_op else grads


def dt_allreduce_coalesced(tensors: Sequence[Sequence[torch.Tensor]], op="sum", stream=None, async_op: bool = False,
                           comm_stream=None):
    """Coalesced in-place AllReduce of tensors[r][t] (rank r, tensor t): one
    launch for up to min(512, 4096 // P) tensors, no flattening."""
    p, nt = len(tensors), len(tensors[0])
    numels = [g.numel() for g in tensors[0]]
    for rank in tensors:
        if len(rank) != nt or [g.numel() for g in rank] != numels:
            raise ValueError("every rank must list tensors of the same sizes")
    flat = [g for rank in tensors for g in rank]
    code = _dtype_code(flat)
    g_arr, n_arr = _ptr_array(flat), _size_array(numels)
    w = _launch(lambda st: _L.dt_allreduce_coalesced(g_arr, n_arr, nt, p, code, _op_code(op), st), flat, async_op,
                stream, comm_stream)
    return w if async_op else tensors


def dt_bucket_plan(numels: Sequence[int], elem_size: int, bucket_bytes: int = DEFAULT_BUCKET_BYTES):
    """Host-side bucket plan: (pieces, nbuckets); each piece is a dict."""
    n_arr = _size_array(numels)
    npieces, nbuckets = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_L.dt_bucket_plan(n_arr, len(numels), elem_size, bucket_bytes, None, 0, ctypes.byref(npieces),
                             ctypes.byref(nbuckets)))
    buf = (_lib.DtPiece * max(1, npieces.value))()
    _check(_L.dt_bucket_plan(n_arr, len(numels), elem_size, bucket_bytes, buf, npieces.value,
                             ctypes.byref(npieces), ctypes.byref(nbuckets)))
    pieces = [dict(tensor=buf[i].tensor, bucket=buf[i].bucket, offset=buf[i].offset, length=buf[i].length,
                   bucket_pos=buf[i].bucket_pos) for i in range(npieces.value)]
    return pieces, nbuckets.value


# ------------------------------------------------------------------ barrier --
DT_BARRIER_PACKED, DT_BARRIER_SPREAD = 0, 1
_LAYOUTS = {"packed": DT_BARRIER_PACKED, "spread": DT_BARRIER_SPREAD}


def dt_barrier(windows: Sequence[torch.Tensor], status: torch.Tensor, first_generation: int, generations: int = 1,
               timeout_ns: int = 0, layout="packed", stream=None) -> None:
    """Signal-window barrier over int32 windows[p] (nranks cells each);
    layout "packed" (one workgroup, a wave per rank) or "spread" (a
    workgroup per rank, cooperative launch)."""
    p = len(windows)
    _check_windows(windows, status, p)
    w_arr = _ptr_array(windows)
    _check(_L.dt_barrier(w_arr, p, first_generation, generations, status.data_ptr(), timeout_ns, _LAYOUTS[layout],
                         _stream_handle(stream)))


def dt_barrier_exchange(src: Sequence[torch.Tensor], stage: Sequence[torch.Tensor], dst: Sequence[torch.Tensor],
                        windows: Sequence[torch.Tensor], status: torch.Tensor, generation: int, timeout_ns: int = 0,
                        layout="packed", stream=None) -> None:
    """Stage src[r], meet the barrier, then dst[r] = stage[(r+1) % P]."""
    p = len(src)
    nbytes = src[0].numel() * src[0].element_size()
    for group in (src, stage, dst):
        if len(group) != p or any(t.numel() * t.element_size() != nbytes for t in group):
            raise ValueError("src, stage and dst need one contiguous buffer of equal bytes per rank")
        _on_gpu(group, "src, stage and dst")
    if len(windows) != p:
        raise ValueError("one window per rank")
    _check_windows(windows, status, p)
    _check(_L.dt_barrier_exchange(_ptr_array(src), _ptr_array(stage), _ptr_array(dst), nbytes, _ptr_array(windows),
                                  p, generation, status.data_ptr(), timeout_ns, _LAYOUTS[layout],
                                  _stream_handle(stream)))


# -------------------------------------------------------------- HSDP -------
class HSDPPipeline:
    """Per-layer ReduceScatter -> fused AllReduce pipeline (dt_hsdp_*).

    The two phases may run on two streams (the page's layout: the
    AllReduce of layer L-1 never blocks the ReduceScatter of layer L) or on
    one.  With every rank on one device both phases draw on the same HBM, and
    issuing them back to back on one stream, in the same order, measured 4%
    faster (30.5 vs 31.8 ms for the 32-layer workload), so one side stream
    for both is the default; pass two streams for the split layout, or the
    stream that produces the gradients as both, for a pipeline without
    cross-stream events (its collectives then queue behind the producer's
    work, in order).

    A layer's fused buffers must not be passed again (as the next layer's)
    before ``finish()``: the previous layer's AllReduce is still pending on
    them, and the library refuses the overlap."""

    def __init__(self, replicate: int, shard: int, bucket_bytes: int = DEFAULT_BUCKET_BYTES,
                 dtype=torch.bfloat16, op="sum", rs_stream=None, ar_stream=None):
        self.replicate, self.shard = replicate, shard
        if rs_stream is None and ar_stream is None:
            rs_stream = ar_stream = torch.cuda.Stream()
        self.rs_stream = rs_stream if rs_stream is not None else torch.cuda.Stream()
        self.ar_stream = ar_stream if ar_stream is not None else torch.cuda.Stream()
        self._h = ctypes.c_void_p()
        self._stash: List[torch.Tensor] = []
        self._lib = _L
        _check(_L.dt_hsdp_create(replicate, shard, bucket_bytes, _DTYPES[dtype], _op_code(op),
                                 _stream_handle(self.rs_stream), _stream_handle(self.ar_stream),
                                 ctypes.byref(self._h)))
        _live_pipelines.add(self)

    def post_backward(self, grads: Sequence[Sequence[torch.Tensor]], fused: Sequence[torch.Tensor],
                      producer=None) -> None:
        """grads[r][t]: rank r's full gradients of one layer; fused[r]: its
        flat shard buffer (sum(numel)/shard elements)."""
        p = self.replicate * self.shard
        nt = len(grads[0])
        numels = [g.numel() for g in grads[0]]
        flat = [g for rank in grads for g in rank]
        _dtype_code(flat + list(fused))
        if len(grads) != p or len(fused) != p:
            raise ValueError("one gradient list and one fused buffer per rank")
        if any(f.numel() != sum(numels) // self.shard for f in fused):
            raise ValueError("fused[r] must hold sum(numels) / shard elements")
        self._stash.extend(flat + list(fused))
        _check(self._lib.dt_hsdp_post_backward(self._h, _ptr_array(flat), _size_array(numels), nt, _ptr_array(fused),
                                        _stream_handle(producer)))

    def finish(self, consumer=None) -> None:
        _check(self._lib.dt_hsdp_finish(self._h, _stream_handle(consumer)))
        self._stash = []

    def close(self) -> None:
        """Release the handle: the library waits for the work it queued to
        stop writing the buffers, then the buffers are let go.  A layer
        posted without finish() gets no AllReduce."""
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.dt_hsdp_destroy(h)
        self._h = None
        self._stash = []

    def __del__(self):
        self.close()


def shard_views(fused: torch.Tensor, numels: Sequence[int], shard: int) -> List[torch.Tensor]:
    """Each parameter's reduced shard as a view of a fused buffer (the page's
    get_param_grad_view): no copy."""
    out, at = [], 0
    for n in numels:
        m = n // shard
        out.append(fused[at:at + m])
        at += m
    return out


# ----------------------------------------------- model-step operators ------
# Layer norm, expert routing, the experts' token exchange and the loss over a
# sharded vocabulary: the steps of a model whose mathematics crosses the ranks.
DT_MAX_EXPERTS, DT_MAX_TOPK = 1024, 64
_SCORES = {"softmax": 0, "sigmoid": 1}


def _refuse(name: str, tensors, sizes, dtype, dev: int) -> None:
    """Say which tensor of a list the call cannot take, and why."""
    if not isinstance(tensors, (list, tuple)):
        raise TypeError(f"{name} must be a list of tensors, got {type(tensors).__name__}")
    if len(tensors) != len(sizes):
        raise ValueError(f"{name} must list one tensor per rank ({len(sizes)}), got {len(tensors)}")
    for r, (t, want) in enumerate(zip(tensors, sizes)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{r}] must be a tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise TypeError(f"{name}[{r}] must be {dtype}, got {t.dtype}")
        if t.numel() != want:
            raise ValueError(f"{name}[{r}] must hold {want} elements, got {t.numel()}")
        if t.get_device() != dev:
            raise ValueError(f"{name}[{r}] must live on the current GPU (cuda:{dev}), got {t.device}")
    raise ValueError(f"{name} must list contiguous tensors")


def _buffers(name: str, tensors, sizes, dtype, dev: int, stash: list):
    """The pointers of a list of contiguous tensors of ``dtype`` on the current
    GPU, rank r's with sizes[r] elements; the tensors join ``stash``."""
    ptrs = _marshal.buffers(tensors, sizes, dtype, dev, stash)
    if ptrs is None:
        _refuse(name, tensors, sizes, dtype, dev)
    return ptrs


def _ranks(tensors, name: str) -> int:
    p = len(tensors)
    if not 1 <= p <= DT_MAX_RANKS:
        raise ValueError(f"{name} must list 1 to {DT_MAX_RANKS} ranks' tensors, got {p}")
    return p


def _row_counts(tensors, cols: int, name: str, times: int = 1):
    """(elements, rows, rows * times, rows as the C ABI takes them) of each
    tensor, whole rows of ``cols``."""
    counts = _marshal.counts(tensors, cols, times)
    if counts is None:
        raise ValueError(f"{name} must be a list of tensors of whole rows of {cols} elements")
    return counts


def _float_dtype(t: torch.Tensor) -> int:
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _workspace(given: Optional[torch.Tensor], nbytes: int, dev: int, stream, async_op: bool, comm_stream,
               stash: list) -> torch.Tensor:
    """The call's workspace: the caller's, or a block of torch's caching
    allocator, taken in the order of the stream that runs the call.  (An async
    call's stream waits for the producer, whose order serves as well.)"""
    if given is not None:
        _on_gpu([given], "workspace")
        if given.numel() * given.element_size() < nbytes:
            raise ValueError(f"workspace must hold {nbytes} bytes, got {given.numel() * given.element_size()}")
        stash.append(given)
        return given
    home = _stream_handle(stream)
    if home == _current_stream_handle():
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    else:
        with torch.cuda.stream(_as_stream(home, dev)):
            ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    if getattr(_preparing, "active", False):
        _preparing.space = _Space(ws, home)
    if async_op:
        ws.record_stream(_as_stream(_stream_handle(comm_stream if comm_stream is not None else side_stream(dev)), dev))
    stash.append(ws)
    return ws


def _sized(nbytes: int) -> int:
    """The result of a *_workspace function: 0 with an error message means refused."""
    if nbytes == 0:
        detail = _L.dt_last_error().decode()
        if detail:
            raise DtError(DT_ERR_ARG, detail)
    return nbytes


def _width(t: torch.Tensor, name: str) -> int:
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must have a last dimension of at least one element")
    return t.shape[-1]


def dt_layer_norm_workspace(rows: Sequence[int], cols: int) -> int:
    """Bytes of workspace dt_layer_norm_backward takes for rows[r] rows of ``cols`` per rank."""
    return _sized(_L.dt_layer_norm_workspace(len(rows), _size_array(rows), cols))


def dt_layer_norm(x: Sequence[torch.Tensor], weight: Sequence[torch.Tensor], bias: Optional[Sequence[torch.Tensor]],
                  y: Sequence[torch.Tensor], mean: Optional[Sequence[torch.Tensor]] = None,
                  rstd: Optional[Sequence[torch.Tensor]] = None, eps: float = 1e-5, stream=None,
                  async_op: bool = False, comm_stream=None):
    """Layer norm of every rank's rows x[r] [..., cols] into y[r]; weight[r],
    bias[r] (None: no bias) hold ``cols`` elements.  mean[r], rstd[r] (fp32,
    one per row) keep the statistics for dt_layer_norm_backward."""
    p, dev, cols = _ranks(x, "x"), torch.cuda.current_device(), _width(weight[0], "weight")
    code, dtype, stash = _float_dtype(x[0]), x[0].dtype, []
    sizes, rows, _, n = _row_counts(x, cols, "x")
    if (mean is None) != (rstd is None):
        raise ValueError("mean and rstd come together")
    xs, ys = _buffers("x", x, sizes, dtype, dev, stash), _buffers("y", y, sizes, dtype, dev, stash)
    ws = _buffers("weight", weight, [cols] * p, dtype, dev, stash)
    bs = _buffers("bias", bias, [cols] * p, dtype, dev, stash) if bias is not None else None
    ms = rs = None
    if mean is not None:
        ms, rs = _buffers("mean", mean, rows, torch.float32, dev, stash), _buffers("rstd", rstd, rows, torch.float32, dev, stash)
    w = _launch(lambda st: _L.dt_layer_norm(xs, ws, bs, ys, ms, rs, p, n, cols, eps, code, st), stash, async_op, stream,
                comm_stream)
    return w if async_op else y


def dt_layer_norm_backward(dy: Sequence[torch.Tensor], x: Sequence[torch.Tensor], weight: Sequence[torch.Tensor],
                           mean: Sequence[torch.Tensor], rstd: Sequence[torch.Tensor], dx: Sequence[torch.Tensor],
                           dweight: Sequence[torch.Tensor], dbias: Optional[Sequence[torch.Tensor]] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None, async_op: bool = False,
                           comm_stream=None):
    """Gradients of dt_layer_norm: dx[r], and dweight[q], dbias[q] (None: not
    formed) summed over the rows of all ranks, for every rank q."""
    p, dev, cols = _ranks(x, "x"), torch.cuda.current_device(), _width(weight[0], "weight")
    code, dtype, stash = _float_dtype(x[0]), x[0].dtype, []
    sizes, rows, _, n = _row_counts(x, cols, "x")
    wide = [cols] * p
    xs, gs = _buffers("x", x, sizes, dtype, dev, stash), _buffers("dy", dy, sizes, dtype, dev, stash)
    ds, ws = _buffers("dx", dx, sizes, dtype, dev, stash), _buffers("weight", weight, wide, dtype, dev, stash)
    ms, rs = _buffers("mean", mean, rows, torch.float32, dev, stash), _buffers("rstd", rstd, rows, torch.float32, dev, stash)
    dw = _buffers("dweight", dweight, wide, dtype, dev, stash)
    db = _buffers("dbias", dbias, wide, dtype, dev, stash) if dbias is not None else None
    space = _workspace(workspace, _sized(_L.dt_layer_norm_workspace(p, n, cols)), dev, stream, async_op, comm_stream, stash)
    at, have = space.data_ptr(), space.numel() * space.element_size()
    w = _launch(lambda st: _L.dt_layer_norm_backward(gs, xs, ws, ms, rs, ds, dw, db, p, n, cols, code, at, have, st), stash,
                async_op, stream, comm_stream)
    return w if async_op else dx


def _score_code(score) -> int:
    return _SCORES[score] if isinstance(score, str) else int(score)


def dt_moe_route(logits: Sequence[torch.Tensor], experts: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                 bias: Optional[torch.Tensor] = None, groups: int = 1, topk_groups: int = 1, score="softmax",
                 renormalize: bool = True, scale: float = 1.0, stream=None, async_op: bool = False, comm_stream=None):
    """Routing: experts[r] int32 and weights[r] fp32 [tokens, topk] from
    logits[r] [tokens, nexperts]; see dt.h for the order and what -inf, NaN
    and ties do.  ``bias`` (fp32 [nexperts]) moves the choice, not the weights."""
    p, dev = _ranks(logits, "logits"), torch.cuda.current_device()
    e, k, stash = _width(logits[0], "logits"), _width(experts[0], "experts"), []
    code, dtype = _float_dtype(logits[0]), logits[0].dtype
    sizes, _, slots, n = _row_counts(logits, e, "logits", k)
    ls, es = _buffers("logits", logits, sizes, dtype, dev, stash), _buffers("experts", experts, slots, torch.int32, dev, stash)
    ws = _buffers("weights", weights, slots, torch.float32, dev, stash)
    b = None
    if bias is not None:
        _buffers("bias", [bias], [e], torch.float32, dev, stash)
        b = bias.data_ptr()
    sc, rn = _score_code(score), int(bool(renormalize))
    w = _launch(lambda st: _L.dt_moe_route(ls, es, ws, p, n, e, k, b, groups, topk_groups, sc, rn, scale, code, st),
                stash, async_op, stream, comm_stream)
    return w if async_op else (experts, weights)


def dt_moe_route_backward(logits: Sequence[torch.Tensor], experts: Sequence[torch.Tensor],
                          dweights: Sequence[torch.Tensor], dlogits: Sequence[torch.Tensor], score="softmax",
                          renormalize: bool = True, scale: float = 1.0, stream=None, async_op: bool = False,
                          comm_stream=None):
    """dlogits[r] from the gradient of dt_moe_route's weights, for its choice."""
    p, dev = _ranks(logits, "logits"), torch.cuda.current_device()
    e, k, stash = _width(logits[0], "logits"), _width(experts[0], "experts"), []
    code, dtype = _float_dtype(logits[0]), logits[0].dtype
    sizes, _, slots, n = _row_counts(logits, e, "logits", k)
    ls, ds = _buffers("logits", logits, sizes, dtype, dev, stash), _buffers("dlogits", dlogits, sizes, dtype, dev, stash)
    es, gs = _buffers("experts", experts, slots, torch.int32, dev, stash), _buffers("dweights", dweights, slots, torch.float32, dev, stash)
    sc, rn = _score_code(score), int(bool(renormalize))
    w = _launch(lambda st: _L.dt_moe_route_backward(ls, es, gs, ds, p, n, e, k, sc, rn, scale, code, st), stash, async_op,
                stream, comm_stream)
    return w if async_op else dlogits


def dt_moe_dispatch_workspace(tokens: Sequence[int], nexperts: int, topk: int) -> int:
    """Bytes of workspace dt_moe_dispatch takes."""
    return _sized(_L.dt_moe_dispatch_workspace(len(tokens), _size_array(tokens), nexperts, topk))


def _exchange(tok, rows, experts, nexperts: int):
    """(p, cols, topk, token elements, slots, tokens, expert row elements, capacity)
    of an exchange between token tensors and the experts' row buffers."""
    p = _ranks(tok, "tokens")
    cols, k = _width(tok[0], "the rows"), _width(experts[0], "experts")
    if nexperts % p:
        raise ValueError(f"{nexperts} experts do not divide by {p} ranks")
    sizes, _, slots, n = _row_counts(tok, cols, "the token tensors", k)
    held, _, _, cap = _row_counts(rows, cols, "the experts' buffers")
    if len(rows) != p:
        raise ValueError(f"the experts' buffers must list one tensor per rank ({p}), got {len(rows)}")
    return p, cols, k, sizes, slots, n, held, cap


def dt_moe_dispatch(x: Sequence[torch.Tensor], experts: Sequence[torch.Tensor], recv: Sequence[torch.Tensor],
                    positions: Sequence[torch.Tensor], offsets: Sequence[torch.Tensor], nexperts: int,
                    workspace: Optional[torch.Tensor] = None, stream=None, async_op: bool = False, comm_stream=None):
    """AllToAll of token rows x[r] [tokens, cols] to the ranks of their
    experts[r] [tokens, topk]: recv[q] [capacity, cols] in expert order,
    positions[r] int32 [tokens, topk] (-1: no row), offsets[q] int32
    [nexperts / P + 1]."""
    dev, dtype, stash, i32 = torch.cuda.current_device(), x[0].dtype, [], torch.int32
    p, cols, k, sizes, slots, n, held, cap = _exchange(x, recv, experts, nexperts)
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    code = _DTYPES[dtype]
    xs, rs = _buffers("x", x, sizes, dtype, dev, stash), _buffers("recv", recv, held, dtype, dev, stash)
    es, ps = _buffers("experts", experts, slots, i32, dev, stash), _buffers("positions", positions, slots, i32, dev, stash)
    fs = _buffers("offsets", offsets, [nexperts // p + 1] * p, i32, dev, stash)
    space = _workspace(workspace, _sized(_L.dt_moe_dispatch_workspace(p, n, nexperts, k)), dev, stream, async_op, comm_stream, stash)
    at, have = space.data_ptr(), space.numel() * space.element_size()
    w = _launch(lambda st: _L.dt_moe_dispatch(xs, es, rs, ps, fs, p, n, cap, cols, nexperts, k, code, at, have, st), stash,
                async_op, stream, comm_stream)
    return w if async_op else recv


def dt_moe_combine(y: Sequence[torch.Tensor], experts: Sequence[torch.Tensor], positions: Sequence[torch.Tensor],
                   weights: Optional[Sequence[torch.Tensor]], out: Sequence[torch.Tensor], nexperts: int, stream=None,
                   async_op: bool = False, comm_stream=None):
    """out[r][t] = sum over its slots of weight * y[owner][position]
    (weights None: all ones, dt_moe_dispatch's backward pass)."""
    dev, dtype, stash, i32 = torch.cuda.current_device(), out[0].dtype, [], torch.int32
    p, cols, k, sizes, slots, n, held, cap = _exchange(out, y, experts, nexperts)
    code = _float_dtype(out[0])
    ys, outs = _buffers("y", y, held, dtype, dev, stash), _buffers("out", out, sizes, dtype, dev, stash)
    es, ps = _buffers("experts", experts, slots, i32, dev, stash), _buffers("positions", positions, slots, i32, dev, stash)
    ws = _buffers("weights", weights, slots, torch.float32, dev, stash) if weights is not None else None
    w = _launch(lambda st: _L.dt_moe_combine(ys, es, ps, ws, outs, p, n, cap, cols, nexperts, k, code, st), stash, async_op,
                stream, comm_stream)
    return w if async_op else out


def dt_moe_combine_backward(dout: Sequence[torch.Tensor], y: Sequence[torch.Tensor], experts: Sequence[torch.Tensor],
                            positions: Sequence[torch.Tensor], weights: Sequence[torch.Tensor],
                            dy: Sequence[torch.Tensor], dweights: Sequence[torch.Tensor], nexperts: int, stream=None,
                            async_op: bool = False, comm_stream=None):
    """Gradients of dt_moe_combine: dy[owner][position] = weight * dout[r][t]
    (other rows of dy are left as they were), dweights[r] fp32."""
    dev, dtype, stash, i32, f32 = torch.cuda.current_device(), dout[0].dtype, [], torch.int32, torch.float32
    p, cols, k, sizes, slots, n, held, cap = _exchange(dout, y, experts, nexperts)
    code = _float_dtype(dout[0])
    gs, ys = _buffers("dout", dout, sizes, dtype, dev, stash), _buffers("y", y, held, dtype, dev, stash)
    es, ps = _buffers("experts", experts, slots, i32, dev, stash), _buffers("positions", positions, slots, i32, dev, stash)
    ws, ds = _buffers("weights", weights, slots, f32, dev, stash), _buffers("dy", dy, held, dtype, dev, stash)
    dw = _buffers("dweights", dweights, slots, f32, dev, stash)
    w = _launch(lambda st: _L.dt_moe_combine_backward(gs, ys, es, ps, ws, ds, dw, p, n, cap, cols, nexperts, k, code, st),
                stash, async_op, stream, comm_stream)
    return w if async_op else dy


def dt_vocab_loss_workspace(vocab_rows: Sequence[int], tokens: int, cols: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace dt_vocab_loss takes."""
    return _sized(_L.dt_vocab_loss_workspace(len(vocab_rows), _size_array(vocab_rows), tokens, cols, _DTYPES[dtype]))


def dt_vocab_loss_backward_workspace(vocab_rows: Sequence[int], tokens: int, cols: int, dtype=torch.bfloat16,
                                     piece_rows: int = 0) -> int:
    """Bytes of workspace dt_vocab_loss_backward takes with pieces of ``piece_rows`` vocabulary rows (0: the library's choice)."""
    return _sized(_L.dt_vocab_loss_backward_workspace(len(vocab_rows), _size_array(vocab_rows), tokens, cols, piece_rows,
                                                      _DTYPES[dtype]))


def _loss_inputs(hidden, weight, targets, dev: int, stash: list):
    p, cols = _ranks(hidden, "hidden"), _width(hidden[0], "hidden")
    code, dtype, tokens = _float_dtype(hidden[0]), hidden[0].dtype, hidden[0].numel() // cols
    held, _, _, n = _row_counts(weight, cols, "weight")
    hs = _buffers("hidden", hidden, [tokens * cols] * p, dtype, dev, stash)
    if len(weight) != p:
        raise ValueError(f"weight must list one tensor per rank ({p}), got {len(weight)}")
    ws = _buffers("weight", weight, held, dtype, dev, stash)
    ts = _buffers("targets", targets, [tokens] * p, torch.int64, dev, stash)
    return p, cols, tokens, code, dtype, held, n, hs, ws, ts


def dt_vocab_loss(hidden: Sequence[torch.Tensor], weight: Sequence[torch.Tensor], targets: Sequence[torch.Tensor],
                  loss: Sequence[torch.Tensor], lse: Sequence[torch.Tensor], ignore_index: int = -100,
                  workspace: Optional[torch.Tensor] = None, stream=None, async_op: bool = False, comm_stream=None):
    """Softmax cross entropy per token over a vocabulary sharded over the
    ranks: hidden[r] [tokens, cols] (the same on every rank; one tensor may be
    listed P times), weight[r] [rows of rank r, cols], targets[r] int64.
    loss[q] and lse[q] fp32 [tokens] are written for every rank."""
    dev, stash = torch.cuda.current_device(), []
    p, cols, tokens, code, dtype, _, n, hs, ws, ts = _loss_inputs(hidden, weight, targets, dev, stash)
    each = [tokens] * p
    ls, es = _buffers("loss", loss, each, torch.float32, dev, stash), _buffers("lse", lse, each, torch.float32, dev, stash)
    space = _workspace(workspace, _sized(_L.dt_vocab_loss_workspace(p, n, tokens, cols, code)), dev, stream, async_op, comm_stream,
                       stash)
    at, have = space.data_ptr(), space.numel() * space.element_size()
    w = _launch(lambda st: _L.dt_vocab_loss(hs, ws, ts, ls, es, p, n, tokens, cols, ignore_index, code, at, have, st), stash,
                async_op, stream, comm_stream)
    return w if async_op else loss


def dt_vocab_loss_backward(hidden: Sequence[torch.Tensor], weight: Sequence[torch.Tensor],
                           targets: Sequence[torch.Tensor], lse: Sequence[torch.Tensor], dloss: Sequence[torch.Tensor],
                           dhidden: Sequence[torch.Tensor], dweight: Sequence[torch.Tensor], ignore_index: int = -100,
                           piece_rows: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                           async_op: bool = False, comm_stream=None):
    """Gradients of dt_vocab_loss for dloss[r] fp32 [tokens]: dhidden[q] is
    the sum over all ranks' shards for every rank q, dweight[r] rank r's own.
    The logits are formed again, ``piece_rows`` vocabulary rows at a time (0:
    the library's choice); the workspace grows with the piece."""
    dev, stash = torch.cuda.current_device(), []
    p, cols, tokens, code, dtype, held, n, hs, ws, ts = _loss_inputs(hidden, weight, targets, dev, stash)
    each = [tokens] * p
    es, gs = _buffers("lse", lse, each, torch.float32, dev, stash), _buffers("dloss", dloss, each, torch.float32, dev, stash)
    dh = _buffers("dhidden", dhidden, [tokens * cols] * p, dtype, dev, stash)
    dw = _buffers("dweight", dweight, held, dtype, dev, stash)
    space = _workspace(workspace, _sized(_L.dt_vocab_loss_backward_workspace(p, n, tokens, cols, piece_rows, code)), dev, stream,
                       async_op, comm_stream, stash)
    at, have = space.data_ptr(), space.numel() * space.element_size()
    w = _launch(lambda st: _L.dt_vocab_loss_backward(hs, ws, ts, es, gs, dh, dw, p, n, tokens, cols, ignore_index, piece_rows,
                                                     code, at, have, st), stash, async_op, stream, comm_stream)
    return w if async_op else dhidden


__all__ = [
    "dt_allreduce", "dt_reduce_scatter", "dt_all_gather", "dt_all_to_all", "dt_bucket_allreduce", "dt_bucket_plan",
    "dt_all_gather_into_vec", "dt_broadcast", "dt_replicate_to_shard", "dt_all_to_all_dims",
    "dt_allreduce_coalesced", "dt_bucket_allreduce_noalloc", "dt_barrier", "dt_barrier_exchange", "HSDPPipeline", "Work", "DtError", "shard_views", "side_stream",
    "status_string", "version",
    "dt_layer_norm", "dt_layer_norm_backward", "dt_layer_norm_workspace", "dt_moe_route", "dt_moe_route_backward",
    "dt_moe_dispatch", "dt_moe_dispatch_workspace", "dt_moe_combine", "dt_moe_combine_backward", "dt_vocab_loss",
    "dt_vocab_loss_backward", "dt_vocab_loss_workspace", "dt_vocab_loss_backward_workspace",
]
