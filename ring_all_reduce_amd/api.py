"""Python binding of librar.so: one function per C entry point, same names.

Argument marshalling only -- every step of the all-reduce runs in the HIP
library.  Device buffers may be given as torch tensors (contiguous, on the
GPU, of the plan's element type: float32 for RAR_F32 and for weights,
bfloat16 for RAR_BF16, with at least as many elements as the call touches;
ValueError otherwise) or as integer device addresses, which are passed on
unchecked.  ``stream`` may be a torch stream, an
integer hipStream_t, or None for torch's current stream on the current
device (the default stream when torch has no GPU).

The operators on matrices (rar_embed_*, rar_linear_*, rar_ckpt_*) take 2-D
tensors whose rows are contiguous; the distance between rows is the leading
dimension.  An integer address stands for a contiguous matrix.  Their tensors
must be on the current device.  ``ws`` is a uint8 tensor of at least the
queried bytes, or None: then one is allocated for the call, and returned to
torch's allocator in the order of the call's stream.

Status codes other than RAR_OK raise RarError carrying the code.
"""
from __future__ import annotations

import ctypes
from typing import Sequence

from ._lib import lib

# enums of rar.h
F32, BF16 = 0, 1
BALANCED, CEIL, ALIGN16 = 0, 1, 2
FUSED, RING, NAIVE = 0, 1, 2
OK, EINVAL, EMISMATCH, EALIGN, ENOMEM, EHIP, ETOOLARGE = 0, -1, -2, -3, -4, -5, -6
MAX_RANKS = 64
MAX_STRIDE_CANDIDATES = 64
STATIC_WS_ELEMS = 1 << 24
ACT_NONE, ACT_RELU, ACT_GELU = 0, 1, 2
CKPT_GROUP = 32


class RarError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {rar_strerror(status)} ({status})")


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise RarError(rc, where)


def rar_strerror(status: int) -> str:
    return lib().rar_strerror(int(status)).decode()


def rar_version() -> int:
    return int(lib().rar_version())


def _addr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensor must be contiguous")
        if x.numel() and not x.is_cuda:
            raise ValueError("tensor must be on the GPU")
        return int(x.data_ptr())
    raise TypeError(f"not a device buffer: {type(x)!r}")


def _ptr_array(xs: Sequence) -> ctypes.Array:
    arr = (ctypes.c_void_p * max(len(xs), 1))()
    for i, x in enumerate(xs):
        arr[i] = _addr(x) or None
    return arr


def _ranks(xs: Sequence, N: int, what: str) -> ctypes.Array:
    # the library reads exactly N pointers from the array
    if len(xs) != N:
        raise ValueError(f"{what}: {len(xs)} entries for {N} ranks")
    return _ptr_array(xs)


_DTYPES = {}


def _torch_dtype(dtype: int):
    if dtype not in _DTYPES:
        import torch
        _DTYPES[dtype] = torch.float32 if dtype == F32 else torch.bfloat16
    return _DTYPES[dtype]


def _check_tensor(x, what: str, dtype: int, min_numel: int) -> None:
    """A tensor argument must have the element type the library will read and
    write through it, and at least as many elements as it will touch (the
    library sees only an address).  Integer addresses are taken as given."""
    if x is None or isinstance(x, int) or not hasattr(x, "data_ptr"):
        return
    want = _torch_dtype(dtype)
    if x.dtype != want:
        raise ValueError(f"{what}: dtype {x.dtype}, expected {want}")
    if x.numel() < min_numel:
        raise ValueError(f"{what}: {x.numel()} elements, at least {min_numel} needed")


def _check_ranks(xs: Sequence, what: str, dtype: int, min_numel: int) -> None:
    for n, x in enumerate(xs):
        if hasattr(x, "data_ptr") and (x.dtype != _torch_dtype(dtype) or x.numel() < min_numel):
            _check_tensor(x, f"{what}[{n}]", dtype, min_numel)  # raises, with the argument's name


def _stream(s) -> int:
    if s is None:
        try:
            import torch
            if torch.cuda.is_available():
                return int(torch.cuda.current_stream().cuda_stream)
        except ImportError:
            pass
        return 0
    if isinstance(s, int):
        return s
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    raise TypeError(f"not a stream: {type(s)!r}")


# ---------------------------------------------------------------------------
# Plans
# ---------------------------------------------------------------------------

class Plan:
    """Owner of a rar_plan_t; destroyed with the object or by rar_plan_destroy."""

    def __init__(self, handle: int, N: int, P: int, dtype: int, chunking: int):
        self.handle = ctypes.c_void_p(handle)
        self.N, self.P, self.dtype, self.chunking = N, P, dtype, chunking

    def __del__(self):
        try:
            rar_plan_destroy(self)
        except Exception:
            pass


def rar_plan(N: int, P: int, dtype: int = F32, chunking: int = BALANCED) -> Plan:
    out = ctypes.c_void_p()
    _check(lib().rar_plan(int(N), int(P), int(dtype), int(chunking), ctypes.byref(out)), "rar_plan")
    return Plan(out.value, int(N), int(P), int(dtype), int(chunking))


def rar_rank_stride(P: int, dtype: int = F32) -> int:
    """Recommended byte distance between rank buffers carved from one allocation."""
    out = ctypes.c_int64()
    _check(lib().rar_rank_stride(int(P), int(dtype), ctypes.byref(out)), "rar_rank_stride")
    return out.value


def rar_rank_stride_candidate(P: int, dtype: int, k: int) -> int:
    """Candidate k of the strides rar_rank_stride_tune times (for sizing its pool)."""
    out = ctypes.c_int64()
    _check(lib().rar_rank_stride_candidate(int(P), int(dtype), int(k), ctypes.byref(out)),
           "rar_rank_stride_candidate")
    return out.value


def rar_rank_stride_tune(N: int, P: int, dtype: int, pool, candidates: int = 64, stream=None) -> int:
    """Measured byte distance between rank buffers carved from `pool` (a
    device tensor or pointer; its contents are overwritten).  Waits for the
    stream."""
    out = ctypes.c_int64()
    nbytes = pool.numel() * pool.element_size() if hasattr(pool, "element_size") else None
    if nbytes is None:
        raise TypeError("pool must be a tensor (its size bounds the candidates)")
    _check(lib().rar_rank_stride_tune(int(N), int(P), int(dtype), _addr(pool), int(nbytes), int(candidates),
                                      _stream(stream), ctypes.byref(out)), "rar_rank_stride_tune")
    return out.value


def rar_rank_stride_tune_stats(N: int, P: int, dtype: int, pool, candidates: int = 64, stream=None):
    """rar_rank_stride_tune and its measurements: (stride, [(candidate stride,
    median ms, spread ms), ...])."""
    if not hasattr(pool, "element_size"):
        raise TypeError("pool must be a tensor (its size bounds the candidates)")
    nbytes = pool.numel() * pool.element_size()
    out, K = ctypes.c_int64(), ctypes.c_int()
    cs = (ctypes.c_int64 * candidates)()
    med, spr = (ctypes.c_float * candidates)(), (ctypes.c_float * candidates)()
    _check(lib().rar_rank_stride_tune_stats(int(N), int(P), int(dtype), _addr(pool), int(nbytes), int(candidates),
                                            _stream(stream), ctypes.byref(out), ctypes.byref(K), cs, med, spr),
           "rar_rank_stride_tune_stats")
    return out.value, [(cs[k], med[k], spr[k]) for k in range(K.value)]


def rar_plan_destroy(plan: Plan) -> None:
    if plan.handle:
        h, plan.handle = plan.handle, ctypes.c_void_p()
        _check(lib().rar_plan_destroy(h), "rar_plan_destroy")


def rar_plan_set_algo(plan: Plan, algo: int) -> None:
    _check(lib().rar_plan_set_algo(plan.handle, int(algo)), "rar_plan_set_algo")


def rar_plan_set_grid(plan: Plan, max_blocks: int) -> None:
    _check(lib().rar_plan_set_grid(plan.handle, int(max_blocks)), "rar_plan_set_grid")


def rar_plan_chunk(plan: Plan, c: int):
    off, ln, own = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
    _check(lib().rar_plan_chunk(plan.handle, int(c), ctypes.byref(off), ctypes.byref(ln), ctypes.byref(own)),
           "rar_plan_chunk")
    return off.value, ln.value, own.value


def rar_plan_traffic(plan: Plan, rank: int):
    s, r = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().rar_plan_traffic(plan.handle, int(rank), ctypes.byref(s), ctypes.byref(r)), "rar_plan_traffic")
    return s.value, r.value


# ---------------------------------------------------------------------------
# All-reduce
# ---------------------------------------------------------------------------

def _check_exec(plan: Plan, bufs: Sequence, P: int) -> None:
    # a P that differs from the plan's is the library's RAR_EMISMATCH, raised
    # before it touches any buffer
    if int(P) == plan.P:
        _check_ranks(bufs, "bufs", plan.dtype, plan.P)


def _check_weights(w, what: str, plan: Plan, P: int) -> None:
    if int(P) == plan.P:
        _check_tensor(w, what, F32, plan.P)


def rar_allreduce_mean(plan: Plan, bufs: Sequence, P: int, stream=None) -> None:
    _check_exec(plan, bufs, P)
    _check(lib().rar_allreduce_mean(plan.handle, _ranks(bufs, plan.N, "bufs"), int(P), _stream(stream)),
           "rar_allreduce_mean")


def rar_allreduce_sgd(plan: Plan, bufs: Sequence, w, lr: float, P: int, stream=None) -> None:
    _check_exec(plan, bufs, P)
    _check_weights(w, "w", plan, P)
    _check(lib().rar_allreduce_sgd(plan.handle, _ranks(bufs, plan.N, "bufs"), _addr(w), ctypes.c_float(lr), int(P),
                                   _stream(stream)), "rar_allreduce_sgd")


def rar_allreduce_ring_noalloc(plan: Plan, bufs: Sequence, w, lr: float, P: int, stream=None) -> None:
    """The ring all-reduce-mean (w None) or + SGD with no device allocation:
    a bf16 plan's partial sums use the library's static workspace."""
    _check_exec(plan, bufs, P)
    if w is not None:
        _check_weights(w, "w", plan, P)
    _check(lib().rar_allreduce_ring_noalloc(plan.handle, _ranks(bufs, plan.N, "bufs"), _addr(w),
                                            ctypes.c_float(lr), int(P), _stream(stream)),
           "rar_allreduce_ring_noalloc")


def rar_reduce_scatter_sgd_allgather(plan: Plan, bufs: Sequence, w_reps: Sequence, lr: float, P: int,
                                     stream=None) -> None:
    _check_exec(plan, bufs, P)
    for n, w in enumerate(w_reps):
        _check_weights(w, f"w_reps[{n}]", plan, P)
    _check(lib().rar_reduce_scatter_sgd_allgather(plan.handle, _ranks(bufs, plan.N, "bufs"),
                                                  _ranks(w_reps, plan.N, "w_reps"),
                                                  ctypes.c_float(lr), int(P), _stream(stream)),
           "rar_reduce_scatter_sgd_allgather")


# ---------------------------------------------------------------------------
# Buckets
# ---------------------------------------------------------------------------

class Buckets:
    def __init__(self, handle: int, numel: Sequence[int], dtype: int):
        self.handle = ctypes.c_void_p(handle)
        self.numel = [int(n) for n in numel]
        self.n_tensors, self.dtype, self.total = len(self.numel), dtype, sum(self.numel)

    def __del__(self):
        try:
            rar_bucket_destroy(self)
        except Exception:
            pass


def rar_bucket_plan(numel: Sequence[int], dtype: int = F32, bucket_bytes: int = 25_000_000) -> Buckets:
    arr = (ctypes.c_int64 * max(len(numel), 1))(*[int(n) for n in numel])
    out = ctypes.c_void_p()
    _check(lib().rar_bucket_plan(len(numel), arr, int(dtype), int(bucket_bytes), ctypes.byref(out)),
           "rar_bucket_plan")
    return Buckets(out.value, numel, int(dtype))


def rar_bucket_destroy(b: Buckets) -> None:
    if b.handle:
        h, b.handle = b.handle, ctypes.c_void_p()
        _check(lib().rar_bucket_destroy(h), "rar_bucket_destroy")


def rar_bucket_count(b: Buckets):
    n, m = ctypes.c_int(), ctypes.c_int64()
    _check(lib().rar_bucket_count(b.handle, ctypes.byref(n), ctypes.byref(m)), "rar_bucket_count")
    return n.value, m.value


def rar_bucket_info(b: Buckets, bucket: int):
    so, el, ns = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
    _check(lib().rar_bucket_info(b.handle, int(bucket), ctypes.byref(so), ctypes.byref(el), ctypes.byref(ns)),
           "rar_bucket_info")
    return so.value, el.value, ns.value


def rar_bucket_segment(b: Buckets, bucket: int, seg: int):
    t, to, bo, ln = ctypes.c_int(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().rar_bucket_segment(b.handle, int(bucket), int(seg), ctypes.byref(t), ctypes.byref(to),
                                    ctypes.byref(bo), ctypes.byref(ln)), "rar_bucket_segment")
    return t.value, to.value, bo.value, ln.value


def _rank_major(b: "Buckets", tensors: Sequence[Sequence]) -> ctypes.Array:
    # the library reads N * n_tensors pointers: every rank must list them all
    want, numel = _torch_dtype(b.dtype), b.numel
    for n, rank in enumerate(tensors):
        if len(rank) != b.n_tensors:
            raise ValueError(f"rank {n} lists {len(rank)} tensors; the bucket plan has {b.n_tensors}")
        for t, x in enumerate(rank):
            # the common case costs two comparisons; the message is built only on failure
            if hasattr(x, "data_ptr") and (x.dtype != want or x.numel() < numel[t]):
                _check_tensor(x, f"tensors[{n}][{t}]", b.dtype, numel[t])
    flat = [x for rank in tensors for x in rank]
    return _ptr_array(flat)


def _check_bucket_bufs(b: Buckets, bucket_bufs: Sequence, elems: int) -> None:
    _check_ranks(bucket_bufs, "bucket_bufs", b.dtype, elems)


def _bucket_elems(b: Buckets, bucket: int) -> int:
    # a bad bucket index is the library's RAR_EINVAL
    nb = rar_bucket_count(b)[0] if b.handle else 0
    return rar_bucket_info(b, bucket)[1] if 0 <= int(bucket) < nb else 0


def rar_bucket_pack(b: Buckets, bucket: int, tensors: Sequence[Sequence], bucket_bufs: Sequence,
                    stream=None) -> None:
    _check_bucket_bufs(b, bucket_bufs, _bucket_elems(b, bucket))
    _check(lib().rar_bucket_pack(b.handle, int(bucket), len(tensors), _rank_major(b, tensors),
                                 _ranks(bucket_bufs, len(tensors), "bucket_bufs"), _stream(stream)),
           "rar_bucket_pack")


def rar_bucket_unpack(b: Buckets, bucket: int, bucket_bufs: Sequence, tensors: Sequence[Sequence],
                      stream=None) -> None:
    _check_bucket_bufs(b, bucket_bufs, _bucket_elems(b, bucket))
    _check(lib().rar_bucket_unpack(b.handle, int(bucket), len(tensors),
                                   _ranks(bucket_bufs, len(tensors), "bucket_bufs"),
                                   _rank_major(b, tensors), _stream(stream)), "rar_bucket_unpack")


def rar_bucket_allreduce_mean(b: Buckets, tensors: Sequence[Sequence], bucket_bufs=None,
                              chunking: int = BALANCED, algo: int = FUSED, stream=None) -> None:
    """bucket_bufs: N buffers of max_bucket_elems, or None when the reduction
    runs straight from the tensors: RAR_ALGO_FUSED at a supported rank count,
    RAR_ALGO_RING on binary32 at N >= 2, and RAR_ALGO_RING on bf16 when every
    rank's tensors lie end to end in one buffer (see rar.h)."""
    if bucket_bufs is not None and b.handle:
        _check_bucket_bufs(b, bucket_bufs, rar_bucket_count(b)[1])
    bufs = None if bucket_bufs is None else _ranks(bucket_bufs, len(tensors), "bucket_bufs")
    _check(lib().rar_bucket_allreduce_mean(b.handle, len(tensors), int(chunking), int(algo),
                                           _rank_major(b, tensors), bufs, _stream(stream)),
           "rar_bucket_allreduce_mean")


def rar_bucket_allreduce_arena(b: Buckets, arenas: Sequence, ready_events=None, chunking: int = BALANCED,
                               algo: int = FUSED, stream=None) -> None:
    """ready_events: None, or one entry per bucket: a torch.cuda.Event, an
    integer hipEvent_t, or None (no wait)."""
    _check_ranks(arenas, "arenas", b.dtype, b.total)
    ev = None
    if ready_events is not None:
        nb = rar_bucket_count(b)[0]
        if len(ready_events) != nb:
            raise ValueError(f"{len(ready_events)} ready events for {nb} buckets")
        ev = (ctypes.c_void_p * max(len(ready_events), 1))()
        for i, e in enumerate(ready_events):
            ev[i] = None if e is None else (e if isinstance(e, int) else int(e.cuda_event)) or None
    _check(lib().rar_bucket_allreduce_arena(b.handle, len(arenas), int(chunking), int(algo), _ptr_array(arenas),
                                            ev, _stream(stream)), "rar_bucket_allreduce_arena")


# ---------------------------------------------------------------------------
# Producers of the gradients: embedding, linear layer, 8-bit checkpoints
# ---------------------------------------------------------------------------

_get_device = None


def _here() -> int:
    """The current device's index, -1 without a GPU."""
    global _get_device
    if _get_device is None:
        import torch
        if not torch.cuda.is_available():
            return -1
        torch.cuda.init()
        # the call behind current_device(), where torch has it
        _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _get_device()


def _on(stream) -> int:
    """The call's stream; torch's current one, where torch has it, costs a tenth of building its Stream object."""
    if stream is None:
        dev = _here()
        if dev >= 0:
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            if raw is not None:
                return raw(dev)
    return _stream(stream)


def _device_of(x, what: str) -> None:
    dev = x.get_device()
    if dev < 0:
        if x.numel():
            raise ValueError(f"{what}: tensor must be on the GPU")
    elif dev != _here():
        raise ValueError(f"{what}: tensor is on {x.device}, the current device is cuda:{_here()}")


def _plain(x) -> bool:
    return x.is_cuda and x.is_contiguous() and x.get_device() == _here()


def _matrix(x, what: str, tdtype, rows: int, cols: int):
    """(address, leading dimension) of a rows x cols matrix argument."""
    if getattr(x, "dtype", None) is tdtype and rows > 0 and x.shape == (rows, cols) and _plain(x):
        return x.data_ptr(), cols  # the usual case; what follows finds out what is wrong with others
    if x is None:
        return 0, cols
    if isinstance(x, int):
        return x, cols
    if not hasattr(x, "data_ptr"):
        raise TypeError(f"{what}: not a device buffer: {type(x)!r}")
    if x.dtype is not tdtype:
        raise ValueError(f"{what}: dtype {x.dtype}, expected {tdtype}")
    if x.shape != (rows, cols):
        raise ValueError(f"{what}: shape {tuple(x.shape)}, expected ({rows}, {cols})")
    if rows == 0:
        return 0, cols
    ld, step = x.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    if rows == 1:
        ld = cols  # the stride of a single row says nothing
    elif ld < cols:
        raise ValueError(f"{what}: rows overlap (stride {ld} for {cols} columns)")
    _device_of(x, what)
    return x.data_ptr(), ld


def _dense(x, what: str, tdtype, numel: int) -> int:
    """Address of a contiguous argument of exactly numel elements."""
    if getattr(x, "dtype", None) is tdtype and x.numel() == numel and _plain(x):
        return x.data_ptr()
    if x is None or isinstance(x, int):
        return x or 0
    if not hasattr(x, "data_ptr"):
        raise TypeError(f"{what}: not a device buffer: {type(x)!r}")
    if x.dtype is not tdtype:
        raise ValueError(f"{what}: dtype {x.dtype}, expected {tdtype}")
    if x.numel() != numel:
        raise ValueError(f"{what}: {x.numel()} elements, expected {numel}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    _device_of(x, what)
    return x.data_ptr()


def _workspace(ws, nbytes: int, stream):
    """(address, bytes, owner) of the call's workspace."""
    if ws is not None:
        if not hasattr(ws, "element_size"):
            raise TypeError("ws must be a tensor (its size is checked)")
        return _dense(ws, "ws", ws.dtype, ws.numel()), ws.numel() * ws.element_size(), ws
    if nbytes == 0:
        return 0, 0, None
    import torch
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    if stream is not None:
        s = stream
        if isinstance(stream, int):
            s = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        if s.cuda_stream != torch.cuda.current_stream().cuda_stream:
            # the allocator may hand the memory out again only once this stream has used it, and this
            # stream may use it only once its last user on the current stream is done
            s.wait_stream(torch.cuda.current_stream())
            t.record_stream(s)
    return t.data_ptr(), nbytes, t


def rar_embed_lookup(V: int, D: int, dtype: int, table, T: int, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]]; rows of ids outside 0..V-1 are zero."""
    import torch
    V, D, T, scale = int(V), int(D), int(T), float(scale)
    td = _torch_dtype(dtype)
    ptr, ldo = _matrix(out, "out", td, T, D)
    _check(lib().rar_embed_lookup(V, D, dtype, _dense(table, "table", td, V * D), T,
                                  _dense(ids, "ids", torch.int64, T), scale, ptr, ldo, _on(stream)),
           "rar_embed_lookup")


def rar_embed_grad_workspace(V: int, D: int, T: int) -> int:
    out = ctypes.c_int64()
    _check(lib().rar_embed_grad_workspace(int(V), int(D), int(T), ctypes.byref(out)), "rar_embed_grad_workspace")
    return out.value


def rar_embed_grad(V: int, D: int, dtype: int, T: int, ids, dy, grad, scale: float = 1.0, accumulate: bool = False,
                   ws=None, stream=None) -> None:
    """grad[v] (+)= scale * the sum of dy[t] over the t with ids[t] == v."""
    import torch
    V, D, T, scale = int(V), int(D), int(T), float(scale)
    td = _torch_dtype(dtype)
    dptr, lddy = _matrix(dy, "dy", td, T, D)
    gptr, iptr = _dense(grad, "grad", td, V * D), _dense(ids, "ids", torch.int64, T)
    wptr, wbytes, _own = _workspace(ws, 0 if ws is not None else rar_embed_grad_workspace(V, D, T), stream)
    _check(lib().rar_embed_grad(V, D, dtype, T, iptr, dptr, lddy, scale, int(bool(accumulate)), gptr, wptr, wbytes,
                                _on(stream)), "rar_embed_grad")


class Linear:
    """Owner of a rar_linear_t; destroyed with the object or by rar_linear_destroy."""

    def __init__(self, handle: int, K: int, N: int, dtype: int, act: int):
        self.handle = ctypes.c_void_p(handle)
        self.K, self.N, self.dtype, self.act = K, N, dtype, act
        self._bytes = {}

    def __del__(self):
        try:
            rar_linear_destroy(self)
        except Exception:
            pass


def rar_linear_plan(K: int, N: int, dtype: int = F32, act: int = ACT_NONE) -> Linear:
    out = ctypes.c_void_p()
    _check(lib().rar_linear_plan(int(K), int(N), int(dtype), int(act), ctypes.byref(out)), "rar_linear_plan")
    return Linear(out.value, int(K), int(N), int(dtype), int(act))


def rar_linear_destroy(plan: Linear) -> None:
    if plan.handle:
        h, plan.handle = plan.handle, ctypes.c_void_p()
        _check(lib().rar_linear_destroy(h), "rar_linear_destroy")


def rar_linear_workspace(plan: Linear, T: int):
    """(forward bytes, backward bytes) for T rows."""
    T = int(T)
    known = plan._bytes.get(T)
    if known is not None and plan.handle:
        return known
    f, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().rar_linear_workspace(plan.handle, T, ctypes.byref(f), ctypes.byref(b)), "rar_linear_workspace")
    if len(plan._bytes) < 64:  # a layer's plan serves a few batch sizes
        plan._bytes[T] = f.value, b.value
    return f.value, b.value


def _kept(x, scales, what: str, td, T: int, cols: int):
    """(address, leading dimension, scales' address) of a matrix or its 8-bit checkpoint."""
    if scales is None:
        return (*_matrix(x, what, td, T, cols), 0)
    import torch
    groups = -(-cols // CKPT_GROUP)
    return (_dense(x, what, torch.uint8, T * groups * CKPT_GROUP), cols,
            _dense(scales, f"{what}_scales", torch.uint8, T * groups))


def rar_linear_forward(plan: Linear, T: int, x, w, bias, residual, y, pre=None, pre_scales=None, ws=None,
                       stream=None) -> None:
    """z = x w + bias, y = act(z) + residual; bias and residual may be None.
    pre receives z, as an 8-bit checkpoint when pre_scales is given."""
    T = int(T)
    td, K, N = _torch_dtype(plan.dtype), plan.K, plan.N
    xp, ldx = _matrix(x, "x", td, T, K)
    wp, bp = _dense(w, "w", td, K * N), _dense(bias, "bias", td, N)
    rp, ldr = _matrix(residual, "residual", td, T, N)
    yp, ldy = _matrix(y, "y", td, T, N)
    pp, ldp, sp = _kept(pre, pre_scales, "pre", td, T, N)
    wsp, wsb, _own = _workspace(ws, 0 if ws is not None else rar_linear_workspace(plan, T)[0], stream)
    _check(lib().rar_linear_forward(plan.handle, T, xp, ldx, wp, bp, rp, ldr, yp, ldy, pp, ldp, sp, wsp, wsb,
                                    _on(stream)), "rar_linear_forward")


def rar_linear_backward(plan: Linear, T: int, dy, x, w, pre, dx, dw, db, x_scales=None, pre_scales=None,
                        accumulate: bool = False, ws=None, stream=None) -> None:
    """dz = dy act'(z); dx = dz w^T, dw (+)= x^T dz, db (+)= column sums of dz.
    dx, dw and db may each be None; x and pre may be 8-bit checkpoints."""
    T = int(T)
    td, K, N = _torch_dtype(plan.dtype), plan.K, plan.N
    dyp, lddy = _matrix(dy, "dy", td, T, N)
    xp, ldx, xs = _kept(x, x_scales, "x", td, T, K)
    wp = _dense(w, "w", td, K * N)
    pp, ldp, ps = _kept(pre, pre_scales, "pre", td, T, N) if plan.act != ACT_NONE else (0, N, 0)
    dxp, lddx = _matrix(dx, "dx", td, T, K)
    dwp, dbp = _dense(dw, "dw", td, K * N), _dense(db, "db", td, N)
    wsp, wsb, _own = _workspace(ws, 0 if ws is not None else rar_linear_workspace(plan, T)[1], stream)
    _check(lib().rar_linear_backward(plan.handle, T, dyp, lddy, xp, ldx, xs, wp, pp, ldp, ps, dxp, lddx, dwp, dbp,
                                     int(bool(accumulate)), wsp, wsb, _on(stream)), "rar_linear_backward")


def rar_ckpt_size(D: int):
    """(bytes of a row of codes, bytes of a row of scales) of an 8-bit checkpoint of D columns."""
    p, g = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().rar_ckpt_size(int(D), ctypes.byref(p), ctypes.byref(g)), "rar_ckpt_size")
    return p.value, g.value


def rar_ckpt_store(T: int, D: int, dtype: int, x, codes, scales, stream=None) -> None:
    """codes (T x pitch) and scales (T x groups), both uint8, receive the 8-bit checkpoint of x (T x D)."""
    T, D = int(T), int(D)
    xp, ldx, cp, sp = *_matrix(x, "x", _torch_dtype(dtype), T, D), *_ckpt(codes, scales, T, D)
    _check(lib().rar_ckpt_store(T, D, dtype, xp, ldx, cp, sp, _on(stream)), "rar_ckpt_store")


def rar_ckpt_load(T: int, D: int, dtype: int, codes, scales, y, act: int = ACT_NONE, stream=None) -> None:
    """y (T x D) = act(what the checkpoint holds)."""
    T, D = int(T), int(D)
    yp, ldy, cp, sp = *_matrix(y, "y", _torch_dtype(dtype), T, D), *_ckpt(codes, scales, T, D)
    _check(lib().rar_ckpt_load(T, D, dtype, cp, sp, act, yp, ldy, _on(stream)), "rar_ckpt_load")


def _ckpt(codes, scales, T: int, D: int):
    import torch
    groups = -(-D // CKPT_GROUP)
    return (_dense(codes, "codes", torch.uint8, T * groups * CKPT_GROUP),
            _dense(scales, "scales", torch.uint8, T * groups))
