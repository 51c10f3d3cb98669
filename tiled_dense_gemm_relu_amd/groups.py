"""Products whose rows choose their weights (the C ABI in include/gemm_relu_groups.h).

``gemm_relu_grouped``: rows grouped by expert, with ``gemm_relu_grouped_backward`` for its gradients;
``gemm_relu_adapters``: a projection shared by all rows with the low-rank adapters of many requests.
As in binding.py this is argument marshalling only, with no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import threading

from . import binding
from .binding import B_KN, B_NK, _check, _dtype_code, _stream_handle

COUNTER_BYTES = 65536      # GEMM_RELU_GROUPS_COUNTER_BYTES

# Kernels (GEMM_RELU_GROUPS_*).
CONFIG_AUTO = -1
CONFIG_TILED = 0
CONFIG_DMA_256 = 1
CONFIG_DMA_128 = 2
CONFIG_DMA_64 = 3
CONFIG_STREAM = 4

_as_it_is = contextlib.nullcontext()
_lock = threading.Lock()
_lib = None
_spaces = {}               # (device, stream handle): the stream's workspace as (pointer, bytes, tensor)


def _library():
    global _lib
    if _lib is None:
        lib = binding.load_library()
        with _lock:
            vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            lib.gemm_relu_grouped.argtypes = [vp] * 4 + [i64] * 4 + [ci] * 4 + [vp, i64, vp]
            lib.gemm_relu_grouped.restype = ci
            lib.gemm_relu_grouped_workspace.argtypes = [i64] * 4 + [ci] * 2
            lib.gemm_relu_grouped_workspace.restype = i64
            lib.gemm_relu_grouped_backward.argtypes = [vp] * 7 + [i64] * 4 + [ci] * 4 + [vp, i64, vp]
            lib.gemm_relu_grouped_backward.restype = ci
            lib.gemm_relu_grouped_backward_workspace.argtypes = [i64] * 4 + [ci] * 3
            lib.gemm_relu_grouped_backward_workspace.restype = i64
            lib.gemm_relu_adapters.argtypes = [vp] * 8 + [i64] * 6 + [ci] * 4 + [vp, i64, vp]
            lib.gemm_relu_adapters.restype = ci
            lib.gemm_relu_adapters_workspace.argtypes = [i64] * 6 + [ci] * 2
            lib.gemm_relu_adapters_workspace.restype = i64
            _lib = lib
    return _lib


@functools.lru_cache(maxsize=4096)
def _bytes(function: str, *args) -> int:
    """What a *_workspace function returns (pure host arithmetic on the sizes)."""
    n = getattr(_library(), function)(*args)
    if n < 0:
        _check(int(n))
    return n


def grouped_workspace_bytes(M: int, N: int, K: int, groups: int, dtype: int, b_layout: int = B_KN) -> int:
    """Workspace of gemm_relu_grouped for these sizes (host only)."""
    return _bytes("gemm_relu_grouped_workspace", M, N, K, groups, dtype, b_layout)


def grouped_backward_workspace_bytes(M: int, N: int, K: int, groups: int, dtype: int, b_layout: int = B_KN,
                                     relu: bool = True) -> int:
    """Workspace of gemm_relu_grouped_backward for these sizes (host only)."""
    return _bytes("gemm_relu_grouped_backward_workspace", M, N, K, groups, dtype, b_layout, int(relu))


def adapters_workspace_bytes(M: int, N: int, K: int, rank: int, adapters: int, segments: int, dtype: int,
                             b_layout: int = B_KN) -> int:
    """Workspace of gemm_relu_adapters for these sizes (host only)."""
    return _bytes("gemm_relu_adapters_workspace", M, N, K, rank, adapters, segments, dtype, b_layout)


def _check_tensor(name, t, dim, dev, dtype):
    """A contiguous ``dim``-D tensor of this dtype on device ``dev`` (one look at each property: these
    checks are a good part of a small call's time on the host)."""
    import torch
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == dim
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"gemm_relu: {name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"gemm_relu: {name} must be a GPU tensor, got {t.device}")
    if t.dim() != dim:
        raise ValueError(f"gemm_relu: {name} must be {dim}-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"gemm_relu: {name} must be contiguous (row-major)")
    if t.dtype != dtype:
        raise TypeError(f"gemm_relu: {name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"gemm_relu: {name} must be on the same device as the other tensors")


def _check_shape(name, t, shape):
    if tuple(t.shape) != shape:
        raise ValueError(f"gemm_relu: {name} must have shape {shape}, got {tuple(t.shape)}")


def _first(name, t):
    """Dtype and device that the other tensors have to share."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"gemm_relu: {name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"gemm_relu: {name} must be a GPU tensor, got {t.device}")
    return _dtype_code(t), t.get_device()


def _check_layout(b_layout):
    if b_layout not in (B_KN, B_NK):
        raise ValueError(f"gemm_relu: b_layout must be B_KN or B_NK, got {b_layout}")


def _refuse_tangents(what, *tensors):
    """Forward-mode derivatives of ``what``'s inputs are refused: there is none to pass on."""
    from torch.autograd import forward_ad
    if forward_ad._current_level < 0:         # no dual tensors without a level
        return
    import torch
    if any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"gemm_relu: {what} has no forward-mode derivative; pass the primal")


def _new(shape, like, stream):
    """An output for work on ``stream``: allocated for that stream, so that its memory is not one
    that still belongs to other work there."""
    if stream is None:
        return like.new_empty(shape)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape)


def _on(stream, dev):
    """Makes the stream that the kernels run on the current one."""
    import torch
    if stream is not None:
        return torch.cuda.stream(stream)
    return _as_it_is if _current_device() == dev else torch.cuda.device(dev)


def _workspace(given, need, like, dev, handle, stream):
    """(pointer, bytes, tensor) of the workspace: ``given``, or the cached one of this stream.  A capture
    takes memory of its own graph, so that replays stay valid when the cached buffer is replaced by a
    larger one or released.  (gemm_relu_splitk's captures hold its cached buffer: these calls have one of
    their own and never replace that.)"""
    if need == 0:
        return None, 0, None
    import torch
    if given is None:
        # On the kernels' stream, which need not be the current one: nothing else orders the clearing
        # before them, or keeps the memory from others while they run.
        with _on(stream, dev):
            capturing = torch.cuda.is_current_stream_capturing()
            known = None if capturing else _spaces.get((dev, handle))
            if known is None or known[1] < need:
                given = torch.empty(need, dtype=torch.uint8, device=like.device)
                given[:COUNTER_BYTES].zero_()
                known = given.data_ptr(), need, given
                if not capturing:
                    _spaces[(dev, handle)] = known
        return known
    if not isinstance(given, torch.Tensor) or not given.is_cuda or not given.is_contiguous():
        raise TypeError("gemm_relu: workspace must be a contiguous GPU tensor")
    if given.get_device() != dev:
        raise ValueError("gemm_relu: workspace must be on the same device as the other tensors")
    return given.data_ptr(), given.numel() * given.element_size(), given


@functools.lru_cache(maxsize=1)
def _functions():
    """The autograd functions behind calls whose inputs require gradients: (grouped, adapters).  Their
    forward runs with gradients off, so it is the plain call."""
    import torch
    from torch.autograd.function import once_differentiable

    class Grouped(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b, ends, b_layout, relu, config, workspace):
            c = gemm_relu_grouped(a, b, ends, b_layout=b_layout, relu=relu, config=config, workspace=workspace)
            need_a, need_b = ctx.needs_input_grad[:2]
            ctx.save_for_backward(a if need_b else None, b if need_a else None, ends, c if relu else None)
            ctx.b_layout, ctx.relu = b_layout, relu
            return c

        @staticmethod
        @once_differentiable
        def backward(ctx, dc):
            a, b, ends, c = ctx.saved_tensors
            da, db = gemm_relu_grouped_backward(dc.contiguous(), c, a, b, ends, b_layout=ctx.b_layout, relu=ctx.relu,
                                                need_da=ctx.needs_input_grad[0], need_db=ctx.needs_input_grad[1])
            return da, db, None, None, None, None, None

    class Adapters(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, u, v, scales, ends, ids, b_layout, relu, config, workspace):
            return gemm_relu_adapters(x, w, u, v, scales, ends, ids, b_layout=b_layout, relu=relu, config=config,
                                      workspace=workspace)

        @staticmethod
        def backward(ctx, dc):
            raise NotImplementedError("gemm_relu: gemm_relu_adapters has no gradient; call it under torch.no_grad()")

    return Grouped, Adapters


def _differentiable(function, dev, out, stream, *args):
    """The call as a node of autograd's graph, on the kernels' stream so that its backward runs there too."""
    if out is not None:
        raise RuntimeError("gemm_relu: out= has no gradient, but an input requires one: leave out= away, or call "
                           "under torch.no_grad()")
    with _on(stream, dev):
        return function.apply(*args)


def release_workspaces():
    """Gives back the cached workspaces: one per stream, as large as its largest call needed (large products
    of odd row lengths need copies of their operands, all groups' weights among them).  Work already queued
    keeps its memory until it is done; the next call takes a new one."""
    _spaces.clear()


def _call(function, dev, *args):
    """The library launches on the current device: make it the tensors' one."""
    import torch
    if _current_device() == dev:
        rc = function(*args)
    else:
        with torch.cuda.device(dev):
            rc = function(*args)
    if rc != 0:
        _check(rc)


def _current_device() -> int:
    import torch
    raw = getattr(torch._C, "_cuda_getDevice", None)
    return raw() if raw is not None else torch.cuda.current_device()


def gemm_relu_grouped(a, b, ends, out=None, b_layout: int = B_KN, relu: bool = True, config: int = CONFIG_AUTO,
                      workspace=None, stream=None):
    """C[m] = ReLU(a[m] @ B[g]) for every row m of group g (``relu=False``: without the ReLU).

    ``a`` (M, K), fp16 or bf16; ``b`` (groups, K, N), or (groups, N, K) with B_NK; ``ends`` (groups,)
    int32 on the GPU, non-decreasing: group g holds rows ends[g-1] .. ends[g]-1 (a running sum of
    row counts).  Rows past the last end get zeros.  ``out`` (M, N) is written if given.
    ``workspace``: at least grouped_workspace_bytes(...) bytes whose first 65536 are zero, or None
    for a cached one per stream.  ``config``: a kernel (CONFIG_*), by default the library's choice.
    Where gradients are on and ``a`` or ``b`` requires one, the result carries them
    (gemm_relu_grouped_backward, on ``stream``); ``out`` is refused then.  A backward pass can be
    captured; as with torch's own operators, no eager graph of the same leaves may be alive meanwhile.
    """
    import torch
    code, dev = _first("a", a)
    _check_layout(b_layout)
    _check_tensor("a", a, 2, dev, a.dtype)
    _check_tensor("b", b, 3, dev, a.dtype)
    _check_tensor("ends", ends, 1, dev, torch.int32)
    M, K = a.shape
    groups, N, k_b = b.shape
    if b_layout != B_NK:
        N, k_b = k_b, N
    if k_b != K:
        raise ValueError(f"gemm_relu: inner dimensions differ: a {tuple(a.shape)}, b {tuple(b.shape)}")
    if ends.shape[0] != groups:
        raise ValueError(f"gemm_relu: ends must have one entry for each of {groups} groups, got {ends.shape[0]}")
    _refuse_tangents("gemm_relu_grouped", a, b)
    if (a.requires_grad or b.requires_grad) and torch.is_grad_enabled():
        return _differentiable(_functions()[0], dev, out, stream, a, b, ends, b_layout, relu, config, workspace)
    if out is None:
        out = _new((M, N), a, stream)
    else:
        _check_tensor("out", out, 2, dev, a.dtype)
        _check_shape("out", out, (M, N))
    handle = _stream_handle(stream, dev)
    ws, ws_bytes, keep = _workspace(workspace, grouped_workspace_bytes(M, N, K, groups, code, b_layout), a, dev,
                                    handle, stream)
    _call(_library().gemm_relu_grouped, dev, a.data_ptr(), b.data_ptr(), ends.data_ptr(), out.data_ptr(), M, N, K,
          groups, code, b_layout, 1 if relu else 0, config, ws, ws_bytes, handle or None)
    return out


def gemm_relu_grouped_backward(dc, c, a, b, ends, b_layout: int = B_KN, relu: bool = True, da=None, db=None,
                               need_da: bool = True, need_db: bool = True, config: int = CONFIG_AUTO, workspace=None,
                               stream=None):
    """Gradients (da, db) of gemm_relu_grouped's C = ``c`` for its gradient ``dc``, both (M, N).

    da has a's shape (zeros in rows of no group), db has b's (zeros for empty groups).
    ``need_da=False`` / ``need_db=False`` leave one out (None is returned for it, and ``b`` / ``a``
    may be None).  ``c`` is only read with ``relu=True`` and may be None without.  The gradients are
    plain tensors, whether or not the inputs require gradients themselves.
    """
    import torch
    code, dev = _first("dc", dc)
    _check_layout(b_layout)
    _check_tensor("dc", dc, 2, dev, dc.dtype)
    _check_tensor("ends", ends, 1, dev, torch.int32)
    if not need_da and not need_db:
        raise ValueError("gemm_relu: neither gradient is asked for")
    M, N = dc.shape
    groups = ends.shape[0]
    if relu:
        _check_tensor("c", c, 2, dev, dc.dtype)
        _check_shape("c", c, (M, N))
    if need_db:
        _check_tensor("a", a, 2, dev, dc.dtype)
        K = a.shape[1]
        _check_shape("a", a, (M, K))
    if need_da:
        _check_tensor("b", b, 3, dev, dc.dtype)
        if not need_db:
            K = b.shape[2 if b_layout == B_NK else 1]
        _check_shape("b", b, (groups, N, K) if b_layout == B_NK else (groups, K, N))
        if da is None:
            da = _new((M, K), dc, stream)
        else:
            _check_tensor("da", da, 2, dev, dc.dtype)
            _check_shape("da", da, (M, K))
    if need_db:
        shape = (groups, N, K) if b_layout == B_NK else (groups, K, N)
        if db is None:
            db = _new(shape, dc, stream)
        else:
            _check_tensor("db", db, 3, dev, dc.dtype)
            _check_shape("db", db, shape)
    handle = _stream_handle(stream, dev)
    ws, ws_bytes, keep = _workspace(workspace, grouped_backward_workspace_bytes(M, N, K, groups, code, b_layout, relu),
                                    dc, dev, handle, stream)
    # An empty gradient still needs an address to be asked for.
    _call(_library().gemm_relu_grouped_backward, dev, dc.data_ptr(), c.data_ptr() if relu else None,
          a.data_ptr() if need_db else None, b.data_ptr() if need_da else None, ends.data_ptr(),
          (da.data_ptr() or 256) if need_da else None, (db.data_ptr() or 256) if need_db else None, M, N, K, groups,
          code, b_layout, 1 if relu else 0, config, ws, ws_bytes, handle or None)
    return (da if need_da else None), (db if need_db else None)


def gemm_relu_adapters(x, w, u, v, scales, ends, ids, out=None, b_layout: int = B_KN, relu: bool = True,
                       config: int = CONFIG_AUTO, workspace=None, stream=None):
    """C[m] = ReLU(x[m] @ W + scales[i] (x[m] @ U_i) @ V_i), i = ids[segment of row m].

    ``x`` (M, K); B_KN: ``w`` (K, N), ``u`` (adapters, K, rank), ``v`` (adapters, rank, N); B_NK:
    ``w`` (N, K), ``u`` (adapters, rank, K), ``v`` (adapters, N, rank); ``scales`` (adapters,) float32.
    ``ends`` and ``ids`` (segments,) int32: segment s holds rows ends[s-1] .. ends[s]-1 and uses adapter
    ids[s]; an id outside 0 .. adapters-1, and rows past the last end, use none.  ``relu=False``
    leaves the ReLU out.  There is no gradient: where gradients are on and an input requires one,
    ``out`` is refused, and so is a backward pass through the result.
    """
    import torch
    code, dev = _first("x", x)
    _check_layout(b_layout)
    nk = b_layout == B_NK
    dtype = x.dtype
    _check_tensor("x", x, 2, dev, dtype)
    _check_tensor("w", w, 2, dev, dtype)
    _check_tensor("u", u, 3, dev, dtype)
    _check_tensor("v", v, 3, dev, dtype)
    _check_tensor("scales", scales, 1, dev, torch.float32)
    _check_tensor("ends", ends, 1, dev, torch.int32)
    _check_tensor("ids", ids, 1, dev, torch.int32)
    M, K = x.shape
    N = w.shape[0 if nk else 1]
    adapters, rank = u.shape[0], u.shape[1 if nk else 2]
    _check_shape("w", w, (N, K) if nk else (K, N))
    _check_shape("u", u, (adapters, rank, K) if nk else (adapters, K, rank))
    _check_shape("v", v, (adapters, N, rank) if nk else (adapters, rank, N))
    _check_shape("scales", scales, (adapters,))
    segments = ends.shape[0]
    _check_shape("ids", ids, (segments,))
    _refuse_tangents("gemm_relu_adapters", x, w, u, v, scales)
    if (x.requires_grad or w.requires_grad or u.requires_grad or v.requires_grad
            or scales.requires_grad) and torch.is_grad_enabled():
        return _differentiable(_functions()[1], dev, out, stream, x, w, u, v, scales, ends, ids, b_layout, relu, config,
                               workspace)
    if out is None:
        out = _new((M, N), x, stream)
    else:
        _check_tensor("out", out, 2, dev, dtype)
        _check_shape("out", out, (M, N))
    handle = _stream_handle(stream, dev)
    ws, ws_bytes, keep = _workspace(workspace, adapters_workspace_bytes(M, N, K, rank, adapters, segments, code,
                                                                        b_layout), x, dev, handle, stream)
    _call(_library().gemm_relu_adapters, dev, x.data_ptr(), w.data_ptr(), u.data_ptr(), v.data_ptr(),
          scales.data_ptr(), ends.data_ptr(), ids.data_ptr(), out.data_ptr(), M, N, K, rank, adapters, segments,
          code, b_layout, 1 if relu else 0, config, ws, ws_bytes, handle or None)
    return out
