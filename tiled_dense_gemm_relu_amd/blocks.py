"""Products of 8-bit floating-point matrices scaled by blocks of 128 (the C ABI in include/gemm_relu_blocks.h).

``quantize_blocks`` makes such matrices, ``gemm_relu_blocks`` multiplies them (dense, or grouped by expert),
``gemm_relu_blocks_backward`` has the gradients of a layer that does, and ``linear_blocks`` is such a layer as a
node of autograd's graph.  ``gemm_relu_experts`` is a whole expert layer for a few tokens, with 16-bit or such
8-bit weights.
As in binding.py this is argument marshalling only, with no fallback.  The marshalling of ordinary calls is compiled
(csrc/blocks_calls.cpp), for what takes the GPU less time than Python; it leaves all others to this file.  Where it
was not built for the torch that runs, this file marshals every call to the same library.

A quantized matrix is a ``torch.float8_e4m3fn`` or ``torch.float8_e5m2`` tensor whose rows start at multiples
of 16 bytes (``stride(-2) % 16 == 0``), with float32 scales: by rows ``(blocks, rows)``, one for 128 elements
of a row, or by tiles ``(row blocks, blocks)``, one for 128 x 128.
"""
from __future__ import annotations

import ctypes
import functools
import threading

from . import binding
from .binding import B_KN, B_NK, _check, _stream_handle
from .groups import (_call, _check_layout, _check_shape, _check_tensor, _first, _new, _on, _refuse_tangents, _spaces,
                     _workspace)

BLOCK = 128                # GEMM_RELU_BLOCK

# Kernels of gemm_relu_blocks (GEMM_RELU_BLOCKS_*).
CONFIG_AUTO = -1
CONFIG_256 = 0
CONFIG_128 = 1
CONFIG_64 = 2
CONFIG_STREAM = 3

_lock = threading.Lock()
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = binding.load_library()
        with _lock:
            vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            lib.gemm_relu_quantize_blocks.argtypes = [vp] * 6 + [i64] * 5 + [ci] * 4 + [vp]
            lib.gemm_relu_quantize_blocks.restype = ci
            lib.gemm_relu_blocks.argtypes = [vp] * 6 + [i64] * 6 + [ci] * 6 + [vp]
            lib.gemm_relu_blocks.restype = ci
            lib.gemm_relu_blocks_backward.argtypes = [vp] * 8 + [i64] * 5 + [ci] * 5 + [vp, i64, vp]
            lib.gemm_relu_blocks_backward.restype = ci
            lib.gemm_relu_blocks_backward_workspace.argtypes = [i64] * 3
            lib.gemm_relu_blocks_backward_workspace.restype = i64
            lib.gemm_relu_experts.argtypes = [vp] * 9 + [i64] * 8 + [ci] * 4 + [vp, i64, vp]
            lib.gemm_relu_experts.restype = ci
            lib.gemm_relu_experts_workspace.argtypes = [i64] * 5 + [ci]
            lib.gemm_relu_experts_workspace.restype = i64
            _lib = lib
    return _lib


_calls = None


class _NotCompiled:
    """Leaves every call to Python."""

    @staticmethod
    def quantize(*args):
        return None

    multiply = backward = experts = quantize


def _compiled():
    """The compiled calls, with the entry points of the loaded library; where they were not built, or for another
    torch, a stand-in that leaves all calls to Python (some 5 to 9 us more a call on the host)."""
    global _calls
    if _calls is None:
        import torch
        lib = _library()
        try:
            from . import _blocks_calls as calls
            built_for = getattr(calls, "torch_version", "unknown")
            if built_for != torch.__version__:
                raise ImportError(f"built for torch {built_for}, this is {torch.__version__}")
        except ImportError as e:
            import warnings
            warnings.warn(f"gemm_relu: the compiled marshalling of 8-bit calls is not used ({e}); build the package again "
                          "for shorter calls", RuntimeWarning, stacklevel=3)
            _calls = _NotCompiled()
            return _calls
        calls.use(*(ctypes.cast(f, ctypes.c_void_p).value
                    for f in (lib.gemm_relu_quantize_blocks, lib.gemm_relu_blocks, lib.gemm_relu_blocks_backward,
                              lib.gemm_relu_blocks_backward_workspace, lib.gemm_relu_experts, lib.gemm_relu_experts_workspace)))
        _calls = calls
    return _calls


@functools.lru_cache(maxsize=4096)
def _bytes(function: str, *args) -> int:
    """What a *_workspace function returns (pure host arithmetic on the sizes)."""
    n = getattr(_library(), function)(*args)
    if n < 0:
        _check(int(n))
    return n


def blocks_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace of gemm_relu_blocks_backward for these sizes (host only)."""
    return _bytes("gemm_relu_blocks_backward_workspace", M, N, K)


def experts_workspace_bytes(tokens: int, N: int, hidden: int, experts: int, top: int, b_layout: int = B_NK) -> int:
    """Workspace of gemm_relu_experts for these sizes (host only)."""
    return _bytes("gemm_relu_experts_workspace", tokens, N, hidden, experts, top, b_layout)


@functools.lru_cache(maxsize=1)
def _formats():
    import torch
    return {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


def _format_code(name, dtype) -> int:
    code = _formats().get(dtype)
    if code is None:
        raise TypeError(f"gemm_relu: {name} must be float8_e4m3fn or float8_e5m2, got {dtype}")
    return code


def _check_8bit(name, t, dim, dev=None):
    """(format, pitch) of a ``dim``-D 8-bit tensor: rows at one pitch, a multiple of 16 bytes, matrices of a
    stack one behind the other, all 16-byte pieces of its rows inside its storage."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"gemm_relu: {name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"gemm_relu: {name} must be a GPU tensor, got {t.device}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"gemm_relu: {name} must be on the same device as the other tensors")
    shape = t.shape
    if len(shape) != dim:
        raise ValueError(f"gemm_relu: {name} must be {dim}-D, got shape {tuple(shape)}")
    code = _format_code(name, t.dtype)
    if t.requires_grad:
        raise RuntimeError(f"gemm_relu: {name} requires a gradient, but 8-bit operands have none; detach it")
    rows, row = shape[-2], shape[-1]
    whole = row + 15 & -16
    if row == whole and rows > 1 and t.is_contiguous() and not t.data_ptr() & 15:
        return code, row
    if t.numel() == 0:
        return code, whole
    stride = t.stride()
    stacked = dim == 3 and shape[0] > 1
    pitch = stride[-2] if rows > 1 else stride[0] if stacked else whole
    if row > 1 and stride[-1] != 1:
        raise ValueError(f"gemm_relu: {name} must be row-major")
    if pitch < row or pitch % 16 or t.data_ptr() % 16:
        raise ValueError(f"gemm_relu: rows of {name} must start at multiples of 16 bytes, got stride {stride}")
    if stacked and stride[0] != rows * pitch:
        raise ValueError(f"gemm_relu: the matrices of {name} must lie one behind the other, got stride {stride}")
    count = rows * (shape[0] if dim == 3 else 1)
    if t.storage_offset() + (count - 1) * pitch + whole > t.untyped_storage().nbytes():
        raise ValueError(f"gemm_relu: the last row of {name} must have storage for whole 16-byte pieces")
    return code, pitch


def _check_scales(name, t, dim, dev, shape):
    """float32 scales of this shape, which have no gradient any more than the values they belong to."""
    import torch
    _check_tensor(name, t, dim, dev, torch.float32)
    _check_shape(name, t, shape)
    if t.requires_grad and torch.is_grad_enabled():
        raise RuntimeError(f"gemm_relu: {name} requires a gradient, but 8-bit operands have none; detach it")
    _refuse_tangents(name, t)


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _empty(shape, dtype, device, stream):
    """A new tensor for work on ``stream`` (groups._new)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_8bit(shape, dtype, device, stream):
    """An 8-bit tensor whose rows start at multiples of 16 bytes, and its pitch.  Long rows start at whole cache
    lines: pieces of 128 bytes would lie in two (products of 4000 x 11000 x 4100 take 214 us at a pitch of 4112,
    185 at 4224; 64 x 16384 x 8100 46 and 30.5)."""
    import torch
    pitch = shape[-1] + 15 & -16 if shape[-1] <= 1024 else shape[-1] + 127 & -128
    if pitch == shape[-1]:
        return _empty(shape, dtype, device, stream), pitch
    return _empty(shape[:-1] + (pitch,), torch.uint8, device, stream)[..., : shape[-1]].view(dtype), pitch


def quantize_blocks(x, dtype=None, tiles: bool = False, mask=None, rows: bool = True, transposed: bool = False,
                    power_of_two: bool = False, stream=None):
    """8-bit values and scales of ``x`` (R, C) or a stack (count, R, C) in fp16 or bf16.

    Returns ``(q, scales)``: q of x's shape in ``dtype`` (float8_e4m3fn by default, or float8_e5m2), its rows at
    multiples of 16 bytes, or of 128 if they are longer than 1024; scales (C/128, R), one for 128 elements of a
    row, or with ``tiles`` (R/128, C/128); counts of blocks are rounded up.  With ``transposed`` also
    ``(qt, scales_t)``: qt (C, R) the transposed matrix, quantized along its own rows, scales_t (R/128, C), or
    with ``tiles`` the same tiles' values, (C/128, R/128).  ``rows=False`` leaves the first pair out.  All from
    one pass over x.

    A block's scale is its largest finite magnitude (at least 2**-80) over the format's largest value, with
    ``power_of_two`` rounded up to a power of two; values are x / scale, rounded to fp32 and then to nearest
    even.  ``mask`` (x's shape and dtype): x counts as zero where it is not above zero (a ReLU's gradient).
    The outputs carry no gradient.
    """
    if stream is None:
        out = (_calls or _compiled()).quantize(x, 0 if dtype is None else _formats().get(dtype), tiles, mask, rows, transposed,
                                               power_of_two)
        if out is not None:
            return out
    import torch
    code, dev = _first("x", x)
    shape = tuple(x.shape)
    if len(shape) not in (2, 3):
        raise ValueError(f"gemm_relu: x must be 2-D or 3-D, got shape {shape}")
    _check_tensor("x", x, len(shape), dev, x.dtype)
    above = None
    if mask is not None:
        _check_tensor("mask", mask, len(shape), dev, x.dtype)
        _check_shape("mask", mask, shape)
        above = mask.data_ptr()
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    fmt = _format_code("dtype", dtype)
    if not rows and not transposed:
        raise ValueError("gemm_relu: neither rows nor transposed is asked for")
    stack, (R, C) = shape[:-2], shape[-2:]
    br, bc, device = _blocks(R), _blocks(C), x.device
    qp = sp = qtp = stp = None
    ldq = ldqt = 0
    out = ()
    if rows:
        q, ldq = _empty_8bit(shape, dtype, device, stream)
        s = _empty(stack + ((br, bc) if tiles else (bc, R)), torch.float32, device, stream)
        qp, sp, out = q.data_ptr(), s.data_ptr(), (q, s)
    if transposed:
        qt, ldqt = _empty_8bit(stack + (C, R), dtype, device, stream)
        st = _empty(stack + ((bc, br) if tiles else (br, C)), torch.float32, device, stream)
        qtp, stp, out = qt.data_ptr(), st.data_ptr(), out + (qt, st)
    if x.numel():
        _call(_library().gemm_relu_quantize_blocks, dev, x.data_ptr(), above, qp, sp, qtp, stp, stack[0] if stack else 1, R,
              C, ldq, ldqt, code, fmt, 1 if tiles else 0, 1 if power_of_two else 0, _stream_handle(stream, dev) or None)
    return out


def _output(out, out_dtype, shape, dev, device, stream):
    """(output, dtype code) of gemm_relu_blocks."""
    import torch
    if out is None:
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        if out_dtype is not torch.bfloat16 and out_dtype is not torch.float16:
            raise TypeError(f"gemm_relu: the output's dtype must be float16 or bfloat16, got {out_dtype}")
        return _empty(shape, out_dtype, device, stream), 0 if out_dtype is torch.float16 else 1
    code = _first("out", out)[0]
    if out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError(f"gemm_relu: out is {out.dtype}, but out_dtype is {out_dtype}")
    _check_tensor("out", out, 2, dev, out.dtype)
    _check_shape("out", out, shape)
    return out, code


def gemm_relu_blocks(a, a_scales, b, b_scales, ends=None, out=None, out_dtype=None, relu: bool = True,
                     b_rows: bool = False, config: int = CONFIG_AUTO, stream=None):
    """C = ReLU(A @ B^T) of the matrices that 8-bit ``a`` (M, K) and ``b`` (N, K) stand for.

    ``a_scales`` (K/128, M) by rows; ``b_scales`` (N/128, K/128) by tiles, or (K/128, N) with ``b_rows``;
    counts of blocks are rounded up.  With ``ends`` (groups,) int32 on the GPU, non-decreasing, ``b`` is
    (groups, N, K), its scales have groups in front, and row m of group g (rows ends[g-1] .. ends[g]-1) is
    multiplied with b[g]; rows past the last end get zeros.  ``relu=False`` leaves the ReLU out.  C (M, N) is
    ``out`` if given, else a new tensor of ``out_dtype`` (bfloat16 by default).  ``config``: a
    kernel (CONFIG_*), by default the library's choice.  8-bit values and their scales have no gradient;
    one that requires it is refused.
    """
    import torch
    if stream is None and out is None and (out_dtype is None or out_dtype is torch.bfloat16 or out_dtype is torch.float16):
        out = (_calls or _compiled()).multiply(a, a_scales, b, b_scales, ends, out_dtype is not torch.float16, relu, b_rows, config)
        if out is not None:
            return out
    fa, lda = _check_8bit("a", a, 2)
    dev = a.get_device()
    grouped = ends is not None
    fb, ldb = _check_8bit("b", b, 3 if grouped else 2, dev)
    M, K = a.shape
    N, groups = b.shape[-2], b.shape[0] if grouped else 1
    if b.shape[-1] != K:
        raise ValueError(f"gemm_relu: inner dimensions differ: a {tuple(a.shape)}, b {tuple(b.shape)}")
    kb = _blocks(K)
    _check_scales("a_scales", a_scales, 2, dev, (kb, M))
    _check_scales("b_scales", b_scales, 3 if grouped else 2, dev,
                  ((groups,) if grouped else ()) + ((kb, N) if b_rows else (_blocks(N), kb)))
    if grouped:
        _check_tensor("ends", ends, 1, dev, torch.int32)
        _check_shape("ends", ends, (groups,))
    out, code = _output(out, out_dtype, (M, N), dev, a.device, stream)
    _call(_library().gemm_relu_blocks, dev, a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(),
          ends.data_ptr() if grouped else None, out.data_ptr(), M, N, K, groups, lda, ldb, fa, fb, 0 if b_rows else 1,
          code, 1 if relu else 0, config, _stream_handle(stream, dev) or None)
    return out


def gemm_relu_blocks_backward(dc, c, xt, xt_scales, wt, wt_scales, relu: bool = True, dtype=None, dx=None, dw=None,
                              need_dx: bool = True, need_dw: bool = True, workspace=None, stream=None):
    """Gradients (dx, dw) of C = ReLU(X @ W^T), X (M, K), W (N, K), for C's gradient ``dc``, both (M, N).

    D, dc where c > 0, is quantized to ``dtype`` (float8_e5m2 by default) in blocks of 128 along the summed
    dimension of each product.  ``xt`` (K, M) with scales (M/128, K) by rows, and ``wt`` (K, N) with scales
    (K/128, N/128) by tiles, are the transposed outputs of quantize_blocks for X and (tiles=True) W.
    ``need_dx=False`` / ``need_dw=False`` leave one out (None is returned, and ``wt`` / ``xt`` with their
    scales may be None).  ``c`` is only read with ``relu=True``.  The gradients have dc's dtype.
    """
    if stream is None and workspace is None and dx is None and dw is None and need_dx and need_dw:
        out = (_calls or _compiled()).backward(dc, c, xt, xt_scales, wt, wt_scales, relu,
                                               1 if dtype is None else _formats().get(dtype), _spaces)
        if out is not None:
            return out
    import torch
    code, dev = _first("dc", dc)
    _check_tensor("dc", dc, 2, dev, dc.dtype)
    dtype = torch.float8_e5m2 if dtype is None else dtype
    fmt = _format_code("dtype", dtype)
    if not need_dx and not need_dw:
        raise ValueError("gemm_relu: neither gradient is asked for")
    M, N = dc.shape
    if relu:
        _check_tensor("c", c, 2, dev, dc.dtype)
        _check_shape("c", c, (M, N))
    fx = fw = ldxt = ldwt = 0
    if need_dw:
        fx, ldxt = _check_8bit("xt", xt, 2, dev)
        K = xt.shape[0]
        _check_shape("xt", xt, (K, M))
        _check_scales("xt_scales", xt_scales, 2, dev, (_blocks(M), K))
    if need_dx:
        fw, ldwt = _check_8bit("wt", wt, 2, dev)
        K = K if need_dw else wt.shape[0]
        _check_shape("wt", wt, (K, N))
        _check_scales("wt_scales", wt_scales, 2, dev, (_blocks(K), _blocks(N)))

    def output(name, t, shape):
        if t is None:
            return _new(shape, dc, stream)
        _check_tensor(name, t, 2, dev, dc.dtype)
        _check_shape(name, t, shape)
        return t
    dx = output("dx", dx, (M, K)) if need_dx else None
    dw = output("dw", dw, (N, K)) if need_dw else None
    handle = _stream_handle(stream, dev)
    ws, ws_bytes, keep = _workspace(workspace, blocks_backward_workspace_bytes(M, N, K), dc, dev, handle, stream)
    # An empty gradient still needs an address to be asked for.
    _call(_library().gemm_relu_blocks_backward, dev, dc.data_ptr(), c.data_ptr() if relu else None,
          xt.data_ptr() if need_dw else None, xt_scales.data_ptr() if need_dw else None,
          wt.data_ptr() if need_dx else None, wt_scales.data_ptr() if need_dx else None,
          (dx.data_ptr() or 256) if need_dx else None, (dw.data_ptr() or 256) if need_dw else None, M, N, K, ldxt, ldwt,
          fmt, fx, fw, code, 1 if relu else 0, ws, ws_bytes, handle or None)
    return dx, dw


@functools.lru_cache(maxsize=1)
def _linear():
    import torch
    from torch.autograd.function import once_differentiable

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, relu, dtype, grad_dtype):
            need_x, need_w = ctx.needs_input_grad[:2]
            # one pass over each matrix writes what forward and backward read
            q, s, xt, sxt = quantize_blocks(x, dtype, transposed=True) if need_w else quantize_blocks(x, dtype) + (None, None)
            qw, sw, wt, swt = (quantize_blocks(w, dtype, tiles=True, transposed=True) if need_x
                               else quantize_blocks(w, dtype, tiles=True) + (None, None))
            c = gemm_relu_blocks(q, s, qw, sw, out_dtype=x.dtype, relu=relu)
            ctx.save_for_backward(c if relu else None, xt, sxt, wt, swt)
            ctx.relu, ctx.grad_dtype = relu, grad_dtype
            return c

        @staticmethod
        @once_differentiable
        def backward(ctx, dc):
            c, xt, sxt, wt, swt = ctx.saved_tensors
            need_x, need_w = ctx.needs_input_grad[:2]
            dx, dw = gemm_relu_blocks_backward(dc.contiguous(), c, xt, sxt, wt, swt, relu=ctx.relu, dtype=ctx.grad_dtype,
                                               need_dx=need_x, need_dw=need_w)
            return dx, dw, None, None, None

    return Linear


def linear_blocks(x, w, relu: bool = True, dtype=None, grad_dtype=None, stream=None):
    """ReLU(x @ w^T) in 8 bits, with gradients: x (M, K) and w (N, K) in fp16 or bf16.

    x is quantized by rows and w by tiles to ``dtype`` (float8_e4m3fn by default), the gradient of the result
    by rows to ``grad_dtype`` (float8_e5m2); gradients pass the rounding of x and w unchanged.  What backward
    needs of x and w is kept in 8 bits.  Forward and backward run on ``stream``, or the current one.  A backward
    pass can be captured; as with torch's own operators, no eager graph of the same leaves may be alive meanwhile.
    Tangents of forward mode are refused.
    """
    _, dev = _first("x", x)
    _check_tensor("x", x, 2, dev, x.dtype)
    _check_tensor("w", w, 2, dev, x.dtype)
    if w.shape[1] != x.shape[1]:
        raise ValueError(f"gemm_relu: inner dimensions differ: x {tuple(x.shape)}, w {tuple(w.shape)}")
    import torch
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    grad_dtype = torch.float8_e5m2 if grad_dtype is None else grad_dtype
    _format_code("dtype", dtype)
    _format_code("grad_dtype", grad_dtype)
    _refuse_tangents("linear_blocks", x, w)
    with _on(stream, dev):
        if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
            return _linear().apply(x, w, bool(relu), dtype, grad_dtype)
        return gemm_relu_blocks(*quantize_blocks(x, dtype), *quantize_blocks(w, dtype, tiles=True), out_dtype=x.dtype,
                                relu=relu)


@functools.lru_cache(maxsize=1)
def _no_gradient():
    import torch

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w1, w2, logits, weights, w1_scales, w2_scales, call):
            return call()

        @staticmethod
        def backward(ctx, dy):
            raise NotImplementedError("gemm_relu: gemm_relu_experts has no gradient; call it under torch.no_grad()")

    return Experts


def gemm_relu_experts(x, w1, w2, logits=None, top=None, ids=None, weights=None, w1_scales=None, w2_scales=None,
                      out=None, b_layout: int = B_NK, renormalize: bool = True, workspace=None, stream=None):
    """A whole expert layer for up to 64 tokens: y[t] = sum_j weights[t, j] ReLU(x[t] @ W1[e]) @ W2[e], e = ids[t, j].

    ``x`` (tokens, K), fp16 or bf16.  ``w1`` (experts, hidden, K) and ``w2`` (experts, N, hidden) with B_NK, or
    (experts, K, hidden) and (experts, hidden, N) with B_KN, in x's dtype; or with B_NK 8-bit, with
    ``w1_scales`` (experts, hidden/128, K/128) and ``w2_scales`` (experts, N/128, hidden/128) by tiles, counts
    rounded up (quantize_blocks with tiles=True).

    Either ``logits`` (tokens, experts) float32 and ``top``, up to 16: each token's ``top`` largest logits
    (ties to the lowest index, -inf never), weighted by their softmax over the chosen (``renormalize``) or all
    logits; a token with a logit of NaN or +inf gets a row of NaN.  Or ``ids`` (tokens, top) int32, ids outside
    0 .. experts-1 skipped, and ``weights`` (tokens, top) float32.  Returns (y, ids, weights), y (tokens, N) in
    x's dtype (``out`` if given).  There is no gradient: a backward pass is refused, and so is ``out`` where
    gradients are on and an input requires one.
    """
    if stream is None and workspace is None and out is None and ids is None and weights is None:
        result = (_calls or _compiled()).experts(x, w1, w2, logits, top, w1_scales, w2_scales, b_layout, renormalize, _spaces)
        if result is not None:
            return result
    import torch
    code, dev = _first("x", x)
    _check_layout(b_layout)
    nk = b_layout == B_NK
    _check_tensor("x", x, 2, dev, x.dtype)
    if not isinstance(w1, torch.Tensor) or not isinstance(w2, torch.Tensor):
        raise TypeError("gemm_relu: w1 and w2 must be torch.Tensors")
    eight = w1.dtype in _formats()
    fmt, ld1, ld2 = -1, 0, 0
    if eight:
        if not nk:
            raise ValueError("gemm_relu: 8-bit weights must be stored (out, in): b_layout=B_NK")
        fmt, ld1 = _check_8bit("w1", w1, 3, dev)
        fmt2, ld2 = _check_8bit("w2", w2, 3, dev)
        if fmt2 != fmt:
            raise TypeError(f"gemm_relu: w1 and w2 must have one format, got {w1.dtype} and {w2.dtype}")
    else:
        _check_tensor("w1", w1, 3, dev, x.dtype)
        _check_tensor("w2", w2, 3, dev, x.dtype)
    tokens, K = x.shape
    experts, hidden = w1.shape[0], w1.shape[1 if nk else 2]
    N = w2.shape[1 if nk else 2]
    _check_shape("w1", w1, (experts, hidden, K) if nk else (experts, K, hidden))
    _check_shape("w2", w2, (experts, N, hidden) if nk else (experts, hidden, N))
    if eight:
        _check_tensor("w1_scales", w1_scales, 3, dev, torch.float32)
        _check_shape("w1_scales", w1_scales, (experts, _blocks(hidden), _blocks(K)))
        _check_tensor("w2_scales", w2_scales, 3, dev, torch.float32)
        _check_shape("w2_scales", w2_scales, (experts, _blocks(N), _blocks(hidden)))
    elif w1_scales is not None or w2_scales is not None:
        raise ValueError("gemm_relu: scales are for 8-bit weights")
    routed = logits is not None
    if routed:
        if ids is not None or weights is not None:
            raise ValueError("gemm_relu: give logits and top, or ids and weights")
        if top is None:
            raise ValueError("gemm_relu: logits need top")
        _check_tensor("logits", logits, 2, dev, torch.float32)
        _check_shape("logits", logits, (tokens, experts))
    else:
        if ids is None or weights is None or top is not None:
            raise ValueError("gemm_relu: give logits and top, or ids and weights")
        _check_tensor("ids", ids, 2, dev, torch.int32)
        top = ids.shape[1]
        _check_shape("ids", ids, (tokens, top))
        _check_tensor("weights", weights, 2, dev, torch.float32)
        _check_shape("weights", weights, (tokens, top))
    inputs = x, w1, w2, logits, weights, w1_scales, w2_scales
    _refuse_tangents("gemm_relu_experts", *inputs)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        if out is not None:
            raise RuntimeError("gemm_relu: out= has no gradient, but an input requires one: leave out= away, or call "
                               "under torch.no_grad()")

        chosen = []

        def call():
            y, *rest = gemm_relu_experts(x, w1, w2, logits, top if routed else None, ids, weights, w1_scales, w2_scales,
                                         None, b_layout, renormalize, workspace, stream)
            chosen.extend(rest)
            return y
        with _on(stream, dev):
            y = _no_gradient().apply(*inputs, call)
        return (y, *chosen)
    need = experts_workspace_bytes(tokens, N, hidden, experts, top, b_layout)
    if routed:
        ids = _empty((tokens, top), torch.int32, x.device, stream)
        weights = _empty((tokens, top), torch.float32, x.device, stream)
    if out is None:
        out = _new((tokens, N), x, stream)
    else:
        _check_tensor("out", out, 2, dev, x.dtype)
        _check_shape("out", out, (tokens, N))
    handle = _stream_handle(stream, dev)
    ws, ws_bytes, keep = _workspace(workspace, need, x, dev, handle, stream)
    _call(_library().gemm_relu_experts, dev, x.data_ptr(), w1.data_ptr(), w1_scales.data_ptr() if eight else None,
          w2.data_ptr(), w2_scales.data_ptr() if eight else None, logits.data_ptr() if routed else None,
          ids.data_ptr(), weights.data_ptr(), out.data_ptr(), tokens, N, K, hidden, experts, top, ld1, ld2,
          1 if renormalize else 0, code, fmt, b_layout, ws, ws_bytes, handle or None)
    return out, ids, weights
