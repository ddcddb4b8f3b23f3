"""The operators of a mixture-of-experts layer (the C ABI in include/experts.h).

A router gives each token ``top_k`` expert ids. ``group_rows`` counts the
(token, choice) pairs of each expert and sorts them; ``matmul`` multiplies the
sorted rows by their experts' weights (``matmul_dx`` and ``matmul_dw`` are its
gradients, ``int8_matmul`` its 8-bit form); ``combine`` adds the results back
to their tokens (``combine_backward``: its gradients). ``linear`` and
``merge`` are the product and the sum for torch's autograd, with gradients of the
first order (a gradient of a gradient raises RuntimeError).

::

    g = experts.group_rows(ids, num_experts)              # ids: [tokens, top_k]
    h = experts.linear(x, w_up, g, gather=True)           # x: [tokens, k] -> [pairs, n]
    y = experts.linear(torch.nn.functional.silu(h), w_down, g)
    out = experts.merge(y, g, weights)                    # [tokens, k]

A pair whose id lies outside [0, experts) is dropped: place -1, no row, nothing
added. Rows of the sorted arrays past the last kept pair are zero.

Tensors are bfloat16 or float16, rows of unit stride (the stride between rows
is free). Every call queues kernels on the current stream of the tensors'
device, allocates its results there, and never synchronises, so it can be
captured into a graph. A bad argument raises ValueError, a status of the
library hist.HistError; there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import hist

MAX_EXPERTS = 1024
MAX_TOP_K = 64
_ONE_WORKGROUP = 8192  # pairs that experts_group sorts without a workspace
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}

_vp, _u32, _u64, _i32, _i64 = (ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int32,
                               ctypes.c_int64)
_SIGNATURES = {
    "experts_group_workspace_size": [_u64, _u32, _u32, ctypes.POINTER(_u64)],
    "experts_group": [_vp, _i32, _u64, _u32, _u32, _vp, _vp, _vp, _vp, _vp, _u64, _vp],
    "experts_matmul": [_vp, _i64, _vp, _i64, _u64, _vp, _i64, _i64, _vp, _vp, _u64, _u32, _u32,
                       _u32, _u32, _i32, _vp],
    "experts_matmul_dx": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _u64, _u32, _u32, _u32,
                          _i32, _vp],
    "experts_matmul_dw": [_vp, _vp, _i64, _vp, _i64, _u64, _vp, _vp, _u64, _u32, _u32, _u32, _u32,
                          _i32, _vp],
    "experts_combine": [_vp, _i64, _vp, _i64, _u64, _vp, _vp, _u64, _u32, _u32, _i32, _vp],
    "experts_combine_backward": [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _u64, _u32,
                                 _u32, _i32, _vp],
    "experts_quantize_rows": [_vp, _i64, _vp, _vp, _i64, _u64, _u32, _i32, _vp],
    "experts_int8_matmul": [_vp, _i64, _vp, _i64, _u64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _u64,
                            _u32, _u32, _u32, _u32, _i32, _vp],
}
PRODUCTS = {"matmul": 0, "matmul_dx": 1, "matmul_dw": 2, "int8_matmul": 3}


class Kernel(ctypes.Structure):
    """The kernel of a product (``preview``)."""
    _fields_ = [("rows", _u32), ("cols", _u32), ("threads", _u32), ("stages", _u32),
                ("per_cu", _u32), ("direct", _u32)]


_SIGNATURES["experts_product_preview"] = [_i32, _u64, _u64, _u32, _u32, _u32, _i64, _i64, _u32,
                                          ctypes.POINTER(Kernel)]
_functions: dict = {}
# 0.1 us; current_stream().cuda_stream takes 2.8. (A torch build for the host alone does not have it; no
# tensor gets as far as a call there.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _library():
    global _functions
    lib = hist.library()
    if not _functions:
        bound = {}
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = _i32, args
            bound[name] = fn
        _functions = bound  # whole at once: another thread sees none of them or all
    return lib


def _call(name: str, device: torch.device, *args):
    """The call on the current stream of the device."""
    if not _functions:
        _library()
    index = device.index
    if torch.cuda.current_device() == index:
        status = _functions[name](*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = _functions[name](*args, _raw_stream(index))
    if status:
        raise hist.HistError(status, name)


class Groups(NamedTuple):
    """The pairs of a routing, sorted by expert (int32 CUDA tensors)."""
    counts: torch.Tensor   # [experts] pairs of each expert
    offsets: torch.Tensor  # [experts + 1] their exclusive sum; the last one: kept pairs
    order: torch.Tensor    # [pairs] sorted place -> pair (token * top_k + choice), -1 past the end
    place: torch.Tensor    # [tokens, top_k] pair -> sorted place, -1 where dropped


# The checks run on every call, so what they say is only put together when one fails.

def _matrix(t: torch.Tensor, name: str, dtypes=_DTYPES, dim: int = 2) -> int:
    """Checks a matrix (or a stack of them) and returns its leading dimension."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == dim):
        raise ValueError(f"{name} must be a CUDA tensor of {dim} dimensions and of type "
                         f"{' or '.join(map(str, dtypes))}")
    rows, width = t.shape[-2:]
    stride = t.stride()
    ld = stride[-2] if rows > 1 else width
    if width == 0 or (rows and width > 1 and stride[-1] != 1) or ld < width:
        raise ValueError(f"{name} must have columns, and rows of unit stride that do not overlap")
    return ld


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: torch.device):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and
            t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")


def _groups(g: Groups, device: torch.device) -> tuple[int, int, int]:
    """Checks the groups and returns (experts, pairs, top_k)."""
    _, offsets, order, place = g
    if place.dim() != 2:
        raise ValueError("place must have the shape [tokens, top_k]")
    tokens, top_k = place.shape
    experts, pairs = offsets.numel() - 1, tokens * top_k
    _vector(offsets, "offsets", torch.int32, (g.counts.numel() + 1,), device)
    _vector(order, "order", torch.int32, (pairs,), device)
    _vector(place, "place", torch.int32, (tokens, top_k), device)
    return experts, pairs, top_k


def _rows(x: torch.Tensor, g: Groups, pairs: int, gather: bool, name: str):
    want = g.place.shape[0] if gather else pairs
    if x.shape[0] != want:
        raise ValueError(
            f"{name} must have {want} rows, one for each {'token' if gather else 'pair'}")


def _weights(w: torch.Tensor, experts: int, device: torch.device, dtype: torch.dtype):
    """Leading dimension and stride of the experts' weights [experts, n, k]."""
    ld = _matrix(w, "w", (dtype,), 3)
    if w.device != device or w.shape[0] != experts or w.shape[1] == 0:
        raise ValueError(f"w must hold {experts} experts' weights, with rows, on {device}")
    return ld, w.stride(0) if experts > 1 else 0


def _same(a: int, b: int, what: str):
    if a != b:
        raise ValueError(f"{what} must agree, not be {a} and {b}")


def _device(a: torch.Tensor, b: torch.Tensor, what: str):
    if a.device != b.device:
        raise ValueError(f"{what} must be on one device")


def group_rows(ids: torch.Tensor, experts: int) -> Groups:
    """Count and sort the pairs of ``ids`` (int32 or int64, [tokens, top_k],
    contiguous) by expert; pairs of one expert keep their order."""
    if not (isinstance(ids, torch.Tensor) and ids.is_cuda and ids.dim() == 2 and
            ids.dtype in (torch.int32, torch.int64) and ids.is_contiguous()):
        raise ValueError("ids must be a contiguous int32 or int64 CUDA tensor of shape "
                         "[tokens, top_k]")
    tokens, top_k = ids.shape
    if top_k <= 0 or experts <= 0:
        raise ValueError("top_k and experts must be positive")
    pairs, work = tokens * top_k, 0
    if pairs > _ONE_WORKGROUP:
        need = _u64()
        _library()
        status = _functions["experts_group_workspace_size"](tokens, top_k, experts,
                                                            ctypes.byref(need))
        if status:
            raise hist.HistError(status, "experts_group_workspace_size")
        work = need.value // 4
    # one allocation, the workspace first (its start is aligned)
    buf = torch.empty(work + 2 * experts + 1 + 2 * pairs, dtype=torch.int32, device=ids.device)
    counts, offsets, order, place = buf[work:].split((experts, experts + 1, pairs, pairs)) \
        if work else buf.split((experts, experts + 1, pairs, pairs))
    at = buf.data_ptr()
    c = at + 4 * work
    _call("experts_group", ids.device, ids.data_ptr(), ids.element_size() * 8, tokens, top_k,
          experts, c, c + 4 * experts, c + 4 * (2 * experts + 1),
          c + 4 * (2 * experts + 1 + pairs), at, 4 * work)
    return Groups(counts, offsets, order, place.view(tokens, top_k))


def matmul(x: torch.Tensor, w: torch.Tensor, g: Groups, gather: bool = False) -> torch.Tensor:
    """y[p] = x[p] w[e(p)]^T over the sorted pairs; w is [experts, n, k]. With
    ``gather`` x has one row a token, and pair p reads its token's."""
    ldx = _matrix(x, "x")
    experts, pairs, top_k = _groups(g, x.device)
    ldw, stride = _weights(w, experts, x.device, x.dtype)
    n, k = w.shape[1:]
    _same(x.shape[1], k, "the last dimensions of x and w")
    _rows(x, g, pairs, gather, "x")
    y = torch.empty(pairs, n, dtype=x.dtype, device=x.device)
    _call("experts_matmul", x.device, y.data_ptr(), n, x.data_ptr(), ldx, x.shape[0], w.data_ptr(),
          ldw, stride, g.offsets.data_ptr(), g.order.data_ptr() if gather else None, pairs, top_k,
          experts, n, k, _DTYPES[x.dtype])
    return y


def matmul_dx(dy: torch.Tensor, w: torch.Tensor, g: Groups) -> torch.Tensor:
    """dx[p] = dy[p] w[e(p)] over the sorted pairs (one row a pair; a token's
    gradient is ``combine(dx, g)``)."""
    lddy = _matrix(dy, "dy")
    experts, pairs, _ = _groups(g, dy.device)
    ldw, stride = _weights(w, experts, dy.device, dy.dtype)
    n, k = w.shape[1:]
    _same(dy.shape[1], n, "the columns of dy and the rows of w")
    _rows(dy, g, pairs, False, "dy")
    dx = torch.empty(pairs, k, dtype=dy.dtype, device=dy.device)
    _call("experts_matmul_dx", dy.device, dx.data_ptr(), k, dy.data_ptr(), lddy, w.data_ptr(), ldw,
          stride, g.offsets.data_ptr(), pairs, experts, n, k, _DTYPES[dy.dtype])
    return dx


def matmul_dw(dy: torch.Tensor, x: torch.Tensor, g: Groups, gather: bool = False) -> torch.Tensor:
    """dw[e] = sum over e's sorted pairs p of dy[p]^T x[p]; x as in ``matmul``."""
    lddy, ldx = _matrix(dy, "dy"), _matrix(x, "x", (dy.dtype,))
    experts, pairs, top_k = _groups(g, dy.device)
    _device(x, dy, "dy and x")
    _rows(dy, g, pairs, False, "dy")
    _rows(x, g, pairs, gather, "x")
    n, k = dy.shape[1], x.shape[1]
    dw = torch.empty(experts, n, k, dtype=dy.dtype, device=dy.device)
    _call("experts_matmul_dw", dy.device, dw.data_ptr(), dy.data_ptr(), lddy, x.data_ptr(), ldx,
          x.shape[0], g.offsets.data_ptr(), g.order.data_ptr() if gather else None, pairs, top_k,
          experts, n, k, _DTYPES[dy.dtype])
    return dw


def combine(y: torch.Tensor, g: Groups, weights: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] y[place[t, j]]; ``weights`` is
    float32 [tokens, top_k] (None: all one)."""
    ldy = _matrix(y, "y")
    _, pairs, top_k = _groups(g, y.device)
    _rows(y, g, pairs, False, "y")
    tokens, n = g.place.shape[0], y.shape[1]
    if weights is not None:
        _vector(weights, "weights", torch.float32, (tokens, top_k), y.device)
    out = torch.empty(tokens, n, dtype=y.dtype, device=y.device)
    _call("experts_combine", y.device, out.data_ptr(), n, y.data_ptr(), ldy, pairs,
          g.place.data_ptr(), None if weights is None else weights.data_ptr(), tokens, top_k, n,
          _DTYPES[y.dtype])
    return out


def combine_backward(dout: torch.Tensor, y: torch.Tensor, g: Groups,
                     weights: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """``combine``'s gradients: (dy [pairs, n], dweights float32 [tokens, top_k])."""
    lddout, ldy = _matrix(dout, "dout"), _matrix(y, "y", (dout.dtype,))
    _, pairs, top_k = _groups(g, y.device)
    _device(dout, y, "dout and y")
    _rows(y, g, pairs, False, "y")
    tokens, n = g.place.shape[0], y.shape[1]
    if dout.shape != (tokens, n):
        raise ValueError(f"dout must have the shape {(tokens, n)}")
    _vector(weights, "weights", torch.float32, (tokens, top_k), y.device)
    dy = torch.empty(pairs, n, dtype=y.dtype, device=y.device)
    dweights = torch.empty(tokens, top_k, dtype=torch.float32, device=y.device)
    _call("experts_combine_backward", y.device, dy.data_ptr(), n, dweights.data_ptr(),
          dout.data_ptr(), lddout, y.data_ptr(), ldy, g.order.data_ptr(), g.place.data_ptr(),
          weights.data_ptr(), tokens, top_k, n, _DTYPES[y.dtype])
    return dy, dweights


def quantize_rows(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """8-bit rows and their float32 scales: sx = max |x| / 127 of the row, xq =
    x / sx to the nearest whole number, ties to even. xq's rows start at
    multiples of 16 bytes (its stride can exceed its width)."""
    ldx = _matrix(x, "x")
    rows, k = x.shape
    ldq = (k + 15) // 16 * 16
    xq = torch.empty(rows, ldq, dtype=torch.int8, device=x.device)
    sx = torch.empty(rows, dtype=torch.float32, device=x.device)
    _call("experts_quantize_rows", x.device, xq.data_ptr(), ldq, sx.data_ptr(), x.data_ptr(), ldx,
          rows, k, _DTYPES[x.dtype])
    return (xq if ldq == k else xq[:, :k]), sx


def int8_matmul(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor,
                g: Groups | None = None, gather: bool = False,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """(xq wq^T) scaled by sx for rows and sw for columns. Dense without ``g``:
    wq is [n, k], sw [n]. By expert with it: wq is [experts, n, k], sw
    [experts, n], and xq and sx are per token with ``gather``, else per pair."""
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float16")
    ldq = _matrix(xq, "xq", (torch.int8,))
    device, x_rows = xq.device, xq.shape[0]
    _vector(sx, "sx", torch.float32, (x_rows,), device)
    if g is None:
        if gather:
            raise ValueError("gather needs the groups")
        ldw, stride = _matrix(wq, "wq", (torch.int8,)), 0
        if wq.device != device or wq.shape[0] == 0:
            raise ValueError(f"wq must have rows and be on {device}")
        experts, pairs, top_k, offsets, order = 1, x_rows, 1, None, None
    else:
        experts, pairs, top_k = _groups(g, device)
        ldw, stride = _weights(wq, experts, device, torch.int8)
        _rows(xq, g, pairs, gather, "xq")
        offsets, order = g.offsets.data_ptr(), g.order.data_ptr() if gather else None
    n, k = wq.shape[-2:]
    _same(xq.shape[1], k, "the last dimensions of xq and wq")
    _vector(sw, "sw", torch.float32, wq.shape[:-1], device)
    y = torch.empty(pairs, n, dtype=out_dtype, device=device)
    _call("experts_int8_matmul", device, y.data_ptr(), n, xq.data_ptr(), ldq, x_rows,
          sx.data_ptr(), wq.data_ptr(), ldw, stride, sw.data_ptr(), offsets, order, pairs, top_k,
          experts, n, k, _DTYPES[out_dtype])
    return y


def preview(product: str, rows: int, experts: int, n: int, k: int, x_rows: int = 0,
            lda: int | None = None, ldb: int | None = None, alignment: int = 16) -> Kernel:
    """The kernel that ``product`` (a key of PRODUCTS) takes for ``rows`` sorted pairs and weights
    [experts, n, k] (experts 0: the dense 8-bit product); ``x_rows``: rows of a gathered x. Needs
    no GPU. The leading dimensions default to those of contiguous operands."""
    kernel = Kernel()
    first = n if product in ("matmul_dx", "matmul_dw") else k
    _library()
    status = _functions["experts_product_preview"](
        PRODUCTS[product], rows, x_rows, experts, n, k, first if lda is None else lda,
        k if ldb is None else ldb, alignment, ctypes.byref(kernel))
    if status:
        raise hist.HistError(status, "experts_product_preview")
    return kernel


def _plain_rows(t: torch.Tensor) -> torch.Tensor:
    """A gradient as autograd hands it over can be expanded or transposed."""
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous()


class _FirstOrder(torch.autograd.Function):
    """A gradient that a kernel computed, tied to what it depends on: a second backward pass
    raises where it would have taken the gradient for a constant."""
    @staticmethod
    def forward(ctx, grad, *_):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("experts.linear and experts.merge have gradients of the first order "
                           "only")


def _first_order(grad: torch.Tensor, *depends_on: torch.Tensor) -> torch.Tensor:
    # (torch's once_differentiable looks at the incoming gradients alone, not at what was saved)
    if torch.is_grad_enabled() and any(t.requires_grad for t in depends_on):
        return _FirstOrder.apply(grad, *depends_on)
    return grad


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, gather, *g):
        ctx.save_for_backward(x, w, *g)
        ctx.gather = gather
        return matmul(x, w, Groups(*g), gather)

    @staticmethod
    def backward(ctx, dy):
        x, w, *g = ctx.saved_tensors
        g = Groups(*g)
        dy = _plain_rows(dy)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = matmul_dx(dy, w, g)
            if ctx.gather:
                # Each pair's row is rounded to 16 bits before the sum over a token's pairs, whose
                # sums are 32-bit and rounded once more: rows of 32 bits would be twice the bytes to
                # write and to read again.
                dx = combine(dx, g)
            dx = _first_order(dx, dy, w)
        if ctx.needs_input_grad[1]:
            dw = _first_order(matmul_dw(dy, x, g, ctx.gather), dy, x)
        return (dx, dw, None) + (None,) * len(g)


class _Merge(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, *g):
        ctx.save_for_backward(y, weights, *g)
        return combine(y, Groups(*g), weights)

    @staticmethod
    def backward(ctx, dout):
        y, weights, *g = ctx.saved_tensors
        g = Groups(*g)
        by = weights if weights is not None else torch.ones(
            g.place.shape, dtype=torch.float32, device=y.device)
        dy, dweights = combine_backward(_plain_rows(dout), y, g, by)
        dy = _first_order(dy, dout, by)
        dweights = None if weights is None else _first_order(dweights, dout, y)
        return (dy, dweights) + (None,) * len(g)


def linear(x: torch.Tensor, w: torch.Tensor, g: Groups, gather: bool = False) -> torch.Tensor:
    """``matmul`` with gradients for x and w. With ``gather``, x's gradient is the sum of its pairs'
    16-bit gradients: off by half a step of each of them, at most, and half a step of the sum."""
    return _Linear.apply(x, w, gather, *g)


def merge(y: torch.Tensor, g: Groups, weights: torch.Tensor | None) -> torch.Tensor:
    """``combine`` with gradients for y and the weights (if there are any)."""
    return _Merge.apply(y, weights, *g)
