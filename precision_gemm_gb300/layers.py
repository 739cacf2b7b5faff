"""Layers of language models on the library's kernels: linear layers with a fused
epilogue, routing to experts, the experts' products, and their backward passes.

The functions mirror the ``sgemm_linear``, ``sgemm_route`` and ``sgemm_expert_*``
declarations of ``include/precision_gemm.h``: they check tensors, allocate results
and call the library; all arithmetic runs in its kernels.

    y             = linear(x, w, bias, act, residual)           act(x w^T + bias) + residual
    dx, dw, dbias = linear_backward(dy, x, w, act, preact)
    weights, ids  = route(logits, top, score, ...)
    dlogits       = route_backward(dweights, logits, ids, score, ...)
    plan          = expert_plan(ids, experts)                    the experts' row lists
    h             = expert_linear(x, w, plan, bias, act, gather=True)
    dx, dw, dbias = expert_linear_backward(dy, x, w, plan, act, preact, gather=True)
    y             = expert_combine(rows, plan, weights, residual)
    drows, dweights = expert_combine_backward(dy, rows, plan, weights)

Tensors are float32 or bfloat16 (one type per call) on the current CUDA device,
with a last dimension of unit stride and rows at any stride that does not overlap
them.  Sums, scores and routing weights are FP32.  `act` is 'none', 'relu',
'silu', 'gelu' or 'gelu_tanh'.  Work is queued on `stream` (torch's current stream
when None); results are allocated on that stream.  Tensors that were made on another
stream must be ready on it and stay alive until its work is done, as for any
asynchronous call.  A bad tensor raises ValueError before the library is called,
a failed call SgemmError.
"""
from __future__ import annotations

import torch

from . import _check, _stream, load_library

SGEMM_F32, SGEMM_BF16 = 0, 1
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
_DTYPES = {torch.float32: SGEMM_F32, torch.bfloat16: SGEMM_BF16}


class _Call:
    """The stream of one call, the device its tensors must be on, and its element
    type; allocations inside `with` belong to the stream."""

    __slots__ = ("handle", "device", "index", "dtype", "code", "_other")

    def __init__(self, stream, first, name, dtype=None):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError("%s: expected a CUDA tensor" % name)
        self.device = first.device
        self.index = first.get_device()
        if self.index != torch.cuda.current_device():
            raise ValueError("%s: the tensor is on %s, the current device is cuda:%d"
                             % (name, first.device, torch.cuda.current_device()))
        self.dtype = first.dtype if dtype is None else dtype
        self.code = _DTYPES.get(self.dtype)
        if self.code is None:
            raise ValueError("%s: expected a float32 or bfloat16 tensor, got %s" % (name, first.dtype))
        self._other = None
        if stream is None:
            self.handle = torch.cuda.current_stream(self.index).cuda_stream
        else:
            self.handle = _stream(stream)
            if self.handle != torch.cuda.current_stream(self.index).cuda_stream:
                self._other = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(self.handle)

    def empty(self, *shape, dtype=None):
        if self._other is None:
            return torch.empty(shape, dtype=self.dtype if dtype is None else dtype, device=self.device)
        with torch.cuda.stream(self._other):
            return torch.empty(shape, dtype=self.dtype if dtype is None else dtype, device=self.device)

    def tensor(self, x, name, shape, dtype=None, packed=False):
        """x checked to be a tensor of this call with the given shape; its row stride
        (its last dimension has unit stride, all of it when packed)."""
        if not isinstance(x, torch.Tensor):
            raise ValueError("%s: expected a tensor, got %r" % (name, type(x)))
        if x.dtype != (self.dtype if dtype is None else dtype):
            raise ValueError("%s: expected a %s tensor, got %s" % (name, dtype or self.dtype, x.dtype))
        if x.get_device() != self.index:
            raise ValueError("%s: expected a tensor on %s, got one on %s" % (name, self.device, x.device))
        if tuple(x.shape) != shape:
            raise ValueError("%s: expected shape %s, got %s" % (name, shape, tuple(x.shape)))
        if packed:
            if not x.is_contiguous():
                raise ValueError("%s: the tensor must be contiguous" % name)
            return shape[-1] if shape else 1
        cols = shape[-1]
        if cols > 1 and x.numel() > 0 and x.stride(-1) != 1:
            raise ValueError("%s: the last dimension must have unit stride" % name)
        if len(shape) < 2 or shape[-2] <= 1 or x.numel() == 0:
            return max(cols, 1)
        ld = x.stride(-2)
        if ld < cols:
            raise ValueError("%s: rows must not overlap (row stride %d, %d columns)" % (name, ld, cols))
        return ld


def _ptr(x):
    return None if x is None else x.data_ptr()


def _act(act):
    try:
        return ACTS[act]
    except KeyError:
        raise ValueError("act: %r is not one of %s" % (act, ", ".join(ACTS))) from None


def _score(score):
    try:
        return SCORES[score]
    except KeyError:
        raise ValueError("score: %r is not one of %s" % (score, ", ".join(SCORES))) from None


def _rows2d(x, name):
    """x as a matrix of its last dimension's rows, without copying."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("%s: expected a tensor, got %r" % (name, type(x)))
    if x.dim() == 2:
        return x
    if x.dim() < 2:
        raise ValueError("%s: expected at least two dimensions, got shape %s" % (name, tuple(x.shape)))
    try:
        return x.view(-1, x.shape[-1])
    except RuntimeError:
        raise ValueError("%s: the leading dimensions of shape %s, strides %s do not form rows of one stride"
                         % (name, tuple(x.shape), x.stride())) from None


def _matrix_shape(w, name, dims):
    if not isinstance(w, torch.Tensor) or w.dim() != dims:
        raise ValueError("%s: expected a tensor of %d dimensions" % (name, dims))
    return tuple(w.shape)


def _result(c, given, name, shape):
    """The caller's tensor for a result, or a new one; and its row stride."""
    if given is None:
        return c.empty(*shape), max(shape[-1], 1)
    return given, c.tensor(given, name, shape)


def linear(x, w, bias=None, act="none", residual=None, out=None, preact=None, stream=None):
    """y = act(x w^T + bias) + residual for x (..., k), w (n, k), bias (n), residual
    (..., n); returns y (..., n).  preact=True also returns x w^T + bias, which
    linear_backward reads; a tensor given as out or preact is written instead.
    residual and out may be the same tensor."""
    lib = load_library()
    x2 = _rows2d(x, "x")
    c = _Call(stream, x2, "x")
    n, k = _matrix_shape(w, "w", 2)
    t = x2.shape[0]
    ldx = c.tensor(x2, "x", (t, k))
    ldw = c.tensor(w, "w", (n, k))
    if bias is not None:
        c.tensor(bias, "bias", (n,), packed=True)
    ldr = 0
    if residual is not None:
        residual = _rows2d(residual, "residual")
        ldr = c.tensor(residual, "residual", (t, n))
    y, ldy = _result(c, None if out is None else _rows2d(out, "out"), "out", (t, n))
    z, ldz = None, 0
    if preact is not None and preact is not False:
        z, ldz = _result(c, None if preact is True else _rows2d(preact, "preact"), "preact", (t, n))
    rc = lib.sgemm_linear(c.code, t, n, k, x2.data_ptr(), ldx, w.data_ptr(), ldw, _ptr(bias), _act(act),
                          _ptr(residual), ldr, y.data_ptr(), ldy, _ptr(z), ldz, c.handle)
    _check(rc, lib)
    y = (y if x.dim() == 2 else y.view(*x.shape[:-1], n)) if out is None else out
    if preact is True:
        return y, z if x.dim() == 2 else z.view(*x.shape[:-1], n)
    return y


def linear_backward(dy, x, w, act="none", preact=None, bias=True, need_dx=True, need_dw=True, stream=None):
    """(dx, dw, dbias) of linear for dy (..., n), with preact as linear returned it
    (needed unless act is 'none'); dbias is None unless `bias`, dx and dw unless
    needed.  The residual's gradient is dy."""
    lib = load_library()
    x2, dy2 = _rows2d(x, "x"), _rows2d(dy, "dy")
    c = _Call(stream, x2, "x")
    n, k = _matrix_shape(w, "w", 2)
    t = x2.shape[0]
    code = _act(act)
    lddy = c.tensor(dy2, "dy", (t, n))
    ldx = c.tensor(x2, "x", (t, k))
    ldw = c.tensor(w, "w", (n, k))
    ldz = 0
    if code:
        if preact is None:
            raise ValueError("preact: the gradient of %r needs it" % act)
        preact = _rows2d(preact, "preact")
        ldz = c.tensor(preact, "preact", (t, n))
    else:
        preact = None
    dx = c.empty(t, k) if need_dx else None
    dw = c.empty(n, k) if need_dw else None
    db = c.empty(n) if bias else None
    rc = lib.sgemm_linear_backward(c.code, t, n, k, dy2.data_ptr(), lddy, x2.data_ptr(), ldx, w.data_ptr(), ldw, code,
                                   _ptr(preact), ldz, _ptr(dx), max(k, 1), _ptr(dw), max(k, 1), _ptr(db), c.handle)
    _check(rc, lib)
    if dx is not None and x.dim() != 2:
        dx = dx.view(x.shape)
    return dx, dw, db


def route(logits, top, score="softmax", bias=None, groups=1, group_top=1, renormalize=True, scale=1.0, mask=None,
          stream=None):
    """(weights, ids), both (tokens, top), of logits (tokens, experts): the `top`
    experts of the best score + bias, best first, and their scores (divided by their
    sum when renormalize, times scale).  bias (experts, float32) steers the choice
    alone; with groups > 1 only the group_top best groups of experts are considered,
    a group scoring the sum of its two best.  Ties go to the lower index.  Tokens
    with mask False (tokens, bool) get ids of -1 and weights of zero."""
    lib = load_library()
    c = _Call(stream, logits, "logits")
    t, e = _matrix_shape(logits, "logits", 2)
    ldl = c.tensor(logits, "logits", (t, e))
    if bias is not None:
        c.tensor(bias, "bias", (e,), torch.float32, packed=True)
    if mask is not None:
        c.tensor(mask, "mask", (t,), torch.bool, packed=True)
    top = int(top)
    weights = c.empty(t, max(top, 0), dtype=torch.float32)
    ids = c.empty(t, max(top, 0), dtype=torch.int32)
    rc = lib.sgemm_route(c.code, t, e, top, logits.data_ptr(), ldl, _score(score), _ptr(bias), groups, group_top,
                         1 if renormalize else 0, scale, _ptr(mask), weights.data_ptr(), ids.data_ptr(), c.handle)
    _check(rc, lib)
    return weights, ids


def route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits of route's weights for dweights (tokens, top), the choice ids held."""
    lib = load_library()
    c = _Call(stream, logits, "logits")
    t, e = _matrix_shape(logits, "logits", 2)
    top = _matrix_shape(ids, "ids", 2)[1]
    ldl = c.tensor(logits, "logits", (t, e))
    c.tensor(dweights, "dweights", (t, top), torch.float32, packed=True)
    c.tensor(ids, "ids", (t, top), torch.int32, packed=True)
    dlogits = c.empty(t, e)
    rc = lib.sgemm_route_backward(c.code, t, e, top, dweights.data_ptr(), logits.data_ptr(), ldl, ids.data_ptr(),
                                  _score(score), 1 if renormalize else 0, scale, dlogits.data_ptr(), max(e, 1),
                                  c.handle)
    _check(rc, lib)
    return dlogits


class ExpertPlan:
    """The experts' row lists (int32 tensors): counts (experts), offsets (experts + 1),
    rows (tokens * top: the pair token * top + choice of each row, -1 for rows of no
    expert) and slots (tokens, top: the row of each pair, -1 where its id names no
    expert)."""

    __slots__ = ("counts", "offsets", "rows", "slots")

    def __init__(self, counts, offsets, rows, slots):
        self.counts, self.offsets, self.rows, self.slots = counts, offsets, rows, slots


def expert_plan(ids, experts, stream=None):
    """The row lists of ids (tokens, top): an expert's rows hold its pairs in order."""
    lib = load_library()
    t, top = _matrix_shape(ids, "ids", 2)
    c = _Call(stream, ids, "ids", torch.float32)
    c.tensor(ids, "ids", (t, top), torch.int32, packed=True)
    counts, offsets = c.empty(experts, dtype=torch.int32), c.empty(experts + 1, dtype=torch.int32)
    rows, slots = c.empty(t * top, dtype=torch.int32), c.empty(t, top, dtype=torch.int32)
    rc = lib.sgemm_expert_plan(t, top, experts, ids.data_ptr(), counts.data_ptr(), offsets.data_ptr(),
                               rows.data_ptr(), slots.data_ptr(), c.handle)
    _check(rc, lib)
    return ExpertPlan(counts, offsets, rows, slots)


def _plan_sizes(c, plan, experts):
    if not isinstance(plan, ExpertPlan):
        raise ValueError("plan: expected an ExpertPlan, got %r" % type(plan))
    t, top = _matrix_shape(plan.slots, "plan.slots", 2)
    c.tensor(plan.slots, "plan.slots", (t, top), torch.int32, packed=True)
    c.tensor(plan.rows, "plan.rows", (t * top,), torch.int32, packed=True)
    if experts is not None:
        c.tensor(plan.offsets, "plan.offsets", (experts + 1,), torch.int32, packed=True)
    return t, top


def _expert_weights(c, w, name="w"):
    e, n, k = _matrix_shape(w, name, 3)
    ld = c.tensor(w, name, (e, n, k))
    stride = w.stride(0) if e > 1 else n * ld
    return e, n, k, ld, stride


def expert_linear(x, w, plan, bias=None, act="none", gather=False, out=None, preact=None, stream=None):
    """Rows r of expert e's list: act(w[e] x[r'] + bias[e]) for w (experts, n, k) and
    bias (experts, n), where r' is the row's token (gather=True, x (tokens, k)) or r
    itself (x (tokens * top, k)).  Returns (tokens * top, n) in the plan's row order,
    rows of no expert zero; preact and out are as in linear."""
    lib = load_library()
    c = _Call(stream, x, "x")
    e, n, k, ldw, stride = _expert_weights(c, w)
    t, top = _plan_sizes(c, plan, e)
    rows = t * top
    ldx = c.tensor(x, "x", (t if gather else rows, k))
    if bias is not None:
        c.tensor(bias, "bias", (e, n), packed=True)
    y, ldy = _result(c, out, "out", (rows, n))
    z, ldz = None, 0
    if preact is not None and preact is not False:
        z, ldz = _result(c, None if preact is True else preact, "preact", (rows, n))
    rc = lib.sgemm_expert_linear(c.code, t, top, e, n, k, 1 if gather else 0, x.data_ptr(), ldx, w.data_ptr(), ldw,
                                 stride, _ptr(bias), _act(act), plan.offsets.data_ptr(), plan.rows.data_ptr(),
                                 y.data_ptr(), ldy, _ptr(z), ldz, c.handle)
    _check(rc, lib)
    return (y, z) if preact is True else y


def expert_linear_backward(dy, x, w, plan, act="none", preact=None, bias=True, gather=False, need_dx=True,
                           need_dw=True, stream=None):
    """(dx, dw, dbias) of expert_linear for dy (tokens * top, n).  With gather, dx
    (tokens, k) is the sum over the token's rows."""
    lib = load_library()
    c = _Call(stream, x, "x")
    e, n, k, ldw, stride = _expert_weights(c, w)
    t, top = _plan_sizes(c, plan, e)
    rows = t * top
    code = _act(act)
    lddy = c.tensor(dy, "dy", (rows, n))
    ldx = c.tensor(x, "x", (t if gather else rows, k))
    ldz = 0
    if code:
        if preact is None:
            raise ValueError("preact: the gradient of %r needs it" % act)
        ldz = c.tensor(preact, "preact", (rows, n))
    else:
        preact = None
    dx = c.empty(t if gather else rows, k) if need_dx else None
    dw = c.empty(e, n, k) if need_dw else None
    db = c.empty(e, n) if bias else None
    rc = lib.sgemm_expert_linear_backward(
        c.code, t, top, e, n, k, 1 if gather else 0, dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), ldw, stride,
        code, _ptr(preact), ldz, plan.offsets.data_ptr(), plan.rows.data_ptr(), plan.slots.data_ptr(), _ptr(dx),
        max(k, 1), _ptr(dw), max(k, 1), n * max(k, 1), _ptr(db), c.handle)
    _check(rc, lib)
    return dx, dw, db


def expert_combine(rows, plan, weights=None, residual=None, out=None, stream=None):
    """y (tokens, n) = residual + the sum over the token's choices of weights
    (tokens, top, float32; ones when None) times its rows (tokens * top, n)."""
    lib = load_library()
    c = _Call(stream, rows, "rows")
    t, top = _plan_sizes(c, plan, None)
    n = _matrix_shape(rows, "rows", 2)[1]
    ldx = c.tensor(rows, "rows", (t * top, n))
    if weights is not None:
        c.tensor(weights, "weights", (t, top), torch.float32, packed=True)
    ldr = c.tensor(residual, "residual", (t, n)) if residual is not None else 0
    y, ldy = _result(c, out, "out", (t, n))
    rc = lib.sgemm_expert_combine(c.code, t, top, n, rows.data_ptr(), ldx, plan.slots.data_ptr(), _ptr(weights),
                                  _ptr(residual), ldr, y.data_ptr(), ldy, c.handle)
    _check(rc, lib)
    return y


def expert_combine_backward(dy, rows, plan, weights=None, need_dweights=True, stream=None):
    """(drows, dweights) of expert_combine for dy (tokens, n); dweights is None unless
    needed.  The residual's gradient is dy."""
    lib = load_library()
    c = _Call(stream, rows, "rows")
    t, top = _plan_sizes(c, plan, None)
    n = _matrix_shape(rows, "rows", 2)[1]
    ldx = c.tensor(rows, "rows", (t * top, n))
    lddy = c.tensor(dy, "dy", (t, n))
    if weights is not None:
        c.tensor(weights, "weights", (t, top), torch.float32, packed=True)
    drows = c.empty(t * top, n)
    dweights = c.empty(t, top, dtype=torch.float32) if need_dweights else None
    rc = lib.sgemm_expert_combine_backward(c.code, t, top, n, dy.data_ptr(), lddy, rows.data_ptr(), ldx,
                                           plan.rows.data_ptr(), plan.slots.data_ptr(), _ptr(weights),
                                           drows.data_ptr(), max(n, 1), _ptr(dweights), c.handle)
    _check(rc, lib)
    return drows, dweights
