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

autograd records none of these calls: a result has no grad_fn, also where its inputs
require gradients.  The _backward functions are called as they are, or from a
torch.autograd.Function of the caller's.
"""
from __future__ import annotations

import math

import torch

from . import _check, _stream, load_library

SGEMM_F32, SGEMM_BF16 = 0, 1
MAX_EXPERTS = 512  # SGEMM_MAX_EXPERTS
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORES = {"softmax": 0, "sigmoid": 1}
_DTYPES = {torch.float32: SGEMM_F32, torch.bfloat16: SGEMM_BF16}


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

_Tensor, _empty, _current_device = torch.Tensor, torch.empty, torch.cuda.current_device


def _on(stream, f, *args, **kw):
    """f on a stream other than the current one: results are allocated on it too."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream))
    with torch.cuda.stream(stream):
        return f(*args, **kw)


# The checks below run on every call, before a kernel that may take 3 us: each goes
# through its conditions once and leaves the wording of a refusal to _refuse.


def _begin(x, name):
    """The device index of the call's first tensor and its element type's code."""
    if not isinstance(x, _Tensor) or not x.is_cuda:
        raise ValueError("%s: expected a CUDA tensor, got %s" % (name, getattr(x, "device", type(x))))
    index = x.get_device()
    if index != _current_device():
        raise ValueError("%s: the tensor is on %s, the current device is cuda:%d" % (name, x.device, _current_device()))
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise ValueError("%s: expected a float32 or bfloat16 tensor, got %s" % (name, x.dtype))
    return index, code


def _matrix(x, name, rows, cols, dtype, index):
    """The row stride of x, checked to be a rows x cols matrix of the call."""
    if isinstance(x, _Tensor) and x.dtype is dtype and x.get_device() == index and x.shape == (rows, cols):
        ld, unit = x.stride()
        if (unit == 1 or cols <= 1) and ld >= cols:
            return ld if ld else 1
        if rows <= 1 and (unit == 1 or cols <= 1) or rows == 0 or cols == 0:
            return cols if cols else 1
    _refuse(x, name, (rows, cols), dtype, index)


def _packed(x, name, shape, dtype, index):
    """x checked to be a contiguous tensor of the call."""
    if not (isinstance(x, _Tensor) and x.dtype is dtype and x.get_device() == index and x.shape == shape and
            x.is_contiguous()):
        _refuse(x, name, shape, dtype, index)


def _refuse(x, name, shape, dtype, index):
    if not isinstance(x, _Tensor):
        raise ValueError("%s: expected a tensor, got %r" % (name, type(x)))
    if x.dtype != dtype:
        raise ValueError("%s: expected a %s tensor, got %s" % (name, dtype, x.dtype))
    if x.get_device() != index:
        raise ValueError("%s: expected a tensor on cuda:%d, got one on %s" % (name, index, x.device))
    if tuple(x.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(x.shape)))
    raise ValueError("%s: strides %s: the last dimension must have unit stride and rows must not overlap (vectors and "
                     "routing tensors must be contiguous)" % (name, x.stride()))


def _ptr(x):
    return None if x is None else x.data_ptr()


def _act(act):
    try:
        return ACTS[act]
    except (KeyError, TypeError):
        raise ValueError("act: %r is not one of %s" % (act, ", ".join(ACTS))) from None


def _score(score):
    try:
        return SCORES[score]
    except (KeyError, TypeError):
        raise ValueError("score: %r is not one of %s" % (score, ", ".join(SCORES))) from None


def _rows2d(x, name):
    """x as a matrix of its last dimension's rows, without copying."""
    if not isinstance(x, _Tensor):
        raise ValueError("%s: expected a tensor, got %r" % (name, type(x)))
    if x.dim() == 2:
        return x
    if x.dim() < 2:
        raise ValueError("%s: expected at least two dimensions, got shape %s" % (name, tuple(x.shape)))
    try:
        return x.view(math.prod(x.shape[:-1]), x.shape[-1])
    except RuntimeError:
        raise ValueError("%s: the leading dimensions of shape %s, strides %s do not form rows of one stride"
                         % (name, tuple(x.shape), x.stride())) from None


def _count(v, name):
    """v as the library's 32-bit integer, which would otherwise be cut off without a word."""
    v = int(v)
    if not -1 << 31 <= v < 1 << 31:
        raise ValueError("%s: %d does not fit in 32 bits" % (name, v))
    return v


def _shape(w, name, dims):
    if not isinstance(w, _Tensor) or w.dim() != dims:
        raise ValueError("%s: expected a tensor of %d dimensions" % (name, dims))
    return w.shape


def linear(x, w, bias=None, act="none", residual=None, out=None, preact=None, stream=None):
    """y = act(x w^T + bias) + residual for x (..., k), w (n, k), bias (n), residual
    (..., n); returns y (..., n).  preact=True also returns x w^T + bias, which
    linear_backward reads; a tensor given as out or preact is written instead.
    residual and out may be the same tensor."""
    if stream is not None:
        return _on(stream, linear, x, w, bias, act, residual, out, preact)
    lib = load_library()
    index, code = _begin(x, "x")
    x2 = x if x.dim() == 2 else _rows2d(x, "x")
    dtype = x.dtype
    n, k = _shape(w, "w", 2)
    t = x2.shape[0]
    ldx = _matrix(x2, "x", t, k, dtype, index)
    ldw = _matrix(w, "w", n, k, dtype, index)
    if bias is not None:
        _packed(bias, "bias", (n,), dtype, index)
    ldr = 0
    if residual is not None:
        residual = _rows2d(residual, "residual")
        ldr = _matrix(residual, "residual", t, n, dtype, index)
    if out is None:
        y, ldy = _empty((t, n), dtype=dtype, device=x.device), n or 1
    else:
        y = _rows2d(out, "out")
        ldy = _matrix(y, "out", t, n, dtype, index)
    z, ldz = None, 0
    if preact is True:
        z, ldz = _empty((t, n), dtype=dtype, device=x.device), n or 1
    elif preact is not None and preact is not False:
        z = _rows2d(preact, "preact")
        ldz = _matrix(z, "preact", t, n, dtype, index)
    rc = lib.sgemm_linear(code, t, n, k, x2.data_ptr(), ldx, w.data_ptr(), ldw, _ptr(bias), _act(act),
                          _ptr(residual), ldr, y.data_ptr(), ldy, _ptr(z), ldz, _raw_stream(index))
    if rc:
        _check(rc, lib)
    if out is not None:
        y = out
    elif x2 is not x:
        y = y.view(*x.shape[:-1], n)
    if preact is True:
        return y, z if x2 is x else z.view(*x.shape[:-1], n)
    return y


def linear_backward(dy, x, w, act="none", preact=None, bias=True, need_dx=True, need_dw=True, stream=None):
    """(dx, dw, dbias) of linear for dy (..., n), with preact as linear returned it
    (needed unless act is 'none'); dbias is None unless `bias`, dx and dw unless
    needed.  The residual's gradient is dy."""
    if stream is not None:
        return _on(stream, linear_backward, dy, x, w, act, preact, bias, need_dx, need_dw)
    lib = load_library()
    index, code = _begin(x, "x")
    x2, dy2 = _rows2d(x, "x"), _rows2d(dy, "dy")
    dtype, device = x.dtype, x.device
    n, k = _shape(w, "w", 2)
    t = x2.shape[0]
    kind = _act(act)
    lddy = _matrix(dy2, "dy", t, n, dtype, index)
    ldx = _matrix(x2, "x", t, k, dtype, index)
    ldw = _matrix(w, "w", n, k, dtype, index)
    ldz = 0
    if kind:
        if preact is None:
            raise ValueError("preact: the gradient of %r needs it" % act)
        preact = _rows2d(preact, "preact")
        ldz = _matrix(preact, "preact", t, n, dtype, index)
    else:
        preact = None
    dx = _empty((t, k), dtype=dtype, device=device) if need_dx else None
    dw = _empty((n, k), dtype=dtype, device=device) if need_dw else None
    db = _empty((n,), dtype=dtype, device=device) if bias else None
    rc = lib.sgemm_linear_backward(code, t, n, k, dy2.data_ptr(), lddy, x2.data_ptr(), ldx, w.data_ptr(), ldw, kind,
                                   _ptr(preact), ldz, _ptr(dx), k or 1, _ptr(dw), k or 1, _ptr(db), _raw_stream(index))
    if rc:
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
    if stream is not None:
        return _on(stream, route, logits, top, score, bias, groups, group_top, renormalize, scale, mask)
    lib = load_library()
    index, code = _begin(logits, "logits")
    device = logits.device
    t, e = _shape(logits, "logits", 2)
    ldl = _matrix(logits, "logits", t, e, logits.dtype, index)
    if bias is not None:
        _packed(bias, "bias", (e,), torch.float32, index)
    if mask is not None:
        _packed(mask, "mask", (t,), torch.bool, index)
    top, groups, group_top = _count(top, "top"), _count(groups, "groups"), _count(group_top, "group_top")
    shape = (t, top if 0 < top <= e else 0)  # the library refuses any other top
    weights = _empty(shape, dtype=torch.float32, device=device)
    ids = _empty(shape, dtype=torch.int32, device=device)
    rc = lib.sgemm_route(code, t, e, top, logits.data_ptr(), ldl, _score(score), _ptr(bias), groups, group_top,
                         1 if renormalize else 0, scale, _ptr(mask), weights.data_ptr(), ids.data_ptr(),
                         _raw_stream(index))
    if rc:
        _check(rc, lib)
    return weights, ids


def route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits of route's weights for dweights (tokens, top), the choice ids held."""
    if stream is not None:
        return _on(stream, route_backward, dweights, logits, ids, score, renormalize, scale)
    lib = load_library()
    index, code = _begin(logits, "logits")
    t, e = _shape(logits, "logits", 2)
    top = _shape(ids, "ids", 2)[1]
    ldl = _matrix(logits, "logits", t, e, logits.dtype, index)
    _packed(dweights, "dweights", (t, top), torch.float32, index)
    _packed(ids, "ids", (t, top), torch.int32, index)
    dlogits = _empty((t, e), dtype=logits.dtype, device=logits.device)
    rc = lib.sgemm_route_backward(code, t, e, top, dweights.data_ptr(), logits.data_ptr(), ldl, ids.data_ptr(),
                                  _score(score), 1 if renormalize else 0, scale, dlogits.data_ptr(), e or 1,
                                  _raw_stream(index))
    if rc:
        _check(rc, lib)
    return dlogits


class ExpertPlan:
    """The experts' row lists (int32 tensors): counts (experts), offsets (experts + 1),
    rows (tokens * top: the pair token * top + choice of each row, -1 for rows of no
    expert) and slots (tokens, top: the row of each pair, -1 where its id names no
    expert).  expert_plan makes one; one can also be made of four such tensors, where an
    entry of rows inside an expert's list may name no pair (-1): gathered, it reads as zeros."""

    __slots__ = ("tokens", "top", "experts", "index", "_store", "_lists", "_addresses")

    def __init__(self, counts, offsets, rows, slots):
        tokens, top = _shape(slots, "slots", 2)
        if not slots.is_cuda:
            raise ValueError("slots: expected a CUDA tensor, got one on %s" % slots.device)
        experts, index = _shape(counts, "counts", 1)[0], slots.get_device()
        for x, name, shape in ((counts, "counts", (experts,)), (offsets, "offsets", (experts + 1,)),
                               (rows, "rows", (tokens * top,)), (slots, "slots", (tokens, top))):
            _packed(x, name, shape, torch.int32, index)
        self.tokens, self.top, self.experts, self.index = tokens, top, experts, index
        self._store, self._lists = None, [counts, offsets, rows, slots]
        self._addresses = tuple(x.data_ptr() for x in self._lists)

    @classmethod
    def _of(cls, store, address, tokens, top, experts, index):
        """The lists one after another in `store`; their tensors are made when asked for."""
        self = cls.__new__(cls)
        self.tokens, self.top, self.experts, self.index = tokens, top, experts, index
        self._store, self._lists = store, [None] * 4
        rows = address + 4 * (2 * experts + 1)
        self._addresses = (address, address + 4 * experts, rows, rows + 4 * tokens * top)
        return self

    def _list(self, i):
        x = self._lists[i]
        if x is None:
            e, r = self.experts, self.tokens * self.top
            at = (0, e, 2 * e + 1, 2 * e + 1 + r)[i]
            if i == 3:
                x = self._store.as_strided((self.tokens, self.top), (self.top, 1), at)
            else:
                x = self._store.as_strided(((e, e + 1, r)[i],), (1,), at)
            self._lists[i] = x
        return x

    counts = property(lambda self: self._list(0))
    offsets = property(lambda self: self._list(1))
    rows = property(lambda self: self._list(2))
    slots = property(lambda self: self._list(3))


def expert_plan(ids, experts, stream=None):
    """The row lists of ids (tokens, top): an expert's rows hold its pairs in order.
    The four lists lie in one allocation."""
    if stream is not None:
        return _on(stream, expert_plan, ids, experts)
    lib = load_library()
    t, top = _shape(ids, "ids", 2)
    if not ids.is_cuda:
        raise ValueError("ids: expected a CUDA tensor, got one on %s" % ids.device)
    index = _current_device()
    _packed(ids, "ids", (t, top), torch.int32, index)
    experts = _count(experts, "experts")
    if experts < 1:
        raise ValueError("experts: %d is less than 1" % experts)
    # more experts than SGEMM_MAX_EXPERTS are the library's to refuse, before it writes a list
    store = _empty((2 * min(experts, MAX_EXPERTS) + 1 + 2 * t * top,), dtype=torch.int32, device=ids.device)
    plan = ExpertPlan._of(store, store.data_ptr(), t, top, experts, index)
    rc = lib.sgemm_expert_plan(t, top, experts, ids.data_ptr(), *plan._addresses, _raw_stream(index))
    if rc:
        _check(rc, lib)
    return plan


def _plan_sizes(plan, experts, index):
    """tokens and top of a plan of the call's device, for `experts` experts (any when None)."""
    if not isinstance(plan, ExpertPlan):
        raise ValueError("plan: expected an ExpertPlan, got %r" % type(plan))
    if plan.index != index:
        raise ValueError("plan: its lists are on cuda:%d, the call is on cuda:%d" % (plan.index, index))
    if experts is not None and plan.experts != experts:
        raise ValueError("plan: made for %d experts, the weights are of %d" % (plan.experts, experts))
    return plan.tokens, plan.top


def _expert_weights(w, dtype, index):
    """experts, n, k, the row stride and the stride between experts of w."""
    e, n, k = _shape(w, "w", 3)
    if w.dtype is dtype and w.get_device() == index:
        stride, ld, unit = w.stride()
        if n <= 1 or w.numel() == 0:
            ld = k or 1
        if (unit == 1 or k <= 1 or w.numel() == 0) and ld >= k:
            return e, n, k, ld, stride if e > 1 and w.numel() else n * ld
    _refuse(w, "w", (e, n, k), dtype, index)


def expert_linear(x, w, plan, bias=None, act="none", gather=False, out=None, preact=None, stream=None):
    """Rows r of expert e's list: act(w[e] x[r'] + bias[e]) for w (experts, n, k) and
    bias (experts, n), where r' is the row's token (gather=True, x (tokens, k)) or r
    itself (x (tokens * top, k)).  Returns (tokens * top, n) in the plan's row order,
    rows of no expert zero; preact and out are as in linear."""
    if stream is not None:
        return _on(stream, expert_linear, x, w, plan, bias, act, gather, out, preact)
    lib = load_library()
    index, code = _begin(x, "x")
    dtype = x.dtype
    e, n, k, ldw, stride = _expert_weights(w, dtype, index)
    t, top = _plan_sizes(plan, e, index)
    rows = t * top
    ldx = _matrix(x, "x", t if gather else rows, k, dtype, index)
    if bias is not None:
        _packed(bias, "bias", (e, n), dtype, index)
    if out is None:
        y, ldy = _empty((rows, n), dtype=dtype, device=x.device), n or 1
    else:
        y, ldy = out, _matrix(out, "out", rows, n, dtype, index)
    z, ldz = None, 0
    if preact is True:
        z, ldz = _empty((rows, n), dtype=dtype, device=x.device), n or 1
    elif preact is not None and preact is not False:
        z, ldz = preact, _matrix(preact, "preact", rows, n, dtype, index)
    rc = lib.sgemm_expert_linear(code, t, top, e, n, k, 1 if gather else 0, x.data_ptr(), ldx, w.data_ptr(), ldw,
                                 stride, _ptr(bias), _act(act), plan._addresses[1], plan._addresses[2],
                                 y.data_ptr(), ldy, _ptr(z), ldz, _raw_stream(index))
    if rc:
        _check(rc, lib)
    return (y, z) if preact is True else y


def expert_linear_backward(dy, x, w, plan, act="none", preact=None, bias=True, gather=False, need_dx=True,
                           need_dw=True, stream=None):
    """(dx, dw, dbias) of expert_linear for dy (tokens * top, n).  With gather, dx
    (tokens, k) is the sum over the token's rows."""
    if stream is not None:
        return _on(stream, expert_linear_backward, dy, x, w, plan, act, preact, bias, gather, need_dx, need_dw)
    lib = load_library()
    index, code = _begin(x, "x")
    dtype, device = x.dtype, x.device
    e, n, k, ldw, stride = _expert_weights(w, dtype, index)
    t, top = _plan_sizes(plan, e, index)
    rows = t * top
    kind = _act(act)
    lddy = _matrix(dy, "dy", rows, n, dtype, index)
    ldx = _matrix(x, "x", t if gather else rows, k, dtype, index)
    ldz = 0
    if kind:
        if preact is None:
            raise ValueError("preact: the gradient of %r needs it" % act)
        ldz = _matrix(preact, "preact", rows, n, dtype, index)
    else:
        preact = None
    dx = _empty((t if gather else rows, k), dtype=dtype, device=device) if need_dx else None
    dw = _empty((e, n, k), dtype=dtype, device=device) if need_dw else None
    db = _empty((e, n), dtype=dtype, device=device) if bias else None
    rc = lib.sgemm_expert_linear_backward(
        code, t, top, e, n, k, 1 if gather else 0, dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), ldw, stride,
        kind, _ptr(preact), ldz, *plan._addresses[1:], _ptr(dx), k or 1, _ptr(dw), k or 1, n * (k or 1), _ptr(db), _raw_stream(index))
    if rc:
        _check(rc, lib)
    return dx, dw, db


def expert_combine(rows, plan, weights=None, residual=None, out=None, stream=None):
    """y (tokens, n) = residual + the sum over the token's choices of weights
    (tokens, top, float32; ones when None) times its rows (tokens * top, n)."""
    if stream is not None:
        return _on(stream, expert_combine, rows, plan, weights, residual, out)
    lib = load_library()
    index, code = _begin(rows, "rows")
    dtype = rows.dtype
    t, top = _plan_sizes(plan, None, index)
    n = _shape(rows, "rows", 2)[1]
    ldx = _matrix(rows, "rows", t * top, n, dtype, index)
    if weights is not None:
        _packed(weights, "weights", (t, top), torch.float32, index)
    ldr = _matrix(residual, "residual", t, n, dtype, index) if residual is not None else 0
    if out is None:
        y, ldy = _empty((t, n), dtype=dtype, device=rows.device), n or 1
    else:
        y, ldy = out, _matrix(out, "out", t, n, dtype, index)
    rc = lib.sgemm_expert_combine(code, t, top, n, rows.data_ptr(), ldx, plan._addresses[3], _ptr(weights),
                                  _ptr(residual), ldr, y.data_ptr(), ldy, _raw_stream(index))
    if rc:
        _check(rc, lib)
    return y


def expert_combine_backward(dy, rows, plan, weights=None, need_dweights=True, stream=None):
    """(drows, dweights) of expert_combine for dy (tokens, n); dweights is None unless
    needed.  The residual's gradient is dy."""
    if stream is not None:
        return _on(stream, expert_combine_backward, dy, rows, plan, weights, need_dweights)
    lib = load_library()
    index, code = _begin(rows, "rows")
    dtype, device = rows.dtype, rows.device
    t, top = _plan_sizes(plan, None, index)
    n = _shape(rows, "rows", 2)[1]
    ldx = _matrix(rows, "rows", t * top, n, dtype, index)
    lddy = _matrix(dy, "dy", t, n, dtype, index)
    if weights is not None:
        _packed(weights, "weights", (t, top), torch.float32, index)
    drows = _empty((t * top, n), dtype=dtype, device=device)
    dweights = _empty((t, top), dtype=torch.float32, device=device) if need_dweights else None
    rc = lib.sgemm_expert_combine_backward(code, t, top, n, dy.data_ptr(), lddy, rows.data_ptr(), ldx,
                                           plan._addresses[2], plan._addresses[3], _ptr(weights),
                                           drows.data_ptr(), n or 1, _ptr(dweights), _raw_stream(index))
    if rc:
        _check(rc, lib)
    return drows, dweights
