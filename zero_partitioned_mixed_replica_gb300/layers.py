"""The operators at a model's ends and between its blocks: embedding, layer
norm, and the language-model head with its loss, with their gradients.

A step of :class:`.engine.ZeroStep` or :class:`.multi.MultiAdamW` begins where
backward has left the weight gradients: in a rank's flat 16-bit replica, or in
a list of tensors.  The ``*_backward`` functions here write them there, into
any tensor that the caller gives (``engine.tensor_view(engine.grads[r], t,
shape)``), overwriting it or adding to it; what else they return is new.

Each operator comes in two forms.  The ``*_forward`` and ``*_backward`` functions
are the library's calls: nothing is recorded, and they can be captured into a
CUDA graph.  :func:`embedding`, :func:`layer_norm` and :func:`lm_loss` are
differentiable by torch's autograd.

All of them run on torch's current stream of the tensors' device and allocate
their workspace from torch's allocator for the call.  Inputs may have any
number of leading dimensions and any strides (rows that are not evenly spaced
with contiguous elements are copied first); gradients that are written in
place are contiguous.  Formulas, ranges and what happens at their edges:
``include/zero.h``.
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple, Union

import torch

from . import binding as B
from .multi import _GRAD as DTYPE
from .multi import _current_device, _raw_stream

_FP32 = torch.float32
_empty = torch.empty         # half the time of a tensor's new_empty


# A short call costs the host more than the GPU: each function looks at its arguments in one condition, and only where
# that does not hold says which one is wrong.
def _shape(t: torch.Tensor) -> str:
    return "x".join(map(str, t.shape)) or "scalar"


def _check_on(device: torch.device, **tensors) -> None:
    """All on one CUDA device; the messages name the first that is not."""
    for name, t in tensors.items():
        if t is not None and (t.device != device or t.device.type != "cuda"):
            raise ValueError("%s is on %s: the call's tensors are on one CUDA device" % (name, t.device))


def _check_dtype(name: str, t: torch.Tensor, *dtypes: torch.dtype) -> None:
    if t.dtype not in (dtypes or DTYPE):
        raise ValueError("%s: dtype %s (need %s)" % (name, t.dtype, " or ".join(map(str, dtypes or DTYPE))))


def _check_weight(name: str, t: torch.Tensor, shape) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: shape %s (need %s)" % (name, _shape(t), "x".join(map(str, shape))))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % name)


def _check_dims(name: str, t: torch.Tensor, dims: int) -> None:
    if t.dim() != dims:
        raise ValueError("%s: shape %s (need %s)" % (name, _shape(t), "vocab x d" if dims == 2 else "one dimension"))


def _check_last(name: str, t: torch.Tensor, d: int) -> None:
    if t.dim() < 1 or t.shape[-1] != d:
        raise ValueError("%s: shape %s (need %d in the last dimension)" % (name, _shape(t), d))


def _like(t: Optional[torch.Tensor], shape, dtype, index) -> bool:
    return t is None or (t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous())


def _rows(t: torch.Tensor, d: int) -> Tuple[torch.Tensor, int]:
    """(t as rows of d, elements between rows); a copy where t is not evenly
    spaced rows of contiguous elements."""
    if t.is_contiguous():
        return t, d
    if t.dim() != 2:
        t = t.reshape(-1, d)
        if t.is_contiguous():
            return t, d
    stride = d if t.shape[0] <= 1 else t.stride(0)
    if (d > 1 and t.stride(1) != 1) or stride < d:
        return t.contiguous(), d
    return t, stride


_embedding_workspace = lru_cache(maxsize=256)(B.zero_embedding_workspace)
_norm_workspace = lru_cache(maxsize=256)(B.zero_layer_norm_workspace)


def _no_capture(*tensors) -> None:
    """Autograd under capture is refused: torch's backward ends the process
    when the leaves also belong to a graph that was recorded outside."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors) \
            and torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("inside a CUDA graph capture use the *_forward and *_backward functions")


# -- embedding -------------------------------------------------------------------------------------------
def embedding_forward(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """``scale * weight[ids]``: weight [vocab, d], ids int64 of any shape; a
    new tensor of ids' shape with d behind it.  An id outside 0 .. vocab-1
    (padding) gives zeros."""
    index, code = weight.get_device(), DTYPE.get(weight.dtype)
    if not (index >= 0 and code is not None and weight.dim() == 2 and weight.is_contiguous() and ids.dtype is torch.int64 and
            ids.get_device() == index):
        _check_dims("weight", weight, 2)
        _check_weight("weight", weight, weight.shape)
        _check_dtype("weight", weight)
        _check_dtype("ids", ids, torch.int64)
        _check_on(weight.device, weight=weight, ids=ids)
    if _current_device() != index:
        with torch.cuda.device(index):
            return embedding_forward(weight, ids, scale)
    vocab, d = weight.shape
    flat = ids.contiguous()
    out = _empty((*ids.shape, d), dtype=weight.dtype, device=index)
    status = B.lib().zero_embedding_forward(weight.data_ptr(), flat.data_ptr(), vocab, d, flat.numel(), code, scale,
                                            out.data_ptr(), _raw_stream(index))
    if status:
        B._check(status)
    return out


def embedding_backward(grad_out: torch.Tensor, ids: torch.Tensor, grad_weight: torch.Tensor, scale: float = 1.0,
                       accumulate: bool = False) -> torch.Tensor:
    """The weight's gradient into ``grad_weight`` [vocab, d] (grad_out's dtype
    or float32): row k gets ``scale`` times the sum of the rows of
    ``grad_out`` whose id is k, the others zeros; with ``accumulate`` that is
    added to what is there.  The same inputs give the same bits."""
    index, dtype = grad_weight.get_device(), grad_out.dtype
    code, to = DTYPE.get(dtype), grad_weight.dtype
    if not (index >= 0 and code is not None and grad_weight.dim() == 2 and grad_weight.is_contiguous() and
            (to is dtype or to is _FP32) and ids.dtype is torch.int64 and ids.get_device() == index and
            grad_out.get_device() == index and grad_out.shape == (*ids.shape, grad_weight.shape[1])):
        _check_dims("grad_weight", grad_weight, 2)
        _check_dtype("grad_out", grad_out)
        _check_weight("grad_weight", grad_weight, grad_weight.shape)
        _check_dtype("grad_weight", grad_weight, dtype, _FP32)
        _check_dtype("ids", ids, torch.int64)
        if tuple(grad_out.shape) != (*ids.shape, grad_weight.shape[1]):
            raise ValueError("grad_out: shape %s (need %s)" % (_shape(grad_out), "x".join(map(str, (*ids.shape, grad_weight.shape[1])))))
        _check_on(grad_weight.device, grad_weight=grad_weight, grad_out=grad_out, ids=ids)
    if _current_device() != index:
        with torch.cuda.device(index):
            return embedding_backward(grad_out, ids, grad_weight, scale, accumulate)
    vocab, d = grad_weight.shape
    g, flat = grad_out.contiguous(), ids.contiguous()
    n = flat.numel()
    ws = _empty(_embedding_workspace(vocab, d, n), dtype=torch.uint8, device=index)
    status = B.lib().zero_embedding_backward(g.data_ptr(), flat.data_ptr(), vocab, d, n, code, DTYPE[to], scale, 1 if accumulate else 0,
                                             grad_weight.data_ptr(), ws.data_ptr(), _raw_stream(index))
    if status:
        B._check(status)
    return grad_weight


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale):
        ctx.save_for_backward(ids)
        ctx.shape, ctx.scale = weight.shape, scale
        return embedding_forward(weight, ids, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        ids, = ctx.saved_tensors
        grad = torch.empty(ctx.shape, dtype=grad_out.dtype, device=grad_out.device)
        return embedding_backward(grad_out, ids, grad, ctx.scale), None, None


def embedding(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """:func:`embedding_forward`, differentiable in ``weight``."""
    _no_capture(weight)
    return _Embedding.apply(weight, ids, scale)


# -- layer norm ------------------------------------------------------------------------------------------
def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       eps: float = 1e-5) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): ``y = (x - mean) * rstd * weight + bias`` over the last
    dimension; mean and rstd are float32, one per row, for
    :func:`layer_norm_backward`.  All tensors have one dtype."""
    index, dtype, shape = x.get_device(), x.dtype, x.shape
    code, per_row, last = DTYPE.get(dtype), shape[:-1], shape[-1:]
    if not (index >= 0 and code is not None and len(last) == 1 and _like(weight, last, dtype, index) and _like(bias, last, dtype, index)):
        _check_dtype("x", x)
        _check_dims("weight", weight, 1)
        _check_last("x", x, weight.shape[0])
        for name, t in (("weight", weight), ("bias", bias)):
            if t is not None:
                _check_weight(name, t, last)
                _check_dtype(name, t, dtype)
        _check_on(x.device, x=x, weight=weight, bias=bias)
    if _current_device() != index:
        with torch.cuda.device(index):
            return layer_norm_forward(x, weight, bias, eps)
    d = last[0]
    rows, stride = _rows(x, d)
    y = _empty(shape, dtype=dtype, device=index)
    mean, rstd = _empty(per_row, dtype=_FP32, device=index), _empty(per_row, dtype=_FP32, device=index)
    status = B.lib().zero_layer_norm_forward(rows.data_ptr(), stride, weight.data_ptr(), None if bias is None else bias.data_ptr(),
                                             mean.numel(), d, code, eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                             _raw_stream(index))
    if status:
        B._check(status)
    return y, mean, rstd


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        grad_weight: torch.Tensor, grad_bias: Optional[torch.Tensor] = None,
                        accumulate: bool = False) -> torch.Tensor:
    """The input's gradient, a new tensor; the weight's and the bias' go into
    ``grad_weight`` and ``grad_bias`` [d] (x's dtype or float32, one for both),
    overwritten or, with ``accumulate``, added to.  mean and rstd are
    :func:`layer_norm_forward`'s."""
    index, dtype, shape = x.get_device(), x.dtype, x.shape
    code, per_row, last, to = DTYPE.get(dtype), shape[:-1], shape[-1:], grad_weight.dtype
    if not (index >= 0 and code is not None and len(last) == 1 and grad_y.shape == shape and grad_y.dtype is dtype and
            grad_y.get_device() == index and _like(weight, last, dtype, index) and (to is dtype or to is _FP32) and
            _like(grad_weight, last, to, index) and _like(grad_bias, last, to, index) and _like(mean, per_row, _FP32, index) and
            _like(rstd, per_row, _FP32, index)):
        _check_dtype("x", x)
        _check_dtype("grad_y", grad_y, dtype)
        _check_dims("weight", weight, 1)
        _check_last("x", x, weight.shape[0])
        if grad_y.shape != shape:
            raise ValueError("grad_y: shape %s (need %s)" % (_shape(grad_y), _shape(x)))
        _check_weight("weight", weight, last)
        _check_dtype("weight", weight, dtype)
        _check_weight("grad_weight", grad_weight, last)
        _check_dtype("grad_weight", grad_weight, dtype, _FP32)
        if grad_bias is not None:
            _check_weight("grad_bias", grad_bias, last)
            _check_dtype("grad_bias", grad_bias, to)
        for name, t in (("mean", mean), ("rstd", rstd)):
            _check_weight(name, t, per_row)
            _check_dtype(name, t, _FP32)
        _check_on(x.device, x=x, grad_y=grad_y, weight=weight, mean=mean, rstd=rstd, grad_weight=grad_weight, grad_bias=grad_bias)
    if _current_device() != index:
        with torch.cuda.device(index):
            return layer_norm_backward(grad_y, x, weight, mean, rstd, grad_weight, grad_bias, accumulate)
    d, n = last[0], mean.numel()
    rows, stride = _rows(x, d)
    g, g_stride = _rows(grad_y, d)
    grad_x = _empty(shape, dtype=dtype, device=index)
    ws = _empty(_norm_workspace(n, d), dtype=torch.uint8, device=index)
    status = B.lib().zero_layer_norm_backward(g.data_ptr(), g_stride, rows.data_ptr(), stride, weight.data_ptr(), mean.data_ptr(),
                                              rstd.data_ptr(), n, d, code, DTYPE[to], 1 if accumulate else 0, grad_x.data_ptr(),
                                              grad_weight.data_ptr(), None if grad_bias is None else grad_bias.data_ptr(),
                                              ws.data_ptr(), _raw_stream(index))
    if status:
        B._check(status)
    return grad_x


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.biased = bias is not None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        grads = torch.empty(2, *weight.shape, dtype=weight.dtype, device=weight.device)
        gx = layer_norm_backward(grad_y, x, weight, mean, rstd, grads[0], grads[1] if ctx.biased else None)
        return gx, grads[0], grads[1] if ctx.biased else None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5) -> torch.Tensor:
    """y of :func:`layer_norm_forward`, differentiable in x, weight and bias."""
    _no_capture(x, weight, bias)
    return _LayerNorm.apply(x, weight, bias, eps)


# -- language-model head and loss ------------------------------------------------------------------------
_REDUCTION = {"mean": B.ZERO_LOSS_MEAN, "sum": B.ZERO_LOSS_SUM}
_LOSS_DTYPE = {torch.bfloat16: B.ZERO_BF16, torch.float16: B.ZERO_FP16}


@lru_cache(maxsize=256)
def _loss_workspace(n: int, d: int, vocab: int, dtype: int, piece: int, weight_at: int) -> Tuple[int, int]:
    return B.zero_lm_loss_query(B.zero_lm_loss_args(n=n, d=d, vocab=vocab, hidden_stride=d, dtype=dtype, piece=piece, weight=256 + weight_at))


def _check_loss(hidden, weight, targets) -> None:
    _check_dims("weight", weight, 2)
    _check_weight("weight", weight, weight.shape)
    _check_dtype("hidden", hidden, *_LOSS_DTYPE)
    _check_dtype("weight", weight, hidden.dtype)
    _check_dtype("targets", targets, torch.int64)
    _check_last("hidden", hidden, weight.shape[1])
    if hidden.shape[:-1] != targets.shape:
        raise ValueError("targets: shape %s (need %s)" % (_shape(targets), "x".join(map(str, hidden.shape[:-1]))))
    _check_on(weight.device, weight=weight, hidden=hidden, targets=targets)


def _loss_args(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, piece: int = 0):
    """(arguments without outputs, their workspaces' sizes, tensors that they point to)."""
    index, dtype = weight.get_device(), hidden.dtype
    code = _LOSS_DTYPE.get(dtype)
    if not (index >= 0 and code is not None and weight.dtype is dtype and weight.dim() == 2 and weight.is_contiguous() and
            targets.dtype is torch.int64 and hidden.get_device() == index and targets.get_device() == index and
            hidden.shape == (*targets.shape, weight.shape[1])):
        _check_loss(hidden, weight, targets)
    vocab, d = weight.shape
    rows, stride = _rows(hidden, d)
    flat = targets.contiguous()
    n, at = flat.numel(), weight.data_ptr()
    a = B.zero_lm_loss_args(n, d, vocab, stride, code, 0, piece, rows.data_ptr(), at, flat.data_ptr(), scale=1.0)
    return a, _loss_workspace(n, d, vocab, code, piece, at & 255), (rows, flat)


def lm_loss_forward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, reduction: str = "mean"):
    """(loss, losses, saved): the cross entropy of softmax(hidden @ weight.T)
    against ``targets``, without the logits in memory.  hidden [..., d] and
    weight [vocab, d] are bf16 or fp16, targets int64 of hidden's leading
    shape; a target outside 0 .. vocab-1 makes a token not count.  ``loss``
    is the mean over the tokens that count (or the sum; 0 without any),
    ``losses`` has a value for each token, both float32; ``saved`` is for
    :func:`lm_loss_backward` (``loss`` is a view of it)."""
    if reduction not in _REDUCTION:
        raise ValueError("reduction must be 'mean' or 'sum'")
    a, (need, _), keep = _loss_args(hidden, weight, targets)
    index = weight.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return lm_loss_forward(hidden, weight, targets, reduction)
    losses = _empty(targets.shape, dtype=_FP32, device=index)
    saved = _empty(2 + a.n, dtype=_FP32, device=index)   # loss, share, log of each token's sum of exponentials
    ws = _empty(need, dtype=torch.uint8, device=index)
    at = saved.data_ptr()
    a.reduction = _REDUCTION[reduction]
    a.losses, a.lse, a.stats, a.workspace = losses.data_ptr(), at + 8, at, ws.data_ptr()
    status = B.lib().zero_lm_loss_forward(a, _raw_stream(index))
    if status:
        B._check(status)
    return saved.select(0, 0), losses, saved


def lm_loss_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, saved,
                     grad_weight: Optional[torch.Tensor] = None, scale: Union[float, torch.Tensor] = 1.0,
                     accumulate: bool = False, need_hidden: bool = True, piece: int = 0) -> Optional[torch.Tensor]:
    """The gradient of ``loss`` times ``scale``: hidden's is returned (None
    without ``need_hidden``), the weight's goes into ``grad_weight`` [vocab, d]
    of its dtype, overwritten or, with ``accumulate``, added to.  ``scale`` is
    a number or a float32 CUDA tensor of one element that is read when the
    kernels run: a loss scale (``MultiAdamW.state_fields()["loss_scale"]``,
    ``ZeroStep.loss_scale``) or the gradient of ``loss``.  ``piece`` columns of
    the vocabulary are in memory at a time (0: chosen)."""
    a, (_, need), keep = _loss_args(hidden, weight, targets, piece)
    index = weight.get_device()
    by_tensor = isinstance(scale, torch.Tensor)
    if by_tensor and (scale.dtype is not _FP32 or scale.numel() != 1):
        raise ValueError("scale: a number or a float32 tensor of one element")
    if not (_like(saved, (2 + a.n,), _FP32, index) and _like(grad_weight, weight.shape, weight.dtype, index) and
            (not by_tensor or scale.get_device() == index)):
        _check_weight("saved", saved, (2 + a.n,))
        _check_dtype("saved", saved, _FP32)
        if grad_weight is not None:
            _check_weight("grad_weight", grad_weight, weight.shape)
            _check_dtype("grad_weight", grad_weight, weight.dtype)
        _check_on(weight.device, saved=saved, grad_weight=grad_weight, scale=scale if by_tensor else None)
    if _current_device() != index:
        with torch.cuda.device(index):
            return lm_loss_backward(hidden, weight, targets, saved, grad_weight, scale, accumulate, need_hidden, piece)
    grad_hidden = _empty(hidden.shape, dtype=hidden.dtype, device=index) if need_hidden else None
    ws = _empty(need, dtype=torch.uint8, device=index)
    if by_tensor:
        a.scale_dev = scale.data_ptr()
    else:
        a.scale = scale
    a.lse, a.stats, a.workspace = saved.data_ptr() + 8, saved.data_ptr(), ws.data_ptr()
    a.grad_hidden = grad_hidden.data_ptr() if need_hidden else None
    a.grad_weight = grad_weight.data_ptr() if grad_weight is not None else None
    a.accumulate = 1 if accumulate else 0
    status = B.lib().zero_lm_loss_backward(a, _raw_stream(index))
    if status:
        B._check(status)
    return grad_hidden


class _LmLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, reduction):
        loss, _, saved = lm_loss_forward(hidden, weight, targets, reduction)
        ctx.save_for_backward(hidden, weight, targets, saved)
        return loss.clone()         # saved is kept: what becomes of the loss does not reach it

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        hidden, weight, targets, saved = ctx.saved_tensors
        need_hidden, need_weight = ctx.needs_input_grad[:2]
        gw = torch.empty_like(weight) if need_weight else None
        gh = lm_loss_backward(hidden, weight, targets, saved, gw, scale=grad.contiguous(), need_hidden=need_hidden)
        return gh, gw, None, None


def lm_loss(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, reduction: str = "mean") -> torch.Tensor:
    """``loss`` of :func:`lm_loss_forward`, differentiable in hidden and weight."""
    _no_capture(hidden, weight)
    return _LmLoss.apply(hidden, weight, targets, reduction)
