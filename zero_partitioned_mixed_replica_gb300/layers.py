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

from typing import Optional, Tuple, Union

import torch

from . import binding as B
from .multi import _GRAD as DTYPE
from .multi import _device, _raw_stream


def _shape(t: torch.Tensor) -> str:
    return "x".join(map(str, t.shape)) or "scalar"


def _check_on(device: torch.device, **tensors) -> None:
    """All on one CUDA device; the messages name the first that is not."""
    for name, t in tensors.items():
        if t is not None and (t.device != device or t.device.type != "cuda"):
            raise ValueError("%s is on %s: the call's tensors are on one CUDA device" % (name, t.device))


def _check_dtype(name: str, t: torch.Tensor, dtype: Optional[torch.dtype] = None) -> None:
    if dtype is None:
        if t.dtype not in DTYPE:
            raise ValueError("%s: dtype %s (need %s)" % (name, t.dtype, "/".join(map(str, DTYPE))))
    elif t.dtype != dtype:
        raise ValueError("%s: dtype %s (need %s)" % (name, t.dtype, dtype))


def _check_weight(name: str, t: torch.Tensor, shape) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: shape %s (need %s)" % (name, _shape(t), "x".join(map(str, shape))))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % name)


def _check_grad(name: str, t: torch.Tensor, shape, dtype: torch.dtype) -> None:
    _check_weight(name, t, shape)
    if t.dtype != dtype and t.dtype != torch.float32:
        raise ValueError("%s: dtype %s (need %s or torch.float32)" % (name, t.dtype, dtype))


def _rows(t: torch.Tensor, d: int) -> Tuple[torch.Tensor, int]:
    """(t as rows of d, elements between rows); a copy where t is not evenly
    spaced rows of contiguous elements."""
    if t.dim() != 2:
        t = t.reshape(-1, d)
    if t.is_contiguous() or t.shape[0] == 0:
        return t, d
    stride = d if t.shape[0] <= 1 else t.stride(0)
    if (d > 1 and t.stride(1) != 1) or stride < d:
        return t.contiguous(), d
    return t, stride


def _check_last(name: str, t: torch.Tensor, d: int) -> None:
    if t.dim() < 1 or t.shape[-1] != d:
        raise ValueError("%s: shape %s (need %d in the last dimension)" % (name, _shape(t), d))


def _check_ids(name: str, ids: torch.Tensor) -> None:
    if ids.dtype != torch.int64:
        raise ValueError("%s: dtype %s (need torch.int64)" % (name, ids.dtype))


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(n, dtype=torch.uint8, device=device)


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
    if weight.dim() != 2:
        raise ValueError("weight: shape %s (need vocab x d)" % _shape(weight))
    _check_weight("weight", weight, weight.shape)
    _check_dtype("weight", weight)
    _check_ids("ids", ids)
    dev = weight.device
    _check_on(dev, weight=weight, ids=ids)
    vocab, d = weight.shape
    with _device(dev.index):
        flat = ids.contiguous()
        out = torch.empty((*ids.shape, d), dtype=weight.dtype, device=dev)
        B.zero_embedding_forward(weight, flat, vocab, d, flat.numel(), DTYPE[weight.dtype], scale, out, _raw_stream(dev.index))
    return out


def embedding_backward(grad_out: torch.Tensor, ids: torch.Tensor, grad_weight: torch.Tensor, scale: float = 1.0,
                       accumulate: bool = False) -> torch.Tensor:
    """The weight's gradient into ``grad_weight`` [vocab, d] (grad_out's dtype
    or float32): row k gets ``scale`` times the sum of the rows of
    ``grad_out`` whose id is k, the others zeros; with ``accumulate`` that is
    added to what is there.  The same inputs give the same bits."""
    if grad_weight.dim() != 2:
        raise ValueError("grad_weight: shape %s (need vocab x d)" % _shape(grad_weight))
    vocab, d = grad_weight.shape
    _check_dtype("grad_out", grad_out)
    _check_grad("grad_weight", grad_weight, grad_weight.shape, grad_out.dtype)
    _check_ids("ids", ids)
    if tuple(grad_out.shape) != (*ids.shape, d):
        raise ValueError("grad_out: shape %s (need %s)" % (_shape(grad_out), "x".join(map(str, (*ids.shape, d)))))
    dev = grad_weight.device
    _check_on(dev, grad_weight=grad_weight, grad_out=grad_out, ids=ids)
    with _device(dev.index):
        g, flat = grad_out.contiguous(), ids.contiguous()
        ws = _bytes(B.zero_embedding_workspace(vocab, d, flat.numel()), dev)
        B.zero_embedding_backward(g, flat, vocab, d, flat.numel(), DTYPE[g.dtype], DTYPE[grad_weight.dtype], scale,
                                  accumulate, grad_weight, ws, _raw_stream(dev.index))
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
    _check_dtype("x", x)
    if weight.dim() != 1:
        raise ValueError("weight: shape %s (need one dimension)" % _shape(weight))
    d = weight.shape[0]
    _check_last("x", x, d)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check_weight(name, t, (d,))
            _check_dtype(name, t, x.dtype)
    dev = x.device
    _check_on(dev, x=x, weight=weight, bias=bias)
    with _device(dev.index):
        rows, stride = _rows(x, d)
        n = rows.shape[0]
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        stats = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=dev)
        mean, rstd = stats[0], stats[1]
        B.zero_layer_norm_forward(rows, stride, weight, bias, n, d, DTYPE[x.dtype], eps, y, mean, rstd, _raw_stream(dev.index))
    return y, mean, rstd


def layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        grad_weight: torch.Tensor, grad_bias: Optional[torch.Tensor] = None,
                        accumulate: bool = False) -> torch.Tensor:
    """The input's gradient, a new tensor; the weight's and the bias' go into
    ``grad_weight`` and ``grad_bias`` [d] (x's dtype or float32, one for both),
    overwritten or, with ``accumulate``, added to.  mean and rstd are
    :func:`layer_norm_forward`'s."""
    _check_dtype("x", x)
    _check_dtype("grad_y", grad_y, x.dtype)
    if weight.dim() != 1:
        raise ValueError("weight: shape %s (need one dimension)" % _shape(weight))
    d = weight.shape[0]
    _check_last("x", x, d)
    if grad_y.shape != x.shape:
        raise ValueError("grad_y: shape %s (need %s)" % (_shape(grad_y), _shape(x)))
    _check_weight("weight", weight, (d,))
    _check_dtype("weight", weight, x.dtype)
    _check_grad("grad_weight", grad_weight, (d,), x.dtype)
    if grad_bias is not None:
        _check_grad("grad_bias", grad_bias, (d,), x.dtype)
        if grad_bias.dtype != grad_weight.dtype:
            raise ValueError("grad_bias: dtype %s (need grad_weight's %s)" % (grad_bias.dtype, grad_weight.dtype))
    for name, t in (("mean", mean), ("rstd", rstd)):
        _check_weight(name, t, x.shape[:-1])
        _check_dtype(name, t, torch.float32)
    dev = x.device
    _check_on(dev, x=x, grad_y=grad_y, weight=weight, mean=mean, rstd=rstd, grad_weight=grad_weight, grad_bias=grad_bias)
    with _device(dev.index):
        rows, stride = _rows(x, d)
        g, g_stride = _rows(grad_y, d)
        n = rows.shape[0]
        grad_x = torch.empty(x.shape, dtype=x.dtype, device=dev)
        ws = _bytes(B.zero_layer_norm_workspace(n, d), dev)
        B.zero_layer_norm_backward(g, g_stride, rows, stride, weight, mean, rstd, n, d, DTYPE[x.dtype],
                                   DTYPE[grad_weight.dtype], accumulate, grad_x, grad_weight, grad_bias, ws,
                                   _raw_stream(dev.index))
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


def _loss_args(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, piece: int):
    """(checked arguments, the tensors that they point to)."""
    if weight.dim() != 2:
        raise ValueError("weight: shape %s (need vocab x d)" % _shape(weight))
    _check_weight("weight", weight, weight.shape)
    if hidden.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("hidden: dtype %s (need torch.bfloat16 or torch.float16)" % hidden.dtype)
    _check_dtype("weight", weight, hidden.dtype)
    _check_ids("targets", targets)
    vocab, d = weight.shape
    _check_last("hidden", hidden, d)
    if hidden.shape[:-1] != targets.shape:
        raise ValueError("targets: shape %s (need %s)" % (_shape(targets), "x".join(map(str, hidden.shape[:-1]))))
    _check_on(weight.device, weight=weight, hidden=hidden, targets=targets)
    rows, stride = _rows(hidden, d)
    flat = targets.contiguous()
    a = B.zero_lm_loss_args(n=rows.shape[0], d=d, vocab=vocab, hidden_stride=stride, dtype=DTYPE[hidden.dtype], piece=piece,
                            hidden=rows.data_ptr(), weight=weight.data_ptr(), targets=flat.data_ptr(), scale=1.0)
    return a, (rows, flat)


def lm_loss_forward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, reduction: str = "mean"):
    """(loss, losses, saved): the cross entropy of softmax(hidden @ weight.T)
    against ``targets``, without the logits in memory.  hidden [..., d] and
    weight [vocab, d] are bf16 or fp16, targets int64 of hidden's leading
    shape; a target outside 0 .. vocab-1 makes a token not count.  ``loss``
    is the mean over the tokens that count (or the sum; 0 without any),
    ``losses`` has a value for each token, both float32; ``saved`` is for
    :func:`lm_loss_backward`."""
    if reduction not in _REDUCTION:
        raise ValueError("reduction must be 'mean' or 'sum'")
    dev = weight.device
    a, keep = _loss_args(hidden, weight, targets, 0)
    with _device(dev.index):
        out = torch.empty((2, *targets.shape), dtype=torch.float32, device=dev)
        stats = torch.empty(2, dtype=torch.float32, device=dev)
        ws = _bytes(B.zero_lm_loss_query(a)[0], dev)
        a.reduction = _REDUCTION[reduction]
        a.losses, a.lse, a.stats, a.workspace = out[0].data_ptr(), out[1].data_ptr(), stats.data_ptr(), ws.data_ptr()
        B.zero_lm_loss_forward(a, _raw_stream(dev.index))
    return stats[0], out[0], (out[1], stats)


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
    dev = weight.device
    a, keep = _loss_args(hidden, weight, targets, piece)
    lse, stats = saved
    _check_weight("saved[0]", lse, targets.shape)
    _check_weight("saved[1]", stats, (2,))
    for name, t in (("saved[0]", lse), ("saved[1]", stats)):
        _check_dtype(name, t, torch.float32)
    if grad_weight is not None:
        _check_weight("grad_weight", grad_weight, weight.shape)
        _check_dtype("grad_weight", grad_weight, weight.dtype)
    if isinstance(scale, torch.Tensor):
        if scale.dtype != torch.float32 or scale.numel() != 1:
            raise ValueError("scale: a number or a float32 tensor of one element")
        a.scale_dev = scale.data_ptr()
    else:
        a.scale = scale
    _check_on(dev, lse=lse, stats=stats, grad_weight=grad_weight, scale=scale if isinstance(scale, torch.Tensor) else None)
    with _device(dev.index):
        grad_hidden = torch.empty(hidden.shape, dtype=hidden.dtype, device=dev) if need_hidden else None
        ws = _bytes(B.zero_lm_loss_query(a)[1], dev)
        a.lse, a.stats, a.workspace = lse.data_ptr(), stats.data_ptr(), ws.data_ptr()
        a.grad_hidden = grad_hidden.data_ptr() if need_hidden else None
        a.grad_weight = grad_weight.data_ptr() if grad_weight is not None else None
        a.accumulate = int(bool(accumulate))
        B.zero_lm_loss_backward(a, _raw_stream(dev.index))
    return grad_hidden


class _LmLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, reduction):
        loss, _, (lse, stats) = lm_loss_forward(hidden, weight, targets, reduction)
        ctx.save_for_backward(hidden, weight, targets, lse, stats)
        return loss.clone()         # stats is kept: what becomes of the loss does not reach it

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        hidden, weight, targets, lse, stats = ctx.saved_tensors
        need_hidden, need_weight = ctx.needs_input_grad[:2]
        gw = torch.empty_like(weight) if need_weight else None
        gh = lm_loss_backward(hidden, weight, targets, (lse, stats), gw, scale=grad.contiguous(), need_hidden=need_hidden)
        return gh, gw, None, None


def lm_loss(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, reduction: str = "mean") -> torch.Tensor:
    """``loss`` of :func:`lm_loss_forward`, differentiable in hidden and weight."""
    _no_capture(hidden, weight)
    return _LmLoss.apply(hidden, weight, targets, reduction)
