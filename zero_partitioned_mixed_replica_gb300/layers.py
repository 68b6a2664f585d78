"""The operators at a model's ends and between its blocks: embedding and layer
norm, with their gradients.

A step of :class:`.engine.ZeroStep` or :class:`.multi.MultiAdamW` begins where
backward has left the weight gradients: in a rank's flat 16-bit replica, or in
a list of tensors.  The ``*_backward`` functions here write them there, into
any tensor that the caller gives (``engine.tensor_view(engine.grads[r], t,
shape)``), overwriting it or adding to it; what else they return is new.

Each operator comes in two forms.  ``embedding_forward`` / ``embedding_backward``
and ``layer_norm_forward`` / ``layer_norm_backward`` are the library's calls:
nothing is recorded, and they can be captured into a CUDA graph.
:func:`embedding` and :func:`layer_norm` are differentiable by torch's autograd.

All of them run on torch's current stream of the tensors' device and allocate
their workspace from torch's allocator for the call.  Inputs may have any
number of leading dimensions and any strides (rows that are not evenly spaced
with contiguous elements are copied first); gradients that are written in
place are contiguous.  Formulas, ranges and what happens at their edges:
``include/zero.h``.
"""
from __future__ import annotations

from typing import Optional, Tuple

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
