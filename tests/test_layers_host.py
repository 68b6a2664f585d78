"""Refusals of the embedding and layer norm calls, before any launch."""
import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import build as zbuild
from zero_partitioned_mixed_replica_gb300 import layers as L

FAKE = 1 << 40          # never dereferenced: refused before any launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    zbuild.build()


def _status(fn, *a, **kw):
    with pytest.raises(B.ZeroError) as e:
        fn(*a, **kw)
    return e.value.status


EMBED = dict(weight=FAKE, ids=FAKE, vocab=10, d=4, n=3, dtype=B.ZERO_BF16, scale=1.0, out=FAKE, stream=0)
EMBED_GRAD = dict(grad_out=FAKE, ids=FAKE, vocab=10, d=4, n=3, dtype=B.ZERO_BF16, grad_dtype=B.ZERO_BF16, scale=1.0,
                  accumulate=False, grad_weight=FAKE, workspace=FAKE, stream=0)
NORM = dict(x=FAKE, x_stride=4, weight=FAKE, bias=FAKE, rows=3, d=4, dtype=B.ZERO_FP16, eps=1e-5, y=FAKE, mean=FAKE,
            rstd=FAKE, stream=0)
NORM_GRAD = dict(grad_y=FAKE, gy_stride=4, x=FAKE, x_stride=4, weight=FAKE, mean=FAKE, rstd=FAKE, rows=3, d=4,
                 dtype=B.ZERO_FP16, grad_dtype=B.ZERO_FP32, accumulate=True, grad_x=FAKE, grad_weight=FAKE, grad_bias=FAKE,
                 workspace=FAKE, stream=0)
SIZES = [dict(vocab=0), dict(vocab=2 ** 31 - 1), dict(d=0), dict(d=2 ** 20 + 1), dict(n=-1), dict(n=2 ** 31), dict(dtype=3),
         dict(dtype=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e300)]
ROWS = [dict(rows=-1), dict(rows=2 ** 31), dict(d=0), dict(d=B.ZERO_MAX_NORM_DIM + 1, x_stride=1 << 20), dict(dtype=7), dict(x_stride=3)]


@pytest.mark.parametrize("fn,base,bad", [
    *[(B.zero_embedding_forward, EMBED, b) for b in SIZES + [dict(weight=0), dict(ids=0), dict(out=0)]],
    *[(B.zero_embedding_backward, EMBED_GRAD, b) for b in SIZES + [
        dict(grad_out=0), dict(ids=0), dict(grad_weight=0), dict(workspace=0), dict(grad_dtype=B.ZERO_FP16), dict(grad_dtype=9)]],
    *[(B.zero_layer_norm_forward, NORM, b) for b in ROWS + [
        dict(x=0), dict(weight=0), dict(y=0), dict(mean=0), dict(rstd=0), dict(eps=-1.0), dict(eps=float("nan"))]],
    *[(B.zero_layer_norm_backward, NORM_GRAD, b) for b in ROWS + [
        dict(gy_stride=2), dict(grad_y=0), dict(x=0), dict(weight=0), dict(mean=0), dict(rstd=0), dict(grad_x=0),
        dict(grad_weight=0), dict(workspace=0), dict(grad_dtype=B.ZERO_BF16)]]])
def test_invalid(fn, base, bad):
    assert _status(fn, **{**base, **bad}) == B.ZERO_ERR_INVALID
    assert B.zero_last_error()


@pytest.mark.parametrize("fn,base,bad", [
    *[(B.zero_embedding_forward, EMBED, b) for b in (dict(weight=FAKE + 1), dict(ids=FAKE + 4), dict(out=FAKE + 1),
                                                    dict(out=FAKE + 2, dtype=B.ZERO_FP32))],
    *[(B.zero_embedding_backward, EMBED_GRAD, b) for b in (
        dict(grad_out=FAKE + 1), dict(ids=FAKE + 2), dict(grad_weight=FAKE + 1), dict(workspace=FAKE + 128),
        dict(grad_weight=FAKE + 2, grad_dtype=B.ZERO_FP32))],
    *[(B.zero_layer_norm_forward, NORM, b) for b in (dict(x=FAKE + 1), dict(weight=FAKE + 1), dict(bias=FAKE + 1),
                                                     dict(y=FAKE + 1), dict(mean=FAKE + 2), dict(rstd=FAKE + 2))],
    *[(B.zero_layer_norm_backward, NORM_GRAD, b) for b in (
        dict(x=FAKE + 1), dict(grad_y=FAKE + 1), dict(weight=FAKE + 1), dict(mean=FAKE + 2), dict(rstd=FAKE + 2),
        dict(grad_x=FAKE + 1), dict(grad_weight=FAKE + 2), dict(grad_bias=FAKE + 2), dict(workspace=FAKE + 16))]])
def test_misaligned(fn, base, bad):
    assert _status(fn, **{**base, **bad}) == B.ZERO_ERR_ALIGN


def test_workspace_queries():
    assert B.zero_embedding_workspace(10, 4, 0) % 256 == 0 and B.zero_layer_norm_workspace(0, 4) % 256 == 0
    assert B.zero_embedding_workspace(50257, 1600, 32768) < 64 << 20
    assert _status(B.zero_embedding_workspace, 0, 4, 1) == B.ZERO_ERR_INVALID
    assert _status(B.zero_layer_norm_workspace, 1, 0) == B.ZERO_ERR_INVALID
    lib = B.lib()
    assert lib.zero_embedding_workspace(1, 1, 1, None) == B.ZERO_ERR_INVALID
    assert lib.zero_layer_norm_workspace(1, 1, None) == B.ZERO_ERR_INVALID


def test_nothing_to_do_needs_no_pointers():
    B.zero_embedding_forward(**{**EMBED, "n": 0, "weight": 0, "ids": 0, "out": 0})
    B.zero_embedding_backward(**{**EMBED_GRAD, "n": 0, "grad_out": 0, "ids": 0, "workspace": 0, "accumulate": True})
    B.zero_layer_norm_forward(**{**NORM, "rows": 0, "x": 0, "y": 0})
    B.zero_layer_norm_backward(**{**NORM_GRAD, "rows": 0, "x": 0, "grad_y": 0, "grad_x": 0, "mean": 0, "rstd": 0})


W, IDS = torch.zeros(10, 4), torch.zeros(3, dtype=torch.int64)
X, V, M = torch.zeros(3, 4), torch.zeros(4), torch.zeros(3)


@pytest.mark.parametrize("call,word", [
    (lambda: L.embedding_forward(torch.zeros(10), IDS), "weight"),
    (lambda: L.embedding_forward(W.double(), IDS), "dtype"),
    (lambda: L.embedding_forward(W.t(), IDS), "contiguous"),
    (lambda: L.embedding_forward(W, IDS.int()), "int64"),
    (lambda: L.embedding_forward(W, IDS), "CUDA"),
    (lambda: L.embedding_backward(X, IDS, torch.zeros(10, 5)), "grad_out"),
    (lambda: L.embedding_backward(X, IDS[:2], W), "grad_out"),
    (lambda: L.embedding_backward(X.half(), IDS, W.bfloat16()), "grad_weight"),
    (lambda: L.embedding_backward(X, IDS, torch.zeros(4, 10).t()), "contiguous"),
    (lambda: L.embedding_backward(X, IDS, W), "CUDA"),
    (lambda: L.embedding(W, IDS), "CUDA"),
    (lambda: L.layer_norm_forward(X, torch.zeros(5)), "x: shape"),
    (lambda: L.layer_norm_forward(X, torch.zeros(1, 4)), "weight"),
    (lambda: L.layer_norm_forward(X, V.half()), "weight"),
    (lambda: L.layer_norm_forward(X.long(), V), "dtype"),
    (lambda: L.layer_norm_forward(X, V, torch.zeros(3)), "bias"),
    (lambda: L.layer_norm_forward(X, V, V), "CUDA"),
    (lambda: L.layer_norm_backward(X[:2], X, V, M, M, V), "grad_y"),
    (lambda: L.layer_norm_backward(X.half(), X, V, M, M, V), "grad_y"),
    (lambda: L.layer_norm_backward(X, X, V, M[:2], M, V), "mean"),
    (lambda: L.layer_norm_backward(X, X, V, M, M.double(), V), "rstd"),
    (lambda: L.layer_norm_backward(X, X, V, M, M, V.half()), "grad_weight"),
    (lambda: L.layer_norm_backward(X.half(), X.half(), V.half(), M, M, V.half(), V), "grad_bias"),
    (lambda: L.layer_norm_backward(X, X, V, M, M, V, V), "CUDA"),
    (lambda: L.layer_norm(X, V), "CUDA")])
def test_python_refusals(call, word):
    with pytest.raises(ValueError, match=word):
        call()


# -- language-model loss ---------------------------------------------------------------------------------
def _loss(**kw):
    a = dict(n=3, d=8, vocab=10, hidden_stride=8, dtype=B.ZERO_BF16, reduction=B.ZERO_LOSS_MEAN, piece=0, hidden=FAKE, weight=FAKE,
             targets=FAKE, losses=FAKE, lse=FAKE, stats=FAKE, workspace=FAKE, scale=1.0, scale_dev=None, grad_hidden=FAKE,
             grad_weight=FAKE, accumulate=0)
    a.update(kw)
    return B.zero_lm_loss_args(**a)


LOSS_SIZES = [dict(n=-1), dict(n=2 ** 30 + 1), dict(d=0), dict(d=65537, hidden_stride=65537), dict(vocab=0), dict(vocab=2 ** 30 + 1),
              dict(hidden_stride=7), dict(dtype=B.ZERO_FP32), dict(dtype=-1), dict(piece=-1)]


@pytest.mark.parametrize("bad", LOSS_SIZES + [dict(reduction=2), dict(hidden=0), dict(weight=0), dict(targets=0), dict(losses=0),
                                              dict(lse=0), dict(stats=0), dict(workspace=0)])
def test_loss_forward_invalid(bad):
    assert _status(B.zero_lm_loss_forward, _loss(**bad), 0) == B.ZERO_ERR_INVALID


@pytest.mark.parametrize("bad", LOSS_SIZES + [dict(hidden=0), dict(weight=0), dict(targets=0), dict(lse=0), dict(stats=0),
                                              dict(workspace=0), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=-1e39)])
def test_loss_backward_invalid(bad):
    assert _status(B.zero_lm_loss_backward, _loss(**bad), 0) == B.ZERO_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(hidden=FAKE + 1), dict(weight=FAKE + 1), dict(targets=FAKE + 4), dict(lse=FAKE + 2),
                                 dict(stats=FAKE + 2), dict(workspace=FAKE + 16)])
def test_loss_misaligned(bad):
    assert _status(B.zero_lm_loss_forward, _loss(**bad), 0) == B.ZERO_ERR_ALIGN
    assert _status(B.zero_lm_loss_backward, _loss(**bad), 0) == B.ZERO_ERR_ALIGN


@pytest.mark.parametrize("bad", [dict(scale_dev=FAKE + 1), dict(grad_hidden=FAKE + 1), dict(grad_weight=FAKE + 1)])
def test_loss_backward_misaligned(bad):
    assert _status(B.zero_lm_loss_backward, _loss(**bad), 0) == B.ZERO_ERR_ALIGN


def test_loss_queries():
    lib = B.lib()
    for fn in (lib.zero_lm_loss_forward, lib.zero_lm_loss_backward):
        assert fn(None, None) == B.ZERO_ERR_INVALID
    assert lib.zero_lm_loss_query(None, None, None) == B.ZERO_ERR_INVALID
    assert _status(B.zero_lm_loss_query, _loss(vocab=0)) == B.ZERO_ERR_INVALID
    f, b = B.zero_lm_loss_query(_loss(n=8192, d=1600, vocab=50257, hidden_stride=1600))
    assert f % 256 == 0 and b % 256 == 0
    assert f < 64 << 20 and b < 800 << 20            # the logits alone would be 824 MB in 16 bits
    # bounded whatever the vocabulary, less with a smaller piece, and a copy of a weight that TMA cannot read
    assert B.zero_lm_loss_query(_loss(n=8192, d=1600, vocab=10 ** 6, hidden_stride=1600))[1] < 800 << 20
    assert B.zero_lm_loss_query(_loss(n=8192, d=1600, vocab=50257, hidden_stride=1600, piece=256))[1] < 128 << 20
    assert B.zero_lm_loss_query(_loss(weight=FAKE + 2))[0] > B.zero_lm_loss_query(_loss())[0]
    assert B.zero_lm_loss_query(_loss(n=0))[0] > 0
    assert lib.zero_lm_loss_device_error(None, None) == B.ZERO_ERR_INVALID
    assert _status(B.zero_lm_loss_device_error, 0) == B.ZERO_ERR_INVALID
    assert _status(B.zero_lm_loss_device_error, FAKE + 8) == B.ZERO_ERR_ALIGN
    B.zero_lm_loss_backward(_loss(grad_hidden=None, grad_weight=None), 0)      # nothing asked for


def test_loss_struct_matches_the_header(tmp_path):
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cls = B.zero_lm_loss_args
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "zero.h"', "int main(void) {",
             'printf("size %zu\\n", sizeof(zero_lm_loss_args));']
    lines += ['printf("%s %%zu\\n", offsetof(zero_lm_loss_args, %s));' % (f[0], f[0]) for f in cls._fields_]
    lines += ['printf("%s %%d\\n", (int)%s);' % (c, c) for c in ("ZERO_MAX_NORM_DIM", "ZERO_LOSS_MEAN", "ZERO_LOSS_SUM")]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f in cls._fields_:
        assert int(got[f[0]]) == getattr(cls, f[0]).offset, f[0]
    for c in ("ZERO_MAX_NORM_DIM", "ZERO_LOSS_MEAN", "ZERO_LOSS_SUM"):
        assert int(got[c]) == getattr(B, c), c


H, HW = torch.zeros(3, 4, dtype=torch.bfloat16), torch.zeros(10, 4, dtype=torch.bfloat16)


@pytest.mark.parametrize("call,word", [
    (lambda: L.lm_loss_forward(H, HW, IDS, reduction="none"), "reduction"),
    (lambda: L.lm_loss_forward(H, HW[0], IDS), "weight"),
    (lambda: L.lm_loss_forward(H, HW.t(), IDS), "contiguous"),
    (lambda: L.lm_loss_forward(H.float(), HW.float(), IDS), "hidden"),
    (lambda: L.lm_loss_forward(H, HW.half(), IDS), "weight"),
    (lambda: L.lm_loss_forward(H, HW, IDS.int()), "int64"),
    (lambda: L.lm_loss_forward(H, HW, IDS[:2]), "targets"),
    (lambda: L.lm_loss_forward(H[:, :3], HW, IDS), "hidden"),
    (lambda: L.lm_loss_forward(H, HW, IDS), "CUDA"),
    (lambda: L.lm_loss(H, HW, IDS), "CUDA")])
def test_loss_python_refusals(call, word):
    with pytest.raises(ValueError, match=word):
        call()
