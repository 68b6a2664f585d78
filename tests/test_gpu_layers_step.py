"""Embedding, layer norm and loss together, as a training step uses them: weights and gradients are tensors of an engine's
flat 16-bit buffers, the loss scale is read on the device, and the sharded step follows."""
import os
import sys

import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import layers as L
from zero_partitioned_mixed_replica_gb300.engine import AdamW, ZeroStep
from zero_partitioned_mixed_replica_gb300.multi import MultiAdamW

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
V, D, N = 1000, 136, 200          # 3 elements before the table: nothing begins on a vector's boundary
SHAPES = [(3,), (V, D), (D,), (D,)]
SCALE = 11.0


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def engine(**kw):
    eng = ZeroStep([3, V * D, D, D], 2, 2, B.ZERO_FP16, adamw=AdamW(lr=1e-2), max_norm=1.0, dynamic_scale=True, loss_scale=1024.0, **kw)
    g = torch.Generator("cuda").manual_seed(3)
    flat = torch.zeros(eng.info.psi_pad, device="cuda")
    eng.tensor_view(flat, 1).copy_(torch.randn(V * D, generator=g, device="cuda") * 0.1)
    eng.tensor_view(flat, 2).fill_(1.0)
    eng.load_master(flat)
    return eng


def batches(seed=5):
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        ids = torch.randint(V, (4, N // 4), generator=g, device="cuda")
        ids[1, -5:] = -1                                    # padding
        targets = torch.roll(ids, -1, 1)
        targets[:, -1] = -100
        out.append((ids, targets))
    return out


def views(eng, r):
    return ([eng.tensor_view(eng.params[r], t, s) for t, s in enumerate(SHAPES)],
            [eng.tensor_view(eng.grads[r], t, s) for t, s in enumerate(SHAPES)])


def backward(eng, r, ids, targets):
    """One rank's forward and backward pass into its gradient replica: a tied table at both ends."""
    (_, table, w, b), (_, g_table, g_w, g_b) = views(eng, r)
    h = L.embedding_forward(table, ids, scale=SCALE)
    y, mean, rstd = L.layer_norm_forward(h, w, b)
    loss, _, saved = L.lm_loss_forward(y, table, targets)
    gy = L.lm_loss_backward(y, table, targets, saved, g_table, scale=eng.loss_scale)
    gh = L.layer_norm_backward(gy, h, w, mean, rstd, g_w, g_b)
    L.embedding_backward(gh, ids, g_table, scale=SCALE, accumulate=True)
    return loss


def exact(eng, r, ids, targets):
    """Gradients of the mean loss in 64 bits, by torch's autograd."""
    (_, table, w, b), _ = views(eng, r)
    p = [t.double().requires_grad_() for t in (table, w, b)]
    inside = ids >= 0
    h = p[0][ids.clamp(min=0)] * SCALE * inside[..., None]
    c = h - h.mean(-1, keepdim=True)
    y = c / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt() * p[1] + p[2]
    loss = torch.nn.functional.cross_entropy((y @ p[0].t()).view(-1, V), targets.reshape(-1), ignore_index=-100)
    # the last column of a row and what follows padding have targets of -1: padding too
    return loss.detach(), torch.autograd.grad(loss, p)


def test_a_training_step_through_the_flat_buffers():
    eng = engine()
    for step in range(3):
        for r, (ids, targets) in enumerate(batches(step)):
            targets = torch.where(targets < 0, -100, targets)
            want_loss, want = exact(eng, r, ids, targets)
            loss = backward(eng, r, ids, targets)
            # 6 tensors of 16 bits between the table and its gradient, each rounded by at most 2^-11 of a value, and norms
            # that pass an error on at most 4 times: 2^-11 * 24 of the gradient's size
            assert abs(float(loss) - float(want_loss)) <= 2.0 ** -8 * float(want_loss)
            scale = float(eng.loss_scale)
            for got, e in zip(views(eng, r)[1][1:], want):
                off = (got.double() / scale - e).norm()
                assert float(off) <= 24 * 2.0 ** -11 * float(e.norm())
            assert not eng.tensor_view(eng.grads[r], 0).any()      # what no operator was given
        norm = sum((eng.tensor_view(eng.grads[0], t).double() / scale / 2 + eng.tensor_view(eng.grads[1], t).double() / scale / 2)
                   .square().sum() for t in range(4)).sqrt()
        eng.step()
        state = eng.read_state()
        assert state["t"] == step + 1 and state["overflow"] == 0
        assert abs(state["grad_norm"] - float(norm)) <= 1e-5 * float(norm)


def test_an_overflow_skips_the_step_and_lowers_the_scale():
    eng = engine()
    B.zero_state_init(eng.state, 0.9, 0.999, 2.0 ** 40, True, 2000)
    before = eng.params.clone()
    for r, (ids, targets) in enumerate(batches()):
        backward(eng, r, ids, targets)
    eng.step()
    state = eng.read_state()
    assert state["overflow"] == 1 and state["t"] == 0 and state["loss_scale"] == 2.0 ** 39
    assert torch.equal(eng.params, before)


def test_a_whole_step_captured():
    eng, twin = engine(), engine()
    (ids0, t0), (ids1, t1) = batches()

    def step(e):
        a = backward(e, 0, ids0, t0)
        b = backward(e, 1, ids1, t1)
        e.step()
        return a, b

    step(twin)
    step(eng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        losses = step(eng)
    for _ in range(3):
        for ids, t in ((ids0, t0), (ids1, t1)):
            ids.copy_(torch.where(ids < 0, ids, (ids * 7 + 1) % V))
            t.copy_(torch.where(t < 0, t, (t * 7 + 1) % V))
        graph.replay()
        want = step(twin)
        assert all(torch.equal(a, b) for a, b in zip(losses, want))
        assert torch.equal(eng.grads, twin.grads) and torch.equal(eng.params, twin.params)
        assert torch.equal(eng.state, twin.state)


def test_views_are_refused_where_there_is_no_such_tensor():
    eng = engine()
    with pytest.raises(ValueError, match="Psi_pad"):
        eng.tensor_view(eng.grads, 0)
    with pytest.raises(ValueError, match="Psi_pad"):
        eng.tensor_view(eng.master[0], 0)
    for t in (-1, 4):
        with pytest.raises(ValueError, match="tensor must be"):
            eng.tensor_view(eng.grads[0], t)
    with pytest.raises(RuntimeError):
        eng.tensor_view(eng.grads[0], 1, (V, D + 1))
    assert eng.tensor_view(eng.grads[1], 1).data_ptr() == eng.grads[1].data_ptr() + 2 * eng.tensor_offsets[1]


def test_gradients_of_a_list_follow_the_list_optimizers_loss_scale():
    g = torch.Generator("cuda").manual_seed(9)
    master = [torch.randn(50, 64, generator=g, device="cuda") * 0.1]
    model = [t.bfloat16() for t in master]
    grads = [torch.zeros_like(t) for t in model]
    opt = MultiAdamW(master, grads, model, loss_scale=8.0, max_norm=1e9)
    ids = torch.randint(50, (96,), generator=g, device="cuda")
    h = L.embedding_forward(model[0], ids)
    _, _, saved = L.lm_loss_forward(h, model[0], (ids + 1) % 50)
    L.lm_loss_backward(h, model[0], (ids + 1) % 50, saved, grads[0], scale=opt.state_fields()["loss_scale"])
    at_8 = grads[0].clone()
    L.lm_loss_backward(h, model[0], (ids + 1) % 50, saved, grads[0])
    assert torch.equal(at_8.float(), grads[0].float() * 8)        # a power of two: exact in bf16
    grads[0].copy_(at_8)
    opt.step()
    assert abs(opt.read_state()["grad_norm"] - float((at_8.double() / 8).norm())) <= 1e-5 * opt.read_state()["grad_norm"]


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_trains_with_the_operators(bits):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import many_tensors
    finally:
        sys.path.pop(0)
    losses = many_tensors.train(steps=20, state_bits=bits, operators=True, say=lambda s: None)
    assert len(losses) == 20 and all(x == x and x < 20 for x in losses)


def test_the_examples_gradients_are_the_plain_ones():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import many_tensors as ex
    finally:
        sys.path.pop(0)
    gen = torch.Generator("cuda").manual_seed(1)
    p = {n: t.bfloat16().requires_grad_() for n, t in ex.parameters(gen).items()}
    x = torch.randint(ex.VOCAB, (512,), generator=gen, device="cuda")
    y = torch.randint(ex.VOCAB, (512,), generator=gen, device="cuda")
    plain, own = (f(p, x, y) for f in (ex.loss_of, ex.loss_of_operators))
    a, b = float(plain.detach()), float(own.detach())
    # what the operators round to bf16 on the way (the embedding is exact): the state before the head and its gradient,
    # dz and the gradients, 2^-9 each, through a norm and two products: 2^-9 * 16
    assert abs(b - a) <= 2.0 ** -7 * a
    for n, a, b in zip(p, torch.autograd.grad(plain, list(p.values())), torch.autograd.grad(own, list(p.values()))):
        assert float((a.double() - b.double()).norm()) <= 16 * 2.0 ** -9 * float(a.double().norm()), n


FIRST = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from zero_partitioned_mixed_replica_gb300 import layers as L
g = torch.Generator("cuda").manual_seed(1)
w = torch.randn(300, 72, generator=g, device="cuda").bfloat16()
n = torch.ones(72, device="cuda").bfloat16()
ids = torch.randint(300, (150,), generator=g, device="cuda")
gw, gn = torch.zeros_like(w), torch.zeros_like(n)
torch.cuda.synchronize()
def work():
    h = L.embedding_forward(w, ids)
    y, mean, rstd = L.layer_norm_forward(h, n)
    loss, _, saved = L.lm_loss_forward(y, w, ids)
    gy = L.lm_loss_backward(y, w, ids, saved, gw)
    L.embedding_backward(L.layer_norm_backward(gy, h, n, mean, rstd, gn), ids, gw, accumulate=True)
    return loss
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):          # the first call of the process
    loss = work()
graph.replay()
torch.cuda.synchronize()
got = loss.clone(), gw.clone(), gn.clone()
want = work(), gw, gn
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("equal")
"""


def test_the_first_call_of_a_process_may_be_captured(tmp_path):
    import subprocess
    src = tmp_path / "first.py"
    src.write_text(FIRST)
    p = subprocess.run([sys.executable, str(src), ROOT], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "equal" in p.stdout, p.stdout + p.stderr
