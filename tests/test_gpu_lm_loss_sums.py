"""The loss' long sums of terms of one sign: over d in the logits, over the tokens in grad_weight, over the vocabulary in
grad_hidden.

Terms are whole numbers times a power of two, so small that the sum of a run of them is at most 2^24 units: exact in binary32,
whether additions round or cut (runs of 32768 in the gradients, of 8192 in the logits).  The runs are then added with rounding to
nearest: R runs are off by at most (R - 1) U of the whole sum, U = 2^-24, and the factors and the last rounding come on top."""
import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import layers as L

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HF, BF = torch.float16, torch.bfloat16
RUN, LOGIT_RUN = 32768, 8192


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    B.zero_set_max_ctas(0)


def whole(g, *shape, run):
    return torch.randint(1, 2 ** 24 // run + 1, shape, generator=g, device="cuda", dtype=torch.int16).to(HF)


def close(got, want, tol):
    tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), "worst %.3g of its tolerance" % float((off / tol).max())


@pytest.mark.parametrize("n,d,pad", [(8192, 64, 0), (32768, 64, 0), (32769, 40, 0), (70001, 24, 0.3), (262144, 64, 0), (600000, 15, 0.1)])
def test_weight_gradient_of_many_tokens(n, d, pad):
    # a weight of zeros and a vocabulary of 256: every probability is 2^-8, exactly so when rounded to 16 bits
    g = torch.Generator("cuda").manual_seed(n)
    h, w = whole(g, n, d, run=RUN), torch.zeros(256, d, dtype=HF, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    t[torch.rand(n, generator=g, device="cuda") < pad] = -1
    count = int((t >= 0).sum())
    _, _, saved = L.lm_loss_forward(h, w, t, "sum")
    gw = torch.empty_like(w)
    L.lm_loss_backward(h, w, t, saved, gw, scale=2.0 ** -12, need_hidden=False)
    want = (h.double() * (t >= 0)[:, None]).sum(0) * 2.0 ** -20
    runs = -(-count // RUN) + 1
    # row 0 is the target's, whose terms are larger
    close(gw[1:], want.expand(255, d), (runs + 4) * U * want)
    first = gw.clone()
    B.zero_set_max_ctas(5)
    L.lm_loss_backward(h, w, t, saved, gw, scale=2.0 ** -12)
    assert torch.equal(gw, first)


# sums in one part and in several, of one run and of two; rows that the product writes itself and others; pieces
@pytest.mark.parametrize("n,d,vocab,piece", [(4096, 256, 65536, 0), (4096, 2048, 65536, 0), (2048, 1000, 65536, 32768), (100, 12288, 2 ** 18, 0),
                                             (3000, 2040, 65536, 20000), (1024, 1024, 2 ** 18, 0)])
def test_hidden_gradient_of_a_large_vocabulary(n, d, vocab, piece):
    # hidden states of zeros: every probability is 1 / vocab, the target's row of the weight is zeros
    g = torch.Generator("cuda").manual_seed(n)
    h, w = torch.zeros(n, d, dtype=HF, device="cuda"), whole(g, vocab, d, run=RUN)
    w[0] = 0
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    _, _, saved = L.lm_loss_forward(h, w, t, "sum")
    gh = L.lm_loss_backward(h, w, t, saved, None, piece=piece)
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for k in range(0, vocab, 16384):
        want += w[k:k + 16384].double().sum(0)
    want /= vocab
    # no sum is longer than the vocabulary; parts and pieces (of which there are 32 at most) add one sum each
    close(gh, want.expand(n, d), (vocab // RUN + 32 + 4) * U * want)


@pytest.mark.parametrize("n,d", [(129, 8192), (129, 8200), (256, 16384), (300, 65535), (256, 65536), (600, 40000), (128, 65536)])
def test_logits_of_a_long_row(n, d):
    g = torch.Generator("cuda").manual_seed(d)
    vocab = 32
    h = torch.full((n, d), 2.0 ** -6, dtype=HF, device="cuda")
    h[1::2] *= 2
    w = whole(g, vocab, d, run=LOGIT_RUN) * 2.0 ** -14
    w[0] = 0
    t = torch.zeros(n, dtype=torch.int64, device="cuda")         # a logit of 0: the loss is the logarithm of the sum
    z = h[:2].double() @ w.double().t()
    lse = z.logsumexp(1)
    # the runs, the exponentials (2^-22 each, their arguments 4 U of the largest logit), their sum, the logarithm
    size = float(z.max() + lse.max() + 1)
    tol = (d // LOGIT_RUN + 128 + 8) * U * size if n <= 128 else (d // LOGIT_RUN + 8) * U * size
    tol = torch.tensor(tol + 2.0 ** -21 + 64 * U, dtype=torch.float64, device="cuda")
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    row = torch.arange(n, device="cuda") % 2
    assert bool(((losses.double() - lse[row]).abs() <= tol).all()), float((losses.double() - lse[row]).abs().max() / tol)
    # the backward call computes them again: dz is a probability, off by its logit's and lse's errors and a rounding to 16 bits
    gw = torch.empty_like(w)
    L.lm_loss_backward(h, w, t, saved, gw, scale=2.0 ** 6, need_hidden=False)
    want = ((z - lse[:, None]).exp()[row] / n * 2.0 ** 6).t() @ h.double()
    close(gw[1:], want[1:], want[1:] * (3 * tol + 2.0 ** -11 + n * 2 * U))


def test_places_of_the_runs_in_a_captured_step_and_on_two_streams():
    g = torch.Generator("cuda").manual_seed(1)
    n, d, vocab = 40000, 72, 3000
    h = torch.randn(n, d, generator=g, device="cuda").to(BF)
    w = (torch.randn(vocab, d, generator=g, device="cuda") * 0.1).to(BF)
    t = torch.randint(vocab, (n,), generator=g, device="cuda")

    def work(gw):
        loss, losses, saved = L.lm_loss_forward(h, w, t)
        return loss, losses, L.lm_loss_backward(h, w, t, saved, gw), gw

    want = [x.clone() for x in work(torch.zeros_like(w))]
    gw = torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(gw)
    graph.replay()
    graph.replay()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            mine = torch.zeros_like(w)
            for _ in range(3):
                out = work(mine)
            outs.append(out)
    torch.cuda.synchronize()
    for o in (got, *outs):
        assert all(torch.equal(a, e) for a, e in zip(o, want))
