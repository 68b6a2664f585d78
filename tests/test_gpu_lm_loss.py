"""The language-model head's loss and gradients against their formulas in 64 bits.

Tolerances count roundings.  U = 2^-24.  The products of 16-bit numbers are exact in binary32; the tensor cores add them
in an order of their own, each addition off by at most 2 U (they may cut instead of rounding): a sum of k terms is off by
at most 2 k U times the sum of their magnitudes.  ex2.approx is off by 2^-22 relatively, plus its argument's rounding.
dz is rounded to 16 bits (fp16 times 2^14, whose smallest step is 2^-24), the results to 16 bits at the end."""
import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import layers as L

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    B.zero_set_max_ctas(0)


def inputs(n, d, vocab, dtype, shift=0, padded=0.3, lean=6.0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + n * 1000003 + d * 1009 + vocab)
    flat = torch.zeros(vocab * d + shift, dtype=dtype, device="cuda")
    w = flat[shift:].view(vocab, d)
    w.copy_(torch.randn(vocab, d, generator=g, device="cuda") * 0.05)
    t = torch.randint(vocab, (n,), generator=g, device="cuda")
    h = torch.randn(n, d, generator=g, device="cuda") + lean * torch.rand(n, 1, generator=g, device="cuda") * w[t].float() / 0.05 / d ** 0.5
    h = h.to(dtype)
    if n > 3:
        out = torch.rand(n, generator=g, device="cuda") < padded
        t = torch.where(out, torch.where(t % 2 == 0, -100, vocab + t), t)
        h[out] = NAN                           # what does not count is not read by a product
    return h, w, t


def exact(h, w, t, scale, share=None, terms=None):
    """(loss, losses, grad_hidden, grad_weight) in 64 bits and what each may be off; `terms` of a logit are added one after another."""
    dtype, (n, d), vocab = h.dtype, h.shape, w.shape[0]
    on = (t >= 0) & (t < vocab)
    hd = torch.where(on[:, None], h.double(), 0.0)
    wd = w.double()
    z = hd @ wd.t()
    ez = (2 * (terms or d) * U * (hd.abs() @ wd.abs().t())).amax(1, keepdim=True)       # of a row's logits
    lse = z.logsumexp(1, keepdim=True)
    at = torch.where(on, t, 0)[:, None]
    zt = z.gather(1, at)
    size = z.abs().amax(1, keepdim=True) + lse.abs() + 1
    # each exponential: 2^-22, and its argument off by 4 U of the largest magnitude; sums of vocab terms with fewer than
    # 300 one after another; the logarithm
    el = ez + 4 * U * size + 2.0 ** -21 + 300 * U
    count = max(1, int(on.sum()))
    share = 1.0 / count if share is None else share
    losses = torch.where(on, (lse - zt)[:, 0], 0.0)
    tl = torch.where(on, (ez + el + 4 * U * size)[:, 0], 0.0)
    loss = losses.sum() * share
    p = (z - lse).exp()
    p1 = p.scatter_add(1, at, torch.full_like(zt, -1.0)) * on[:, None]
    eps = torch.finfo(dtype).eps / 2
    dp = (p * (torch.expm1(ez + el + 4 * U * size) + 2.0 ** -21) + 2 * U) * on[:, None]
    dp = dp + eps * (p1.abs() + dp) + (2.0 ** -39 if dtype == HF else 2.0 ** -130)
    dp = dp * on[:, None]
    f = scale * share
    gh, gw = p1 @ wd * f, p1.t() @ hd * f
    fa = abs(f)
    th = fa * (dp @ wd.abs() + 2 * vocab * U * (p1.abs() @ wd.abs())) + 4 * U * gh.abs()
    tw = fa * (dp.t() @ hd.abs() + 2 * n * U * (p1.abs().t() @ hd.abs())) + 4 * U * gw.abs()
    return (loss, losses, gh, gw), ((tl.sum() + 4 * U * losses.abs().sum()) * share, tl, th, tw)


def rounding(x, dtype):
    if dtype == torch.float32:
        return U * x.abs()
    return torch.finfo(dtype).eps / 2 * x.abs() + (2.0 ** -25 if dtype == HF else 0.0)


def close(got, want, tol):
    tol = tol + rounding(want.abs() + tol, got.dtype)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%d of %d off, worst %.3g of its tolerance" % (
        bad.sum(), bad.numel(), float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


CASES = [(1, 8, 16, BF, 0), (3, 7, 5, HF, 0), (2, 64, 1, BF, 0), (37, 64, 97, BF, 0), (64, 128, 256, BF, 0), (128, 72, 300, HF, 0),
         (129, 65, 257, BF, 0), (255, 768, 1000, BF, 0), (256, 256, 512, HF, 0), (300, 1600, 2011, BF, 0), (513, 264, 3001, HF, 5),
         (700, 100, 999, BF, 1), (1023, 136, 50257, BF, 0), (64, 4104, 513, HF, 8), (2048, 512, 4096, BF, 0), (5000, 48, 64, HF, 0),
         (40, 33, 70001, BF, 3), (9, 1, 33, HF, 0), (2500, 1000, 8191, BF, 0), (70000, 16, 300, BF, 0), (5, 65536, 50, BF, 0),
         (200, 1600, 700, HF, 1), (130, 31, 513, BF, 7)]


@pytest.mark.parametrize("n,d,vocab,dtype", [(1, 512, 100, BF), (128, 513, 300, HF), (37, 1024, 1001, BF), (5, 1032, 65, HF), (100, 4100, 2050, BF),
                                             (3, 16383, 129, BF), (7, 65536, 200, HF)])
def test_few_tokens_add_a_logit_in_runs(n, d, vocab, dtype):
    """Up to 128 tokens: the tensor cores add up to 512 terms, then the d / 512 (or fewer) sums, of alike lengths, are added."""
    h, w, t = inputs(n, d, vocab, dtype)
    want, tol = exact(h, w, t, 1.0, terms=512 + -(-d // 512))
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    close(losses, want[1], tol[1])
    close(loss, want[0], tol[0])
    gw = torch.empty_like(w)
    gh = L.lm_loss_backward(h, w, t, saved, gw)
    close(gh, want[2], tol[2])
    close(gw, want[3], tol[3])


@pytest.mark.parametrize("n,d,vocab,dtype,shift", CASES)
def test_forward_and_backward(n, d, vocab, dtype, shift):
    h, w, t = inputs(n, d, vocab, dtype, shift)
    scale = 2.0 ** 10 if dtype == HF else 1.5
    want, tol = exact(h, w, t, scale)
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    close(losses, want[1], tol[1])
    close(loss, want[0], tol[0])
    guarded = torch.full((vocab * d + 64 + shift,), 7.0, dtype=dtype, device="cuda")
    gw = guarded[32 + shift:32 + shift + vocab * d].view(vocab, d)
    gh = L.lm_loss_backward(h, w, t, saved, gw, scale=torch.tensor([scale], device="cuda"))
    close(gh, want[2], tol[2])
    close(gw, want[3], tol[3])
    assert bool((guarded[:32 + shift] == 7).all()) and bool((guarded[32 + shift + vocab * d:] == 7).all())
    first = gw.clone()
    # the same bits again, on few CTAs and on other streams' shares of the GPU
    for cap in (1, 5):
        B.zero_set_max_ctas(cap)
        again, lagain, _ = L.lm_loss_forward(h, w, t)
        assert torch.equal(again, loss) and torch.equal(lagain, losses)
        assert torch.equal(L.lm_loss_backward(h, w, t, saved, gw, scale=scale), gh) and torch.equal(gw, first)
        if n * d * vocab > 1e8:
            break
    B.zero_set_max_ctas(0)
    old = (torch.randn(vocab, d, generator=torch.Generator("cuda").manual_seed(1), device="cuda") * 0.1).to(dtype)
    gw.copy_(old)
    assert L.lm_loss_backward(h, w, t, saved, gw, scale=scale, accumulate=True, need_hidden=False) is None
    close(gw, want[3] + old.double(), tol[3] + U * (want[3].abs() + old.double().abs()))
    assert bool((guarded[:32 + shift] == 7).all()) and bool((guarded[32 + shift + vocab * d:] == 7).all())
    assert torch.equal(L.lm_loss_backward(h, w, t, saved, None, scale=scale), gh)


@pytest.mark.parametrize("piece", [1, 256, 512, 1000, 1 << 40])
def test_pieces_of_the_vocabulary(piece):
    h, w, t = inputs(300, 200, 1777, BF)
    want, tol = exact(h, w, t, 1.0)
    _, _, saved = L.lm_loss_forward(h, w, t)
    gw = torch.full_like(w, NAN)
    close(L.lm_loss_backward(h, w, t, saved, gw, piece=piece), want[2], tol[2])
    close(gw, want[3], tol[3])


def test_pieces_with_sums_in_memory_until_the_last():
    # enough tokens that grad_hidden is not summed in parts: its binary32 sums pass from piece to piece, and the last rounds
    for dtype in (BF, HF):
        h, w, t = inputs(3000, 256, 3000, dtype)
        want, tol = exact(h, w, t, 64.0)
        _, _, saved = L.lm_loss_forward(h, w, t)
        gw = torch.full_like(w, NAN)
        close(L.lm_loss_backward(h, w, t, saved, gw, scale=64.0, piece=512), want[2], tol[2])
        close(gw, want[3], tol[3])


def test_one_token_without_leading_dimensions():
    h, w, t = inputs(1, 64, 100, BF)
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    gw = torch.empty_like(w)
    gh = L.lm_loss_backward(h, w, t, saved, gw)
    first = gw.clone()
    loss0, losses0, saved0 = L.lm_loss_forward(h[0], w, t[0])
    assert losses0.shape == () and torch.equal(loss0, loss) and torch.equal(losses0, losses[0])
    assert torch.equal(L.lm_loss_backward(h[0], w, t[0], saved0, gw), gh[0]) and torch.equal(gw, first)


@pytest.mark.parametrize("n", [1, 5, 128, 300])
@pytest.mark.parametrize("kind", ["none", "all", "the last", "the first"])
def test_which_tokens_count(n, kind):
    h, w, t = inputs(n, 96, 515, BF, padded=0.0)
    i = torch.arange(n, device="cuda")
    on = {"none": i < 0, "all": i >= 0, "the last": i == n - 1, "the first": i == 0}[kind]
    t = torch.where(on, t, -1)
    h[~on] = float("inf")
    want, tol = exact(h, w, t, 1.0)
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    close(losses, want[1], tol[1])
    close(loss, want[0], tol[0])
    gw = torch.full_like(w, NAN)
    close(L.lm_loss_backward(h, w, t, saved, gw), want[2], tol[2])
    close(gw, want[3], tol[3])
    if kind == "none":
        assert float(loss) == 0 and not losses.any() and not gw.any()
        gw.fill_(2.0)
        L.lm_loss_backward(h, w, t, saved, gw, accumulate=True)
        assert bool((gw == 2).all())


def test_sum_and_no_tokens():
    h, w, t = inputs(200, 64, 300, HF)
    want, tol = exact(h, w, t, 2.0, share=1.0)
    loss, losses, saved = L.lm_loss_forward(h, w, t, reduction="sum")
    close(loss, want[0], tol[0])
    gw = torch.empty_like(w)
    close(L.lm_loss_backward(h, w, t, saved, gw, scale=2.0), want[2], tol[2])
    close(gw, want[3], tol[3])
    e, te = h[:0], t[:0]
    loss, losses, saved = L.lm_loss_forward(e, w, te)
    assert float(loss) == 0 and losses.shape == (0,)
    assert L.lm_loss_backward(e, w, te, saved, gw).shape == (0, 64) and not gw.any()


def test_exact_products():
    # small whole numbers: every logit is exact, so that any element read from another place shows
    g = torch.Generator("cuda").manual_seed(5)
    for n, d, vocab in ((300, 200, 700), (100, 520, 300)):
        h = torch.randint(-2, 3, (n, d), generator=g, device="cuda").to(BF)
        w = torch.randint(-1, 2, (vocab, d), generator=g, device="cuda").to(BF) * 0.0625
        t = torch.randint(vocab, (n,), generator=g, device="cuda")
        z = h.double() @ w.double().t()
        losses = z.logsumexp(1) - z.gather(1, t[:, None])[:, 0]
        got = L.lm_loss_forward(h, w, t)[1]
        # exact logits: only the exponentials, their sum and the logarithm round
        assert float((got.double() - losses).abs().max()) <= 2.0 ** -20 + 16 * U * float(z.abs().max() + losses.max())


def test_extreme_logits():
    g = torch.Generator("cuda").manual_seed(6)
    n, d, vocab = 140, 128, 400
    w = torch.randn(vocab, d, generator=g, device="cuda").to(BF)
    t = torch.randint(vocab, (n,), generator=g, device="cuda")
    h = (w[t].float() * 100).to(BF)            # logits of about 12800, a one-hot softmax
    want, tol = exact(h, w, t, 1.0)
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    close(losses, want[1], tol[1])
    assert bool((losses == 0).all())           # exactly: the target is the maximum by far
    gw = torch.empty_like(w)
    gh = L.lm_loss_backward(h, w, t, saved, gw)
    assert not gh.any() and not gw.any()
    wrong = (t + 1) % vocab                    # and all of it on another token
    want, tol = exact(h, w, wrong, 1.0)
    loss, losses, saved = L.lm_loss_forward(h, w, wrong)
    close(losses, want[1], tol[1])
    gh = L.lm_loss_backward(h, w, wrong, saved, gw)
    close(gh, want[2], tol[2])
    close(gw, want[3], tol[3])
    h[3] = NAN                                 # a token that counts and is bad spoils its own loss and the mean
    loss, losses, saved = L.lm_loss_forward(h, w, wrong)
    assert bool(losses[3].isnan()) and bool(loss.isnan()) and int(losses.isnan().sum()) == 1
    gh = L.lm_loss_backward(h, w, wrong, saved, gw)
    assert bool(gh[3].isnan().all()) and int(gh.isnan().any(1).sum()) == 1 and bool(gw.isnan().any())


def test_fp16_overflow_shows_as_inf():
    h, w, t = inputs(64, 64, 128, HF, padded=0.0)
    loss, _, saved = L.lm_loss_forward(h, w, t)
    gw = torch.empty_like(w)
    L.lm_loss_backward(h, w, t, saved, gw, scale=2.0 ** 30)
    assert bool(gw.isinf().any())


def test_gradients_against_differences():
    # d loss along a direction: central differences of the losses over a step of the hidden states (or the weight) that
    # 16 bits hold exactly.  Off by the losses' tolerance over the step, and by the third derivative: step^2 / 6 times at
    # most |direction . w|^3
    n, d, vocab, step = 20, 64, 150, 2.0 ** -4
    h, w, t = inputs(n, d, vocab, BF, padded=0.0)
    h = (h * 8).round() / 8                    # multiples of 1/8 below 32: adding 1/16 is exact in bf16 up to 16
    h = h.clamp(-7, 7)
    w = ((w * 64).round() / 64).clamp(-0.25, 0.25)   # and 2^-9 to multiples of 2^-6 up to 1/4
    _, _, saved = L.lm_loss_forward(h, w, t)
    gw = torch.empty_like(w)
    gh = L.lm_loss_backward(h, w, t, saved, gw)
    (_, _, xh, xw), (tl, _, th, tw) = exact(h, w, t, 1.0)
    dh = xh.sign().to(BF) * step               # uphill: the difference is large
    assert torch.equal((h + dh).double(), h.double() + dh.double()) and torch.equal((h - dh).double(), h.double() - dh.double())
    a, b = (L.lm_loss_forward(x, w, t)[0] for x in (h + dh, h - dh))
    along = float((gh.double() * dh.double()).sum())
    third = float((dh.double().abs() @ w.double().abs().t()).amax(1).pow(3).mean())
    tol = 2 * float(tl) + 4 * U * float(a) + float(((th + rounding(xh, BF)) * dh.double().abs()).sum()) + third
    assert abs((float(a) - float(b)) / 2 - along) <= tol
    assert abs(along) > 4 * tol                # the comparison says something
    dw = xw.sign().to(BF) * 2.0 ** -9
    assert torch.equal((w + dw).double(), w.double() + dw.double()) and torch.equal((w - dw).double(), w.double() - dw.double())
    a, b = (L.lm_loss_forward(h, x, t)[0] for x in (w + dw, w - dw))
    along = float((gw.double() * dw.double()).sum())
    third = float((h.double().abs() @ dw.double().abs().t()).amax(1).pow(3).mean())
    tol = 2 * float(tl) + 4 * U * float(a) + float(((tw + rounding(xw, BF)) * dw.double().abs()).sum()) + third
    assert abs((float(a) - float(b)) / 2 - along) <= tol


def test_offsets_pass_32_bits():
    # a weight and a gradient of more than 2^31 elements
    vocab, d, n = 2 ** 20 + 300, 2056, 6
    w = torch.zeros(vocab, d, device="cuda", dtype=BF)
    g = torch.Generator("cuda").manual_seed(8)
    rows = torch.tensor([0, 5, vocab - 300, vocab - 2, vocab - 1], device="cuda")
    w[rows] = (torch.randn(5, d, generator=g, device="cuda") * 0.1).to(BF)
    h = torch.randn(n, d, generator=g, device="cuda").to(BF)
    t = torch.tensor([0, vocab - 1, vocab - 300, 5, 77, vocab - 2], device="cuda")
    loss, losses, saved = L.lm_loss_forward(h, w, t)
    z = h.double() @ w[rows].double().t()
    lse = torch.logaddexp(z.logsumexp(1), torch.log(torch.tensor(float(vocab - 5), dtype=torch.float64, device="cuda")))
    place = torch.tensor([0, 4, 2, 1, -1, 3], device="cuda")
    zt = torch.where(place >= 0, z.gather(1, place.clamp(min=0)[:, None])[:, 0], 0.0)
    # 2 d U of the magnitudes, 4100 tiles joined
    tol = 4 * d * U * float((h.double().abs() @ w[rows].double().abs().t()).max()) + 2.0 ** -20 + 600 * U * 20
    assert float((losses.double() - (lse - zt)).abs().max()) <= tol
    gw = torch.full((vocab, d), 1.0, device="cuda", dtype=BF)
    gh = L.lm_loss_backward(h, w, t, saved, gw, scale=float(n))
    p = (z - lse[:, None]).exp()
    p[place >= 0, place[place >= 0]] -= 1
    eps = torch.finfo(BF).eps / 2
    bound = (2 * tol + 3 * eps) * (p.abs() + 2 * tol)
    assert bool(((gw[rows].double() - p.t() @ h.double()).abs() <= bound.t() @ h.double().abs() + 2.0 ** -60).all())
    assert bool(((gh.double() - p @ w[rows].double()).abs() <= bound @ w[rows].double().abs() + 2.0 ** -60).all())
    # everywhere else a row is the sum of the other tokens' probabilities times their states
    rest = (-lse).exp()[:, None] * h.double()
    for k in (1, vocab // 2, vocab - 3, vocab - 299):
        assert bool(((gw[k].double() - rest.sum(0)).abs() <= (3 * eps + 2 * tol) * rest.abs().sum(0) + 1e-12).all())


def test_autograd_and_strides():
    h, w, t = inputs(6 * 40, 64, 333, BF, padded=0.2)
    h = torch.where(h.isnan(), 0.0, h.float()).to(BF)
    loss, _, saved = L.lm_loss_forward(h, w, t)
    gw = torch.empty_like(w)
    gh = L.lm_loss_backward(h, w, t, saved, gw, scale=3.0)
    x, y = h.view(6, 40, 64).clone().requires_grad_(), w.clone().requires_grad_()
    out = L.lm_loss(x, y, t.view(6, 40))
    assert torch.equal(out, loss)
    a, b = torch.autograd.grad(out * 3.0, [x, y])
    assert torch.equal(a.view(-1, 64), gh) and torch.equal(b, gw)
    a, = torch.autograd.grad(L.lm_loss(x.detach(), y, t.view(6, 40)) * 3.0, [y])
    assert torch.equal(a, gw)
    # the hidden states of a sequence without its last token, and rows of a wider array at an odd place
    seq = torch.cat([h.view(6, 40, 64), torch.full((6, 1, 64), NAN, device="cuda", dtype=BF)], 1)
    assert torch.equal(L.lm_loss_forward(seq[:, :-1], w, t.view(6, 40))[0], loss)
    wide = torch.full((240, 75), NAN, device="cuda", dtype=BF)
    wide[:, 3:67] = h
    assert torch.equal(L.lm_loss_forward(wide[:, 3:67], w, t)[0], loss)
    assert torch.equal(L.lm_loss_backward(wide[:, 3:67], w, t, saved, gw, scale=3.0), gh)


def test_captured_replayed_and_on_two_streams():
    h, w, t = inputs(300, 128, 1000, BF, padded=0.0)
    scale = torch.ones(1, device="cuda")
    gw = torch.zeros_like(w)

    def work(gw):
        loss, losses, saved = L.lm_loss_forward(h, w, t)
        return loss, losses, L.lm_loss_backward(h, w, t, saved, gw, scale=scale)

    work(gw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(gw)
    for k in range(3):
        t.copy_(torch.roll(t, k))
        t[: 50 * k] = -1
        scale.fill_(2.0 ** k)
        graph.replay()
        seen = [x.clone() for x in (*got, gw)]
        for a, e in zip(seen, (*work(gw), gw)):
            assert torch.equal(a, e)
    # two calls at once, each with its own workspace
    want = [x.clone() for x in (*work(gw), gw)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            mine = torch.zeros_like(w)
            for _ in range(4):
                out = work(mine)
            outs.append((*out, mine))
    torch.cuda.synchronize()
    for o in outs:
        for a, e in zip(o, want):
            assert torch.equal(a, e)
    x = h.clone().requires_grad_()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        t.add_(0)
        with pytest.raises(RuntimeError, match="capture"):
            L.lm_loss(x, w, t)


def test_no_errors_reported():
    h, w, t = inputs(50, 64, 300, BF)
    a, (need, _), keep = L._loss_args(h, w, t)
    assert need == B.zero_lm_loss_query(a)[0]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, stats = torch.empty(2, 50, device="cuda"), torch.empty(2, device="cuda")
    a.losses, a.lse, a.stats, a.workspace = out[0].data_ptr(), out[1].data_ptr(), stats.data_ptr(), ws.data_ptr()
    B.zero_lm_loss_forward(a)
    assert B.zero_lm_loss_device_error(ws) == 0
