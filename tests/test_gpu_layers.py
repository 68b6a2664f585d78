"""Embedding and layer norm against their formulas in 64 bits.

Tolerances count roundings: a binary32 operation is off by at most U = 2^-24 of
its result, a sum of k terms in any order by at most k U times the sum of the
magnitudes, and the last rounding to the output's type by half a step, eps / 2
(for fp16 also half its smallest step, 2^-25, where the result is subnormal)."""
import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import layers as L

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    B.zero_set_max_ctas(0)


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def placed(t, shift, guard=64):
    """t as a tensor that begins `shift` elements after a 256-byte boundary, with guard bands of 7 around it."""
    flat = torch.full((guard * 8 + shift + t.numel() + guard,), 7.0, dtype=t.dtype, device=t.device)
    at = guard * 8 + shift
    flat[at:at + t.numel()] = t.reshape(-1)
    return flat, flat[at:at + t.numel()].view(t.shape)


def untouched(flat, view):
    at = view.storage_offset()
    return bool((flat[:at] == 7).all()) and bool((flat[at + view.numel():] == 7).all())


def rounding(exact, dtype):
    if dtype == FP:
        return U * exact.abs()
    return torch.finfo(dtype).eps / 2 * exact.abs() + (2.0 ** -25 if dtype == HF else 0.0)


def close(got, exact, tol):
    tol = tol + rounding(exact.abs() + tol, got.dtype)
    off = (got.double() - exact).abs()
    bad = ~(off <= tol)
    assert not bad.any(), "%d of %d off, worst %.3g of its tolerance" % (
        bad.sum(), bad.numel(), float((off / tol.clamp(min=1e-300)).max()))


# -- embedding -------------------------------------------------------------------------------------------
TABLES = [(1, 1, 1, BF, 0), (5, 3, 7, BF, 1), (97, 64, 512, BF, 0), (257, 8, 1000, HF, 0), (50257, 768, 1023, BF, 0),
          (1000, 1600, 300, HF, 5), (300, 33, 2500, FP, 0), (65536, 16, 70000, FP, 2), (40, 4104, 64, BF, 8), (33, 1001, 9000, HF, 3),
          (7, 70000, 40, HF, 0), (5, 70001, 20, BF, 1)]


@pytest.mark.parametrize("vocab,d,n,dtype,shift", TABLES)
def test_embedding_forward_is_the_rounded_product(vocab, d, n, dtype, shift):
    g = gen(1)
    _, w = placed(torch.randn(vocab, d, generator=g, device="cuda").to(dtype), shift)
    ids = torch.randint(-2, vocab + 2, (n,), generator=g, device="cuda")
    for scale in (1.0, 1.0 / 3.0):
        got = L.embedding_forward(w, ids, scale)
        inside = (ids >= 0) & (ids < vocab)
        want = torch.where(inside[:, None], w[ids.clamp(0, vocab - 1)].float() * torch.tensor(scale, dtype=FP), 0.0).to(dtype)
        assert torch.equal(got, want)


def embed_grad_exact(g, ids, vocab, scale):
    inside = (ids >= 0) & (ids < vocab)
    exact = torch.zeros(vocab, g.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(exact)
    count = torch.zeros(vocab, 1, dtype=torch.float64, device="cuda")
    exact.index_add_(0, ids[inside], g[inside].double() * scale)
    size.index_add_(0, ids[inside], g[inside].double().abs() * abs(scale))
    count.index_add_(0, ids[inside], torch.ones(int(inside.sum()), 1, dtype=torch.float64, device="cuda"))
    return exact, (count + 3) * U * size


@pytest.mark.parametrize("fp32_grad", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("vocab,d,n,dtype,shift", TABLES)
def test_embedding_backward(vocab, d, n, dtype, shift, fp32_grad):
    g = gen(2)
    ids = torch.randint(-1, vocab + 1, (n,), generator=g, device="cuda")
    if n > 100:
        ids[: n // 3] = ids[0].clamp(0, vocab - 1)            # one id in a third of the tokens
    go = torch.randn(n, d, generator=g, device="cuda").to(dtype)
    go[(ids < 0) | (ids >= vocab)] = NAN                      # padding is not read
    flat, gw = placed(torch.full((vocab, d), 3.0, device="cuda", dtype=FP if fp32_grad else dtype), shift)
    exact, tol = embed_grad_exact(go, ids, vocab, 0.75)
    L.embedding_backward(go, ids, gw, scale=0.75)
    close(gw, exact, tol)
    assert untouched(flat, gw)
    first = gw.clone()
    old = torch.randn(vocab, d, generator=g, device="cuda").to(gw.dtype)
    gw.copy_(old)
    L.embedding_backward(go, ids, gw, scale=0.75, accumulate=True)
    close(gw, exact + old.double(), tol + U * (exact.abs() + old.double().abs()))
    assert untouched(flat, gw)
    for cap in (1, 3, 12):
        B.zero_set_max_ctas(cap)
        assert torch.equal(L.embedding_backward(go, ids, gw, scale=0.75), first), cap


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 2048, 2049, 8192, 8193, 50001, 98304, 98305, 200003])
@pytest.mark.parametrize("kind", ["one id", "none", "two alternating", "sorted", "each once"])
def test_embedding_backward_token_orders(n, kind):
    vocab = max(70000, n)
    go = torch.randn(n, 24, generator=gen(3), device="cuda")
    i = torch.arange(n, device="cuda")
    ids = {"one id": torch.full((n,), 69999, device="cuda"), "none": torch.full((n,), -100, device="cuda"),
           "two alternating": 255 + i % 2, "sorted": i // 3, "each once": (n - 1 - i)}[kind]
    gw = torch.full((vocab, 24), NAN, device="cuda")
    L.embedding_backward(go, ids, gw)
    exact, tol = embed_grad_exact(go, ids, vocab, 1.0)
    close(gw, exact, tol)


def test_embedding_without_tokens():
    w = torch.ones(7, 6, device="cuda", dtype=BF)
    ids = torch.empty(0, 3, dtype=torch.int64, device="cuda")
    assert L.embedding_forward(w, ids).shape == (0, 3, 6)
    gw = torch.full((7, 6), 2.0, device="cuda", dtype=BF)
    L.embedding_backward(torch.empty(0, 3, 6, device="cuda", dtype=BF), ids, gw, accumulate=True)
    assert bool((gw == 2).all())
    L.embedding_backward(torch.empty(0, 3, 6, device="cuda", dtype=BF), ids, gw)
    assert not gw.any()


def test_embedding_offsets_pass_32_bits():
    # a table of 2^31 + elements: rows behind the 4 GiB mark, forward and backward
    vocab, d = 2 ** 20 + 3, 2056
    w = torch.zeros(vocab, d, device="cuda", dtype=BF)
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1], device="cuda")
    w[ids[:3]] = torch.randn(3, d, generator=gen(4), device="cuda").to(BF)
    out = L.embedding_forward(w, ids)
    assert torch.equal(out, w[ids])
    L.embedding_backward(out, ids, w)
    exact, tol = embed_grad_exact(out, torch.tensor([2, 0, 1, 2], device="cuda"), 3, 1.0)
    close(w[[0, vocab - 2, vocab - 1]], exact, tol)
    assert not w[1:vocab - 2].any()


# -- layer norm ------------------------------------------------------------------------------------------
def norm_exact(x, w, b, eps):
    """y, mean, rstd in 64 bits, with what their binary32 forms may be off: K terms follow one another in a sum at most."""
    K = 80
    x, w = x.double(), w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    dm = K * U * x.abs().mean(1, keepdim=True)
    dr = (K / 2 + 5) * U + (dm.square() + 4 * U * dm * (var.sqrt() + dm)) / (2 * (var + eps))
    y = (x - mean) * rstd * w + b
    dy = (w * rstd).abs() * (dm + U * (x - mean).abs()) + ((x - mean) * rstd * w).abs() * (dr + 3 * U) + U * y.abs()
    return (y, mean[:, 0], rstd[:, 0]), (dy + (w * rstd).abs() * dm * dr, dm[:, 0], (rstd * dr)[:, 0])


SHAPES = [(1, 1, BF, 0), (3, 2, FP, 1), (5, 7, HF, 0), (70, 8, BF, 0), (9, 33, FP, 0), (64, 768, BF, 0), (33, 1000, HF, 0),
          (21, 1001, FP, 3), (130, 1600, BF, 0), (17, 1600, HF, 1), (9, 1602, BF, 2), (12, 2048, FP, 0), (6, 2056, BF, 0),
          (5, 4096, BF, 0), (4, 4104, HF, 8), (3, 5001, BF, 0), (3, 8192, FP, 0), (2, 16383, BF, 1), (3, 16384, BF, 0),
          (2, 16384, FP, 0), (2, 16384, HF, 2), (2000, 24, BF, 0), (3001, 768, BF, 0)]


def norm_inputs(rows, d, dtype, shift):
    g = gen(rows * 7 + d)
    x = (torch.randn(rows, d, generator=g, device="cuda") * 1.5 + 2.0 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    w = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    b = (0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    gy = torch.randn(rows, d, generator=g, device="cuda").to(dtype)
    return x, placed(w, shift)[1], placed(b, shift)[1], gy


@pytest.mark.parametrize("rows,d,dtype,shift", SHAPES)
def test_layer_norm_forward(rows, d, dtype, shift):
    x, w, b, _ = norm_inputs(rows, d, dtype, shift)
    for bias in (b, None):
        got = L.layer_norm_forward(x, w, bias)
        for a, e, t in zip(got, *norm_exact(x, w, bias, 1e-5)):
            close(a, e, t)
    wide = torch.full((rows, d + 9), NAN, device="cuda", dtype=dtype)     # rows of a wider array
    wide[:, 4:d + 4] = x
    for a, e, t in zip(L.layer_norm_forward(wide[:, 4:d + 4], w, None), *norm_exact(x, w, None, 1e-5)):
        close(a, e, t)


def norm_grad_exact(gy, x, w, mean, rstd, per_block):
    K = 64
    gy, x, w = gy.double(), x.double(), w.double()
    mean, rstd, d = mean.double()[:, None], rstd.double()[:, None], x.shape[1]
    u, h = (x - mean) * rstd, gy * w
    s1, s2 = h.mean(1, keepdim=True), (h * u).mean(1, keepdim=True)
    gx = rstd * (h - s1 - u * s2)
    e1 = (K + 3) * U * h.abs().mean(1, keepdim=True)
    e2 = (K + 6) * U * (h * u).abs().mean(1, keepdim=True)
    tx = rstd * (4 * U * h.abs() + 3 * U * s1.abs() + 7 * U * (u * s2).abs() + e1 + u.abs() * e2)
    k = (per_block + 50 + 4) * U
    return (gx, (gy * u).sum(0), gy.sum(0)), (tx, k * (gy * u).abs().sum(0), k * gy.abs().sum(0))


@pytest.mark.parametrize("fp32_grad", [False, True], ids=["same", "fp32"])
@pytest.mark.parametrize("rows,d,dtype,shift", SHAPES)
def test_layer_norm_backward(rows, d, dtype, shift, fp32_grad):
    x, w, b, gy = norm_inputs(rows, d, dtype, shift)
    _, mean, rstd = L.layer_norm_forward(x, w, b)
    gt = FP if fp32_grad else dtype
    fw, gw = placed(torch.full((d,), 3.0, device="cuda", dtype=gt), shift)
    fb, gb = placed(torch.full((d,), 3.0, device="cuda", dtype=gt), shift)
    exact, tol = norm_grad_exact(gy, x, w, mean, rstd, max(4, -(-rows // 456)))
    gx = L.layer_norm_backward(gy, x, w, mean, rstd, gw, gb)
    for a, e, t in zip((gx, gw, gb), exact, tol):
        close(a, e, t)
    assert untouched(fw, gw) and untouched(fb, gb)
    first = gw.clone(), gb.clone()
    old = torch.randn(d, generator=gen(5), device="cuda").to(gt)
    gw.copy_(old)
    gb.copy_(old)
    wide = torch.full((2, rows, d + 9), NAN, device="cuda", dtype=dtype)
    wide[0, :, 4:d + 4], wide[1, :, 4:d + 4] = gy, x
    close(L.layer_norm_backward(wide[0, :, 4:d + 4], wide[1, :, 4:d + 4], w, mean, rstd, gw, gb, accumulate=True), exact[0], tol[0])
    for a, e, t in zip((gw, gb), exact[1:], tol[1:]):
        close(a, e + old.double(), t + U * (e.abs() + old.double().abs()))
    assert untouched(fw, gw) and untouched(fb, gb)
    L.layer_norm_backward(gy, x, w, mean, rstd, gw, None)
    assert torch.equal(gw, first[0])
    for cap in (1, 7):
        B.zero_set_max_ctas(cap)
        assert torch.equal(L.layer_norm_backward(gy, x, w, mean, rstd, gw, gb), gx)
        assert torch.equal(gw, first[0]) and torch.equal(gb, first[1])


@pytest.mark.parametrize("rows,d,dtype,shift", [(400, 1001, FP, 1), (310, 1600, FP, 0), (470, 1602, BF, 2), (200, 4104, HF, 8), (307, 5001, BF, 0),
                                                (160, 10000, BF, 0), (333, 2500, FP, 0), (153, 10008, FP, 0), (305, 9002, HF, 2), (154, 16383, BF, 1)])
def test_layer_norm_of_several_rows_a_block(rows, d, dtype, shift):
    """More rows than blocks and, capped, many for each CTA: a row is loaded while another is worked on."""
    x, w, b, gy = norm_inputs(rows, d, dtype, shift)
    first = L.layer_norm_forward(x, w, b)
    for a, e, t in zip(first, *norm_exact(x, w, b, 1e-5)):
        close(a, e, t)
    B.zero_set_max_ctas(3)
    assert all(torch.equal(a, e) for a, e in zip(L.layer_norm_forward(x, w, b), first))
    gw, gb = torch.empty_like(w), torch.empty_like(b)
    gx = L.layer_norm_backward(gy, x, w, *first[1:], gw, gb)
    exact, tol = norm_grad_exact(gy, x, w, *first[1:], -(-rows // 152))
    for a, e, t in zip((gx, gw, gb), exact, tol):
        close(a, e, t)


def test_layer_norm_rows_of_one_value_and_far_from_zero():
    d = 640
    x = torch.zeros(4, d, device="cuda")
    x[1] = 5.0                                              # variance 0: y is the bias
    x[2] = 1e4 + torch.randn(d, generator=gen(6), device="cuda")
    x[3] = 1e-3 * torch.randn(d, generator=gen(6), device="cuda")
    w, b = torch.full((d,), 2.0, device="cuda"), torch.full((d,), 0.5, device="cuda")
    got = L.layer_norm_forward(x, w, b)
    for a, e, t in zip(got, *norm_exact(x, w, b, 1e-5)):
        close(a, e, t)
    assert bool((got[0][:2] == 0.5).all())
    x[0, 3] = NAN                                           # a bad row spoils itself alone
    x[1, 7] = float("inf")
    bad = L.layer_norm_forward(x, w, b)[0]
    assert bool(bad[:2].isnan().any(1).all()) and torch.equal(bad[2:], got[0][2:])


def test_layer_norm_without_rows():
    w = torch.ones(6, device="cuda")
    x = torch.empty(0, 6, device="cuda")
    y, mean, rstd = L.layer_norm_forward(x, w)
    assert y.shape == (0, 6) and mean.shape == (0,)
    gw, gb = torch.full((6,), 2.0, device="cuda"), torch.full((6,), 2.0, device="cuda")
    L.layer_norm_backward(x, x, w, mean, rstd, gw, gb, accumulate=True)
    assert bool((gw == 2).all()) and bool((gb == 2).all())
    L.layer_norm_backward(x, x, w, mean, rstd, gw, gb)
    assert not gw.any() and not gb.any()


def test_layer_norm_gradient_against_differences():
    # f = sum(y * c), central differences in binary32: the quotient is off by the rounding of f (its y's tolerances, over
    # the step) and by a third-derivative term below step^2 * |f'''| / 6; with step 2^-6 and rstd near 1 both are small
    rows, d, step = 3, 40, 2.0 ** -6
    x, w, b, c = norm_inputs(rows, d, FP, 0)
    y, mean, rstd = L.layer_norm_forward(x, w, b)
    gw, gb = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    gx = L.layer_norm_backward(c, x, w, mean, rstd, gw, gb)

    def f(x, w, b):
        return (L.layer_norm_forward(x, w, b)[0].double() * c.double()).sum()

    (ye, _, _), (ty, _, _) = norm_exact(x, w, b, 1e-5)
    noise = float((c.double().abs() * (ty + U * ye.abs())).sum()) / step
    curve = step ** 2 * float((rstd.max().double() ** 3) * (w.abs().max() * c.abs().max()).double() * 15)
    for t, grad in ((x, gx), (w, gw), (b, gb)):
        for k in range(0, t.numel(), 13):
            one = torch.zeros(t.numel(), device="cuda")
            one[k] = step
            one = one.view(t.shape)
            args = [[x, w, b], [x, w, b]]
            j = 0 if t is x else 1 if t is w else 2
            args[0][j], args[1][j] = t + one, t - one
            diff = (f(*args[0]) - f(*args[1])) / float((args[0][j] - args[1][j]).double().sum())
            assert abs(float(diff) - float(grad.view(-1)[k])) <= noise + curve


def test_without_leading_dimensions():
    g = gen(11)
    w, x = torch.randn(9, 40, generator=g, device="cuda"), torch.randn(1, 40, generator=g, device="cuda")
    one = torch.tensor(4, device="cuda")
    assert torch.equal(L.embedding_forward(w, one), w[4])
    gw = torch.empty_like(w)
    L.embedding_backward(x[0], one, gw)
    assert torch.equal(gw[4], x[0]) and int((gw != 0).any(1).sum()) == 1
    y, mean, rstd = L.layer_norm_forward(x, w[0], w[1])
    y0, mean0, rstd0 = L.layer_norm_forward(x[0], w[0], w[1])
    assert torch.equal(y0, y[0]) and mean0.shape == () and torch.equal(rstd0, rstd[0])
    a, b = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    gx = L.layer_norm_backward(y, x, w[0], mean, rstd, a, b)
    first = a.clone()
    assert torch.equal(L.layer_norm_backward(y0, x[0], w[0], mean0, rstd0, a, b), gx[0]) and torch.equal(a, first)


# -- how they are called ----------------------------------------------------------------------------------
def test_autograd_gives_the_same_gradients():
    g = gen(8)
    w = torch.randn(50, 96, generator=g, device="cuda").to(BF).requires_grad_()
    lw = torch.ones(96, device="cuda", dtype=BF).requires_grad_()
    lb = torch.zeros(96, device="cuda", dtype=BF).requires_grad_()
    ids = torch.randint(50, (4, 9), generator=g, device="cuda")
    c = torch.randn(4, 9, 96, generator=g, device="cuda").to(BF)
    h = L.embedding(w, ids, 2.0)
    y = L.layer_norm(h, lw, lb)
    grads = torch.autograd.grad(y, [w, lw, lb], c)
    with torch.no_grad():
        h2 = L.embedding_forward(w, ids, 2.0)
        y2, mean, rstd = L.layer_norm_forward(h2, lw, lb)
        want = [torch.empty_like(t) for t in (w, lw, lb)]
        gh = L.layer_norm_backward(c, h2, lw, mean, rstd, want[1], want[2])
        L.embedding_backward(gh, ids, want[0], 2.0)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    for a, e in zip(grads, want):
        assert torch.equal(a, e)
    y = L.layer_norm(L.embedding(w, ids), lw)               # no bias, and an expanded gradient
    a, = torch.autograd.grad(y.float().sum(), [lw])
    assert a.shape == lw.shape


def test_captured_and_replayed_with_other_inputs():
    g = gen(9)
    w = torch.randn(300, 64, generator=g, device="cuda").to(BF)
    lw, lb = (torch.randn(64, generator=g, device="cuda").to(BF) for _ in range(2))
    ids = torch.randint(300, (700,), generator=g, device="cuda")
    gw, glw, glb = torch.zeros_like(w), torch.zeros_like(lw), torch.zeros_like(lb)

    def work():
        h = L.embedding_forward(w, ids)
        y, mean, rstd = L.layer_norm_forward(h, lw, lb)
        gh = L.layer_norm_backward(y, h, lw, mean, rstd, glw, glb)
        L.embedding_backward(gh, ids, gw)
        return y

    work()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = work()
    with torch.cuda.graph(graph2):                           # a second one, with workspaces of its own
        y2 = work()
    for k in range(3):
        ids.copy_(torch.randint(-1, 300, (700,), generator=g, device="cuda"))
        (graph if k % 2 else graph2).replay()
        got = (y if k % 2 else y2).clone(), gw.clone(), glw.clone(), glb.clone()
        want = work(), gw, glw, glb
        for a, e in zip(got, want):
            assert torch.equal(a, e)
    wg = w.clone().requires_grad_()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        ids.add_(0)
        with pytest.raises(RuntimeError, match="capture"):
            L.embedding(wg, ids)


def test_another_stream_and_odd_strides():
    g = gen(10)
    w = torch.randn(64, 40, generator=g, device="cuda").to(BF)
    lw = torch.randn(40, generator=g, device="cuda").to(BF)
    ids = torch.randint(64, (6, 50), generator=g, device="cuda")
    x = torch.randn(40, 50, 6, generator=g, device="cuda").to(BF)
    want = L.embedding_forward(w, ids.t().contiguous()), L.layer_norm_forward(x.permute(2, 1, 0).contiguous(), lw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = L.embedding_forward(w, ids.t()), L.layer_norm_forward(x.permute(2, 1, 0), lw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, e) for a, e in zip(got[1], want[1]))
    one = torch.randn(1, 40, generator=g, device="cuda").to(BF).expand(5, 40)      # rows that are one row
    a, e = L.layer_norm_forward(one, lw), L.layer_norm_forward(one.contiguous(), lw)
    assert torch.equal(a[0], e[0])
