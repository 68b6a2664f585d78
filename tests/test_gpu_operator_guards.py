"""The operators' calls write their outputs and their workspaces and nothing beside them, and leave their inputs alone: every
array of a call lies between guard bands, workspaces are of exactly the size that the query gives."""
import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
CODE = {BF: B.ZERO_BF16, HF: B.ZERO_FP16, FP: B.ZERO_FP32}
BAND = 4096


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


class Arrays:
    """Arrays between bands of BAND bytes of 0xA5, filled with 0xFF: NaN in every type, which no output of the finite inputs
    here is.  An odd one begins one element after a 256-byte boundary."""

    def __init__(self):
        self.gen = torch.Generator("cuda").manual_seed(11)
        self.all, self.inputs = [], []

    def out(self, dtype, *shape, odd=False):
        n, size = 1, torch.empty(0, dtype=dtype).element_size()
        for s in shape:
            n *= s
        at = BAND + (size if odd else 0)
        raw = torch.full((at + n * size + BAND,), 0xA5, dtype=torch.uint8, device="cuda")
        raw[at:at + n * size] = 0xFF
        self.all.append((raw, at, n * size))
        return raw[at:at + n * size].view(dtype).view(shape)

    def given(self, values, odd=False):
        v = self.out(values.dtype, *values.shape, odd=odd)
        v.copy_(values)
        self.inputs.append((v, v.clone()))
        return v

    def randn(self, dtype, *shape, odd=False):
        return self.given(torch.randn(*shape, generator=self.gen, device="cuda").to(dtype), odd)

    def ids(self, n, below):
        return self.given(torch.randint(-1, below + 1, (n,), generator=self.gen, device="cuda"))

    def bytes(self, n):
        return self.out(torch.uint8, n)

    def check(self, *outs):
        torch.cuda.synchronize()
        for raw, at, n in self.all:
            assert bool((raw[:at] == 0xA5).all()) and bool((raw[at + n:] == 0xA5).all())
        for v, was in self.inputs:
            assert torch.equal(v.view(torch.uint8), was.view(torch.uint8))
        for o in outs:          # written from end to end
            assert not bool(o.isnan().any())


ROWS = [(1, 1, BF, False), (3, 1001, BF, False), (200, 768, HF, False), (200, 768, HF, True), (153, 4104, BF, False), (153, 4104, BF, True),
        (310, 8200, FP, False), (33, 16384, BF, False), (33, 16383, HF, True), (999, 96, FP, True)]


@pytest.mark.parametrize("n,d,dtype,odd", ROWS)
@pytest.mark.parametrize("bias", [False, True])
def test_layer_norm(n, d, dtype, odd, bias):
    a = Arrays()
    x, w, b = a.randn(dtype, n, d, odd=odd), a.randn(dtype, d, odd=odd), a.randn(dtype, d, odd=odd)
    y, mean, rstd = a.out(dtype, n, d, odd=odd), a.out(FP, n), a.out(FP, n)
    B.zero_layer_norm_forward(x, d, w, b if bias else None, n, d, CODE[dtype], 1e-5, y, mean, rstd)
    a.check(y, mean, rstd)
    gy, gx = a.randn(dtype, n, d), a.out(dtype, n, d)
    for to in {dtype, FP}:
        gw, gb = a.out(to, d, odd=odd), a.out(to, d)
        ws = a.bytes(B.zero_layer_norm_workspace(n, d))
        B.zero_layer_norm_backward(gy, d, x, d, w, mean, rstd, n, d, CODE[dtype], CODE[to], False, gx, gw, gb if bias else None, ws)
        a.check(gx, gw, *([gb] if bias else []))


@pytest.mark.parametrize("n,d,dtype,odd", ROWS + [(2049, 64, BF, False), (9000, 40, HF, True), (100000, 24, BF, False), (100, 70001, BF, True)])
@pytest.mark.parametrize("vocab", [1, 257, 5003])
def test_embedding(n, d, dtype, odd, vocab):
    if vocab * d > 50_000_000:
        vocab = 50
    a = Arrays()
    w, ids, out = a.randn(dtype, vocab, d, odd=odd), a.ids(n, vocab), a.out(dtype, n, d)
    B.zero_embedding_forward(w, ids, vocab, d, n, CODE[dtype], 1.5, out)
    a.check(out)
    g = a.randn(dtype, n, d)
    for to in {dtype, FP}:
        gw, ws = a.out(to, vocab, d, odd=odd), a.bytes(B.zero_embedding_workspace(vocab, d, n))
        for accumulate in (False, True):
            B.zero_embedding_backward(g, ids, vocab, d, n, CODE[dtype], CODE[to], 0.5, accumulate, gw, ws)
            a.check(gw)


# one CTA's tiles and pairs', copied weights, rows that the products write themselves, pieces, parts, sums in several runs
@pytest.mark.parametrize("n,d,vocab,dtype,odd,piece", [
    (1, 8, 16, BF, False, 0), (5, 24, 40, BF, True, 0), (128, 512, 1000, HF, False, 256), (128, 520, 777, BF, False, 0), (129, 64, 256, HF, False, 0),
    (300, 200, 1777, BF, False, 512), (300, 31, 513, HF, True, 0), (3000, 256, 3000, BF, False, 512), (1000, 1600, 5000, HF, False, 0),
    (130, 8256, 300, BF, False, 0), (33000, 48, 500, BF, False, 256), (257, 1, 1, BF, False, 0)])
def test_loss(n, d, vocab, dtype, odd, piece):
    a = Arrays()
    args = B.zero_lm_loss_args(n=n, d=d, vocab=vocab, hidden_stride=d, dtype=CODE[dtype], piece=piece)
    h, w, t = a.randn(dtype, n, d), a.randn(dtype, vocab, d, odd=odd), a.ids(n, vocab)
    losses, lse, stats = a.out(FP, n), a.out(FP, n), a.out(FP, 2)
    args.hidden, args.weight, args.targets = h.data_ptr(), w.data_ptr(), t.data_ptr()
    args.losses, args.lse, args.stats = losses.data_ptr(), lse.data_ptr(), stats.data_ptr()
    forward, backward = B.zero_lm_loss_query(args)
    ws = a.bytes(forward)
    args.workspace = ws.data_ptr()
    B.zero_lm_loss_forward(args)
    a.check(losses, lse, stats)
    assert B.zero_lm_loss_device_error(ws) == 0
    a.inputs += [(x, x.clone()) for x in (lse, stats)]
    ws = a.bytes(backward)
    args.workspace, args.scale = ws.data_ptr(), 8.0
    for odd_gradients in (False, True):
        gh, gw = a.out(dtype, n, d, odd=odd_gradients), a.out(dtype, vocab, d, odd=odd_gradients)
        for hidden, weight in ((True, True), (True, False), (False, True)):
            args.grad_hidden, args.grad_weight = gh.data_ptr() if hidden else None, gw.data_ptr() if weight else None
            B.zero_lm_loss_backward(args)
            a.check(*([gh] if hidden else []), *([gw] if weight else []))
    assert B.zero_lm_loss_device_error(ws) == 0
