"""AdamW over a list of tensors on the GPU: 32-bit and 8-bit states, the norm and the codec, against plain references."""
import math

import numpy as np
import pytest
import torch

from tests import _multi_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HP = [(1e-3, 1e-8, 0.01), (4e-4, 1e-6, 0.0), (2e-3, 1e-8, 0.1)]
BETAS = (0.9, 0.999)
SIZES = [0, 1, 7, 8, 9, 31, 32, 33, 255, 256, 257, 2047, 2048, 2049, 4095, 5000, 100_003, 0, 1600]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, None: None}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from zero_partitioned_mixed_replica_gb300 import build
    build.build()


def _views(flat, offs, sizes):
    return [flat[o:o + n] for o, n in zip(offs, sizes)]


class Setup:
    """A list of tensors inside flat buffers; `gap` elements between tensors (0: odd offsets everywhere) hold a
    marker that no call may touch."""

    def __init__(self, sizes, grad, out, bits, gap="aligned", scale=1.0, seed=0, **kw):
        from zero_partitioned_mixed_replica_gb300 import multi
        from zero_partitioned_mixed_replica_gb300.engine import AdamW
        self.sizes, self.scale, self.bits = sizes, scale, bits
        gen = torch.Generator().manual_seed(seed)
        at, self.offs = 1 if gap == "odd" else 0, []
        for n in sizes:
            self.offs.append(at)
            at += n if gap == "odd" else -(-(n + 1) // 256) * 256
        total = self.total = at + 64
        r = lambda: torch.randn(total, generator=gen)  # noqa: E731
        self.g = (r() * 1e-3 * scale).to(DT[grad])
        self.p = r() * 0.02
        self.m, self.v = r() * 3e-4, (r() ** 2 + 0.01) * 1e-6
        inside = torch.zeros(total, dtype=torch.bool)
        for o, n in zip(self.offs, sizes):
            inside[o:o + n] = True
        self.inside = inside
        self.groups = [i % 3 for i in range(len(sizes))]
        dev = "cuda"
        self.dg, self.dp = self.g.to(dev), self.p.to(dev)
        self.dout = torch.full((total,), 7.0, dtype=DT[out], device=dev) if out else None
        self.out = out
        groups = [AdamW(lr=a, eps=b, weight_decay=c, beta1=BETAS[0], beta2=BETAS[1]) for a, b, c in HP]
        common = dict(groups=groups, group_of_tensor=self.groups, loss_scale=scale, **kw)
        outs = _views(self.dout, self.offs, sizes) if out else None
        args = (_views(self.dp, self.offs, sizes), _views(self.dg, self.offs, sizes), outs)
        if bits == 32:
            self.dm, self.dv = self.m.to(dev), self.v.to(dev)
            self.opt = multi.MultiAdamW(*args, m=_views(self.dm, self.offs, sizes), v=_views(self.dv, self.offs, sizes), **common)
        else:
            self.opt = multi.MultiAdamW(*args, state_bits=8, **common)
            self.opt.load_states([x.contiguous().to(dev) for x in _views(self.m, self.offs, sizes)],
                                 [x.contiguous().to(dev) for x in _views(self.v, self.offs, sizes)])

    def untouched(self):
        out = ~self.inside
        assert torch.equal(self.dp.cpu()[out], self.p[out])
        assert torch.equal(self.dg.cpu(), self.g)
        if self.dout is not None:
            assert bool((self.dout.cpu()[out] == 7).all())
        if self.bits == 32:
            assert torch.equal(self.dm.cpu()[out], self.m[out]) and torch.equal(self.dv.cpu()[out], self.v[out])


def _check32(s, t, clip):
    """One step against binary64.  Per element, in units u = 2^-24 of the magnitudes involved: m is two products of rounded
    constants and inputs and one sum (constants, unscale and clip at most 1 u each: 6 u of the terms), v 8 u of itself;
    the update takes m's error over den, and sqrt, division, sum, two constants and the product: 16 u of itself; p two
    roundings more and a rounded decay: 4 u of p."""
    dp, dm, dv = s.dp.cpu(), s.dm.cpu(), s.dv.cpu()
    for i, (o, n) in enumerate(zip(s.offs, s.sizes)):
        lr, eps, wd = HP[s.groups[i]]
        sl = slice(o, o + n)
        p, m, v, upd, mmag, mm = R.adamw64(s.p[sl], s.m[sl], s.v[sl], s.g[sl], lr=lr, eps=eps, wd=wd, beta1=BETAS[0],
                                           beta2=BETAS[1], t=t, clip=clip, scale=s.scale)
        assert bool(((dm[sl].double() - m).abs() <= 6 * U * mm + 1e-44).all()), i
        assert bool(((dv[sl].double() - v).abs() <= 8 * U * v + 1e-44).all()), i
        bound = 6 * U * mmag + 16 * U * upd + 4 * U * s.p[sl].double().abs() + 1e-44
        assert bool(((dp[sl].double() - p).abs() <= bound).all()), i
        if s.out:
            assert torch.equal(s.dout.cpu()[sl], dp[sl].to(DT[s.out])), i


@pytest.mark.parametrize("gap", ["aligned", "odd"])
@pytest.mark.parametrize("grad,out", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"), ("fp32", None), ("bf16", None),
                                      ("fp16", "bf16")])
def test_adamw32_against_binary64(grad, out, gap):
    scale = 1024.0 if grad == "fp16" else 1.0
    s = Setup(SIZES, grad, out, 32, gap, scale)
    s.opt.resume_at(6)
    s.opt.update(1)                                  # no norm
    st = s.opt.read_state()
    assert (st["t"], st["apply"], st["skipped"], st["clip_coef"], st["good_steps"]) == (7, 1, 0, 1.0, 1)
    assert st["beta1_pow"] == math.prod([0.9] * 7)
    _check32(s, 7, 1.0)
    s.untouched()


@pytest.mark.parametrize("grad,gap", [("bf16", "aligned"), ("fp16", "odd"), ("fp32", "odd"), ("fp32", "aligned")])
def test_step_with_norm_and_clip(grad, gap):
    scale = 512.0 if grad == "fp16" else 1.0
    s = Setup(SIZES, grad, "bf16", 32, gap, scale, max_norm=0.05)
    s.opt.step()
    g = torch.cat([s.g[o:o + n] for o, n in zip(s.offs, s.sizes)]).double() / scale
    norm = float(g.square().sum().sqrt())
    st = s.opt.read_state()
    # squares and their sums in binary32, groups of 8 (8 roundings), the rest carried: 9 u of the sum, half of that on the norm
    assert abs(st["grad_norm"] - norm) <= 5 * U * norm
    assert abs(st["clip_coef"] - 0.05 / (norm + 1e-6)) <= 6 * U
    assert st["t"] == 1 and st["overflow"] == 0
    _check32(s, 1, st["clip_coef"])
    s.untouched()


def test_list_equals_the_flat_step_bit_for_bit():
    # one rank's flat buffer, once through the flat engine and once as a list of its tensors (odd offsets); the second
    # run takes the flat run's decision, so that both have the same clip coefficient
    from zero_partitioned_mixed_replica_gb300 import binding as B
    from zero_partitioned_mixed_replica_gb300 import multi
    from zero_partitioned_mixed_replica_gb300.engine import AdamW, ZeroStep
    for dtype, dt, max_norm, scale in ((B.ZERO_BF16, torch.bfloat16, 0.0, 1.0), (B.ZERO_FP16, torch.float16, 0.1, 4096.0)):
        numels = [1001, 64, 3, 70_000, 1, 4096]
        hp = AdamW(lr=2e-3, weight_decay=0.05)
        eng = ZeroStep(numels, 1, 2, dtype, adamw=hp, max_norm=max_norm, loss_scale=scale, dynamic_scale=scale > 1)
        gen = torch.Generator("cuda").manual_seed(5)
        p0 = torch.zeros(eng.info.psi_pad, device="cuda")
        p0[:eng.info.psi] = torch.randn(eng.info.psi, generator=gen, device="cuda") * 0.02
        eng.load_master(p0)
        offs = eng.tensor_offsets
        p, m, v = p0.clone(), torch.zeros_like(p0), torch.zeros_like(p0)
        out, g = torch.zeros_like(p0).to(dt), torch.zeros_like(p0).to(dt)
        opt = multi.MultiAdamW(*[_views(x, offs, numels) for x in (p, g, out)], m=_views(m, offs, numels), v=_views(v, offs, numels),
                               groups=[hp], loss_scale=scale, decide=scale > 1)
        for step in range(3):
            g.copy_(torch.randn(p0.numel(), generator=gen, device="cuda") * 1e-2 * scale)
            g[20_000:40_000] = 0                      # a region of zeros, whose update takes another path
            g[eng.info.psi:] = 0
            eng.grads[0].copy_(g)
            eng.step()
            if scale > 1:
                norm = eng.read_state()["grad_norm"]
                opt.grad_norm()
                assert abs(opt.read_state()["grad_norm"] / norm - 1) < 1e-6
                opt.state.copy_(eng.state)            # the scale of opt.grad_norm()'s gradients is kept
                opt.update()
            else:
                opt.step()
            for a, b in ((p, eng.master[0]), (m, eng.m[0]), (v, eng.v[0])):
                assert torch.equal(a.view(torch.int32), b.view(torch.int32)), (dtype, step)
            assert torch.equal(out.view(torch.int16), eng.params[0].view(torch.int16))


@pytest.mark.parametrize("gap", ["aligned", "odd"])
@pytest.mark.parametrize("grad,out", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", None)])
def test_adamw8_against_references(grad, out, gap):
    """Codes and scales bit for bit against the documented form (binary32 operations in the documented order), the
    parameters against binary64 from the same decoded states: the update's bound of the 32-bit step with the approximate
    square root (1 u ... 2 u), division (4 u) and the fused sum inside the same 16 u."""
    scale = 256.0 if grad == "fp16" else 1.0
    s = Setup(SIZES, grad, out, 8, gap, scale, decide=False, seed=4)
    s.opt.seed = 99
    s.opt.resume_at(2)
    m0 = [R.decode_ref(x.cpu(), y.cpu().view(torch.uint8)) for x, y in zip(s.opt.m, s.opt.m_scale)]
    v0 = [R.decode_ref(x.cpu(), y.cpu().view(torch.uint8)) for x, y in zip(s.opt.v, s.opt.v_scale)]
    s.opt.step()
    assert s.opt.read_state()["t"] == 3
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    dp = s.dp.cpu()
    for i, (o, n) in enumerate(zip(s.offs, s.sizes)):
        lr, eps, wd = HP[s.groups[i]]
        sl = slice(o, o + n)
        g = s.g[sl].float() * f(1.0 / scale)
        m = f(0.9) * m0[i] + f(1 - 0.9) * g
        v = f(0.999) * v0[i] + f(1 - 0.999) * (g * g)
        rm, rv = R.random_ints(n, 99, 3, i)
        for what, x, kind, r, code, byte in (("m", m, R.E4M3, rm, s.opt.m[i], s.opt.m_scale[i]),
                                             ("v", v, R.E5M2, rv, s.opt.v[i], s.opt.v_scale[i])):
            c, b = R.encode_ref(x, kind, r)
            assert torch.equal(byte.cpu().view(torch.uint8), b), (what, i)
            assert torch.equal(code.cpu().view(torch.uint8), c.view(torch.uint8)), (what, i)
        p, _, _, upd, mmag, _ = R.adamw64(s.p[sl], m0[i], v0[i], s.g[sl], lr=lr, eps=eps, wd=wd, beta1=BETAS[0], beta2=BETAS[1],
                                          t=3, scale=scale)
        bound = 6 * U * mmag + 16 * U * upd + 4 * U * s.p[sl].double().abs() + 1e-44
        assert bool(((dp[sl].double() - p).abs() <= bound).all()), i
        if out:
            assert torch.equal(s.dout.cpu()[sl], dp[sl].to(DT[out])), i
    s.untouched()


def _check8(s, t, clip, m0, v0):
    """States bit for bit against the documented form, parameters against binary64 (see test_adamw8_against_references)."""
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    dp = s.dp.cpu()
    for i, (o, n) in enumerate(zip(s.offs, s.sizes)):
        lr, eps, wd = HP[s.groups[i]]
        sl = slice(o, o + n)
        g = s.g[sl].float() * f(1.0 / s.scale) * f(clip)
        m = f(0.9) * m0[i] + f(1 - 0.9) * g
        v = f(0.999) * v0[i] + f(1 - 0.999) * (g * g)
        rm, rv = R.random_ints(n, s.opt.seed, t, i)
        for x, kind, r, code, byte in ((m, R.E4M3, rm, s.opt.m[i], s.opt.m_scale[i]), (v, R.E5M2, rv, s.opt.v[i], s.opt.v_scale[i])):
            c, b = R.encode_ref(x, kind, r)
            assert torch.equal(byte.cpu().view(torch.uint8), b), i
            assert torch.equal(code.cpu().view(torch.uint8), c.view(torch.uint8)), i
        p, _, _, upd, mmag, _ = R.adamw64(s.p[sl], m0[i], v0[i], s.g[sl], lr=lr, eps=eps, wd=wd, beta1=BETAS[0], beta2=BETAS[1],
                                          t=t, scale=s.scale, clip=clip)
        bound = 6 * U * mmag + 16 * U * upd + 4 * U * s.p[sl].double().abs() + 1e-44
        assert bool(((dp[sl].double() - p).abs() <= bound).all()), i
        if s.out:
            assert torch.equal(s.dout.cpu()[sl], dp[sl].to(DT[s.out])), i


@pytest.mark.parametrize("seed", range(24))
def test_random_lists(seed):
    rng = np.random.default_rng(1000 + seed)
    sizes = [int(x) for x in np.exp(rng.uniform(0, np.log(60_000), rng.integers(1, 25)))]
    sizes = [0 if rng.random() < 0.1 else n for n in sizes]
    grad = ["bf16", "fp16", "fp32"][rng.integers(3)]
    out = [None, "bf16", "fp16"][rng.integers(3)]
    gap = ["aligned", "odd"][rng.integers(2)]
    bits = [32, 8][rng.integers(2)]
    scale = float(2.0 ** rng.integers(0, 11)) if grad == "fp16" else 1.0
    max_norm = float(10.0 ** rng.uniform(-3, 1))
    s = Setup(sizes, grad, out, bits, gap, scale, seed=seed, max_norm=max_norm, decide=True)
    s.opt.seed = int(rng.integers(1 << 32))
    s.opt.resume_at(int(rng.integers(0, 50)))
    t = s.opt.read_state()["t"] + 1
    if bits == 8:
        m0 = [R.decode_ref(x.cpu(), y.cpu().view(torch.uint8)) for x, y in zip(s.opt.m, s.opt.m_scale)]
        v0 = [R.decode_ref(x.cpu(), y.cpu().view(torch.uint8)) for x, y in zip(s.opt.v, s.opt.v_scale)]
    s.opt.step()
    st = s.opt.read_state()
    norm = math.sqrt(sum(float((s.g[o:o + n].double() / scale).square().sum()) for o, n in zip(s.offs, sizes)))
    assert abs(st["grad_norm"] - norm) <= 5 * U * norm
    assert (st["t"], st["error"], st["apply"]) == (t, 0, 1)
    if bits == 32:
        _check32(s, t, st["clip_coef"])
    else:
        _check8(s, t, st["clip_coef"], m0, v0)
    s.untouched()


@pytest.mark.parametrize("bits", [32, 8])
def test_every_distance_to_a_boundary(bits):
    """Arrays that begin anywhere, each at a distance of its own, give what aligned ones do, bit for bit."""
    from zero_partitioned_mixed_replica_gb300 import multi
    from zero_partitioned_mixed_replica_gb300.engine import AdamW
    n = 5000
    gen = torch.Generator("cuda").manual_seed(8)
    r = lambda: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    g, p, m, v = r() * 1e-3, r() * 0.02, r() * 3e-4, (r() ** 2 + 0.01) * 1e-6
    want = {}
    for case in range(24):
        for dt in (torch.bfloat16, torch.float32):
            # distances in elements: equal ones, one array off, all different
            d = [0] * 5 if case == 0 else [case % 8] * 5 if case < 8 else \
                [(case - 8) % 8 if k == (case - 8) // 4 else 0 for k in range(5)] if case < 20 else [(case * (k + 2)) % 9 for k in range(5)]

            def at(x, off):
                buf = torch.full((n + 32,), 3.0, dtype=x.dtype, device="cuda")
                buf[off:off + n] = x
                return buf, buf[off:off + n]

            bufs = [at(x, off) for x, off in zip((g.to(dt), p, m, v, p.bfloat16()), d)]
            views = [b[1] for b in bufs]
            if bits == 32:
                opt = multi.MultiAdamW([views[1]], [views[0]], [views[4]], m=[views[2]], v=[views[3]], decide=False, groups=[AdamW()])
            else:
                opt = multi.MultiAdamW([views[1]], [views[0]], [views[4]], state_bits=8, decide=False, groups=[AdamW()], seed=5)
                opt.load_states([m], [v])
            opt.step()
            got = [views[1], views[4], opt.m[0], opt.v[0]] + (opt.m_scale + opt.v_scale if bits == 8 else [])
            got = [x.contiguous().view(torch.uint8).clone() for x in got]
            for a, b in zip(got, want.setdefault(dt, got)):
                assert torch.equal(a, b), (case, dt, d)
            for (buf, _), off in zip(bufs[1:2] + bufs[4:], (d[1], d[4])):
                assert bool((buf[:off] == 3).all()) and bool((buf[off + n:] == 3).all())


def _codec_case(x, v):
    from zero_partitioned_mixed_replica_gb300 import multi
    n = x.numel()
    nb = multi.scale_count(n)
    z = lambda k, dt: torch.zeros(k, dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    m32, v32 = x.cuda(), v.cuda()
    m8, v8, ms, vs = z(n, multi.M8), z(n, multi.V8), z(nb, multi.SCALE8), z(nb, multi.SCALE8)
    c = multi.StateCodec8([m32], [v32], [m8], [ms], [v8], [vs])
    c.encode()
    m32.zero_(), v32.zero_()
    c.decode()
    from zero_partitioned_mixed_replica_gb300 import binding as B
    assert B.zero_multi_device_error(c._list.M) == 0
    return m8.cpu(), ms.cpu().view(torch.uint8), v8.cpu(), vs.cpu().view(torch.uint8), m32.cpu(), v32.cpu()


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 2048, 2049, 50_000])
def test_codec_against_references(n):
    rng = np.random.default_rng(n)
    x = torch.from_numpy((rng.standard_normal(n) * np.exp2(rng.integers(-30, 30, n))).astype(np.float32))
    v = x.square() * 2.0 ** -20
    if n >= 64:
        x[:32], v[:32] = 0, 0
        x[32:64] = torch.linspace(-1e-38, 1e-38, 32)          # subnormal values, the smallest scale
        v[32:64] = torch.linspace(0, 1e-44, 32)
    m8, ms, v8, vs, m, w = _codec_case(x, v)
    for val, kind, code, byte, back in ((x, R.E4M3, m8, ms, m), (v, R.E5M2, v8, vs, w)):
        c, b = R.encode_ref(val, kind)
        assert torch.equal(byte, b)
        assert torch.equal(code.view(torch.uint8), c.view(torch.uint8))
        assert torch.equal(back.view(torch.int32), R.decode_ref(c, b).view(torch.int32))


def _placed(x, off, mark):
    """x at `off` elements behind a 256-byte boundary, between marks: (the buffer's bytes, the view)."""
    buf = torch.full(((x.numel() + off + 64) * x.element_size(),), mark, dtype=torch.uint8, device="cuda")
    view = buf[off * x.element_size():(off + x.numel()) * x.element_size()].view(x.dtype)
    view.copy_(x)
    return buf, view


def _marks_stand(buf, view, off, mark):
    a, b = off * view.element_size(), (off + view.numel()) * view.element_size()
    return bool((buf[:a] == mark).all()) and bool((buf[b:] == mark).all())


# distances of (m, v, codes of m, codes of v, scales of m, scales of v) from a boundary, in elements
DISTANCES = [(1, 1, 0, 0, 0, 0), (3, 3, 0, 0, 0, 0), (4, 4, 0, 0, 0, 0), (0, 5, 0, 0, 0, 0), (0, 0, 1, 1, 0, 0), (0, 0, 8, 8, 0, 0),
             (0, 0, 16, 0, 0, 0), (0, 0, 0, 7, 0, 0), (0, 0, 0, 0, 1, 1), (0, 0, 0, 0, 2, 0), (0, 0, 0, 0, 0, 3), (2, 2, 3, 5, 1, 2),
             (7, 6, 15, 13, 3, 1)]


@pytest.mark.parametrize("n", [1, 15, 16, 33, 2048, 5001])
def test_codec_wherever_the_states_begin(n):
    """What aligned states give, bit for bit, and nothing around them is touched."""
    from zero_partitioned_mixed_replica_gb300 import multi
    gen = torch.Generator("cuda").manual_seed(n)
    m, v = torch.randn(n, generator=gen, device="cuda") * 3e-4, torch.rand(n, generator=gen, device="cuda") * 1e-6
    nb = multi.scale_count(n)
    zero = lambda k, dt: torch.zeros(k, dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    want = None
    for d in [(0,) * 6] + DISTANCES:
        arrays = [m, v, zero(n, multi.M8), zero(n, multi.V8), zero(nb, multi.SCALE8), zero(nb, multi.SCALE8)]
        placed = [_placed(x, off, 0xA5) for x, off in zip(arrays, d)]
        pm, pv, m8, v8, ms, vs = (view for _, view in placed)
        codec = multi.StateCodec8([pm], [pv], [m8], [ms], [v8], [vs])
        codec.encode()
        assert torch.equal(pm, m) and torch.equal(pv, v)
        pm.zero_(), pv.zero_()
        codec.decode()
        codec.check()
        got = [x.contiguous().view(torch.uint8).clone() for x in (pm, pv, m8, v8, ms, vs)]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want)), d
        assert all(_marks_stand(*p, off, 0xA5) for p, off in zip(placed, d)), d


@pytest.mark.parametrize("n", [1, 15, 16, 33, 2048, 5001])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_adamw8_wherever_the_states_begin(grad, n):
    from zero_partitioned_mixed_replica_gb300 import multi
    gen = torch.Generator("cuda").manual_seed(n)
    r = lambda: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    g, p, m, v = (r() * 1e-3).to(DT[grad]), r() * 0.02, r() * 3e-4, (r() ** 2 + 0.01) * 1e-6
    nb = multi.scale_count(n)
    zero = lambda k, dt: torch.zeros(k, dtype=torch.uint8, device="cuda").view(dt)  # noqa: E731
    eight = [zero(n, multi.M8), zero(n, multi.V8), zero(nb, multi.SCALE8), zero(nb, multi.SCALE8)]
    multi.StateCodec8([m], [v], [eight[0]], [eight[2]], [eight[1]], [eight[3]]).encode()
    want = None
    for d in [(0,) * 6] + [d for d in DISTANCES if any(d[2:])]:
        for off in (0, 1, 3):                       # of the parameters, their copies and the gradients
            placed = [_placed(x, o, 0xA5) for x, o in zip([p, p.bfloat16(), g] + eight, (off,) * 3 + d[2:])]
            pp, out, pg, m8, v8, ms, vs = (view for _, view in placed)
            opt = multi.MultiAdamW([pp], [pg], [out], state_bits=8, m=[m8], v=[v8], m_scale=[ms], v_scale=[vs], decide=False, seed=6)
            opt.step()
            opt.step()
            assert opt.read_state()["error"] == 0
            got = [x.contiguous().view(torch.uint8).clone() for x in (pp, out, m8, v8, ms, vs)]
            want = want or got
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (d, off)
            assert all(_marks_stand(*x, o, 0xA5) for x, o in zip(placed, (off,) * 3 + d[2:])), (d, off)


def test_codec_of_values_that_are_not_finite():
    x = torch.ones(128)
    x[5], x[40] = math.inf, math.nan
    x[100] = 3.4e38                                             # finite: its block stays finite
    m8, ms, v8, vs, m, v = _codec_case(x, x.abs())
    for back, byte in ((m, ms), (v, vs)):
        assert byte.tolist()[:2] == [255, 255] and bool(torch.isnan(back[:64]).all())
        assert bool(torch.isfinite(back[64:]).all()) and byte[2] != 255


def test_zero_bytes_are_zero_states():
    s = Setup([100, 5], "fp32", None, 8, decide=False)
    m, v = s.opt.states32()
    from zero_partitioned_mixed_replica_gb300 import multi
    fresh = multi.MultiAdamW(_views(s.dp, s.offs, s.sizes), _views(s.dg, s.offs, s.sizes), state_bits=8)
    m, v = fresh.states32()
    assert all(float(x.abs().sum()) == 0 for x in m + v)


def test_loaded_states_come_back_and_the_width_can_change():
    s = Setup([5000, 33, 0, 64], "bf16", "bf16", 8, decide=False)
    m, v = s.opt.states32()
    for a, x, kind in ((m, s.m, R.E4M3), (v, s.v, R.E5M2)):
        for t, o, n in zip(a, s.offs, s.sizes):
            assert torch.equal(t.cpu(), R.decode_ref(*R.encode_ref(x[o:o + n], kind)))
    s.opt.load_states(m, v)
    m2, v2 = s.opt.states32()
    assert all(torch.equal(a, b) for a, b in zip(m + v, m2 + v2))


@pytest.mark.parametrize("bits", [32, 8])
def test_loaded_states_outlast_a_step_under_way_on_another_stream(bits):
    stream = torch.cuda.Stream()
    s = Setup(SIZES + [500_000], "bf16", "bf16", bits, decide=False, stream=stream)
    m = [x.contiguous().cuda() * 2 for x in _views(s.m, s.offs, s.sizes)]
    v = [x.contiguous().cuda() * 2 for x in _views(s.v, s.offs, s.sizes)]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    s.opt.step()
    s.opt.load_states(m, v)
    torch.cuda.synchronize()
    got_m, got_v = s.opt.states32()
    for got, want, kind in ((got_m, m, R.E4M3), (got_v, v, R.E5M2)):
        for a, b in zip(got, want):
            assert torch.equal(a.cpu(), b.cpu() if bits == 32 else R.decode_ref(*R.encode_ref(b.cpu(), kind)))


@pytest.mark.parametrize("bits", [32, 8])
def test_states_that_are_read_are_those_of_one_step(bits):
    # the copies are held up on the current stream while the next step, on another one, is already issued
    stream = torch.cuda.Stream()
    s, other = (Setup(SIZES + [500_000], "bf16", "bf16", bits, decide=False, stream=x) for x in (stream, None))
    other.opt.step()
    want = other.opt.states32()
    torch.cuda.synchronize()
    s.opt.step()
    torch.cuda._sleep(20_000_000)
    got = s.opt.states32()
    s.opt.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0] + got[1], want[0] + want[1]))


# -- the step's decision ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 3e38])
def test_overflow_skips_the_step(bits, value):
    # 3e38: finite, but its square is beyond binary32
    s = Setup([3000, 1, 100], "bf16", "bf16", bits, max_norm=1.0, scale=2.0 ** 15, dynamic_scale=True)
    before = [x.clone() for x in (s.dp, s.dout)] + [x.clone().view(torch.uint8) for x in s.opt.m + s.opt.v]
    s.dg[s.offs[0] + 2999] = value
    s.opt.step()
    st = s.opt.read_state()
    assert (st["t"], st["skipped"], st["overflow"], st["apply"], st["loss_scale"]) == (0, 1, 1, 0, 2.0 ** 14)
    assert st["grad_norm"] == math.inf
    after = [s.dp, s.dout] + [x.view(torch.uint8) for x in s.opt.m + s.opt.v]
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_growing_scale_is_not_applied_to_the_gradients_of_the_step_that_grows_it():
    s = Setup(SIZES, "fp16", "fp16", 32, scale=128.0, dynamic_scale=True, growth_interval=1)
    s.opt.step()
    st = s.opt.read_state()
    assert st["loss_scale"] == 256.0 and st["t"] == 1 and st["good_steps"] == 0
    _check32(s, 1, 1.0)


def test_a_list_of_empty_tensors_still_advances():
    from zero_partitioned_mixed_replica_gb300 import multi
    e = torch.empty(0, device="cuda")
    for bits in (32, 8):
        opt = multi.MultiAdamW([e, e], [e, e], state_bits=bits)
        opt.step()
        opt.grad_norm()
        assert opt.read_state()["t"] == 2 and opt.read_state()["grad_norm"] == 0.0


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_without_the_norm_clears_the_last_decision(bits):
    s = Setup([300, 5], "bf16", "bf16", bits, decide=False)
    s.dg[7] = math.inf
    s.opt.grad_norm()
    assert s.opt.read_state()["overflow"] == 1
    s.dg[7] = 0
    s.opt.step()
    st = s.opt.read_state()
    assert (st["t"], st["overflow"], st["nonfinite"], st["apply"], st["skipped"]) == (1, 0, 0, 1, 1)


def test_zero_gradients_move_nothing_but_the_decay():
    for bits in (32, 8):
        s = Setup([5000], "bf16", "bf16", bits, decide=False)
        s.dg.zero_()
        s.opt.load_states([torch.zeros(5000, device="cuda")], [torch.zeros(5000, device="cuda")])
        s.opt.step()
        lr, _, wd = HP[0]
        want = s.p[:5000] * torch.tensor(1.0 - lr * wd, dtype=torch.float64).float()
        assert torch.equal(s.dp.cpu()[:5000], want)
        m, v = s.opt.states32()
        assert float(m[0].abs().sum() + v[0].sum()) == 0.0


def test_not_finite_gradient_without_a_decision_spoils_its_block_only():
    s = Setup([4096], "fp32", None, 8, decide=False)
    s.dg[100] = math.nan
    s.opt.step()
    m, v = s.opt.states32()
    bad = torch.isnan(m[0]).cpu()
    assert bool(bad[96:128].all()) and int(bad.sum()) == 32
    assert int(torch.isnan(s.dp).sum()) == 1


# -- how it runs --------------------------------------------------------------------------------------------------
def _outputs(s):
    return [s.dp] + ([s.dout] if s.dout is not None else []) + [x.view(torch.uint8) for x in s.opt.m + s.opt.v] + \
        ([x.view(torch.uint8) for x in s.opt.m_scale + s.opt.v_scale] if s.bits == 8 else []) + [s.opt.state]


@pytest.mark.parametrize("bits", [32, 8])
def test_results_do_not_depend_on_the_launch_shape_or_stream(bits):
    from zero_partitioned_mixed_replica_gb300 import binding as B
    sizes = SIZES + [3_000_001]
    ref = None
    for cap, own_stream, graph in ((0, False, False), (1, False, False), (7, True, False), (152, False, True), (0, True, True)):
        old = B.zero_set_max_ctas(cap)
        try:
            stream = torch.cuda.Stream() if own_stream else None
            s = Setup(sizes, "bf16", "bf16", bits, "odd" if bits == 32 else "aligned", max_norm=0.5, stream=stream)
            if graph:
                g = s.opt.capture()
                if stream is not None:
                    torch.cuda.current_stream().wait_stream(stream)
                g.replay()
                g.replay()
            else:
                s.opt.step()
                s.opt.step()
            torch.cuda.synchronize()
        finally:
            B.zero_set_max_ctas(old)
        out = _outputs(s)
        ref = ref or [x.clone() for x in out]
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), (cap, own_stream, graph)


def test_seeds_and_steps_round_differently_and_equal_seeds_alike():
    runs = {}
    for name, seed in (("a", 1), ("b", 1), ("c", 2)):
        s = Setup([20_000], "bf16", "bf16", 8, decide=False)
        s.opt.seed = seed
        s.opt.step()
        runs[name] = [x.cpu().view(torch.uint8) for x in s.opt.m + s.opt.v]
    assert all(torch.equal(a, b) for a, b in zip(runs["a"], runs["b"]))
    assert not any(torch.equal(a, b) for a, b in zip(runs["a"], runs["c"]))


def test_binding_between_the_norm_and_the_update_keeps_the_scale():
    s = Setup(SIZES, "fp16", "fp16", 32, scale=128.0, dynamic_scale=True, growth_interval=1)
    s.opt.grad_norm()                                # the scale grows to 256
    moved = s.dg.clone()
    s.opt.rebind_grads(_views(moved, s.offs, s.sizes))
    s.opt.update()
    _check32(s, 1, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[2048, 2048, 5000], [2048] * 3000, [1, 4096, 0, 2047]], ids=["few", "many", "mixed"])
def test_a_replay_follows_gradients_that_moved(bits, sizes):
    """Recorded with gradients at one distance from a boundary and replayed with them at others, which give a list other
    numbers of tiles: what the same calls give without a recording, bit for bit."""
    from zero_partitioned_mixed_replica_gb300 import multi
    gen = torch.Generator("cuda").manual_seed(9)
    starts = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    r = lambda: torch.randn(starts[-1], generator=gen, device="cuda")  # noqa: E731
    g, p = (r() * 1e-3).bfloat16(), r() * 0.02
    room = [-(-(n + 8) // 8) * 8 for n in sizes]

    def grads(off):                              # every tensor `off` elements behind a boundary
        buf, views, at = torch.zeros(sum(room), dtype=g.dtype, device="cuda"), [], off
        for n, k, o in zip(sizes, room, starts):
            views.append(buf[at:at + n])
            views[-1].copy_(g[o:o + n])
            at += k
        return views

    def run(first, moves, graph):
        q = [p[o:o + n].clone() for o, n in zip(starts, sizes)]
        opt = multi.MultiAdamW(q, grads(first), [x.bfloat16() for x in q], state_bits=bits, max_norm=0.05)
        step = opt.capture().replay if graph else opt.step
        for off in moves:
            opt.rebind_grads(grads(off))
            step()
        st = opt.read_state()
        assert (st["t"], st["error"]) == (len(moves), 0)
        return q + opt.out16 + [x.view(torch.uint8) for x in opt.m + opt.v] + [opt.state]

    for first, moves in ((0, (1, 0, 5)), (1, (0, 0, 7)), (3, (4, 3, 0))):
        for a, b in zip(run(first, moves, True), run(first, moves, False)):
            assert torch.equal(a, b), (first, moves)


def test_rebound_gradients_are_used():
    s = Setup(SIZES, "bf16", "bf16", 32, decide=False)
    s.g = s.g * 2
    moved = s.g.cuda()
    s.opt.rebind_grads(_views(moved, s.offs, s.sizes))
    s.dg.copy_(s.g)                  # for untouched() only
    s.opt.step()
    _check32(s, 1, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_objects_may_go_while_their_work_on_another_stream_is_under_way(bits):
    import gc
    from zero_partitioned_mixed_replica_gb300 import multi
    results = []
    for stream in (None, torch.cuda.Stream()):
        s = Setup(SIZES + [500_000], "bf16", "bf16", bits, decide=False, stream=stream)
        sizes = [x.numel() for x in s.opt.m] + [s.opt._list.workspace.numel()]
        m = [torch.zeros(n, device="cuda") for n in s.sizes]
        v = [torch.zeros(n, device="cuda") for n in s.sizes]
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        moved = _views(s.dg.clone(), s.offs, s.sizes)
        s.opt.rebind_grads(moved)
        s.opt.step()
        if bits == 8:
            multi.StateCodec8(m, v, s.opt.m, s.opt.m_scale, s.opt.v, s.opt.v_scale, stream).decode()
        else:
            s.opt.rebind_grads(_views(s.dg, s.offs, s.sizes))
        del moved, s.opt
        gc.collect()
        junk = [torch.full((n * k,), 255, dtype=torch.uint8, device="cuda") for n in sizes for k in (1, 2, 4)]
        torch.cuda.synchronize()
        results.append([s.dp, s.dout] + (m + v if bits == 8 else [s.dm, s.dv]))
        del junk
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("bits", [32, 8])
def test_memory_comes_back_with_the_last_reference(bits):
    import gc
    s = Setup([100_000, 77], "bf16", "bf16", bits, max_norm=1.0)
    s.opt.step()
    torch.cuda.synchronize()
    gc.collect()
    gc.disable()
    try:
        before = torch.cuda.memory_allocated()
        kept = s.opt.states32()
        s.opt.load_states(*kept)
        del kept
        assert torch.cuda.memory_allocated() == before
        held = s.opt._list.workspace.numel() + (sum(x.numel() for x in s.opt.m + s.opt.v) if bits == 8 else 0)
        del s.opt
        assert torch.cuda.memory_allocated() <= before - held
    finally:
        gc.enable()


@pytest.mark.parametrize("bits", [32, 8])
def test_update_alone_on_an_object_without_decisions_is_a_step(bits):
    a, b = (Setup(SIZES, "bf16", "bf16", bits, decide=False) for _ in range(2))
    a.opt.step(), a.opt.update()
    b.opt.step(), b.opt.step()
    assert a.opt.read_state()["t"] == 2
    assert all(torch.equal(x, y) for x, y in zip(_outputs(a), _outputs(b)))
    a.opt.grad_norm(), a.opt.update()                # a decision all the same: t moves once
    assert a.opt.read_state()["t"] == 3
    a.opt.grad_norm(), a.opt.step()                  # the norm to look at, then a step without a decision
    a.opt.update()
    assert a.opt.read_state()["t"] == 6


def test_refusals():
    from zero_partitioned_mixed_replica_gb300 import binding as B
    from zero_partitioned_mixed_replica_gb300 import multi
    from zero_partitioned_mixed_replica_gb300.engine import AdamW
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    ok = dict(master=[z(64)], grads=[z(64)])
    for bad in (dict(grads=[z(65)]), dict(grads=[z(64, torch.float64)]), dict(grads=[]), dict(master=[z(64, torch.bfloat16)]),
                dict(grads=[z(128)[::2]]), dict(grads=[torch.zeros(64)]), dict(out16=[z(64)]), dict(state_bits=16),
                dict(m=[z(64)]), dict(m=[z(64)], v=[z(64)], state_bits=8), dict(groups=[AdamW(), AdamW(beta2=0.95)]),
                dict(decide=False, max_norm=1.0), dict(decide=False, dynamic_scale=True), dict(master=[z(64), z(64)])):
        with pytest.raises(ValueError):
            multi.MultiAdamW(**{**ok, **bad})
    opt = multi.MultiAdamW(**ok)
    opt.hp[0].lr = -1.0
    with pytest.raises(B.ZeroError) as e:
        opt.step()
    assert e.value.status == B.ZERO_ERR_INVALID
    opt.hp[0].lr = 1e-3
    for call, status in ((lambda: opt.update(4), B.ZERO_ERR_INVALID),
                         (lambda: B.zero_multi_adamw8(opt._list.M, opt.hp, 0, 0, opt.state), B.ZERO_ERR_STATE),
                         (lambda: B.zero_multi_encode8(opt._list.M), B.ZERO_ERR_STATE),
                         (lambda: B.zero_multi_grad_norm(opt._list.M, math.nan, opt.state), B.ZERO_ERR_INVALID),
                         (lambda: B.zero_multi_adamw(opt._list.M, opt.hp, 1, opt.state[16:]), B.ZERO_ERR_ALIGN)):
        with pytest.raises(B.ZeroError) as e:
            call()
        assert e.value.status == status
    with pytest.raises(ValueError):
        opt.resume_at(-1)
    norm_only = multi.MultiAdamW(None, [z(64)])
    norm_only.grad_norm()
    with pytest.raises(B.ZeroError) as e:
        norm_only.step()
    assert e.value.status == B.ZERO_ERR_STATE


@pytest.mark.slow
def test_tensor_beyond_32_bit_offsets():
    # 2^32 + 77 elements: element and byte offsets pass 32 bits.  Everything before the last chunks is zero and stays so.
    from zero_partitioned_mixed_replica_gb300 import multi
    from zero_partitioned_mixed_replica_gb300.engine import AdamW
    n, tail = (1 << 32) + 77, 5000
    gen = torch.Generator().manual_seed(2)
    g = (torch.randn(tail, generator=gen) * 1e-3).bfloat16()
    p = torch.randn(tail, generator=gen) * 0.02
    dg = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    dp = torch.zeros(n, device="cuda")
    dg[-tail:], dp[-tail:] = g.cuda(), p.cuda()
    opt = multi.MultiAdamW([dp], [dg], state_bits=8, groups=[AdamW(lr=1e-3)], max_norm=1e6, seed=3)
    opt.step()
    st = opt.read_state()
    norm = float(g.double().square().sum().sqrt())
    assert abs(st["grad_norm"] - norm) <= 5 * U * norm
    want, m, v, upd, mmag, _ = R.adamw64(p, torch.zeros(tail), torch.zeros(tail), g, lr=1e-3, eps=1e-8, wd=0.01, beta1=0.9,
                                         beta2=0.999, t=1)
    bound = 6 * U * mmag + 16 * U * upd + 4 * U * p.double().abs() + 1e-44
    assert bool(((dp[-tail:].cpu().double() - want).abs() <= bound).all())
    for at in range(0, n - tail, 1 << 30):
        end = min(n - tail, at + (1 << 30))
        assert not bool(dp[at:end].any()) and not bool(opt.m[0][at:end].view(torch.uint8).any())

    back = opt.m[0][-tail:].cpu().float()
    assert int((back != 0).sum()) > tail // 2
