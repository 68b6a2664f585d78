"""ZeroStep with 8-bit states: the flat engine's split step with the list update on its rank shards."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle.step import FMT_BF16, FMT_FP16
from tests import _multi_ref as R
from tests._cases import Case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CASES = {
    "zero2_bf16": Case([1001, 64, 3, 70_000, 1, 4096], 4, 2, FMT_BF16, bucket_elems=32_768, grad_std=1e-2),
    "zero1_fp16_clip": Case([50_000, 777, 33], 3, 1, FMT_FP16, grad_std=1e-2, max_norm=0.5, loss_scale=1024.0, dynamic=True),
    "zero3_bf16": Case([30_000, 60_000, 640, 45_000, 7, 20_000, 3], 2, 3, FMT_BF16, units=[0, 1, 1, 2, 0, 3, 3], grad_std=1e-2),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from zero_partitioned_mixed_replica_gb300 import build
    build.build()


def _engine(c, bits=8, **kw):
    from zero_partitioned_mixed_replica_gb300.engine import ZeroStep
    return ZeroStep(c.numels, c.n_d, c.stage, c.fmt, c.bucket_elems, c.units, max_norm=c.max_norm, loss_scale=c.loss_scale,
                    dynamic_scale=c.dynamic, state_bits=bits, seed=11, **kw)


def _feed(eng, c, L, step):
    for r, g in enumerate(c.grads_torch(L, step, c.loss_scale)):
        eng.grads[r].copy_(g.cuda())


@pytest.mark.parametrize("name", list(CASES))
def test_states_bit_for_bit_and_parameters_within_the_update_s_bound(name):
    c = CASES[name]
    L = c.layout()
    eng = _engine(c)
    eng.load_master(torch.from_numpy(c.master0(L)))
    for step in (1, 2, 3):
        m0, v0 = (x.cpu() for x in eng.states32())
        p0 = eng.master.cpu().clone()
        _feed(eng, c, L, step)
        eng.step()
        st = eng.read_state()
        assert (st["t"], st["apply"], st["error"]) == (step, 1, 0)
        clip = torch.tensor(st["clip_coef"], dtype=torch.float32)
        f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
        for r in range(c.n_d):
            g = eng.gshard[r].cpu() * clip
            m = f(0.9) * m0[r] + f(1 - 0.9) * g
            v = f(0.999) * v0[r] + f(1 - 0.999) * (g * g)
            rm, rv = R.random_ints(g.numel(), 11, step, r)
            for x, kind, rnd, code, byte in ((m, R.E4M3, rm, eng.m[r], eng.m_scale[r]), (v, R.E5M2, rv, eng.v[r], eng.v_scale[r])):
                q, b = R.encode_ref(x, kind, rnd)
                assert torch.equal(byte.cpu().view(torch.uint8), b)
                assert torch.equal(code.cpu().view(torch.uint8), q.view(torch.uint8))
            p, _, _, upd, mmag, _ = R.adamw64(p0[r], m0[r], v0[r], eng.gshard[r].cpu(), lr=1e-3, eps=1e-8, wd=0.01, beta1=0.9,
                                              beta2=0.999, t=step, clip=float(clip))
            # the bound of the list update (tests/test_gpu_multi.py)
            bound = 6 * U * mmag + 16 * U * upd + 4 * U * p0[r].double().abs() + 1e-44
            assert bool(((eng.master[r].cpu().double() - p).abs() <= bound).all())
        want = eng.flat("master").to(eng.grads.dtype)
        if c.stage == 3:
            assert torch.equal(eng.flat("shard16").view(torch.int16), want.view(torch.int16))
        else:
            for r in range(c.n_d):
                assert torch.equal(eng.params[r].view(torch.int16), want.view(torch.int16))


def test_overflow_skips_and_halves_the_scale():
    c = CASES["zero1_fp16_clip"]
    L = c.layout()
    eng = _engine(c)
    eng.load_master(torch.from_numpy(c.master0(L)))
    _feed(eng, c, L, 1)
    eng.step()
    before = [x.clone().view(torch.uint8) for x in (eng.master, eng.m, eng.v, eng.m_scale, eng.v_scale, eng.params)]
    eng.grads[1][5] = float("inf")
    eng.step()
    st = eng.read_state()
    assert (st["t"], st["skipped"], st["overflow"], st["loss_scale"]) == (1, 1, 1, 512.0)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in
               zip(before, (eng.master, eng.m, eng.v, eng.m_scale, eng.v_scale, eng.params)))


@pytest.mark.parametrize("stage", [1, 2, 3])
def test_accumulated_micro_batches_equal_one_batch_of_their_sum(stage):
    # the same gradients twice: the accumulated average is the gradient itself (sums of two equal numbers are exact)
    c = Case([3000, 500, 41], 2, stage, FMT_BF16, units=[0, 1, 1] if stage == 3 else None, grad_std=1e-2)
    L = c.layout()
    a, b = _engine(c, n_micro=2), _engine(c)
    for e in (a, b):
        e.load_master(torch.from_numpy(c.master0(L)))
        _feed(e, c, L, 1)
    a.micro_step(0)
    a.micro_step(1)
    b.step()
    for x, y in ((a.master, b.master), (a.m, b.m), (a.v, b.v), (a.m_scale, b.m_scale)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert a.read_state()["t"] == b.read_state()["t"] == 1


@pytest.mark.parametrize("stage", [1, 2, 3])
def test_a_whole_step_of_an_accumulating_engine_is_one_batch(stage):
    c = Case([3000, 500, 41], 2, stage, FMT_BF16, units=[0, 1, 1] if stage == 3 else None, grad_std=1e-2)
    L = c.layout()
    a, b = _engine(c, n_micro=2), _engine(c)
    for e in (a, b):
        e.load_master(torch.from_numpy(c.master0(L)))
    for step in (1, 2, 3):
        for e in (a, b):
            _feed(e, c, L, step)
        if step < 3:
            a.step()
        else:
            a.capture().replay()
        b.step()
        for x, y in ((a.gshard, b.gshard), (a.master, b.master), (a.m, b.m), (a.v, b.v), (a.m_scale, b.m_scale)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), step
        assert a.read_state() == b.read_state()


def test_captured_step_and_transients():
    c = CASES["zero3_bf16"]
    L = c.layout()
    a, b = _engine(c), _engine(c)
    seen = []
    a.transient_hook = lambda kind, unit, rows: seen.append((kind, unit))
    for e in (a, b):
        e.load_master(torch.from_numpy(c.master0(L)))
        _feed(e, c, L, 1)
    g = b.capture()
    g.replay()
    g.replay()
    a.step()
    a.step()
    n = len(a.units)
    assert seen == 2 * ([("fwd", u) for u in range(n)] + [("bwd", u) for u in reversed(range(n))])
    for x, y in ((a.master, b.master), (a.m, b.m), (a.v, b.v), (a.shard16, b.shard16)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_checkpoints_cross_widths_and_partitions(tmp_path):
    c = CASES["zero2_bf16"]
    L = c.layout()
    eng = _engine(c)
    eng.load_master(torch.from_numpy(c.master0(L)))
    for step in (1, 2):
        _feed(eng, c, L, step)
        eng.step()
    eng.save_checkpoint(str(tmp_path))
    psi = eng.info.psi
    m, v, p = (eng.flat(x)[:psi].clone() for x in ("m", "v", "master"))
    same = _engine(c)
    same.load_checkpoint(str(tmp_path))
    assert torch.equal(same.flat("m")[:psi], m) and torch.equal(same.flat("v")[:psi], v)      # values survive
    assert torch.equal(same.params.view(torch.int16), eng.params.view(torch.int16))
    assert same.read_state()["t"] == 2
    wide = _engine(Case(c.numels, 2, 1, c.fmt), bits=32)
    wide.load_checkpoint(str(tmp_path))
    assert torch.equal(wide.flat("m")[:psi], m) and torch.equal(wide.flat("v")[:psi], v) and torch.equal(wide.flat("master")[:psi], p)
    # another partition has other blocks: each value within half a step of its block's code (E4M3: 2^-4 of it, or the
    # smallest code's half, 2^-10 of the scale; E5M2: 2^-3, 2^-17), the scale at most 2^-7 (2^-14) of the block's largest
    other = _engine(Case(c.numels, 3, 1, c.fmt))
    other.load_checkpoint(str(tmp_path))
    for name, want, rel, least in (("m", m, 2.0 ** -4, 2.0 ** -17), ("v", v, 2.0 ** -3, 2.0 ** -30)):
        got = other.flat(name)[:psi]
        top = torch.nn.functional.max_pool1d(want.abs()[None, None], 127, 1, 63)[0, 0]      # any block that holds it lies in there
        assert bool(((got - want).abs() <= rel * want.abs() + least * top).all()), name


@pytest.mark.parametrize("n_d,elems", [(2, 1 << 18), (3, 400_001)])
def test_checkpoints_of_8_bit_states_take_little_device_memory(tmp_path, monkeypatch, n_d, elems):
    """The fp32 values go through pieces, not through whole copies of the states (8 bytes a parameter): with pieces of
    65,536 bytes, less than a quarter of that."""
    from zero_partitioned_mixed_replica_gb300 import engine
    monkeypatch.setattr(engine, "STAGE_BYTES", 1 << 16)
    c = Case([elems, 3001, 77], n_d, 2, FMT_BF16, grad_std=1e-2)
    L = c.layout()
    eng = _engine(c)
    eng.load_master(torch.from_numpy(c.master0(L)))
    _feed(eng, c, L, 1)
    eng.step()
    m, v = (x.cpu() for x in eng.states32())
    whole = 8 * eng.master.numel()
    other = _engine(c)
    for call in (eng.save_checkpoint, other.load_checkpoint):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call(str(tmp_path))
        assert torch.cuda.max_memory_allocated() - before <= whole / 4
    S = eng.info.shard_len
    for r in range(n_d):
        f32 = np.fromfile(tmp_path / ("rank%03d.bin" % r), np.float32, 3 * S)
        assert np.array_equal(f32[S:2 * S], m[r].numpy()) and np.array_equal(f32[2 * S:], v[r].numpy())
    for a, b in zip(other.states32(), (m, v)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("bits", [32, 8])
def test_loads_and_reads_around_steps_under_way_on_another_stream(tmp_path, bits):
    c = CASES["zero2_bf16"]
    L = c.layout()
    stream = torch.cuda.Stream()
    p0 = torch.from_numpy(c.master0(L))
    p1 = torch.from_numpy(c.master0(L)) * 2
    eng, ref = _engine(c, bits, stream=stream), _engine(c, bits)
    for e in (eng, ref):
        e.load_master(p0)
        _feed(e, c, L, 1)
    torch.cuda.synchronize()
    ref.step()
    ref.save_checkpoint(str(tmp_path))
    want = {x: ref.flat(x) for x in ("master", "m", "v")}
    hold = lambda: torch.cuda._sleep(20_000_000)  # noqa: E731

    eng.step()                              # reads: the copies are held up, the next step is already issued
    hold()
    got = {x: eng.flat(x) for x in want}
    eng.step()
    torch.cuda.synchronize()
    assert all(torch.equal(got[x], want[x]) for x in want)
    with torch.cuda.stream(stream):         # loads: the step before is held up
        hold()
    eng.step()
    eng.load_checkpoint(str(tmp_path))
    assert all(torch.equal(eng.flat(x), want[x]) for x in want)
    with torch.cuda.stream(stream):
        hold()
    eng.step()
    eng.load_master(p1.cuda())
    torch.cuda.synchronize()
    assert torch.equal(eng.flat("master").cpu(), p1) and not bool(eng.flat("m").any())


def test_an_error_of_the_codec_is_not_lost(tmp_path, monkeypatch):
    """Nothing is made to fail on the GPU: the error word that a kernel would set is set behind it."""
    from zero_partitioned_mixed_replica_gb300 import binding as B
    from zero_partitioned_mixed_replica_gb300 import multi
    c = Case([3000, 500, 41], 2, 2, FMT_BF16)
    eng = _engine(c)
    eng.save_checkpoint(str(tmp_path))
    opt = multi.MultiAdamW([torch.zeros(100, device="cuda")], [torch.zeros(100, device="cuda")], state_bits=8)
    m, v = opt.states32()
    opt.load_states(m, v)
    assert opt.read_state()["error"] == 0 and eng.flat("m").any() == False and eng.read_state()["error"] == 0  # noqa: E712
    seen = []

    def after(call):
        def run(self):
            call(self)
            self._list.error_word().fill_(4)
            seen.append(B.zero_multi_device_error(self._list.M))
        return run

    monkeypatch.setattr(multi.StateCodec8, "decode", after(multi.StateCodec8.decode))
    opt.states32()
    assert opt.read_state()["error"] == 4
    eng.flat("m")
    assert eng.read_state()["error"] == 4
    with pytest.raises(RuntimeError, match="8-bit states"):
        eng.save_checkpoint(str(tmp_path / "other"))
    monkeypatch.setattr(multi.StateCodec8, "encode", after(multi.StateCodec8.encode))
    opt.state.zero_()
    opt.load_states(m, v)
    assert opt.read_state()["error"] == 4
    with pytest.raises(RuntimeError, match="8-bit states"):
        eng.load_checkpoint(str(tmp_path))
    assert seen and set(seen) == {4}


def test_refusals():
    from zero_partitioned_mixed_replica_gb300.engine import ZeroStep
    for kw in (dict(state_bits=16), dict(state_bits=8, fused=True), dict(state_bits=8, live_units=2, unit_of_tensor=[0])):
        with pytest.raises(ValueError):
            ZeroStep([100], 2, 3 if "live_units" in kw else 2, **kw)
    eng = ZeroStep([100], 2, 2, state_bits=8)
    with pytest.raises(ValueError):
        eng.step_from_host(torch.zeros(eng.grads.shape, dtype=eng.grads.dtype).pin_memory())


def test_the_example_learns_with_either_width():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import many_tensors
    last = {}
    for bits in (32, 8):
        losses = many_tensors.train(steps=200, state_bits=bits, say=lambda s: None)
        assert all(np.isfinite(losses))
        last[bits] = float(np.mean(losses[-10:]))
        assert losses[0] > 4.0 and last[bits] < 0.5        # from ln(97) = 4.6
    assert last[8] < 3 * last[32] + 0.1
