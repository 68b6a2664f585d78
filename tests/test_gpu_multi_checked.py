"""The list updates and the codec in the bounds-checked build: their suites run inside the tensors, and with every
extent shortened by the build's test hook each kind of launch reports the accesses it skipped."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def checked_env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from zero_partitioned_mixed_replica_gb300 import build
    env = dict(os.environ)
    env["ZERO_LIB"] = build.build(checked=True)
    return env


def test_suites_run_inside_their_tensors(checked_env):
    p = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_multi.py", "tests/test_gpu_state8_engine.py", "-q", "-x",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=checked_env, capture_output=True, text=True, timeout=900)
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-2000:]
    assert " passed" in p.stdout


CONTROL = r"""
import torch
from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300.multi import MultiAdamW, StateCodec8
assert B.zero_checked_build()
sizes = [10000, 33, 4096, 0, 700]
new = lambda dt=torch.float32: [torch.full((n,), 0.5, dtype=dt, device="cuda") for n in sizes]
res = {}
for bits in (32, 8):
    opt = MultiAdamW(new(), new(torch.bfloat16), new(torch.bfloat16), state_bits=bits, max_norm=1.0)
    calls = {"norm%d" % bits: opt.grad_norm, "update%d" % bits: opt.update}
    if bits == 8:
        codec = StateCodec8(new(), new(), opt.m, opt.m_scale, opt.v, opt.v_scale)
        calls.update(encode=codec.encode, decode=codec.decode)
    for name, run in calls.items():
        for slack in (0, 40, 0):
            B.zero_checked_set_slack(slack)
            run()
            torch.cuda.synchronize()
            hits = B.zero_bounds_violations(reset=True)
            assert (hits > 0) == (slack > 0), (name, slack, hits)
            assert opt.read_state()["error"] == 0
        res[name] = True
    if bits == 8:
        assert B.zero_multi_device_error(codec._list.M) == 0
assert len(res) == 6
"""


def test_checks_fire_when_the_extents_are_short(checked_env):
    p = subprocess.run([sys.executable, "-c", CONTROL], cwd=ROOT, env=checked_env, capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stdout[-3000:] + p.stderr[-3000:]
