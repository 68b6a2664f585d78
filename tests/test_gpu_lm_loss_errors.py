"""What a loss call leaves behind when one of its kernels has reported an error: NaN that every later reader meets, the
backward call and the step's decision among them.  A test program sets the error word between the kernels; no wait runs out."""
import os
import subprocess

import pytest
import torch

from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import layers as L
from zero_partitioned_mixed_replica_gb300.engine import ZeroStep

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from zero_partitioned_mixed_replica_gb300 import build
    build.build()


def test_an_error_shows_in_the_loss_and_in_the_gradients(tmp_path):
    exe = str(tmp_path / "loss_errors")
    pkg = os.path.join(ROOT, "zero_partitioned_mixed_replica_gb300")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-fmad=false",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(pkg, "csrc"),
                    os.path.join(ROOT, "tests", "native", "loss_errors.cu"), "-L", pkg, "-lzero", "-Xlinker", "-rpath," + pkg, "-o", exe],
                   check=True, capture_output=True, timeout=600)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "failures=0 cuda=0" in p.stdout, p.stdout + p.stderr


@pytest.mark.parametrize("dtype,d", [(torch.float16, 64), (torch.bfloat16, 64), (torch.bfloat16, 65)])
def test_a_forward_calls_error_skips_the_step(dtype, d):
    # what such a call saves: NaN as the loss and as the share of a token in it
    vocab, n = 100, 200
    eng = ZeroStep([3, vocab * d], 2, 2, B.ZERO_FP16 if dtype is torch.float16 else B.ZERO_BF16, max_norm=1.0, dynamic_scale=True,
                   loss_scale=64.0)
    g = torch.Generator("cuda").manual_seed(2)
    eng.load_master(torch.randn(eng.info.psi_pad, generator=g, device="cuda"))
    before = eng.params.clone()
    h = torch.randn(n, d, generator=g, device="cuda").to(dtype)
    t = torch.randint(vocab, (n,), generator=g, device="cuda")
    for r in range(2):
        table = eng.tensor_view(eng.params[r], 1, (vocab, d))
        _, _, saved = L.lm_loss_forward(h, table, t)
        if r == 1:
            saved[:2] = float("nan")
        gh = L.lm_loss_backward(h, table, t, saved, eng.tensor_view(eng.grads[r], 1, (vocab, d)), scale=eng.loss_scale)
        assert bool(gh.isnan().all()) == (r == 1)
    eng.step()
    state = eng.read_state()
    assert state["overflow"] == 1 and state["t"] == 0 and state["loss_scale"] == 32.0
    assert torch.equal(eng.params, before)
