"""The grids that the operators' calls launch, read from captured graphs: capped as the header says, and chosen by the call's
own sizes whatever calls came before."""
import ctypes
import json
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
from zero_partitioned_mixed_replica_gb300 import binding as B  # noqa: E402
from zero_partitioned_mixed_replica_gb300 import layers as L  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
KERNEL_NODE = 0


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in
                                              ("gx", "gy", "gz", "bx", "by", "bz", "shared")] + [
        ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """[(CTAs, threads of a CTA)] of the kernels that a call launches, in order, torch's own left out by capturing the
    call alone; nothing of it is run."""
    cu = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    count = ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    out = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == KERNEL_NODE:
            k = KernelNode()
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)) == 0
            out.append((k.gx * k.gy * k.gz, k.bx * k.by * k.bz))
    return out


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    B.zero_set_max_ctas(0)


@pytest.mark.parametrize("cap", [1, 2, 3, 4, 5, 7, 8, 12, 15, 16, 31, 100])
@pytest.mark.parametrize("n", [100, 2048, 2049, 30000, 200000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_within_the_cap(n, cap, accumulate):
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    g = torch.zeros(n, 8, dtype=BF, device="cuda")
    gw = torch.zeros(40000, 8, dtype=BF, device="cuda")
    B.zero_set_max_ctas(cap)
    got = launches(lambda: L.embedding_backward(g, ids, gw, accumulate=accumulate))
    assert len(got) == 3
    # the first launch sorts and zeroes: two CTAs at least, where there are zeros to write
    assert got[0][0] <= max(cap, 1 if accumulate else 2), got
    assert all(ctas <= cap for ctas, _ in got[1:]), got


@pytest.mark.parametrize("n", [2049, 9000, 98304, 98305, 200000])
def test_embedding_gradient_under_caps_is_the_same(n):
    # clusters of 1, 2, 4 and 8 that sort, in shared memory and outside it
    g = torch.Generator("cuda").manual_seed(n)
    ids = torch.randint(-3, 70000, (n,), generator=g, device="cuda")
    ids[: n // 2] %= 50
    go = torch.randn(n, 24, generator=g, device="cuda").to(BF)
    want = L.embedding_backward(go, ids, torch.empty(66000, 24, dtype=BF, device="cuda"))
    inside = (ids >= 0) & (ids < 66000)
    count = torch.bincount(ids[inside], minlength=66000)
    plain = torch.zeros(66000, 24, dtype=torch.float64, device="cuda").index_add_(0, ids[inside], go[inside].double())
    size = torch.zeros_like(plain).index_add_(0, ids[inside], go[inside].double().abs())
    # each addition and the product off by 2^-24 of the magnitudes, then the rounding to bf16
    tol = (count[:, None] + 3) * 2.0 ** -24 * size
    assert bool(((want.double() - plain).abs() <= tol + 2.0 ** -8 * (plain.abs() + tol)).all())
    for accumulate in (False, True):
        for cap in (1, 2, 4, 5, 7, 8, 15, 16, 100):
            B.zero_set_max_ctas(cap)
            got = L.embedding_backward(go, ids, torch.zeros_like(want) if accumulate else torch.full_like(want, 5.0), accumulate=accumulate)
            assert torch.equal(got, want), (accumulate, cap)


OPERATORS = ["embedding", "norm", "norm gradient", "loss", "loss gradient", "loss gradient, copies"]


@pytest.mark.parametrize("cap", [1, 2, 7, 40])
@pytest.mark.parametrize("n", [3, 129, 5000])
@pytest.mark.parametrize("op", OPERATORS)
def test_the_other_operators_within_the_cap(op, n, cap):
    d, vocab, at = 128, 3000, 1 if "copies" in op else 0
    x, w = torch.zeros(n, d, dtype=BF, device="cuda"), torch.zeros(vocab * d + 8, dtype=BF, device="cuda")[at:at + vocab * d].view(vocab, d)
    ids, row, per_row = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(d, dtype=BF, device="cuda"), torch.zeros(n, device="cuda")
    gw, grow, saved = torch.zeros_like(w), torch.zeros_like(row), torch.zeros(2 + n, device="cuda")
    B.zero_set_max_ctas(cap)
    got = launches({"embedding": lambda: L.embedding_forward(w, ids),
                    "norm": lambda: L.layer_norm_forward(x, row),
                    "norm gradient": lambda: L.layer_norm_backward(x, x, row, per_row, per_row, grow),
                    "loss": lambda: L.lm_loss_forward(x, w, ids)}.get(op, lambda: L.lm_loss_backward(x, w, ids, saved, gw, piece=1024)))
    assert got and all(ctas <= cap + cap % 2 for ctas, _ in got if "loss" in op), got   # the next even number
    assert "loss" in op or all(ctas <= cap for ctas, _ in got), got


WIDTHS = [2304, 4096, 8192, 9000, 16384, 1025, 2049, 8191, 16383, 1026, 5002, 16382]    # 16-byte pieces, single elements, pairs


def _grids(widths):
    out = {}
    for d in widths:
        x, w = torch.zeros(9000, d, dtype=BF, device="cuda"), torch.zeros(d, dtype=BF, device="cuda")
        out[str(d)] = launches(lambda: L.layer_norm_forward(x, w))
    return out


def test_a_norms_grid_does_not_depend_on_earlier_widths():
    seen = []
    for order in (WIDTHS, WIDTHS[::-1]):
        p = subprocess.run([sys.executable, os.path.abspath(__file__), *map(str, order)], capture_output=True, text=True, timeout=300)
        assert p.returncode == 0, p.stdout + p.stderr
        seen.append(json.loads(p.stdout.splitlines()[-1]))
    assert seen[0] == seen[1]
    assert all(len(v) == 1 for v in seen[0].values())
    # and every CTA is resident: 64 warps and 32 CTAs an SM at most
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for (ctas, threads), in seen[0].values():
        assert ctas <= min(9000, sms * min(32, 2048 // threads))


if __name__ == "__main__":
    print(json.dumps(_grids([int(d) for d in sys.argv[1:]])))
