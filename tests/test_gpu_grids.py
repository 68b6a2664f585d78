"""The grids that the operators' calls launch, read from captured graphs: chosen by the call's own sizes
whatever calls came before."""
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
