"""The many-tensor calls without a GPU: structs, sizes, refusals before any launch, and the 8-bit form's reference."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from tests import _multi_ref as R
from zero_partitioned_mixed_replica_gb300 import binding as B
from zero_partitioned_mixed_replica_gb300 import build as zbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40          # never dereferenced: refused before any launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    zbuild.build()


def _status(fn, *a, **kw):
    with pytest.raises(B.ZeroError) as e:
        fn(*a, **kw)
    return e.value.status


def test_structs_match_the_header(tmp_path):
    structs = {"zero_multi_arrays": B.zero_multi_arrays, "zero_multi_info": B.zero_multi_info,
               "zero_step_state": B.zero_step_state}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "zero.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for f in cls._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f[0], name, f[0]))
    for c in ("ZERO_MAX_GROUPS", "ZERO_FP32", "ZERO_NO_OUT", "ZERO_MULTI_DECIDED", "ZERO_MULTI_ADVANCE", "ZERO_MULTI_UNSCALED"):
        lines.append('printf("%s %%d\\n", (int)%s);' % (c, c))
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f in cls._fields_:
            assert int(got["%s.%s" % (name, f[0])]) == getattr(cls, f[0]).offset, (name, f[0])
    for c in ("ZERO_MAX_GROUPS", "ZERO_FP32", "ZERO_NO_OUT", "ZERO_MULTI_DECIDED", "ZERO_MULTI_ADVANCE", "ZERO_MULTI_UNSCALED"):
        assert int(got[c]) == getattr(B, c), c


def test_query_counts():
    M = B.zero_multi_init([0, 1, 32, 33, 100_000], [0, 1, 1, 0, 0], 2, B.ZERO_FP32, B.ZERO_NO_OUT)
    i = B.zero_multi_query(M)
    assert (i.n_tensors, i.n_groups, i.grad_dtype, i.param_dtype) == (5, 2, B.ZERO_FP32, B.ZERO_NO_OUT)
    assert i.numel == 100_066
    assert i.state8_bytes == 2 * (100_066 + 0 + 1 + 1 + 2 + 3125)
    assert i.workspace_bytes % 256 == 0 and i.workspace_bytes > 0
    B.zero_multi_destroy(M)
    B.zero_multi_destroy(M)     # a second time does nothing


@pytest.mark.parametrize("kw", [
    dict(numels=[]), dict(numels=[-1]), dict(numels=[(1 << 34) + 1]), dict(n_groups=0), dict(n_groups=17),
    dict(group_of_tensor=[0, 2], n_groups=2), dict(group_of_tensor=[0, -1], n_groups=2), dict(group_of_tensor=[0]),
    dict(grad_dtype=3), dict(grad_dtype=-1), dict(param_dtype=2), dict(param_dtype=-2),
    dict(numels=[1 << 34] * 200)])
def test_init_refuses(kw):
    a = dict(numels=[5, 6], group_of_tensor=None, n_groups=1, grad_dtype=B.ZERO_BF16, param_dtype=B.ZERO_BF16)
    a.update(kw)
    assert _status(B.zero_multi_init, **a) == B.ZERO_ERR_INVALID


def test_bind_refuses_before_any_launch():
    M = B.zero_multi_init([100, 6], None, 1, B.ZERO_FP32, B.ZERO_BF16)
    two = [FAKE, FAKE]
    bind = lambda ws=FAKE, **kw: _status(B.zero_multi_bind, M, ws, 0, **kw)  # noqa: E731
    assert bind(ws=0, grads=two) == B.ZERO_ERR_INVALID
    assert bind(ws=FAKE + 16, grads=two) == B.ZERO_ERR_ALIGN
    assert bind(grads=[FAKE, 0]) == B.ZERO_ERR_INVALID
    assert bind(grads=[FAKE, FAKE + 2]) == B.ZERO_ERR_ALIGN          # fp32 gradients
    assert bind(master=[FAKE + 1, FAKE]) == B.ZERO_ERR_ALIGN
    assert bind(param16=[FAKE, FAKE + 1]) == B.ZERO_ERR_ALIGN
    assert bind(m=two) == B.ZERO_ERR_INVALID                         # without v
    assert bind(m8=two, v8=two, m8_scale=two) == B.ZERO_ERR_INVALID  # without v8_scale
    assert bind(grads=[FAKE]) == B.ZERO_ERR_INVALID                  # one pointer for two tensors
    with pytest.raises(TypeError):
        B.zero_multi_bind(M, FAKE, 0, gradients=two)
    assert B.lib().zero_multi_bind(None, None, None, None) == B.ZERO_ERR_INVALID
    assert B.lib().zero_multi_bind(M, None, FAKE, None) == B.ZERO_ERR_INVALID


def test_calls_on_an_unbound_list_are_refused():
    M = B.zero_multi_init([100], None, 1, B.ZERO_BF16, B.ZERO_BF16)
    hp = B.zero_adamw_hp(lr=1e-3, eps=1e-8, weight_decay=0.0)
    assert _status(B.zero_multi_grad_norm, M, 0.0, FAKE, 0) == B.ZERO_ERR_STATE
    assert _status(B.zero_multi_adamw, M, hp, 0, FAKE, 0) == B.ZERO_ERR_STATE
    assert _status(B.zero_multi_adamw8, M, hp, 0, 1, FAKE, 0) == B.ZERO_ERR_STATE
    assert _status(B.zero_multi_encode8, M, 0) == B.ZERO_ERR_STATE
    assert _status(B.zero_multi_decode8, M, 0) == B.ZERO_ERR_STATE
    assert _status(B.zero_multi_device_error, M) == B.ZERO_ERR_STATE
    assert _status(B.zero_multi_adamw, M, [hp, hp], 0, FAKE, 0) == B.ZERO_ERR_INVALID     # one group
    for fn, args in (("zero_multi_grad_norm", (None, 0.0, FAKE, None)), ("zero_multi_encode8", (None, None)),
                     ("zero_multi_adamw", (None, None, 0, FAKE, None)), ("zero_multi_query", (None, None))):
        assert getattr(B.lib(), fn)(*args) == B.ZERO_ERR_INVALID, fn


# -- the reference of the 8-bit form against other ways to say the same ----------------------------------------
@pytest.mark.parametrize("kind", [R.E4M3, R.E5M2], ids=["e4m3", "e5m2"])
def test_nearest_codes_equal_a_search_of_the_code_table(kind):
    rng = np.random.default_rng(3)
    x = rng.standard_normal(32 * 64) * np.exp2(rng.integers(-20, 20, 32 * 64))
    x[:32] = 0
    x[32:64] = 1.75 * 2.0 ** 5            # the largest code exactly
    x[64] = np.nextafter(np.float32(1.75 * 2.0 ** 30), np.float32(4e9))   # one above it: the next power of two
    x = np.abs(x) if kind["floor"] else x
    x = x.astype(np.float32)
    got = R.decode_ref(*R.encode_ref(torch.from_numpy(x), kind)).double().numpy()
    assert np.array_equal(got, R.nearest64(x.astype(np.float64), kind))
    again = R.decode_ref(*R.encode_ref(torch.from_numpy(got.astype(np.float32)), kind)).double().numpy()
    assert np.array_equal(again, got)     # stored values store as themselves


def test_stochastic_rounding_is_unbiased():
    # x between two codes: the mean over many steps is x.  4096 elements x 64 steps, each rounding off by at most one
    # code step (2^-3 of the power of two below x): 6 standard deviations of the mean are 6 * 0.5 * 2^-3 / 512
    n, steps = 4096, 64
    x = torch.full((n,), 1.3)
    x[::32] = 1.75                        # the block's scale
    tot = torch.zeros(n, dtype=torch.float64)
    for t in range(steps):
        rm, _ = R.random_ints(n, 7, t, 3)
        tot += R.decode_ref(*R.encode_ref(x, R.E4M3, rm)).double()
    keep = torch.arange(n) % 32 != 0
    assert abs(float(tot[keep].mean()) / steps - 1.3) < 6 * 0.5 * 0.125 / math.sqrt(n * steps * 31 / 32)
    assert float((tot[~keep] / steps - 1.75).abs().max()) == 0.0


def test_v_follows_small_steps_with_stochastic_rounding_only():
    # v under a constant gradient, beta2 = 0.999: after 3000 steps v is 1 - 0.999^3000 = 95% of g^2 in exact arithmetic;
    # nearest rounding stays where one step is less than half a code apart
    n, g2 = 1024, 1.0
    v = {True: torch.full((n,), 0.05), False: torch.full((n,), 0.05)}
    for t in range(3000):
        _, rv = R.random_ints(n, 1, t, 0)
        for s in v:
            new = 0.999 * v[s] + 0.001 * g2
            v[s] = R.decode_ref(*R.encode_ref(new, R.E5M2, rv if s else None))
    exact = 0.05 * 0.999 ** 3000 + (1 - 0.999 ** 3000)
    assert abs(float(v[True].mean()) / exact - 1) < 0.05
    assert float(v[False].mean()) < 0.5 * exact
