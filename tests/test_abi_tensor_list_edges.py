"""Arguments at the edge of what the tensor-list calls' arithmetic holds: the
ones beyond it are refused on the host, before any launch.  No GPU: the
pointers are never dereferenced."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
STEP = 1 << 16      # far enough apart for the tensors used here


@pytest.fixture(scope="module")
def sp():
    from spatiotemporal_neural_field_b200 import build
    build.build()
    from spatiotemporal_neural_field_b200 import spin4d
    return spin4d


def statuses(entry, calls):
    """What the calls return when ``entry`` fails by injection behind its checks, in a process of their own:
    ERR_INJECTED is an argument that was taken, and nothing is launched."""
    code = """
import json, sys
sys.path.insert(0, %r)
from spatiotemporal_neural_field_b200 import spin4d as sp
F, S = %d, %d
print(json.dumps([eval(c) for c in json.loads(sys.argv[1])]))
""" % (ROOT, FAKE, STEP)
    out = subprocess.run([sys.executable, "-c", code, json.dumps(calls)], capture_output=True, text=True,
                         env=dict(os.environ, SPIN4D_FAULT=entry), timeout=300)
    assert out.returncode == 0, out.stderr
    return json.loads(out.stdout)


FMAX = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("scale", [
    1e39, 1.7e308,                  # infinite in fp32: the coefficient of a zero norm would be too, and inf * 0 is NaN
    FMAX + 2.0 ** 103,              # half a step above the largest: the tie goes to infinity
    1e-46, 5e-324,                  # 0 in fp32, which is the coefficient that drops a gradient
    2.0 ** -150,                    # rounds to 0 (ties to even)
])
def test_grad_norm_refuses_scales_that_fp32_does_not_hold(sp, scale):
    g = (sp.GradTensor * 1)(sp.GradTensor(FAKE, None, 100, 0, 0))
    assert sp.lib.spin4d_grad_norm(g, 1, 2, scale, 1.0, FAKE, None, FAKE, 1 << 20, None) == sp.ERR_INVALID
    assert sp.lib.spin4d_grad_norm(None, 0, 2, scale, 1.0, FAKE, None, FAKE, 1 << 20, None) == sp.ERR_INVALID


def test_grad_norm_takes_scales_that_round_into_fp32(sp):
    scales = [FMAX, FMAX * (1 + 2.0 ** -25),      # less than half a step (2^103) above the largest
              2.0 ** -149, 1.001 * 2.0 ** -150, 1.0]
    call = "sp.lib.spin4d_grad_norm((sp.GradTensor * 1)(sp.GradTensor(F, None, 9, 0, 0)), 1, 2, %r, 1.0, F, None, F, 1 << 20, None)"
    assert statuses("spin4d_grad_norm", [call % x for x in scales]) == [sp.ERR_INJECTED] * len(scales)


ADAM = ("sp.lib.spin4d_adam_step_tensors((sp.AdamTensor * 1)(sp.AdamTensor(F, None, F + S, F + 2 * S, F + 3 * S, 9, 1e-3,"
        " 0.0, 0, 0)), 1, 1, 0.9, 0.99, %r, 0, None, None, None)")


def test_adam_refuses_eps_outside_the_range_of_its_quotient(sp):
    """The quotient is within 2 ulp for denominators from 2^-126 to 2^126 (and 0, where it is infinite or NaN as it should
    be); the root reaches 2^64."""
    taken = [0.0, 2.0 ** -126, 1e-30, 1e-15, 1e-8, 1.0, 2.0 ** 125]
    refused = [2.0 ** -149, 1e-40, 2.0 ** -127, 2.0 ** 125 * (1 + 2.0 ** -23), 2.0 ** 126, 1e38, FMAX]
    assert statuses("spin4d_adam_step_tensors", [ADAM % x for x in taken]) == [sp.ERR_INJECTED] * len(taken)
    assert statuses("spin4d_adam_step_tensors", [ADAM % x for x in refused]) == [sp.ERR_INVALID] * len(refused)
    assert statuses("spin4d_adam_step_tensors", [ADAM % 1e-46]) == [sp.ERR_INJECTED]      # 0 in fp32


def test_pointers_of_a_tensor_without_values_are_not_looked_at(sp):
    """Odd and overlapping addresses of n = 0, with the types that go with them."""
    odd = FAKE + 1
    for w, wt in ((odd, 1), (FAKE, 0), (odd, 9)):
        row = sp.AdamTensor(odd, w, odd, odd, odd, 0, 1e-3, 0.0, 0, wt)
        assert sp.lib.spin4d_adam_step_tensors((sp.AdamTensor * 2)(row, row), 2, 1, 0.9, 0.99, 1e-8, 1, None, None,
                                               None) == sp.OK
    row = sp.GradTensor(odd, odd, 0, 0, 9)
    assert sp.lib.spin4d_clip_grads((sp.GradTensor * 2)(row, row), 2, FAKE, None) == sp.OK


def test_adam_refuses_a_flag_without_a_value(sp, monkeypatch):
    """An empty tensor's address is 0, which the library takes as no flag."""
    lst = object.__new__(sp.AdamList)
    lst.index, lst.count, lst.address = -1, 0, 0           # as CPU tensors number their device
    monkeypatch.setattr(sp, "_list_call", lambda *args: None)
    sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, step=1, nonfinite_flag=torch.zeros(1, dtype=torch.int32))
    for flag in (torch.zeros(0, dtype=torch.int32), torch.zeros(1)):
        with pytest.raises(ValueError):
            sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, step=1, nonfinite_flag=flag)
