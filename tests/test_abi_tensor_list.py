"""The tensor-list entry points refuse bad arguments on the host, before any
launch.  No GPU: the pointers are never dereferenced."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
STEP = 1 << 16      # far enough apart for the tensors used here
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def sp():
    from spatiotemporal_neural_field_b200 import build
    build.build()
    from spatiotemporal_neural_field_b200 import spin4d
    return spin4d


def _grads(sp, *rows):
    return (sp.GradTensor * len(rows))(*[sp.GradTensor(*r) for r in rows])


def _norm(sp, rows, count=None, kind=2, scale=1.0, max_norm=1.0, control=FAKE, norms=None, ws=FAKE, nbytes=1 << 20):
    arr = _grads(sp, *rows) if rows else None
    return sp.lib.spin4d_grad_norm(arr, len(rows) if count is None else count, kind, scale, max_norm, control, norms, ws,
                                   nbytes, None)


GOOD = (FAKE, None, 100, 0, 0)


@pytest.mark.parametrize("kw", [
    dict(count=-1), dict(count=65537), dict(rows=[], count=1),
    dict(kind=3), dict(kind=-1),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF),
    dict(max_norm=-1.0), dict(max_norm=NAN),
    dict(control=None), dict(control=FAKE + 4), dict(norms=FAKE + 2),
    dict(ws=None), dict(ws=FAKE + 16), dict(nbytes=100),
    dict(rows=[(FAKE, None, -1, 0, 0)]), dict(rows=[(FAKE, None, (1 << 40) + 1, 0, 0)]),
    dict(rows=[(None, None, 1, 0, 0)]), dict(rows=[(FAKE + 2, None, 1, 0, 0)]), dict(rows=[(FAKE + 1, None, 1, 1, 0)]),
    dict(rows=[(FAKE, None, 1, 3, 0)]), dict(rows=[(FAKE, None, 1, -1, 0)]),
    dict(rows=[GOOD, (FAKE, None, -1, 0, 0)]),
    dict(rows=[(FAKE, None, 1 << 40, 0, 0)] * 5),     # more tiles than a launch can number
])
def test_grad_norm_refuses(sp, kw):
    assert _norm(sp, kw.pop("rows", [GOOD]), **kw) == sp.ERR_INVALID


def test_grad_norm_workspace_size(sp):
    assert sp.lib.spin4d_grad_norm_workspace(-1) == 0
    assert sp.lib.spin4d_grad_norm_workspace(65537) == 0
    need = sp.lib.spin4d_grad_norm_workspace(1)
    assert need > 0
    assert _norm(sp, [GOOD], nbytes=need - 1) == sp.ERR_INVALID


def _clip(sp, rows, control=FAKE):
    return sp.lib.spin4d_clip_grads(_grads(sp, *rows), len(rows), control, None)


@pytest.mark.parametrize("rows", [
    [(FAKE, None, -1, 0, 0)], [(None, None, 1, 0, 0)], [(FAKE + 2, None, 1, 0, 0)], [(FAKE, None, 1, 7, 0)],
    [(FAKE, FAKE + STEP, 1, 0, 5)], [(FAKE, FAKE + STEP + 2, 1, 0, 0)],
    [GOOD, GOOD],                                              # the same tensor twice, in place
    [GOOD, (FAKE + 396, None, 100, 0, 0)],                     # one value shared
    [(FAKE, FAKE + 4, 100, 0, 0)],                             # an output a value behind its gradient
    [(FAKE, FAKE, 100, 0, 1)],                                 # its own gradient's place in another type
    [(FAKE, FAKE + STEP, 100, 0, 0), (FAKE + 4 * STEP, FAKE + STEP + 200, 100, 0, 2)],
    [(FAKE, FAKE + STEP, 100, 0, 0), (FAKE + STEP, None, 100, 0, 0)],
])
def test_clip_refuses(sp, rows):
    assert _clip(sp, rows) == sp.ERR_INVALID


def test_clip_refuses_control_and_long_overlapping_lists(sp):
    assert _clip(sp, [GOOD], control=None) == sp.ERR_INVALID
    assert _clip(sp, [GOOD], control=FAKE + 8) == sp.ERR_INVALID
    many = [(FAKE + STEP * ((7 * i) % 1000), None, 100, 0, 0) for i in range(1000)]
    assert _clip(sp, many + [(FAKE + 500 * STEP + 4, None, 1, 0, 0)]) == sp.ERR_INVALID


def _adam(sp, rows, step=1, b1=0.9, b2=0.99, eps=1e-15, zero=0, control=None, flag=None, count=None):
    arr = (sp.AdamTensor * max(len(rows), 1))(*[sp.AdamTensor(*r) for r in rows])
    return sp.lib.spin4d_adam_step_tensors(arr if rows else None, len(rows) if count is None else count, step, b1, b2, eps,
                                           zero, control, flag, None)


def _row(p=FAKE, w=None, g=FAKE + STEP, m=FAKE + 2 * STEP, v=FAKE + 3 * STEP, n=100, lr=1e-3, wd=0.0, gd=0, wt=0):
    return (p, w, g, m, v, n, lr, wd, gd, wt)


@pytest.mark.parametrize("kw", [
    dict(step=-1), dict(step=0), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=NAN), dict(eps=-1e-9),
    dict(eps=NAN), dict(eps=1e39), dict(b1=1 - 1e-12),          # 1 in fp32
    dict(control=FAKE + 4), dict(flag=FAKE + 1), dict(count=-1), dict(count=65537), dict(rows=[], count=1),
    dict(rows=[_row(n=-1)]), dict(rows=[_row(n=(1 << 40) + 1)]), dict(rows=[_row(lr=NAN)]), dict(rows=[_row(lr=INF)]),
    dict(rows=[_row(wd=NAN)]), dict(rows=[_row(p=None)]), dict(rows=[_row(g=None)]), dict(rows=[_row(m=FAKE + 2)]),
    dict(rows=[_row(v=FAKE + 2)]), dict(rows=[_row(gd=3)]), dict(rows=[_row(g=FAKE + STEP + 1, gd=1)]),
    dict(rows=[_row(w=FAKE + 4 * STEP, wt=0)]),                  # a working copy in fp32
    dict(rows=[_row(w=FAKE + 4 * STEP + 1, wt=1)]),
    dict(rows=[_row(m=FAKE)]), dict(rows=[_row(v=FAKE + 2 * STEP + 396)]), dict(rows=[_row(g=FAKE + 8)]),
    dict(rows=[_row(w=FAKE + 2 * STEP, wt=1)]),
    dict(rows=[_row(), _row(p=FAKE + 5 * STEP, m=FAKE + 6 * STEP, v=FAKE + 7 * STEP)], zero=1),   # a shared gradient, cleared
])
def test_adam_refuses(sp, kw):
    assert _adam(sp, kw.pop("rows", [_row()]), **kw) == sp.ERR_INVALID


def test_empty_lists_and_tensors_launch_nothing(sp):
    assert _clip(sp, [(None, None, 0, 0, 0)] * 3) == sp.OK
    assert sp.lib.spin4d_clip_grads(None, 0, FAKE, None) == sp.OK
    assert _adam(sp, []) == sp.OK
    assert _adam(sp, [_row(p=None, g=None, m=None, v=None, n=0)]) == sp.OK


@pytest.mark.parametrize("name,call", [
    ("spin4d_grad_norm", "spin4d_grad_norm(r(g), 1, %s, 1.0, 1.0, F, None, F, 1 << 20, None)"),
    ("spin4d_clip_grads", "spin4d_clip_grads(r(g), %s, F, None)"),
    ("spin4d_adam_step_tensors", "spin4d_adam_step_tensors(r(a), 1, %s, 0.9, 0.99, 1e-8, 0, None, None, None)"),
])
def test_injected_faults_come_after_validation(sp, name, call):
    good = {"spin4d_grad_norm": "2"}.get(name, "1")
    code = r"""
import ctypes, sys
sys.path.insert(0, %r)
from spatiotemporal_neural_field_b200 import spin4d as sp
F, S, r = 1 << 20, 1 << 16, ctypes.byref
g = sp.GradTensor(F, None, 100, 0, 0)
a = sp.AdamTensor(F, None, F + S, F + 2 * S, F + 3 * S, 100, 1e-3, 0.0, 0, 0)
print(sp.lib.%s, sp.lib.%s)
""" % (ROOT, call % good, call % "-1")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         env=dict(os.environ, SPIN4D_FAULT=name), timeout=300)
    assert out.returncode == 0, out.stderr
    assert list(map(int, out.stdout.split())) == [sp.ERR_INJECTED, sp.ERR_INVALID]


def test_binding_refuses(sp):
    cpu = torch.zeros(8)
    with pytest.raises(ValueError):
        sp.grad_list([cpu])                                    # not on a GPU
    with pytest.raises(ValueError):
        sp.grad_list([torch.zeros(4, 4).t()[1:]])              # not contiguous
    with pytest.raises(ValueError):
        sp.grad_list([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError):
        sp.grad_list([cpu], [])
    with pytest.raises(ValueError):
        sp.grad_list([cpu], [torch.zeros(7)])
    with pytest.raises(ValueError):
        sp.grad_list([None])
    with pytest.raises(ValueError):
        sp.adam_list([cpu], [None], [cpu], [cpu], lr=1e-3)
    with pytest.raises(ValueError):
        sp.adam_list([cpu], [cpu], [cpu], [], lr=1e-3)
    with pytest.raises(ValueError):
        sp.adam_list([cpu], [torch.zeros(7)], [cpu], [cpu], lr=1e-3)
    with pytest.raises(ValueError):
        sp.adam_list([cpu], [cpu], [cpu], [cpu], lr=[1e-3, 1e-3])
    with pytest.raises(ValueError):
        sp.adam_list([cpu.half()], [cpu], [cpu], [cpu], lr=1e-3)          # fp32 masters only
    with pytest.raises(ValueError):
        sp.adam_list([cpu], [cpu], [cpu], [cpu], lr=1e-3, params_work=[cpu])
    with pytest.raises(ValueError):
        sp.grad_control("cpu")
    assert len(sp.grad_list([])) == 0 and len(sp.adam_list([], [], [], [], lr=1e-3)) == 0
    assert ctypes.sizeof(sp.GradTensor) == 32 and ctypes.sizeof(sp.AdamTensor) == 64
