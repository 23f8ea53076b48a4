"""The tensor-list kernels in the build with device checks: what is checked
(read from the source), and lists of every capacity through them on a B200,
which leave no bounds error behind.  No test drives an index out of range: the
host admits no such list."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "spatiotemporal_neural_field_b200", "csrc", "tensor_list.cu")


def test_vectors_slots_and_owners_are_behind_checks():
    lines = open(SOURCE).read().split("\n")
    assert any("bounds_ok(" in x for x in lines)
    calls = [i for i, x in enumerate(lines)
             if re.search(r"\b(load_raw<(H|kKeep|kStream)>|store_raw)\(static_cast|load_raw<kKeep>\(", x)]
    assert len(calls) == 5                                 # two loads, two stores, the norm's own loop
    for i in calls:
        assert "expect(" in lines[i - 1], lines[i]
    stores = [x for x in lines if re.search(r"f\.slots\[[^\]]*\]\]* = ", x)]
    assert len(stores) == 1 and "expect(" in stores[0]
    walks = [x for x in lines if re.search(r"for \(int k = .*(owner|last).*;", x)]
    assert len(walks) == 3 and all("expect(" in x for x in walks)
    assert "expect(" in "".join(lines[i + 2] for i, x in enumerate(lines) if "int owner(uint32_t tile)" in x)


CHILD = r"""
import sys
sys.path.insert(0, %r)
import torch
from spatiotemporal_neural_field_b200 import spin4d as sp
sp.check_device_errors(clear=True)
gen = torch.Generator(device="cuda").manual_seed(1)
types = (torch.float32, torch.float16, torch.bfloat16)
total = 0
for count, big in ((0, 0), (1, 1), (16, 5000), (17, 40_000_001), (64, 9), (65, 31_000_003), (224, 0), (225, 12_000_001),
                   (320, 4097), (321, 30_000_001), (448, 0), (449, 8), (1025, 25_000_001)):
    lens = [(k * 977) %% 4111 for k in range(count)]
    if count:
        lens[count // 2] = big
    def views(dtype, gap, seed):
        flat = torch.randn(sum(lens) + gap * (count + 1), device="cuda", generator=gen).to(dtype)
        out, at = [], gap
        for n in lens:
            out.append(flat[at:at + n])
            at += n + gap
        return out, flat
    dtype = types[count %% 3]
    (g, gf), (p, pf), (m, mf), (v, vf), (w, wf) = (views(dtype, 2, 0), views(torch.float32, 1, 1), views(torch.float32, 1, 2),
                                                   views(torch.float32, 1 if count %% 2 else 3, 3), views(torch.float16, 1, 4))
    vf.square_()
    for kind in ("l1", "inf", "l2"):
        ctl, norms = sp.grad_control(), torch.zeros(count, device="cuda")
        sp.grad_norm(g, ctl, max_norm=1.0, norm_type=kind)
        sp.grad_norm(g, ctl, max_norm=1.0, norm_type=kind, norms=norms)
    sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=1e-2, params_work=w), 0.9, 0.99, 1e-8, control=ctl)
    sp.clip_grads(sp.grad_list(g, m), ctl)
    sp.clip_grads(g, ctl)
    sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=1e-2), 0.9, 0.99, 1e-8, step=1, zero_grad=True)
    torch.cuda.synchronize()
    sp.check_device_errors(clear=False)
    for f in (gf, pf, mf, vf, wf):
        x = f.view(torch.int32 if f.element_size() == 4 else torch.int16).long()
        total += int((x * torch.arange(1, x.numel() + 1, device="cuda")).sum())
    total += int((torch.cat([ctl.buf, norms.view(torch.int32)]).long()).sum())
print("BITS", sp.lib.spin4d_checked_build(), total %% (1 << 61))
""" % ROOT


@pytest.mark.gpu
def test_lists_of_every_capacity_run_clean_and_with_the_same_bits():
    seen = {}
    for flag in ("1", "0"):
        r = subprocess.run([sys.executable, "-c", CHILD], env=dict(os.environ, SPIN4D_CHECKED=flag), cwd=ROOT,
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
        _, checked, bits = r.stdout.split()
        assert checked == flag
        seen[flag] = bits
    assert seen["0"] == seen["1"]
