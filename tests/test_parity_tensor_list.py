"""GPU parity of the tensor-list calls (global gradient norm, clipping, Adam
with decoupled weight decay) with the fp64 oracle, through the binding."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import decoder as dec
from oracle import tensor_list as tl
from spatiotemporal_neural_field_b200 import synthetic as S
from tests import tensor_list_tol as tt
from tests import tol

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# lengths around a thread's 8 values, a warp's 256 and a tile's 2048
EDGES = [0, 1, 2, 7, 8, 9, 0, 31, 255, 256, 257, 2039, 2040, 2041, 2047, 2048, 2049, 4096, 6987, 100003]


@pytest.fixture(scope="module")
def sp():
    from spatiotemporal_neural_field_b200 import spin4d
    return spin4d


def host(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def packed(lens, dtype, seed, scale=1e-2, gap=1):
    """Views of one buffer with ``gap`` values between them (so that they start at every
    alignment of their type), the buffer, and a copy of it."""
    total = sum(lens) + gap * (len(lens) + 1)
    flat = (torch.randn(total, device="cuda", generator=gen(seed)) * scale).to(TYPES[dtype])
    views, at = [], gap
    for n in lens:
        views.append(flat[at:at + n])
        at += n + gap
    return views, flat, flat.clone()


def gaps_unchanged(flat, before, lens, gap=1):
    at = 0
    for n in list(lens) + [0]:
        assert torch.equal(flat[at:at + gap], before[at:at + gap])
        at += gap + n


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm_of_ragged_lists(sp, dtype, kind):
    for lens, gap in ((EDGES, 1), (EDGES[::-1], 3), ([1], 1), ([0], 1), ([0, 0, 5], 2), ([2048 * 7], 8)):
        views, flat, before = packed(lens, dtype, 1, gap=gap)
        ctl = sp.grad_control()
        norms = torch.full((len(lens),), -1.0, device="cuda")
        scale = float(np.float32(0.3))
        sp.grad_norm(views, ctl, max_norm=0.5, norm_type=kind, grad_scale=scale, norms=norms)
        want, coef, each = tl.grad_norm([host(v) for v in views], max_norm=0.5, kind=kind, scale=scale)
        tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
        tt.within(host(ctl.coef), coef, tt.scalar_bound(coef), "coef")
        tt.within(host(norms), each, tt.scalar_bound(np.array(each)), "norms")
        assert int(ctl.step) == 1 and int(ctl.skipped) == 0
        assert torch.equal(flat, before)


@pytest.mark.parametrize("count", [0, 1, 16, 17, 200, 1024, 1025, 2500])
def test_norm_of_many_tensors(sp, count):
    """Lists on both sides of each launch's capacity; every tensor's norm is its own."""
    lens = [int(x) for x in np.random.default_rng(count).integers(0, 400, count)]
    views, _, _ = packed(lens, "f32", 2)
    ctl, norms = sp.grad_control(), torch.full((count,), -1.0, device="cuda")
    sp.grad_norm(views, ctl, max_norm=1e-3, norms=norms)
    want, coef, each = tl.grad_norm([host(v) for v in views], max_norm=1e-3)
    tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
    tt.within(host(ctl.coef), coef, tt.scalar_bound(coef), "coef")
    tt.within(host(norms), each, tt.scalar_bound(np.array(each)), "norms")


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("big_at", [0, 60, 120])
def test_norms_of_long_and_short_tensors_of_every_type(sp, big_at, kind):
    """A tensor of many blocks among 120 of a few values, types mixed: the parts of each are kept apart."""
    lens = [int(x) for x in np.random.default_rng(4).integers(0, 5000, 120)]
    lens[3] = lens[70] = 0
    lens.insert(big_at, 3_000_001)
    views = []
    for k, n in enumerate(lens):
        t = list(TYPES)[k % 3]
        views.append(packed([n], t, 200 + k, scale=10.0 ** -(k % 5), gap=1 + k % 4)[0][0])
    ctl, norms = sp.grad_control(), torch.full((len(lens),), -1.0, device="cuda")
    want, coef, each = tl.grad_norm([host(v) for v in views], max_norm=0.5, kind=kind)
    for given in (norms, None):
        sp.grad_norm(views, ctl, max_norm=0.5, norm_type=kind, norms=given)
        tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
        tt.within(host(ctl.coef), coef, tt.scalar_bound(coef), "coef")
    tt.within(host(norms), each, tt.scalar_bound(np.array(each)), "norms")
    old = [host(v) for v in views]
    sp.clip_grads(views, ctl)
    for k, (v, o) in enumerate(zip(views, old)):
        w = tl.clip(o, float(ctl.coef))
        tt.within(host(v), w, tt.clip_bound(w, list(TYPES)[k % 3]), "clip of %d" % lens[k])


@pytest.mark.parametrize("n", [16_777_216 + 6987, 134_217_728 + 3])
def test_norm_of_long_tensors_is_deterministic(sp, n):
    g = torch.randn(n, device="cuda", generator=gen(3))
    want = float(g.double().square().sum().sqrt())
    got = []
    for _ in range(3):
        ctl = sp.grad_control()
        sp.grad_norm([g[:n // 3], g[n // 3:]], ctl, max_norm=1.0)
        got.append(ctl.buf.clone())
    assert all(torch.equal(got[0], x) for x in got)
    tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")


def test_norm_over_the_whole_range_of_fp32(sp):
    """Squares of neither the largest nor the smallest values leave the 64-bit sum's range."""
    for value in (3e38, 1e25, 1e-25, 2.0 ** -149):
        for n in (1, 1000):
            g = torch.full((n,), value, device="cuda")
            v = float(g[0])
            for scale in (1.0, float(np.float32(1e-4))):
                ctl = sp.grad_control()
                sp.grad_norm([g], ctl, max_norm=1.0, grad_scale=scale)
                want, coef, _ = tl.grad_norm([np.full(n, v)], max_norm=1.0, scale=scale)
                if want > float(np.finfo(np.float32).max):         # not a number of fp32: treated as infinite
                    assert torch.isinf(ctl.norm) and float(ctl.coef) == 0 and int(ctl.skipped) == 1
                    continue
                tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm of %g" % value)
                tt.within(host(ctl.coef), coef, tt.scalar_bound(coef), "coef of %g" % value)


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_non_finite_gradients_are_found_and_dropped(sp, dtype, kind):
    lens = [5000, 0, 3, 2049]
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t, i in ((0, 0), (0, 4999), (2, 1), (3, 2048)):
            views, flat, before = packed(lens, dtype, 4)
            views[t][i] = bad
            ctl, norms = sp.grad_control(step=7), torch.zeros(4, device="cuda")
            sp.grad_norm(views, ctl, max_norm=1.0, norm_type=kind, norms=norms)
            assert not np.isfinite(float(ctl.norm)) and float(ctl.coef) == 0.0
            assert np.isnan(float(ctl.norm)) == np.isnan(bad)
            assert int(ctl.step) == 7 and int(ctl.skipped) == 1
            fine = torch.isfinite(norms).tolist()
            assert fine == [k != t for k in range(4)]
            sp.clip_grads(views, ctl)
            assert all(not v.any() for v in views)           # zeros, NaN and infinity included
            gaps_unchanged(flat, before, lens)
            # and the next good gradient is taken
            views[0].fill_(0.25)
            sp.grad_norm(views, ctl, max_norm=1.0, norm_type=kind)
            assert int(ctl.step) == 8 and int(ctl.skipped) == 1


@pytest.mark.parametrize("out", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_clip_matches_oracle(sp, dtype, out):
    for gap, out_gap in ((1, 1), (8, 8), (3, 2)):            # alike, aligned, and at different offsets
        views, flat, before = packed(EDGES, dtype, 5, gap=gap)
        outs, oflat, obefore = packed(EDGES, out or "f32", 6, gap=out_gap)
        lst = sp.grad_list(views, outs if out else None)
        ctl = sp.grad_control()
        sp.grad_norm(lst, ctl, max_norm=0.05, grad_scale=2.0)
        sp.clip_grads(lst, ctl)
        coef, at = float(ctl.coef), gap
        assert 0 < coef < 2
        for k, n in enumerate(EDGES):
            want = tl.clip(host(before[at:at + n]), coef)
            tt.within(host(outs[k] if out else views[k]), want, tt.clip_bound(want, out or dtype), "clip %d" % n)
            at += n + gap
        if out:
            assert torch.equal(flat, before)
            gaps_unchanged(oflat, obefore, EDGES, out_gap)
        else:
            gaps_unchanged(flat, before, EDGES, gap)


def test_clip_of_many_tensors_and_infinite_or_zero_max_norm(sp):
    lens = [int(x) for x in np.random.default_rng(9).integers(0, 300, 1030)]
    views, flat, before = packed(lens, "f32", 7)
    ctl = sp.grad_control()
    sp.grad_norm(views, ctl)
    sp.clip_grads(views, ctl)
    assert float(ctl.coef) == 1.0 and torch.equal(flat, before)
    sp.grad_norm(views, ctl, max_norm=0.0)
    assert float(ctl.coef) == 0.0 and int(ctl.step) == 2
    sp.clip_grads(views, ctl)
    assert all(not v.any() for v in views)
    gaps_unchanged(flat, before, lens)


def _adam_state(lens, dtype, seed, gap=1, work=None):
    p, pf, p0 = packed(lens, "f32", seed, 1.0, gap)
    g, gf, g0 = packed(lens, dtype, seed + 1, 1e-2, gap)
    m, mf, m0 = packed(lens, "f32", seed + 2, 1e-2, gap)
    v, vf, _ = packed(lens, "f32", seed + 3, 1.0, gap)
    vf.copy_(mf * mf * (1 + vf.abs()) + 1e-10)
    v0 = vf.clone()
    w = packed(lens, work, seed + 4, 1.0, gap) if work else (None, None, None)
    return (p, g, m, v, w[0]), (pf, gf, mf, vf, w[1]), (p0, g0, m0, v0, w[2])


def _check_adam(lens, state, before, gap, step, lr, betas, eps, decay, coef, work, what):
    at = gap
    for k, n in enumerate(lens):
        old = [host(b[at:at + n]) for b in before[:4]]
        old = [old[0], old[1], old[2], old[3]]
        h = dict(step=step, lr=lr[k], b1=betas[0], b2=betas[1], eps=eps, decay=decay[k], coef=coef)
        want = tl.adamw_step(*old, **h)
        bounds = tt.adam_bounds(*old, **h)
        for name, got, w, b in zip("pmv", (state[0][k], state[2][k], state[3][k]), want, bounds):
            tt.within(host(got), w, b, "%s %s of %d" % (what, name, n))
        if work:
            assert torch.equal(state[4][k], state[0][k].to(TYPES[work]))
        at += n + gap


@pytest.mark.parametrize("dtype,work", [("f32", "f16"), ("f32", None), ("f16", "bf16"), ("bf16", None)])
@pytest.mark.parametrize("gap", [1, 8])
def test_adam_step_matches_oracle(sp, dtype, work, gap):
    lens = EDGES
    state, flats, before = _adam_state(lens, dtype, 20, gap, work)
    lr = [1e-3 * (k + 1) for k in range(len(lens))]
    decay = [0.0 if k % 2 else 0.05 for k in range(len(lens))]
    ctl = sp.grad_control(step=4)
    sp.grad_norm(state[1], ctl, max_norm=0.5)
    lst = sp.adam_list(*state[:4], lr=lr, weight_decay=decay, params_work=state[4])
    sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, control=ctl)
    coef = float(ctl.coef)
    assert coef < 1.0 and int(ctl.step) == 5
    _check_adam(lens, state, before, gap, 5, lr, (0.9, 0.99), 1e-8, decay, coef, work, "adam")
    assert torch.equal(flats[1], before[1])
    for k in (0, 2, 3) + ((4,) if work else ()):
        gaps_unchanged(flats[k], before[k], lens, gap)


def test_adam_step_with_arrays_at_different_offsets(sp):
    lens = [2500, 9, 4096]
    p, pf, p0 = packed(lens, "f32", 30, 1.0, gap=1)
    g, gf, g0 = packed(lens, "f16", 31, 1e-2, gap=2)
    m, mf, m0 = packed(lens, "f32", 32, 1e-2, gap=5)
    v, vf, v0 = packed(lens, "f32", 33, 1.0, gap=7)
    vf.square_()
    v0 = vf.clone()
    w, wf, w0 = packed(lens, "f16", 34, gap=3)
    old = [[host(x) for x in a] for a in (p, g, m, v)]
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=1e-2, params_work=w), 0.9, 0.99, 1e-8, step=2, zero_grad=True,
                         nonfinite_flag=flag)
    for k in range(3):
        args = [a[k] for a in old]
        h = dict(step=2, lr=1e-2, b1=0.9, b2=0.99, eps=1e-8)
        for name, got, want, b in zip("pmv", (p[k], m[k], v[k]), tl.adamw_step(*args, **h), tt.adam_bounds(*args, **h)):
            tt.within(host(got), want, b, name)
        assert torch.equal(w[k], p[k].half()) and not g[k].any()
    for f, b, gap in ((pf, p0, 1), (gf, g0, 2), (mf, m0, 5), (vf, v0, 7), (wf, w0, 3)):
        gaps_unchanged(f, b, lens, gap)
    assert int(flag) == 0


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_adam_step_with_gradients_from_a_packed_bucket(sp, dtype, zero):
    """Parameters and state of their own, gradients at every offset of one buffer: read, and cleared, in place."""
    lens = EDGES
    own = [_adam_state([n], "f32", 500 + 10 * k, gap=8, work="f16") for k, n in enumerate(lens)]
    p, m, v, w = ([x[0][j][0] for x in own] for j in (0, 2, 3, 4))
    for gap in (1, 2, 3):
        g, gf, g0 = packed(lens, dtype, 700 + gap, gap=gap)
        old = [[host(x) for x in a] for a in (p, g, m, v)]
        sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=1e-2, params_work=w), 0.9, 0.99, 1e-8, step=2, zero_grad=zero)
        for k, n in enumerate(lens):
            args = [a[k] for a in old]
            h = dict(step=2, lr=1e-2, b1=0.9, b2=0.99, eps=1e-8)
            for name, got, want, b in zip("pmv", (p[k], m[k], v[k]), tl.adamw_step(*args, **h), tt.adam_bounds(*args, **h)):
                tt.within(host(got), want, b, "%s of %d" % (name, n))
            assert torch.equal(w[k], p[k].half())
        gaps_unchanged(gf, g0, lens, gap)
        assert all(not x.any() for x in g) if zero else torch.equal(gf, g0)


@pytest.mark.parametrize("count", [1, 17, 512, 513, 1300])
def test_adam_step_of_many_tensors(sp, count):
    lens = [int(x) for x in np.random.default_rng(count).integers(0, 300, count)]
    state, flats, before = _adam_state(lens, "f32", 40)
    lr, decay = [1e-3 + 1e-5 * k for k in range(count)], [0.01] * count
    sp.adam_step_tensors(sp.adam_list(*state[:4], lr=lr, weight_decay=decay), 0.9, 0.99, 1e-8, step=3)
    at = 1
    want, bound, got = [], [], []
    for k, n in enumerate(lens):
        old = [host(b[at:at + n]) for b in before[:4]]
        h = dict(step=3, lr=lr[k], b1=0.9, b2=0.99, eps=1e-8, decay=0.01)
        want.append(np.concatenate(tl.adamw_step(*old, **h)))
        bound.append(np.concatenate(tt.adam_bounds(*old, **h)))
        got.append(np.concatenate([host(state[j][k]) for j in (0, 2, 3)]))
        at += n + 1
    tt.within(np.concatenate(got), np.concatenate(want), np.concatenate(bound), "%d tensors" % count)


def test_adam_step_agrees_with_the_single_tensor_call(sp):
    """Without decay and control it is spin4d_adam_step: both inside the bound around the oracle, which
    counts the single call's 1 - b, taken from b in fp32, by 2^-24 / (1 - b)."""
    n, b1, b2, eps = 70_001, 0.5, 0.75, 1e-15                # betas that fp32 holds
    (p, g, m, v, w), _, _ = _adam_state([n], "f32", 50, gap=8, work="f16")
    one = [x[0].clone() for x in (p, g, m, v)]
    w1 = torch.zeros(n, dtype=torch.float16, device="cuda")
    for step in (1, 2, 3):
        old = [host(x) for x in one]
        h = dict(step=step, lr=1e-3, b1=b1, b2=b2, eps=eps)
        bounds = tt.adam_bounds(*old, **h)
        sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=1e-3, params_work=w), b1, b2, eps, step=step)
        sp.adam_step(one[0], one[1], one[2], one[3], step, 1e-3, b1, b2, eps, params_work=w1)
        for name, a, b, bound in zip("pmv", (p[0], m[0], v[0]), (one[0], one[2], one[3]), bounds):
            tt.within(host(a), host(b), 2 * bound, "step %d %s" % (step, name))
        for a, b in zip((p, m, v), (one[0], one[2], one[3])):
            a[0].copy_(b)


def test_adam_skips_and_clears_after_a_non_finite_norm(sp):
    lens = [3000, 5]
    state, flats, before = _adam_state(lens, "f32", 60, work="f16")
    state[1][1][2] = float("nan")
    ctl = sp.grad_control(step=9)
    lst = sp.adam_list(*state[:4], lr=1e-3, weight_decay=0.1, params_work=state[4])
    sp.grad_norm(state[1], ctl, max_norm=1.0)
    for zero in (False, True):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, control=ctl, zero_grad=zero, nonfinite_flag=flag)
        for k in (0, 2, 3, 4):
            assert torch.equal(flats[k], before[k])
        assert int(flag) == 0 and int(ctl.step) == 9
    assert all(not x.any() for x in state[1])
    # a control block that grad_norm has not been run on takes no step either
    fresh = sp.grad_control()
    sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, control=fresh)
    assert all(torch.equal(flats[k], before[k]) for k in (0, 2, 3, 4))


def test_adam_flags_updates_that_are_not_finite(sp):
    g = torch.ones(3000, device="cuda")
    g[2999] = float("inf")
    p, m, v = torch.zeros_like(g), torch.zeros_like(g), torch.zeros_like(g)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    sp.adam_step_tensors(sp.adam_list([p], [g], [m], [v], lr=1e-3), 0.9, 0.99, 1e-8, step=1, nonfinite_flag=flag)
    assert int(flag) == 1 and bool(torch.isfinite(p[:2999]).all())


def test_entries_without_gradient_stay(sp):
    """g = m = v = 0 moves nothing, with the smallest eps; eps = 0 in the tail's padding flags nothing."""
    p = torch.randn(2049, device="cuda", generator=gen(8))
    z = [torch.zeros_like(p) for _ in range(3)]
    q = p.clone()
    sp.adam_step_tensors(sp.adam_list([p], [z[0]], [z[1]], [z[2]], lr=1e-2), 0.9, 0.99, 1e-15, step=1)
    assert torch.equal(p, q)
    g = torch.full_like(p, 0.5)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    sp.adam_step_tensors(sp.adam_list([p], [g], [z[1]], [z[2]], lr=2.0 ** -6), 0.0, 0.0, 0.0, step=1, nonfinite_flag=flag)
    assert int(flag) == 0
    args = (host(q), host(g), np.zeros(2049), np.zeros(2049))
    h = dict(step=1, lr=2.0 ** -6, b1=0.0, b2=0.0, eps=0.0)
    tt.within(host(p), host(q) - 2.0 ** -6, tt.adam_bounds(*args, **h)[0], "g / sqrt(g^2) = 1")


@pytest.mark.parametrize("work", [None, "bf16"])
def test_updates_over_the_range_of_gradients(sp, work):
    """From parameters of zero, so that nothing hides the update: gradients from 1e-25 (whose squares vanish next
    to eps) to 1e15."""
    n = 200_003
    g = 10.0 ** (torch.rand(n, device="cuda", generator=gen(10)) * 40 - 25) * torch.randn(n, device="cuda", generator=gen(11)).sign()
    m = g * torch.rand(n, device="cuda", generator=gen(12))
    v = (g * g) * torch.rand(n, device="cuda", generator=gen(13))
    p = torch.zeros(n, device="cuda")
    w = None if work is None else [torch.zeros(n, dtype=TYPES[work], device="cuda")]
    old = [host(x) for x in (p, g, m, v)]
    for step in (1, 1000, 2_000_000):
        pp, mm, vv = p.clone(), m.clone(), v.clone()
        sp.adam_step_tensors(sp.adam_list([pp], [g], [mm], [vv], lr=2.0 ** -7, params_work=w), 0.9, 0.999, 1e-15, step=step)
        h = dict(step=step, lr=2.0 ** -7, b1=0.9, b2=0.999, eps=1e-15)
        for name, got, want, b in zip("pmv", (pp, mm, vv), tl.adamw_step(*old, **h), tt.adam_bounds(*old, **h)):
            tt.within(host(got), want, b, "step %d %s" % (step, name))
        if w:
            assert torch.equal(w[0], pp.to(TYPES[work]))


def test_two_graphs_with_the_default_workspace(sp):
    """Each capture gets a workspace of its own; replayed in turn and on two streams at once they do not meet."""
    lens = [400_000, 3, 70_001]
    sides = []
    for k in range(2):
        views, flat, before = packed(lens, "f32", 300 + k)
        ctl, graph, stream = sp.grad_control(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        lst = sp.grad_list(views)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            sp.grad_norm(lst, ctl, max_norm=1.0)
        sides.append((views, ctl, graph, stream))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, graph, stream in sides:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for views, ctl, _, _ in sides:
        want, coef, _ = tl.grad_norm([host(v) for v in views], max_norm=1.0)
        tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
        tt.within(host(ctl.coef), coef, tt.scalar_bound(coef), "coef")
        assert int(ctl.step) == 10


def test_shared_gradient(sp):
    g = torch.randn(5000, device="cuda", generator=gen(9))
    ps = [torch.zeros_like(g) for _ in range(6)]
    lst = sp.adam_list(ps[:2], [g, g], ps[2:4], ps[4:], lr=[1e-2, 1e-2])
    sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, step=1)
    assert torch.equal(ps[0], ps[1]) and bool(ps[0].any())
    with pytest.raises(sp.Spin4dError) as e:
        sp.adam_step_tensors(lst, 0.9, 0.99, 1e-8, step=1, zero_grad=True)
    assert e.value.status == sp.ERR_INVALID
    ctl = sp.grad_control()
    sp.grad_norm([g, g], ctl)
    want = float(g.double().square().sum().mul(2).sqrt())
    tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm of a tensor listed twice")


@pytest.mark.parametrize("count", [3, 40])
def test_captured_sequence_replays_as_the_eager_one(sp, count):
    """The whole update in a graph: the step counts itself, new gradients are clipped anew, a bad one is skipped."""
    lens = [int(x) for x in np.random.default_rng(count).integers(1, 9000, count)]

    def make():
        state, flats, _ = _adam_state(lens, "f32", 70, work="f16")
        ws = torch.empty(sp.grad_norm_workspace(count), dtype=torch.uint8, device="cuda")
        return state, flats, sp.grad_list(state[1]), sp.adam_list(*state[:4], lr=1e-2, weight_decay=0.01,
                                                                  params_work=state[4]), sp.grad_control(), ws

    def update(x):
        sp.grad_norm(x[2], x[4], max_norm=0.1, workspace=x[5])
        sp.adam_step_tensors(x[3], 0.9, 0.99, 1e-8, control=x[4], zero_grad=True)

    eager, graphed = make(), make()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        update(graphed)
    for i in range(4):
        grads = torch.randn(eager[1][1].numel(), device="cuda", generator=gen(100 + i)) * 10.0 ** -i
        if i == 2:
            grads[lens[0] // 2 + 1] = float("nan")
        for x in (eager, graphed):
            x[1][1].copy_(grads)
        update(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager[4].buf[1:], graphed[4].buf[1:])
        assert int(eager[4].step) == (i + 1 if i < 2 else i) and int(eager[4].skipped) == (i >= 2)
        for k in (0, 1, 2, 3, 4):
            assert torch.equal(eager[1][k], graphed[1][k])


def test_captured_across_streams(sp):
    """Gradients written on two streams, joined, measured and used on a third: in a graph, replayed."""
    n = 50_001
    g = [torch.zeros(n, device="cuda") for _ in range(2)]
    src = [torch.randn(n, device="cuda", generator=gen(90 + k)) for k in range(2)]
    p, m, v = ([torch.zeros(n, device="cuda") for _ in range(2)] for _ in range(3))
    ctl, ws = sp.grad_control(), torch.empty(sp.grad_norm_workspace(2), dtype=torch.uint8, device="cuda")
    grads, adam = sp.grad_list(g), sp.adam_list(p, g, m, v, lr=1e-2)
    streams = [torch.cuda.Stream() for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[2]):
        for k in range(2):
            streams[k].wait_stream(streams[2])
            with torch.cuda.stream(streams[k]):
                g[k].add_(src[k])
            streams[2].wait_stream(streams[k])
        sp.grad_norm(grads, ctl, max_norm=1.0, workspace=ws)
        sp.adam_step_tensors(adam, 0.9, 0.99, 1e-8, control=ctl, zero_grad=True)
    for i in range(3):
        old = [[host(x[k]) for x in (p, src, m, v)] for k in range(2)]
        graph.replay()
        torch.cuda.synchronize()
        want, coef, _ = tl.grad_norm([o[1] for o in old], max_norm=1.0)
        tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
        h = dict(step=i + 1, lr=1e-2, b1=0.9, b2=0.99, eps=1e-8, coef=float(ctl.coef))
        for k in range(2):
            for name, got, w, b in zip("pmv", (p[k], m[k], v[k]), tl.adamw_step(*old[k], **h), tt.adam_bounds(*old[k], **h)):
                tt.within(host(got), w, b, "%s of replay %d" % (name, i))
    assert int(ctl.step) == 3


def test_two_streams_at_once(sp):
    lens = [300_000, 70_001]
    sides = []
    for k in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        views, flat, before = packed(lens, "f32", 80 + k)
        sides.append((s, views, before, sp.grad_control()))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, views, _, ctl in sides:
            sp.grad_norm(views, ctl, max_norm=1.0, stream=s)      # its own workspace, by default
    for s, views, _, ctl in sides:
        sp.clip_grads(views, ctl, stream=s)
    torch.cuda.synchronize()
    for s, views, before, ctl in sides:
        at = [1, 2 + lens[0]]
        old = [host(before[a:a + n]) for a, n in zip(at, lens)]
        want, coef, _ = tl.grad_norm(old, max_norm=1.0)
        tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
        assert int(ctl.step) == 20
        for v, o in zip(views, old):
            w = tl.clip(o, float(ctl.coef))
            tt.within(host(v), w, tt.clip_bound(w, "f32"), "clip")


def test_offsets_past_32_bits(sp):
    """An fp16 gradient of more than 2^32 values: the parts behind the border are measured and clipped."""
    n = (1 << 32) + 4099
    g = torch.zeros(n, dtype=torch.float16, device="cuda")
    places = torch.tensor([0, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1], device="cuda")
    g[places] = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0, 6.0], dtype=torch.float16, device="cuda")
    ctl = sp.grad_control()
    sp.grad_norm([g], ctl, max_norm=1.0)
    want = float(np.sqrt(91.0))
    tt.within(host(ctl.norm), want, tt.scalar_bound(want), "norm")
    sp.clip_grads([g], ctl)
    w = np.arange(1.0, 7.0) * float(ctl.coef)
    tt.within(host(g[places]), w, tt.clip_bound(w, "f16"), "clip")
    assert int(torch.count_nonzero(g[:1 << 31])) == 2 and int(torch.count_nonzero(g[1 << 31:])) == 4


def test_checked_build_gives_the_same_bits():
    """Norm, clip and update in the build with device checks, in processes of their own."""
    code = r"""
import sys
sys.path.insert(0, %r)
import torch
from spatiotemporal_neural_field_b200 import spin4d as sp
gen = torch.Generator(device="cuda").manual_seed(1)
r = lambda n: torch.randn(n, device="cuda", generator=gen)
g, p, m, v = ([r(n) for n in (70001, 0, 9)] for _ in range(4))
v = [x.square() for x in v]
ctl = sp.grad_control()
sp.grad_norm(g, ctl, max_norm=1.0)
sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=1e-2), 0.9, 0.99, 1e-8, control=ctl)
sp.clip_grads(g, ctl)
torch.cuda.synchronize()
sp.check_device_errors(clear=False)
out = torch.cat([x.view(torch.int32) for x in g + p + m + v] + [ctl.buf]).long()
print("BITS", sp.lib.spin4d_checked_build(), int((out * torch.arange(1, out.numel() + 1, device="cuda")).sum()))
""" % ROOT
    seen = {}
    for flag in ("0", "1"):
        r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, SPIN4D_CHECKED=flag), cwd=ROOT,
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-3000:]
        _, checked, bits = r.stdout.split()
        assert checked == flag
        seen[flag] = bits
    assert seen["0"] == seen["1"]


def test_a_decoder_trains_through_them(sp):
    """Forward, backward, norm, clipped step on the tiny decoder: the parameters that the oracle's
    gradients, norm and update give."""
    w = S.WORKLOADS["tiny_fp32"]
    grid, mlp, n = w["grid"], w["mlp"], 1500
    pos, tables = S.uniform_positions(n), S.hash_tables(grid, scale=1.0)
    weights, ups = S.mlp_weights(mlp, bias_scale=0.5), S.upstream_grads(n, S.DECODE_OUT_WIDTHS, 1.0)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()   # noqa: E731
    g, m = sp.grid_from_spec(grid), sp.mlp_from_spec(mlp)
    P, params = dev(pos), [dev(tables).float(), dev(weights).float()]
    start = [host(p) for p in params]
    grads, ms, vs = ([torch.zeros_like(p) for p in params] for _ in range(3))
    lst, ctl = sp.grad_list(grads), sp.grad_control()
    adam = sp.adam_list(params, grads, ms, vs, lr=[1e-2, 1e-3])
    sp.decode_bwd(g, m, P, params[0], params[1], {k: dev(v) for k, v in ups.items()}, grads[0], grads[1])
    before = [host(x) for x in grads]
    sp.grad_norm(lst, ctl, max_norm=1.0)
    sp.adam_step_tensors(adam, 0.9, 0.99, 1e-15, control=ctl, zero_grad=True)
    ot, ow = dec.decode_backward(pos, tables, weights, grid, mlp, ups)
    norm, coef, _ = tl.grad_norm([ot, ow], max_norm=1.0)
    # the gradients are within 1e-5 of the oracle's by their own test, and so is their norm
    assert abs(float(ctl.norm) - norm) <= 2e-5 * norm and 0 < float(ctl.coef) < 1
    for p0, p, m_, v_, gr, lr in zip(start, params, ms, vs, before, (1e-2, 1e-3)):
        h = dict(step=1, lr=lr, b1=0.9, b2=0.99, eps=1e-15, coef=float(ctl.coef))
        zero = np.zeros_like(p0)
        for name, got, want, b in zip("pmv", (p, m_, v_), tl.adamw_step(p0, gr, zero, zero, **h),
                                      tt.adam_bounds(p0, gr, zero, zero, **h)):
            tt.within(host(got), want, b, name)
    assert all(not x.any() for x in grads) and int(ctl.step) == 1
    for o, gr in zip((ot, ow), before):
        tol.normwise(gr, np.asarray(o).reshape(gr.shape), 1e-4, "gradient")
    out = sp.decode_fwd(g, m, P, params[0], params[1])
    assert all(bool(torch.isfinite(x).all()) for x in out.values())
