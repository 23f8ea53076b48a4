"""Pins for the tensor-list oracle (norms, clipping, Adam with decoupled
weight decay) and for the bounds that hold the kernels to it: closed forms,
invariants, fp32 restatements that the bounds admit, planted mistakes that
they do not."""
import numpy as np
import pytest

from oracle import decoder as dec
from oracle import tensor_list as tl
from tests import tensor_list_tol as tt


def test_norm_closed_forms():
    g = [np.array([3.0, -4.0]), np.array([]), np.array([[12.0]])]
    assert tl.grad_norm(g)[0] == 13.0 and tl.grad_norm(g)[2] == [5.0, 0.0, 12.0]
    assert tl.grad_norm(g, kind="l1")[0] == 19.0
    assert tl.grad_norm(g, kind="inf")[0] == 12.0
    assert tl.grad_norm(g, scale=0.5)[0] == 6.5
    assert tl.grad_norm([], max_norm=1.0)[:2] == (0.0, 1.0)


def test_coefficient_brings_the_norm_to_max_norm():
    g = [np.random.default_rng(0).standard_normal(1000), np.random.default_rng(1).standard_normal(7)]
    for kind in ("l2", "l1", "inf"):
        for scale in (1.0, 1 / 128):
            norm, coef, _ = tl.grad_norm(g, max_norm=0.01, kind=kind, scale=scale)
            after = tl.grad_norm([tl.clip(x, coef) for x in g], kind=kind)[0]
            assert abs(after - 0.01 * norm / (norm + 1e-6)) <= 1e-14
            norm, coef, _ = tl.grad_norm(g, max_norm=1e9, kind=kind, scale=scale)
            assert coef == scale                     # a small gradient is only unscaled


def test_non_finite_gradients_are_dropped_whole():
    for bad in (np.nan, np.inf, -np.inf):
        norm, coef, each = tl.grad_norm([np.ones(3), np.array([1.0, bad])], max_norm=1.0)
        assert not np.isfinite(norm) and coef == 0.0 and each[0] == np.sqrt(3.0)
        assert np.array_equal(tl.clip(np.array([1.0, bad]), coef), [0.0, 0.0])


def test_adamw_is_adam_without_decay_and_shrinks_with_it():
    r = np.random.default_rng(2)
    p, g, m = (r.standard_normal(50) for _ in range(3))
    v = r.random(50)
    for a, b in zip(tl.adamw_step(p, g, m, v, 3, 1e-2, 0.9, 0.99, 1e-8),
                    dec.adam_step(p, g, m, v, 3, 1e-2, 0.9, 0.99, 1e-8)):
        assert np.allclose(a, b, rtol=1e-15, atol=0)
    q, _, _ = tl.adamw_step(p, 0 * g, 0 * m, 0 * v, 1, 1e-2, 0.9, 0.99, 1e-8, decay=0.1)
    assert np.allclose(q, p * (1 - 1e-3), rtol=1e-15, atol=0)


def _adam32(p, g, m, v, step, lr, b1, b2, eps, decay, coef, mistake=None):
    """The formula in fp32, as a kernel has it; ``mistake`` plants one."""
    f = np.float32
    p, g, m, v = (np.asarray(x, f) for x in (p, g, m, v))
    g = f(coef) * g
    if mistake == "coupled decay":
        g = g + f(decay) * p
    m = f(b1) * m + f(1 - b1) * g
    v = f(b2) * v + f(1 - b2) * ((g if mistake != "squares unclipped" else g / f(coef)) ** 2)
    t = step + (1 if mistake == "step off by one" else 0)
    i1, i2 = f(1 / f(1 - b1 ** t)), f(1 / f(1 - b2 ** t))
    if mistake == "no correction":
        i1 = i2 = f(1)
    upd = f(lr) * (m * i1) / (np.sqrt(v * i2) + f(eps))
    if mistake == "eps inside":
        upd = f(lr) * (m * i1) / np.sqrt(v * i2 + f(eps))
    rate = f(decay) if mistake == "decay without rate" else f(lr) * f(decay)
    q = p - (upd + (0 if mistake == "coupled decay" else rate * p))
    return q, m, v


def _state(n=4096, seed=5):
    r = np.random.default_rng(seed)
    g = (r.standard_normal(n) * 10.0 ** r.uniform(-6, 0, n)).astype(np.float32)
    g[::7] = 0
    m = (r.standard_normal(n) * 1e-2).astype(np.float32)
    v = (m.astype(np.float64) ** 2 * (1 + r.random(n)) + 1e-12).astype(np.float32)
    return r.standard_normal(n).astype(np.float32), g, m, v


MISTAKES = ("coupled decay", "squares unclipped", "step off by one", "no correction", "eps inside",
            "decay without rate")


@pytest.mark.parametrize("mistake", (None,) + MISTAKES)
def test_bounds_admit_fp32_and_catch_mistakes(mistake):
    s = _state()
    # rates and coefficient that fp32 holds exactly: the bound counts their rounding as well
    hyper = dict(step=5, lr=2.0 ** -7, b1=0.9, b2=0.99, eps=1e-5, decay=2.0 ** -4, coef=0.25)
    want = tl.adamw_step(*s, **hyper)
    bounds = tt.adam_bounds(*s, **hyper)
    got = _adam32(*s, mistake=mistake, **hyper)
    inside = [bool(np.all(np.abs(a.astype(np.float64) - b) <= c)) for a, b, c in zip(got, want, bounds)]
    assert all(inside) == (mistake is None), (mistake, inside)


def test_clip_bounds_admit_rounding_to_each_type():
    import torch
    g = torch.randn(5000, generator=torch.Generator().manual_seed(0)) * 1e-2
    coef = np.float32(0.123)
    for name, t in (("f32", torch.float32), ("f16", torch.float16), ("bf16", torch.bfloat16)):
        got = (g * float(coef)).to(t).double().numpy()
        want = tl.clip(g.numpy(), float(coef))
        assert np.all(np.abs(got - want) <= tt.clip_bound(want, name))
        assert not np.all(np.abs(got * (1 + 4 * tt.HALF_STEP[name]) - want) <= tt.clip_bound(want, name))
