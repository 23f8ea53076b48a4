"""GPU parity of the tensor-list calls on both sides of each kernel's list
capacity (norm and clip 16, 64, 320 and 1024 tensors, Adam 16, 64, 224 and
448), and on lists so long that a block walks several tiles and crosses from one
tensor to the next.  The 64-bit formulas and their bounds are computed on the
device."""
import numpy as np
import pytest

from oracle import tensor_list as tl
from tests import tensor_list_tol as tt

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U, TINY = tt.U, tt.TINY
TYPES = (torch.float32, torch.float16, torch.bfloat16)
NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
B1, B2, EPS = 0.9, 0.99, 1e-8


@pytest.fixture(scope="module")
def sp():
    from spatiotemporal_neural_field_b200 import spin4d
    return spin4d


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def views(lens, dtype, seed, scale=1e-2, gap=1):
    """Tensors of one buffer, `gap` values apart, so that they start at every alignment of their type; and the buffer."""
    flat = (torch.randn(sum(lens) + gap * (len(lens) + 1), device="cuda", generator=gen(seed)) * scale).to(dtype)
    out, at = [], gap
    for n in lens:
        out.append(flat[at:at + n])
        at += n + gap
    return out, flat


def inside(got, want, bound, what):
    """Every |got - want| <= bound, on the device."""
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    ratio = float(((got - want).abs() / bound).max()) if got.numel() else 0.0
    assert ratio <= 1.0, (what, ratio)


def clip_bound(want, dtype):
    w, name = want.abs(), NAMES[dtype]
    narrow = 0.0 if name == "f32" else tt.HALF_STEP[name] * (1 + 4 * U)
    return (2 * U * (1 + 2 * U) + narrow) * w + tt.HALF_SUBNORMAL[name] + 2.0 ** -149


def adam64(p, g, m, v, step, lr, decay, coef):
    """(p, m, v) after the step and the bounds of tensor_list_tol.adam_bounds around them."""
    p, g, m, v = p.double(), coef * g.double(), m.double(), v.double()
    terms = B1 * m.abs() + (1 - B1) * g.abs()
    m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
    den = (v / (1 - B2 ** step)).sqrt() + EPS
    upd, most, shrink = lr / (1 - B1 ** step) * m / den, lr / (1 - B1 ** step) * terms / den, lr * decay * p.abs()
    dp = (21.1 + 5.05 + 1) * U * most + 5.05 * U * shrink + U * (p.abs() + most + shrink) + TINY
    return (p - upd - lr * decay * p, m, v), (dp, 5.05 * U * terms + TINY, 7.05 * U * v + TINY)


def small_lens(count, seed):
    lens = [int(x) for x in np.random.default_rng(seed).integers(0, 5000, count)]
    lens[count // 3] = 0
    return lens


def norm64(tensors, kind):
    each = [float({"l2": lambda a: a.square().sum().sqrt(), "l1": lambda a: a.sum(), "inf": lambda a: a.max()}[kind](
        t.double().abs())) if t.numel() else 0.0 for t in tensors]
    whole = {"l2": lambda e: float(np.sqrt(np.sum(np.square(e)))), "l1": np.sum, "inf": np.max}[kind](each)
    return float(whole), np.array(each)


def near(got, want, what):
    tt.within(got.double().cpu().numpy(), want, tt.scalar_bound(want), what)


@pytest.mark.parametrize("kind", ["l2", "l1", "inf"])
@pytest.mark.parametrize("count", [16, 17, 64, 65, 320, 321, 1024, 1025])
def test_norm_on_both_sides_of_a_capacity(sp, count, kind):
    lens = small_lens(count, count)
    for big in (None, count - 1):                        # short tensors alone, and one of many blocks at the end
        if big is not None:
            lens[big] = 3_000_001
        grads = [views([n], TYPES[k % 3], 1000 + k, 10.0 ** -(k % 4), 1 + k % 5)[0][0] for k, n in enumerate(lens)]
        ctl, norms = sp.grad_control(), torch.full((count,), -1.0, device="cuda")
        want, each = norm64(grads, kind)
        for given in (norms, None):
            sp.grad_norm(grads, ctl, max_norm=0.5, norm_type=kind, norms=given)
            near(ctl.norm, want, "norm")
            near(ctl.coef, min(1.0, 0.5 / (want + tl.CLIP_EPS)), "coef")
        near(norms, each, "norms")


def check_clip(sp, lens, dtype, out):
    grads, flat = views(lens, dtype, 11)
    outs, oflat = views(lens, out, 12, gap=2) if out is not None else (grads, flat)
    before, obefore = flat.clone(), oflat.clone()
    lst, ctl = sp.grad_list(grads, outs if out is not None else None), sp.grad_control()
    sp.grad_norm(lst, ctl, max_norm=0.05)
    coef = float(ctl.coef)
    assert 0 < coef < 1
    sp.clip_grads(lst, ctl)
    gap = 1 if out is None else 2
    want, written, a, b = oflat.double(), torch.zeros(oflat.numel(), dtype=torch.bool, device="cuda"), 1, gap
    for n in lens:
        want[b:b + n] = before[a:a + n].double() * coef
        written[b:b + n] = True
        a, b = a + n + 1, b + n + gap
    inside(oflat[written], want[written], clip_bound(want[written], oflat.dtype), "clip")
    assert torch.equal(oflat[~written], obefore[~written])
    if out is not None:
        assert torch.equal(flat, before)


@pytest.mark.parametrize("dtype,out", [(torch.float32, None), (torch.float16, torch.float32), (torch.bfloat16, None)])
@pytest.mark.parametrize("count", [16, 17, 64, 65, 320, 321, 1024, 1025])
def test_clip_on_both_sides_of_a_capacity(sp, count, dtype, out):
    check_clip(sp, small_lens(count, count), dtype, out)


@pytest.mark.parametrize("dtype,out", [(torch.float32, None), (torch.float16, torch.float32)])
@pytest.mark.parametrize("count,big_at", [(5, 2), (40, 0), (120, 60), (500, 499)])
def test_clip_blocks_that_cross_tensors(sp, count, big_at, dtype, out):
    """32 blocks a SM have a tile each up to 9.7M values; 21M give them three."""
    lens = small_lens(count, 50 + count)
    lens[big_at] = 21_000_003
    check_clip(sp, lens, dtype, out)


def check_adam(sp, lens, dtype, work, zero, loose, step, seed):
    """All tensors of a list, those of each kind views of one buffer; `loose`: gradients at other offsets."""
    count = len(lens)
    p, pf = views(lens, torch.float32, seed, 1.0)
    m, mf = views(lens, torch.float32, seed + 1)
    v, vf = views(lens, torch.float32, seed + 2)
    vf.square_().add_(1e-10)
    g, gf = views(lens, dtype, seed + 3, gap=2 if loose else 1)
    w, wf = views(lens, work, seed + 4) if work is not None else (None, None)
    flats = [f for f in (pf, mf, vf, gf, wf) if f is not None]
    before = [f.clone() for f in flats]
    old = [[t.clone() for t in ts] for ts in (p, g, m, v)]
    lr, decay = [2.0 ** -7 * (1 + k % 3) for k in range(count)], [0.0 if k % 2 else 0.05 for k in range(count)]
    ctl, flag = sp.grad_control(step=step - 1), torch.zeros(1, dtype=torch.int32, device="cuda")
    sp.grad_norm(g, ctl, max_norm=0.5)
    sp.adam_step_tensors(sp.adam_list(p, g, m, v, lr=lr, weight_decay=decay, params_work=w), B1, B2, EPS, control=ctl,
                         zero_grad=zero, nonfinite_flag=flag)
    coef = float(ctl.coef)
    assert 0 < coef < 1 and int(ctl.step) == step and int(flag) == 0
    for k in range(count):
        want, bounds = adam64(*(o[k] for o in old), step, lr[k], decay[k], coef)
        for name, got, x, b in zip("pmv", (p[k], m[k], v[k]), want, bounds):
            inside(got, x, b, "%s of tensor %d, %d values" % (name, k, lens[k]))
        if work is not None:
            assert torch.equal(w[k], p[k].to(work))
        assert not bool(g[k].any()) if zero else torch.equal(g[k], old[1][k])
    # what lies between the tensors
    for f, b, gap in zip(flats, before, (1, 1, 1, 2 if loose else 1, 1)):
        keep, at = torch.ones(f.numel(), dtype=torch.bool, device="cuda"), gap
        for n in lens:
            keep[at:at + n] = False
            at += n + gap
        assert torch.equal(f[keep], b[keep])


@pytest.mark.parametrize("dtype,work,zero,loose", [
    (torch.float32, torch.float16, True, False), (torch.bfloat16, None, False, True), (torch.float16, torch.bfloat16, True, True)])
@pytest.mark.parametrize("count", [16, 17, 64, 65, 224, 225, 448, 449])
def test_adam_on_both_sides_of_a_capacity(sp, count, dtype, work, zero, loose):
    check_adam(sp, small_lens(count, count), dtype, work, zero, loose, 3, 60)


@pytest.mark.parametrize("count,big_at,big,dtype,work,zero,loose", [
    (3, 1, 33_000_005, torch.float32, torch.float16, False, False),
    (40, 0, 60_000_001, torch.float16, None, True, False),
    (120, 60, 31_000_001, torch.bfloat16, torch.float16, False, True),
    (120, 119, 31_000_003, torch.float32, None, True, True),
    (300, 299, 61_000_001, torch.float32, torch.bfloat16, True, False),
    (300, 150, 31_000_007, torch.bfloat16, None, False, False),
    (460, 0, 31_000_001, torch.float32, torch.float16, False, True),
])
def test_adam_blocks_that_cross_tensors(sp, count, big_at, big, dtype, work, zero, loose):
    """96 blocks a SM have a tile each up to 29M values; 31M give them two, 60M three."""
    lens = small_lens(count, 90 + count)
    lens[big_at] = big
    check_adam(sp, lens, dtype, work, zero, loose, 5, 80)


def test_coefficients_at_the_edges_of_fp32(sp):
    """One below fp32's range is 0: zeros are written, and the step counts; the largest scale leaves zeros zeros."""
    g = torch.full((5000,), 1e36, device="cuda")
    ctl = sp.grad_control()
    for max_norm in (1e-3, 1e-8):
        sp.grad_norm([g], ctl, max_norm=max_norm)
        want = max_norm / float(g.double().square().sum().sqrt())
        near(ctl.coef, want, "coef of max_norm %g" % max_norm)
    assert float(ctl.coef) == 0.0 and int(ctl.step) == 2 and int(ctl.skipped) == 0
    sp.clip_grads([g], ctl)
    assert not bool(g.any())
    scale = float(np.finfo(np.float32).max)
    p, m, v = (torch.ones_like(g) for _ in range(3))
    ctl = sp.grad_control()
    sp.grad_norm([g], ctl, max_norm=1.0, grad_scale=scale)
    sp.adam_step_tensors(sp.adam_list([p], [g], [m], [v], lr=1e-3), B1, B2, EPS, control=ctl)
    sp.clip_grads([g], ctl)
    assert float(ctl.coef) == scale and not bool(g.any())
    assert all(bool(torch.isfinite(x).all()) for x in (p, m, v))


def test_eps_from_the_smallest_to_the_largest(sp):
    """Denominators of every size that an accepted eps gives, entries without gradient among them."""
    n = 5000
    g = 10.0 ** (torch.rand(n, device="cuda", generator=gen(1)) * 40 - 25)
    g[::5] = 0
    for eps in (2.0 ** -126, 1e-30, 1.0, 2.0 ** 60, 2.0 ** 125):
        p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
        sp.adam_step_tensors(sp.adam_list([p], [g], [m], [v], lr=2.0 ** -7), B1, B2, eps, step=1)
        z = np.zeros(n)
        h = dict(step=1, lr=2.0 ** -7, b1=B1, b2=B2, eps=eps)
        want = tl.adamw_step(z, g.double().cpu().numpy(), z, z, **h)
        bounds = tt.adam_bounds(z, g.double().cpu().numpy(), z, z, **h)
        # g^2 / 100 below fp32's range: v is 0 and the denominator eps alone, the step's own size is then bounded instead
        fine = want[2] >= 2.0 ** -126
        for name, got, w, b in zip("pmv", (p, m, v), want, bounds):
            tt.within(got.double().cpu().numpy()[fine], w[fine], b[fine], "eps %g %s" % (eps, name))
        assert not bool(p[::5].any()) and bool(torch.isfinite(p).all())
