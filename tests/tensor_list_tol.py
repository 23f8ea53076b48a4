"""Bounds for the tensor-list kernels against the fp64 oracle, by counting
roundings.  u = 2^-24 is half a step of fp32; a rounding to a narrower type is
off by at most half of that type's step, or half of its smallest subnormal.

* norm, a tensor's norm, coef: 64-bit arithmetic, rounded once to fp32; the
  64-bit sum of N < 2^33 terms is off by less than N 2^-53 < 2^-20 u' of its
  own, and is halved by the root: u (1 + 2^-10) covers both for the sizes here
  (a thread adds < 2^12 terms, a tree joins the threads: 2^13 2^-53 < u 2^-16).
* clip: coef is fp32 (u), the product is rounded (u), then the output's type.
* Adam.  g = coef * grad: 1 rounding, coef given.
    m: b1, its product, 1-b1, its product, the sum: at most 4u of either term
       and the gradient's u: 5u (|b1 m| + |(1-b1) g|);
    v: the same with g twice rounded and squared: 7u of the (positive) sum;
    1/(1-b^t): t log b rounded (at most u after expm1, whose condition is
       x e^x/(e^x - 1) <= 1 for x < 0), expm1f within 1 ulp = 2u, division u: 4u;
    mh: m's error and 5u |mh|; sqrt(vh), itself within 2^-23 = 2u: (7u + 5u)/2 + 2u
       = 8u; + eps (rounded u, added u): 10u of the denominator; lr rounded u,
       product u, quotient within 2 ulp = 4u: in all 21u |update| + lr * (5u (|b1 m| +
       |(1-b1) g|)) / (1-b1^t) / denominator;
    p: decay * p: lr * decay rounded twice over (lr u, decay u, product u, product u): 4u;
       the sum of both and the difference from p: u of each.
  fp32 subnormals add at most 2^-148 to m and v.
"""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -148
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_SUBNORMAL = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def scalar_bound(want):
    return U * (1 + 2.0 ** -10) * abs(want) + TINY


def clip_bound(want, dtype):
    w = np.abs(np.asarray(want, np.float64))
    bound = 2 * U * w * (1 + 2 * U)
    if dtype != "f32":
        bound = bound + HALF_STEP[dtype] * (1 + 4 * U) * w
    return bound + HALF_SUBNORMAL[dtype] + 2.0 ** -149


def adam_bounds(p, g, m, v, step, lr, b1, b2, eps, decay=0.0, coef=1.0):
    """Bounds on (p, m, v) after the step, from the values before it."""
    p, g, m, v = (np.abs(np.asarray(x, np.float64)) for x in (p, g, m, v))
    g = abs(coef) * g
    terms = b1 * m + (1 - b1) * g
    dm = 5.05 * U * terms + TINY
    vn = b2 * v + (1 - b2) * g * g
    dv = 7.05 * U * vn + TINY
    den = np.sqrt(vn / (1 - b2 ** step)) + eps
    with np.errstate(divide="ignore", invalid="ignore"):
        scale = lr / (1 - b1 ** step) / den
        upd = np.where(terms > 0, terms * scale, 0.0)      # no smaller than |update|
        dp = np.where(terms > 0, (21.1 + 5.05) * U * upd, 0.0)
    shrink = lr * decay * p
    dp = dp + 4.05 * U * shrink + U * (upd + shrink) + U * (p + upd + shrink) + TINY
    return dp, dm, dv


def within(got, want, bound, what=""):
    """Every |got - want| <= bound; prints the worst ratio."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.size == 0:
        return 0.0
    assert np.all(np.isfinite(got)), what + ": non-finite values"
    ratio = float(np.max(np.abs(got - want) / bound))
    print("%-40s worst %.3f of the bound" % (what, ratio))
    assert ratio <= 1.0, (what, ratio, int(np.argmax(np.abs(got - want) / bound)))
    return ratio
