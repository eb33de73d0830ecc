"""64-bit references of the head norms with the rotation, written from their definitions in
include/fa.h, and the tolerances of their tests.

Tolerances.  u = 2^-24.  The sum of d squares in fp32, in any order, is off by at most d u of itself, the
mean and its sum with eps by 2 u more; r, the root's reciprocal, by half of that and u for its own rounding:
(d / 2 + 2) u.  x r w is two products more: a normed value n = w x r is off by (d / 2 + 4) u |n|.  The rotation
mixes the two values of a pair, a and b, with sines and cosines to 2^-22 and three roundings
(tests/paged_ref.py): (|a| + |b|) 2^-21, besides their own errors.
  Backward.  g = R^T dy is off by A 2^-21 with A = |a| + |b| of dy's pair (A = |g|, exactly, behind the pairs).  m =
mean(w g x) sums d products of three factors: off by (d + 4) u mean(|w| A |x|) besides g's error.  dx =
r (w g - x r^2 m): r carries (d / 2 + 2) u, and each product or sum u, so that with
S = r (|w| A + |x| r^2 mean(|w| A |x|)) >= |dx| all of it stays below S (2^-21 + (3 d + 16) u): three factors of r
(3 d / 2 + 6), the mean (d + 4), and six roundings.
  dw sums N terms g x r, each off by A |x| r (2^-21 + (d / 2 + 4) u), in fp32 in some order: N u sum A |x| r.
A 16-bit output adds half a step, 2^-8 of the value; a 32-bit one u.
"""
from __future__ import annotations

import numpy as np

import paged_ref as R

U = 2.0 ** -24


def _mixed(x, n, inter):
    """|a| + |b| of the pair that each feature belongs to; |x| behind the pairs."""
    ia, ib = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if inter else (np.arange(n), np.arange(n, 2 * n))
    out = np.abs(x)
    out[..., ia] = out[..., ib] = np.abs(x[..., ia]) + np.abs(x[..., ib])
    return out


def rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def forward(x, w, eps, pos, freqs, axis, inter):
    """x [..., T, d] normed by w [d] and turned by pos [axes][T]; the tolerance of an fp32 computation."""
    n = x * rms(x, eps) * w
    y, tol = R.rotate(n, pos, freqs, axis, inter)
    return y, tol + (x.shape[-1] / 2 + 4) * U * _mixed(n, len(freqs), inter)


def backward(dy, x, w, eps, pos, freqs, axis, inter):
    """dx, the terms of dw (to be summed over the rows), and the tolerances of dx and of the summed dw's terms
    (without the sum's own)."""
    d = x.shape[-1]
    g, _ = R.rotate(dy, pos, freqs, axis, inter, inverse=True)
    a = _mixed(dy, len(freqs), inter)
    far = np.abs(pos).max(initial=0) * max(abs(f) for f in freqs) * 2.0 ** -53   # the reference's own angles
    r = rms(x, eps)
    dx = r * (w * g - x * r * r * (w * g * x).mean(-1, keepdims=True))
    s = r * (np.abs(w) * a + np.abs(x) * r * r * (np.abs(w) * a * np.abs(x)).mean(-1, keepdims=True))
    return dx, g * x * r, s * (2.0 ** -21 + far + (3 * d + 16) * U), a * np.abs(x) * r * (2.0 ** -21 + far + (d / 2 + 4) * U), a * np.abs(x) * r
