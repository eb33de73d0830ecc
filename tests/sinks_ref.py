"""64-bit reference of attention under a causal window with sinks (include/fa.h: fa_fwd_sinks, fa_bwd_sinks), and
the tolerances of its tests.

Tolerances.  u = 2^-24; a bf16 rounding is off by 2^-8 of the value.  Forward: a score is off by at most
e = (d + 4) u c sum_i |q_i k_i| (e: the largest over a row), its exponential by 2^-18 of itself besides, and P enters its
product as bf16: with A = sum p |v| an output is off by (2 e + 2^-18 + 2^-8) A, and 2^-8 |o| for its own rounding.
lse: e + 2^-20 (1 + |lse|).
  Backward.  P comes from the scores and from lse: f = 2 e + 2^-18 + 2^-20 (1 + |lse|) of itself off.  dP = dO v^T: (d + 4) u
sum_i |dO_i v_i|.  D = dO . o with the forward's o: sum_i |dO_i| (its tolerance), and (d + 4) u sum |dO_i o_i|.
dS = P (dP - D): P times the two, f |dS|, and 2^-8 of what comes out for its rounding.  dV = P^T dO with P in bf16:
sum_r p (f + 2^-8) |dO_r|; dK = c dS^T Q and dQ = c dS K by dS's; their sums of N terms in fp32 add N u of the terms'
magnitudes, their own rounding 2^-8.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
BF = 2.0 ** -8


def visible(Tq, Tk, left, sinks):
    p = np.arange(Tq)[:, None] + Tk - Tq
    l = np.arange(Tk)
    return (l <= p) & ((l >= p - left) | (l < sinks)) if left >= 0 else l <= p


def forward(q, k, v, scale, see):
    """o, lse of one head, and their tolerances (that of o with its rounding), P and the errors of its scores."""
    d = q.shape[1]
    s = np.where(see, scale * (q @ k.T), -np.inf)
    e = np.where(see, (d + 4) * U * scale * (np.abs(q) @ np.abs(k).T), 0.0).max(1, initial=0.0)
    m = s.max(1, initial=-np.inf)
    live = np.isfinite(m)
    z = np.exp(s - np.where(live, m, 0.0)[:, None])
    l = z.sum(1)
    p = z / np.where(live, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(live, m + np.log(l), -np.inf)
    o = p @ v
    to = (2 * e + 2.0 ** -18 + BF)[:, None] * (p @ np.abs(v)) + BF * np.abs(o)
    tl = e + 2.0 ** -20 * (1 + np.abs(np.where(live, lse, 0.0)))
    return o, lse, to, tl, p, e


def backward(q, k, v, do, scale, see):
    """(dq, dk, dv) of one head and their tolerances, without the rounding of the outputs."""
    d = q.shape[1]
    o, lse, to, tl, p, e = forward(q, k, v, scale, see)
    f = (2 * e + 2.0 ** -18 + tl)[:, None]
    dp, D = do @ v.T, (do * o).sum(1, keepdims=True)
    ds = p * (dp - D)
    off = (d + 4) * U * (np.abs(do) @ np.abs(v).T)
    off_d = (np.abs(do) * to).sum(1, keepdims=True) + (d + 4) * U * (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
    t = p * (1 + f) * (off + off_d) + f * np.abs(ds)
    t += BF * (np.abs(ds) + t)
    n = max(q.shape[0], k.shape[0])
    mag = np.abs(ds) + t
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    tq = scale * (t + n * U * mag) @ np.abs(k)
    tk = scale * (t + n * U * mag).T @ np.abs(q)
    tv = (p * (f + BF + n * U)).T @ np.abs(do)
    return (dq, dk, dv), (tq, tk, tv)
