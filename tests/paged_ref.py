"""64-bit references of the rotary positions and the paged-cache operators, written from their
definitions in include/fa.h, and the tolerances of their tests.

Tolerances.  u = 2^-24 is half a step of fp32, 2^-8 of bf16, 2^-4 of e4m3 (relative; 2^-10
absolute below e4m3's smallest normal number).
  Rotation: an angle in [-pi/4, pi/4] carries the rounding of a 32-bit integer to fp32, of the
    constant 2 pi 2^-34 and of their product (3 u each, times pi/4) and of 2^-34 turns; the series
    adds 1.5 u: sine and cosine are off by at most 4 u = 2^-22.  a cos - b sin adds the rounding of
    one product and of the sum: (|a| + |b|) (2^-22 + 2^-23) < (|a| + |b|) 2^-21.  The reference's own
    p f is off by |p f| 2^-53 radians.  bf16 output adds 2^-8 |y|.
  Attention: a score is off by at most e = (d + 4) u c sum_i |q_i k_i| (fp32 sums of exact
    products, in any order), a probability by a factor e^{2e} and 2^-20 (exp2, the joins), so with
    A = sum p |v| an output is off by (2 e + 2^-18) A; probabilities that enter the second product
    with 11 bits or more add 2^-12 A, the bf16 output 2^-8 |o|.  In an e4m3 cache they enter as f16 after
    a factor of 2^15 on e^{s - m}: below 2^-14 f16 goes in steps of 2^-24, so that each e^{s - m} is off by up to
    2^-25 2^-15 = 2^-40 instead, where 2^-12 of it is less.  m only grows, and a later m scales the error down with
    the value; the sum l >= 1 divides it.  That adds 2^-40 sum |v|, over the entries that the row sees.  lse: e + 2^-20 (1 + |lse|).
    weight: (2 e + 2^-18) sum p, and u (M + 1) |w| for the additions.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def e4m3_values() -> np.ndarray:
    """The 256 code values."""
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def rotate(x: np.ndarray, pos: np.ndarray, freqs, axis, interleaved=False, inverse=False):
    """x [..., T, d] float64 turned by pos [axes][T]; and the tolerance of an fp32 computation."""
    n = len(freqs)
    f = np.asarray(freqs, dtype=np.float64)
    ang = pos[np.asarray(axis)].astype(np.float64).T * f          # [T][pairs]
    off = np.abs(ang) * 2.0 ** -53
    c, s = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
    ia, ib = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    y, tol = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    t = (np.abs(a) + np.abs(b)) * (2.0 ** -21 + off)
    tol[..., ia], tol[..., ib] = t, t
    return y, tol


def attend(q, k, v, scale, causal, group, codes=False):
    """q [Hq][Tq][d], k, v [Hkv][n][d] float64 -> o, lse, weight sums [Hkv][n] and the tolerances
    of the three (module docstring; codes: of an e4m3 cache), without the rounding of o to bf16."""
    Hq, Tq, d = q.shape
    n = k.shape[1]
    o, lse = np.zeros_like(q), np.full((Hq, Tq), -np.inf)
    w = np.zeros((k.shape[0], n))
    to, tl, tw = np.zeros_like(q), np.zeros((Hq, Tq)), np.zeros((k.shape[0], n))
    for h in range(Hq):
        kv = h // group
        for t in range(Tq):
            m = max(0, min(n, n - Tq + t + 1)) if causal else n
            if m == 0:
                continue
            s = scale * (k[kv, :m] @ q[h, t])
            e = (d + 4) * U * scale * float((np.abs(k[kv, :m]) @ np.abs(q[h, t])).max())
            mx = s.max()
            z = np.exp(s - mx).sum()
            p = np.exp(s - mx) / z
            o[h, t], lse[h, t] = p @ v[kv, :m], mx + np.log(z)
            w[kv, :m] += p
            to[h, t] = (2 * e + 2.0 ** -18 + 2.0 ** -12) * (p @ np.abs(v[kv, :m]))
            if codes:
                to[h, t] += 2.0 ** -40 * np.abs(v[kv, :m]).sum(0)
            tl[h, t] = e + 2.0 ** -20 * (1 + abs(lse[h, t]))
            tw[kv, :m] += (2 * e + 2.0 ** -18) * p
    return o, lse, w, to, tl, tw


def evict(weight, order, n, seen, budget, n_first, n_recent):
    """The old slot of each entry kept of one (sequence, KV head) with n entries."""
    end = min(n, budget)

    def rank(i):
        prot = order is not None and (order[i] < n_first or (n_recent > 0 and order[i] >= seen - n_recent))
        w = float(weight[i])
        return (0 if prot else 1, 0.0 if prot else (np.inf if np.isnan(w) else -w), 1 if (not prot and np.isnan(w)) else 0, i)

    stay = set(sorted(range(n), key=rank)[:end])
    late = iter(sorted(i for i in stay if i >= end))
    return [i if i in stay else next(late) for i in range(end)]
