"""The 64-bit references of a training step's operators (norm_ref, sinks_ref), one after the other."""
import numpy as np

import norm_ref as N
import sinks_ref as S

EPS = 1e-5


def freqs_of(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def test_training_gradients_against_differences():
    """The references' chain of one head against difference quotients of their forward pass."""
    d, T, left, sinks, scale = 16, 24, 5, 2, 0.25
    rng = np.random.default_rng(4)
    x, k, v, do = (rng.standard_normal((T, d)) for _ in range(4))
    w = [1.0 + 0.3 * rng.standard_normal(d) for _ in range(2)]
    freqs, axis, pos, see = freqs_of(d), [0] * (d // 2), np.arange(T)[None], S.visible(T, T, left, sinks)

    def forward(x, k, v, wq, wk):
        a, b = (N.forward(t, u, EPS, pos, freqs, axis, False)[0] for t, u in ((x, wq), (k, wk)))
        return a, b, (do * S.forward(a, b, v, scale, see)[0]).sum()
    qn, kn, _ = forward(x, k, v, *w)
    dqn, dkn, dv = S.backward(qn, kn, v, do, scale, see)[0]
    dx, tx = N.backward(dqn, x, w[0], EPS, pos, freqs, axis, False)[:2]
    dk, tk = N.backward(dkn, k, w[1], EPS, pos, freqs, axis, False)[:2]
    at, grads = [x, k, v, *w], [dx, dk, dv, tx.sum(0), tk.sum(0)]
    for i, gr in enumerate(grads):
        u, h = rng.standard_normal(gr.shape), 1e-5
        f = [forward(*at[:i], at[i] + s * h * u, *at[i + 1:])[2] for s in (1, -1)]
        # the quotient's error: h^2 of a third derivative, and 2^-53 / h of the loss's terms
        assert abs((f[0] - f[1]) / (2 * h) - (gr * u).sum()) <= 1e-7 * (np.abs(gr * u).sum() + np.abs(do).sum())
