"""Mistakes planted in the fp64 gradients of the scan and the norm (CPU): the
comparison with differences sees each of them."""
import numpy as np
import pytest

import block_reference as R
from test_block_reference import differences, rng

KEYS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0")


def scan_args(seed):
    g = rng(seed)
    B, T, D, N = 2, 6, 4, 3
    a = [g.standard_normal((B, T, D)), 0.3 * g.standard_normal((B, T, D)),
         -np.exp(g.standard_normal((D, N))), g.standard_normal((B, T, 2, N)),
         g.standard_normal((B, T, 2, N)), g.standard_normal(D), g.standard_normal((B, T, D)),
         0.3 * g.standard_normal(D), g.standard_normal((B, D, N))]
    return a, g.standard_normal((B, T, D)), g.standard_normal((B, D, N))


def scan_loss(dout, dh):
    def f(*a):
        y, h, _ = R.scan_fwd(*a)
        return (y * dout).sum() + (h * dh).sum()
    return f


def test_scan_without_the_carried_gradient():
    """Each token's gradients from its own output alone: a_{t+1} g_{t+1} left
    out of g_t."""
    a, dout, dh = scan_args(1)
    right = R.scan_bwd(*a, dout, dh)
    differences(scan_loss(dout, dh), a, [right[k] for k in KEYS], 2)
    _, _, hs = R.scan_fwd(*a)
    T = dout.shape[1]
    cut = (0, 1, 3, 4, 6)
    own = [R.scan_bwd(*[v[:, t:t + 1] if k in cut else hs[t] if k == 8 else v
                        for k, v in enumerate(a)],
                      dout[:, t:t + 1], dh if t == T - 1 else None) for t in range(T)]
    wrong = {k: np.concatenate([o[k] for o in own], 1) if k in ("dx", "ddt", "dB", "dC", "dz")
             else own[0][k] if k == "dh0" else sum(o[k] for o in own) for k in KEYS}
    # what has no carried gradient in it is as it was
    for k in ("dC", "dD", "dz"):
        np.testing.assert_allclose(wrong[k], right[k], rtol=1e-12, atol=1e-12)
    with pytest.raises(AssertionError):
        differences(scan_loss(dout, dh), a, [wrong[k] for k in KEYS], 2)


@pytest.mark.parametrize("k", KEYS)
def test_scan_with_one_gradient_off(k):
    """One gradient taken a place too far along its first axis longer than one."""
    a, dout, dh = scan_args(3)
    o = R.scan_bwd(*a, dout, dh)
    o[k] = np.roll(o[k], 1, 1 if o[k].ndim > 1 else 0)
    with pytest.raises(AssertionError):
        differences(scan_loss(dout, dh), a, [o[j] for j in KEYS], 4)


@pytest.mark.parametrize("term", ["mean dn", "n mean(dn n)"])
def test_norm_without_a_mean(term):
    g = rng(5)
    x, w, b = g.standard_normal((4, 9)), g.standard_normal(9), g.standard_normal(9)
    dy = g.standard_normal((4, 9))
    (dx, dw, db), _ = R.norm_bwd(x, w, dy, 1e-5, None)

    def f(x, w, b):
        return (R.norm_fwd(x, w, b, 1e-5) * dy).sum()

    differences(f, (x, w, b), (dx, dw, db), 6)
    c = x - x.mean(-1, keepdims=True)
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + 1e-5)
    n, dn = c * r, dy * w
    gone = dn.mean(-1, keepdims=True) if term == "mean dn" else \
        n * (dn * n).mean(-1, keepdims=True)
    with pytest.raises(AssertionError):
        differences(f, (x, w, b), (dx + r * gone, dw, db), 6)
