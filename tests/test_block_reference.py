"""The fp64 forms of block_reference against central differences, and their
majorants against the values (CPU)."""
import numpy as np
import pytest

import block_reference as R


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def differences(f, args, grads, seed, h=1e-6):
    """sum_i grad_i . v_i against (f(x + h v) - f(x - h v)) / 2h along one
    random direction of all arguments; f's third derivatives are O(1), so the
    difference errs by O(h^2) plus rounding 1e-16 |f| / h."""
    g = rng(seed)
    v = [None if a is None else g.standard_normal(a.shape) for a in args]
    up = f(*[None if a is None else a + h * d for a, d in zip(args, v)])
    dn = f(*[None if a is None else a - h * d for a, d in zip(args, v)])
    want = sum((gr * d).sum() for gr, d in zip(grads, v) if d is not None)
    scale = sum(np.abs(gr * d).sum() for gr, d in zip(grads, v) if d is not None)
    assert abs((up - dn) / (2 * h) - want) <= 1e-7 * scale


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 9])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients(K, T, silu):
    g = rng(K + T)
    x, w, b = g.standard_normal((2, T, 5)), g.standard_normal((5, K)), g.standard_normal(5)
    s0, dy = g.standard_normal((2, K - 1, 5)), g.standard_normal((2, T, 5))
    ds = g.standard_normal((2, K - 1, 5))

    def f(x, w, b, s0):
        y, sf, _, _ = R.conv_fwd(x, w, b, s0, silu)
        return (y * dy).sum() + (sf * ds).sum()

    (dx, dw, db, ds0), _ = R.conv_bwd(x, w, b, s0, dy, ds, silu)
    differences(f, (x, w, b, s0), (dx, dw, db, ds0), 1)


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("sp", [True, False])
def test_scan_gradients(G, sp):
    g = rng(G)
    B, T, D, N = 2, 7, 6, 3
    x, dt = g.standard_normal((B, T, D)), g.standard_normal((B, T, D)) * 0.3
    A, Bm = -np.exp(g.standard_normal((D, N))), g.standard_normal((B, T, G, N))
    Cm, Dk, z = g.standard_normal((B, T, G, N)), g.standard_normal(D), g.standard_normal((B, T, D))
    bias, h0 = g.standard_normal(D) * 0.3, g.standard_normal((B, D, N))
    dout, dh = g.standard_normal((B, T, D)), g.standard_normal((B, D, N))
    args = (x, dt, A, Bm, Cm, Dk, z, bias, h0)

    def f(*a):
        y, hf, _ = R.scan_fwd(*a, sp=sp)
        return (y * dout).sum() + (hf * dh).sum()

    o = R.scan_bwd(*args, dout, dh, sp=sp)
    differences(f, args, [o[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0")],
                2)
    m = R.scan_bwd(*args, dout, dh, sp=sp, majorant=True)
    assert all((np.abs(o[k]) <= m[k] * (1 + 1e-12)).all() for k in o)


def test_norm_gradients():
    g = rng(4)
    x, w, b = g.standard_normal((4, 9)), g.standard_normal(9), g.standard_normal(9)
    dy = g.standard_normal((4, 9))
    (dx, dw, db), _ = R.norm_bwd(x, w, dy, 1e-5, None)
    differences(lambda x, w, b: (R.norm_fwd(x, w, b, 1e-5) * dy).sum(), (x, w, b), (dx, dw, db), 3)


def test_a_planted_mistake_fails_its_difference():
    """A decay taken before the step's token enters the gradient twice is seen."""
    g = rng(5)
    x, w, b = g.standard_normal((1, 6, 3)), g.standard_normal((3, 4)), g.standard_normal(3)
    dy = g.standard_normal((1, 6, 3))
    (dx, dw, db, ds0), _ = R.conv_bwd(x, w, b, None, dy, None, True)

    def f(x, w, b):
        return (R.conv_fwd(x, w, b, None, True)[0] * dy).sum()

    differences(f, (x, w, b), (dx, dw, db), 6)
    with pytest.raises(AssertionError):
        differences(f, (x, w, b), (np.roll(dx, 1, 1), dw, db), 6)
