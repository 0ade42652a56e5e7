"""The fp64 forms of linear_reference against central differences and against each
other, and mistakes planted in them that the differences see (CPU)."""
import numpy as np
import pytest

import linear_reference as R
from test_block_reference import differences


def la_args(seed, B=2, T=7, H=4, Hk=2, Dk=3, Dv=5, head=False):
    g = R.rng(seed)
    a = [g.standard_normal((B, T, Hk, Dk)), g.standard_normal((B, T, Hk, Dk)),
         g.standard_normal((B, T, H, Dv)), -np.exp(g.standard_normal(H if head else (B, T, H))),
         g.standard_normal((B, H, Dv, Dk))]
    return a, g.standard_normal((B, T, H, Dv)), g.standard_normal((B, H, Dv, Dk))


def la_loss(do, ds, scale):
    def f(q, k, v, g, s0):
        (o, s), _, _ = R.la_fwd(q, k, v, g, s0, scale)
        return (o * do).sum() + (s * ds).sum()
    return f


def la_grads(a, do, ds, scale):
    r = R.la_bwd(*a, do, ds, scale)[0]
    if a[3].ndim == 1:
        r["dg"] = r["dg"].sum((0, 1))
    return [r[n] for n in ("dq", "dk", "dv", "dg", "ds0")]


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("T", [1, 2, 9])
def test_linear_attention_gradients(head, T):
    a, do, ds = la_args(T, T=T, head=head)
    differences(la_loss(do, ds, 0.7), a, la_grads(a, do, ds, 0.7), 3)


@pytest.mark.parametrize("i", range(5))
def test_one_gradient_off(i):
    a, do, ds = la_args(11)
    g = la_grads(a, do, ds, 0.7)
    g[i] = np.roll(g[i], 1, 1)
    with pytest.raises(AssertionError):
        differences(la_loss(do, ds, 0.7), a, g, 4)


def test_shared_heads_not_summed():
    a, do, ds = la_args(12)
    g = la_grads(a, do, ds, 0.7)
    g[0] = g[0] / 2
    with pytest.raises(AssertionError):
        differences(la_loss(do, ds, 0.7), a, g, 4)


def test_decay_gradient_is_the_running_sum():
    """dg_t = a_t <G_t, S_{t-1}> is also the sum from t on of q . dq - k . dk plus
    what the final state's gradient says."""
    (q, k, v, g, s0), do, ds = la_args(13)
    (_, s), _, _ = R.la_fwd(q, k, v, g, s0, 0.7)
    r = R.la_bwd(q, k, v, g, s0, do, ds, 0.7)[0]
    H, B, T = 4, 2, 7
    one = R.la_bwd(R.spread(q, H), R.spread(k, H), v, g, s0, do, ds, 0.7)[0]
    e = (R.spread(q, H) * one["dq"]).sum(-1) - (R.spread(k, H) * one["dk"]).sum(-1)
    want = np.flip(np.cumsum(np.flip(e, 1), 1), 1) + (ds * s).sum((2, 3))[:, None]
    np.testing.assert_allclose(r["dg"], want, rtol=1e-10, atol=1e-10)
    assert r["dg"].shape == (B, T, H)


def test_chunks_and_tokens_agree():
    """The chunk formulas that the kernels evaluate, in fp64."""
    (q, k, v, g, s0), _, _ = la_args(14, T=9, Hk=4)
    (o, s), _, _ = R.la_fwd(q, k, v, g, s0, 0.7)
    L = np.cumsum(g, 1)
    D = np.exp(np.minimum(L[:, :, None] - L[:, None], 0)) * np.tril(np.ones((9, 9)))[None, ..., None]
    P = 0.7 * np.einsum("bihd,bjhd->bijh", q, k) * D
    want = np.einsum("bijh,bjhd->bihd", P, v) + \
        0.7 * np.exp(L)[..., None] * np.einsum("bhvk,bihk->bihv", s0, q)
    np.testing.assert_allclose(o, want, rtol=1e-11, atol=1e-11)
    end = np.exp(L[:, -1])[..., None, None] * s0 + \
        np.einsum("bjh,bjhv,bjhk->bhvk", np.exp(L[:, -1:] - L), v, k)
    np.testing.assert_allclose(s, end, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_turns_back(inter):
    g = R.rng(5)
    x, pos = g.standard_normal((2, 6, 3, 10)), np.arange(12).reshape(2, 6) * 1000
    f = 10000.0 ** (-np.arange(4) / 4)
    y, _ = R.rotary(x, pos, f, inter, 1.5, False)
    z, _ = R.rotary(y, pos, f, inter, 1 / 1.5, True)
    np.testing.assert_allclose(x, z, atol=1e-12)
    # the reverse mode: <dy, y> = <dx, x> for every dy
    dy = g.standard_normal(x.shape)
    dx, _ = R.rotary(dy, pos, f, inter, 1.5, True)
    np.testing.assert_allclose((dy * y).sum(), (dx * x).sum(), rtol=1e-12)
    # the angle between two tokens is that of their distance
    d = [(R.rotary(x[0, 0], np.int64(p), f, inter, 1, False)[0] *
          R.rotary(x[0, 1], np.int64(p + 7), f, inter, 1, False)[0])[..., :8].sum(-1)
         for p in (0, 50)]
    np.testing.assert_allclose(d[0], d[1], rtol=1e-9)


@pytest.mark.parametrize("weight", [True, False])
def test_rms_gradients(weight):
    g = R.rng(6)
    x, w, dy = g.standard_normal((4, 9)), g.standard_normal(9), g.standard_normal((4, 9))
    w = w if weight else None
    (dx, dw), _ = R.rms_bwd(x, w, dy, 1e-3, None)

    def f(x, w):
        return (R.rms_fwd(x, w, 1e-3) * dy).sum()

    differences(f, (x, w), (dx, dw), 7)
    with pytest.raises(AssertionError):
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-3)
        m2 = (dy * (1 if w is None else w) * n).mean(-1, keepdims=True)
        differences(f, (x, w), (dx + n * m2, dw), 7)
