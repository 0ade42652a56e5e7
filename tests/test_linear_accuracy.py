"""How exact linear attention is, beside how far off it may be at worst: norms of the
errors over whole outputs on fixed inputs.

Roundings are independent and the terms of random sign, so a sum's partial sums are in
norm no larger than the sum and the errors of n roundings add up as sqrt(n): an output
errs in norm by at most U (4 + sqrt(n)) of it, n the roundings one after the other on
its longest chain, each of them at most U, and 4 U for the factors of the decays (their
exponent's and the exponential's own) and the scale.  bf16 inputs: three terms of every
32 tokens or channels and the state's decay at every 64; fp32 inputs: every 4, and at
every 32.

Two bf16 terms for a computed operand in place of three leave 2^-18 of it, which these
bounds see (planted below, on the CPU) and the worst case of every rounding does not."""
import numpy as np
import pytest
import torch

import linear_reference as R
from test_linear_attn import DT, F32, make, n64

U = R.U


def depth(T, D, dt):
    if dt == "bf16":
        return 3 * -(-T // 32) + -(-T // 64) + -(-D // 32)
    return -(-T // 4) + -(-T // 32) + -(-D // 4)


def bound(T, D, dt):
    return U * (4 + depth(T, D, dt) ** 0.5)


def off(got, want):
    return np.linalg.norm(n64(got) - want) / np.linalg.norm(want)


# ---- the chunk's formulas with operands in a number of terms (CPU) -------------------------


def terms(x, n):
    """x as the sum of n bf16 terms, the largest first."""
    out, rest = np.zeros_like(x), x.copy()
    for _ in range(n):
        h = torch.from_numpy(rest.astype(np.float32)).bfloat16().double().numpy()
        out, rest = out + h, rest - h
    return out


def chunks(q, k, v, g, s0, scale, of_out, of_state):
    """o and the state of one head in chunks of 64 tokens, in 64 bits but for the terms
    of what the matrix cores take: the pairs' products and the state in `of_out`, the
    values scaled by their decays in `of_state`."""
    S, o = s0.T.copy(), np.zeros_like(v)
    for c in range(0, len(q), 64):
        s = slice(c, c + 64)
        L = np.cumsum(g[s])
        P = scale * np.tril(q[s] @ k[s].T * np.exp(np.minimum(L[:, None] - L, 0)))
        o[s] = terms(P, of_out) @ v[s] + scale * np.exp(L)[:, None] * (q[s] @ terms(S, of_out))
        S = np.exp(L[-1]) * S + k[s].T @ terms(np.exp(L[-1] - L)[:, None] * v[s], of_state)
    return o, S.T


@pytest.mark.parametrize("T,D", [(64, 64), (192, 64), (192, 128), (300, 128)])
def test_bounds_see_a_missing_term(T, D):
    g = R.rng(T + D)
    q, k, v = (torch.from_numpy(g.standard_normal((T, D))).bfloat16().double().numpy()
               for _ in range(3))
    d, s0 = -np.exp(1.5 * g.standard_normal(T) - 2), g.standard_normal((D, D))
    (o, s), _, _ = R.la_fwd(*[x[None, :, None] for x in (q, k, v, d)], s0[None, None], 0.3)
    o, s = o[0, :, 0], s[0, 0]

    def errors(*n):
        return [np.linalg.norm(x - y) / np.linalg.norm(y)
                for x, y in zip(chunks(q, k, v, d, s0, 0.3, *n), (o, s))]

    most = bound(T, D, "bf16")
    assert max(errors(3, 3)) < most / 20
    assert errors(2, 3)[0] > 2 * most
    assert errors(3, 2)[1] > 1.5 * most


# ---- the kernels ----------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(64, 64), (192, 64), (192, 128), (300, 128), (700, 64)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_forward(gdr_lib, T, D, dt):
    a, _, _ = make(81, 2, T, 3, 3, D, D, dt)
    o, s = gdr_lib.gdr_linear_attn_fwd(*a, scale=0.3, out_dtype=F32)
    torch.cuda.synchronize()
    (ow, sw), _, _ = R.la_fwd(*[n64(x) for x in a], 0.3)
    assert off(o, ow) <= bound(T, D, dt) and off(s, sw) <= bound(T, D, dt), (off(o, ow), off(s, sw))


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(64, 64), (192, 64), (192, 128), (700, 64)])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_backward(gdr_lib, T, D, state, dt):
    """dlog_decay_t sums (q dq)_ic and (k dk)_ic over the tokens from t on and the
    channels, and G S over a state: independent errors of each.  6 in place of 4: the
    products' own rounding and that of their sums over 16 channels."""
    a, do, ds = make(82, 2, T, 3, 3, D, D, dt, state=state)
    got = gdr_lib.gdr_linear_attn_bwd(*a, do, ds, scale=0.3)
    torch.cuda.synchronize()
    ref = [n64(x) for x in a]
    r = R.la_bwd(*ref, n64(do), n64(ds), 0.3)[0]
    for n, x in zip(("dq", "dk", "dv", "dg", "ds0"), got):
        if n != "dg" and np.any(r[n]):
            assert off(x, r[n]) <= bound(T, D, dt), (n, off(x, r[n]))
    one = U * (6 + depth(T, D, dt) ** 0.5)
    sq = ((ref[0] * r["dq"]) ** 2 + (ref[1] * r["dk"]) ** 2).sum(-1)
    var = np.flip(np.cumsum(np.flip(sq, 1), 1), 1)
    if state:
        (_, s), _, _ = R.la_fwd(*ref, 0.3)
        var = var + ((n64(ds) * s) ** 2).sum((2, 3))[:, None]
    assert np.linalg.norm(n64(got[3]) - r["dg"]) <= one * np.sqrt(var.sum())
    if not state:
        # no pair lies across the first token: the sum's error (of one value in place of
        # a norm, so six times as much) is taken out, and leaves the roundings of the
        # share that is taken
        assert (np.abs(n64(got[3])[:, 0]) <= 4 * U * 6 * one * np.sqrt(var[:, 0])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 31, 48, 64])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dots_lose_nothing_to_cancellation(gdr_lib, T, dt):
    """Whole numbers, no decay: q . dq and k . dk of 16 channels are below 2^24, but sums
    of products past it that cancel, channel by channel in pairs.  dlog_decay is exact."""
    g = torch.Generator().manual_seed(T)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g).double()

    B, H, D, Dv = 2, 2, 32, 16
    k = ints(-250, 250, B, T, H, D // 2).repeat_interleave(2, -1)
    q = ints(150, 250, B, T, H, D // 2).repeat_interleave(2, -1)
    q[..., 1::2] = ints(-1, 1, B, T, H, D // 2) - q[..., 1::2]
    v, do = ints(-10, 10, B, T, H, Dv), ints(-10, 10, B, T, H, Dv)
    one = R.la_bwd(*(x.numpy() for x in (q, k, v)), np.zeros((B, T, H)), None, do.numpy(), None, 1.0)[0]
    for x, dx in ((q, one["dq"]), (k, one["dk"])):
        p = x.numpy() * dx
        assert np.abs(p.reshape(B, T, H, 2, 16).sum(-1)).max() < 2 ** 24 and np.abs(dx).max() < 2 ** 24
        assert T < 31 or np.abs(p).max() > 2 ** 25
    assert np.abs(one["dg"]).max() < 2 ** 24
    a = [x.to(DT[dt]).cuda() for x in (q, k, v)]
    dg = gdr_lib.gdr_linear_attn_bwd(*a, torch.zeros(B, T, H, device="cuda"), None,
                                     do.to(DT[dt]).cuda())[3]
    torch.cuda.synchronize()
    assert (n64(dg) == one["dg"]).all(), np.abs(n64(dg) - one["dg"]).max()
