"""GPU parity of gdr_rotary with the fp64 form, at the bounds derived in
linear_reference; its frequencies (CPU)."""
import math

import numpy as np
import pytest
import torch

import linear_reference as R

BF, F32 = torch.bfloat16, torch.float32
DT = {"f32": F32, "bf16": BF}


def n64(t):
    return t.detach().cpu().double().numpy()


def close(name, got, want, bound):
    err = np.abs(n64(got) - want)
    assert got.shape == want.shape and np.isfinite(err).all() and (err - bound).max() <= 0, \
        f"{name}: error {err.max():.3e}, worst over its bound by {(err - bound).max():.3e}"


def make(seed, B, T, Hq, Hk, D, dt):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((B, T, (Hq + Hk) * D + 3), generator=g).to(DT[dt]).cuda()
    return wide[..., 1:1 + Hq * D].unflatten(-1, (Hq, D)), \
        wide[..., 1 + Hq * D:1 + (Hq + Hk) * D].unflatten(-1, (Hk, D))


def check(gdr, q, k, pos, f, inter=False, scale=1.0, inverse=False, dt="f32"):
    got = gdr.gdr_rotary(q, k, pos, f, interleaved=inter, scale=scale, inverse=inverse)
    torch.cuda.synchronize()
    p = n64(pos) if isinstance(pos, torch.Tensor) else pos + np.arange(q.shape[1])
    p = np.broadcast_to(p, q.shape[:2])
    for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
        want, m = R.rotary(n64(x), p, n64(f), inter, scale, inverse)
        close(name, y, want, R.rotary_bound(want, m, dt, np.abs(p).max()))
        assert torch.equal(y[..., 2 * len(f):], x[..., 2 * len(f):])
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (128, 128), (7, 2), (7, 6), (40, 24),
                                   (33, 18), (100, 100), (256, 80), (1024, 1024), (9, 8)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sizes(gdr_lib, D, rot, inter, dt):
    q, k = make(D + rot, 2, 5, 4, 2, D, dt)
    f = gdr_lib.gdr_rotary_frequencies(rot)
    pos = torch.arange(10, device="cuda").view(2, 5) * 17
    check(gdr_lib, q, k, pos, f, inter, 1.25, False, dt)
    check(gdr_lib, q, k, pos, f, inter, 1.25, True, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (32, 8), (5, 1), (17, 3)])
@pytest.mark.parametrize("T", [1, 3, 700])
def test_heads_and_lengths(gdr_lib, Hq, Hk, T):
    q, k = make(Hq + T, 3, T, Hq, Hk, 64, "bf16")
    f = gdr_lib.gdr_rotary_frequencies(64)
    check(gdr_lib, q, k, 11, f, dt="bf16")
    check(gdr_lib, q, k, torch.arange(T, device="cuda"), f, dt="bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("start", [0, -5, 131072, 1 << 20, (1 << 31) - 3, 1 << 40])
def test_far_positions(gdr_lib, start):
    """The angle is right where fp32 has long lost it."""
    q, k = make(3, 1, 6, 2, 1, 64, "f32")
    check(gdr_lib, q, k, start, gdr_lib.gdr_rotary_frequencies(64))


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (96, 50), (33, 18)])
def test_in_place_and_one_token(gdr_lib, inter, D, rot):
    q, k = make(4, 6, 5, 3, 2, D, "bf16")
    f = gdr_lib.gdr_rotary_frequencies(rot)
    pos = torch.randint(0, 5000, (6, 5), device="cuda")
    want = gdr_lib.gdr_rotary(q, k, pos, f, interleaved=inter)
    one = [gdr_lib.gdr_rotary(q[:, t], k[:, t], pos[:, t], f, interleaved=inter) for t in range(5)]
    only = gdr_lib.gdr_rotary(q, None, pos, f, interleaved=inter)
    # a slice of a wider tensor, turned where it lies: its neighbours stay
    wide = torch.cat([q.flatten(2), k.flatten(2), q.flatten(2)], -1)
    kept = wide.clone()
    n, m = 3 * D, 2 * D
    qi, ki = wide[..., :n].unflatten(-1, (3, D)), wide[..., n:n + m].unflatten(-1, (2, D))
    got = gdr_lib.gdr_rotary(qi, ki, pos, f, interleaved=inter, q_out=qi, k_out=ki)
    torch.cuda.synchronize()
    assert got[0] is qi and torch.equal(qi, want[0]) and torch.equal(ki, want[1])
    assert torch.equal(wide[..., n + m:], kept[..., n + m:])
    assert torch.equal(torch.stack([x[0] for x in one], 1), want[0])
    assert torch.equal(torch.stack([x[1] for x in one], 1), want[1])
    assert torch.equal(only[0], want[0]) and only[1] is None


@pytest.mark.gpu
def test_bad_values_stay_in_their_pair(gdr_lib):
    q, k = make(5, 2, 9, 3, 3, 64, "f32")
    f = gdr_lib.gdr_rotary_frequencies(48)
    want = gdr_lib.gdr_rotary(q, k, 3, f)
    q[1, 4, 2, 10] = float("nan")
    q[0, 0, 0, 60] = float("inf")
    got = gdr_lib.gdr_rotary(q, k, 3, f)
    torch.cuda.synchronize()
    hit = torch.zeros_like(want[0], dtype=torch.bool)
    hit[1, 4, 2, [10, 34]] = True
    hit[0, 0, 0, 60] = True
    assert torch.equal(got[0][~hit], want[0][~hit]) and torch.equal(got[1], want[1])
    assert not torch.isfinite(got[0][hit]).any()


# ---- frequencies (CPU) ---------------------------------------------------------------


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_16_amd as g
    return g


def freqs(gdr, *a, **kw):
    return gdr.gdr_rotary_frequencies(*a, device="cpu", **kw).numpy()


@pytest.mark.parametrize("rot", [2, 4, 64, 1024])
def test_plain_and_linear(gdr, rot):
    f = freqs(gdr, rot, 5e5)
    want = 5e5 ** (-2 * np.arange(rot // 2) / rot)
    np.testing.assert_allclose(f, want, rtol=1e-14)
    np.testing.assert_allclose(freqs(gdr, rot, 5e5, scaling="linear", factor=4), want / 4, rtol=1e-14)


def test_base(gdr):
    """The slowest rate is divided by the factor, the fastest kept."""
    f, s = freqs(gdr, 64), freqs(gdr, 64, scaling="base", factor=8)
    assert s[0] == f[0] == 1
    assert abs(s[-1] * 8 / f[-1] - 1) < 1e-12 and (np.diff(f / s) > 0).all()


def test_parts(gdr):
    f = freqs(gdr, 128)
    s = freqs(gdr, 128, scaling="parts", factor=16, low=1, high=32, original=4096)
    turns = 4096 * f / (2 * math.pi)
    assert (s[turns >= 32] == f[turns >= 32]).all()
    np.testing.assert_allclose(s[turns <= 1], f[turns <= 1] / 16, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    w = (turns[mid] - 1) / 31
    np.testing.assert_allclose(s[mid], f[mid] * w + f[mid] / 16 * (1 - w), rtol=1e-12)
    assert mid.any()


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=0), dict(scaling="linear", factor=-2),
                                dict(base=0.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(scaling="parts", factor=2, low=4, high=4),
                                dict(scaling="parts", factor=2, low=-1),
                                dict(scaling="parts", factor=2, original=0),
                                dict(scaling="base", factor=float("inf"))])
def test_frequencies_refused(gdr, kw):
    with pytest.raises(gdr.GdrError):
        freqs(gdr, 64, **kw)


def test_more_frequencies_refused(gdr):
    for rot in (0, -2, 1026):
        with pytest.raises(ValueError):
            freqs(gdr, rot)
    with pytest.raises(gdr.GdrError):
        freqs(gdr, 7)
    with pytest.raises(gdr.GdrError):
        freqs(gdr, 2, scaling="base", factor=2)
    with pytest.raises(ValueError):
        freqs(gdr, 64, scaling="other")
