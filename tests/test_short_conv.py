"""GPU parity of gdr_short_conv_fwd, _step and _bwd with the fp64 form, at the
bounds derived in block_reference."""
import numpy as np
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def make(B, T, C, K, dt, seed, bias=True, state=True):
    g = rng(seed)

    def t(*shape, dtype=torch.float32, scale=1.0):
        return torch.from_numpy((scale * g.standard_normal(shape)).astype(np.float32)).to(dtype)

    return dict(x=t(B, T, C, dtype=DT[dt]), w=t(C, K, scale=0.6),
                bias=t(C, scale=0.3) if bias else None,
                s0=t(B, K - 1, C, dtype=DT[dt]) if state else None,
                dy=t(B, T, C), dsf=t(B, K - 1, C))


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def cu(t):
    return None if t is None else t.cuda()


def close(name, got, want, bound):
    err = np.abs(n64(got) - want)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if want.size:
        over = err - bound
        assert np.isfinite(err).all() and over.max() <= 0, \
            f"{name}: error {err.max():.3e}, worst over its bound by {over.max():.3e}"


def check_fwd(gdr, i, K, silu, out):
    y, sf = gdr.gdr_short_conv_fwd(cu(i["x"]), cu(i["w"]), cu(i["bias"]), cu(i["s0"]), silu=silu,
                                   out_dtype=DT[out])
    torch.cuda.synchronize()
    want, wsf, u, m = R.conv_fwd(n64(i["x"]), n64(i["w"]), n64(i["bias"]), n64(i["s0"]), silu)
    close("y", y, want, R.conv_fwd_bound(want, u, m, K, silu, out))
    assert (n64(sf) == wsf).all(), "the state is not a copy of the last inputs"


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 17, 64, 257, 1030])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_fwd_lengths(gdr_lib, T, K):
    check_fwd(gdr_lib, make(3, T, 72, K, "bf16", 10 * T + K), K, True, "f32")


@pytest.mark.parametrize("C", [1, 7, 8, 9, 513, 1030])
@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_fwd_channels_and_types(gdr_lib, C, dt, out):
    check_fwd(gdr_lib, make(2, 21, C, 4, dt, C), 4, True, out)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("silu", [True, False])
def test_fwd_options(gdr_lib, bias, state, silu):
    check_fwd(gdr_lib, make(2, 40, 33, 3, "f32", 5, bias, state), 3, silu, "f32")


@pytest.mark.parametrize("T", [0, 1, 2, 3, 9])
def test_state_in_place_and_empty(gdr_lib, T):
    """s_final in s0's buffer, also where it keeps rows of the old state."""
    i = make(2, T, 19, 4, "bf16", 77 + T)
    s = cu(i["s0"])
    y, sf = gdr_lib.gdr_short_conv_fwd(cu(i["x"]), cu(i["w"]), cu(i["bias"]), s, s_final=s)
    torch.cuda.synchronize()
    assert sf is s and y.shape == (2, T, 19)
    assert (n64(s) == R.conv_full(n64(i["x"]), n64(i["s0"]), 4)[:, T:]).all()


def test_slices_and_batch_order(gdr_lib):
    """A channel slice of a wider projection at an odd offset, batch and token
    axes swapped in memory, a broadcast batch."""
    g = rng(3)
    wide = torch.from_numpy(g.standard_normal((2, 30, 101)).astype(np.float32)).bfloat16()
    i = make(2, 30, 37, 4, "bf16", 4)
    swapped = torch.from_numpy(g.standard_normal((30, 2, 37)).astype(np.float32)).bfloat16()
    for x in (wide.cuda()[:, :, 5:42], swapped.cuda().transpose(0, 1),
              wide.cuda()[:1, :, 64:101].expand(2, 30, 37)):
        y, sf = gdr_lib.gdr_short_conv_fwd(x, cu(i["w"]), cu(i["bias"]), cu(i["s0"]))
        y2, sf2 = gdr_lib.gdr_short_conv_fwd(x.contiguous(), cu(i["w"]), cu(i["bias"]),
                                             cu(i["s0"]))
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(sf, sf2)


def test_whole_equals_chunks_and_steps(gdr_lib):
    """One call, two chunks through the state, and single tokens: equal bits."""
    i = make(3, 50, 65, 4, "bf16", 8)
    x, w, b, s0 = (cu(i[k]) for k in ("x", "w", "bias", "s0"))
    y, sf = gdr_lib.gdr_short_conv_fwd(x, w, b, s0)
    s = s0.clone()
    parts = [gdr_lib.gdr_short_conv_fwd(x[:, :2], w, b, s, s_final=s)[0],
             gdr_lib.gdr_short_conv_fwd(x[:, 2:31], w, b, s, s_final=s)[0]]
    for t in range(31, 50):
        parts.append(gdr_lib.gdr_short_conv_step(x[:, t], w, b, s).unsqueeze(1))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(s, sf)


@pytest.mark.parametrize("N,C,K,dt,out", [(1, 1, 2, "f32", "f32"), (5, 130, 3, "bf16", "f32"),
                                          (300, 67, 4, "bf16", "bf16"), (2, 4096, 4, "f32", "bf16")])
@pytest.mark.parametrize("silu", [True, False])
def test_step(gdr_lib, N, C, K, dt, out, silu):
    i = make(N, 1, C, K, dt, N + C)
    s = cu(i["s0"])
    y = gdr_lib.gdr_short_conv_step(cu(i["x"])[:, 0], cu(i["w"]), cu(i["bias"]), s, silu=silu,
                                    out_dtype=DT[out])
    torch.cuda.synchronize()
    want, wsf, u, m = R.conv_fwd(n64(i["x"]), n64(i["w"]), n64(i["bias"]), n64(i["s0"]), silu)
    close("y", y.unsqueeze(1), want, R.conv_fwd_bound(want, u, m, K, silu, out))
    assert (n64(s) == wsf).all()


def check_bwd(gdr, i, K, silu, grad="f32", dy="f32", dsf=True):
    d = i["dy"].to(DT[dy])
    df = i["dsf"] if dsf else None
    got = gdr.gdr_short_conv_bwd(cu(i["x"]), cu(i["w"]), cu(i["bias"]), cu(i["s0"]), cu(d), cu(df),
                                 silu=silu, grad_dtype=DT[grad])
    torch.cuda.synchronize()
    want, bound = R.conv_bwd(n64(i["x"]), n64(i["w"]), n64(i["bias"]), n64(i["s0"]), n64(d),
                             n64(df), silu)
    bound[0] = bound[0] + R.HALF[grad] * (np.abs(want[0]) + bound[0])
    for name, g, v, b in zip(("dx", "dw", "dbias", "ds0"), got, want, bound):
        if name == "dbias" and i["bias"] is None:
            assert g is None
            continue
        close(name, g, v, b)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 31, 33, 300])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_bwd_lengths(gdr_lib, T, K):
    check_bwd(gdr_lib, make(3, T, 70, K, "bf16", T + K), K, True)


@pytest.mark.parametrize("C", [1, 3, 4, 257, 1030])
@pytest.mark.parametrize("dt,dy,grad", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                        ("f32", "bf16", "f32")])
def test_bwd_channels_and_types(gdr_lib, C, dt, dy, grad):
    check_bwd(gdr_lib, make(2, 37, C, 4, dt, C), 4, True, grad, dy)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("silu", [True, False])
def test_bwd_options(gdr_lib, bias, state, silu):
    check_bwd(gdr_lib, make(4, 25, 40, 3, "f32", 6, bias, state), 3, silu, dsf=state)


def test_bwd_more_stretches_than_workgroup_rows(gdr_lib):
    """So many sequences that a workgroup walks several."""
    check_bwd(gdr_lib, make(1500, 9, 1100, 2, "bf16", 12), 2, True, dsf=False)


def test_bwd_repeats_bit_for_bit_and_empty(gdr_lib):
    i = make(5, 130, 66, 4, "bf16", 14)
    a = [cu(i[k]) for k in ("x", "w", "bias", "s0", "dy", "dsf")]
    one = gdr_lib.gdr_short_conv_bwd(*a)
    two = gdr_lib.gdr_short_conv_bwd(*a)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    e = torch.empty((5, 0, 66), device="cuda", dtype=torch.bfloat16)
    dx, dw, db, ds0 = gdr_lib.gdr_short_conv_bwd(e, a[1], a[2], a[3], e, a[5])
    torch.cuda.synchronize()
    assert dx.shape == e.shape and not dw.any() and not db.any() and torch.equal(ds0, a[5])


@pytest.mark.parametrize("C", [4, 12, 17, 33, 100, 130, 255, 256, 300])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_narrow_rows(gdr_lib, C, dt):
    """Few channels: several stretches of tokens share a wave."""
    i = make(3, 333, C, 4, dt, C)
    check_fwd(gdr_lib, i, 4, True, dt)
    check_bwd(gdr_lib, i, 4, True, dt, dt)
