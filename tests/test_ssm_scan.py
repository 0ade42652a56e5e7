"""GPU parity of gdr_ssm_scan_fwd, gdr_ssm_step and gdr_ssm_scan_bwd with the
fp64 token-by-token form, at the bounds derived in block_reference."""
import numpy as np
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0")


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def make(B, T, D, G, N, dt, seed, gate=True, skip=True, bias=True, state=True, slow=1.0):
    g = rng(seed)

    def t(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return torch.from_numpy((shift + scale * g.standard_normal(shape)).astype(np.float32)
                                ).to(dtype)

    i = dict(x=t(B, T, D, dtype=DT[dt]), dt=t(B, T, D, dtype=DT[dt]),
             A=-torch.exp(t(D, N, scale=0.7)) * slow, Bm=t(B, T, G, N, dtype=DT[dt]),
             Cm=t(B, T, G, N, dtype=DT[dt]), D=t(D) if skip else None,
             z=t(B, T, D, dtype=DT[dt]) if gate else None,
             bias=t(D, shift=-3.0) if bias else None, h0=t(B, D, N) if state else None)
    i["dout"], i["dh"] = t(B, T, D), (t(B, D, N) if state else None)
    return i


KEYS = ("x", "dt", "A", "Bm", "Cm", "D", "z", "bias", "h0")


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
            f"{name}: error {err.max():.3e} (rms {np.sqrt((want ** 2).mean()):.2e}), worst over " \
            f"its bound by {over.max():.3e}"


def check_fwd(gdr, i, out="f32", sp=True):
    y, hf = gdr.gdr_ssm_scan_fwd(*[cu(i[k]) for k in KEYS], softplus=sp, out_dtype=DT[out])
    torch.cuda.synchronize()
    a = [n64(i[k]) for k in KEYS]
    want, wh, _ = R.scan_fwd(*a, sp=sp)
    my, mh, _ = R.scan_fwd(*a, sp=sp, majorant=True)
    T = i["x"].shape[1]
    close("y", y, want, R.scan_bound(my, T, out, want))
    close("h", hf, wh, R.scan_bound(mh, T))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 63, 65, 200, 515])
def test_fwd_lengths(gdr_lib, T):
    check_fwd(gdr_lib, make(2, T, 70, 1, 16, "bf16", T))


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 32, 33, 63, 64])
@pytest.mark.parametrize("T", [11, 150])
def test_fwd_states(gdr_lib, N, T):
    check_fwd(gdr_lib, make(2, T, 37, 1, N, "f32", N))


@pytest.mark.parametrize("D,G", [(1, 1), (3, 3), (64, 1), (65, 1), (130, 2), (300, 4), (259, 7)])
def test_fwd_channels_and_groups(gdr_lib, D, G):
    check_fwd(gdr_lib, make(3, 40, D, G, 16, "bf16", D + G))


@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("opt", [dict(), dict(gate=False), dict(skip=False), dict(bias=False),
                                 dict(state=False)])
def test_fwd_types_and_options(gdr_lib, dt, out, opt):
    check_fwd(gdr_lib, make(2, 77, 66, 1, 12, dt, 1, **opt), out)


def test_fwd_without_softplus(gdr_lib):
    i = make(2, 50, 40, 1, 16, "f32", 2)
    i["dt"], i["bias"] = i["dt"].abs() * 0.1, i["bias"].abs() * 0.01
    check_fwd(gdr_lib, i, sp=False)


def test_fwd_extreme_steps(gdr_lib):
    """Steps that forget everything, steps that underflow, far tails of the
    softplus and of the gate."""
    i = make(2, 90, 64, 1, 16, "f32", 3)
    i["dt"][:, ::3] = 60.0
    i["dt"][:, 1::5] = -110.0
    i["z"][:, ::4] = -120.0
    i["z"][:, 1::4] = 90.0
    check_fwd(gdr_lib, i)


@pytest.mark.parametrize("B,D", [(1, 64), (1, 512), (16, 2048)])
def test_fwd_segments_and_whole_agree(gdr_lib, B, D):
    """Few channels run as segments, many as whole sequences: both against
    the fp64 form on a part, and the states through a cut at an odd place."""
    T = 700 if D < 2048 else 150
    i = make(B, T, D, 1, 16, "bf16", D, slow=0.05)
    need = gdr_lib.gdr_ssm_scan_fwd_workspace_size(B, T, D, 1, 16)
    assert (need > 0) == (D < 2048)
    a = [cu(i[k]) for k in KEYS]
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a, out_dtype=torch.float32)
    cut = 333 if T > 333 else 70
    parts, h = [], a[8].clone()
    for lo, hi in ((0, cut), (cut, T)):
        sl = [x[:, lo:hi] if k in ("x", "dt", "Bm", "Cm", "z") else x for k, x in zip(KEYS, a)]
        parts.append(gdr_lib.gdr_ssm_scan_fwd(*sl[:8], h, h_final=h, out_dtype=torch.float32)[0])
    torch.cuda.synchronize()
    sub = {k: v for k, v in i.items()}
    if B * D > 4000:
        c = torch.arange(5, D, 97)
        for k in ("x", "dt", "z"):
            sub[k] = i[k][:2][..., c]
        for k in ("Bm", "Cm"):
            sub[k] = i[k][:2]
        for k in ("A", "D", "bias"):
            sub[k] = i[k][c]
        sub["h0"] = i["h0"][:2][:, c]
        y, hf = y[:2][..., c], hf[:2][:, c]
        parts, h = [p[:2][..., c] for p in parts], h[:2][:, c]
    ref = [n64(sub[k]) for k in KEYS]
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    for yy, hh in ((y, hf), (torch.cat(parts, 1), h)):
        close("y", yy, want, R.scan_bound(my, T))
        close("h", hh, wh, R.scan_bound(mh, T))


@pytest.mark.parametrize("T", [700, 40])
def test_state_in_place(gdr_lib, T):
    """h_final in h0's buffer gives the same bits, with segments (T 700) too."""
    i = make(1, T, 96, 1, 16, "bf16", 21)
    a = [cu(i[k]) for k in KEYS]
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a)
    h = a[8].clone()
    y2, h2 = gdr_lib.gdr_ssm_scan_fwd(*a[:8], h, h_final=h)
    torch.cuda.synchronize()
    assert h2 is h and torch.equal(y, y2) and torch.equal(hf, h)


def test_empty(gdr_lib):
    i = make(2, 0, 24, 1, 8, "f32", 4)
    a = [cu(i[k]) for k in KEYS]
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a)
    _, hz = gdr_lib.gdr_ssm_scan_fwd(*a[:8])
    g = gdr_lib.gdr_ssm_scan_bwd(*a, cu(i["dout"]), cu(i["dh"]))
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 24) and torch.equal(hf, a[8]) and not hz.any()
    assert not g[2].any() and not g[5].any() and not g[7].any() and torch.equal(g[8], cu(i["dh"]))


def sliced(i):
    """x and z halves of one projection, B and C of another at odd offsets, dt
    with tokens before sequences."""
    B, T, D = i["x"].shape
    G, N = i["Bm"].shape[2:]
    xz = torch.cat([i["x"], i["z"]], -1).cuda()
    bc = torch.cat([i["x"][..., :1], i["Bm"].flatten(2), i["Cm"].flatten(2)], -1).cuda()
    o = {k: cu(v) for k, v in i.items()}
    o["x"], o["z"] = xz[..., :D], xz[..., D:]
    o["Bm"] = bc[..., 1:1 + G * N].unflatten(-1, (G, N))
    o["Cm"] = bc[..., 1 + G * N:].unflatten(-1, (G, N))
    o["dt"] = i["dt"].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    o["dout"] = torch.cat([i["dout"], i["dout"][..., :3]], -1).cuda()[..., :D]
    return o


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_slices(gdr_lib, dt):
    i = make(2, 70, 51, 1, 10, dt, 31)
    a, s = {k: cu(v) for k, v in i.items()}, sliced(i)
    one = gdr_lib.gdr_ssm_scan_fwd(*[a[k] for k in KEYS])
    two = gdr_lib.gdr_ssm_scan_fwd(*[s[k] for k in KEYS])
    g1 = gdr_lib.gdr_ssm_scan_bwd(*[a[k] for k in KEYS], a["dout"], a["dh"])
    g2 = gdr_lib.gdr_ssm_scan_bwd(*[s[k] for k in KEYS], s["dout"], s["dh"])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one + g1, two + g2))


@pytest.mark.parametrize("B,D,G,N", [(1, 1, 1, 1), (3, 70, 1, 16), (5, 66, 2, 7), (2, 40, 1, 33),
                                     (300, 48, 1, 4), (2, 129, 3, 64)])
@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16")])
def test_step(gdr_lib, B, D, G, N, dt, out):
    i = make(B, 1, D, G, N, dt, D + N)
    a = {k: cu(v) for k, v in i.items()}
    h = a["h0"].clone()
    y = gdr_lib.gdr_ssm_step(a["x"][:, 0], a["dt"][:, 0], a["A"], a["Bm"][:, 0], a["Cm"][:, 0], h,
                             a["D"], a["z"][:, 0], a["bias"], out_dtype=DT[out])
    torch.cuda.synchronize()
    ref = [n64(i[k]) for k in KEYS]
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    close("y", y.unsqueeze(1), want, R.scan_bound(my, 1, out, want))
    close("h", h, wh, R.scan_bound(mh, 1))


def test_prompt_then_tokens(gdr_lib):
    """A prompt and then single tokens against the whole sequence."""
    T = 60
    i = make(2, T, 50, 1, 16, "bf16", 41)
    a = {k: cu(v) for k, v in i.items()}
    h = a["h0"].clone()
    cutk = ("x", "dt", "Bm", "Cm", "z")
    got = [gdr_lib.gdr_ssm_scan_fwd(*[a[k][:, :45] if k in cutk else a[k] for k in KEYS[:8]], h,
                                    h_final=h, out_dtype=torch.float32)[0]]
    for t in range(45, T):
        got.append(gdr_lib.gdr_ssm_step(a["x"][:, t], a["dt"][:, t], a["A"], a["Bm"][:, t],
                                        a["Cm"][:, t], h, a["D"], a["z"][:, t], a["bias"],
                                        out_dtype=torch.float32).unsqueeze(1))
    torch.cuda.synchronize()
    ref = [n64(i[k]) for k in KEYS]
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    close("y", torch.cat(got, 1), want, R.scan_bound(my, T))
    close("h", h, wh, R.scan_bound(mh, T))


def check_bwd(gdr, i, dout="f32", grad="f32", sp=True):
    d = i["dout"].to(DT[dout])
    got = gdr.gdr_ssm_scan_bwd(*[cu(i[k]) for k in KEYS], cu(d), cu(i["dh"]), softplus=sp,
                               grad_dtype=DT[grad])
    torch.cuda.synchronize()
    a = [n64(i[k]) for k in KEYS] + [n64(d), n64(i["dh"])]
    want = R.scan_bwd(*a, sp=sp)
    maj = R.scan_bwd(*a, sp=sp, majorant=True)
    B, T, D = i["x"].shape
    gone = {"dD": i["D"], "dz": i["z"], "db": i["bias"]}
    for k, g in zip(NAMES, got):
        if k in gone and gone[k] is None:
            assert g is None
            continue
        # a chain forwards and one backwards; then the sums over channels or tokens
        steps = 2 * T + (D if k in ("dB", "dC") else B * T if k in ("dA", "dD", "db") else 0)
        narrow = k in ("dx", "ddt", "dB", "dC", "dz")
        close(k, g, want[k], R.scan_bound(maj[k], steps, grad if narrow else "f32", want[k]))


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 64, 65, 130, 300])
def test_bwd_lengths(gdr_lib, T):
    check_bwd(gdr_lib, make(2, T, 70, 1, 16, "bf16", T))


@pytest.mark.parametrize("N", [1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 63, 64])
@pytest.mark.parametrize("T", [13, 140])
def test_bwd_states(gdr_lib, N, T):
    check_bwd(gdr_lib, make(2, T, 37, 1, N, "f32", N))


@pytest.mark.parametrize("D,G", [(1, 1), (3, 3), (64, 1), (65, 1), (130, 2), (300, 4), (259, 7)])
def test_bwd_channels_and_groups(gdr_lib, D, G):
    check_bwd(gdr_lib, make(3, 37, D, G, 16, "bf16", D + G))


@pytest.mark.parametrize("dt,dout,grad", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                          ("bf16", "f32", "f32")])
@pytest.mark.parametrize("opt", [dict(), dict(gate=False), dict(skip=False), dict(bias=False),
                                 dict(state=False)])
def test_bwd_types_and_options(gdr_lib, dt, dout, grad, opt):
    check_bwd(gdr_lib, make(2, 77, 66, 1, 12, dt, 1, **opt), dout, grad)


def test_bwd_without_softplus(gdr_lib):
    i = make(2, 50, 40, 1, 16, "f32", 2)
    i["dt"], i["bias"] = i["dt"].abs() * 0.1, i["bias"].abs() * 0.01
    check_bwd(gdr_lib, i, sp=False)


def test_bwd_extreme_steps(gdr_lib):
    i = make(2, 90, 64, 1, 16, "f32", 3)
    i["dt"][:, ::3] = 60.0
    i["dt"][:, 1::5] = -110.0
    i["z"][:, ::4] = -120.0
    i["z"][:, 1::4] = 90.0
    check_bwd(gdr_lib, i)


def test_bwd_long_memory(gdr_lib):
    """States that decay slowly, over many segments."""
    check_bwd(gdr_lib, make(1, 1500, 33, 1, 16, "f32", 5, slow=0.02))


def test_bwd_one_segment(gdr_lib):
    """Enough channels for one segment per sequence: a part against fp64."""
    B, T, D = 16, 70, 2048
    i = make(B, T, D, 1, 16, "bf16", 6)
    got = dict(zip(NAMES, gdr_lib.gdr_ssm_scan_bwd(*[cu(i[k]) for k in KEYS], cu(i["dout"]),
                                                   cu(i["dh"]))))
    torch.cuda.synchronize()
    ref = [n64(i[k][:1] if k in ("x", "dt", "Bm", "Cm", "z", "h0") else i[k]) for k in KEYS]
    ref += [n64(i["dout"][:1]), n64(i["dh"][:1])]
    want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
    for k in ("dx", "ddt", "dz", "dB", "dC", "dh0"):
        steps = 2 * T + (D if k in ("dB", "dC") else 0)
        close(k, got[k][:1], want[k], R.scan_bound(maj[k], steps))


def test_bwd_repeats_bit_for_bit(gdr_lib):
    i = make(2, 300, 200, 1, 16, "bf16", 7)
    a = [cu(i[k]) for k in KEYS] + [cu(i["dout"]), cu(i["dh"])]
    one, two = gdr_lib.gdr_ssm_scan_bwd(*a), gdr_lib.gdr_ssm_scan_bwd(*a)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))


@pytest.mark.parametrize("N,D", [(16, 20), (3, 70), (40, 9)])
def test_many_segments(gdr_lib, N, D):
    """A long sequence of few channels: more segments than one batch of their
    states, forward and backward."""
    i = make(1, 4000, D, 1, N, "f32", N, slow=0.05)
    check_fwd(gdr_lib, i)
    check_bwd(gdr_lib, i)
