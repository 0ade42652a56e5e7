"""GPU parity of gdr_linear_attn_fwd, _step and _bwd with the fp64 forms, at the
bounds derived in linear_reference."""
import numpy as np
import pytest
import torch

import linear_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = {"f32": F32, "bf16": BF}


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(name, got, want, bound):
    got = n64(got)
    assert got.shape == want.shape, name
    over = np.abs(got - want) - bound
    assert np.isfinite(got).all() and (got.size == 0 or over.max() <= 0), \
        f"{name}: error {np.abs(got - want).max():.3e}, worst over its bound by {over.max():.3e}"


def make(seed, B, T, H, Hk, Dk, Dv, dt="bf16", decay="token", state=True, reset=0.0):
    """Inputs on the GPU, q, k and v as slices of one projection."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((B, T, 2 * Hk * Dk + H * Dv), generator=g).to(DT[dt]).cuda()
    q = wide[..., :Hk * Dk].unflatten(-1, (Hk, Dk))
    k = wide[..., Hk * Dk:2 * Hk * Dk].unflatten(-1, (Hk, Dk))
    v = wide[..., 2 * Hk * Dk:].unflatten(-1, (H, Dv))
    d = None
    if decay == "head":
        d = -torch.exp(torch.randn(H, generator=g) - 2).cuda()
    elif decay == "token":
        d = -torch.exp(1.5 * torch.randn((B, T, H), generator=g) - 2)
        d[torch.rand((B, T, H), generator=g) < reset] = float("-inf")
        d = d.cuda()
    s0 = torch.randn((B, H, Dv, Dk), generator=g).cuda() if state else None
    do = torch.randn((B, T, H, Dv), generator=g).to(DT[dt]).cuda()
    ds = torch.randn((B, H, Dv, Dk), generator=g).cuda() if state else None
    return [q, k, v, d, s0], do, ds


def check_fwd(gdr, a, scale=0.3, out="f32", **kw):
    o, s = gdr.gdr_linear_attn_fwd(*a, scale=scale, out_dtype=DT[out], **kw)
    torch.cuda.synchronize()
    B, T, H, Dv = a[2].shape
    Dk = a[0].shape[-1]
    (ow, sw), (mo, ms), (do, ds) = R.la_fwd(*[n64(x) for x in a], scale)
    close("o", o, ow, R.la_bound(ow, mo, do, T, Dk, Dv, out))
    close("s", s, sw, R.la_bound(sw, ms, ds, T, Dk, Dv))
    return o, s


def check_bwd(gdr, a, do, ds, scale=0.3, grad="f32", **kw):
    got = gdr.gdr_linear_attn_bwd(*a, do, ds, scale=scale, grad_dtype=DT[grad], **kw)
    torch.cuda.synchronize()
    B, T, H, Dv = a[2].shape
    Hk, Dk = a[0].shape[2:]
    r = R.la_bwd(*[n64(x) for x in a], n64(do), n64(ds), scale)
    for n, x in zip(("dq", "dk", "dv"), got):
        close(n, x, r[0][n], R.la_bound(r[0][n], r[1][n], r[2][n], T, Dk, Dv, grad, H // Hk))
    close("ds0", got[4], r[0]["ds0"], R.la_bound(r[0]["ds0"], r[1]["ds0"], r[2]["ds0"], T, Dk, Dv))
    if a[3] is None:
        assert got[3] is None
    else:
        b = R.la_dg_bound(r, T, Dk, Dv)
        if a[3].dim() == 1:
            close("dg", got[3], r[0]["dg"].sum((0, 1)), b.sum((0, 1)))
        else:
            close("dg", got[3], r[0]["dg"], b)
    return got


# lengths about a chunk (64 tokens, 32 in fp32), its tiles and several of them
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_lengths(gdr_lib, T, dt):
    a, do, ds = make(T, 2, T, 2, 2, 64, 64, dt)
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)


@pytest.mark.parametrize("Dk,Dv", [(8, 8), (16, 128), (128, 8), (72, 40), (40, 72), (104, 56),
                                   (128, 128), (64, 128), (128, 64), (24, 120)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_head_sizes(gdr_lib, Dk, Dv, dt):
    a, do, ds = make(Dk + Dv, 2, 70, 3, 1, Dk, Dv, dt)
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (6, 2), (5, 5), (8, 1)])
@pytest.mark.parametrize("decay", ["token", "head", "none"])
@pytest.mark.parametrize("state", [True, False])
def test_heads_decays_states(gdr_lib, H, Hk, decay, state):
    a, do, ds = make(H, 3, 90, H, Hk, 32, 48, "bf16", decay, state)
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_types(gdr_lib, dt, out):
    a, do, ds = make(7, 2, 100, 4, 2, 64, 72, dt)
    o, s = check_fwd(gdr_lib, a, out=out)
    g = check_bwd(gdr_lib, a, do, ds, grad=out)
    assert o.dtype == DT[out] and g[0].dtype == g[1].dtype == g[2].dtype == DT[out]
    assert s.dtype == g[3].dtype == g[4].dtype == F32


# enough tokens for segments side by side, and (from 1025 on) kept states inside them
@pytest.mark.parametrize("B,T,H,Dk,Dv", [(1, 512, 1, 64, 64), (1, 777, 2, 40, 128),
                                         (2, 1100, 1, 128, 64), (1, 2100, 1, 64, 64)])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_segments(gdr_lib, B, T, H, Dk, Dv, decay, dt):
    assert gdr_lib.gdr_linear_attn_fwd_workspace_size(B, T, H, Dk, Dv, DT[dt]) > 0
    a, do, ds = make(T, B, T, H, H, Dk, Dv, dt, decay, reset=0.002)
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)
    a[4] = None
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, None)


def test_kept_states_of_one_segment(gdr_lib):
    """Enough heads that a sequence is one segment, longer than 1024 tokens."""
    a, do, ds = make(3, 16, 1300, 16, 16, 16, 16, "bf16", reset=0.002)
    assert gdr_lib.gdr_linear_attn_fwd_workspace_size(16, 1300, 16, 16, 16, BF) == 0
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)


@pytest.mark.parametrize("B,T,H,Hk,Dk,Dv", [(2, 2300, 1, 1, 128, 64), (130, 2100, 1, 1, 8, 72),
                                            (43, 3200, 3, 1, 8, 16)])
@pytest.mark.parametrize("decay", ["token", "none"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_from_kept_states(gdr_lib, B, T, H, Hk, Dk, Dv, decay, dt):
    """dv in a launch of its own, in segments that start from the states that dk's
    chain has left, with and without a decay's gradient."""
    a, do, ds = make(8, B, T, H, Hk, Dk, Dv, dt, decay, state=B < 100)
    want = check_bwd(gdr_lib, a, do, ds)
    got = gdr_lib.gdr_linear_attn_bwd(*a, do, ds, scale=0.3, want_ddecay=False, want_ds0=False)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got[:3], want[:3]))
    if dt == "bf16" and decay == "none":        # products in fewer terms
        check_bwd(gdr_lib, a, do, ds, grad=dt)


@pytest.mark.parametrize("reset", [0.02, 0.3, 1.0])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_resets(gdr_lib, reset, dt):
    """Minus infinity forgets what was before, exactly: the same as separate calls;
    its own gradient is 0, and the tokens after it keep their precision."""
    a, do, ds = make(5, 2, 150, 2, 2, 64, 64, dt, reset=reset)
    o, s = check_fwd(gdr_lib, a)
    g = check_bwd(gdr_lib, a, do, ds)
    assert not g[3][a[3] == float("-inf")].any()
    if reset == 1.0:
        assert not g[4].any() and not g[3].any()


@pytest.mark.parametrize("low", [-1e38, torch.finfo(F32).min, -2e4, -200.0, -60.0])
def test_decays_far_below(gdr_lib, low):
    """Every third token forgets almost, or wholly; sums of such exponents lose none
    of the others' precision."""
    a, do, ds = make(6, 1, 140, 2, 2, 64, 64, "bf16")
    a[3][:, ::3] = low
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)


def test_packed_documents_are_separate(gdr_lib):
    a, do, _ = make(8, 1, 300, 2, 2, 64, 64, "bf16", state=False)
    cuts = [0, 70, 71, 200, 300]
    for c in cuts[1:-1]:
        a[3][:, c] = float("-inf")
    o, s = gdr_lib.gdr_linear_attn_fwd(*a, out_dtype=F32)
    g = gdr_lib.gdr_linear_attn_bwd(*a, do)
    for lo, hi in zip(cuts, cuts[1:]):
        one = [x[:, lo:hi] for x in a[:4]] + [None]
        one[3] = one[3].contiguous()
        check_fwd(gdr_lib, one)
        (ow, _), (mo, _), (dm, _) = R.la_fwd(*[n64(x) for x in one], 1.0)
        close("o", o[:, lo:hi], ow, R.la_bound(ow, mo, dm, 300, 64, 64))
        r = R.la_bwd(*[n64(x) for x in one], n64(do[:, lo:hi]), None, 1.0)
        for n, x in zip(("dq", "dk", "dv"), g):
            close(n, x[:, lo:hi], r[0][n], R.la_bound(r[0][n], r[1][n], r[2][n], 300, 64, 64))
    torch.cuda.synchronize()


# ---- one token ----------------------------------------------------------------------


@pytest.mark.parametrize("Dk,Dv", [(8, 8), (64, 64), (128, 128), (72, 40), (40, 104), (16, 72)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["token", "head", "none"])
def test_step(gdr_lib, Dk, Dv, dt, decay):
    a, _, _ = make(Dk, 5, 1, 6, 3, Dk, Dv, dt, decay)
    want = R.la_fwd(*[n64(x) for x in a], 0.3)
    st = a[4].clone()
    g = a[3][:, 0].contiguous() if decay == "token" else a[3]
    o = gdr_lib.gdr_linear_attn_step(a[0][:, 0], a[1][:, 0], a[2][:, 0], g, st, scale=0.3,
                                     out_dtype=F32)
    torch.cuda.synchronize()
    (ow, sw), (mo, ms), (do, ds) = want
    close("o", o, ow[:, 0], R.la_bound(ow, mo, do, 1, Dk, Dv)[:, 0])
    close("s", st, sw, R.la_bound(sw, ms, ds, 1, Dk, Dv))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_prompt_then_tokens(gdr_lib, dt):
    """A prompt, then single tokens on the state that it left (held in place): the
    whole sequence."""
    T, P = 90, 77
    a, _, _ = make(9, 3, T, 4, 2, 64, 64, dt, reset=0.05)
    st = a[4].clone()
    pre = [x[:, :P] for x in a[:4]]
    pre[3] = pre[3].contiguous()
    outs = [gdr_lib.gdr_linear_attn_fwd(*pre, st, s_final=st, out_dtype=F32)[0]]
    for t in range(P, T):
        outs.append(gdr_lib.gdr_linear_attn_step(
            *[x[:, t] for x in a[:3]], a[3][:, t].contiguous(), st, out_dtype=F32).unsqueeze(1))
    torch.cuda.synchronize()
    (ow, sw), (mo, ms), (do, ds) = R.la_fwd(*[n64(x) for x in a], 1.0)
    close("o", torch.cat(outs, 1), ow, R.la_bound(ow, mo, do, T, 64, 64))
    close("s", st, sw, R.la_bound(sw, ms, ds, T, 64, 64))


# ---- gradients by differences -----------------------------------------------------------


def test_gradients_by_differences(gdr_lib):
    """The fp32 backward against central differences of the fp32 forward, along one
    direction per input.  A step h errs by h^2 / 6 times the third derivative (the
    loss is cubic in all and linear in each of q, k, v, s0, so 0 there; for g the
    moments of |g| <= 1 over 40 tokens, below 40^2 of the value) and by the forward's
    bound over h."""
    a, do, ds = make(21, 1, 40, 2, 1, 16, 24, "f32")
    a = [x.contiguous() for x in a]
    a[3].clamp_(min=-1)
    got = gdr_lib.gdr_linear_attn_bwd(*a, do, ds)
    ref = [n64(x) for x in a]
    (ow, sw), (mo, ms), (dmo, dms) = R.la_fwd(*ref, 1.0)
    noise = (R.la_bound(ow, mo, dmo, 40, 16, 24) * np.abs(n64(do))).sum() + \
        (R.la_bound(sw, ms, dms, 40, 16, 24) * np.abs(n64(ds))).sum()
    major = (mo * np.abs(n64(do))).sum() + (ms * np.abs(n64(ds))).sum()
    g = torch.Generator().manual_seed(22)
    for i, name in enumerate(("q", "k", "v", "g", "s0")):
        d = torch.randn(a[i].shape, generator=g).cuda()
        h = 2.0 ** -6

        def loss(sign):
            b = list(a)
            b[i] = a[i] + sign * h * d
            o, s = gdr_lib.gdr_linear_attn_fwd(*b)
            return ((o.double() * do.double()).sum() + (s.double() * ds.double()).sum()).item()

        diff = (loss(1) - loss(-1)) / (2 * h)
        val = (n64(got[i]) * n64(d)).sum()
        lim = 2 * noise / h + (h * h / 6 * 1600 * 8 * major if name == "g" else 0.0)
        assert abs(diff - val) <= lim, (name, diff, val, lim)


# ---- values that are not numbers --------------------------------------------------------


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bad_values_reach_no_token_before(gdr_lib, bad, dt):
    """One value that is no number in v, q or k: other sequences and heads, and the
    tokens before it, are what they were."""
    a, _, _ = make(31, 2, 150, 2, 2, 64, 64, dt)
    want = check_fwd(gdr_lib, a)[0]
    (ow, _), (mo, _), (dm, _) = R.la_fwd(*[n64(x) for x in a], 0.3)
    lim = R.la_bound(ow, mo, dm, 150, 64, 64)
    for i in range(3):
        b = [x.clone() for x in a]
        b[i][1, 77, 0, 5] = bad
        o, s = gdr_lib.gdr_linear_attn_fwd(*b, scale=0.3, out_dtype=F32)
        torch.cuda.synchronize()
        keep = torch.ones_like(o, dtype=torch.bool)
        keep[1, 77:, 0] = False
        assert torch.isfinite(o[keep]).all()
        assert (np.abs(n64(o) - ow)[keep.cpu().numpy()] <= lim[keep.cpu().numpy()]).all()
        assert torch.equal(o[0], want[0]) and torch.equal(o[1, :, 1], want[1, :, 1])
        assert not torch.isfinite(o[1, 77, 0]).all()
        assert torch.isfinite(s[0]).all() and torch.isfinite(s[1, 1]).all()


def test_large_values_in_masked_pairs(gdr_lib):
    """Products of later tokens that overflow are never formed into a result."""
    a, _, _ = make(32, 1, 64, 1, 1, 64, 64, "f32", state=False)
    a = [x.contiguous() if x is not None else None for x in a]
    a[1][:, 40:] = 3e38
    a[0][:, :40] = a[0][:, :40].abs() + 1
    o, _ = gdr_lib.gdr_linear_attn_fwd(*a)
    torch.cuda.synchronize()
    part = [x[:, :40].contiguous() if x is not None else None for x in a]
    (ow, _), (mo, _), (dm, _) = R.la_fwd(*[n64(x) for x in part], 1.0)
    close("o", o[:, :40], ow, R.la_bound(ow, mo, dm, 64, 64, 64))


# ---- many heads, many sequences, a decay per head over several blocks ---------------------


@pytest.mark.parametrize("B,T,H,Hk,Dk,Dv", [(1, 5, 2048, 1, 8, 8), (3000, 2, 1, 1, 8, 16),
                                            (2, 70, 96, 3, 16, 8)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_heads_or_sequences(gdr_lib, B, T, H, Hk, Dk, Dv, dt):
    a, do, ds = make(41, B, T, H, Hk, Dk, Dv, dt)
    check_fwd(gdr_lib, a)
    check_bwd(gdr_lib, a, do, ds)


@pytest.mark.parametrize("B,T,Dk,Dv", [(130, 700, 8, 8), (2, 1500, 16, 72), (1, 515, 64, 64)])
@pytest.mark.parametrize("state", ["none", "start", "both"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_decay_per_head_over_blocks(gdr_lib, B, T, Dk, Dv, state, dt):
    """The sums over blocks of tokens, with and without states at either end."""
    a, do, ds = make(42, B, T, 1, 1, Dk, Dv, dt, "head", state=state != "none")
    check_bwd(gdr_lib, a, do, ds if state == "both" else None)


def test_sum_per_head_is_as_exact_as_its_tokens(gdr_lib):
    """A decay per head is the same call with the decay of every token; its gradient is
    the sum of theirs.  Both err by at most the bound of one of them."""
    a, do, _ = make(43, 2, 1300, 2, 2, 64, 64, "f32", "head", state=False)
    b = list(a)
    b[3] = a[3].expand(2, 1300, 2).contiguous()
    one = gdr_lib.gdr_linear_attn_bwd(*a, do, scale=0.3)
    all_ = gdr_lib.gdr_linear_attn_bwd(*b, do, scale=0.3)
    torch.cuda.synchronize()
    r = R.la_bwd(*[n64(x) for x in b], n64(do), None, 0.3)
    bound = R.la_dg_bound(r, 1300, 64, 64).sum((0, 1))
    close("dg", one[3], r[0]["dg"].sum((0, 1)), bound)
    close("sum", all_[3].double().sum((0, 1)), r[0]["dg"].sum((0, 1)), bound)
    for x, y, n in zip(one[:3], all_[:3], ("dq", "dk", "dv")):
        close(n, x, r[0][n], R.la_bound(r[0][n], r[1][n], r[2][n], 1300, 64, 64))
        close(n, y, r[0][n], R.la_bound(r[0][n], r[1][n], r[2][n], 1300, 64, 64))
