"""The operators around the mixer as they are used: one after the other, into
the mixer and its gate, from a prompt into single tokens; captured into graphs
and replayed; on streams and in buffers of the caller's; with padded tokens,
tokens that are not numbers, and offsets past 2^31 elements."""
import numpy as np
import pytest
import torch

import block_reference as R
import oracle

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = {"f32": F32, "bf16": BF}
KEYS = ("x", "dt", "A", "Bm", "Cm", "D", "z", "bias", "h0")


def draw(seed):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, dtype=F32, scale=1.0, shift=0.0):
        return (shift + scale * torch.randn(shape, generator=g)).to(dtype).cuda()

    return t


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(name, got, want, bound):
    err = np.abs(n64(got) - want)
    over = err - bound
    assert got.shape == want.shape and np.isfinite(err).all() and over.max() <= 0, \
        f"{name}: error {err.max():.3e}, worst over its bound by {over.max():.3e}"


def scan_set(seed, B, T, D, G=1, N=16, dt=BF):
    t = draw(seed)
    i = dict(x=t(B, T, D, dtype=dt), dt=t(B, T, D, dtype=dt), A=-torch.exp(t(D, N, scale=0.7)),
             Bm=t(B, T, G, N, dtype=dt), Cm=t(B, T, G, N, dtype=dt), D=t(D),
             z=t(B, T, D, dtype=dt), bias=t(D, shift=-3.0), h0=t(B, D, N))
    return [i[k] for k in KEYS], t(B, T, D, dtype=dt), t(B, D, N)


def scan_fwd_close(i, y, h=None, out="f32"):
    ref = [n64(v) for v in i]
    T = i[0].shape[1]
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    close("y", y, want, R.scan_bound(my, T, out, want))
    if h is not None:
        close("h", h, wh, R.scan_bound(mh, T))


# ---- one after the other ----------------------------------------------------------


def test_norm_conv_delta_rule_gate(gdr_lib):
    """Residual and norm, one projection, the convolution on slices of it, the
    delta rule and its gate: each stage against its fp64 form on the bits that
    the stage before it left."""
    B, T, H, d, C = 2, 130, 2, 64, 200
    t = draw(1)
    x, res, w, b = t(B, T, C, dtype=BF), t(B, T, C), t(C, scale=0.2, shift=1), t(C, scale=0.2)
    y, h = gdr_lib.gdr_layer_norm_fwd(x, w, b, residual=res)
    hr = n64(x.float() + res)
    close("norm", y, R.norm_fwd(hr, n64(w), n64(b), 1e-5),
          R.norm_fwd_bound(hr, n64(w), n64(b), 1e-5, "bf16"))
    wide = (y.float() @ t(C, 4 * H * d + 2 * H, scale=C ** -0.5)).to(BF)
    cw, cb = t(3 * H * d, 4, scale=0.6), t(3 * H * d, scale=0.3)
    u, _ = gdr_lib.gdr_short_conv_fwd(wide[..., :3 * H * d], cw, cb)
    want, _, pre, m = R.conv_fwd(n64(wide[..., :3 * H * d]), n64(cw), n64(cb), None, True)
    close("conv", u, want, R.conv_fwd_bound(want, pre, m, 4, True, "bf16"))
    q, k, v = (s.unflatten(-1, (H, d)).contiguous() for s in u.split(H * d, -1))
    q = torch.nn.functional.normalize(q.float(), dim=-1).to(BF)
    k = torch.nn.functional.normalize(k.float(), dim=-1).to(BF)
    ab = wide[..., 4 * H * d:].float()
    alpha = torch.sigmoid(ab[..., :H] + 3).contiguous()
    beta = torch.sigmoid(ab[..., H:]).contiguous()
    o, s = gdr_lib.gdr_chunk_fwd(q, k, v, alpha, beta, None, out_dtype=F32)
    g = wide[..., 3 * H * d:4 * H * d].reshape(B * T, H, d).contiguous()
    og = gdr_lib.gdr_output_gate(o.reshape(B * T, H, d), g, None, 1e-6, out_dtype=F32)
    torch.cuda.synchronize()
    o_ref, s_ref = oracle.gdn_fwd(*(z.cpu() for z in (q, k, v, alpha, beta)), None)
    assert oracle.err_rms(n64(o), o_ref) <= 2e-2 and oracle.err_rms(n64(s), s_ref) <= 2e-2
    assert og.shape == (B * T, H, d) and torch.isfinite(og).all()


def test_state_space_block_and_its_gradient(gdr_lib):
    """Norm, convolution and scan with their reverse modes, each stage against
    its fp64 form on the bits that it was given."""
    B, T, D, N, C = 2, 75, 52, 16, 52
    t = draw(2)
    x, w, b = t(B, T, C), t(C, scale=0.2, shift=1), t(C, scale=0.2)
    h, wide = gdr_lib.gdr_layer_norm_fwd(x, w, b), t(C, 2 * D + D + 2 * N, scale=C ** -0.5)
    p = h @ wide
    cw, cb = t(D, 4, scale=0.6), t(D, scale=0.3)
    u, _ = gdr_lib.gdr_short_conv_fwd(p[..., :D], cw, cb)
    a = [u, p[..., 2 * D:3 * D], -torch.exp(t(D, N, scale=0.7)),
         p[..., 3 * D:3 * D + N].unsqueeze(2), p[..., 3 * D + N:].unsqueeze(2), t(D),
         p[..., D:2 * D], t(D, shift=-3.0), None]
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a)
    scan_fwd_close(a, y, hf)
    dy = t(B, T, D)
    gs = gdr_lib.gdr_ssm_scan_bwd(*a, dy)
    torch.cuda.synchronize()
    ref = [n64(v) for v in a] + [n64(dy), None]
    want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
    for k, g in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0"), gs):
        steps = 2 * T + (D if k in ("dB", "dC") else B * T if k in ("dA", "dD", "db") else 0)
        close(k, g, want[k], R.scan_bound(maj[k], steps))
    gc = gdr_lib.gdr_short_conv_bwd(p[..., :D], cw, cb, None, gs[0])
    torch.cuda.synchronize()
    cv, bound = R.conv_bwd(n64(p[..., :D]), n64(cw), n64(cb), None, n64(gs[0]), None, True)
    for k, g, v, e in zip(("dx", "dw", "dbias", "ds0"), gc, cv, bound):
        close(k, g, v, e)
    dp = torch.cat([gc[0], gs[6], gs[1], gs[3].squeeze(2), gs[4].squeeze(2)], -1)
    dh = dp @ wide.T
    gn = gdr_lib.gdr_layer_norm_bwd(x, w, dh)
    torch.cuda.synchronize()
    nv, bound = R.norm_bwd(n64(x).reshape(-1, C), n64(w), n64(dh).reshape(-1, C), 1e-5, None)
    for k, g, v, e in zip(("dx", "dw", "db"), gn, nv, bound):
        close(k, g.reshape(v.shape), v, e)


def test_prompt_then_tokens(gdr_lib):
    """A prompt through convolution and scan, then single tokens on the states
    that it left (held in place): the convolution bit for bit, the scan within
    its bound of the whole sequence."""
    B, T, P, D, N = 3, 40, 29, 130, 16
    t = draw(3)
    xz, cw, cb = t(B, T, 2 * D, dtype=BF), t(D, 4, scale=0.6), t(D, scale=0.3)
    full, _, _ = scan_set(4, B, T, D, 2, N)
    u, _ = gdr_lib.gdr_short_conv_fwd(xz[..., :D], cw, cb)
    cs, hs = torch.zeros(B, 3, D, dtype=BF, device="cuda"), full[8].clone()
    up, _ = gdr_lib.gdr_short_conv_fwd(xz[:, :P, :D], cw, cb, cs, s_final=cs)
    cut = (0, 1, 3, 4, 6)
    pr = [v[:, :P] if k in cut else v for k, v in enumerate(full)]
    ys = [gdr_lib.gdr_ssm_scan_fwd(up, *pr[1:8], hs, h_final=hs, out_dtype=F32)[0]]
    us = [up]
    for s in range(P, T):
        us.append(gdr_lib.gdr_short_conv_step(xz[:, s, :D], cw, cb, cs).unsqueeze(1))
        st = [v[:, s] if k in cut else v for k, v in enumerate(full)]
        ys.append(gdr_lib.gdr_ssm_step(us[-1][:, 0], *st[1:5], hs, *st[5:8],
                                       out_dtype=F32).unsqueeze(1))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(us, 1), u)
    scan_fwd_close([u] + full[1:], torch.cat(ys, 1), hs)


# ---- states in place, blocks that share channels ------------------------------------


@pytest.mark.parametrize("B,T,D,G", [(48, 20, 531, 1), (70, 9, 402, 2), (1, 600, 67, 1),
                                     (2, 40, 9, 3)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan_state_in_place_at_odd_widths(gdr_lib, B, T, D, G, dt):
    a, _, _ = scan_set(5, B, T, D, G, 16, DT[dt])
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a)
    h = a[8].clone()
    y2, _ = gdr_lib.gdr_ssm_scan_fwd(*a[:8], h, h_final=h)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(hf, h)


@pytest.mark.parametrize("C", [5, 8, 67, 521, 1030])
def test_conv_state_in_place_at_odd_widths(gdr_lib, C):
    t = draw(6)
    x, w, s0 = t(5, 300, C, dtype=BF), t(C, 4), t(5, 3, C, dtype=BF)
    y, sf = gdr_lib.gdr_short_conv_fwd(x, w, None, s0)
    s = s0.clone()
    y2, _ = gdr_lib.gdr_short_conv_fwd(x, w, None, s, s_final=s)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(sf, s)


@pytest.mark.parametrize("C", [5, 9, 67, 521, 1111, 2055, 8191, 9001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_norm_in_place_at_odd_widths(gdr_lib, C, dt):
    t = draw(7)
    x, r, w = t(33, C, dtype=DT[dt]), t(33, C, dtype=DT[dt]), t(C)
    y, h = gdr_lib.gdr_layer_norm_fwd(x, w, w, residual=r)
    dx, dw, db = gdr_lib.gdr_layer_norm_bwd(h, w, y, dres=x, grad_dtype=DT[dt])
    x2, r2 = x.clone(), r.clone()
    gdr_lib.gdr_layer_norm_fwd(x2, w, w, residual=r2, y=x2, h=r2)
    torch.cuda.synchronize()
    assert torch.equal(y, x2) and torch.equal(h, r2)
    dx2, dw2, db2 = gdr_lib.gdr_layer_norm_bwd(r2, w, x2, dres=x, grad_dtype=DT[dt])
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_rows_behind_the_outputs_stay(gdr_lib):
    """Outputs in the middle of a buffer: what lies before and behind them is
    left as it was, at odd widths too."""
    def inside(*shape, dtype=F32):
        n = int(np.prod(shape))
        buf = torch.full((n + 128,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[64:64 + n].view(shape)

    a, _, _ = scan_set(8, 2, 150, 77, 1, 13)
    by, y = inside(2, 150, 77, dtype=BF)
    bh, h = inside(2, 77, 13)
    gdr_lib.gdr_ssm_scan_fwd(*a, y=y, h_final=h)
    t = draw(9)
    bc, yc = inside(2, 150, 77, dtype=BF)
    bs, sf = inside(2, 3, 77, dtype=BF)
    gdr_lib.gdr_short_conv_fwd(a[0], t(77, 4), y=yc, s_final=sf)
    bn, yn = inside(300, 77, dtype=BF)
    br, hn = inside(300, 77, dtype=BF)
    gdr_lib.gdr_layer_norm_fwd(a[0].view(300, 77), residual=a[6].view(300, 77), y=yn, h=hn)
    torch.cuda.synchronize()
    for buf in (by, bh, bc, bs, bn, br):
        assert (buf[:64] == 7).all() and (buf[-64:] == 7).all()


# ---- graphs, streams, workspaces ------------------------------------------------------


def _everything(gdr, B, T, D, N, seed):
    """A function that runs every call on fixed inputs and returns its outputs."""
    a, do, dh = scan_set(seed, B, T, D, 1, N)
    t = draw(seed + 50)
    cw, cb, s0, ds = t(D, 4, scale=0.6), t(D), t(B, 3, D, dtype=BF), t(B, 3, D)
    w, b = t(D), t(D)
    h, cs = torch.empty_like(a[8]), torch.empty_like(s0)

    def run():
        y, hf = gdr.gdr_ssm_scan_fwd(*a)
        g = gdr.gdr_ssm_scan_bwd(*a, do, dh)
        h.copy_(a[8])
        cs.copy_(s0)
        st = [v[:, 0] if v is not None and v.dim() > 2 and k in (0, 1, 3, 4, 6) else v
              for k, v in enumerate(a)]
        ys = gdr.gdr_ssm_step(*st[:5], h, *st[5:8])
        c, sf = gdr.gdr_short_conv_fwd(a[0], cw, cb, s0)
        ct = gdr.gdr_short_conv_step(st[0], cw, cb, cs)
        gc = gdr.gdr_short_conv_bwd(a[0], cw, cb, s0, do, ds)
        n, hn = gdr.gdr_layer_norm_fwd(c, w, b, residual=a[6])
        gn = gdr.gdr_layer_norm_bwd(hn, w, do, dres=g[0])
        return (y, hf, *g, h, ys, c, sf, ct, cs, *gc, n, hn, *gn)

    return run


@pytest.mark.parametrize("B,T,D,N", [(2, 300, 96, 16), (3, 170, 131, 5)])
def test_graph_of_every_call(gdr_lib, B, T, D, N):
    """Captured once, replayed with eager work of the same calls between the
    replays: equal bits every time (the scan runs as segments here)."""
    assert gdr_lib.gdr_ssm_scan_fwd_workspace_size(B, T, D, 1, N) > 0
    run = _everything(gdr_lib, B, T, D, N, 10)
    other = _everything(gdr_lib, B, T + 3, D, N, 11)
    eager = [v.clone() for v in run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for i in range(4):
        other()
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for j, (p, q) in enumerate(zip(outs, eager)):
            assert torch.equal(p, q), f"replay {i} output {j} differs"


def test_two_graphs_share_a_workspace(gdr_lib):
    """A workspace of the caller's that both graphs (and eager calls between
    them) write: nothing is kept in it from one call for the next."""
    a, do, dh = scan_set(12, 1, 400, 80)
    b, eo, eh = scan_set(13, 2, 210, 72, 1, 9)
    n = max(gdr_lib.gdr_ssm_scan_bwd_workspace_size(*s) for s in ((1, 400, 80, 1, 16),
                                                                   (2, 210, 72, 1, 9)))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def one(i, d, e):
        return (*gdr_lib.gdr_ssm_scan_fwd(*i, workspace=ws),
                *gdr_lib.gdr_ssm_scan_bwd(*i, d, e, workspace=ws))

    sets = ((a, do, dh), (b, eo, eh))
    want = [[v.clone() for v in one(*s)] for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = one(*s)
        graphs.append((g, outs))
    for i in range(4):
        for k in (0, 1) if i % 2 else (1, 0):
            ws.fill_(255)
            graphs[k][0].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(graphs[k][1], want[k])), (i, k)
        one(*sets[i % 2])
        torch.cuda.synchronize()


def test_streams(gdr_lib):
    """On a stream of the caller's, given or current, behind work that writes
    the inputs there; and two calls at once on two streams."""
    run = _everything(gdr_lib, 2, 120, 100, 16, 14)
    want = [v.clone() for v in run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    a, do, dh = scan_set(15, 2, 500, 100)
    yw = gdr_lib.gdr_ssm_scan_fwd(*a)[0].clone()
    gw = [v.clone() for v in gdr_lib.gdr_ssm_scan_bwd(*a, do, dh)]
    late = [torch.zeros_like(a[0]), *a[1:]]
    torch.cuda.synchronize()
    s2 = torch.cuda.Stream()
    with torch.cuda.stream(s):
        junk = torch.randn(1 << 24, device="cuda").sort()
        late[0].copy_(a[0])
    y = gdr_lib.gdr_ssm_scan_fwd(*late, stream=s)[0]
    g = gdr_lib.gdr_ssm_scan_bwd(*a, do, dh, stream=s2)
    torch.cuda.synchronize()
    del junk
    assert torch.equal(y, yw) and all(torch.equal(p, q) for p, q in zip(g, gw))


# ---- padded tokens, values that are not numbers ------------------------------------------


@pytest.mark.parametrize("pad", [float("-inf"), torch.finfo(BF).min])
@pytest.mark.parametrize("T", [60, 700])
def test_padded_tokens_leave_the_state(gdr_lib, pad, T):
    """dt at minus infinity, or the type's lowest value, is a step of 0: the
    state passes the token unchanged, and no gradient enters through it."""
    a, do, dh = scan_set(16, 3, T, 70)
    keep = torch.ones(3, T, dtype=torch.bool, device="cuda")
    keep[0, 40:] = False                 # behind the sequence
    keep[1, :17] = False                 # before it
    keep[2] = False                      # nothing left
    a[1][~keep] = pad
    do[~keep] = 0
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a, out_dtype=F32)
    g = gdr_lib.gdr_ssm_scan_bwd(*a, do, dh)
    torch.cuda.synchronize()
    assert torch.equal(hf[2], a[8][2]) and torch.equal(g[8][2], dh[2])
    for v in (g[0], g[1], g[3]):
        assert not v[~keep].any()
    for b, sl in ((0, slice(0, 40)), (1, slice(17, T))):
        part = [v[b:b + 1, sl] if k in (0, 1, 3, 4, 6) else v[b:b + 1] if k == 8 else v
                for k, v in enumerate(a)]
        scan_fwd_close(part, y[b:b + 1, sl], hf[b:b + 1])
        ref = [n64(v) for v in part] + [n64(do[b:b + 1, sl]), n64(dh[b:b + 1])]
        want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
        for name, j in (("dx", 0), ("ddt", 1), ("dB", 3), ("dC", 4), ("dz", 6)):
            close(name, g[j][b:b + 1, sl], want[name],
                  R.scan_bound(maj[name], 2 * T + (70 if name in ("dB", "dC") else 0)))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_channel(gdr_lib, bad):
    """One value that is no number: other sequences and channels, and the tokens
    before it, keep their bits."""
    B, T, D, ch, tk = 3, 90, 77, 40, 33
    a, do, _ = scan_set(17, B, T, D)
    t = draw(18)
    cw, w = t(D, 4), t(D)
    y = gdr_lib.gdr_ssm_scan_fwd(*a)[0].clone()
    gx = gdr_lib.gdr_ssm_scan_bwd(*a, do)[0].clone()
    c = gdr_lib.gdr_short_conv_fwd(a[0], cw)[0].clone()
    n = gdr_lib.gdr_layer_norm_fwd(a[0], w).clone()
    a[0][1, tk, ch] = bad
    y2 = gdr_lib.gdr_ssm_scan_fwd(*a)[0]
    gx2 = gdr_lib.gdr_ssm_scan_bwd(*a, do)[0]
    c2 = gdr_lib.gdr_short_conv_fwd(a[0], cw)[0]
    n2 = gdr_lib.gdr_layer_norm_fwd(a[0], w)
    torch.cuda.synchronize()
    hit = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    hit[1, tk:, ch] = True
    assert torch.equal(y[~hit], y2[~hit]) and not torch.isfinite(y2[1, tk, ch])
    col = torch.zeros_like(hit)
    col[1, :, ch] = True
    assert torch.equal(gx[~col], gx2[~col])
    hit[1, tk + 4:, ch] = False
    assert torch.equal(c[~hit], c2[~hit]) and not torch.isfinite(c2[1, tk, ch])
    row = torch.zeros_like(hit)
    row[1, tk] = True
    assert torch.equal(n[~row], n2[~row]) and torch.isnan(n2[1, tk]).all()


# ---- arguments through the binding ------------------------------------------------------------


def test_binding_refuses(gdr_lib):
    a, do, dh = scan_set(19, 2, 10, 24)
    g = gdr_lib
    x, w = a[0], torch.zeros(24, 4, device="cuda")
    with pytest.raises(ValueError):
        g.gdr_ssm_scan_fwd(x.cpu(), *a[1:])
    with pytest.raises(TypeError):
        g.gdr_ssm_scan_fwd(x.float(), *a[1:])
    with pytest.raises(TypeError):
        g.gdr_ssm_scan_fwd(x.half(), *a[1:])
    with pytest.raises(ValueError):
        g.gdr_ssm_scan_fwd(*a[:3], a[3][..., :8], *a[4:])
    with pytest.raises(ValueError):
        g.gdr_ssm_scan_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), *a[1:])
    with pytest.raises(ValueError):
        g.gdr_ssm_scan_fwd(*a[:8], a[8][:1])
    with pytest.raises(TypeError):
        g.gdr_ssm_scan_fwd(*a, y=torch.empty_like(x), out_dtype=F32)
    with pytest.raises(ValueError):
        g.gdr_ssm_scan_bwd(*a, do[:, :5])
    with pytest.raises(ValueError):
        g.gdr_ssm_scan_bwd(*a, do, dh.transpose(1, 2))
    with pytest.raises(TypeError):
        g.gdr_ssm_scan_bwd(*a, do, grad_dtype=torch.float16)
    with pytest.raises(ValueError):
        g.gdr_short_conv_fwd(x, w[:20])
    with pytest.raises(ValueError):
        g.gdr_short_conv_fwd(x, w, s0=torch.zeros(2, 4, 24, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        g.gdr_layer_norm_fwd(x, w[:, 0])
    with pytest.raises(ValueError):
        g.gdr_layer_norm_fwd(x, h=torch.empty_like(x))
    with pytest.raises(RuntimeError):
        g.gdr_short_conv_fwd(x, w, y=x)
    with pytest.raises(RuntimeError):
        g.gdr_ssm_scan_fwd(*a, y=a[6])
    with pytest.raises(RuntimeError):
        g.gdr_ssm_scan_bwd(*a, do, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError):
        g.gdr_short_conv_fwd(x, torch.zeros(24, 5, device="cuda"))


# ---- offsets past 2^31 elements -----------------------------------------------------------------


@pytest.fixture(scope="module")
def wide():
    """One buffer of 2.2e9 bf16 elements that the tests below view."""
    buf = torch.empty(2101 << 20, dtype=BF, device="cuda")
    step = 1 << 28
    for i in range(0, buf.numel(), step):
        buf[i:i + step].normal_()
    return buf


def test_conv_past_2_31(gdr_lib, wide):
    T, C = wide.numel() // 8192, 8192
    x = wide[:T * C].view(1, T, C)
    t = draw(20)
    w, b = t(C, 4, scale=0.6), t(C)
    y, _ = gdr_lib.gdr_short_conv_fwd(x, w, b)
    dx, dw, db, _ = gdr_lib.gdr_short_conv_bwd(x, w, b, None, y, grad_dtype=BF)
    torch.cuda.synchronize()
    for lo in (0, T // 2, T - 9):
        i = x[:, max(lo - 3, 0):lo + 9]
        skip = lo - max(lo - 3, 0)
        want, _, u, m = R.conv_fwd(n64(i), n64(w), n64(b), None, True)
        bound = R.conv_fwd_bound(want, u, m, 4, True, "bf16")
        close("y", y[:, lo:lo + 9], want[:, skip:], bound[:, skip:])
    i, dy = x[:, T - 12:], y[:, T - 12:]
    want, bound = R.conv_bwd(n64(i), n64(w), n64(b), None, n64(dy), None, True)
    bound[0] = bound[0] + R.HALF["bf16"] * (np.abs(want[0]) + bound[0])
    close("dx", dx[:, T - 8:], want[0][:, 4:], bound[0][:, 4:])


def test_norm_past_2_31(gdr_lib, wide):
    C = 4096
    x = wide.view(-1, C)
    t = draw(21)
    w, b = t(C), t(C)
    y, h = gdr_lib.gdr_layer_norm_fwd(x, w, b, residual=x)
    dx, _, _ = gdr_lib.gdr_layer_norm_bwd(h, w, y, grad_dtype=BF)
    torch.cuda.synchronize()
    for r in (0, x.shape[0] // 2, x.shape[0] - 2):
        i = n64((2 * x[r:r + 2].float()).to(BF))
        close("y", y[r:r + 2], R.norm_fwd(i, n64(w), n64(b), 1e-5),
              R.norm_fwd_bound(i, n64(w), n64(b), 1e-5, "bf16"))
        want, bound = R.norm_bwd(i, n64(w), n64(y[r:r + 2]), 1e-5, None)
        close("dx", dx[r:r + 2], want[0], bound[0] + R.HALF["bf16"] * (np.abs(want[0]) + bound[0]))


def test_scan_strides_past_2_31(gdr_lib, wide):
    """Channel slices of rows 2^20 apart, whose last rows lie past 2^31."""
    B, T, D, N = 1, 2100, 70, 16
    rows = wide.view(1, -1, 1 << 20)[:, :T]
    t = draw(22)
    cols = [rows[..., k * 100003:][..., :n] for k, n in enumerate((D, D, N, N, D, D))]
    a = [cols[0], cols[1], -torch.exp(t(D, N, scale=0.7)), cols[2].unsqueeze(2),
         cols[3].unsqueeze(2), t(D), cols[4], t(D, shift=-3.0), None]
    y, hf = gdr_lib.gdr_ssm_scan_fwd(*a, out_dtype=F32)
    g = gdr_lib.gdr_ssm_scan_bwd(*a, cols[5])
    torch.cuda.synchronize()
    scan_fwd_close(a, y, hf)
    ref = [n64(v) for v in a] + [n64(cols[5]), None]
    want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
    for name, j in (("dx", 0), ("ddt", 1), ("dB", 3), ("dC", 4), ("dz", 6)):
        close(name, g[j], want[name],
              R.scan_bound(maj[name], 2 * T + (D if name in ("dB", "dC") else 0)))


def test_scan_states_past_2_31(gdr_lib):
    """So many tokens and states that the kept states take more than 2^31 floats
    of the workspace: channels of the first and last sequence against fp64."""
    B, T, D, N = 16, 4128, 8192, 64
    assert gdr_lib.gdr_ssm_scan_bwd_workspace_size(B, T, D, 1, N) > 4 * 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(23)

    def big(*s, dtype=BF):
        return torch.empty(s, dtype=dtype, device="cuda").normal_(generator=g)

    t = draw(24)
    a = [big(B, T, D), big(B, T, D), -torch.exp(t(D, N, scale=0.7)), big(B, T, 1, N),
         big(B, T, 1, N), t(D), None, t(D, shift=-3.0), None]
    do = big(B, T, D)
    y, _ = gdr_lib.gdr_ssm_scan_fwd(*a)
    gr = gdr_lib.gdr_ssm_scan_bwd(*a, do, grad_dtype=BF)
    torch.cuda.synchronize()
    c = torch.tensor([0, 77, D - 1], device="cuda")
    for b in (0, B - 1):
        part = [v[b:b + 1][..., c] if k < 2 else v[c] if k in (2, 5, 7) else
                v[b:b + 1] if v is not None else None for k, v in enumerate(a)]
        ref = [n64(v) for v in part]
        want, _, _ = R.scan_fwd(*ref)
        maj, _, _ = R.scan_fwd(*ref, majorant=True)
        close("y", y[b:b + 1][..., c], want, R.scan_bound(maj, T, "bf16", want))
        ref += [n64(do[b:b + 1][..., c]), None]
        want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
        for name, j in (("dx", 0), ("ddt", 1)):
            close(name, gr[j][b:b + 1][..., c], want[name],
                  R.scan_bound(maj[name], 2 * T, "bf16", want[name]))
