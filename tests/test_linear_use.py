"""Linear attention, rotary positions and RMS norm as they are used: one after the
other into the output gate and back, from a prompt into single tokens; captured into
graphs and replayed; on streams and in buffers of the caller's; with padded tokens,
shared and broadcast inputs, and offsets past 2^31 elements."""
import numpy as np
import pytest
import torch

import linear_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = {"f32": F32, "bf16": BF}


def draw(seed):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, dtype=F32, scale=1.0, shift=0.0):
        return (shift + scale * torch.randn(shape, generator=g)).to(dtype).cuda()

    return t


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(name, got, want, bound):
    got = n64(got)
    assert got.shape == want.shape, name
    over = np.abs(got - want) - bound
    assert np.isfinite(got).all() and over.max() <= 0, \
        f"{name}: error {np.abs(got - want).max():.3e}, worst over its bound by {over.max():.3e}"


def decay(t, *shape):
    return -torch.exp(t(*shape, scale=1.5, shift=-2.0))


def la_set(seed, B, T, H, Hk, Dk, Dv, dt=BF):
    t = draw(seed)
    a = [t(B, T, Hk, Dk, dtype=dt), t(B, T, Hk, Dk, dtype=dt), t(B, T, H, Dv, dtype=dt),
         decay(t, B, T, H), t(B, H, Dv, Dk)]
    return a, t(B, T, H, Dv, dtype=dt), t(B, H, Dv, Dk)


def la_close(a, o, s=None, out="f32", scale=1.0):
    B, T, H, Dv = a[2].shape
    Dk = a[0].shape[-1]
    (ow, sw), (mo, ms), (do, ds) = R.la_fwd(*[n64(x) for x in a], scale)
    close("o", o, ow, R.la_bound(ow, mo, do, T, Dk, Dv, out))
    if s is not None:
        close("s", s, sw, R.la_bound(sw, ms, ds, T, Dk, Dv))


def la_back_close(a, do, ds, got, grad="f32", scale=1.0):
    B, T, H, Dv = a[2].shape
    Hk, Dk = a[0].shape[2:]
    r = R.la_bwd(*[n64(x) for x in a], n64(do), n64(ds), scale)
    for n, x in zip(("dq", "dk", "dv"), got):
        close(n, x, r[0][n], R.la_bound(r[0][n], r[1][n], r[2][n], T, Dk, Dv, grad, H // Hk))
    if got[3] is not None:
        close("dg", got[3], r[0]["dg"], R.la_dg_bound(r, T, Dk, Dv))
    if got[4] is not None:
        close("ds0", got[4], r[0]["ds0"],
              R.la_bound(r[0]["ds0"], r[1]["ds0"], r[2]["ds0"], T, Dk, Dv))


def rotated_close(x, y, pos, f, out, inverse=False):
    want, m = R.rotary(n64(x), pos, n64(f), False, 1.0, inverse)
    close("rotary", y, want, R.rotary_bound(want, m, out, np.abs(pos).max()))


# ---- one after the other -------------------------------------------------------------


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (2, 2, 128)])
def test_block_and_its_gradient(gdr_lib, H, Hk, d):
    """Residual and norm, one projection, rotary positions in place in it, linear
    attention on its slices and the output gate, then back: each stage against its
    fp64 form on the bits that the stage before it left."""
    B, T, C = 2, 150, 264
    t = draw(1)
    x, res, w = t(B, T, C, dtype=BF), t(B, T, C), t(C, scale=0.2, shift=1)
    y, h = gdr_lib.gdr_rms_norm_fwd(x, w, residual=res)
    hr = n64(x.float() + res)
    close("norm", y, R.rms_fwd(hr, n64(w), 1e-6), R.rms_fwd_bound(hr, n64(w), 1e-6, "bf16"))
    wide_w = t(C, (2 * Hk + H) * d, scale=C ** -0.5)
    p = (y.float() @ wide_w).to(BF)
    plain = p.clone()
    n = Hk * d
    q, k = p[..., :n].unflatten(-1, (Hk, d)), p[..., n:2 * n].unflatten(-1, (Hk, d))
    v = p[..., 2 * n:].unflatten(-1, (H, d))
    f, pos = gdr_lib.gdr_rotary_frequencies(d), np.arange(T) + 5
    gdr_lib.gdr_rotary(q, k, 5, f, q_out=q, k_out=k)
    torch.cuda.synchronize()
    rotated_close(plain[..., :n].unflatten(-1, (Hk, d)), q, pos, f, "bf16")
    rotated_close(plain[..., n:2 * n].unflatten(-1, (Hk, d)), k, pos, f, "bf16")
    assert torch.equal(v, plain[..., 2 * n:].unflatten(-1, (H, d)))
    a = [q, k, v, decay(t, B, T, H), None]
    o, s = gdr_lib.gdr_linear_attn_fwd(*a, scale=d ** -0.5, out_dtype=F32)
    torch.cuda.synchronize()
    la_close(a, o, s, scale=d ** -0.5)
    g = t(B, T, H, d, dtype=BF)
    z = gdr_lib.gdr_output_gate(o, g, None, 1e-6, out_dtype=BF)
    dz = t(B, T, H, d, dtype=BF)
    do = gdr_lib.gdr_output_gate_bwd(o, g, None, dz, want_dw=False)[0].to(BF)
    assert torch.isfinite(z).all()
    ga = gdr_lib.gdr_linear_attn_bwd(*a, do, scale=d ** -0.5)
    torch.cuda.synchronize()
    la_back_close(a, do, None, ga, scale=d ** -0.5)
    rq, rk = gdr_lib.gdr_rotary(ga[0], ga[1], 5, f, inverse=True)
    torch.cuda.synchronize()
    rotated_close(ga[0], rq, pos, f, "f32", True)
    rotated_close(ga[1], rk, pos, f, "f32", True)
    dy = torch.cat([rq.flatten(2), rk.flatten(2), ga[2].flatten(2)], -1) @ wide_w.T
    dx, dw = gdr_lib.gdr_rms_norm_bwd(h, w, dy, dres=res)
    torch.cuda.synchronize()
    want, bound = R.rms_bwd(hr.reshape(-1, C), n64(w), n64(dy).reshape(-1, C), 1e-6,
                            n64(res).reshape(-1, C))
    close("dx", dx.view(-1, C), want[0], bound[0])
    close("dw", dw, want[1], bound[1])


def test_gradient_through_rotary_and_attention(gdr_lib):
    """The chain of both backwards against central differences of the chain of both
    forwards in fp32: quadratic in q and k together and linear in each, so the step
    costs nothing beyond the roundings over it."""
    B, T, H, d = 1, 45, 2, 32
    t = draw(2)
    q, k, v, do = (t(B, T, H, d) for _ in range(4))
    g = decay(t, B, T, H)
    f = gdr_lib.gdr_rotary_frequencies(24, scaling="linear", factor=4.0)

    def run(q, k):
        r = gdr_lib.gdr_rotary(q, k, 2, f, interleaved=True)
        return r, gdr_lib.gdr_linear_attn_fwd(*r, v, g)[0]

    r, o = run(q, k)
    gr = gdr_lib.gdr_linear_attn_bwd(*r, v, g, None, do)
    dq, dk = gdr_lib.gdr_rotary(gr[0], gr[1], 2, f, interleaved=True, inverse=True)
    torch.cuda.synchronize()
    (ow, _), (mo, _), (dm, _) = R.la_fwd(*[n64(x) for x in (*r, v, g)], None, 1.0)
    # rotary's own error moves o by its relative size of the majorant
    noise = ((R.la_bound(ow, mo, dm, T, d, d) + 4 * (2.0 ** -22 + 4 * R.U) * mo) *
             np.abs(n64(do))).sum()
    for i, (name, got) in enumerate((("q", dq), ("k", dk))):
        e, h = t(B, T, H, d), 2.0 ** -6

        def loss(sign):
            x = [q, k]
            x[i] = x[i] + sign * h * e
            return (run(*x)[1].double() * do.double()).sum().item()

        diff = (loss(1) - loss(-1)) / (2 * h)
        assert abs(diff - (n64(got) * n64(e)).sum()) <= 2 * noise / h, name


@pytest.mark.parametrize("H,Hk,d,rot", [(4, 2, 64, 64), (3, 3, 40, 16)])
def test_prompt_then_tokens(gdr_lib, H, Hk, d, rot):
    """A prompt through rotary and attention, then single tokens (in place, positions
    of each sequence its own) on the state that it left."""
    B, T, P = 3, 60, 41
    t = draw(3)
    p = t(B, T, (2 * Hk + H) * d, dtype=BF)
    n = Hk * d
    g, st = decay(t, B, T, H), t(B, H, d, d)
    s0 = st.clone()
    f = gdr_lib.gdr_rotary_frequencies(rot)
    first = torch.tensor([0, 9, 700], device="cuda")
    pos = first[:, None] + torch.arange(T, device="cuda")

    def cut(x):
        return (x[..., :n].unflatten(-1, (Hk, d)), x[..., n:2 * n].unflatten(-1, (Hk, d)),
                x[..., 2 * n:].unflatten(-1, (H, d)))

    q, k, v = cut(p)
    whole = gdr_lib.gdr_rotary(q, k, pos, f)
    outs = []
    for lo, hi in [(0, P)] + [(i, i + 1) for i in range(P, T)]:
        one = hi - lo == 1
        at = (slice(None), lo) if one else (slice(None), slice(lo, hi))
        q1, k1, v1 = cut(p[at])
        gdr_lib.gdr_rotary(q1, k1, pos[at], f, q_out=q1, k_out=k1)
        if one:
            o = gdr_lib.gdr_linear_attn_step(q1, k1, v1, g[at].contiguous(), st, out_dtype=F32)
            outs.append(o.unsqueeze(1))
        else:
            outs.append(gdr_lib.gdr_linear_attn_fwd(q1, k1, v1, g[at].contiguous(), st, s_final=st,
                                                    out_dtype=F32)[0])
    torch.cuda.synchronize()
    assert torch.equal(q, whole[0]) and torch.equal(k, whole[1])
    la_close([q, k, v, g, s0], torch.cat(outs, 1), st)


# ---- layouts ---------------------------------------------------------------------------


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 3, 8])
def test_strides_and_alignment(gdr_lib, dt, off):
    """Slices that begin at any element, sequence before or behind the batch, heads
    apart: the bits of contiguous inputs."""
    B, T, H, Hk, d = 2, 133, 4, 2, 40
    t = draw(4)
    a, do, ds = la_set(5, B, T, H, Hk, d, d, DT[dt])
    want = gdr_lib.gdr_linear_attn_fwd(*a)
    back = gdr_lib.gdr_linear_attn_bwd(*a, do, ds)
    one = gdr_lib.gdr_linear_attn_step(*[x[:, 3].contiguous() for x in a[:4]], a[4].clone())

    def apart(x, order):                  # the same values at odd places
        h = x.shape[2]
        buf = t(off + x.shape[order[0]] * (x.shape[order[1]] + 1) * (h + 1) * (d + 2), dtype=DT[dt])
        y = buf[off:].view(x.shape[order[0]], x.shape[order[1]] + 1, h + 1, d + 2)
        y = y[:, :x.shape[order[1]], :h, 1:1 + d]
        y = y if order == (0, 1) else y.transpose(0, 1)
        y.copy_(x)
        return y

    for order in ((0, 1), (1, 0)):
        b = [apart(x, order) for x in a[:3]] + a[3:]
        e = apart(do, order)
        got = gdr_lib.gdr_linear_attn_fwd(*b)
        gb = gdr_lib.gdr_linear_attn_bwd(*b, e, ds)
        g1 = gdr_lib.gdr_linear_attn_step(*[x[:, 3] for x in b[:3]], a[3][:, 3].contiguous(),
                                          a[4].clone())
        torch.cuda.synchronize()
        for x, y in zip((*want, *back, one), (*got, *gb, g1)):
            assert torch.equal(x, y)
        r = gdr_lib.gdr_rotary(b[0], b[1], 4, f := gdr_lib.gdr_rotary_frequencies(d))
        rc = gdr_lib.gdr_rotary(a[0], a[1], 4, f)
        ro = [apart(x, order) for x in rc]
        gdr_lib.gdr_rotary(b[0], b[1], 4, f, q_out=ro[0], k_out=ro[1])
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(r[i], rc[i]) and torch.equal(ro[i], rc[i])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_broadcast_inputs(gdr_lib, dt):
    """Inputs with a stride of 0 (one key of all heads and tokens, one value for all
    sequences): as their copies."""
    B, T, H, d = 3, 90, 4, 64
    t = draw(6)
    k = t(1, 1, 1, d, dtype=DT[dt]).expand(B, T, H, d)
    v = t(1, T, H, d, dtype=DT[dt]).expand(B, T, H, d)
    q = t(B, T, 1, d, dtype=DT[dt]).expand(B, T, H, d)
    do, g = t(B, 1, H, d, dtype=DT[dt]).expand(B, T, H, d), decay(t, B, T, H)
    got = gdr_lib.gdr_linear_attn_fwd(q, k, v, g)
    back = gdr_lib.gdr_linear_attn_bwd(q, k, v, g, None, do)
    c = [x.contiguous() for x in (q, k, v)]
    want = gdr_lib.gdr_linear_attn_fwd(*c, g)
    wb = gdr_lib.gdr_linear_attn_bwd(*c, g, None, do.contiguous())
    f = gdr_lib.gdr_rotary_frequencies(d)
    r, rc = gdr_lib.gdr_rotary(q, k, 1, f), gdr_lib.gdr_rotary(c[0], c[1], 1, f)
    torch.cuda.synchronize()
    for x, y in zip((*got, *back, *r), (*want, *wb, *rc)):
        assert torch.equal(x, y)
    la_back_close([*c, g, None], do, None, back)
    with pytest.raises(RuntimeError):
        gdr_lib.gdr_rotary(q, k, 1, f, q_out=q, k_out=k)
    with pytest.raises(RuntimeError):
        gdr_lib.gdr_rotary(c[0], None, 1, f, q_out=torch.empty_like(c[0][:1]).expand(B, T, H, d))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_same_tensor_as_all_inputs(gdr_lib, dt):
    t = draw(7)
    x, g = t(2, 100, 2, 64, dtype=DT[dt]), decay(t, 2, 100, 2)
    c = [x.clone(), x.clone(), x.clone(), g, None]
    o, s = gdr_lib.gdr_linear_attn_fwd(x, x, x, g)
    b = gdr_lib.gdr_linear_attn_bwd(x, x, x, g, None, x)
    torch.cuda.synchronize()
    la_close(c, o, s, dt)
    la_back_close(c, x, None, b)
    f = gdr_lib.gdr_rotary_frequencies(64)
    q, k = gdr_lib.gdr_rotary(x, x, 0, f)
    torch.cuda.synchronize()
    assert torch.equal(q, k)


def test_rows_behind_the_outputs_stay(gdr_lib):
    """Outputs in the middle of a buffer: what lies before and behind them is left as
    it was, at odd widths and lengths too; and so are the inputs."""
    def inside(*shape, dtype=F32):
        n = int(np.prod(shape))
        buf = torch.full((n + 128,), 7.0, dtype=dtype, device="cuda")
        bufs.append(buf)
        return buf[64:64 + n].view(shape)

    bufs = []
    for B, T, H, Hk, Dk, Dv, dt in ((2, 83, 3, 1, 24, 40, BF), (1, 700, 2, 2, 64, 104, F32)):
        a, do, ds = la_set(8, B, T, H, Hk, Dk, Dv, dt)
        f = gdr_lib.gdr_rotary_frequencies(Dk // 2)
        kept = [x.clone() for x in (*a, do, ds)]
        gdr_lib.gdr_linear_attn_fwd(*a, o=inside(B, T, H, Dv, dtype=dt),
                                    s_final=inside(B, H, Dv, Dk))
        gdr_lib.gdr_linear_attn_step(*[x[:, 0].contiguous() for x in a[:4]], a[4].clone(),
                                     o=inside(B, H, Dv, dtype=dt))
        n = gdr_lib.gdr_linear_attn_bwd_workspace_size(B, T, H, Hk, Dk, Dv, dt)
        ws = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
        gdr_lib.gdr_linear_attn_bwd(*a, do, ds, workspace=ws[128:128 + n])
        gdr_lib.gdr_rotary(a[0], a[1], 3, f, q_out=inside(*a[0].shape, dtype=dt),
                           k_out=inside(*a[1].shape, dtype=dt))
        x = a[2].reshape(B * T, H * Dv)
        gdr_lib.gdr_rms_norm_fwd(x, residual=x, y=inside(*x.shape, dtype=dt),
                                 h=inside(*x.shape, dtype=dt))
        q8 = torch.full((x.numel() + 128,), 7, dtype=torch.int8, device="cuda")
        gdr_lib.gdr_rms_norm_quant(x, y=q8[64:64 + x.numel()].view(x.shape),
                                   scales=inside(B * T, 1), out_dtype=torch.int8)
        torch.cuda.synchronize()
        assert all((b[:64] == 7).all() and (b[-64:] == 7).all() for b in (*bufs, q8))
        assert (ws[:128] == 77).all() and (ws[128 + n:] == 77).all()
        assert all(torch.equal(x, y) for x, y in zip((*a, do, ds), kept))


# ---- graphs, streams, workspaces ---------------------------------------------------------


def _everything(gdr, B, T, H, Hk, d, seed, dt=BF):
    """A function that runs every call on fixed inputs and returns its outputs."""
    a, do, ds = la_set(seed, B, T, H, Hk, d, d, dt)
    t = draw(seed + 50)
    C = H * d
    w, f = t(C), gdr.gdr_rotary_frequencies(d // 2)
    pos = torch.arange(T, device="cuda") * 3
    st = torch.empty_like(a[4])

    def run():
        o, s = gdr.gdr_linear_attn_fwd(*a)
        g = gdr.gdr_linear_attn_bwd(*a, do, ds)
        st.copy_(a[4])
        o1 = gdr.gdr_linear_attn_step(*[x[:, 0] for x in a[:3]], a[3][:, 0].contiguous(), st)
        r = gdr.gdr_rotary(a[0], a[1], pos, f)
        n, h = gdr.gdr_rms_norm_fwd(o.flatten(2), w, residual=do.flatten(2))
        q8, sc = gdr.gdr_rms_norm_quant(n, w, out_dtype=torch.int8)
        gn = gdr.gdr_rms_norm_bwd(h, w, n, dres=g[2].flatten(2))
        return (o, s, *g, st, o1, *r, n, h, q8, sc, *gn)

    return run


@pytest.mark.parametrize("B,T,H,Hk,d,dt", [(1, 900, 2, 1, 64, "bf16"), (3, 130, 3, 3, 40, "f32")])
def test_graph_of_every_call(gdr_lib, B, T, H, Hk, d, dt):
    """Captured once, replayed with eager work of the same calls between the replays:
    equal bits every time (the first case runs as segments and sums heads)."""
    run = _everything(gdr_lib, B, T, H, Hk, d, 10, DT[dt])
    other = _everything(gdr_lib, B, T + 3, H, Hk, d, 11, DT[dt])
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


def test_segments_in_the_graph_case(gdr_lib):
    assert gdr_lib.gdr_linear_attn_fwd_workspace_size(1, 900, 2, 64, 64, BF) > 0


def test_two_graphs_share_a_workspace(gdr_lib):
    """A workspace of the caller's that both graphs (and eager calls between them)
    write: nothing is kept in it from one call for the next."""
    sizes = ((1, 800, 2, 1, 64, 64), (2, 400, 3, 3, 40, 56))
    sets = [la_set(12 + i, *z) for i, z in enumerate(sizes)]
    n = max(gdr_lib.gdr_linear_attn_bwd_workspace_size(*z, BF) for z in sizes)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def one(a, d, e):
        return (*gdr_lib.gdr_linear_attn_fwd(*a, workspace=ws),
                *gdr_lib.gdr_linear_attn_bwd(*a, d, e, workspace=ws))

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
    """On a stream of the caller's, given or current, behind work that writes the
    inputs there; and two calls at once on two streams."""
    run = _everything(gdr_lib, 2, 200, 4, 2, 64, 14)
    want = [v.clone() for v in run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    a, do, ds = la_set(15, 2, 500, 4, 4, 64, 64)
    f = gdr_lib.gdr_rotary_frequencies(64)
    ow = gdr_lib.gdr_linear_attn_fwd(*a)[0].clone()
    gw = [v.clone() for v in gdr_lib.gdr_linear_attn_bwd(*a, do, ds)]
    rw = gdr_lib.gdr_rotary(a[0], a[1], 0, f)[0].clone()
    nw = gdr_lib.gdr_rms_norm_fwd(a[0]).clone()
    late = [torch.zeros_like(a[0]), *a[1:]]
    torch.cuda.synchronize()
    s2 = torch.cuda.Stream()
    with torch.cuda.stream(s):
        junk = torch.randn(1 << 24, device="cuda").sort()
        late[0].copy_(a[0])
    o = gdr_lib.gdr_linear_attn_fwd(*late, stream=s)[0]
    r = gdr_lib.gdr_rotary(late[0], a[1], 0, f, stream=s)[0]
    n = gdr_lib.gdr_rms_norm_fwd(late[0], stream=s)
    g = gdr_lib.gdr_linear_attn_bwd(*a, do, ds, stream=s2)
    torch.cuda.synchronize()
    del junk
    assert torch.equal(o, ow) and torch.equal(r, rw) and torch.equal(n, nw)
    assert all(torch.equal(p, q) for p, q in zip(g, gw))


# ---- padded tokens, states in place -----------------------------------------------------


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_padded_tokens_leave_the_state(gdr_lib, T, dt):
    """Tokens with a zero value and no decay: the state passes them unchanged, bit for
    bit, and its gradient too."""
    a, do, ds = la_set(16, 2, T, 2, 2, 64, 72, DT[dt])
    keep = T // 2
    a[2][1, keep:] = 0                   # behind the sequence
    a[3][1, keep:] = 0
    a[2][0] = 0                          # nothing left
    a[3][0] = 0
    do[0] = 0
    do[1, keep:] = 0
    o, s = gdr_lib.gdr_linear_attn_fwd(*a, out_dtype=F32)
    g = gdr_lib.gdr_linear_attn_bwd(*a, do, ds)
    torch.cuda.synchronize()
    assert torch.equal(s[0], a[4][0]) and torch.equal(g[4][0], ds[0])
    if keep:
        part = [x[1:, :keep] for x in a[:3]] + [a[3][1:, :keep], a[4][1:]]
        la_close(part, o[1:, :keep], s[1:])
    else:
        assert torch.equal(s, a[4])
    assert not g[0][0].any()


def test_tokens_of_no_value_or_key(gdr_lib):
    """All of q, k, v zero, every token a reset: outputs are zeros, not NaN."""
    z = torch.zeros(2, 70, 2, 64, dtype=BF, device="cuda")
    g = torch.full((2, 70, 2), float("-inf"), device="cuda")
    s0 = torch.randn(2, 2, 64, 64, device="cuda")
    o, s = gdr_lib.gdr_linear_attn_fwd(z, z, z, g, s0)
    b = gdr_lib.gdr_linear_attn_bwd(z, z, z, g, s0, z, s0)
    torch.cuda.synchronize()
    assert not o.any() and not s.any()
    assert not any(x.any() for x in b)


@pytest.mark.parametrize("T,Dk,Dv", [(1, 8, 8), (130, 64, 72), (1100, 128, 40)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_state_in_place(gdr_lib, T, Dk, Dv, dt):
    a, _, _ = la_set(17, 2, T, 2, 1, Dk, Dv, DT[dt])
    o, s = gdr_lib.gdr_linear_attn_fwd(*a)
    st = a[4].clone()
    o2, _ = gdr_lib.gdr_linear_attn_fwd(*a[:4], st, s_final=st)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, st)


def test_empty(gdr_lib):
    """No tokens: the state and its gradient pass through; no sequences or heads."""
    a, do, ds = la_set(18, 2, 0, 2, 2, 64, 64)
    o, s = gdr_lib.gdr_linear_attn_fwd(*a)
    g = gdr_lib.gdr_linear_attn_bwd(*a, do, ds)
    head = gdr_lib.gdr_linear_attn_bwd(*a[:3], torch.zeros(2, device="cuda"), a[4], do)
    st = a[4].clone()
    gdr_lib.gdr_linear_attn_fwd(*a[:4], st, s_final=st)
    none = gdr_lib.gdr_linear_attn_fwd(*a[:4])[1]
    f = gdr_lib.gdr_rotary_frequencies(64)
    r = gdr_lib.gdr_rotary(a[0], a[1], 0, f)
    torch.cuda.synchronize()
    assert o.numel() == 0 and torch.equal(s, a[4]) and torch.equal(g[4], ds)
    assert torch.equal(st, a[4]) and not none.any()
    assert not head[3].any() and not head[4].any() and r[0].shape == a[0].shape
    for z in (dict(B=0, T=5, H=2, Hk=2), dict(B=2, T=5, H=0, Hk=0)):
        b, e, _ = la_set(19, Dk=64, Dv=64, **z)
        assert gdr_lib.gdr_linear_attn_fwd(*b)[0].numel() == 0
        assert gdr_lib.gdr_linear_attn_bwd(*b, e)[0].numel() == 0
        st = [x[:, 0].contiguous() for x in b[:4]]
        assert gdr_lib.gdr_linear_attn_step(*st, b[4]).numel() == 0
        gdr_lib.gdr_rotary(b[0], b[1], 0, f)
    torch.cuda.synchronize()


# ---- arguments through the binding ---------------------------------------------------------


def test_binding_refuses(gdr_lib):
    a, do, ds = la_set(20, 2, 10, 4, 2, 64, 64)
    g, f = gdr_lib, gdr_lib.gdr_rotary_frequencies(64)
    q, k, v, d, s0 = a
    V, T, E = ValueError, TypeError, RuntimeError
    for err, call in (
            (V, lambda: g.gdr_linear_attn_fwd(q.cpu(), k, v)),
            (V, lambda: g.gdr_linear_attn_fwd(q, k.cpu(), v)),
            (T, lambda: g.gdr_linear_attn_fwd(q.float(), k, v)),
            (T, lambda: g.gdr_linear_attn_fwd(q.half(), k.half(), v.half())),
            (V, lambda: g.gdr_linear_attn_fwd(q[:, :5], k, v)),
            (V, lambda: g.gdr_linear_attn_fwd(q.transpose(2, 3), k.transpose(2, 3), v)),
            (V, lambda: g.gdr_linear_attn_fwd(q, k, v, d[:, :5].contiguous())),
            (T, lambda: g.gdr_linear_attn_fwd(q, k, v, d.to(BF))),
            (V, lambda: g.gdr_linear_attn_fwd(q, k, v, d.transpose(1, 2))),
            (V, lambda: g.gdr_linear_attn_fwd(q, k, v, d, s0[:1])),
            (V, lambda: g.gdr_linear_attn_fwd(q, k, v, d, s0.transpose(1, 2))),
            (T, lambda: g.gdr_linear_attn_fwd(q, k, v, out_dtype=torch.float16)),
            (T, lambda: g.gdr_linear_attn_fwd(q, k, v, o=torch.empty_like(v), out_dtype=F32)),
            (E, lambda: g.gdr_linear_attn_fwd(q, k, v, o=v)),
            (E, lambda: g.gdr_linear_attn_fwd(q, k, v[:, :, :3])),
            (E, lambda: g.gdr_linear_attn_fwd(q[..., :60], k[..., :60], v)),
            (V, lambda: g.gdr_linear_attn_step(q[:, 0], k[:, 0], v[:, 0], d, s0)),
            (V, lambda: g.gdr_linear_attn_step(q[:, 0], k[:, 0], v[:, 0], None, s0[:1])),
            (T, lambda: g.gdr_linear_attn_step(q[:, 0], k[:, 0], v[:, 0], None, s0.to(BF))),
            (V, lambda: g.gdr_linear_attn_bwd(q, k, v, d, s0, do[:, :5])),
            (T, lambda: g.gdr_linear_attn_bwd(q, k, v, d, s0, do.float())),
            (V, lambda: g.gdr_linear_attn_bwd(q, k, v, d, s0, do, ds.transpose(1, 2))),
            (T, lambda: g.gdr_linear_attn_bwd(q, k, v, d, s0, do, grad_dtype=torch.float16)),
            (E, lambda: g.gdr_linear_attn_bwd(q, k, v, d, s0, do, workspace=torch.empty(
                16, dtype=torch.uint8, device="cuda"))),
            (V, lambda: g.gdr_rotary(q[0, 0], None, 0, f)),
            (V, lambda: g.gdr_rotary(q, k, 0, f[None])),
            (T, lambda: g.gdr_rotary(q, k, 0, f.float())),
            (T, lambda: g.gdr_rotary(q, k.float(), 0, f)),
            (V, lambda: g.gdr_rotary(q, k[:, :3], 0, f)),
            (V, lambda: g.gdr_rotary(q, k, 0, f.cpu())),
            (V, lambda: g.gdr_rotary(q, k, torch.arange(9, device="cuda"), f)),
            (T, lambda: g.gdr_rotary(q, k, torch.arange(10, device="cuda").int(), f)),
            (V, lambda: g.gdr_rotary(q, None, 0, f, k_out=k)),
            (V, lambda: g.gdr_rotary(q, k, 0, f, q_out=v)),
            (E, lambda: g.gdr_rotary(q, k, 0, f, q_out=k)),
            (E, lambda: g.gdr_rotary(q[..., :32], None, 0, f)),
            (V, lambda: g.gdr_rms_norm_fwd(q, d)), (V, lambda: g.gdr_rms_norm_fwd(q, h=q)),
            (V, lambda: g.gdr_rms_norm_fwd(q, residual=v)),
            (V, lambda: g.gdr_rms_norm_quant(q, group=48)),
            (T, lambda: g.gdr_rms_norm_quant(q, out_dtype=BF)),
            (V, lambda: g.gdr_rms_norm_quant(q, scales=torch.empty(2, 10, 2, 2, device="cuda"))),
            (V, lambda: g.gdr_rms_norm_bwd(q, None, v)),
            (T, lambda: g.gdr_rms_norm_bwd(q, None, q, dres=q)),
            (E, lambda: g.gdr_rms_norm_bwd(q, None, q, workspace=torch.empty(
                16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(err):
            call()


# ---- offsets past 2^31 elements ---------------------------------------------------------------


@pytest.fixture(scope="module")
def wide():
    """One buffer of 2.2e9 bf16 elements that the tests below view."""
    buf = torch.empty(2101 << 20, dtype=BF, device="cuda")
    step = 1 << 28
    for i in range(0, buf.numel(), step):
        buf[i:i + step].normal_()
    return buf


def test_largest_token_stride(gdr_lib, wide):
    """Rows as far apart as a token's may lie, the last ones past 2^31."""
    T, H, d = 262, 2, 64
    rows = wide.view(-1)[:T << 23].view(1, T, 1 << 23)
    cut = [rows[..., i * 100003:][..., :H * d].unflatten(-1, (H, d)) for i in range(4)]
    a = [*cut[:3], decay(draw(21), 1, T, H), None]
    o, s = gdr_lib.gdr_linear_attn_fwd(*a, out_dtype=F32)
    g = gdr_lib.gdr_linear_attn_bwd(*a, cut[3])
    f = gdr_lib.gdr_rotary_frequencies(d)
    r = gdr_lib.gdr_rotary(cut[0], cut[1], 3, f)
    torch.cuda.synchronize()
    la_close(a, o, s)
    la_back_close(a, cut[3], None, g)
    rotated_close(cut[1], r[1], np.arange(T) + 3, f, "bf16")
    further = wide[:1 << 25].as_strided((1, 3, 1, 64), (0, (1 << 23) + 8, 64, 1))
    with pytest.raises(RuntimeError):
        gdr_lib.gdr_linear_attn_fwd(further, further, further)


def test_attention_past_2_31(gdr_lib, wide):
    """q, k, v, o and the gradients of 2.2e9 elements each: heads of the first, a
    middle and the last sequence."""
    B, T, H, d = 508, 264, 128, 128
    assert B * T * H * d > 2 ** 31
    x = wide[:B * T * H * d].view(B, T, H, d)
    v = x.flip(3)
    g = -torch.rand(B, T, H, device="cuda")
    o, s = gdr_lib.gdr_linear_attn_fwd(x, x, v, g)
    gr = gdr_lib.gdr_linear_attn_bwd(x, x, v, g, None, x, grad_dtype=BF)
    f = gdr_lib.gdr_rotary_frequencies(d)
    torch.cuda.synchronize()
    for b, h in ((0, 0), (300, 77), (B - 1, H - 1)):
        at = (slice(b, b + 1), slice(None), slice(h, h + 1))
        a = [x[at], x[at], v[at], g[at], None]
        la_close(a, o[at], s[b:b + 1, h:h + 1], "bf16")
        la_back_close(a, x[at], None, [*(y[at] for y in gr[:4]), gr[4][b:b + 1, h:h + 1]], "bf16")
    del gr, s, v
    r = gdr_lib.gdr_rotary(x, None, 5, f, q_out=o)[0]
    torch.cuda.synchronize()
    for b, h in ((0, 0), (B - 1, H - 1)):
        at = (slice(b, b + 1), slice(None), slice(h, h + 1))
        rotated_close(x[at], r[at], np.arange(T) + 5, f, "bf16")


def test_step_past_2_31(gdr_lib):
    """States of more than 2^31 floats."""
    N, H, d = 1100, 128, 128
    t = draw(22)
    st = torch.empty(N, H, d, d, device="cuda")
    for i in range(0, N, 100):
        st[i:i + 100].normal_()
    assert st.numel() > 2 ** 31
    q, k, v = (t(N, H, d, dtype=BF) for _ in range(3))
    g = decay(t, N, H)
    at = ((0, 0), (700, 3), (N - 1, H - 1))
    before = [st[n:n + 1, h:h + 1].clone() for n, h in at]
    o = gdr_lib.gdr_linear_attn_step(q, k, v, g, st, out_dtype=F32)
    torch.cuda.synchronize()
    for (n, h), s0 in zip(at, before):
        a = [x[n:n + 1, None, h:h + 1] for x in (q, k, v)] + [g[n:n + 1, None, h:h + 1], s0]
        la_close(a, o[n:n + 1, None, h:h + 1], st[n:n + 1, h:h + 1])


def test_rms_norm_past_2_31(gdr_lib, wide):
    C = 4096
    x = wide.view(-1, C)
    w = draw(23)(C)
    y, h = gdr_lib.gdr_rms_norm_fwd(x, w, residual=x)
    q, sc = gdr_lib.gdr_rms_norm_quant(x, w, out_dtype=torch.int8)
    dx, _ = gdr_lib.gdr_rms_norm_bwd(h, w, y, grad_dtype=BF)
    torch.cuda.synchronize()
    for r in (0, x.shape[0] // 2, x.shape[0] - 2):
        i = n64((2 * x[r:r + 2].float()).to(BF))
        close("y", y[r:r + 2], R.rms_fwd(i, n64(w), 1e-6), R.rms_fwd_bound(i, n64(w), 1e-6, "bf16"))
        want, bound = R.rms_bwd(i, n64(w), n64(y[r:r + 2]), 1e-6, None)
        close("dx", dx[r:r + 2], want[0], bound[0] + R.HALF["bf16"] * (np.abs(want[0]) + bound[0]))
        i = n64(x[r:r + 2])
        z, e = R.rms_fwd(i, n64(w), 1e-6), R.rms_fwd_bound(i, n64(w), 1e-6)
        close("q", q[r:r + 2].float() * sc[r:r + 2], z,
              (0.5 * n64(sc[r:r + 2]) + e + 4 * R.U * np.abs(z)) * (1 + 1e-6))
