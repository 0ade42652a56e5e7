"""Edges of the operators around the mixer: sizes of zero that leave some
outputs with elements, values at the ends of the type's range, and buffers that
are their own outputs."""
import numpy as np
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LOWEST = torch.finfo(F32).min


def draw(seed):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, dtype=F32, scale=1.0, shift=0.0):
        return (shift + scale * torch.randn(shape, generator=g)).to(dtype).cuda()

    return t


# ---- no channels ------------------------------------------------------------------


@pytest.mark.parametrize("grad", [F32, BF])
@pytest.mark.parametrize("G", [1, 3])
def test_scan_bwd_of_no_channels(gdr_lib, grad, G):
    """dB and dC are sums over channels: zeros where there are none, whatever
    their memory held before."""
    B, T, N = 2, 9, 16
    t = draw(1)
    x, bc = torch.empty(B, T, 0, device="cuda"), t(B, T, G, N)
    held = [torch.full((B, T, G, N), 7.0, dtype=grad, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del held
    z, none = torch.empty_like(x), torch.empty(0, device="cuda")
    o = gdr_lib.gdr_ssm_scan_bwd(x, x, torch.empty(0, N, device="cuda"), bc, bc, none, z, none,
                                 None, x, grad_dtype=grad)
    torch.cuda.synchronize()
    assert [tuple(v.shape) for v in o] == [
        (B, T, 0), (B, T, 0), (0, N), (B, T, G, N), (B, T, G, N), (0,), (B, T, 0), (0,), (B, 0, N)]
    for v in (o[3], o[4]):
        assert v.dtype == grad and not v.any()


# ---- states that forget at once -----------------------------------------------------


def forgetting(seed, B, T, D, N, dt):
    t = draw(seed)
    i = [t(B, T, D, dtype=dt), t(B, T, D, dtype=dt), -torch.exp(t(D, N, scale=0.7)),
         t(B, T, 1, N, dtype=dt), t(B, T, 1, N, dtype=dt), t(D), t(B, T, D, dtype=dt),
         t(D, shift=-3.0), t(B, D, N)]
    return i, t(B, T, D, dtype=dt), t(B, D, N)


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(name, got, want, bound):
    err = np.abs(n64(got) - want)
    over = err - bound
    assert got.shape == want.shape and np.isfinite(err).all() and over.max() <= 0, \
        f"{name}: error {err.max():.3e}, worst over its bound by {over.max():.3e}"


@pytest.mark.parametrize("A", [float("-inf"), LOWEST])
@pytest.mark.parametrize("T,D,N", [(1, 70, 16), (5, 70, 16), (8, 9, 3), (30, 130, 7), (75, 70, 33),
                                   (700, 70, 16)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_scan_that_forgets_at_once(gdr_lib, A, T, D, N, dt):
    """A of minus infinity, or fp32's lowest value: with the steps of these
    tokens (all above 1e-9) the decay is 0, as it is in fp64 at A = -1e30, where
    the reference takes it.  Padded tokens, ends of segments and of the tensors
    inside a block meet steps of 0."""
    a, do, dh = forgetting(T + N, 2, T, D, N, dt)
    a[2][:, 0] = A
    a[2][5 % D] = A
    y, h = gdr_lib.gdr_ssm_scan_fwd(*a, out_dtype=F32)
    o = gdr_lib.gdr_ssm_scan_bwd(*a, do, dh)
    torch.cuda.synchronize()
    ref = [n64(v) for v in a]
    ref[2] = np.maximum(ref[2], -1e30)
    assert np.logaddexp(ref[1] + ref[7], 0).min() > 1e-9
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    close("y", y, want, R.scan_bound(my, T, "f32", want))
    close("h", h, wh, R.scan_bound(mh, T))
    ref += [n64(do), n64(dh)]
    want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
    for k, g in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0"), o):
        steps = 2 * T + (D if k in ("dB", "dC") else 2 * T if k in ("dA", "dD", "db") else 0)
        close(k, g, want[k], R.scan_bound(maj[k], steps))


@pytest.mark.parametrize("A", [float("-inf"), LOWEST])
@pytest.mark.parametrize("T", [40, 700])
def test_padded_tokens_of_states_that_forget_at_once(gdr_lib, A, T):
    """dt at minus infinity is a step of 0 there too: the state passes, the
    token's own gradients are 0 whatever arrives at it, and all others are those
    of the tokens before it."""
    D = 70
    a, do, dh = forgetting(6, 2, T, D, 16, BF)
    a[2][:, 0] = A
    a[1][:, T - 13:] = float("-inf")
    do[:, T - 13:] = 0
    y, h = gdr_lib.gdr_ssm_scan_fwd(*a, out_dtype=F32)
    o = gdr_lib.gdr_ssm_scan_bwd(*a, do, dh)
    torch.cuda.synchronize()
    assert not o[1][:, T - 13:].any() and not o[0][:, T - 13:].any()
    part = [v[:, :T - 13] if k in (0, 1, 3, 4, 6) else v for k, v in enumerate(a)]
    ref = [n64(v) for v in part]
    ref[2] = np.maximum(ref[2], -1e30)
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    close("y", y[:, :T - 13], want, R.scan_bound(my, T, "f32", want))
    close("h", h, wh, R.scan_bound(mh, T))
    ref += [n64(do[:, :T - 13]), n64(dh)]
    want, maj = R.scan_bwd(*ref), R.scan_bwd(*ref, majorant=True)
    for k, g in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0"), o):
        steps = 2 * T + (D if k in ("dB", "dC") else 2 * T if k in ("dA", "dD", "db") else 0)
        g = g[:, :T - 13] if g.shape[1:2] == (T,) else g
        close(k, g, want[k], R.scan_bound(maj[k], steps))


@pytest.mark.parametrize("A", [float("-inf"), LOWEST])
def test_token_that_forgets_at_once(gdr_lib, A):
    """The decode token: a step above 0 forgets, a step of 0 (dt at minus
    infinity, a padded sequence) keeps the state bit for bit."""
    a, _, _ = forgetting(3, 2, 1, 70, 16, BF)
    a[2][:, 0] = A
    a[1][1] = float("-inf")
    h = a[8].clone()
    st = [v[:, 0] if k in (0, 1, 3, 4, 6) else v for k, v in enumerate(a)]
    y = gdr_lib.gdr_ssm_step(*st[:5], h, *st[5:8], out_dtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(h[1], a[8][1]) and torch.isfinite(y).all()
    ref = [n64(v[:1]) if k in (0, 1, 3, 4, 6, 8) else n64(v) for k, v in enumerate(a)]
    ref[2] = np.maximum(ref[2], -1e30)
    want, wh, _ = R.scan_fwd(*ref)
    my, mh, _ = R.scan_fwd(*ref, majorant=True)
    close("y", y[:1].unsqueeze(1), want, R.scan_bound(my, 1, "f32", want))
    close("h", h[:1], wh, R.scan_bound(mh, 1))


def test_scan_of_a_rate_that_is_no_number(gdr_lib):
    """NaN in A is not taken for a value: it reaches its channel, and no other."""
    a, _, _ = forgetting(4, 2, 50, 70, 16, BF)
    want, hw = gdr_lib.gdr_ssm_scan_fwd(*a)
    a[2][7, 2] = float("nan")
    y, h = gdr_lib.gdr_ssm_scan_fwd(*a)
    torch.cuda.synchronize()
    other = torch.arange(70, device="cuda") != 7
    assert torch.equal(y[..., other], want[..., other]) and torch.isnan(y[..., 7]).all()
    assert torch.equal(h[:, other], hw[:, other]) and torch.isnan(h[:, 7, 2]).all()


# ---- the convolution's state is a copy ------------------------------------------------


@pytest.mark.parametrize("C", [8192, 5000, 259, 6])
@pytest.mark.parametrize("K", [2, 4])
def test_conv_state_keeps_every_bit(gdr_lib, C, K):
    """Every bit pattern of bf16 (signalling NaNs among them) goes through the
    state as it is: from x, from the old state, and one token at a time."""
    n = K - 1
    B = -(-65536 // (n * C))
    bits = torch.arange(B * n * C, dtype=torch.int32, device="cuda").to(torch.int16)
    rows = bits.view(B, n, C).view(BF)
    w = draw(5)(C, K)
    x = torch.cat([torch.zeros(B, 5, C, dtype=BF, device="cuda"), rows], 1)
    _, sf = gdr_lib.gdr_short_conv_fwd(x, w)
    _, kept = gdr_lib.gdr_short_conv_fwd(x[:, :1], w, s0=rows)
    st = torch.zeros_like(rows)
    held = rows.clone()
    for t in range(n):
        gdr_lib.gdr_short_conv_step(rows[:, t], w, None, st)
    gdr_lib.gdr_short_conv_fwd(x[:, :1], w, s0=held, s_final=held)
    torch.cuda.synchronize()

    def same(a, b):
        return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))

    assert same(sf, rows) and same(st, rows)
    if n > 1:
        assert same(kept[:, :n - 1], rows[:, 1:]) and same(held[:, :n - 1], rows[:, 1:])


def test_conv_state_keeps_every_bit_in_fp32(gdr_lib):
    word = torch.tensor([0x7f800001, 0x7fc12345, 1, 0x007fffff, -1, -0x7fffffff, -0x400001],
                        dtype=torch.int32, device="cuda").repeat(5).view(1, 1, 35)
    x, w = word.view(F32), draw(6)(35, 2)
    _, sf = gdr_lib.gdr_short_conv_fwd(x, w)
    st = torch.zeros_like(x)
    gdr_lib.gdr_short_conv_step(x[:, 0], w, None, st)
    torch.cuda.synchronize()
    assert torch.equal(sf.view(torch.int32), word) and torch.equal(st.view(torch.int32), word)


# ---- one row -----------------------------------------------------------------------------


@pytest.mark.parametrize("C", [5, 24, 2049, 9001])
def test_one_row_of_a_wider_tensor_in_place(gdr_lib, C):
    """A single row is contiguous whatever lies behind it: a decode step's row
    of a wider buffer is its own output."""
    t = draw(7)
    wide, rwide, w = t(3, C + 16), t(3, C + 16), t(C)
    x, r = wide[:1, :C], rwide[:1, :C]
    y, h = gdr_lib.gdr_layer_norm_fwd(x, w, residual=r)
    behind = wide.clone(), rwide.clone()
    y2, h2 = gdr_lib.gdr_layer_norm_fwd(x, w, residual=r, y=x, h=r)
    torch.cuda.synchronize()
    assert y2 is x and h2 is r and torch.equal(y, x) and torch.equal(h, r)
    for now, before in zip((wide, rwide), behind):
        now[:1, :C] = before[:1, :C]
        assert torch.equal(now, before)


# ---- the chain's last stage -------------------------------------------------------------


def gate64(o, g, w, eps):
    """The output gate, and its bound: the mean square errs by 66 U (64 squares
    and their sum, no cancellation), its root by half of that and 8 U more,
    sigmoid by 2 |g| U (the exponent's argument) and 6 U, five products by one
    step each."""
    ms = (o * o).mean(-1, keepdims=True) + eps
    y = o / np.sqrt(ms) * (1.0 if w is None else w) * g * R.sigmoid(g)
    return y, (33 + 8 + 6 + 5 + 2 * np.abs(g)) * R.U * np.abs(y) * 1.05 + 1e-30


@pytest.mark.parametrize("weight", [True, False])
def test_gate_of_a_projections_slice(gdr_lib, weight):
    """Norm, projection, convolution, delta rule and output gate, the gate's
    branch the projection's last columns: the gate against fp64 on the bits of
    o and of that slice.  Neighbouring columns, or g without its sigmoid, are
    far outside the bound."""
    B, T, H, d, C = 2, 70, 2, 64, 96
    t = draw(8)
    x = gdr_lib.gdr_layer_norm_fwd(t(B, T, C, dtype=BF), t(C, scale=0.2, shift=1), t(C))
    wide = (x.float() @ t(C, 4 * H * d, scale=C ** -0.5)).to(BF)
    u, _ = gdr_lib.gdr_short_conv_fwd(wide[..., :3 * H * d], t(3 * H * d, 4, scale=0.6))
    q, k, v = (s.unflatten(-1, (H, d)).contiguous() for s in u.split(H * d, -1))
    q, k = (torch.nn.functional.normalize(s.float(), dim=-1).to(BF) for s in (q, k))
    ab = torch.sigmoid(t(2, B, T, H) + 1)
    o, _ = gdr_lib.gdr_chunk_fwd(q, k, v, ab[0].contiguous(), ab[1].contiguous(), None,
                                 out_dtype=F32)
    g = wide[..., 3 * H * d:].reshape(B * T, H, d).contiguous()
    w = t(d, scale=0.2, shift=1) if weight else None
    y = gdr_lib.gdr_output_gate(o.reshape(B * T, H, d), g, w, 1e-6, out_dtype=F32)
    torch.cuda.synchronize()
    oo, gg = n64(o).reshape(B * T, H, d), n64(g)
    want, bound = gate64(oo, gg, n64(w), 1e-6)
    close("gate", y, want, bound)
    for wrong in (gate64(oo, n64(wide[..., 2 * H * d:3 * H * d]).reshape(gg.shape), n64(w), 1e-6),
                  (want / R.sigmoid(gg), bound)):
        assert (np.abs(n64(y) - wrong[0]) > bound).mean() > 0.9
