"""GPU parity of gdr_rms_norm_fwd, _quant and _bwd with the fp64 form, at the bounds
derived in linear_reference."""
import numpy as np
import pytest
import torch

import linear_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3, I8 = torch.float8_e4m3fn, torch.int8
WIDTHS = [1, 7, 8, 64, 500, 512, 513, 1024, 1025, 2047, 2048, 2049, 4097, 8192, 8193, 20001]


def make(rows, C, dt, seed):
    g = R.rng(seed)

    def t(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return torch.from_numpy((shift + scale * g.standard_normal(shape)).astype(np.float32)
                                ).to(dtype).cuda()

    return dict(x=t(rows, C, dtype=DT[dt], shift=0.3), res=t(rows, C), w=t(C, scale=0.2, shift=1),
                dy=t(rows, C), dres=t(rows, C))


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(name, got, want, bound):
    err = np.abs(n64(got) - want)
    assert got.shape == want.shape
    assert np.isfinite(err).all() and (err - bound).max() <= 0, \
        f"{name}: error {err.max():.3e}, worst over its bound by {(err - bound).max():.3e}"


def summed(i, res):
    """(residual, h) as the call takes and leaves them."""
    if res is None:
        return None, i["x"]
    r = i["res"].to(DT[res])
    return r, (i["x"].float() + r.float()).to(DT[res])


def check_fwd(gdr, i, out="f32", res=None, w=True, eps=1e-6):
    wt = i["w"] if w else None
    r, h = summed(i, res)
    y = gdr.gdr_rms_norm_fwd(i["x"], wt, eps, residual=r, out_dtype=DT[out])
    if res is not None:
        y, hg = y
        assert torch.equal(hg, h), "the residual sum is the rounded fp32 sum"
    torch.cuda.synchronize()
    close("y", y, R.rms_fwd(n64(h), n64(wt), eps), R.rms_fwd_bound(n64(h), n64(wt), eps, out))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_fwd_widths(gdr_lib, C, res):
    check_fwd(gdr_lib, make(5, C, "bf16", C), res=res)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 1000])
@pytest.mark.parametrize("dt,out,res", [("f32", "f32", None), ("bf16", "bf16", "bf16"),
                                        ("bf16", "f32", "f32"), ("f32", "bf16", None)])
def test_fwd_rows_and_types(gdr_lib, rows, dt, out, res):
    check_fwd(gdr_lib, make(rows, 129, dt, rows), out, res)
    check_fwd(gdr_lib, make(rows, 129, dt, rows), out, res, w=False, eps=0.25)


def check_quant(gdr, i, kind, group, res=None, w=True, eps=1e-6):
    wt = i["w"] if w else None
    r, h = summed(i, res)
    got = gdr.gdr_rms_norm_quant(i["x"], wt, eps, residual=r, group=group, out_dtype=kind)
    torch.cuda.synchronize()
    if res is not None:
        assert torch.equal(got[2], h)
    q, s = got[:2]
    R_, C = i["x"].shape
    n = C // (group or C)
    assert q.dtype == kind and tuple(s.shape) == (R_, n)
    y, e = R.rms_fwd(n64(h), n64(wt), eps), R.rms_fwd_bound(n64(h), n64(wt), eps)
    top = 448.0 if kind == E4M3 else 127.0
    yg, eg = y.reshape(R_, n, -1), e.reshape(R_, n, -1)
    most = np.abs(yg).max(-1)
    # the largest moves by no more than the largest error, then one division
    close("scales", s, most / top, (eg.max(-1) + 2 * R.U * most) / top)
    # half a step of the code at the value (e4m3: 2^-4 of it, or half of the smallest
    # step 2^-9; int8: half), the quotient's 3 roundings, and y's own error
    sc = n64(s)[..., None]
    step = np.maximum(2.0 ** -4 * (np.abs(yg) + eg), 2.0 ** -10 * sc) if kind == E4M3 else 0.5 * sc
    close("q", (n64_t(q) * torch.from_numpy(sc.repeat(yg.shape[-1], -1).reshape(R_, C))), y,
          (step + eg + 4 * R.U * np.abs(yg)).reshape(R_, C) * (1 + 1e-6))
    # the largest of each group is the largest code
    assert np.abs(n64_t(q).numpy().reshape(R_, n, -1)).max(-1).min() == top


def n64_t(q):
    return q.cpu().float().double()


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("kind", [E4M3, I8])
@pytest.mark.parametrize("res", [None, "bf16"])
def test_quant_widths(gdr_lib, C, kind, res):
    check_quant(gdr_lib, make(5, C, "bf16", C), kind, None, res)


@pytest.mark.parametrize("C", [128, 640, 896, 1152, 2048, 2176, 4224, 8320, 16384, 17024])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", [E4M3, I8])
def test_quant_groups(gdr_lib, C, group, kind):
    check_quant(gdr_lib, make(5, C, "bf16", C), kind, group, "f32")
    if C < 1000:
        check_quant(gdr_lib, make(3, 3 * group, "f32", C), kind, group, None, w=False)


def test_quant_zeros_and_tiny(gdr_lib):
    """Rows and groups of zeros: scale 0, codes 0; so where the scale would be below
    fp32's normal numbers."""
    x = torch.randn(4, 256, device="cuda")
    x[1] = 0
    x[2, 64:128] = 0
    x[3, 128:192] = 1e-37
    for kind in (E4M3, I8):
        q, s = gdr_lib.gdr_rms_norm_quant(x, eps=1.0, group=64, out_dtype=kind)
        torch.cuda.synchronize()
        zero = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
        zero[1] = zero[2, 1] = zero[3, 2] = True
        assert (s == 0).equal(zero)
        assert not q.float().view(4, 4, 64)[zero].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("C", [64, 2048, 4096, 20480])
def test_bad_values_stay_in_their_row(gdr_lib, bad, C):
    i = make(9, C, "f32", C)
    y = gdr_lib.gdr_rms_norm_fwd(i["x"], i["w"])
    two = [gdr_lib.gdr_rms_norm_quant(i["x"], i["w"], group=g, out_dtype=k)
           for k in (E4M3, I8) for g in (None, 64)]
    dx, _ = gdr_lib.gdr_rms_norm_bwd(i["x"], i["w"], i["dy"])
    i["x"][4, 37] = bad
    y2 = gdr_lib.gdr_rms_norm_fwd(i["x"], i["w"])
    two2 = [gdr_lib.gdr_rms_norm_quant(i["x"], i["w"], group=g, out_dtype=k)
            for k in (E4M3, I8) for g in (None, 64)]
    dx2, _ = gdr_lib.gdr_rms_norm_bwd(i["x"], i["w"], i["dy"])
    torch.cuda.synchronize()
    other = torch.arange(9, device="cuda") != 4
    assert torch.equal(y[other], y2[other]) and torch.isnan(y2[4, 37])
    assert torch.equal(dx[other], dx2[other]) and not torch.isfinite(dx2[4, 37])
    for (q, s), (q2, s2) in zip(two, two2):
        assert torch.equal(q[other].view(torch.uint8), q2[other].view(torch.uint8))
        assert torch.equal(s[other], s2[other])
        assert torch.isnan(s2[4, 0])        # the scale of channel 37


def check_bwd(gdr, i, dy="f32", grad="f32", dres=False, w=True, eps=1e-6):
    d, q = i["dy"].to(DT[dy]), (i["dres"].to(DT[grad]) if dres else None)
    wt = i["w"] if w else None
    got = gdr.gdr_rms_norm_bwd(i["x"], wt, d, eps, dres=q, grad_dtype=DT[grad])
    torch.cuda.synchronize()
    want, bound = R.rms_bwd(n64(i["x"]), n64(wt), n64(d), eps, n64(q))
    bound[0] = bound[0] + R.HALF[grad] * (np.abs(want[0]) + bound[0])
    for name, g, v, e in zip(("dx", "dw"), got, want, bound):
        close(name, g, v, e)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dres", [False, True])
def test_bwd_widths(gdr_lib, C, dres):
    check_bwd(gdr_lib, make(6, C, "bf16", C), dres=dres)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 2600])
@pytest.mark.parametrize("dt,dy,grad", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                        ("bf16", "f32", "f32")])
def test_bwd_rows_and_types(gdr_lib, rows, dt, dy, grad):
    check_bwd(gdr_lib, make(rows, 65, dt, rows), dy, grad, True)


@pytest.mark.parametrize("C", [77, 2100, 8200])
def test_bwd_many_rows_without_weight(gdr_lib, C):
    """More rows than workgroups of each variant."""
    check_bwd(gdr_lib, make(1300, C, "bf16", C), "bf16", "bf16", True, w=False)


def test_rows_apart_and_in_place(gdr_lib):
    g = torch.Generator().manual_seed(1)
    for C in (129, 521, 2055, 8191, 9001, 20001):
        wide = torch.randn((9, 2 * C + 75), generator=g).bfloat16().cuda()
        x, r = wide[:, 3:3 + C], wide[:, C + 50:2 * C + 50]
        y, h = gdr_lib.gdr_rms_norm_fwd(x, residual=r)
        xc, rc, rq = x.contiguous(), r.contiguous(), r.contiguous()
        q, s, hq = gdr_lib.gdr_rms_norm_quant(x, residual=r)
        q2, s2, hq2 = gdr_lib.gdr_rms_norm_quant(xc, residual=rq, h=rq)
        dx, dw = gdr_lib.gdr_rms_norm_bwd(h, None, x, dres=r, grad_dtype=torch.bfloat16)
        y2, h2 = gdr_lib.gdr_rms_norm_fwd(xc, residual=rc, y=xc, h=rc)
        torch.cuda.synchronize()
        assert y2 is xc and h2 is rc and torch.equal(y, y2) and torch.equal(h, h2)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
        assert torch.equal(hq, h) and torch.equal(hq2, h) and hq2 is rq
        dx2, dw2 = gdr_lib.gdr_rms_norm_bwd(h2, None, x, dres=r, grad_dtype=torch.bfloat16)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    three = gdr_lib.gdr_rms_norm_quant(wide[:, :128].reshape(3, 3, 128), group=32)
    flat = gdr_lib.gdr_rms_norm_quant(wide[:, :128], group=32)
    torch.cuda.synchronize()
    assert tuple(three[1].shape) == (3, 3, 4) and torch.equal(three[1].view(9, 4), flat[1])
    assert torch.equal(three[0].view(9, 128).view(torch.uint8), flat[0].view(torch.uint8))


def test_empty(gdr_lib):
    x = torch.empty(0, 64, device="cuda")
    assert gdr_lib.gdr_rms_norm_fwd(x).shape == (0, 64)
    q, s = gdr_lib.gdr_rms_norm_quant(x, group=32)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    dx, dw = gdr_lib.gdr_rms_norm_bwd(x, None, x)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not dw.any()
