"""GPU parity of gdr_layer_norm_fwd and _bwd with the fp64 form, at the bounds
derived in block_reference."""
import numpy as np
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
WIDTHS = [1, 7, 8, 64, 500, 512, 513, 1024, 1025, 2047, 2048, 2049, 4097, 8192, 8193, 20001]


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def make(rows, C, dt, seed, mean=0.3):
    g = rng(seed)

    def t(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return torch.from_numpy((shift + scale * g.standard_normal(shape)).astype(np.float32)
                                ).to(dtype)

    return dict(x=t(rows, C, dtype=DT[dt], shift=mean), res=t(rows, C), w=t(C, scale=0.2, shift=1),
                b=t(C, scale=0.2), dy=t(rows, C), dres=t(rows, C))


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def cu(t):
    return None if t is None else t.cuda()


def close(name, got, want, bound):
    err = np.abs(n64(got) - want)
    assert got.shape == want.shape
    over = err - bound
    assert np.isfinite(err).all() and over.max() <= 0, \
        f"{name}: error {err.max():.3e}, worst over its bound by {over.max():.3e}"


def check_fwd(gdr, i, out="f32", res=None, w=True, b=True, eps=1e-5):
    wt, bt = (i["w"] if w else None), (i["b"] if b else None)
    if res is None:
        y = gdr.gdr_layer_norm_fwd(cu(i["x"]), cu(wt), cu(bt), eps, out_dtype=DT[out])
        h = i["x"]
    else:
        r = i["res"].to(DT[res])
        y, hg = gdr.gdr_layer_norm_fwd(cu(i["x"]), cu(wt), cu(bt), eps, residual=cu(r),
                                       out_dtype=DT[out])
        h = (i["x"].float() + r.float()).to(DT[res])
        torch.cuda.synchronize()
        assert torch.equal(hg.cpu(), h), "the residual sum is the rounded fp32 sum"
    torch.cuda.synchronize()
    h = n64(h)
    close("y", y, R.norm_fwd(h, n64(wt), n64(bt), eps),
          R.norm_fwd_bound(h, n64(wt), n64(bt), eps, out))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
def test_fwd_widths(gdr_lib, C, res):
    check_fwd(gdr_lib, make(5, C, "bf16", C), res=res)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 1000])
@pytest.mark.parametrize("dt,out,res", [("f32", "f32", None), ("bf16", "bf16", "bf16"),
                                        ("bf16", "f32", "f32"), ("f32", "bf16", None)])
def test_fwd_rows_and_types(gdr_lib, rows, dt, out, res):
    check_fwd(gdr_lib, make(rows, 129, dt, rows), out, res)


@pytest.mark.parametrize("w", [True, False])
@pytest.mark.parametrize("b", [True, False])
@pytest.mark.parametrize("C", [96, 3001, 9000])
def test_fwd_without_weights(gdr_lib, w, b, C):
    check_fwd(gdr_lib, make(3, C, "f32", 3), w=w, b=b)


@pytest.mark.parametrize("C", [100, 2500, 10000])
def test_fwd_large_mean_and_constant_rows(gdr_lib, C):
    """A mean 300 times the spread loses only what its rounding loses; a
    constant row gives b."""
    check_fwd(gdr_lib, make(4, C, "f32", 9, mean=300.0))
    x = torch.full((2, C), 2.5, device="cuda")
    b = torch.randn(C, device="cuda")
    y = gdr_lib.gdr_layer_norm_fwd(x, None, b)
    torch.cuda.synchronize()
    # 2.5 C is exact in fp32 but its quotient by C need not be: off by half a step
    lim = 2.5 * R.U * 4 / np.sqrt(1e-5)
    assert ((y - b).abs().max() <= lim + 1e-6).item()


def test_rows_apart_and_in_place(gdr_lib):
    g = torch.Generator().manual_seed(1)
    wide = torch.randn((9, 333), generator=g).bfloat16().cuda()
    x, r = wide[:, 3:132], wide[:, 180:309]
    y, h = gdr_lib.gdr_layer_norm_fwd(x, residual=r)
    xc, rc = x.contiguous(), r.contiguous()
    y2, h2 = gdr_lib.gdr_layer_norm_fwd(xc, residual=rc, y=xc, h=rc)
    torch.cuda.synchronize()
    assert y2 is xc and h2 is rc and torch.equal(y, y2) and torch.equal(h, h2)
    three = gdr_lib.gdr_layer_norm_fwd(x.reshape(3, 3, 129))
    torch.cuda.synchronize()
    assert torch.equal(three.reshape(9, 129), gdr_lib.gdr_layer_norm_fwd(x))


def check_bwd(gdr, i, dy="f32", grad="f32", dres=False, w=True, eps=1e-5):
    d, q = i["dy"].to(DT[dy]), (i["dres"].to(DT[grad]) if dres else None)
    wt = i["w"] if w else None
    got = gdr.gdr_layer_norm_bwd(cu(i["x"]), cu(wt), cu(d), eps, dres=cu(q), grad_dtype=DT[grad])
    torch.cuda.synchronize()
    want, bound = R.norm_bwd(n64(i["x"]), n64(wt), n64(d), eps, n64(q))
    bound[0] = bound[0] + R.HALF[grad] * (np.abs(want[0]) + bound[0])
    for name, g, v, e in zip(("dx", "dw", "db"), got, want, bound):
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
    check_bwd(gdr_lib, make(700, C, "bf16", C), "bf16", "bf16", True, w=False)


def test_bwd_options_and_empty(gdr_lib):
    i = make(50, 300, "f32", 4)
    x, w, dy, q = (cu(i[k]) for k in ("x", "w", "dy", "dres"))
    one = gdr_lib.gdr_layer_norm_bwd(x, w, dy, dres=q)
    two = gdr_lib.gdr_layer_norm_bwd(x, w, dy, dres=q)
    dx, dw, db = gdr_lib.gdr_layer_norm_bwd(x, w, dy, dres=q, want_dw=False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert dw is None and db is None and torch.equal(dx, one[0])
    dx, dw, db = gdr_lib.gdr_layer_norm_bwd(x[:0], w, dy[:0])
    assert gdr_lib.gdr_layer_norm_fwd(x[:0], w).shape == (0, 300)
    torch.cuda.synchronize()
    assert dx.shape == (0, 300) and not dw.any() and not db.any()


@pytest.mark.parametrize("C", [8192, 8193, 12000, 16379, 16384, 16385])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_longest_rows_in_registers(gdr_lib, C, dt):
    i = make(40, C, dt, C)
    check_fwd(gdr_lib, i, dt, dt)
    check_bwd(gdr_lib, i, dt, dt, True)
