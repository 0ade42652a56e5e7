"""Argument checks of the operators around the mixer, on the CPU: nothing is
launched (fake device addresses, and calls that end before a launch)."""
import ctypes
import os
import re

import pytest

A16 = 1 << 20          # a fake, 16-byte aligned "device" address
ODD = A16 + 1          # no element's alignment
F32, BF16 = 0, 1
HUGE = 1 << 62


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_16_amd as g
    return g


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def conv(gdr, B=1, T=8, C=16, K=4, dt=BF16, x=A16, st=None, w=A16, b=A16, s0=None, flags=1,
         odt=BF16, y=A16, sf=None):
    return gdr.lib.gdr_short_conv_fwd(B, T, C, K, dt, x, st, w, b, s0, flags, odt, y, sf, None)


def conv_step(gdr, N=1, C=16, K=4, dt=BF16, x=A16, xs=16, w=A16, b=A16, s=A16, flags=1, odt=BF16,
              y=A16):
    return gdr.lib.gdr_short_conv_step(N, C, K, dt, x, xs, w, b, s, flags, odt, y, None)


def conv_bwd(gdr, B=1, T=8, C=16, K=4, dt=BF16, x=A16, w=A16, b=A16, s0=None, ddt=BF16, dy=A16,
             st=None, dsf=None, flags=1, gdt=F32, dx=A16, dw=A16, db=A16, ds0=None, ws=A16,
             nb=1 << 30):
    return gdr.lib.gdr_short_conv_bwd(B, T, C, K, dt, x, w, b, s0, ddt, dy, st, dsf, flags, gdt, dx,
                                      dw, db, ds0, ws, nb, None)


def scan(gdr, B=1, T=8, D=16, G=1, N=16, dt=BF16, x=A16, d=A16, A=A16, Bm=A16, Cm=A16, D_=None,
         z=None, b=None, h0=None, st=None, flags=1, odt=BF16, y=A16, hf=None, ws=None, nb=0):
    return gdr.lib.gdr_ssm_scan_fwd(B, T, D, G, N, dt, x, d, A, Bm, Cm, D_, z, b, h0, st, flags,
                                    odt, y, hf, ws, nb, None)


def step(gdr, B=1, D=16, G=1, N=16, dt=BF16, x=A16, d=A16, A=A16, Bm=A16, Cm=A16, D_=None, z=None,
         b=None, s=A16, st=None, flags=1, odt=BF16, y=A16):
    return gdr.lib.gdr_ssm_step(B, D, G, N, dt, x, d, A, Bm, Cm, D_, z, b, s, st, flags, odt, y,
                                None)


def scan_bwd(gdr, B=1, T=8, D=16, G=1, N=16, dt=BF16, x=A16, d=A16, A=A16, Bm=A16, Cm=A16, D_=None,
             z=None, b=None, h0=None, odt=BF16, do=A16, dh=None, st=None, flags=1, gdt=F32, dx=A16,
             dd=A16, dA=A16, dB=A16, dC=A16, dD=None, dz=None, db=None, dh0=None, ws=A16,
             nb=1 << 40):
    return gdr.lib.gdr_ssm_scan_bwd(B, T, D, G, N, dt, x, d, A, Bm, Cm, D_, z, b, h0, odt, do, dh,
                                    st, flags, gdt, dx, dd, dA, dB, dC, dD, dz, db, dh0, ws, nb,
                                    None)


def norm(gdr, R=4, C=16, dt=BF16, x=A16, xs=16, rdt=BF16, r=None, rs=0, w=None, b=None, eps=1e-5,
         odt=BF16, y=A16, h=None):
    return gdr.lib.gdr_layer_norm_fwd(R, C, dt, x, xs, rdt, r, rs, w, b, eps, odt, y, h, None)


def norm_bwd(gdr, R=4, C=16, dt=BF16, x=A16, xs=16, w=None, ddt=BF16, dy=A16, ys=16, eps=1e-5,
             gdt=F32, dr=None, rs=0, dx=A16, dw=A16, db=A16, ws=A16, nb=1 << 30):
    return gdr.lib.gdr_layer_norm_bwd(R, C, dt, x, xs, w, ddt, dy, ys, eps, gdt, dr, rs, dx, dw, db,
                                      ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(x=ODD), 1), (dict(w=A16 + 2), 1),
    (dict(b=ODD), 1), (dict(s0=ODD), 1), (dict(sf=ODD), 1), (dict(y=ODD), 1), (dict(B=-1), 1),
    (dict(T=-1), 1), (dict(C=-1), 1), (dict(K=1), 2), (dict(K=5), 2), (dict(K=0), 2),
    (dict(dt=4), 2), (dict(odt=9), 2), (dict(flags=2), 2), (dict(st=strides(-1, 16)), 1),
    (dict(st=strides(1 << 41, 16)), 1), (dict(B=HUGE, T=HUGE), 1), (dict(B=1 << 24, C=1 << 16), 1),
])
def test_conv_fwd(gdr, kw, code):
    assert conv(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(s=None), 1), (dict(s=ODD), 1), (dict(y=None), 1), (dict(w=None), 1),
    (dict(N=-1), 1), (dict(K=6), 2), (dict(dt=3), 2), (dict(xs=-4), 1), (dict(flags=8), 2),
    (dict(N=1 << 31, C=1 << 20), 1),
])
def test_conv_step(gdr, kw, code):
    assert conv_step(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dy=ODD), 1),
    (dict(ws=None), 1), (dict(ws=A16 + 4), 1), (dict(nb=0), 1), (dict(ds0=ODD), 1),
    (dict(gdt=3), 2), (dict(ddt=3), 2), (dict(K=7), 2), (dict(st=strides(8, 8, -1, 8)), 1),
    (dict(T=-1), 1), (dict(flags=4), 2),
])
def test_conv_bwd(gdr, kw, code):
    assert conv_bwd(gdr, **kw) == code


SCAN_BAD = [
    (dict(x=None), 1), (dict(d=None), 1), (dict(A=None), 1), (dict(Bm=None), 1), (dict(Cm=None), 1),
    (dict(x=ODD), 1), (dict(z=ODD), 1), (dict(D_=ODD), 1), (dict(b=ODD), 1), (dict(B=-1), 1),
    (dict(D=-16), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(N=0), 1), (dict(N=65), 2),
    (dict(dt=2), 2), (dict(odt=2), 2), (dict(flags=2), 2),
]


@pytest.mark.parametrize("kw,code", SCAN_BAD + [
    (dict(y=None), 1), (dict(h0=ODD), 1), (dict(hf=ODD), 1), (dict(T=-1), 1),
    (dict(st=strides(*[16] * 9, -1)), 1), (dict(T=4096), 1), (dict(T=4096, ws=A16, nb=64), 1),
    (dict(B=1 << 20, T=1 << 20, D=1 << 20), 1), (dict(B=1 << 30, D=64), 1),
])
def test_scan_fwd(gdr, kw, code):
    assert scan(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", SCAN_BAD + [(dict(y=None), 1), (dict(s=None), 1),
                                                (dict(s=ODD), 1), (dict(B=1 << 31, D=256), 1),
                                                (dict(st=strides(1, 1, 1, 1, -1)), 1)])
def test_step(gdr, kw, code):
    assert step(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", SCAN_BAD + [
    (dict(do=None), 1), (dict(dx=None), 1), (dict(dd=None), 1), (dict(dA=None), 1),
    (dict(dB=None), 1), (dict(dC=None), 1), (dict(z=A16), 1), (dict(gdt=7), 2), (dict(ws=None), 1),
    (dict(nb=1), 1), (dict(dh=ODD), 1), (dict(st=strides(*[16] * 11, -1)), 1),
])
def test_scan_bwd(gdr, kw, code):
    assert scan_bwd(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(x=ODD), 1), (dict(w=ODD), 1), (dict(b=ODD), 1),
    (dict(r=A16), 1), (dict(r=ODD, h=A16), 1), (dict(R=-1), 1), (dict(C=-1), 1),
    (dict(C=(1 << 20) + 1), 2), (dict(dt=5), 2), (dict(rdt=5), 2), (dict(odt=5), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(xs=-1), 1), (dict(R=1 << 25), 1),
])
def test_norm_fwd(gdr, kw, code):
    assert norm(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dr=ODD), 1),
    (dict(ws=None), 1), (dict(nb=0), 1), (dict(ws=A16 + 8), 1), (dict(dw=ODD), 1), (dict(gdt=5), 2),
    (dict(ys=-1), 1), (dict(eps=-1.0), 1), (dict(R=-2), 1),
])
def test_norm_bwd(gdr, kw, code):
    assert norm_bwd(gdr, **kw) == code


def test_empty_calls_launch_nothing(gdr):
    none = dict(x=None, w=None, y=None, b=None)
    assert conv(gdr, B=0, **none) == 0 and conv(gdr, C=0, **none) == 0
    assert conv(gdr, T=0, **none) == 0
    assert conv_step(gdr, N=0, s=None, **none) == 0
    assert conv_bwd(gdr, C=0, x=None, ws=None) == 0
    assert conv_bwd(gdr, B=0, x=None, dw=None, db=None, ws=None) == 0
    assert scan(gdr, B=0, x=None) == 0 and scan(gdr, D=0, x=None) == 0
    assert scan(gdr, T=0, x=None, y=None) == 0
    assert step(gdr, B=0, x=None, s=None) == 0
    assert scan_bwd(gdr, D=0, dA=None) == 0
    assert norm(gdr, R=0, x=None, y=None) == 0 and norm(gdr, C=0, x=None) == 0
    assert norm_bwd(gdr, C=0, x=None) == 0
    assert norm_bwd(gdr, R=0, x=None, dw=None, db=None) == 0


def test_workspace_sizes(gdr):
    L = gdr.lib
    assert L.gdr_short_conv_bwd_workspace_size(0, 8, 16, 4) == 0
    assert L.gdr_short_conv_bwd_workspace_size(1, 8, 16, 9) == 0
    assert L.gdr_short_conv_bwd_workspace_size(1, 8, 16, 4) >= 16 * 5 * 4
    assert L.gdr_ssm_scan_fwd_workspace_size(1, 1, 2048, 1, 16) == 0
    assert L.gdr_ssm_scan_fwd_workspace_size(1, 32768, 2048, 1, 16) > 2048 * 16 * 4
    assert L.gdr_ssm_scan_fwd_workspace_size(1, 32768, 2048, 3, 16) == 0
    assert L.gdr_ssm_scan_bwd_workspace_size(1, 64, 32, 1, 65) == 0
    # a kept state in 16 tokens, and the partials of dB and dC
    assert L.gdr_ssm_scan_bwd_workspace_size(2, 64, 32, 1, 16) >= 2 * 4 * 32 * 16 * 4 + \
        2 * 64 * 32 * 4
    assert L.gdr_layer_norm_bwd_workspace_size(0, 8) == 0
    assert L.gdr_layer_norm_bwd_workspace_size(4, 1 << 21) == 0
    assert L.gdr_layer_norm_bwd_workspace_size(100, 2048) >= 2 * 2048 * 4


def test_binding_refuses_cpu_tensors(gdr):
    import torch
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: gdr.gdr_short_conv_fwd(x, w),
                 lambda: gdr.gdr_short_conv_step(x[0], w, None, x),
                 lambda: gdr.gdr_short_conv_bwd(x, w, None, None, x),
                 lambda: gdr.gdr_ssm_scan_fwd(x, x, w, x, x),
                 lambda: gdr.gdr_layer_norm_fwd(x), lambda: gdr.gdr_layer_norm_bwd(x, None, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gdr.gdr_layer_norm_fwd([1.0])


B16 = A16 + 4096       # other fake addresses
C16 = A16 + 8192


@pytest.mark.parametrize("name,kw", [
    ("conv", dict(x=A16, y=A16)), ("conv", dict(s0=B16, y=B16)), ("conv", dict(y=B16, sf=A16)),
    ("conv", dict(y=B16, sf=B16, x=C16)), ("conv_step", dict(s=B16)), ("conv_step", dict(y=B16)),
    ("conv_bwd", dict(dy=B16)), ("conv_bwd", dict(dy=B16, dx=B16)),
    ("conv_bwd", dict(dy=B16, dx=C16, dsf=B16 + 64, ds0=B16 + 64)),
    ("scan", dict()), ("scan", dict(z=B16, y=B16)), ("scan", dict(h0=B16, y=B16)),
    ("step", dict(s=B16)), ("step", dict(s=B16, y=B16)),
    ("scan_bwd", dict(dx=B16, dd=B16 + 64, dB=B16 + 128)), ("scan_bwd", dict(do=B16, dx=B16)),
    ("norm", dict(r=B16, h=A16, y=C16, rs=16)), ("norm", dict(r=B16, h=C16, y=C16, rs=16)),
    ("norm", dict(r=B16, h=C16, y=B16, rs=16)), ("norm", dict(xs=32)), ("norm", dict(odt=F32)),
    ("norm", dict(y=C16, r=B16, h=B16, rs=32)), ("norm_bwd", dict(dy=B16)),
    ("norm_bwd", dict(dy=B16, dx=B16)), ("norm_bwd", dict(dy=B16, dx=C16, dr=C16, rs=32)),
])
def test_outputs_at_inputs(gdr, name, kw):
    """What cannot be done in place is refused, not done wrongly."""
    assert globals()[name](gdr, **kw) == 1


def test_conv_bwd_of_more_channels_than_its_sums_launch(gdr):
    """The sums of dw over 2^28 channels would not fit a launch: refused before
    anything runs."""
    C = 1 << 28
    need = gdr.gdr_short_conv_bwd_workspace_size(1, 1, C, 4)
    assert conv_bwd(gdr, B=1, T=1, C=C, dy=B16, dx=C16, nb=need) == 1


def test_header_and_library_agree(gdr):
    """Every function that gdr_block.h declares is exported, and bound under its
    own name where it is a call of the user's; constants are the binding's."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                        "gdr_block.h")
    src = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    names = re.findall(r"^(?:gdr_status_t|size_t)\s+(gdr_[a-z_]+)\s*\(", src, flags=re.M)
    assert len(names) == 12
    for n in names:
        assert getattr(gdr.lib, n) and callable(getattr(gdr, n)) and n in gdr.__all__
    for name, value in re.findall(r"#define (GDR_[A-Z_]+) (\d+)u?$", src, flags=re.M):
        assert getattr(gdr, name) == int(value), name
