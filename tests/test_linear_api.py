"""Argument checks of linear attention, rotary positions and RMS norm, on the CPU:
nothing is launched (fake device addresses, and calls that end before a launch)."""
import ctypes
import os
import re

import pytest

A = [(i + 1) << 20 for i in range(20)]     # fake, 16-byte aligned "device" addresses
ODD = A[0] + 1                             # no element's alignment
F32, BF16 = 0, 1
HUGE = 1 << 62
SOME = 1 << 30


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_16_amd as g
    return g


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def fwd(gdr, B=1, T=8, H=4, Hk=2, Dk=16, Dv=24, dt=BF16, q=A[0], k=A[1], v=A[2], st=None, g=A[3],
        s0=A[4], scale=1.0, flags=0, odt=BF16, o=A[5], sf=A[6], ws=A[7], nb=SOME):
    return gdr.lib.gdr_linear_attn_fwd(B, T, H, Hk, Dk, Dv, dt, q, k, v, st, g, s0, scale, flags,
                                       odt, o, sf, ws, nb, None)


def step(gdr, N=1, H=4, Hk=2, Dk=16, Dv=24, dt=BF16, q=A[0], k=A[1], v=A[2], st=None, g=A[3],
         s=A[4], scale=1.0, flags=0, odt=BF16, o=A[5]):
    return gdr.lib.gdr_linear_attn_step(N, H, Hk, Dk, Dv, dt, q, k, v, st, g, s, scale, flags, odt,
                                        o, None)


def bwd(gdr, B=1, T=8, H=4, Hk=2, Dk=16, Dv=24, dt=BF16, q=A[0], k=A[1], v=A[2], st=None, g=A[3],
        s0=A[4], do=A[5], ds=A[6], scale=1.0, flags=0, gdt=F32, dq=A[7], dk=A[8], dv=A[9],
        dg=A[10], ds0=A[11], ws=A[12], nb=SOME):
    return gdr.lib.gdr_linear_attn_bwd(B, T, H, Hk, Dk, Dv, dt, q, k, v, st, g, s0, do, ds, scale,
                                       flags, gdt, dq, dk, dv, dg, ds0, ws, nb, None)


def rot(gdr, B=2, T=8, Hq=4, Hk=2, D=16, r=16, dt=BF16, q=A[0], k=A[1], st=None, pos=A[2], ps=8,
        start=0, f=A[3], scale=1.0, flags=0, qo=A[4], ko=A[5]):
    return gdr.lib.gdr_rotary(B, T, Hq, Hk, D, r, dt, q, k, st, pos, ps, start, f, scale, flags, qo,
                              ko, None)


def norm(gdr, R=4, C=64, dt=BF16, x=A[0], xs=64, rdt=BF16, r=None, rs=64, w=A[2], eps=1e-6,
         odt=BF16, y=A[3], h=None):
    return gdr.lib.gdr_rms_norm_fwd(R, C, dt, x, xs, rdt, r, rs, w, eps, odt, y, h, None)


def quant(gdr, R=4, C=64, dt=BF16, x=A[0], xs=64, rdt=BF16, r=None, rs=64, w=A[2], eps=1e-6,
          kind=0, group=32, y=A[3], sc=A[4], h=None):
    return gdr.lib.gdr_rms_norm_quant(R, C, dt, x, xs, rdt, r, rs, w, eps, kind, group, y, sc, h,
                                      None)


def norm_bwd(gdr, R=4, C=64, dt=BF16, x=A[0], xs=64, w=A[1], ddt=BF16, dy=A[2], ys=64, eps=1e-6,
             gdt=F32, dr=None, rs=64, dx=A[3], dw=A[4], ws=A[5], nb=SOME):
    return gdr.lib.gdr_rms_norm_bwd(R, C, dt, x, xs, w, ddt, dy, ys, eps, gdt, dr, rs, dx, dw, ws,
                                    nb, None)


LA_BAD = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q=ODD), 1), (dict(k=ODD), 1),
    (dict(v=ODD), 1), (dict(g=A[3] + 2), 1), (dict(H=-1), 1), (dict(Hk=-1), 1), (dict(Hk=0), 1),
    (dict(Hk=3), 1), (dict(H=1 << 17, Hk=1), 1), (dict(Dk=-8), 1), (dict(Dk=0), 2),
    (dict(Dk=12), 2), (dict(Dv=4), 2), (dict(Dk=136), 2), (dict(Dv=256), 2), (dict(dt=2), 2),
    (dict(flags=2), 2),
]


@pytest.mark.parametrize("kw,code", LA_BAD + [
    (dict(odt=2), 2), (dict(B=-1), 1), (dict(T=-1), 1), (dict(o=None), 1), (dict(o=ODD), 1),
    (dict(s0=A[4] + 2), 1), (dict(sf=A[6] + 1), 1), (dict(B=HUGE, T=HUGE), 1),
    (dict(T=1 << 41), 1), (dict(B=1 << 22, H=16), 1),
    (dict(st=i64(*[64] * 8, -1)), 1), (dict(st=i64(1 << 41, *[64] * 8)), 1),
    (dict(st=i64(64, (1 << 23) + 1, *[64] * 7)), 1),
    # outputs where inputs or other outputs are
    (dict(o=A[0]), 1), (dict(o=A[2]), 1), (dict(o=A[3]), 1), (dict(o=A[4]), 1), (dict(o=A[6]), 1),
    (dict(sf=A[1]), 1), (dict(sf=A[3]), 1),
    # segments: a workspace that is missing, small, not aligned, or another tensor
    (dict(T=32768, ws=None), 1), (dict(T=32768, nb=64), 1), (dict(T=32768, ws=A[7] + 4), 1),
    (dict(T=32768, ws=A[0]), 1), (dict(T=32768, ws=A[4]), 1), (dict(T=32768, ws=A[5]), 1),
    (dict(T=32768, ws=A[6]), 1),
])
def test_linear_attn_fwd(gdr, kw, code):
    assert fwd(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", LA_BAD + [
    (dict(odt=2), 2), (dict(N=-1), 1), (dict(s=None), 1), (dict(s=A[4] + 1), 1), (dict(o=None), 1),
    (dict(o=ODD), 1), (dict(st=i64(64, 64, 64, 64, 64, -1)), 1), (dict(o=A[0]), 1),
    (dict(o=A[4]), 1), (dict(s=A[1]), 1), (dict(N=1 << 40), 1), (dict(N=1 << 24, H=512, Hk=1), 1),
])
def test_linear_attn_step(gdr, kw, code):
    assert step(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", LA_BAD + [
    (dict(gdt=2), 2), (dict(B=-1), 1), (dict(T=-1), 1), (dict(do=None), 1), (dict(do=ODD), 1),
    (dict(ds=A[6] + 1), 1), (dict(s0=A[4] + 1), 1), (dict(dq=None), 1), (dict(dk=None), 1),
    (dict(dv=None), 1), (dict(dv=ODD), 1), (dict(dg=A[10] + 2), 1), (dict(ds0=A[11] + 1), 1),
    (dict(g=None), 1), (dict(ws=None), 1), (dict(ws=A[12] + 8), 1), (dict(nb=64), 1),
    (dict(B=1 << 22, H=16), 1), (dict(st=i64(*[64] * 11, -1)), 1),
    (dict(st=i64(*[64] * 10, (1 << 23) + 1, 64)), 1),
    (dict(dq=A[0]), 1), (dict(dk=A[1]), 1), (dict(dv=A[5]), 1), (dict(dk=A[7]), 1),
    (dict(dg=A[3]), 1), (dict(ds0=A[6]), 1), (dict(ds0=A[4]), 1), (dict(ws=A[9]), 1),
    (dict(ws=A[2]), 1),
])
def test_linear_attn_bwd(gdr, kw, code):
    assert bwd(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(f=None), 1),
    (dict(q=ODD), 1), (dict(ko=ODD), 1), (dict(pos=A[2] + 4), 1), (dict(f=A[3] + 4), 1),
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(Hk=-1), 1), (dict(D=-1), 1),
    (dict(D=1025), 2), (dict(r=0), 1), (dict(r=-2), 1), (dict(r=7), 1), (dict(r=18), 1),
    (dict(dt=3), 2), (dict(flags=4), 2), (dict(ps=-1), 1), (dict(st=i64(*[64] * 11, -1)), 1),
    (dict(Hq=HUGE, Hk=HUGE), 1), (dict(Hq=65536), 1), (dict(B=HUGE, T=HUGE), 1),
    (dict(B=1 << 25, Hq=512), 1),
    (dict(qo=A[1]), 1), (dict(ko=A[0]), 1), (dict(ko=A[4]), 1), (dict(qo=A[2]), 1),
    (dict(ko=A[3]), 1),
    # in place with other strides
    (dict(qo=A[0], st=i64(512, 64, 16, 256, 32, 16, 1024, 128, 16, 256, 32, 16)), 1),
    (dict(ko=A[1], st=i64(512, 64, 16, 256, 32, 16, 512, 64, 16, 512, 64, 16)), 1),
    # heads, tokens or sequences of an output that share memory
    (dict(st=i64(512, 64, 16, 256, 32, 16, 512, 64, 0, 256, 32, 16)), 1),
    (dict(st=i64(512, 64, 16, 256, 32, 16, 512, 64, 8, 256, 32, 16)), 1),
    (dict(st=i64(512, 64, 16, 256, 32, 16, 512, 64, 16, 256, 0, 16)), 1),
    (dict(st=i64(512, 64, 16, 256, 32, 16, 504, 64, 16, 256, 32, 16)), 1),
    (dict(st=i64(0, 64, 16, 256, 32, 16, 0, 64, 16, 256, 32, 16)), 1),
])
def test_rotary(gdr, kw, code):
    assert rot(gdr, **kw) == code


NORM_BAD = [
    (dict(x=None), 1), (dict(y=None), 1), (dict(x=ODD), 1), (dict(w=A[2] + 2), 1),
    (dict(r=A[5]), 1), (dict(h=A[6]), 1), (dict(r=ODD, h=A[6]), 1), (dict(r=A[5], h=ODD), 1),
    (dict(R=-1), 1), (dict(C=-1), 1), (dict(C=(1 << 20) + 32), 2), (dict(dt=5), 2),
    (dict(rdt=5), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(xs=-1), 1), (dict(rs=-1), 1), (dict(R=1 << 25), 1), (dict(R=HUGE), 1), (dict(y=A[2]), 1),
    (dict(r=A[5], h=A[0]), 1), (dict(r=A[5], h=A[2]), 1), (dict(r=A[5], h=A[6], y=A[5]), 1),
    (dict(r=A[5], h=A[3]), 1), (dict(r=A[5], h=A[5], rs=128), 1),
]


@pytest.mark.parametrize("kw,code", NORM_BAD + [
    (dict(odt=5), 2), (dict(y=ODD), 1), (dict(y=A[0], odt=F32), 1), (dict(y=A[0], xs=128), 1),
])
def test_rms_norm_fwd(gdr, kw, code):
    assert norm(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", NORM_BAD + [
    (dict(kind=2), 2), (dict(group=16), 2), (dict(group=128), 1), (dict(group=-32), 2),
    (dict(sc=None), 1), (dict(sc=A[4] + 2), 1), (dict(y=A[0]), 1), (dict(sc=A[3]), 1),
    (dict(sc=A[0]), 1), (dict(r=A[5], h=A[4]), 1),
])
def test_rms_norm_quant(gdr, kw, code):
    assert quant(gdr, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(x=ODD), 1), (dict(dy=ODD), 1),
    (dict(dr=ODD), 1), (dict(w=A[1] + 2), 1), (dict(ws=None), 1), (dict(nb=0), 1),
    (dict(ws=A[5] + 8), 1), (dict(dw=ODD), 1), (dict(gdt=5), 2), (dict(ddt=5), 2), (dict(dt=5), 2),
    (dict(ys=-1), 1), (dict(xs=-1), 1), (dict(rs=-1), 1), (dict(eps=-1.0), 1), (dict(R=-2), 1),
    (dict(C=(1 << 20) + 1), 2), (dict(R=1 << 25), 1), (dict(dx=A[0]), 1), (dict(dx=A[2]), 1),
    (dict(dw=A[1]), 1), (dict(dw=A[3]), 1), (dict(ws=A[0]), 1), (dict(ws=A[4]), 1),
    (dict(dr=A[3], rs=128), 1), (dict(dr=A[4]), 1),
])
def test_rms_norm_bwd(gdr, kw, code):
    assert norm_bwd(gdr, **kw) == code


def test_empty_calls_launch_nothing(gdr):
    none = dict(q=None, k=None, v=None, o=None, g=None)
    assert fwd(gdr, B=0, **none) == 0 and fwd(gdr, H=0, Hk=0, **none) == 0
    assert fwd(gdr, T=0, sf=None, **none) == 0 and fwd(gdr, T=0, s0=A[4], sf=A[4], **none) == 0
    assert step(gdr, N=0, s=None, **none) == 0 and step(gdr, H=0, s=None, **none) == 0
    gone = dict(q=None, k=None, v=None, do=None, dq=None, dk=None, dv=None, ws=None)
    assert bwd(gdr, H=0, Hk=0, **gone) == 0 and bwd(gdr, B=0, **gone) == 0
    assert bwd(gdr, T=0, ds0=None, **gone) == 0 and bwd(gdr, T=0, ds0=A[6], **gone) == 0
    away = dict(q=None, k=None, f=None, qo=None, ko=None, pos=None)
    assert rot(gdr, B=0, **away) == 0 and rot(gdr, T=0, **away) == 0
    assert rot(gdr, Hq=0, Hk=0, **away) == 0
    for call in (norm, quant):
        assert call(gdr, R=0, x=None, y=None) == 0 and call(gdr, C=0, x=None, y=None) == 0
    assert norm_bwd(gdr, C=0, x=None, dy=None, dx=None, ws=None) == 0
    assert norm_bwd(gdr, R=0, x=None, dy=None, dx=None, dw=None) == 0


def test_workspace_sizes(gdr):
    L = gdr.lib
    size = L.gdr_linear_attn_fwd_workspace_size

    def back(*a, flags=0):
        return L.gdr_linear_attn_bwd_workspace_size(*a, flags)

    assert size(1, 64, 4, 64, 64, BF16) == 0            # one segment
    assert size(1, 32768, 4, 64, 64, BF16) >= 4 * 4 * 64 * 64
    for a in ((-1, 64, 4, 64, 64, 1), (1, 32768, 4, 60, 64, 1), (1, 32768, 4, 64, 136, 1),
              (1, 32768, 1 << 17, 64, 64, 1), (1, 32768, 4, 64, 64, 3), (0, 32768, 4, 64, 64, 1),
              (1, 0, 4, 64, 64, 1), (HUGE, HUGE, 4, 64, 64, 1)):
        assert size(*a) == 0, a
    # the state at the end of the only block (its gradient is ds_final), the decay's
    # partial sums, dq and dk per head
    assert back(2, 100, 4, 4, 64, 32, BF16) >= 4 * 2 * 4 * 64 * 32 + 8 * 2 * 100 * 4 * 4
    assert back(2, 100, 4, 2, 64, 32, BF16) >= \
        back(2, 100, 4, 4, 64, 32, BF16) + 8 * 2 * 100 * 4 * 64
    # a decay per head: states at every 256 tokens in place of 512
    assert back(64, 4096, 4, 4, 64, 32, BF16, flags=1) >= \
        back(64, 4096, 4, 4, 64, 32, BF16) + 2 * 8 * 4 * 256 * 64 * 32
    assert back(2, 100, 4, 4, 64, 32, BF16, flags=2) == 0
    for a in ((2, 100, 4, 3, 64, 32, 1), (2, 100, 4, 0, 64, 32, 1), (2, 100, 4, 4, 64, 30, 1),
              (2, -5, 4, 4, 64, 32, 1), (2, 100, 4, 4, 64, 32, 2), (0, 100, 4, 4, 64, 32, 1),
              (2, 0, 4, 4, 64, 32, 1), (HUGE, HUGE, 4, 4, 64, 32, 1), (2, 100, 0, 0, 64, 32, 1)):
        assert back(*a) == 0, a
    assert L.gdr_rms_norm_bwd_workspace_size(0, 8) == 0
    assert L.gdr_rms_norm_bwd_workspace_size(4, 1 << 21) == 0
    assert L.gdr_rms_norm_bwd_workspace_size(100, 2048) >= 2048 * 4


def test_binding_refuses_cpu_tensors(gdr):
    import torch
    x, f = torch.zeros(1, 4, 2, 8), torch.zeros(4, dtype=torch.float64)
    for call in (lambda: gdr.gdr_linear_attn_fwd(x, x, x), lambda: gdr.gdr_rotary(x, x, 0, f),
                 lambda: gdr.gdr_linear_attn_step(x[0], x[0], x[0], None, x),
                 lambda: gdr.gdr_linear_attn_bwd(x, x, x, None, None, x),
                 lambda: gdr.gdr_rms_norm_fwd(x), lambda: gdr.gdr_rms_norm_quant(x),
                 lambda: gdr.gdr_rms_norm_bwd(x, None, x)):
        with pytest.raises(ValueError):
            call()
    for call in (gdr.gdr_linear_attn_fwd, gdr.gdr_linear_attn_step):
        with pytest.raises((TypeError, ValueError)):
            call(1, 2, 3, None, None)
    with pytest.raises(TypeError):
        gdr.gdr_rotary(None, None, 0, f)
    with pytest.raises(TypeError):
        gdr.gdr_rms_norm_quant([1.0])


def test_header_library_and_binding_agree(gdr):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                        "gdr_linear.h")
    text = open(path).read()
    names = set(re.findall(r"^(?:gdr_status_t|size_t) (gdr_\w+)\(", text, re.M))
    assert len(names) == 11
    for n in names:
        assert hasattr(gdr.lib, n) and n in gdr.__all__, n
    for c, v in re.findall(r"^#define (GDR_\w+) (\d+)u?$", text, re.M):
        assert getattr(gdr, c) == int(v), c
