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
