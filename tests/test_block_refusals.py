"""What the operators around the mixer refuse before anything runs, beside the
checks of test_block_api (CPU: fake device addresses, no call here may reach a
launch)."""
import pytest

from test_block_api import (A16, B16, BF16, C16, F32, conv, conv_bwd, conv_step, gdr,  # noqa: F401
                            norm, norm_bwd, scan, scan_bwd, step)


@pytest.mark.parametrize("R,C", [(1 << 23, 8193), (1 << 23, 16384), (1 << 23, 8200),
                                 (1 << 24, 10000), (1 << 24, 8192), (1 << 24, 7)])
def test_norm_of_more_rows_than_a_launch_holds(gdr, R, C):
    """A workgroup per row, of 512 threads from 8193 to 16384 channels: 2^32
    work-items are refused, not handed to a launch that fails."""
    assert norm(gdr, R=R, C=C, xs=C, y=B16) == 1


# ---- an output (or the workspace) where another tensor of the call starts -------------
#
# Every tensor has an address of its own, all arguments are valid, and one output
# at a time is put on each other tensor in turn.


def at(names):
    return {n: A16 + 4096 * (k + 1) for k, n in enumerate(names.split())}


CALLS = {
    # call, fixed arguments, inputs, outputs, pairs that may be one buffer
    "conv": (conv, dict(), "x w b s0", "y sf", {("sf", "s0")}),
    "conv_step": (conv_step, dict(), "x w b", "s y", set()),
    "conv_bwd": (conv_bwd, dict(), "x w b s0 dy dsf", "dx dw db ds0 ws", set()),
    "norm": (norm, dict(rs=16), "x r w b", "y h", {("y", "x"), ("h", "r")}),
    "norm_bwd": (norm_bwd, dict(rs=16), "x w dy dr", "dx dw db ws", {("dx", "dr")}),
    # 512 tokens of 16 channels: segments, and a workspace
    "scan": (scan, dict(T=512, nb=1 << 40), "x d A Bm Cm D_ z b h0", "y hf ws", {("hf", "h0")}),
    "step": (step, dict(), "x d A Bm Cm D_ z b", "s y", set()),
    "scan_bwd": (scan_bwd, dict(), "x d A Bm Cm D_ z b h0 do dh",
                 "dx dd dA dB dC dD dz db dh0 ws", set()),
}


def pairs():
    for name, (_, _, ins, outs, same) in CALLS.items():
        for o in outs.split():
            for p in (ins + " " + outs).split():
                if o != p and (o, p) not in same:
                    yield name, o, p


@pytest.mark.parametrize("name,out,other", list(pairs()))
def test_outputs_on_other_tensors(gdr, name, out, other):
    call, kw, ins, outs, _ = CALLS[name]
    where = at(ins + " " + outs)
    where[out] = where[other]
    assert call(gdr, **{**kw, **where}) == 1


def test_the_workspace_of_segments_is_needed(gdr):
    assert gdr.gdr_ssm_scan_fwd_workspace_size(1, 512, 16, 1, 16) > 0


@pytest.mark.parametrize("name,sizes,call,kw", [
    ("gdr_short_conv_bwd_workspace_size", (1, 1, 1 << 28, 4), conv_bwd,
     dict(B=1, T=1, C=1 << 28, dy=B16, dx=C16)),
    ("gdr_short_conv_bwd_workspace_size", (1 << 31, 1 << 31, 1, 4), conv_bwd,
     dict(B=1 << 31, T=1 << 31, C=1, dy=B16, dx=C16)),
    ("gdr_layer_norm_bwd_workspace_size", ((1 << 24) + 1, 16), norm_bwd,
     dict(R=(1 << 24) + 1, dy=B16, dx=C16)),
    ("gdr_ssm_scan_bwd_workspace_size", (1 << 30, 1, 64, 1, 16), scan_bwd,
     dict(B=1 << 30, T=1, D=64)),
    ("gdr_ssm_scan_fwd_workspace_size", (1 << 30, 1, 64, 1, 16), scan,
     dict(B=1 << 30, T=1, D=64, y=B16)),
])
def test_no_workspace_for_what_is_refused(gdr, name, sizes, call, kw):
    """Sizes that the call refuses need no workspace, so nobody allocates one."""
    assert getattr(gdr.lib, name)(*sizes) == 0
    assert call(gdr, **kw) == 1
