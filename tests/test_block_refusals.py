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
