"""Refusals of rotary calls whose tensors lie over one another (no GPU needed)."""

import pytest

import hadamard_rotated_int8_amd as cr
import test_block_boundary as boundary

FAKE = boundary.FAKE


@boundary.cpu_only
@pytest.mark.parametrize("t", [
    [dict(x=FAKE, y=FAKE + 0x1000), dict(x=FAKE + 0x1000, y=FAKE)],            # exchanged
    [dict(x=FAKE, y=FAKE), dict(x=FAKE + 0x1000, y=FAKE)],                     # the second over the first
    [dict(x=FAKE, y=FAKE + 0x2000), dict(x=FAKE + 0x1000, y=FAKE + 0x2000)],   # one place for both
    [dict(x=FAKE, y=FAKE), dict(x=FAKE, y=FAKE)]])                             # turned twice, or once
def test_rope_outputs_over_other_tensors_are_refused(t):
    assert boundary._rope(t=t, count=2) == cr.ERR_UNSUPPORTED
