"""The upper end of attention's range of scales, on the host (no GPU)."""

import hadamard_rotated_int8_amd as cr
import test_attention_boundary as boundary


def test_scales_that_overflow_are_refused():
    assert boundary._apply(scale=2.3e38) == cr.OK
    for scale in (2.36e38, 3e38, 3.4e38):
        assert boundary._apply(scale=scale) == cr.ERR_UNSUPPORTED
