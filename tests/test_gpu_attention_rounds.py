"""Which last rounds of tiles have their keys split (GPU)."""

import pytest
import torch

import hadamard_rotated_int8_amd as cr
from kernel_names import launched
from test_gpu_attention import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m, l, heads, d, split", [
    (2304, 12288, 40, 128, True), (2304, 12287, 40, 128, False), (2304, 12288, 40, 96, True),
    (2304, 12288, 40, 64, False), (4095, 12288, 40, 64, True), (2688, 12288, 40, 128, False),
    (1664, 1100, 40, 64, True), (1664, 1100, 40, 128, True), (2304, 1100, 20, 160, True)])
def test_last_rounds(m, l, heads, d, split):
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the rule goes by the compute units")
    q, k, v = _inputs(1, m, l, heads, heads, d, seed=l)
    names = launched(lambda: cr.attention(q, k, v))
    assert len(names) == 1 + split and names[0].startswith("attention_kernel")
    assert names[1:] == ["attention_join_kernel"] * split
    out = cr.attention(q, k, v)
    at, rows = [heads - 1], slice(m - 130, m)  # (among the tiles that are split)
    _check(q[:, rows, at], k[:, :, at], v[:, :, at], out[:, rows, at])
