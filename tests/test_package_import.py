"""The package imports on a torch without the E8M0 type (CPU): only what makes or takes such scales
needs it."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import torch
del torch.float8_e8m0fnu
import hadamard_rotated_int8_amd as cr
from hadamard_rotated_int8_amd import block
assert callable(cr.pack_activations) and callable(cr.block_norm) and callable(cr.rope)
assert cr.rope_plan(8, device="cpu").inv_freq.shape == (4,)
try:
    block._new_activation(4, 128, torch.device("cpu"))
except RuntimeError as e:
    assert "float8_e8m0fnu" in str(e), e
else:
    raise AssertionError("no error")
print("imported")
"""


def test_import_without_the_e8m0_type():
    r = subprocess.run([sys.executable, "-c", WITHOUT], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]


def test_the_type_is_used_where_it_is_there():
    torch = pytest.importorskip("torch")
    from hadamard_rotated_int8_amd import block

    a = block._new_activation(5, 300, torch.device("cpu"))
    assert a.scale.dtype == torch.float8_e8m0fnu and a.scale.shape == (5, 3) and a.scale.stride() == (1, 8)
