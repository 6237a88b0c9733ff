"""Which of the library's kernels a call launches."""

import re

import pytest
import torch
from torch.profiler import ProfilerActivity, profile


def launched(call):
    """The names of the library's kernels that call() launches, without their arguments."""
    with profile(activities=[ProfilerActivity.CUDA]) as trace:
        call()
        torch.cuda.synchronize()
    if not trace.events():
        pytest.skip("nothing is recorded (another profiler is at work?)")
    found = [re.search(r"convrot::(\w+(?:<[^>]*>)?)\(", e.name.replace("(anonymous namespace)::", "")) for e in trace.events()]
    return [m[1] for m in found if m]
