"""Rules that decide the order of sums take the call's sizes alone.  No GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deterministic_w8a8_int8_gb300", "csrc")


@pytest.mark.parametrize("name", ["linear_w4g.cu", "kv_plan.cuh"])
def test_cuts_do_not_ask_the_device(name):
    """Slices of K and pieces of keys are cut for a fixed number of SMs."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "kSms" in text and "sm_count" not in text
