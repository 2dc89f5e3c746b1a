"""What the attention kernels do when a bounded wait expires, read from their
sources.  (No test makes a wait expire on a GPU: nothing in a call that the
library accepts does.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_attention_recurrent_int8_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["lq_attn_decode.cu", "lq_attn_prefill.cu"])
def test_an_expired_wait_has_one_outcome_for_the_warp(name):
    """Each lane reads the clock for itself, so the lanes of a warp may see a
    wait expire apart; what a wait returned is acted on after a vote only."""
    s = source(name)
    assert not re.findall(r"!\s*bar_wait\(", s)
    assert s.count("warp_wait(") > 0
