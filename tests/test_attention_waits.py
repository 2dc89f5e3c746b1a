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


def test_a_key_group_out_of_time_counts_for_the_block():
    """FP32 prefill: the groups of a block hold parts of the same rows' keys,
    so that the rows are not valid when any group gave up."""
    s = source("lq_attn_prefill.cu")
    body = s[s.index("attn_prefill_f32(const"):s.index("int group_shift_of(")]
    loop_end = body.index("mbar_arrive(&empty[kg][1][buf])")
    joined = body.index("ok = __syncthreads_and(ok);")
    assert loop_end < joined < body.index("JLD")  # before the parts are handed over
    assert "dst[D] = ok ? top : NAN" in body[joined:] and "if (split == 1 && !ok) continue;" in body[joined:]


def test_copies_and_products_in_flight_outlive_no_block():
    """Before a block hands its shared memory on, or leaves it and its TMEM,
    whoever issued copies or products has waited for them, whatever the waits
    before returned."""
    decode = source("lq_attn_decode.cu")
    gave_up = decode[decode.index("if (!warp_wait(full + st, ph)) {"):]
    gave_up = gave_up[:gave_up.index("return;")]
    assert "for (int k = i; k < filled; ++k)" in gave_up and "bar_wait(full + st, ph)" in gave_up

    s = source("lq_attn_prefill.cu")
    f32 = s[s.index("attn_prefill_f32(const"):s.index("int group_shift_of(")]
    drain = f32.index("for (int i = it; i < sent[kg][v]; ++i) bar_wait(&full[kg][v][i % NBUF], i / NBUF & 1);")
    assert f32.index("mbar_arrive(&empty[kg][1][buf])") < drain < f32.index("__syncthreads_and(ok)")

    tc = s[s.index("attn_prefill_tc(const"):]
    load, rest = tc[tc.index("if (warp == T::kLoadWarp) {"):].split("} else if (warp == T::kMmaWarp) {")
    products, softmax = rest.split("} else if (warp < 4 * streams) {")
    assert "bar_wait(&bars.q_full, 0)" in load and "for (int i = max(0, fills - T::kSlots); i < fills; ++i) bar_wait(" in load
    last = products.rindex("mma_commit(")
    assert "all_done" in products[last:] and "bar_wait(&bars.all_done, 0)" in products[last:]
    # the parts of a split call are written after every warp has passed there
    assert softmax.index("operands_free()") < softmax.index("row[D] =")
    assert "if (warp >= 4 * streams) operands_free();" in softmax
