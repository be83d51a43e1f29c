"""Waits of the cache's attention kernels, read from their source: none is decided by a lane alone.

A wait that runs out is seen by each lane for itself (clock and abort flag). Where lanes of one warp, or the two warps of a
row, act on it apart, some of them end and the others stay at the next collective operation; that shows only when a wait runs
out, so it is looked for in the source.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_sequence_flash_gb300", "csrc")
# A barrier's vote, or a value that is only ever handed to one.
VOTED = [r"both\(wait_bar\(", r"consumers_all\(wait_bar\(", r"const bool up = wait_bar\("]


@pytest.mark.parametrize("name", ["cache_prompt.cuh", "cache_attn.cuh"])
def test_waits_are_voted_on(name):
    with open(os.path.join(CSRC, name)) as fh:
        text = re.sub(r"//[^\n]*", "", fh.read())
    voted = sum(len(re.findall(v, text)) for v in VOTED)
    assert voted and voted == len(re.findall(r"\bwait_bar\(", text))
    assert ("bool up =" in text) == ("both(up)" in text)  # the vote of the softmax's wait for its scores
    assert re.search(r"\bwait_bar_warp\(", text)


def test_the_vote_is_one():
    with open(os.path.join(CSRC, "common.cuh")) as fh:
        text = fh.read()
    body = text[text.index("bool wait_bar_warp("):]
    assert "__all_sync(0xffffffffu, wait_bar(bar, parity, c))" in body[:body.index("\n}\n")]


def test_a_short_limit_does_not_cut_the_drain():
    """What is under way when a block gives up ends within a limit that the caller's does not shorten."""
    with open(os.path.join(CSRC, "common.cuh")) as fh:
        text = fh.read()
    assert float(re.search(r"kDrainLimitNs = (\d+);", text).group(1)) >= 1e8
    body = text[text.index("void wait_bar_drain("):]
    body = body[:body.index("\n}\n")]
    assert "limit_ns > kDrainLimitNs ? limit_ns : kDrainLimitNs" in body and "- t0 > limit)" in body
