"""What orders one CTA's work before another's in the kernels of CTA pairs, read from their sources.

An arrival on the other CTA's barrier in the default scope orders no shared memory that this CTA wrote: not even stores that a
fence has handed to the async proxy.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_block_scaled_04_gb300", "csrc")


def source(name):
    """A file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def statements_before(text, at, count):
    """The last `count` statements that end before position `at`."""
    return [s.strip() for s in re.split(r"[;{}]", text[:at])[-count - 1:-1]]


PAIRS = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cuh") and n != "tcgen05.cuh" and "mbar_arrive_peer" in source(n)]


def test_the_pair_kernels_are_found():
    assert {"mxfp4_pair.cuh", "mxfp8_pair.cuh"} <= set(PAIRS)


@pytest.mark.parametrize("name", PAIRS)
def test_no_arrival_stands_for_stores(name):
    text = source(name)
    for m in re.finditer(r"mbar_arrive_peer\(", text):
        assert not any("fence_proxy_async" in s for s in statements_before(text, m.start(), 3)), text[m.start() - 200:m.end() + 40]


@pytest.mark.parametrize("name", PAIRS)
def test_arrivals_follow_the_accumulators_reads(name):
    """Every arrival that frees accumulators comes behind the fence that orders this thread's reads of them."""
    text = source(name)
    for m in re.finditer(r"mbar_arrive_peer\(", text):
        assert "tc_fence_before()" in statements_before(text, m.start(), 3), text[m.start() - 200:m.end() + 40]
