"""The four-bit kernels and the rule on read-only loads: rows, scales, tables and
weights may all be what the call ahead on the stream is still writing (a weight
set is quantised right before its first product), so none of their loads takes
the read-only path."""
from __future__ import annotations

import re

import pytest

from tests.test_load_rule import READ_ONLY, code


@pytest.mark.parametrize("name", ["nvfp4_pack.cu", "nvfp4.cuh", "nvfp4_grouped.cu"])
def test_four_bit_kernels_take_no_read_only_loads(name):
    assert not re.search(READ_ONLY, code(name))


def test_every_load_comes_after_the_wait_for_the_call_ahead():
    """Each kernel waits for its predecessor before the first use of a pointer:
    nothing but the setup of barriers and tensor memory stands ahead of it."""
    seen = 0
    for name in ("nvfp4_pack.cu", "nvfp4_grouped.cu"):
        for body in re.findall(r"__global__ void(.*?)\n}\n", code(name), re.S):
            head, wait, _ = body[body.index("{"):].partition("pdl_wait();")
            assert wait and not re.search(r"\ba\.(x|codes|scale|given|sti|offsets)\b\s*\[", head)
            seen += 1
    assert seen == 5
