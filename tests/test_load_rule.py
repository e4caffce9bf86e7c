"""Which loads may go through the read-only path, checked on the sources.

Every kernel of the library lets its successor on the stream become resident
before it has finished, so a grid may be there while the one in front still
writes what it will read.  ld.global.nc (`__ldg`, `ld_stream16`) asks for data
that nothing writes during a grid's whole life: it may serve weights, never
what an earlier call of the library may have written."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "expert_routing_alignment_gb300", "csrc")
READ_ONLY = r"__ldg|ld_stream16|ld\.global\.nc"


def code(name: str) -> str:
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_row_kernels_take_no_read_only_loads():
    """Their rows, scales, tables and weights are all a call's own buffers."""
    for name in ("dispatch.cu", "rmsnorm.cu", "route_grad.cu", "rows.cuh"):
        assert not re.search(READ_ONLY, code(name)), name
