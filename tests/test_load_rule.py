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


def test_layer_kernels_take_them_for_weights_alone():
    """No read-only load of the layer's kernels has the tokens' rows in its
    argument (x, or a row of it), but for the row form of the FP8 tensor-core
    kernel: that one is never resident before x is final, by the launch that
    its entry points ask for."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        name = os.path.basename(path)
        text = code(name)
        for m in re.finditer(r"\b(?:__ldg|ld_stream16)\s*\(", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            arg = text[m.end(): end - 1]
            seen += 1
            if name == "verify_tc.cu" and "xr + c" in arg:
                continue
            assert not re.search(r"(?<![\w.])(?:a\.|p\.)?(?:x|xr|xs|y|h)\b", arg), (name, arg)
    assert seen > 20
    assert re.search(r"launch_coop\(\s*x_final \|\| a\.tok\s*,\s*verify_ffn_kernel",
                     code("verify_tc.cu"))
    # the layer's alignment stands between x and the kernel; the expert half may
    # follow whatever wrote x
    calls = re.findall(r"moe::run_experts\([^;]*?v, (\w+), err_word", code("layer.cu"))
    assert calls == ["true", "false"]
