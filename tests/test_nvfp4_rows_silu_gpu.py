"""Gate and up of four-bit rows where the gate is far below zero, whose SiLU
leaves fp32's normal numbers.  Tolerances as in test_nvfp4_rows_gpu."""
from __future__ import annotations

import pytest
import torch

import expert_routing_alignment_gb300 as moe
from tests.test_nvfp4_rows_gpu import FL, U, align

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("power", [0, 40, 100])
def test_gates_down_to_where_silu_leaves_fp32(rows, power):
    """silu(g) * u for gates of one product each, which are exact, and u = 2^power.
    In units of U = 2^-24: two for e^-|g|, one each for its product with g and for
    the denominator 1 + e^-|g|, two for the reciprocal, one each for its product and
    for that with u, 8 in all.  Where e^-|g| and silu are below fp32's normal numbers:
    a unit of the least ones, 2^-149, for the exponential, which g multiplies, and half
    a one for each of two products."""
    scales = torch.arange(0x28, 0x73, dtype=torch.uint8)       # 1/4 to 160 by eighths of a power
    R, C = 4 * len(scales), 32
    t, n = align([rows], 1)

    def rows_of_one(k, code, scale):
        codes = torch.zeros(k, C // 2, dtype=torch.uint8, device="cuda")
        s = torch.zeros(k, 2, dtype=torch.uint8, device="cuda")
        codes[:, 0], s[:, 0] = code, scale
        return codes, s

    x = (*rows_of_one(rows, 2, 0x38), torch.ones(rows, device="cuda"))     # 1, then zeros
    code = torch.tensor([2, 3, 10, 11], dtype=torch.uint8, device="cuda").repeat(len(scales))
    gc, gs = rows_of_one(R, code, scales.cuda().repeat_interleave(4))
    uc, us = rows_of_one(R, 2, 0x38)
    gate = gc[None], gs[None], torch.ones(1, device="cuda")
    up = uc[None], us[None], torch.full((1,), 2.0 ** power, device="cuda")
    out = moe.moe_grouped_gate_up_nvfp4(gate, up, x, t, 1, out_dtype=FL)
    mag = torch.tensor([1.0, 1.5, -1.0, -1.5], dtype=torch.float64, device="cuda")
    g = torch.repeat_interleave(scales.cuda().view(torch.float8_e4m3fn).double(), 4) * mag.repeat(
        len(scales))
    assert float(g.min()) == -240 and bool(((g > -88.7) & (g < -87.4)).any())
    h = g / (1.0 + torch.exp(-g)) * 2.0 ** power
    tol = 8 * U * h.abs() + (g.abs() + 1) * 2.0 ** (-149 + power)
    bad = ~((out.double() - h).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), g.expand_as(bad)[bad][:6], out[bad][:6],
                           h.expand_as(bad)[bad][:6])
