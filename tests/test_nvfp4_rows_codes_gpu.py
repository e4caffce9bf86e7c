"""Codes of the four-bit quantiser where a quotient x / t lies next to a border
between two codes, where x is a negative zero, and where a block's elements are
many powers of two apart: the very bytes of the definition

    t = fl(s g),  code = e2m1(fl(x / t)), ties to even, at most 6

whose rounded quotients the restatement takes from float64 divisions (a
quotient of fp32 numbers rounded to float64 and then to fp32 is the rounded
quotient).  Every comparison is equality."""
from __future__ import annotations

import pytest
import torch

import expert_routing_alignment_gb300 as moe
from tests.test_nvfp4_rows_gpu import ALL, BF, FL, HF, check_quantized, gen, randn, ref_quantize

pytestmark = pytest.mark.gpu

BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
# All 24-bit steps t for which some x has a quotient so near the middle between a
# border and its neighbour in fp32 that a reciprocal one unit off, corrected by
# one residual, or one Newton step from it, rounds it to the other side (by a
# search over every t and border, with the floats around border * t).
STEPS = (12582909, 16777209, 16777210, 16777211, 16777212, 16777213, 16777214, 16777215)


def nibbles(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def check_bytes(q, x, given=None):
    """The codes' own bits, the sign of zeros among them."""
    code, s, _, _ = ref_quantize(x, given)
    a = code.abs()
    want = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4))
    live = torch.repeat_interleave(s > 0, 16, -1)
    want = want + 8.0 * (torch.signbit(x) & live)
    got = nibbles(q["codes"]).double()
    bad = got != want
    assert not bad.any(), (int(bad.sum()), x[bad][:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("power", [-103, -41, -24, 0, 7, 76])
def test_quotients_next_to_a_border(power):
    lanes, given = [], []
    for t in STEPS + tuple(range(8388608, 8388612)) + tuple(range(12582912, 12582916)):
        g = t * 2.0 ** power
        for c in BORDERS:
            x = torch.tensor(c * g, dtype=torch.float64).float()
            near = [x]
            for _ in range(3):
                near = [torch.nextafter(near[0], torch.tensor(0.0)), *near,
                        torch.nextafter(near[-1], torch.tensor(3e38))]
            # 6 g first, so that the block's scale is 1 and its step g
            lanes.append([6.0 * g] + [float(v) for v in near] + [-float(v) for v in near] + [0.0])
            given.append(g)
    x = torch.tensor(lanes, dtype=torch.float64, device="cuda").float()
    given = torch.tensor(given, dtype=torch.float64, device="cuda").float()
    q = moe.moe_quantize_nvfp4(x, global_scale=given, want=ALL)
    assert bool((q["scale"] == 0x38).all())
    check_quantized(q, x, given)
    check_bytes(q, x, given)


def test_every_step_next_to_every_border():
    """Every mantissa that a step can have: the two floats on either side of border * t
    and the one between, which are all whose rounded quotient can lie beside the border."""
    c = torch.tensor(BORDERS, dtype=torch.float64, device="cuda")
    tie_up = torch.tensor([False, True, False, True, False, True, False], device="cuda")
    for first in range(1 << 23, 1 << 24, 1 << 20):
        g = torch.arange(first, first + (1 << 20), device="cuda").double() * 2.0 ** -24
        x = (c * g[:, None]).float().view(torch.int32)
        x = torch.stack([x + d for d in (-2, -1, 0, 1, 2)], -1).view(torch.float32).flatten(1)
        first_of_block = (6.0 * g).float()[:, None]
        row = torch.cat([first_of_block, x[:, :15], first_of_block, x[:, 15:30], first_of_block,
                         x[:, 30:], torch.zeros(len(g), 10, device="cuda")], 1)
        q = moe.moe_quantize_nvfp4(row, global_scale=g.float(), want=("codes", "scale"))
        assert bool((q["scale"] == 0x38).all())
        quotient = (row.double() / g[:, None]).float().double()
        above = torch.bucketize(quotient, c)     # borders below the quotient
        on = above.clamp(max=6)
        tie = (c[on] == quotient) & tie_up[on]
        assert torch.equal(nibbles(q["codes"]).long(), above + tie)


@pytest.mark.parametrize("dtype", [BF, HF, FL])
def test_zeros_keep_their_sign(dtype):
    x = randn(gen(3), 9, 64, dtype=dtype)
    x[:, ::3] = 0.0
    x[:, 1::3] = -0.0
    x[0, 16:32] = -0.0      # a block of zeros alone
    x[1] = -0.0             # a row of them
    for shape in ((9, 64), (3, 3, 64)):
        q = moe.moe_quantize_nvfp4(x.view(shape), want=ALL)
        check_quantized(q, x.view(shape))
        check_bytes(q, x.view(shape))
        v, live = q["values"].view(9, 64), torch.repeat_interleave(
            q["scale"].view(9, 4).view(torch.float8_e4m3fn).float() > 0, 16, -1)
        assert torch.equal(torch.signbit(v)[live], torch.signbit(x)[live])


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("power", [-30, 20, 53, 55, 60, 127])
def test_ties_beside_an_element_far_above_the_scale(power, dtype):
    """Under a given scale far below a block's maximum the codes of its small
    elements are still the division's."""
    lanes, given = [], []
    for k in (*range(16, 37), *range(128, 256, 3)):
        g = k * 2.0 ** (-84 if k < 128 else -87)
        t = 448.0 * g           # 11 bits at most, c t 14: exact in fp32
        row = [2.0 ** power] + [c * t for c in BORDERS] + [-c * t for c in BORDERS] + [-0.0]
        lanes.append(row)
        given.append(g)
    x = torch.tensor(lanes, dtype=torch.float64, device="cuda").to(dtype)
    given = torch.tensor(given, dtype=torch.float64, device="cuda").float()
    q = moe.moe_quantize_nvfp4(x, global_scale=given, want=ALL)
    assert bool((q["scale"] == 0x7E).all())
    check_quantized(q, x, given)
    check_bytes(q, x, given)
