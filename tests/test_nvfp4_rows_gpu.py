"""Four-bit rows and expert weights, and their grouped products, on the GPU
against plain restatements in float64.

Tolerances, from the arithmetic (u = 2^-24 is the fp32 rounding, h(T) =
finfo(T).eps / 2 the rounding to T):
  * quantisation is equality: every operation of the definition is one fp32
    rounding, which the restatement makes of the float64 result (a quotient of
    fp32 numbers rounded to float64 and then to fp32 is the rounded quotient);
  * a value is code * t with t rounded once: u, and h(T) for its storage;
  * a sum of K products of codes and scales: the products are exact (E2M1 has 2
    bits, E4M3 4, so 2 * (2 + 4) = 12), and each of the at most K additions in
    the tensor cores' fp32 accumulators is off by at most a unit of the last of
    24 bits of a partial sum, which is at most the sum of the magnitudes: K 2^-23 of
    that; the two global scales round twice, u each.  Over all outputs the
    errors do not line up: their 2-norm is held to sqrt(K) 2^-22 of the outputs'
    (independent errors of 2^-23 of partial sums whose spread is at most the
    output's);
  * silu(g) * u: |silu'| <= 1.1, so 1.1 |u| times g's error and |silu(g)| times
    u's, and 8 u of its own (the exponential, the addition, the division and the
    product)."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import pytest
import torch

import expert_routing_alignment_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn
MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@pytest.fixture(scope="module", autouse=True)
def _loaded():
    moe.load()


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=FL, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# --------------------------------------------------------------------------
# restatements
# --------------------------------------------------------------------------

def fl(x):
    return x.float().double()


def ref_quantize(x, given=None):
    """(codes [.., C], scale values, global scales, values), float64 holding fp32
    numbers; codes as signed E2M1 values."""
    f = x.double()
    b = f.unflatten(-1, (-1, 16))
    m = b.abs().amax(-1)
    whole = torch.isfinite(m)
    if given is None:
        top = torch.where(whole, m, torch.zeros_like(m)).flatten(1).amax(1)
        g = fl(top / torch.full_like(top, 2688.0)).clamp(min=2.0 ** -80)
    else:
        g = given.double()
    gb = g.view(-1, *[1] * (m.dim() - 1))
    r = fl(m / fl(6.0 * gb)).clamp(max=448.0)
    e = (torch.frexp(r)[1].long() - 1).clamp(min=-6)
    unit = ((e - 3 + 1023) << 52).view(torch.float64)
    s = torch.where(whole, torch.round(r / unit) * unit, torch.full_like(r, math.nan))
    t = fl(s * gb)[..., None]
    live = s[..., None] > 0
    q = torch.where(live, fl(b / torch.where(live, t, torch.ones_like(t))), torch.zeros_like(b))
    a = q.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    code = torch.round(a / step) * step * torch.where(b < 0, -1.0, 1.0)
    code = torch.where(live, code, torch.zeros_like(code))
    return (code.flatten(-2), s, g, fl(code * t).flatten(-2))


def code_values(codes):
    mag = torch.tensor(MAG, dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64,
                    device=codes.device)
    for i in (0, 1):
        c = (codes >> (4 * i)) & 15
        v[..., i::2] = mag[(c & 7).int()] * (1.0 - 2.0 * (c >> 3).double())
    return v


def wide(q):
    """The float64 values of a packed set, without any rounding."""
    codes, scale, g = moe._packed("q", q)
    s = scale.view(E4).to(torch.float64)
    return code_values(codes) * torch.repeat_interleave(s, 16, -1) * g.double().view(
        -1, *[1] * (codes.dim() - 1))


def same(a, b, what=""):
    """Equal, NaN to NaN."""
    a, b = a.double(), b.double()
    assert a.shape == b.shape, (what, a.shape, b.shape)
    bad = ~((a == b) | (a.isnan() & b.isnan()))
    assert not bad.any(), (what, int(bad.sum()), a[bad][:4], b[bad][:4])


def check_quantized(q, x, given=None):
    code, s, g, values = ref_quantize(x, given)
    same(q["global_scale"], g, "global_scale")
    same(q["scale"].view(E4).float(), s, "scale")
    same(code_values(q["codes"]), code, "codes")
    if "values" in q:
        same(q["values"], values.to(x.dtype), "values")


ALL = ("codes", "scale", "global_scale", "values")


# --------------------------------------------------------------------------
# quantisation
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("M,H", [(1, 16), (1, 2048), (3, 48), (257, 96), (5, 512), (7, 528),
                                 (300, 1040), (8, 4096), (2, 4112), (3, 8192), (2, 16384)])
def test_rows(dtype, M, H):
    x = randn(gen(M * 7 + H), M, H, scale=3.0).to(dtype)
    x[0, :: 5] = 0
    check_quantized(moe.moe_quantize_nvfp4(x, want=ALL), x)


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("E,R,C", [(1, 2, 16), (3, 5, 48), (2, 300, 144), (4, 65, 2048),
                                   (70, 3, 32), (1, 1536, 1024), (1, 1, 64)])
def test_expert_matrices(dtype, E, R, C):
    x = randn(gen(E + R + C), E, R, C, scale=0.02)
    x = (x * torch.exp2(torch.arange(E, device="cuda").float())[:, None, None]).to(dtype)
    check_quantized(moe.moe_quantize_nvfp4(x, want=ALL), x)


@pytest.mark.parametrize("at", [0, 1, 300000, 8388600, 8388607])
def test_one_large_matrix_finds_its_maximum_anywhere(at):
    """More parts of the maximum than a CTA has threads."""
    x = randn(gen(7), 1, 4096, 2048, dtype=BF, scale=0.02)
    x.view(-1)[at] = -9.0
    q = moe.moe_quantize_nvfp4(x, want=ALL)
    assert float(q["global_scale"][0]) == float(torch.tensor(9.0) / torch.tensor(2688.0))
    check_quantized(q, x)


@pytest.mark.parametrize("groups", [4096, 4097, 70000])
def test_many_small_matrices(groups):
    x = randn(gen(groups), groups, 2, 16)
    check_quantized(moe.moe_quantize_nvfp4(x, want=ALL), x)


def test_every_tie_of_a_code_and_of_a_scale():
    """Steps that are powers of two and of other E4M3 values, elements on each
    border between two codes and next to it."""
    lanes = []
    for s in range(8, 16):
        for e in (-9, -3, 0, 5):
            t = s * 2.0 ** e
            for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                lanes.append([6 * t] + [v * t for v in (b, -b)] + [0.0] * 13)
    x = torch.tensor(lanes, dtype=torch.float64, device="cuda").float()
    ulp = torch.nextafter(x, torch.full_like(x, math.inf))
    low = torch.nextafter(x, torch.full_like(x, -math.inf))
    x = torch.cat([x, torch.where(x.abs() > 0, ulp, x), torch.where(x.abs() > 0, low, x)])
    x = x.reshape(-1, 16)
    ones = torch.ones(x.shape[0], device="cuda")
    check_quantized(moe.moe_quantize_nvfp4(x, want=ALL), x)
    check_quantized({**moe.moe_quantize_nvfp4(x, global_scale=ones, want=ALL)}, x, ones)


def test_blocks_with_nan_and_infinity_are_nan_and_leave_the_others_alone():
    for dtype in (BF, HF, FL):
        x = randn(gen(4), 6, 64, dtype=dtype)
        x[0, 3], x[1, 20], x[2, 63] = math.nan, math.inf, -math.inf
        x[3] = math.nan
        x[4] = 0
        q = moe.moe_quantize_nvfp4(x, want=ALL)
        check_quantized(q, x)
        assert int(q["values"].isnan().sum()) == 3 * 16 + 64
        m = moe.moe_quantize_nvfp4(x.view(2, 3, 64), want=ALL)
        check_quantized(m, x.view(2, 3, 64))


@pytest.mark.parametrize("scale", [3e38, 1e30, 1e-20, 2.0 ** -79, 1e-30, 1e-38, 1e-44])
def test_magnitudes_to_the_ends_of_fp32(scale):
    """Down to the least global scale codes are those of the definition; rows
    below it lose their small elements to zero, and nothing becomes NaN."""
    x = (randn(gen(9), 4, 256).clamp(-3, 3) / 3.0).double() * scale
    x = x.float()
    q = moe.moe_quantize_nvfp4(x, want=ALL)
    check_quantized(q, x)
    assert torch.isfinite(q["values"]).all()


def test_given_scales():
    x = randn(gen(12), 5, 288, dtype=BF)
    for g in (1.0, 2.0 ** -80, 2.0 ** 100, 1e-3, 7e-5):
        given = torch.full((5,), g, device="cuda")
        q = moe.moe_quantize_nvfp4(x, global_scale=given, want=ALL)
        check_quantized(q, x, given)
        assert q["global_scale"].data_ptr() != given.data_ptr()
    m = x.view(1, 5, 288)
    given = torch.full((1,), 3e-4, device="cuda")
    check_quantized(moe.moe_quantize_nvfp4(m, global_scale=given, want=ALL), m, given)


@pytest.mark.parametrize("want", [("codes",), ("scale",), ("global_scale",), ("values",),
                                  ("codes", "values")])
def test_outputs_alone(want):
    for x in (randn(gen(3), 9, 176, dtype=BF), randn(gen(3), 3, 9, 176, dtype=BF)):
        full = moe.moe_quantize_nvfp4(x, want=ALL)
        q = moe.moe_quantize_nvfp4(x, want=want)
        assert set(q) == set(want)
        for n in want:
            assert torch.equal(q[n].view(torch.uint8), full[n].view(torch.uint8)), n


@pytest.mark.parametrize("dtype", [BF, FL])
def test_strides_and_alignments(dtype):
    base = randn(gen(5), 40, 1000, dtype=dtype)
    for x in (base[:, 1:65], base[::3, 8:168], base[:, 3:995], base[:1, 5:21],
              base[0].expand(7, 1000)[:, :992], base.view(4, 10, 1000)[:, :, 4:100],
              base.view(4, 10, 1000)[1:2, 2:5, 8:40], base.view(40, 1, 1000)[:, :, :32]):
        check_quantized(moe.moe_quantize_nvfp4(x, want=ALL), x)
    x = base[:, :992].contiguous()
    flat = torch.empty(40 * 992 + 1, dtype=dtype, device="cuda")
    out = dict(values=flat[1:].view(40, 992))
    moe.moe_quantize_nvfp4(x, out=out)
    assert torch.equal(out["values"], moe.moe_quantize_nvfp4(x, want=ALL)["values"])
    own = x.clone()   # values in x's own place
    moe.moe_quantize_nvfp4(own, out=dict(values=own))
    assert torch.equal(own, out["values"])


def align(counts, BS, E=None):
    """Tables of experts with these many slots each (top_k = 1), slots in a
    scrambled order; token t is slot t."""
    ids = torch.cat([torch.full((c,), e, dtype=torch.int32) for e, c in enumerate(counts)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))]
    return moe.moe_align(ids.cuda(), E or len(counts), BS), len(ids)


def test_rows_in_expert_order_skip_the_padding():
    t, n = align([5, 0, 17, 1], 16)
    rows = t["max_total"]
    x = randn(gen(6), rows, 96, dtype=BF)
    real = t["sorted_token_ids"][:rows] < n
    assert int(real.sum()) == n
    x[~real] = math.nan
    out = moe.alloc_quantize_nvfp4_outputs(x, ALL)
    for v in out.values():
        v.view(torch.uint8).fill_(0x5A)
    before = {k: v.clone() for k, v in out.items()}
    moe.moe_quantize_nvfp4(x, tables=t, out=out)
    for k, v in out.items():
        assert torch.equal(v[~real].view(torch.uint8), before[k][~real].view(torch.uint8)), k
    check_quantized({k: v[real] for k, v in out.items()}, x[real])


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("shape", [(1, 16), (5, 48), (1000, 2880), (3, 7, 32), (2, 129, 512)])
def test_dequantize(dtype, shape):
    x = randn(gen(8), *shape)
    q = moe.moe_quantize_nvfp4(x, want=ALL)
    codes, scale, glob = (q[n] for n in ("codes", "scale", "global_scale"))
    got = moe.moe_dequantize_nvfp4(codes, scale, glob, dtype=dtype)
    same(got, q["values"].to(dtype))
    ref = wide(q)
    tol = half(dtype) * ref.abs() + tiny(dtype) + 2 * U * ref.abs()
    assert ((got.double() - ref).abs() <= tol).all()
    flat = torch.zeros(got.numel() + 1, dtype=dtype, device="cuda")
    moe.moe_dequantize_nvfp4(codes, scale.view(E4), glob, out=flat[1:].view(got.shape))
    assert torch.equal(flat[1:].view(got.shape), got)


def test_every_code_under_every_scale():
    """All 256 pairs of codes, all 256 scale bytes (NaN where the byte is)."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)
    scale = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 32)
    glob = torch.ones(256, device="cuda")
    got = moe.moe_dequantize_nvfp4(codes, scale, glob, dtype=FL)
    ref = code_values(codes) * scale[:, :1].view(E4).to(torch.float64)
    same(got, ref)


def test_quantized_values_quantise_to_themselves():
    x = randn(gen(21), 64, 1024, dtype=FL)
    q = moe.moe_quantize_nvfp4(x, want=ALL)
    again = moe.moe_quantize_nvfp4(q["values"], global_scale=q["global_scale"], want=ALL)
    assert torch.equal(again["values"], q["values"])


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------

def weights(g, E, R, C):
    return moe.moe_quantize_nvfp4(randn(g, E, R, C, scale=0.05, dtype=BF))


def rows_of(t, k, by_token):
    """(positions, row that each reads, expert of each) of the real positions."""
    offs = t["expert_offsets"].long()
    n = t["token_to_perm"].numel()
    p = torch.arange(t["max_total"], device="cuda")
    s = t["sorted_token_ids"][: t["max_total"]].long()
    real = s < n
    p, s = p[real], s[real]
    e = torch.searchsorted(offs, p, right=True) - 1
    return p, (s // k if by_token else p), e


def sums(x, w, at, e):
    """The products of rows at and matrices e in float64, and the sums of the
    magnitudes."""
    X, W = wide(x), wide(w)
    y = torch.zeros(len(at), W.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for i in e.unique().tolist():
        rows = X[at[e == i]]
        y[e == i] = rows @ W[i].T
        mag[e == i] = rows.abs() @ W[i].abs().T
    return y, mag


def check_product(got, y, err, K, norm=True):
    t = got.dtype
    tol = half(t) * y.abs() + tiny(t) + (1 + half(t)) * err
    bad = ~((got.double() - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], y[bad][:4])
    if norm and y.numel():
        off = float((got.double() - y).norm()) / max(float(y.norm()), 1e-300)
        assert off <= half(t) + math.sqrt(K) * 2.0 ** -22, off


def run_product(counts, R, C, BS=16, k=1, by_token=True, dtype=BF, seed=0, E=None):
    E = E or len(counts)
    g = gen(seed)
    if k == 1:
        t, n = align(counts, BS, E)
    else:
        ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:k]
                           for i in range(sum(counts))]).int().cuda()
        t, n = moe.moe_align(ids, E, BS), ids.numel()
    M = n // k
    x = moe.moe_quantize_nvfp4(randn(g, M if by_token else t["max_total"], C, dtype=BF))
    w = weights(g, E, R, C)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fill = torch.full((t["max_total"], R), 7.0, dtype=dtype, device="cuda")
    out = moe.moe_grouped_product_nvfp4(w, x, t, k, M=None if by_token else M, out=fill.clone(),
                                        err_word=err)
    p, at, e = rows_of(t, k, by_token)
    assert len(p) == n
    y, mag = sums(x, w, at, e)
    check_product(out[p], y, (C * 2.0 ** -23 + 2 * U) * mag, C)
    rest = torch.ones(t["max_total"], dtype=torch.bool, device="cuda")
    rest[p] = False
    assert torch.equal(out[rest], fill[rest])
    assert int(err) == 0
    return out


@pytest.mark.parametrize("C", [32, 64, 96, 128, 224, 256, 288, 512, 1024, 2048])
def test_product_depths(C):
    run_product([3, 0, 20], 128, C, seed=C)


@pytest.mark.parametrize("R", [1, 7, 40, 128, 130, 256, 264, 384, 520])
def test_product_widths(R):
    run_product([3, 0, 20], R, 256, seed=R)
    run_product([3, 0, 20], R, 96, seed=R, dtype=FL)


@pytest.mark.parametrize("n", [1, 2, 8, 15, 16, 17, 31, 33, 64, 65, 96, 127, 128, 129, 255, 256,
                               257, 300])
def test_product_rows(n):
    run_product([n], 256, 512, BS=1, seed=n)
    run_product([1, n, 0, n // 2], 128, 128, BS=64, seed=n, dtype=FL)


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("by_token", [True, False])
@pytest.mark.parametrize("BS", [1, 16, 128, 300])
def test_product_layouts(dtype, by_token, BS):
    run_product([40, 1, 0, 130], 200, 288, BS=BS, by_token=by_token, dtype=dtype)
    run_product([37], 96, 320, BS=BS, k=3, E=7, by_token=by_token, dtype=dtype)


def test_product_of_many_experts():
    run_product([2] * 40, 64, 64, k=4, E=1024, BS=16)
    run_product([600], 128, 64, k=8, E=333, BS=1, dtype=FL)


def test_product_of_many_tiles():
    """More tiles than the device has CTAs, of several row tiles each."""
    run_product([700, 10, 300, 0, 129, 128], 4096, 544, BS=1, seed=5, dtype=FL)
    run_product([700, 10, 300, 0, 129, 128], 2048, 1024, BS=64, seed=6)


def gate_up_reference(x, gate, up, at, e, C):
    g, mg = sums(x, gate, at, e)
    u, mu = sums(x, up, at, e)
    per = C * 2.0 ** -23 + 2 * U
    silu = g * torch.sigmoid(g)
    h = silu * u
    err = 1.1 * per * mg * (u.abs() + per * mu) + silu.abs() * per * mu + 8 * U * h.abs()
    return h, err


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("counts,R,C,by_token", [
    ([1], 128, 256, True), ([3, 0, 70, 129], 200, 288, True), ([20, 300], 40, 64, False),
    ([5] * 30, 768, 1024, True)])
def test_gate_up(dtype, counts, R, C, by_token):
    t, n = align(counts, 16)
    g = gen(R + C)
    x = moe.moe_quantize_nvfp4(randn(g, n if by_token else t["max_total"], C, dtype=BF))
    gate, up = weights(g, len(counts), R, C), weights(g, len(counts), R, C)
    fill = torch.full((t["max_total"], R), 7.0, dtype=dtype, device="cuda")
    out = moe.moe_grouped_gate_up_nvfp4(gate, up, x, t, 1, M=None if by_token else n,
                                        out=fill.clone())
    p, at, e = rows_of(t, 1, by_token)
    h, err = gate_up_reference(x, gate, up, at, e, C)
    check_product(out[p], h, err, C, norm=False)
    off = float((out[p].double() - h).norm() / h.norm())
    assert off <= half(dtype) + 2 * math.sqrt(C) * 2.0 ** -22 + 8 * U, off
    rest = torch.ones(t["max_total"], dtype=torch.bool, device="cuda")
    rest[p] = False
    assert torch.equal(out[rest], fill[rest])


def test_products_take_nan_scales_where_they_belong():
    t, n = align([40, 20], 16)
    g = gen(2)
    x, w = moe.moe_quantize_nvfp4(randn(g, n, 128)), weights(g, 2, 160, 128)
    ref = moe.moe_grouped_product_nvfp4(w, x, t, 1, out_dtype=FL,
                                        out=torch.zeros(t["max_total"], 160, device="cuda"))
    x["scale"][7, 3] = 0x7F
    w["scale"][1, 33, 0] = 0x7F
    got = moe.moe_grouped_product_nvfp4(w, x, t, 1, out=torch.zeros_like(ref))
    p, at, e = rows_of(t, 1, True)
    nan = torch.zeros_like(ref, dtype=torch.bool)
    nan[p[at == 7]] = True
    nan[p[e == 1], 33] = True
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], ref[~nan])


def test_a_rows_bits_do_not_depend_on_the_rows_around_it():
    g = gen(3)
    w = weights(g, 3, 384, 512)
    x = moe.moe_quantize_nvfp4(randn(g, 400, 512))
    ids = torch.randint(0, 3, (400, 1), generator=g, device="cuda").int()

    def rows(sel, BS):
        t = moe.moe_align(ids[sel].contiguous(), 3, BS)
        q = {n: v[sel].contiguous() for n, v in x.items()}
        y = moe.moe_grouped_product_nvfp4(w, q, t, 1, out_dtype=FL)
        return y[t["token_to_perm"].long()]

    whole = rows(torch.arange(400, device="cuda"), 16)
    for sel in (torch.arange(1, device="cuda"), torch.arange(200, 231, device="cuda"),
                torch.arange(399, -1, -3, device="cuda")):
        assert torch.equal(rows(sel, 64), whole[sel])


def test_tables_that_are_none_compute_nothing_and_say_so():
    t, n = align([20, 30], 16)
    g = gen(3)
    w, x = weights(g, 2, 64, 64), moe.moe_quantize_nvfp4(randn(g, n, 64))
    for offs in ([0, 48, 32], [0, 32, 10 ** 6], [-16, 32, 64]):
        bad = {**t, "expert_offsets": torch.tensor(offs, dtype=torch.int32, device="cuda")}
        out = torch.full((t["max_total"], 64), 3.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.moe_grouped_product_nvfp4(w, x, bad, 1, out=out, err_word=err)
        assert int(err) == moe.MOE_ERR_BAD_POSITION and bool((out == 3.0).all())
    ids = t["sorted_token_ids"].clone()
    ids[3], ids[5] = -7, n + 50
    out = torch.full((t["max_total"], 64), 3.0, device="cuda")
    err.zero_()
    moe.moe_grouped_product_nvfp4(w, x, {**t, "sorted_token_ids": ids}, 1, out=out, err_word=err)
    good = moe.moe_grouped_product_nvfp4(w, x, t, 1, out=torch.full_like(out, 3.0))
    good[[3, 5]] = 3.0
    assert int(err) == moe.MOE_ERR_BAD_POSITION and torch.equal(out, good)


def test_no_slots_at_all():
    t = moe.moe_align(torch.full((6,), -1, dtype=torch.int32, device="cuda"), 4, 16)
    g = gen(1)
    out = torch.full((t["max_total"], 64), 3.0, device="cuda")
    moe.moe_grouped_product_nvfp4(weights(g, 4, 64, 64), moe.moe_quantize_nvfp4(randn(g, 6, 64)), t,
                                  1, out=out)
    assert bool((out == 3.0).all())


# --------------------------------------------------------------------------
# the operators together
# --------------------------------------------------------------------------

def layer_inputs(seed, M, E, k, H, I):
    g = gen(seed)
    ids, w = moe.moe_topk_softmax(randn(g, M, E), k)
    sets = [weights(g, E, I, H), weights(g, E, I, H), weights(g, E, H, I)]
    return randn(g, M, H, dtype=BF), ids, w, sets


def layer_calls(x, ids, w, sets, E, k, BS):
    t = moe.moe_align(ids, E, BS)
    q = moe.moe_quantize_nvfp4(x)
    h = moe.moe_grouped_gate_up_nvfp4(sets[0], sets[1], q, t, k)
    hq = moe.moe_quantize_nvfp4(h, tables=t)
    y = moe.moe_grouped_product_nvfp4(sets[2], hq, t, k, M=x.shape[0])
    return t, q, h, hq, y, moe.moe_combine(y, w, t)


@pytest.mark.parametrize("M,E,k,H,I,BS", [(1, 16, 4, 256, 128, 16), (9, 8, 2, 512, 384, 16),
                                          (200, 12, 3, 256, 320, 64)])
def test_layer_of_four_bit_rows(M, E, k, H, I, BS):
    x, ids, w, sets = layer_inputs(M, M, E, k, H, I)
    t, q, h, hq, y, out = layer_calls(x, ids, w, sets, E, k, BS)
    check_quantized(q, x)
    p, at, e = rows_of(t, k, True)
    ref, err = gate_up_reference(q, sets[0], sets[1], at, e, H)
    check_product(h[p], ref, err, H, norm=False)
    check_quantized({n: v[p] for n, v in hq.items()}, h[p])
    sel = {n: v[p] for n, v in hq.items()}
    ref, mag = sums(sel, sets[2], torch.arange(len(p), device="cuda"), e)
    check_product(y[p], ref, (I * 2.0 ** -23 + 2 * U) * mag, I)
    perm = t["token_to_perm"].view(M, k).long()
    exact = (y[perm].double() * w.double()[:, :, None]).sum(1)
    bound = (half(BF) + k * U) * (y[perm].double().abs() * w.double()[:, :, None]).sum(1)
    assert ((out.double() - exact).abs() <= bound + tiny(BF)).all()


def test_layer_in_a_graph_and_on_another_stream():
    x, ids, w, sets = layer_inputs(5, 33, 8, 2, 256, 128)
    eager = layer_calls(x, ids, w, sets, 8, 2, 16)[-1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = layer_calls(x, ids, w, sets, 8, 2, 16)[-1]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer_calls(x, ids, w, sets, 8, 2, 16)[-1]
    x2, ids2, w2, _ = layer_inputs(6, 33, 8, 2, 256, 128)
    want = layer_calls(x2, ids2, w2, sets, 8, 2, 16)[-1]
    x.copy_(x2), ids.copy_(ids2), w.copy_(w2)
    graph.replay()
    assert torch.equal(out, want)
    m = randn(gen(4), 3, 40, 64, dtype=BF)   # a workspace inside a capture
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
        q = moe.moe_quantize_nvfp4(m, want=ALL)
    m.copy_(randn(gen(5), 3, 40, 64, dtype=BF))
    graph.replay()
    check_quantized(q, m)


def test_calls_on_a_given_stream_write_new_outputs_there():
    x = randn(gen(7), 64, 512, dtype=BF)
    m = randn(gen(7), 4, 64, 512, dtype=BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = moe.moe_quantize_nvfp4(x, want=ALL, stream=s)
    w = moe.moe_quantize_nvfp4(m, stream=s)
    v = moe.moe_dequantize_nvfp4(w["codes"], w["scale"], w["global_scale"], stream=s)
    t, n = align([30, 4, 0, 30], 16)
    s.wait_stream(torch.cuda.current_stream())
    y = moe.moe_grouped_product_nvfp4(w, q, t, 1, stream=s)
    s.synchronize()
    check_quantized(q, x)
    check_quantized({**w}, m)
    same(v, ref_quantize(m)[3].to(BF))
    p, at, e = rows_of(t, 1, True)
    ref, mag = sums(q, w, at, e)
    check_product(y[p], ref, (512 * 2.0 ** -23 + 2 * U) * mag, 512)


def test_gradient_through_the_transposed_set():
    """d(sum_p dy[p] . W_e x[p]) / dx = W_e^T dy: the same product on the
    transposed matrices, quantised along the outputs."""
    g = gen(31)
    E, R, C = 3, 96, 160
    t, n = align([20, 0, 50], 16)
    W = randn(g, E, R, C, dtype=BF, scale=0.05)
    wt = moe.moe_quantize_nvfp4(W.transpose(1, 2).contiguous(), want=ALL)
    dy = randn(g, t["max_total"], R, dtype=BF)
    dq = moe.moe_quantize_nvfp4(dy, tables=t, want=ALL)
    dx = moe.moe_grouped_product_nvfp4(wt, dq, t, 1, M=n, out_dtype=FL)
    p, _, e = rows_of(t, 1, False)
    x = torch.zeros(len(p), C, dtype=torch.float64, device="cuda", requires_grad=True)
    y = torch.einsum("pc,pcr->pr", x, wide(wt)[e])
    (y * wide({k: v[p] for k, v in dq.items()})).sum().backward()
    _, mag = sums({k: v[p] for k, v in dq.items()}, wt, torch.arange(len(p), device="cuda"), e)
    check_product(dx[p], x.grad, (R * 2.0 ** -23 + 2 * U) * mag, R)


def test_straight_through_gradient():
    """Values as a torch function whose gradient passes the rounding: against
    differences of the loss in the rounded values."""
    class Rounded(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return moe.moe_quantize_nvfp4(x, want=("values",))["values"]

        @staticmethod
        def backward(ctx, d):
            return d

    x = randn(gen(13), 4, 64).requires_grad_()
    c = randn(gen(14), 4, 64)
    v = Rounded.apply(x)
    (v.square() * c).sum().backward()
    v = v.detach().double()
    step = 2.0 ** -20
    diff = ((v + step).square() - (v - step).square()) * c.double() / (2 * step)
    # two fp32 products in the gradient, and the differences' cancellation in float64
    tol = 4 * U * diff.abs() + 2.0 ** -52 * (v.square() + 1) * c.abs() / step
    assert ((x.grad.double() - diff).abs() <= tol).all()


# --------------------------------------------------------------------------
# sizes and uses at the ends
# --------------------------------------------------------------------------

def test_two_products_at_once():
    """Two streams with products of their own on the same weights."""
    g = gen(41)
    w, up = weights(g, 6, 640, 512), weights(g, 6, 640, 512)
    t, n = align([200, 3, 0, 90, 1, 300], 16)
    x = moe.moe_quantize_nvfp4(randn(g, n, 512, dtype=BF))
    one = moe.moe_grouped_gate_up_nvfp4(w, up, x, t, 1, out=torch.zeros(
        t["max_total"], 640, dtype=BF, device="cuda"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(one) for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, o in zip(streams, outs):
            moe.moe_grouped_gate_up_nvfp4(w, up, x, t, 1, out=o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, one)


def test_products_repeat_to_the_bit():
    g = gen(42)
    w = weights(g, 5, 1000, 1120)
    t, n = align([700, 0, 33, 32, 129], 1)
    x = moe.moe_quantize_nvfp4(randn(g, n, 1120, dtype=BF))
    first = moe.moe_grouped_product_nvfp4(w, x, t, 1, out_dtype=FL)
    for _ in range(50):
        assert torch.equal(moe.moe_grouped_product_nvfp4(w, x, t, 1, out_dtype=FL), first)


def test_outputs_at_any_element_address():
    """Outputs whose rows no 16-byte piece fits."""
    for dtype, R, by_token in ((BF, 130, True), (HF, 256, False), (FL, 96, True), (FL, 257, False)):
        g = gen(R)
        t, n = align([70, 5, 140], 16)
        w = weights(g, 3, R, 256)
        x = moe.moe_quantize_nvfp4(randn(g, n if by_token else t["max_total"], 256, dtype=BF))
        M = None if by_token else n
        flat = torch.full((t["max_total"] * R + 1,), 5.0, dtype=dtype, device="cuda")
        moe.moe_grouped_product_nvfp4(w, x, t, 1, M=M, out=flat[1:].view(-1, R))
        p, at, e = rows_of(t, 1, by_token)
        y, mag = sums(x, w, at, e)
        check_product(flat[1:].view(-1, R)[p], y, (256 * 2.0 ** -23 + 2 * U) * mag, 256)
        rest = torch.ones(t["max_total"], dtype=torch.bool, device="cuda")
        rest[p] = False
        assert bool((flat[1:].view(-1, R)[rest] == 5.0).all()) and float(flat[0]) == 5.0


def test_scales_of_any_width_at_the_arrays_ends():
    """Rows of scales that are no whole words or pieces: the last row of the last
    expert, the last token."""
    for C in (32, 96, 160, 288, 352, 64, 192, 320):
        for R in (1, 3, 97, 129, 193):
            run_product([2, 40, 1], R, C, BS=1, seed=C + R, dtype=FL)


def test_weights_beyond_four_gigabytes():
    E, R, C = 600, 8192, 2048
    codes = torch.randint(0, 256, (E, R, C // 2), dtype=torch.uint8, device="cuda",
                          generator=gen(50))
    scale = torch.randint(0x28, 0x40, (E, R, C // 16), dtype=torch.uint8, device="cuda",
                          generator=gen(51))
    glob = torch.full((E,), 0.01, device="cuda")
    ids = torch.tensor([[0], [599], [598], [599], [300]], dtype=torch.int32, device="cuda")
    t = moe.moe_align(ids, E, 1)
    x = moe.moe_quantize_nvfp4(randn(gen(52), 5, C, dtype=BF))
    y = moe.moe_grouped_product_nvfp4((codes, scale, glob), x, t, 1, out_dtype=FL)
    got = y[t["token_to_perm"].long()]
    X = wide(x)
    for i, e in enumerate(ids.view(-1).tolist()):
        W = wide((codes[e], scale[e], glob[e].expand(R)))
        check_product(got[i: i + 1], (X[i] @ W.T)[None],
                      ((C * 2.0 ** -23 + 2 * U) * (X[i].abs() @ W.abs().T))[None], C)


def test_rows_beyond_two_billion_elements():
    M, H = 270001, 8192
    x = torch.empty(M, H, dtype=BF, device="cuda").normal_(generator=gen(60))
    q = moe.moe_quantize_nvfp4(x)
    pick = torch.tensor([0, 1, 131072, 262143, 262144, M - 2, M - 1], device="cuda")
    check_quantized({n: v[pick] for n, v in q.items()}, x[pick])
    got = moe.moe_dequantize_nvfp4(q["codes"], q["scale"], q["global_scale"])
    same(got[pick], ref_quantize(x[pick])[3].to(BF))
    m = x[:262144].view(2, 131072, H)
    q = moe.moe_quantize_nvfp4(m)
    tail = m[1, -3:]
    check_quantized({"codes": q["codes"][1, -3:], "scale": q["scale"][1, -3:],
                     "global_scale": q["global_scale"][1:].expand(3)}, tail,
                    q["global_scale"][1:].expand(3))
    top = m[1].abs().amax().double() / torch.full((), 2688.0, dtype=torch.float64, device="cuda")
    assert float(q["global_scale"][1]) == float(top.float())


def test_a_single_row_and_a_single_expert():
    for C, R in ((32, 1), (16384, 5), (16384, 300)):
        run_product([1], R, C, BS=1, seed=C + R, dtype=FL)
    run_product([65], 65536, 64, BS=1, seed=9)


def test_first_calls_inside_a_capture():
    """A process whose first calls of these entry points are inside a capture."""
    code = """
import torch, expert_routing_alignment_gb300 as moe
moe.load()
torch.manual_seed(0)
M, H, I, E, k = 40, 512, 256, 8, 2
x = torch.randn(M, H, device="cuda").bfloat16()
wide = [torch.randn(E, *s, device="cuda").bfloat16() for s in ((I, H), (I, H), (H, I))]
ids, tw = moe.moe_topk_softmax(torch.randn(M, E, device="cuda"), k)
t = moe.moe_align(ids, E, 16)
def run():
    g, u, d = ((q["codes"], q["scale"], q["global_scale"]) for q in
               map(moe.moe_quantize_nvfp4, wide))
    q = moe.moe_quantize_nvfp4(x)
    h = moe.moe_grouped_gate_up_nvfp4(g, u, q, t, k)
    hq = moe.moe_quantize_nvfp4(h, tables=t)
    y = moe.moe_grouped_product_nvfp4(d, hq, t, k, M=M)
    return moe.moe_combine(y, tw, t), moe.moe_dequantize_nvfp4(*d)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, run()):
    assert torch.equal(a, b)
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root,
                       timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stdout + p.stderr


def test_tables_of_a_layer_call():
    """The tables that a layer call leaves in its workspace serve the products."""
    import synth
    shape = synth.tiny()
    dev = synth.make_layer(shape, 7, device="cpu").to("cuda")
    layer = moe.LayerDesc(top_k=shape.top_k, block_size=shape.BS,
                          routed=moe.Experts.from_synth(dev.experts))
    ws = moe.alloc_workspace(layer, shape.M)
    out = torch.empty(shape.M, shape.H, dtype=BF, device="cuda")
    moe.moe_decode_layer(layer, dev.x, out, ws, router_logits=dev.logits)
    v = moe.workspace_view(layer, shape.M, ws)
    w = weights(gen(3), shape.E, 96, shape.H)
    x = moe.moe_quantize_nvfp4(dev.x)
    got = moe.moe_grouped_product_nvfp4(w, x, v, shape.top_k, out_dtype=FL)
    p, at, e = rows_of(v, shape.top_k, True)
    y, mag = sums(x, w, at, e)
    check_product(got[p], y, (shape.H * 2.0 ** -23 + 2 * U) * mag, shape.H)


def test_long_padded_runs():
    """Blocks of many tiles, of which few have a row; and runs whose real rows do
    not come first (tables of the user's own)."""
    run_product([3, 0, 300, 1], 160, 256, BS=1000, seed=70)
    run_product([3, 0, 300, 1], 160, 288, BS=700, by_token=False, seed=71, dtype=FL)
    t, n = align([40, 20], 400)
    ids = t["sorted_token_ids"].clone()
    ids[:400] = ids[:400].flip(0)     # expert 0: its rows at the run's end
    t2 = {**t, "sorted_token_ids": ids}
    g = gen(72)
    w, x = weights(g, 2, 96, 128), moe.moe_quantize_nvfp4(randn(g, n, 128, dtype=BF))
    a = moe.moe_grouped_product_nvfp4(w, x, t, 1, out=torch.zeros(
        t["max_total"], 96, device="cuda"))
    b = moe.moe_grouped_product_nvfp4(w, x, t2, 1, out=torch.zeros_like(a))
    assert torch.equal(b[:400], a[:400].flip(0)) and torch.equal(b[400:], a[400:])
