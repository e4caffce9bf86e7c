"""Token dispatch and combination, the RMS norm ahead of the router and every
gradient on the GPU, against plain float64 restatements.

Tolerances, from the arithmetic (u = 2^-24 is the fp32 rounding; h(T) =
finfo(T).eps / 2 the rounding to T; tiny(T) half of T's smallest subnormal):
  * a copy is exact;
  * a sum of k products by fmaf is off by at most k u of the sum of their
    magnitudes, then rounded to T;
  * a dot product of H products likewise by H u;
  * the mean of squares: a thread adds at most 32 squares, then 5 levels of a
    butterfly and at most 16 warps, each a rounding of a positive sum, so it
    is within 56 u; rstd, its inverse root, within 28 u + 3 u (root, division
    and the addition of eps) < 32 u;
  * an e4m3 code is at most half a step from its quotient; the quotient of
    16-bit inputs is known to one rounding (u), others to four."""
from __future__ import annotations

import math
import os

import pytest
import torch

import expert_routing_alignment_gb300 as moe
import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn


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


def close(got, ref, mag, err, msg=""):
    """|got - ref| <= rounding of ref to got's type + err * mag, elementwise."""
    t = got.dtype
    tol = half(t) * ref.abs() + tiny(t) + err * (1 + half(t)) * mag
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (msg, int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


def bits(t):
    return t.contiguous().view(torch.uint8)


def route(M, E, k, BS, seed, skipped=0.0):
    """ids, weights and the framework's alignment; ``skipped``: the share of
    slots whose expert is not here."""
    g = gen(seed)
    ids, w = moe.moe_topk_softmax(randn(g, M, E), k)
    if skipped:
        gone = torch.rand(M, k, generator=g, device="cuda") < skipped
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
        if M > 2:
            ids[1] = -1   # a token without any expert
    return ids, w, moe.moe_align(ids, E, BS)


def perm_of(t, M, k):
    return t["token_to_perm"][: M * k].view(M, k).long()


def taken(rows, perm):
    """float64 rows by slot [M, k, H], zero where skipped."""
    v = rows.double()[perm.clamp(min=0)]
    return torch.where((perm >= 0)[..., None], v, torch.zeros((), dtype=torch.float64,
                                                              device=v.device))


def padding(t, n):
    """Which rows of the sorted order are padding below the total, and which
    lie behind it."""
    p = torch.arange(t["max_total"], device="cuda")
    below = p < t["num_tokens_post_padded"]
    return below & (t["sorted_token_ids"][: t["max_total"]] >= n), ~below


# (M, H, E, k, BS, skipped): one token to many; whole vectors, whole blocks,
# odd widths below and above a warp's; top_k to 32; blocks of one row
SHAPES = [(1, 128, 8, 2, 16, 0.0), (8, 2048, 128, 8, 16, 0.0), (3, 1, 4, 1, 1, 0.0),
          (37, 999, 16, 3, 8, 0.4), (128, 4096, 256, 8, 64, 0.0), (65, 264, 64, 32, 16, 0.2),
          (1000, 520, 24, 6, 128, 0.5), (2, 8192, 8, 8, 64, 0.0), (300, 12, 1024, 10, 4, 0.9),
          (17, 2050, 4, 4, 64, 1.0), (5, 16384, 8, 3, 16, 0.0), (700, 72, 16, 1, 16, 0.3),
          (90, 10007, 8, 2, 32, 0.0), (2500, 1024, 64, 8, 16, 0.2),
          (40, 1540, 8, 3, 16, 0.2), (1100, 100, 8, 5, 4, 0.0), (1030, 77, 8, 2, 16, 0.3),
          (1200, 264, 8, 4, 8, 0.5), (1101, 33, 64, 32, 4, 0.0), (1500, 48, 8, 1, 16, 0.0),
          (1027, 131, 8, 7, 16, 0.9)]


def _shape_id(v):
    return "x".join(map(str, v)) if isinstance(v, tuple) else str(v).replace("torch.", "")


shapes = pytest.mark.parametrize("shape", SHAPES, ids=_shape_id)


# --------------------------------------------------------------------------
# dispatch
# --------------------------------------------------------------------------

@shapes
@pytest.mark.parametrize("dtype", [BF, FL, E4], ids=_shape_id)
def test_dispatch_copies_rows_clears_padding_and_leaves_the_rest(shape, dtype):
    M, H, E, k, BS, skipped = shape
    ids, w, t = route(M, E, k, BS, 10 + M, skipped)
    n, perm = M * k, perm_of(t, M, k)
    g = gen(20 + M)
    scales = {}
    if dtype == E4:
        x = randn(g, M, H, scale=60.0).clamp(-448, 448).to(E4)
        blocks = -(-H // 128)
        scales = dict(x_scale=torch.rand(M, blocks, generator=g, device="cuda"),
                      rows_scale=torch.full((t["max_total"], blocks), 7.0, device="cuda"))
    else:
        x = randn(g, M, H, dtype=dtype)
    rows = torch.full((t["max_total"], H), 3.0, device="cuda").to(dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.moe_dispatch(x, t, k, rows=rows, err_word=err, **scales)
    torch.cuda.synchronize()
    assert int(err) == 0
    pad, behind = padding(t, n)

    def check(out, src, filled):
        real = perm >= 0
        tok = torch.arange(M, device="cuda")[:, None].expand(M, k)
        assert torch.equal(bits(out[perm[real]]), bits(src[tok[real]]))
        assert not bits(out[pad]).any()
        assert torch.equal(bits(out[behind]), bits(filled[behind]))
    if dtype == E4:
        assert got[0] is rows
        check(rows.view(torch.uint8), x.view(torch.uint8),
              torch.full_like(rows.float(), 3.0).to(E4).view(torch.uint8))
        check(got[1], scales["x_scale"], torch.full_like(got[1], 7.0))
    else:
        check(rows, x, torch.full_like(rows, 3.0))


@shapes
@pytest.mark.parametrize("dtype", [BF, HF, FL], ids=_shape_id)
def test_dispatch_gradient(shape, dtype):
    M, H, E, k, BS, skipped = shape
    _, _, t = route(M, E, k, BS, 30 + M, skipped)
    perm = perm_of(t, M, k)
    drows = randn(gen(31), t["max_total"], H, dtype=dtype)
    pad, behind = padding(t, M * k)
    drows[pad | behind] = float("nan")   # never read
    v = taken(drows, perm)
    dx = moe.moe_dispatch_backward(drows, t, M, k)
    assert dx.dtype == dtype
    close(dx, v.sum(1), v.abs().sum(1), k * U)
    assert not dx[(perm < 0).all(1)].any()


@pytest.mark.parametrize("H,shift", [(264, 0), (264, 4), (1028, 0), (999, 0), (999, 3), (17, 1),
                                     (1, 0), (8, 5), (2051, 7)])
@pytest.mark.parametrize("dtype", [BF, FL], ids=_shape_id)
def test_nothing_outside_the_outputs_is_written(H, shift, dtype):
    """Outputs inside larger buffers, at every kind of alignment, with guards
    on both sides; the same bits as in buffers of their own."""
    M, k, E = 13, 3, 4
    _, w, t = route(M, E, k, 8, 130)
    n = t["max_total"]
    g = gen(131)
    x, r, dout = (randn(g, M, H, dtype=dtype) for _ in range(3))
    rows, weight = randn(g, n, H, dtype=dtype), randn(g, H, dtype=dtype)
    made = []

    def guarded(count):
        buf = torch.full((count * H + 64,), 77.0, dtype=dtype, device="cuda")
        made.append((buf, count))
        return buf[32 + shift: 32 + shift + count * H].view(count, H)
    total = int(t["num_tokens_post_padded"])
    a = moe.moe_dispatch(x, t, k, rows=guarded(n))[:total]
    b = moe.moe_dispatch(x, t, k)[:total]
    pairs_ = [(a, b), (moe.moe_dispatch_backward(rows, t, M, k, dx=guarded(M)),
                       moe.moe_dispatch_backward(rows, t, M, k)),
              (moe.moe_combine(rows, w, t, out=guarded(M)), moe.moe_combine(rows, w, t)),
              (moe.moe_combine_backward(dout, rows, w, t, drows=guarded(n))[0][:total],
               moe.moe_combine_backward(dout, rows, w, t)[0][:total])]
    o = moe.moe_add_rmsnorm(x, weight, residual=r, want=("out", "sum", "rstd"))
    p = moe.moe_add_rmsnorm(x, weight, residual=r, out=dict(out=guarded(M), sum=guarded(M)))
    pairs_ += [(p["out"], o["out"]), (p["sum"], o["sum"]),
               (moe.moe_add_rmsnorm_backward(dout, r, weight, o["rstd"], dsum=x, dx=guarded(M))[0],
                moe.moe_add_rmsnorm_backward(dout, r, weight, o["rstd"], dsum=x)[0])]
    torch.cuda.synchronize()
    for i, (got, want) in enumerate(pairs_):
        assert torch.equal(bits(got), bits(want)), i
    for i, (buf, count) in enumerate(made):
        assert (buf[: 32 + shift] == 77.0).all() and (buf[32 + shift + count * H:] == 77.0).all(), i


@pytest.mark.parametrize("H,start,width", [(256, 8, 512), (256, 1, 400), (100, 4, 104),
                                           (33, 3, 70), (256, 0, 0)])
def test_dispatch_of_strided_and_misaligned_rows(H, start, width):
    """Views into wider buffers, at 16-byte and at 2-byte offsets, and one row
    for every token (stride 0)."""
    M, k = 9, 2
    _, _, t = route(M, 8, k, 4, 40)
    g = gen(41)
    for dtype in (BF, FL):
        x = (randn(g, 1, H, dtype=dtype).expand(M, H) if width == 0
             else randn(g, M, width, dtype=dtype)[:, start: start + H])
        a = moe.moe_dispatch(x, t, k, rows=torch.zeros(t["max_total"], H, dtype=dtype,
                                                       device="cuda"))
        b = moe.moe_dispatch(x.contiguous(), t, k,
                             rows=torch.zeros(t["max_total"], H, dtype=dtype, device="cuda"))
        assert torch.equal(bits(a), bits(b))
        assert torch.equal(a[perm_of(t, M, k)[:, 1]], x)
    # an output at an odd place
    buf = torch.zeros(t["max_total"] * H + 1, dtype=BF, device="cuda")
    x = randn(g, M, H, dtype=BF)
    c = moe.moe_dispatch(x, t, k, rows=buf[1:].view(t["max_total"], H))
    assert torch.equal(c[perm_of(t, M, k)[:, 0]], x) and float(buf[0]) == 0


# --------------------------------------------------------------------------
# combine
# --------------------------------------------------------------------------

PAIRS = [(BF, BF), (HF, HF), (FL, FL), (FL, BF), (FL, HF)]
pairs = pytest.mark.parametrize("rt,ot", PAIRS, ids=_shape_id)


@shapes
@pairs
def test_combine_matches_float64(shape, rt, ot):
    M, H, E, k, BS, skipped = shape
    _, w, t = route(M, E, k, BS, 50 + M, skipped)
    perm = perm_of(t, M, k)
    rows = randn(gen(51), t["max_total"], H, dtype=rt)
    pad, behind = padding(t, M * k)
    rows[pad | behind] = float("nan")
    out = moe.moe_combine(rows, w, t, out_dtype=ot)
    v = taken(rows, perm) * w.double()[:, :, None]
    assert out.dtype == ot
    close(out, v.sum(1), v.abs().sum(1), k * U)
    assert not out[(perm < 0).all(1)].any()


@shapes
@pairs
def test_combine_gradient_matches_float64(shape, rt, ot):
    M, H, E, k, BS, skipped = shape
    _, w, t = route(M, E, k, BS, 60 + M, skipped)
    perm = perm_of(t, M, k)
    g = gen(61)
    rows, dout = randn(g, t["max_total"], H, dtype=rt), randn(g, M, H, dtype=ot)
    pad, behind = padding(t, M * k)
    rows[pad | behind] = float("nan")
    drows = torch.full((t["max_total"], H), 3.0, dtype=rt, device="cuda")
    got, dw = moe.moe_combine_backward(dout, rows, w, t, drows=drows)
    assert got is drows
    real = perm >= 0
    d = dout.double()[:, None, :].expand(M, k, H)
    ref = w.double()[:, :, None] * d
    close(drows[perm[real]], ref[real], ref[real].abs(), U)
    assert not bits(drows[pad]).any()
    assert (drows[behind] == 3.0).all()
    v = taken(rows, perm) * d
    close(dw, v.sum(2), v.abs().sum(2), H * U)
    assert not dw[~real].any()
    # one output alone has the same bits
    alone, none = moe.moe_combine_backward(dout, None, w, t, want_dtopk_w=False, rows_dtype=rt,
                                           drows=torch.full_like(drows, 3.0))
    assert none is None and torch.equal(bits(alone), bits(drows))
    none, alone = moe.moe_combine_backward(dout, rows, w, t, want_drows=False)
    assert none is None and torch.equal(bits(alone), bits(dw))


def test_combine_gradient_of_broadcast_and_strided_dout():
    """A gradient with stride 0 (one row for all tokens) and a slice."""
    M, k, H = 21, 3, 136
    _, w, t = route(M, 8, k, 8, 70)
    g = gen(71)
    rows = randn(g, t["max_total"], H, dtype=BF)
    for dout in (randn(g, 1, H, dtype=BF).expand(M, H), randn(g, M, 300, dtype=BF)[:, 5: 5 + H],
                 randn(g, M, 304, dtype=BF)[:, 8: 8 + H]):
        a = moe.moe_combine_backward(dout, rows, w, t,
                                     drows=torch.zeros(t["max_total"], H, dtype=BF, device="cuda"))
        b = moe.moe_combine_backward(dout.contiguous(), rows, w, t,
                                     drows=torch.zeros(t["max_total"], H, dtype=BF, device="cuda"))
        for x, y in zip(a, b):
            assert torch.equal(bits(x), bits(y))


def test_values_that_are_not_finite_stay_in_their_rows():
    """An infinity or a NaN in one token's or one slot's row reaches that token
    and no other."""
    M, k, H = 12, 2, 264
    _, w, t = route(M, 8, k, 4, 80)
    perm = perm_of(t, M, k)
    rows = randn(gen(81), t["max_total"], H, dtype=BF)
    rows[perm[3, 1], 5] = float("inf")
    rows[perm[7, 0], 9] = float("nan")
    out = moe.moe_combine(rows, w, t)
    off = ~torch.isfinite(out)
    assert off[3, 5] and off[7, 9] and int(off.sum()) == 2 and float(out[3, 5]) == math.inf
    _, dw = moe.moe_combine_backward(torch.ones(M, H, dtype=BF, device="cuda"), rows, w, t)
    off = ~torch.isfinite(dw)
    assert off[3, 1] and off[7, 0] and int(off.sum()) == 2


# --------------------------------------------------------------------------
# positions outside the rows, no rows, rows past 2^31 elements
# --------------------------------------------------------------------------

def test_bad_positions_are_skipped_and_reported():
    M, k, H = 6, 2, 72
    _, w, t = route(M, 4, k, 8, 90)
    good = perm_of(t, M, k).clone()
    t = dict(t, token_to_perm=t["token_to_perm"].clone())
    t["token_to_perm"][3] = t["max_total"]          # slot (1, 1)
    t["token_to_perm"][8] = -2                      # slot (4, 0)
    t["token_to_perm"][9] = 2 ** 31 - 1             # slot (4, 1)
    perm = good.clone()
    perm[1, 1] = perm[4, 0] = perm[4, 1] = -1
    g = gen(91)
    x, rows = randn(g, M, H, dtype=BF), randn(g, t["max_total"], H, dtype=BF)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def flagged():
        v = int(err)
        err.zero_()
        return v == moe.MOE_ERR_BAD_POSITION
    out = moe.moe_combine(rows, w, t, err_word=err)
    v = taken(rows, perm) * w.double()[:, :, None]
    close(out, v.sum(1), v.abs().sum(1), k * U)
    assert flagged() and not out[4].any()
    dx = moe.moe_dispatch_backward(rows, t, M, k, err_word=err)
    v = taken(rows, perm)
    close(dx, v.sum(1), v.abs().sum(1), k * U)
    assert flagged()
    buf = torch.full_like(rows, 3.0)
    moe.moe_dispatch(x, t, k, rows=buf, err_word=err)
    assert flagged()
    assert torch.equal(buf[good[0]], x[0].expand(k, H)) and (buf[good[4]] == 3.0).all()
    dr, dw = moe.moe_combine_backward(x, rows, w, t, drows=torch.full_like(rows, 3.0),
                                      err_word=err)
    assert flagged() and not dw[perm < 0].any() and (dr[good[4]] == 3.0).all()
    moe.moe_combine(rows, w, t)   # without an error word the slots are skipped all the same


def test_no_tokens():
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    t = moe.moe_align(ids, 8, 16)
    w = torch.empty(0, 2, device="cuda")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    rows = moe.moe_dispatch(x, t, 2)
    assert rows.shape == (0, 64)
    assert moe.moe_dispatch_backward(rows, t, 0, 2).shape == (0, 64)
    assert moe.moe_combine(rows, w, t).shape == (0, 64)
    dr, dw = moe.moe_combine_backward(x, rows, w, t)
    assert dr.shape == (0, 64) and dw.shape == (0, 2)
    assert moe.moe_topk_softmax_backward(ids, w, w, 8).shape == (0, 8)
    weight = torch.ones(64, dtype=BF, device="cuda")
    o = moe.moe_add_rmsnorm(x, weight, residual=x, want=("out", "sum", "rstd", "codes", "scale"))
    dx, dweight = moe.moe_add_rmsnorm_backward(x, o["sum"], weight, o["rstd"])
    assert dx.shape == (0, 64) and dweight.shape == (64,) and not dweight.any()


def test_rows_past_two_to_the_thirty_one_elements():
    """Byte and element offsets of the last rows need 64 bits."""
    M, H, E, k, BS = 33000, 8192, 16, 8, 16
    _, w, t = route(M, E, k, BS, 95)
    perm = perm_of(t, M, k)
    assert int(t["num_tokens_post_padded"]) * H > 2 ** 31
    x = randn(gen(96), M, H, dtype=BF)
    rows = torch.zeros(t["max_total"], H, dtype=BF, device="cuda")
    moe.moe_dispatch(x, t, k, rows=rows)
    last = int(torch.argmax(perm.max(1).values))
    for tok in (0, last, M - 1):
        assert torch.equal(rows[perm[tok]], x[tok].expand(k, H))
    out = moe.moe_combine(rows, w, t)
    for tok in (0, last, M - 1):
        v = x[tok].double() * w[tok].double()[:, None]
        close(out[tok], v.sum(0), v.abs().sum(0), k * U)
    dr, dw = moe.moe_combine_backward(x, rows, w, t)
    for tok in (0, last, M - 1):
        ref = w[tok].double()[:, None] * x[tok].double()
        close(dr[perm[tok]], ref, ref.abs(), U)
        sq = x[tok].double().square().sum().expand(k)
        close(dw[tok], sq, sq, H * U)


# --------------------------------------------------------------------------
# gradient of the top-k softmax
# --------------------------------------------------------------------------

def topk_grad_ref(ids, w, dw, E):
    w, dw = w.double(), dw.double()
    g = w * (dw - (w * dw).sum(1, keepdim=True))
    here = (ids >= 0) & (ids < E)
    out = torch.zeros(ids.shape[0], E, dtype=torch.float64, device=ids.device)
    out.scatter_add_(1, ids.long().clamp(0, E - 1), torch.where(here, g, torch.zeros_like(g)))
    mag = torch.zeros_like(out)
    m = w.abs() * (dw.abs() + (w * dw).abs().sum(1, keepdim=True))
    mag.scatter_add_(1, ids.long().clamp(0, E - 1), torch.where(here, m, torch.zeros_like(m)))
    return out, mag


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (8, 128, 8), (5, 33, 32), (301, 1024, 10),
                                   (4, 2, 2), (1000, 256, 8), (3, 31, 5)])
def test_topk_softmax_gradient(M, E, k):
    g = gen(100 + M)
    logits = randn(g, M, E)
    ids, w = moe.moe_topk_softmax(logits, k)
    dw = randn(g, M, k)
    got = moe.moe_topk_softmax_backward(ids, w, dw, E)
    ref, mag = topk_grad_ref(ids, w, dw, E)
    # the dot product of k terms, one subtraction, one product
    close(got, ref, mag, (k + 3) * U)
    assert int((got != 0).sum()) <= M * k


def test_topk_softmax_gradient_against_differences():
    """The gradient of sum(c * softmax over the selected logits) by central
    differences of the float64 function, at a fixed selection."""
    M, E, k = 6, 40, 5
    g = gen(110)
    logits, c = randn(g, M, E), randn(g, M, k)
    ids, w = moe.moe_topk_softmax(logits, k)
    got = moe.moe_topk_softmax_backward(ids, w, c, E).double()
    l64 = logits.double()
    step = 1e-5

    def f(l):
        return (torch.softmax(torch.gather(l, 1, ids.long()), 1) * c.double()).sum(1)
    for e in range(E):
        d = torch.zeros_like(l64)
        d[:, e] = step
        num = (f(l64 + d) - f(l64 - d)) / (2 * step)
        # third derivatives of a softmax are below 1; the weights w are the
        # router's, within 2e-6 of softmax
        assert float((got[:, e] - num).abs().max()) < 2e-5


def test_topk_softmax_gradient_of_repeated_and_missing_ids():
    ids = torch.tensor([[2, 2, 5], [0, -1, 7], [1, 1, 1], [8, 3, 4]], dtype=torch.int32,
                       device="cuda")
    g = gen(120)
    w, dw = torch.softmax(randn(g, 4, 3), 1), randn(g, 4, 3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.moe_topk_softmax_backward(ids, w, dw, 8, err_word=err)
    ref, mag = topk_grad_ref(ids, w, dw, 8)
    close(got, ref, mag, 8 * U)
    assert int(err) == moe.MOE_ERR_BAD_ID
    err.zero_()
    moe.moe_topk_softmax_backward(ids[::2].contiguous(), w[::2].contiguous(),
                                  dw[::2].contiguous(), 8, err_word=err)
    assert int(err) == 0


# --------------------------------------------------------------------------
# residual addition and RMS norm
# --------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (2, 128), (9, 200), (4, 257), (8, 2048), (33, 2880),
               (3, 4096), (2, 5001), (7, 8192), (2, 12345), (2, 16384), (600, 256), (6, 2884),
               (400, 513)]
TYPES = [(BF, BF), (BF, FL), (HF, HF), (HF, FL), (FL, FL)]
norm_shapes = pytest.mark.parametrize("M,H", NORM_SHAPES)
types = pytest.mark.parametrize("dt,wt", TYPES, ids=_shape_id)


def norm_inputs(M, H, dt, wt, seed):
    g = gen(seed)
    return (randn(g, M, H, dtype=dt), randn(g, M, H, dtype=dt, scale=3.0),
            (1 + randn(g, H, scale=0.2)).to(wt))


def norm_ref(x, r, w, eps):
    """(sum as stored, rstd, s * w, out) in float64."""
    s = x if r is None else (x.double() + r.double()).to(x.dtype)
    s = s.double()
    rstd = 1 / torch.sqrt(s.square().mean(1) + eps)
    p = s * w.double()
    return s, rstd, p, p * rstd[:, None]


def e4m3_step(q):
    """The step of E4M3 at |q| <= 448."""
    e = (torch.frexp(q)[1].long() - 1).clamp(min=-6) - 3
    return ((e + 1023) << 52).view(torch.float64)   # 2^e (torch.ldexp is off in the last bit)


def check_codes(codes, scale, p, rstd, dt):
    M, H = p.shape
    blocks = -(-H // 128)
    assert codes.shape == (M, H) and scale.shape == (M, blocks)
    most = torch.stack([p[:, 128 * b: 128 * (b + 1)].abs().amax(1) for b in range(blocks)], 1)
    want = (most * rstd[:, None] / 448).clamp(min=2.0 ** -126)
    assert ((scale.double() - want).abs() <= 40 * U * want).all()
    q = p * rstd[:, None] / want.repeat_interleave(128, 1)[:, :H]
    c = codes.float().double()
    err = U if dt != FL else 4 * U
    low = want.repeat_interleave(128, 1)[:, :H] == 2.0 ** -126   # rstd is in the quotient there
    err = torch.where(low, torch.full_like(q, 40 * U), torch.full_like(q, err))
    assert ((c - q).abs() <= e4m3_step(q) / 2 + 2 * err * q.abs()).all()


@norm_shapes
@types
def test_add_rmsnorm_matches_float64(M, H, dt, wt):
    x, r, w = norm_inputs(M, H, dt, wt, 200 + H)
    eps = 1e-6
    o = moe.moe_add_rmsnorm(x, w, eps, residual=r, want=("out", "sum", "rstd", "codes", "scale"))
    s, rstd, p, v = norm_ref(x, r, w, eps)
    assert torch.equal(o["sum"].double(), s)
    assert ((o["rstd"].double() - rstd).abs() <= 32 * U * rstd).all()
    close(o["out"], v, v.abs(), 36 * U)
    check_codes(o["codes"], o["scale"], p, rstd, dt if wt != FL else FL)
    # without a residual, and each output alone: the same bits
    q = moe.moe_add_rmsnorm(o["sum"], w, eps, want=("out", "sum"))
    assert torch.equal(bits(q["out"]), bits(o["out"])) and torch.equal(bits(q["sum"]),
                                                                       bits(o["sum"]))
    for name in ("out", "sum", "rstd"):
        one = moe.moe_add_rmsnorm(x, w, eps, residual=r, want=(name,))
        assert set(one) == {name} and torch.equal(bits(one[name]), bits(o[name]))
    two = moe.moe_add_rmsnorm(x, w, eps, residual=r, want=("codes", "scale"))
    assert torch.equal(bits(two["codes"]), bits(o["codes"]))
    assert torch.equal(bits(two["scale"]), bits(o["scale"]))


def test_codes_of_bf16_rows_are_the_nearest_exactly():
    """bf16 rows and weights: the quotient's products are exact in fp32 and its
    rounding cannot reach or leave a tie, so every code is the nearest one
    (ties to even) to the exact quotient."""
    M, H = 64, 4096
    x, r, w = norm_inputs(M, H, BF, BF, 7)
    o = moe.moe_add_rmsnorm(x, w, residual=r, want=("codes", "scale"))
    p = (x.double() + r.double()).to(BF).double() * w.double()
    most = p.abs().view(M, H // 128, 128).amax(2).repeat_interleave(128, 1)
    q = p * 448 / most   # float64: the product is exact, the quotient off by 2^-53
    step = e4m3_step(q)
    assert torch.equal(o["codes"].float().double(), torch.round(q / step) * step)


def test_norm_of_rows_without_size_and_of_extremes():
    H = 300
    w = torch.ones(H, dtype=BF, device="cuda")
    x = torch.zeros(8, H, dtype=BF, device="cuda")
    x[1] = 2.0 ** -60                      # squares far below eps
    x[2] = 2.0 ** 55                       # squares up to 2^110
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5, 299] = 1.0                        # the last, short block alone
    x[6] = -1.0
    o = moe.moe_add_rmsnorm(x, w, 1e-6, want=("out", "rstd", "codes", "scale"))
    f, c, sc = o["out"].float(), o["codes"].float(), o["scale"]
    assert not f[0].any() and not c[0].any() and (sc[0] == 2.0 ** -126).all()
    assert float(o["rstd"][0]) == pytest.approx(1e3, rel=1e-6)
    close(o["out"][1], x[1].double() * 1e3, x[1].double() * 1e3, 36 * U)
    assert (f[2] == 1).all() and (c[2] == 448).all()
    assert float(o["rstd"][3]) == 0 and torch.isnan(f[3, 7]) and not f[3, :7].any()
    assert torch.isnan(f[4]).all() and torch.isnan(c[4]).all() and torch.isnan(sc[4]).all()
    assert (sc[5, :2] == 2.0 ** -126).all() and float(c[5, 299]) == 448 and not c[5, :299].any()
    assert (f[6] == -1).all() and (c[6] == -448).all()
    # scales below 2^-126 are held there
    tiny_row = torch.full((1, H), 2.0 ** -126, dtype=FL, device="cuda")
    o = moe.moe_add_rmsnorm(tiny_row, torch.ones(H, device="cuda"), 1.0, want=("codes", "scale"))
    assert (o["scale"] == 2.0 ** -126).all() and (o["codes"].float() == 1).all()


@pytest.mark.parametrize("dtype,lo,hi", [(BF, -0x7F80, 0x7F80), (HF, -0x7C00, 0x7C00)],
                         ids=["bfloat16", "float16"])
def test_sums_of_any_two_finite_values(dtype, lo, hi):
    """Random finite bit patterns, subnormal ones and near overflow among them:
    the stored sum is the exact sum rounded once."""
    g = gen(140)
    M, H = 64, 1024

    def any_finite():
        m = torch.randint(0, hi, (M, H), generator=g, device="cuda")
        sign = torch.randint(0, 2, (M, H), generator=g, device="cuda") << 15
        return (m | sign).to(torch.int32).to(torch.int16).view(dtype)
    x, r = any_finite(), any_finite()
    x[0, :512] = (torch.randint(0, 128, (512,), generator=g, device="cuda")).to(
        torch.int16).view(dtype)   # subnormal + subnormal
    r[0, :512] = x[0, :512].flip(0)
    w = torch.ones(H, dtype=dtype, device="cuda")
    s = moe.moe_add_rmsnorm(x, w, residual=r, want=("sum",))["sum"]
    # the fp32 sum of two such values is exact or far from a tie (their bits
    # would span more than 24), so rounding it once more is rounding once
    assert torch.equal(bits(s), bits((x.float() + r.float()).to(dtype)))


def test_norm_in_place_and_of_strided_rows():
    M, H = 6, 520
    for dt in (BF, FL):
        x, r, w = norm_inputs(M, H, dt, FL, 31)
        want = moe.moe_add_rmsnorm(x, w, residual=r, want=("out", "sum"))
        xc, rc = x.clone(), r.clone()
        o = moe.moe_add_rmsnorm(xc, w, residual=rc, out=dict(sum=rc, out=xc))
        assert torch.equal(bits(rc), bits(want["sum"])) and torch.equal(bits(xc),
                                                                        bits(want["out"]))
        for start, width in ((8, 560), (3, 533)):
            wide = torch.zeros(M, width, dtype=dt, device="cuda")
            wide[:, start: start + H] = x
            o = moe.moe_add_rmsnorm(wide[:, start: start + H], w, residual=r,
                                    want=("out", "sum"))
            for k in o:
                assert torch.equal(bits(o[k]), bits(want[k]))
        one = moe.moe_add_rmsnorm(x, w, residual=r[:1].expand(M, H), want=("out",))
        two = moe.moe_add_rmsnorm(x, w, residual=r[:1].repeat(M, 1), want=("out",))
        assert torch.equal(bits(one["out"]), bits(two["out"]))


@norm_shapes
@types
def test_add_rmsnorm_gradient_matches_float64(M, H, dt, wt):
    x, s, w = norm_inputs(M, H, dt, wt, 300 + H)
    dsum = randn(gen(301), M, H, dtype=dt)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    d, xh = x.double(), s.double() * rstd.double()[:, None]
    gw = d * w.double()
    mean = (gw * xh).mean(1, keepdim=True)
    mag = rstd.double()[:, None] * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    # 32 terms a thread, 5 levels, 16 warps, then eight roundings
    for extra in (dsum, None):
        ref = rstd.double()[:, None] * (gw - xh * mean)
        m = mag
        if extra is not None:
            ref, m = ref + extra.double(), mag + extra.double().abs()
        dx, dw = moe.moe_add_rmsnorm_backward(x, s, w, rstd, dsum=extra)
        close(dx, ref, m, 64 * U)
        # the rows of a CTA one after the other, its row groups, the CTAs
        v = d * xh
        close(dw, v.sum(0), v.abs().sum(0), (M / 456 + 8 + 456 / 16 + 16 + 2) * U)
        alone, none = moe.moe_add_rmsnorm_backward(x, s, w, rstd, dsum=extra, want_dweight=False)
        assert none is None and torch.equal(bits(alone), bits(dx))


def test_add_rmsnorm_gradient_of_many_rows_is_the_same_every_time():
    M, H = 5003, 1024
    x, s, w = norm_inputs(M, H, BF, BF, 400)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    dx, dw = moe.moe_add_rmsnorm_backward(x, s, w, rstd)
    v = x.double() * s.double() * rstd.double()[:, None]
    close(dw, v.sum(0), v.abs().sum(0), (M / 456 + 60) * U)
    ws = torch.full((moe.add_rmsnorm_backward_workspace_bytes(M, H),), 255, dtype=torch.uint8,
                    device="cuda")   # it needs no clearing
    for _ in range(3):
        a, b = moe.moe_add_rmsnorm_backward(x, s, w, rstd, workspace=ws)
        assert torch.equal(bits(a), bits(dx)) and torch.equal(bits(b), bits(dw))
    # in place, and strided inputs
    xc = x.clone()
    a, _ = moe.moe_add_rmsnorm_backward(xc, s, w, rstd, dx=xc)
    assert a is xc and torch.equal(bits(xc), bits(dx))
    wide = torch.zeros(M, H + 3, dtype=BF, device="cuda")
    wide[:, 3:] = x
    a, b = moe.moe_add_rmsnorm_backward(wide[:, 3:], s, w, rstd)
    assert torch.equal(bits(a), bits(dx)) and torch.equal(bits(b), bits(dw))


@pytest.mark.parametrize("H", [256, 2884, 77])
def test_add_rmsnorm_gradient_of_broadcast_rows(H):
    """A gradient that is one row for all (stride 0), as a sum's is, and a
    strided sum; the same bits as from dense copies."""
    M = 37
    x, s, w = norm_inputs(M, H, BF, FL, 450)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    wide = torch.zeros(M, H + 24, dtype=BF, device="cuda")
    wide[:, 8: 8 + H] = s
    one = x[:1].expand(M, H)
    a, b = moe.moe_add_rmsnorm_backward(one, wide[:, 8: 8 + H], w, rstd, dsum=one)
    c, d = moe.moe_add_rmsnorm_backward(one.contiguous(), s, w, rstd, dsum=one.contiguous())
    assert torch.equal(bits(a), bits(c)) and torch.equal(bits(b), bits(d))
    # a workspace for more rows serves fewer
    ws = torch.empty(moe.add_rmsnorm_backward_workspace_bytes(10 * M, H), dtype=torch.uint8,
                     device="cuda")
    for n in (1, 5, M):
        p = moe.moe_add_rmsnorm_backward(x[:n], s[:n], w, rstd[:n], workspace=ws)
        q = moe.moe_add_rmsnorm_backward(x[:n], s[:n], w, rstd[:n])
        assert torch.equal(bits(p[0]), bits(q[0])) and torch.equal(bits(p[1]), bits(q[1]))


def test_add_rmsnorm_gradient_against_differences():
    """fp32 rows against central differences of the float64 norm, along random
    directions of the input and of the weight."""
    M, H, eps = 4, 96, 1e-3
    x, r, w = norm_inputs(M, H, FL, FL, 500)
    g = gen(501)
    dout, dsum = randn(g, M, H), randn(g, M, H)
    o = moe.moe_add_rmsnorm(x, w, eps, residual=r, want=("sum", "rstd"))
    dx, dw = moe.moe_add_rmsnorm_backward(dout, o["sum"], w, o["rstd"], dsum=dsum)

    def f(s, w):
        y = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w
        return (y * dout.double()).sum() + (s * dsum.double()).sum()
    s, w64, h = o["sum"].double(), w.double(), 1e-5
    for seed in range(4):
        a, b = randn(gen(510 + seed), M, H).double(), randn(gen(520 + seed), H).double()
        num = (f(s + h * a, w64) - f(s - h * a, w64)) / (2 * h)
        assert float(num) == pytest.approx(float((dx.double() * a).sum()), rel=1e-4, abs=1e-4)
        num = (f(s, w64 + h * b) - f(s, w64 - h * b)) / (2 * h)
        assert float(num) == pytest.approx(float((dw.double() * b).sum()), rel=1e-4, abs=1e-4)


# --------------------------------------------------------------------------
# batch invariance, streams, graphs, refusals
# --------------------------------------------------------------------------

def test_a_rows_bits_do_not_depend_on_the_batch():
    M, H, k, E = 200, 2880, 4, 16
    ids, w, t = route(M, E, k, 16, 600)
    perm = perm_of(t, M, k)
    g = gen(601)
    rows, x, r = (randn(g, n, H, dtype=BF) for n in (t["max_total"], M, M))
    weight = torch.ones(H, dtype=BF, device="cuda")
    out = moe.moe_combine(rows, w, t)
    dr, dw = moe.moe_combine_backward(x, rows, w, t)
    o = moe.moe_add_rmsnorm(x, weight, residual=r, want=("out", "rstd"))
    dx, _ = moe.moe_add_rmsnorm_backward(x, r, weight, o["rstd"])
    for n in (1, 7):
        sub = dict(t, token_to_perm=t["token_to_perm"][: n * k].contiguous())
        assert torch.equal(bits(moe.moe_combine(rows, w[:n], sub)), bits(out[:n]))
        _, b = moe.moe_combine_backward(x[:n], rows, w[:n], sub, want_drows=False)
        assert torch.equal(bits(b), bits(dw[:n]))
        p = moe.moe_add_rmsnorm(x[:n], weight, residual=r[:n], want=("out",))
        assert torch.equal(bits(p["out"]), bits(o["out"][:n]))
        a, _ = moe.moe_add_rmsnorm_backward(x[:n], r[:n], weight, o["rstd"][:n])
        assert torch.equal(bits(a), bits(dx[:n]))


def chain(x, r, weight, wr, E, k, BS, dout, stream=None):
    """Residual addition, norm, router, alignment, dispatch, a stand-in for the
    experts (each row times its expert's number + 1), combination; then every
    gradient back to x."""
    o = moe.moe_add_rmsnorm(x, weight, residual=r, want=("out", "sum", "rstd"), stream=stream)
    logits = moe.moe_router_logits(o["out"], wr, stream=stream)
    ids, w = moe.moe_topk_softmax(logits, k, stream=stream)
    t = moe.moe_align(ids, E, BS, stream=stream)
    rows = moe.moe_dispatch(o["out"], t, k, stream=stream)
    factor = (t["sorted_expert_ids"].float() + 1).repeat_interleave(BS)[:, None]
    y = (rows.float() * factor).to(BF)
    out = moe.moe_combine(y, w, t, stream=stream)
    dy, dw = moe.moe_combine_backward(dout, y, w, t, stream=stream)
    drows = (dy.float() * factor).to(BF)
    dlogits = moe.moe_topk_softmax_backward(ids, w, dw, E, stream=stream)
    dn = moe.moe_dispatch_backward(drows, t, x.shape[0], k, stream=stream)
    dn = (dn.float() + dlogits @ wr.float()).to(BF)
    dx, dweight = moe.moe_add_rmsnorm_backward(dn, o["sum"], weight, o["rstd"], dsum=dout,
                                               stream=stream)
    return dict(out=out, sum=o["sum"], ids=ids, dx=dx, dweight=dweight,
                dwr=dlogits.T @ o["out"].float())


def chain_inputs(M, H, E, seed):
    g = gen(seed)
    return (randn(g, M, H, dtype=BF), randn(g, M, H, dtype=BF),
            (1 + randn(g, H, scale=0.1)).to(BF), randn(g, E, H, dtype=BF, scale=H ** -0.5),
            randn(g, M, H, dtype=BF))


def test_the_block_and_its_gradients_against_autograd():
    """The chain as a training step runs it, against float64 autograd of the
    same function with the same selection.  Six bf16 roundings lie between x
    and a gradient (each 2^-8 of a value at most, 2^-9 as a typical error), so
    6 * 2^-9 = 1.2 percent of the norm bounds what they add up to."""
    M, H, E, k, BS = 50, 256, 16, 4, 8
    x, r, weight, wr, dout = chain_inputs(M, H, E, 700)
    got = chain(x, r, weight, wr, E, k, BS, dout)
    s = (x.double() + r.double()).to(BF).double().requires_grad_()
    w64, wr64 = weight.double().requires_grad_(), wr.double().requires_grad_()
    nrm = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * w64
    lg = nrm @ wr64.T
    pw = torch.softmax(torch.gather(lg, 1, got["ids"].long()), 1)
    out = nrm * (pw * (got["ids"].double() + 1)).sum(1, keepdim=True)
    loss = (out * dout.double()).sum() + (s * dout.double()).sum()
    loss.backward()
    for name, ref in (("out", out.detach()), ("dx", s.grad), ("dweight", w64.grad),
                      ("dwr", wr64.grad)):
        rel = float((got[name].double() - ref).norm() / ref.norm())
        assert rel < 6 * 2.0 ** -9, (name, rel)


def test_captured_chain_replays_on_new_inputs():
    M, H, E, k, BS = 24, 512, 16, 2, 8
    a, b = chain_inputs(M, H, E, 800), chain_inputs(M, H, E, 801)
    want = [chain(*v[:4], E, k, BS, v[4]) for v in (a, b)]
    held = [v.clone() for v in a]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(*held[:4], E, k, BS, held[4])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(*held[:4], E, k, BS, held[4])
    for inputs, ref in ((b, want[1]), (a, want[0]), (b, want[1])):
        for dst, src in zip(held, inputs):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for name in ref:
            assert torch.equal(bits(got[name]), bits(ref[name])), name


def test_first_calls_can_be_captured():
    """A process whose first calls of these entry points are inside a capture."""
    code = """
import torch, expert_routing_alignment_gb300 as moe
moe.load()
torch.manual_seed(0)
M, H, E, k = 40, 4096, 8, 2
x, d = (torch.randn(M, H, device="cuda").bfloat16() for _ in range(2))
w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
ids, tw = moe.moe_topk_softmax(torch.randn(M, E, device="cuda"), k)
t = moe.moe_align(ids, E, 16)
nbytes = moe.add_rmsnorm_backward_workspace_bytes(4 * M, H)
ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
def run():
    o = moe.moe_add_rmsnorm(x, w, residual=d, want=("out", "sum", "rstd", "codes", "scale"))
    rows = moe.moe_dispatch(o["out"], t, k)
    r8, rs = moe.moe_dispatch(o["codes"], t, k, x_scale=o["scale"])
    out = moe.moe_combine(rows, tw, t)
    dr, dw = moe.moe_combine_backward(out, rows, tw, t)
    dx = moe.moe_dispatch_backward(dr, t, M, k)
    dl = moe.moe_topk_softmax_backward(ids, tw, dw, E)
    g, gw = moe.moe_add_rmsnorm_backward(dx, o["sum"], w, o["rstd"], workspace=ws)
    return out, dw, dl, g, gw, o["codes"].view(torch.uint8), o["scale"]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, run()):
    assert torch.equal(a, b)
print("captured")
"""
    import subprocess
    import sys
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]


def test_calls_on_two_streams_at_once():
    """Two chains at once, each on its own stream, the stream given by argument
    and by context; outputs that the calls make belong to their stream."""
    M, H, E, k, BS = 64, 1024, 32, 4, 16
    ins = [chain_inputs(M, H, E, 900 + i) for i in range(2)]
    want = [chain(*v[:4], E, k, BS, v[4]) for v in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = chain(*ins[i][:4], E, k, BS, ins[i][4])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for name in w:
            assert torch.equal(bits(g[name]), bits(w[name])), name
    weight, x = ins[0][2], ins[0][0]
    ref = moe.moe_add_rmsnorm(x, weight, want=("out",))["out"]
    torch.cuda.synchronize()
    for handle in (streams[0], streams[1].cuda_stream, 0):
        o = moe.moe_add_rmsnorm(x, weight, want=("out",), stream=handle)["out"]
        torch.cuda.synchronize()
        assert torch.equal(bits(o), bits(ref))


def test_refusals_reach_python():
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_add_rmsnorm(torch.zeros(1, 16385, dtype=BF, device="cuda"),
                            torch.zeros(16385, dtype=BF, device="cuda"))
    assert e.value.status == moe.MOE_EUNSUPPORTED
    with pytest.raises(moe.MoeError) as e:
        moe.moe_add_rmsnorm(x, torch.ones(64, dtype=HF, device="cuda"))
    assert e.value.status == moe.MOE_EUNSUPPORTED
    with pytest.raises(moe.MoeError) as e:
        moe.moe_add_rmsnorm(x, torch.ones(64, dtype=BF, device="cuda"), eps=-1.0)
    assert e.value.status == moe.MOE_EINVAL
    _, w, t = route(4, 8, 2, 8, 1)
    rows = torch.zeros(t["max_total"], 64, dtype=BF, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_combine(rows, w, t, out_dtype=FL)
    assert e.value.status == moe.MOE_EUNSUPPORTED
    with pytest.raises(ValueError):
        moe.moe_combine(rows, w.cpu(), t)
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm_backward(x, x, torch.ones(64, dtype=BF, device="cuda"),
                                     torch.ones(4))


# --------------------------------------------------------------------------
# with the decode layer
# --------------------------------------------------------------------------

LAYERS = [(synth.tiny(), 0), (synth.decode_fp8(8), 0), (synth.decode_fp8(8), 1),
          (synth.decode_fp8(8), 3), (synth.decode_nvfp4(8), 0)]
layers = pytest.mark.parametrize("shape,path", LAYERS, ids=lambda v: getattr(v, "name", str(v)))


def make_layer(shape, path, router=False):
    inp = synth.make_layer(shape, 1000, device="cuda")
    routed = moe.Experts.from_synth(inp.experts)
    shared = moe.Experts.from_synth(inp.shared) if inp.shared is not None else None
    wr = synth.make_router_weight(shape.E, shape.H, 2024, device="cuda") if router else None
    return inp, moe.LayerDesc(top_k=shape.top_k, block_size=shape.BS, routed=routed,
                              shared=shared, path=path, router_weight=wr)


@layers
def test_decode_block_is_the_norm_and_the_layer(shape, path):
    inp, layer = make_layer(shape, path, router=True)
    M, H = shape.M, shape.H
    g = gen(1100)
    res, weight = randn(g, M, H, dtype=BF), (1 + randn(g, H, scale=0.1)).to(BF)
    o = moe.moe_add_rmsnorm(inp.x, weight, 1e-5, residual=res, want=("out", "sum"))
    ws, ref = moe.alloc_workspace(layer, M), torch.empty(M, H, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_decode_layer(layer, o["out"], ref, ws, err_word=err)
    out, ws2 = torch.empty_like(ref), moe.alloc_workspace(layer, M)
    s, n = moe.moe_decode_block(layer, inp.x, res, weight, out, ws2, eps=1e-5, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for a, b in ((s, o["sum"]), (n, o["out"]), (out, ref)):
        assert torch.equal(bits(a), bits(b))
    # the residual stream in place, captured and replayed; and no residual
    held, out2 = res.clone(), torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_decode_block(layer, inp.x, held, weight, out2, ws2, eps=1e-5, sum_out=held,
                             normed=n)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(held), bits(s)) and torch.equal(bits(out2), bits(out))
    s, n = moe.moe_decode_block(layer, inp.x, None, weight, out2, ws2, eps=1e-5)
    assert torch.equal(bits(s), bits(inp.x))
    o = moe.moe_add_rmsnorm(inp.x, weight, 1e-5)
    assert torch.equal(bits(n), bits(o["out"]))


@layers
def test_router_gradient_behind_a_frozen_layer(shape, path):
    """What a layer call leaves in its workspace (fp32 expert rows by sorted
    position, ids, weights, positions) gives the logits' gradient: against
    float64 central differences of the loss with the rows held."""
    inp, layer = make_layer(shape, path)
    M, H, k, E = shape.M, shape.H, shape.top_k, shape.E
    ws, out = moe.alloc_workspace(layer, M), torch.empty(M, H, dtype=BF, device="cuda")
    moe.moe_decode_layer(layer, inp.x, out, ws, router_logits=inp.logits)
    v = moe.workspace_view(layer, M, ws)
    w, ids = v["topk_w"].view(M, k), v["topk_ids"].view(M, k)
    dout = randn(gen(1200), M, H, dtype=BF)
    none, dw = moe.moe_combine_backward(dout, v["y"], w, v, want_drows=False)
    assert none is None
    perm = perm_of(v, M, k)
    y = taken(v["y"], perm)
    prod = y * dout.double()[:, None, :]
    close(dw, prod.sum(2), prod.abs().sum(2), H * U)
    got = moe.moe_topk_softmax_backward(ids, w, dw, E).double()
    l64, c = inp.logits.double(), prod.sum(2)

    def f(l):
        return (torch.softmax(torch.gather(l, 1, ids.long()), 1) * c).sum(1)
    for j in range(k):
        d = torch.zeros_like(l64).scatter_(1, ids[:, j: j + 1].long(), 1e-5)
        num = (f(l64 + d) - f(l64 - d)) / 2e-5
        have = torch.gather(got, 1, ids[:, j: j + 1].long())[:, 0]
        # w is within 2e-6 of the softmax; the difference's own error is below that
        assert ((have - num).abs() <= 1e-5 * c.abs().sum(1) + 1e-9).all()
    # the combination of those rows is the layer's output when nothing is shared
    if layer.shared is None:
        back = moe.moe_combine(v["y"], w, v, out_dtype=BF)
        assert int((bits(back).view(torch.int16).int() - bits(out).view(torch.int16).int())
                   .abs().max()) <= 1


# --------------------------------------------------------------------------
# the norm at the ends of fp32's range
# --------------------------------------------------------------------------

def walk_err(M):
    """Roundings of a weight gradient's sum: xh; a group's rows one after the
    other (152 CTAs of 1 to 24 groups); the groups; five parts a thread; five
    levels of a butterfly."""
    rows = -(-M // 152)
    return max(rows + 1, -(-rows // 24) + 24) + 11


@pytest.mark.parametrize("scale,gscale", [(1e-20, 1.0), (3e-20, 1.0), (1e-30, 1e-3), (1e18, 1e-3),
                                          (1e30, 1e-3)])
@pytest.mark.parametrize("H", [77, 520, 4100])
@pytest.mark.parametrize("dt", [BF, FL], ids=_shape_id)
def test_norm_gradient_of_tiny_and_huge_rows(dt, H, scale, gscale):
    """Rows whose rstd squared, or its product with the mean, leaves fp32's
    range; elements that are zero among them."""
    M = 6
    g = gen(1600 + H)
    s, d = randn(g, M, H, dtype=dt, scale=scale), randn(g, M, H, dtype=dt, scale=gscale)
    s[1, 5] = 0
    w = (1 + randn(g, H, scale=0.2)).to(dt)
    rstd = (1 / torch.sqrt(s.double().square().mean(1))).float()
    r64 = rstd.double()[:, None]
    xh, gw = s.double() * r64, d.double() * w.double()
    mean = (gw * xh).mean(1, keepdim=True)
    mag = r64 * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    ref = r64 * (gw - xh * mean)
    for dsum in (None, (randn(g, M, H) * float(mag.mean())).to(dt)):
        extra = 0 if dsum is None else dsum.double()
        dx, dw = moe.moe_add_rmsnorm_backward(d, s, w, rstd, dsum=dsum)
        close(dx, ref + extra, mag + (0 if dsum is None else extra.abs()), 64 * U)
        v = d.double() * xh
        close(dw, v.sum(0), v.abs().sum(0), walk_err(M) * U)


@pytest.mark.parametrize("H", [64, 300, 1111, 4096, 12340, 16384])
@pytest.mark.parametrize("dt", [BF, FL], ids=_shape_id)
def test_norm_of_rows_whose_squares_leave_the_range(dt, H):
    """Squares that overflow or vanish in fp32, or whose sum does, with eps 0
    and others; ordinary rows between them keep their bits."""
    w = (1 + randn(gen(1700), H, scale=0.2)).to(dt)
    scales = [1.0, 1e-12, 1e-20, 1e-23, 1e-30, 2.0 ** 62, 1.5 * 2.0 ** 63, 1e25, 1e30, 3.0, 1e19]
    M = len(scales)
    x = randn(gen(1701 + H), M, H, dtype=dt)
    x = (x.double() * torch.tensor(scales, device="cuda", dtype=torch.float64)[:, None]).to(dt)
    x[5] = 2.0 ** 62   # mean 2^124, but the sum of 4096 squares is 2^136
    every = ("out", "sum", "rstd", "codes", "scale")
    for eps in (0.0, 1e-6, 1e-37):
        o = moe.moe_add_rmsnorm(x, w, eps, want=every)
        s, rstd, p, v = norm_ref(x, None, w, eps)
        assert ((o["rstd"].double() - rstd).abs() <= 32 * U * rstd).all()
        close(o["out"], v, v.abs(), 36 * U)
        check_codes(o["codes"], o["scale"], p, rstd, dt)
        for i in (0, 9):
            q = moe.moe_add_rmsnorm(x[i: i + 1], w, eps, want=every)
            for name in every:
                assert torch.equal(bits(q[name]), bits(o[name][i: i + 1])), (name, i)
    # no size at all, and rows that are not finite, with eps 0
    z = torch.zeros(3, H, dtype=dt, device="cuda")
    z[1, 3], z[2, 3] = float("inf"), float("nan")
    o = moe.moe_add_rmsnorm(z, w, 0.0, want=("rstd", "out"))
    assert float(o["rstd"][0]) == math.inf and float(o["rstd"][1]) == 0
    assert torch.isnan(o["rstd"][2]) and torch.isnan(o["out"][2]).all()


def test_codes_and_scales_reach_expert_order_in_one_stream():
    """The norm's E4M3 rows and scales dispatched by the call right behind it,
    eagerly, replayed, and over new inputs in the same buffers: the dispatch
    may be resident while the norm still writes them."""
    M, H, k, E = 700, 2048, 4, 16
    _, _, t = route(M, E, k, 16, 1800)
    perm, total = perm_of(t, M, k), int(t["num_tokens_post_padded"])
    x, r, w = norm_inputs(M, H, BF, BF, 1801)
    o = moe.alloc_add_rmsnorm_outputs(x, ("codes", "scale"))
    rows = torch.empty(t["max_total"], H, dtype=E4, device="cuda")
    scale = torch.empty(t["max_total"], H // 128, device="cuda")

    def both():
        moe.moe_add_rmsnorm(x, w, residual=r, out=o)
        moe.moe_dispatch(o["codes"], t, k, rows=rows, x_scale=o["scale"], rows_scale=scale)

    def check():
        torch.cuda.synchronize()
        s, rstd, p, _ = norm_ref(x, r, w, 1e-6)
        check_codes(o["codes"], o["scale"], p, rstd, BF)
        for got, src in ((rows, o["codes"]), (scale, o["scale"])):
            assert torch.equal(bits(got[perm]), bits(src[:, None].expand(M, k, -1)))
        pad, _ = padding(t, M * k)
        assert not bits(rows[pad]).any() and not scale[:total][pad[:total]].any()
    both()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
        both()
    for seed in range(4):
        a, b, _ = norm_inputs(M, H, BF, BF, 1810 + seed)
        x.copy_(a)
        r.copy_(b)
        graph.replay()
        check()


@pytest.mark.parametrize("shape,path", LAYERS + [(synth.decode_fp8(32), 0)],
                         ids=lambda v: getattr(v, "name", str(v)))
def test_the_layers_calls_right_behind_the_norm_that_writes_their_rows(shape, path):
    """The router, the layer and its expert half on rows that the norm in front
    writes into the same buffer each time, replayed without a gap: the bits of
    calls that wait for it."""
    inp, layer = make_layer(shape, path, router=True)
    M, H = shape.M, shape.H
    weight = torch.ones(H, dtype=BF, device="cuda")
    rows = [randn(gen(1900 + i), M, H, dtype=BF) for i in range(3)]
    ws, out = moe.alloc_workspace(layer, M), torch.empty(M, H, dtype=BF, device="cuda")
    moe.moe_decode_layer(layer, inp.x, out, ws)
    n = torch.empty(M, H, dtype=BF, device="cuda")
    lg = torch.empty(M, shape.E, device="cuda")

    def router(o):
        moe.moe_router_logits(n, layer.router_weight, logits=lg)
        o.copy_(lg[:, :1])

    calls = [lambda o: moe.moe_decode_experts(layer, n, o, ws),
             lambda o: moe.moe_decode_layer(layer, n, o, ws, router_logits=inp.logits), router]
    for call in calls:
        want = []
        for x in rows:
            moe.moe_add_rmsnorm(x, weight, out=dict(out=n))
            torch.cuda.synchronize()
            want.append(torch.empty_like(out))
            call(want[-1])
            torch.cuda.synchronize()
        got = [torch.empty_like(out) for _ in rows]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for x, o in zip(rows, got):
                moe.moe_add_rmsnorm(x, weight, out=dict(out=n))
                call(o)
        for _ in range(5):
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(bits(a), bits(b))


# --------------------------------------------------------------------------
# walks of several rows a group, batches beyond the plans' thresholds
# --------------------------------------------------------------------------

# (M, H, type, weights' type): more rows than the groups of a full grid take at
# once, and no whole number of turns.  Pieces a thread 1, 2, 4 and 8; rows of
# whole pieces, of halves, and of other widths.
WALKS = [(9001, 128, BF, BF), (4001, 2048, BF, BF), (1801, 3600, BF, FL), (2001, 12344, BF, BF),
         (9001, 132, HF, HF), (6001, 1028, BF, BF), (3001, 2884, BF, BF), (2001, 12340, HF, FL),
         (9001, 77, BF, BF), (3001, 513, BF, BF), (3001, 2885, HF, HF), (2001, 12345, BF, BF),
         (3001, 512, FL, FL), (3001, 1600, FL, FL), (2001, 4096, FL, FL), (1001, 16384, FL, FL),
         (3001, 514, FL, FL), (1001, 16382, FL, FL), (3001, 513, FL, FL), (2001, 2005, FL, FL),
         (2001, 5001, FL, FL), (1001, 16383, FL, FL)]
walks = pytest.mark.parametrize("M,H,dt,wt", WALKS, ids=_shape_id)


@walks
def test_norm_of_more_rows_than_a_grid_takes_at_once(M, H, dt, wt):
    """Against float64, and bit for bit the rows of small batches."""
    x, r, w = norm_inputs(M, H, dt, wt, 1300 + H)
    every = ("out", "sum", "rstd", "codes", "scale")
    o = moe.moe_add_rmsnorm(x, w, residual=r, want=every)
    s, rstd, p, v = norm_ref(x, r, w, 1e-6)
    assert torch.equal(o["sum"].double(), s)
    assert ((o["rstd"].double() - rstd).abs() <= 32 * U * rstd).all()
    close(o["out"], v, v.abs(), 36 * U)
    check_codes(o["codes"], o["scale"], p, rstd, dt if wt != FL else FL)
    for at in range(0, M, 150):
        b = slice(at, min(at + 150, M))
        q = moe.moe_add_rmsnorm(x[b], w, residual=r[b], want=every)
        for name in every:
            assert torch.equal(bits(q[name]), bits(o[name][b])), (name, at)


@walks
def test_norm_gradient_of_more_rows_than_a_grid_takes_at_once(M, H, dt, wt):
    x, s, w = norm_inputs(M, H, dt, wt, 1400 + H)
    dsum = randn(gen(1401), M, H, dtype=dt)
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    r64 = rstd.double()[:, None]
    d, xh = x.double(), s.double() * r64
    gw = d * w.double()
    mean = (gw * xh).mean(1, keepdim=True)
    dx, dw = moe.moe_add_rmsnorm_backward(x, s, w, rstd, dsum=dsum)
    mag = r64 * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True)) + dsum.double().abs()
    close(dx, r64 * (gw - xh * mean) + dsum.double(), mag, 64 * U)
    v = d * xh
    close(dw, v.sum(0), v.abs().sum(0), walk_err(M) * U)
    plain, _ = moe.moe_add_rmsnorm_backward(x, s, w, rstd, want_dweight=False)
    for at in range(0, M, 150):
        b = slice(at, min(at + 150, M))
        a, _ = moe.moe_add_rmsnorm_backward(x[b], s[b], w, rstd[b], dsum=dsum[b],
                                            want_dweight=False)
        assert torch.equal(bits(a), bits(dx[b])), at
        a, _ = moe.moe_add_rmsnorm_backward(x[b], s[b], w, rstd[b], want_dweight=False)
        assert torch.equal(bits(a), bits(plain[b])), at


@pytest.mark.parametrize("H", [1024, 1028, 1111, 2880])
@pytest.mark.parametrize("k", [1, 2, 4, 8])
@pytest.mark.parametrize("rt,ot", [(BF, BF), (FL, FL), (FL, BF)], ids=_shape_id)
def test_a_tokens_bits_in_batches_of_every_plan(H, k, rt, ot):
    """A batch whose plan takes several tokens a CTA, and its first tokens in
    batches of one, of seven and of a thousand."""
    M, E = 9000, 16
    _, w, t = route(M, E, k, 16, 1500 + k, 0.2)
    perm = perm_of(t, M, k)
    g = gen(1501)
    rows, dout = randn(g, t["max_total"], H, dtype=rt), randn(g, M, H, dtype=ot)
    x = randn(g, M, H, dtype=rt)
    out = moe.moe_combine(rows, w, t, out_dtype=ot)
    dr, dw = moe.moe_combine_backward(dout, rows, w, t)
    dx = moe.moe_dispatch_backward(rows, t, M, k)
    put = moe.moe_dispatch(x, t, k)
    for n in (1, 7, 1000):
        sub = dict(t, token_to_perm=t["token_to_perm"][: n * k].contiguous())
        real = perm[:n][perm[:n] >= 0]
        a, b = moe.moe_combine_backward(dout[:n], rows, w[:n], sub)
        for got, want in ((moe.moe_combine(rows, w[:n], sub, out_dtype=ot), out[:n]),
                          (a[real], dr[real]), (b, dw[:n]),
                          (moe.moe_dispatch_backward(rows, sub, n, k), dx[:n]),
                          (moe.moe_dispatch(x[:n], sub, k)[real], put[real])):
            assert torch.equal(bits(got), bits(want)), n
