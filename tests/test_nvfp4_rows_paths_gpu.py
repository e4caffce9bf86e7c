"""Four-bit products on the ways through the kernel that the other sizes leave
out: expert-order rows whose scales come by TMA over several stages and tiles,
gate and up of such rows, tables in larger buffers; and gradients against
float64 from the definition of the rounding.  Tolerances as in test_nvfp4_rows_gpu,
whose helpers these are."""
from __future__ import annotations

import pytest
import torch

import expert_routing_alignment_gb300 as moe
from tests.test_nvfp4_rows_gpu import (BF, FL, HF, U, align, check_product, gate_up_reference,
                                       gen, half, randn, ref_quantize, rows_of, run_product, sums,
                                       weights)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# rows in expert order, scales by TMA
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("C", [768, 1024, 1536])
def test_expert_order_over_several_stages(C, dtype):
    run_product([1, 31, 0, 33, 129, 300], 200, C, BS=1, by_token=False, seed=C, dtype=dtype)
    run_product([1, 31, 0, 33, 129, 300], 264, C, BS=16, by_token=False, seed=C + 1, dtype=dtype)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 128, 129, 300])
def test_expert_order_of_one_run(n):
    run_product([n], 256, 768, BS=1, by_token=False, seed=n)


@pytest.mark.parametrize("C", [256, 1024, 1536])
def test_expert_order_over_more_tiles_than_sms(C):
    run_product([700, 10, 300, 0, 129, 128, 1, 33], 4096, C, BS=16, by_token=False, seed=C)


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("counts,R,C", [
    ([1, 31, 33, 129], 200, 256), ([300, 0, 5], 128, 1024), ([2, 140], 40, 768),
    ([129, 20, 0, 300, 33, 1], 2560, 512)])
def test_gate_up_in_expert_order(counts, R, C, dtype):
    t, n = align(counts, 16)
    g = gen(R + C)
    x = moe.moe_quantize_nvfp4(randn(g, t["max_total"], C, dtype=BF))
    gate, up = weights(g, len(counts), R, C), weights(g, len(counts), R, C)
    fill = torch.full((t["max_total"], R), 7.0, dtype=dtype, device="cuda")
    out = moe.moe_grouped_gate_up_nvfp4(gate, up, x, t, 1, M=n, out=fill.clone())
    p, at, e = rows_of(t, 1, False)
    h, err = gate_up_reference(x, gate, up, at, e, C)
    check_product(out[p], h, err, C, norm=False)
    rest = torch.ones(t["max_total"], dtype=torch.bool, device="cuda")
    rest[p] = False
    assert torch.equal(out[rest], fill[rest])


@pytest.mark.parametrize("C", [512, 768, 320, 288])
@pytest.mark.parametrize("both", [False, True])
def test_a_rows_bits_are_its_own_in_either_order(C, both):
    """By token or in expert order, among many rows or few, with any block size,
    a row has the same bits."""
    g = gen(C)
    E, R, n = 3, 384, 400
    sets = [weights(g, E, R, C) for _ in range(1 + both)]
    call = moe.moe_grouped_gate_up_nvfp4 if both else moe.moe_grouped_product_nvfp4
    x = moe.moe_quantize_nvfp4(randn(g, n, C))
    ids = torch.randint(0, E, (n, 1), generator=g, device="cuda").int()

    def rows(sel, BS, by_token):
        t = moe.moe_align(ids[sel].contiguous(), E, BS)
        perm = t["token_to_perm"].long()
        if by_token:
            q = {name: v[sel].contiguous() for name, v in x.items()}
        else:
            q = {name: torch.zeros((t["max_total"], *v.shape[1:]), dtype=v.dtype, device="cuda")
                 for name, v in x.items()}
            for name, v in x.items():
                q[name][perm] = v[sel]
        return call(*sets, q, t, 1, M=None if by_token else len(sel), out_dtype=FL)[perm]

    whole = rows(torch.arange(n, device="cuda"), 16, True)
    for sel, BS in ((torch.arange(1, device="cuda"), 1), (torch.arange(200, 231, device="cuda"), 64),
                    (torch.arange(n - 1, -1, -3, device="cuda"), 16),
                    (torch.arange(n, device="cuda"), 1)):
        for by_token in (True, False):
            assert torch.equal(rows(sel, BS, by_token), whole[sel]), (len(sel), by_token)


# --------------------------------------------------------------------------
# buffers of a larger batch
# --------------------------------------------------------------------------

def test_tables_in_buffers_of_a_larger_batch():
    """moe_align into buffers that an earlier, larger batch used: the smaller one's
    rows are its own, and the padding of its runs stays as it was."""
    g = gen(5)
    E, C, R, BS, k = 4, 256, 96, 16, 2
    big = moe.alloc_align_outputs(200 * k, E, BS)
    ids = torch.randint(0, E, (200, k), generator=g, device="cuda").int()
    moe.moe_align(ids, E, BS, out=big)
    few = ids[:21].contiguous()
    t, fresh = moe.moe_align(few, E, BS, out=big), moe.moe_align(few, E, BS)
    n, total = few.numel(), int(fresh["num_tokens_post_padded"])
    assert t["max_total"] > fresh["max_total"] and t["num_slots"] == n
    real = fresh["sorted_token_ids"][:total] < n
    assert torch.equal(t["sorted_token_ids"][:total], fresh["sorted_token_ids"][:total])
    assert 0 < int(real.sum()) < total
    h = randn(g, t["max_total"], C, dtype=BF)
    q = moe.alloc_quantize_nvfp4_outputs(h)
    for v in q.values():
        v.view(torch.uint8).fill_(0x5A)
    before = {name: v.clone() for name, v in q.items()}
    moe.moe_quantize_nvfp4(h, tables=t, out=q)
    whole = moe.moe_quantize_nvfp4(h)
    for name, v in q.items():
        assert torch.equal(v[:total][real], whole[name][:total][real]), name
        assert torch.equal(v[:total][~real].view(torch.uint8),
                           before[name][:total][~real].view(torch.uint8)), name
    w = weights(g, E, R, C)
    fill = torch.full((t["max_total"], R), 7.0, dtype=BF, device="cuda")
    y = moe.moe_grouped_product_nvfp4(w, q, t, k, M=21, out=fill.clone())
    part = {name: v[: fresh["max_total"]].contiguous() for name, v in q.items()}
    want = moe.moe_grouped_product_nvfp4(w, part, fresh, k, M=21)
    assert torch.equal(y[:total][real], want[:total][real])
    assert torch.equal(y[:total][~real], fill[:total][~real]) and torch.equal(y[total:],
                                                                             fill[total:])
    with pytest.raises(ValueError):
        moe.moe_grouped_product_nvfp4(w, q, t, k, M=200)


# --------------------------------------------------------------------------
# gradients
# --------------------------------------------------------------------------

def test_gradients_straight_through_the_rounding():
    """Loss L = sum_p dy[p] . W_e v[p], v the four-bit values of x and dy constant: dL/dx
    straight through the rounding is the product of the quantised dy with the
    transposed set, dL/dW the outer products of dy and v.  Both against float64 from
    the definition of the rounding, not from what the calls returned, and against
    differences of the loss, which is linear in each."""
    g = gen(77)
    E, R, C = 3, 96, 256
    t, n = align([20, 0, 50], 16)
    W, x = randn(g, E, R, C, dtype=BF, scale=0.05), randn(g, t["max_total"], C, dtype=BF)
    dy = randn(g, t["max_total"], R, dtype=BF)
    p, _, e = rows_of(t, 1, False)
    wt = moe.moe_quantize_nvfp4(W.transpose(1, 2).contiguous())
    dx = moe.moe_grouped_product_nvfp4(wt, moe.moe_quantize_nvfp4(dy, tables=t), t, 1, M=n,
                                       out_dtype=FL)[p].double()
    v = moe.moe_quantize_nvfp4(x, want=("values",), tables=t)["values"][p]

    def wide(z):   # the definition's values in float64, unrounded
        code, s, glob, _ = ref_quantize(z)
        return code * torch.repeat_interleave(s, 16, -1) * glob.view(-1, *[1] * (z.dim() - 1))

    WT, DY, V = wide(W.transpose(1, 2).contiguous()), wide(dy[p]), wide(x[p])

    def loss_x(rows):
        return (torch.einsum("pc,pcr->pr", rows, WT[e]) * DY).sum()

    leaf = V.clone().requires_grad_()
    loss_x(leaf).backward()
    mag = torch.einsum("pr,pcr->pc", DY.abs(), WT[e].abs())
    tol = (1 + half(FL)) * (R * 2.0 ** -23 + 2 * U) * mag + half(FL) * leaf.grad.abs()
    assert bool((leaf.grad.abs() > 0).any())
    assert ((dx - leaf.grad).abs() <= tol).all()
    dW = torch.stack([dy[p][e == i].double().T @ v[e == i].double() for i in range(E)])
    ref = torch.stack([dy[p][e == i].double().T @ V[e == i] for i in range(E)])
    # a value has the roundings of its step, of the product and of its type
    mag = torch.stack([dy[p][e == i].double().abs().T @ V[e == i].abs() for i in range(E)])
    assert ((dW - ref).abs() <= (half(BF) + 4 * U) * mag).all()
    for i, c in ((0, 0), (7, 100), (len(p) - 1, C - 1)):
        for step in (2.0 ** -10, 1.0):
            d = torch.zeros_like(V)
            d[i, c] = step
            diff = float((loss_x(V + d) - loss_x(V - d)) / (2 * step))
            # two sums of float64: their terms' magnitudes times 2^-53 for each
            slack = 2 * V.numel() * 2.0 ** -53 * float(
                (torch.einsum("pc,pcr->pr", (V.abs() + d), WT[e].abs()) * DY.abs()).sum()) / step
            assert abs(float(dx[i, c]) - diff) <= float(tol[i, c]) + slack
