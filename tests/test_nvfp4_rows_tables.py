"""The products of four-bit rows refuse a token count or a top_k that is not
the tables': the kernels know a padding position by its slot alone, which is
the number of slots the tables were made for."""
from __future__ import annotations

import pytest
import torch

import expert_routing_alignment_gb300 as moe
from tests.test_nvfp4_rows_abi import packed, rec, tables  # noqa: F401 (rec is a fixture)

W, ROWS, SORTED = packed(8, 40, cols=96), packed(4, cols=96), packed(64, cols=96)


def calls(rows, t, k, M=None):
    return (lambda: moe.moe_grouped_product_nvfp4(W, rows, t, k, M=M, out=torch.zeros(64, 40),
                                                  stream=7),
            lambda: moe.moe_grouped_gate_up_nvfp4(W, W, rows, t, k, M=M, out=torch.zeros(64, 40),
                                                  stream=7))


@pytest.mark.parametrize("rows,k,M", [
    (ROWS, 1, None), (ROWS, 3, None),                    # a wrong top_k
    (packed(5, cols=96), 2, None), (packed(3, cols=96), 2, None),   # other rows than were aligned
    (SORTED, 2, 5), (SORTED, 2, 3), (SORTED, 2, 0)])     # a wrong M in expert order
def test_slots_other_than_the_tables_are_refused(rec, rows, k, M):  # noqa: F811
    for t in (tables(8, 8, 64), {**tables(8, 50, 64), "num_slots": 8}):
        for f in calls(rows, t, k, M):
            with pytest.raises(ValueError, match="slots"):
                f()
    assert not rec.calls


def test_the_tables_own_slots_are_taken(rec):  # noqa: F811
    """By moe_align's own count where the buffers are larger than the batch; tables
    that say nothing of it as before."""
    plain = tables(8, 8, 64)
    alone = {n: plain[n] for n in ("sorted_token_ids", "expert_offsets")}
    for t in (plain, {**tables(8, 50, 64), "num_slots": 8}, alone):
        for f in (*calls(ROWS, t, 2), *calls(SORTED, t, 2, 4)):
            rec.calls.clear()
            f()
            assert len(rec.calls) == 1


def test_align_says_how_many_slots_it_was_given(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(moe, "_lib", Lib())
    ids = torch.zeros(3, 2, dtype=torch.int32)
    big = dict(sorted_token_ids=torch.zeros(64, dtype=torch.int32),
               token_to_perm=torch.zeros(50, dtype=torch.int32), max_total=64,
               **{n: torch.zeros(9, dtype=torch.int32) for n in (
                   "sorted_expert_ids", "expert_offsets", "active_experts", "active_count",
                   "num_tokens_post_padded")})
    assert moe.moe_align(ids, 8, 4, out=big, stream=0) is big and big["num_slots"] == 6
    moe.moe_align(ids[:1], 8, 4, out=big, stream=0)
    assert big["num_slots"] == 2


def test_rows_in_expert_order_are_known_by_the_same_count(rec):  # noqa: F811
    t = {**tables(8, 50, 64), "num_slots": 8}
    x = torch.zeros(64, 96, dtype=torch.bfloat16)
    moe.moe_quantize_nvfp4(x, tables=t, out=dict(codes=torch.zeros(64, 48, dtype=torch.uint8)),
                           stream=7)
    assert rec.calls["moe_quantize_nvfp4"][8] == 8
