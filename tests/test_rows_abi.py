"""Host side of the token dispatch and combination, the RMS norm and the
gradients, without a GPU: every refusal returns before anything is launched,
the binding refuses what the C entry points cannot read, and passes each
argument at the position the header declares it."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import expert_routing_alignment_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = ctypes.c_void_p(4096)         # 16-byte aligned; never read: each call is refused
ODD = ctypes.c_void_p(4096 + 1)
BF, HF, FL, E4 = moe.DTYPE_BF16, moe.DTYPE_F16, moe.DTYPE_F32, moe.DTYPE_E4M3
OK, EINVAL, EUNS = moe.MOE_OK, moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED


def header_params(fn: str) -> list:
    text = open(os.path.join(ROOT, "include", "moe_gb300.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    m = re.search(r"\b" + fn + r"\s*\(([^;]*?)\)\s*;", text, flags=re.S)
    assert m, fn
    return [re.findall(r"\w+", p)[-1] for p in m.group(1).split(",")]


def call(fn: str, base: dict, **changed):
    names = header_params(fn)
    args = {**base, **changed}
    assert set(args) == set(names), set(args) ^ set(names)
    return getattr(moe.load(), fn)(*[args[n] for n in names])


DISPATCH = dict(x=F, x_stride=256, x_scale=None, dtype=BF, M=4, top_k=2, hidden=256,
                token_to_perm=F, sorted_token_ids=F, num_tokens_post_padded=F, num_rows=64, rows=F,
                rows_scale=None, err_word=None, stream=None)
DISPATCH_BWD = dict(drows=F, dtype=BF, M=4, top_k=2, hidden=256, token_to_perm=F, num_rows=64,
                    dx=F, err_word=None, stream=None)
COMBINE = dict(rows=F, rows_dtype=BF, topk_w=F, token_to_perm=F, M=4, top_k=2, hidden=256,
               num_rows=64, out_dtype=BF, out=F, err_word=None, stream=None)
COMBINE_BWD = dict(dout=F, dout_stride=256, out_dtype=BF, rows=F, rows_dtype=BF, topk_w=F,
                   token_to_perm=F, sorted_token_ids=F, num_tokens_post_padded=F, M=4, top_k=2,
                   hidden=256, num_rows=64, drows=F, dtopk_w=F, err_word=None, stream=None)
TOPK_BWD = dict(topk_ids=F, topk_w=F, dtopk_w=F, M=4, num_experts=8, top_k=2, dlogits=F,
                err_word=None, stream=None)
F2 = ctypes.c_void_p(8192)
NORM = dict(x=F, x_stride=256, residual=F, residual_stride=256, weight=F, dtype=BF,
            weight_dtype=BF, M=4, hidden=256, eps=1e-6, sum_out=F, out=F2, out_codes=F,
            out_scale=F, rstd=F, stream=None)
NORM_BWD = dict(dout=F, dout_stride=256, sum=F, sum_stride=256, weight=F, rstd=F, dsum=F,
                dsum_stride=256, dtype=BF, weight_dtype=BF, M=4, hidden=256, dx=F, dweight=F,
                workspace=F, workspace_bytes=1 << 20, stream=None)

REFUSED = [
    ("moe_dispatch", DISPATCH, EINVAL, [
        dict(x=None), dict(token_to_perm=None), dict(sorted_token_ids=None), dict(rows=None),
        dict(num_tokens_post_padded=None), dict(M=-1), dict(top_k=0), dict(hidden=0),
        dict(num_rows=-1), dict(x_stride=-1), dict(dtype=0), dict(dtype=9), dict(x=ODD),
        dict(rows=ODD), dict(x_scale=F), dict(rows_scale=F), dict(dtype=E4),
        dict(dtype=E4, x_scale=F), dict(dtype=E4, rows_scale=F),
        dict(dtype=E4, x_scale=ODD, rows_scale=F)]),
    ("moe_dispatch", DISPATCH, EUNS, [dict(hidden=16385), dict(top_k=33), dict(M=1 << 20)]),
    ("moe_dispatch_backward", DISPATCH_BWD, EINVAL, [
        dict(drows=None), dict(dx=None), dict(token_to_perm=None), dict(dtype=E4), dict(dtype=0),
        dict(M=-1), dict(drows=ODD), dict(dx=ODD), dict(hidden=0), dict(top_k=0)]),
    ("moe_dispatch_backward", DISPATCH_BWD, EUNS, [
        dict(hidden=16385), dict(top_k=33), dict(M=1 << 20)]),
    ("moe_combine", COMBINE, EINVAL, [
        dict(rows=None), dict(out=None), dict(topk_w=None), dict(token_to_perm=None),
        dict(rows_dtype=E4), dict(out_dtype=0), dict(M=-1), dict(rows=ODD), dict(out=ODD)]),
    ("moe_combine", COMBINE, EUNS, [
        dict(hidden=16385), dict(out_dtype=HF), dict(out_dtype=FL), dict(rows_dtype=HF),
        dict(top_k=33),
        dict(M=1 << 20)]),
    ("moe_combine_backward", COMBINE_BWD, EINVAL, [
        dict(dout=None), dict(rows=None), dict(topk_w=None), dict(token_to_perm=None),
        dict(sorted_token_ids=None), dict(num_tokens_post_padded=None), dict(dout_stride=-1),
        dict(drows=None, dtopk_w=None), dict(dout=ODD), dict(rows=ODD), dict(drows=ODD),
        dict(rows_dtype=E4), dict(out_dtype=E4), dict(M=-1), dict(hidden=0)]),
    ("moe_combine_backward", COMBINE_BWD, EUNS, [
        dict(hidden=16385), dict(out_dtype=HF), dict(rows_dtype=HF), dict(top_k=33),
        dict(M=1 << 20)]),
    ("moe_topk_softmax_backward", TOPK_BWD, EINVAL, [
        dict(topk_ids=None), dict(topk_w=None), dict(dtopk_w=None), dict(dlogits=None), dict(M=-1),
        dict(top_k=0), dict(top_k=9), dict(num_experts=0), dict(dlogits=ODD), dict(topk_ids=ODD)]),
    ("moe_topk_softmax_backward", TOPK_BWD, EUNS, [
        dict(num_experts=1025), dict(num_experts=64, top_k=33)]),
    ("moe_add_rmsnorm", NORM, EINVAL, [
        dict(x=None), dict(weight=None), dict(M=-1), dict(hidden=0), dict(x_stride=-1),
        dict(residual_stride=-1), dict(dtype=E4), dict(weight_dtype=0), dict(eps=-1.0),
        dict(eps=float("nan")), dict(eps=float("inf")), dict(out_scale=None), dict(out_codes=None),
        dict(sum_out=None, out=None, out_codes=None, out_scale=None, rstd=None), dict(x=ODD),
        dict(residual=ODD), dict(weight=ODD), dict(rstd=ODD), dict(out_scale=ODD),
        dict(out=F),   # the same as sum_out
        dict(x_stride=512), dict(residual_stride=0)]),   # strided, and sum_out == x == residual
    ("moe_add_rmsnorm", NORM, EUNS, [
        dict(hidden=16385), dict(weight_dtype=HF), dict(dtype=FL, weight_dtype=BF)]),
    ("moe_add_rmsnorm_backward", NORM_BWD, EINVAL, [
        dict(dout=None), dict(sum=None), dict(weight=None), dict(rstd=None), dict(dx=None),
        dict(workspace=None), dict(workspace_bytes=16), dict(workspace=ODD), dict(M=-1),
        dict(dout_stride=-1), dict(sum_stride=-1), dict(dsum_stride=-1), dict(dout=ODD),
        dict(dweight=ODD), dict(dout_stride=512), dict(sum_stride=0), dict(dsum_stride=512),
        dict(dtype=E4), dict(hidden=0)]),
    ("moe_add_rmsnorm_backward", NORM_BWD, EUNS, [
        dict(hidden=16385), dict(weight_dtype=HF), dict(dtype=FL, weight_dtype=BF)]),
]


@pytest.mark.parametrize("fn,base,status,changes", REFUSED,
                         ids=[f"{r[0]}-{r[2]}" for r in REFUSED])
def test_refusals_come_before_any_launch(fn, base, status, changes):
    for ch in changes:
        assert call(fn, base, **ch) == status, ch


def test_no_rows_at_all_is_a_call_without_work():
    """M = 0 returns with nothing launched (there is no device here)."""
    none = dict(x=None, token_to_perm=None, num_rows=0, rows=None, sorted_token_ids=None,
                num_tokens_post_padded=None)
    assert call("moe_dispatch", DISPATCH, M=0, **none) == OK
    assert call("moe_dispatch_backward", DISPATCH_BWD, M=0, dx=None, token_to_perm=None) == OK
    assert call("moe_combine", COMBINE, M=0, out=None, topk_w=None) == OK
    assert call("moe_combine_backward", COMBINE_BWD, M=0, dout=None, drows=None) == OK
    assert call("moe_topk_softmax_backward", TOPK_BWD, M=0, dlogits=None) == OK
    assert call("moe_add_rmsnorm", NORM, M=0, x=None) == OK
    assert call("moe_add_rmsnorm_backward", NORM_BWD, M=0, dout=None, dweight=None) == OK
    # but its sizes are still looked at
    assert call("moe_combine", COMBINE, M=0, out_dtype=HF) == EUNS
    assert call("moe_add_rmsnorm", NORM, M=0, hidden=16385) == EUNS


def test_norm_gradient_workspace():
    f = moe.load().moe_add_rmsnorm_backward_workspace_bytes
    assert f(-1, 256) == f(4, 0) == f(4, 16385) == 0
    assert f(0, 256) > 0
    for H in (1, 255, 4096, 16384):
        sizes = [f(M, H) for M in (1, 2, 100, 5000, 100000, 2 ** 31 - 1)]
        assert sizes == sorted(sizes) and sizes[0] >= 4 * H and sizes[-1] < 1 << 26


class _FakeTensor:
    def __init__(self, addr):
        self.addr = addr

    def data_ptr(self):
        return self.addr


def _layer(router=4096, H=256):
    t = lambda: _FakeTensor(256)
    proj = (t(), t(), None)
    ex = moe.Experts(moe.FMT_FP8_B128, 8, H, 256, proj, proj, proj)
    return moe.LayerDesc(top_k=2, block_size=16, routed=ex,
                         router_weight=None if router is None else _FakeTensor(router))


def test_block_refuses_before_any_launch():
    lib = moe.load()
    layer = _layer()
    ws = ctypes.c_void_p(1 << 20)
    nb = moe.workspace_bytes(layer, 4)
    A, B, C, D = (ctypes.c_void_p(4096 * i) for i in (2, 3, 4, 5))

    def go(lay=layer, x=A, residual=B, w=F, eps=1e-6, M=4, sum_out=B, normed=C, out=D, ws=ws,
           nb=nb):
        return lib.moe_decode_block(ctypes.pointer(lay._struct), x, residual, w, eps, M, sum_out,
                                    normed, out, ws, nb, None, None)
    for kw in (dict(x=None), dict(w=None), dict(sum_out=None), dict(normed=None), dict(out=None),
               dict(ws=None), dict(nb=16), dict(ws=ctypes.c_void_p((1 << 20) + 64)),
               dict(eps=-1.0), dict(M=0), dict(normed=D), dict(sum_out=C), dict(out=B),
               dict(lay=_layer(router=None)), dict(lay=_layer(router=4096 + 8)),
               dict(normed=ctypes.c_void_p(4096 * 4 + 8))):
        assert go(**kw) == EINVAL, kw
    assert go(M=5000) == EUNS


# --------------------------------------------------------------------------
# the binding
# --------------------------------------------------------------------------

class _Recorder:
    def __init__(self):
        self.calls = {}

    def moe_add_rmsnorm_backward_workspace_bytes(self, M, H):
        return 4096

    def __getattr__(self, name):
        def record(*args):
            self.calls[name] = args
            return 0
        return record


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(moe, "_lib", r)
    monkeypatch.setattr(moe, "_on_device", lambda *a: None)   # CPU tensors stand in
    return r


def _val(a):
    return a.value if isinstance(a, ctypes.c_void_p) else a


def _holds(rec, fn, **want):
    names = header_params(fn)
    got = dict(zip(names, rec.calls[fn]))
    assert len(rec.calls[fn]) == len(names)
    for name, v in {**want, "stream": 7}.items():
        exp = v.data_ptr() if isinstance(v, torch.Tensor) else v
        assert _val(got[name]) == exp, name


M, H, E, K, R = 4, 200, 8, 2, 64


def _t():
    i32 = dict(dtype=torch.int32)
    return dict(token_to_perm=torch.zeros(M * K, **i32), sorted_token_ids=torch.zeros(R, **i32),
                num_tokens_post_padded=torch.zeros(1, **i32))


def test_binding_passes_arguments_in_the_headers_order(rec):
    t, err = _t(), torch.zeros(1, dtype=torch.int32)
    bf = torch.bfloat16
    wide = torch.zeros(M, 300, dtype=bf)
    x = wide[:, 8: 8 + H]
    rows = torch.zeros(R, H, dtype=bf)
    w = torch.zeros(M, K)
    moe.moe_dispatch(x, t, K, rows=rows, err_word=err, stream=7)
    _holds(rec, "moe_dispatch", x=x, x_stride=300, x_scale=None, dtype=BF, M=M, top_k=K, hidden=H,
           num_rows=R, rows=rows, rows_scale=None, err_word=err, **t)
    x8 = torch.zeros(M, H, dtype=torch.float8_e4m3fn)
    xs, r8, rs = torch.zeros(M, 2), torch.zeros(R, H, dtype=torch.float8_e4m3fn), torch.zeros(R, 2)
    moe.moe_dispatch(x8, t, K, rows=r8, x_scale=xs, rows_scale=rs, stream=7)
    _holds(rec, "moe_dispatch", x=x8, x_stride=H, x_scale=xs, dtype=E4, rows=r8, rows_scale=rs)
    dx = torch.zeros(M, H, dtype=bf)
    moe.moe_dispatch_backward(rows, t, M, K, dx=dx, err_word=err, stream=7)
    _holds(rec, "moe_dispatch_backward", drows=rows, dtype=BF, M=M, top_k=K, hidden=H, num_rows=R,
           token_to_perm=t["token_to_perm"], dx=dx, err_word=err)
    rows32 = torch.zeros(R, H)
    moe.moe_combine(rows32, w, t, out=dx, err_word=err, stream=7)
    _holds(rec, "moe_combine", rows=rows32, rows_dtype=FL, topk_w=w, M=M, top_k=K, hidden=H,
           token_to_perm=t["token_to_perm"], num_rows=R, out_dtype=BF, out=dx, err_word=err)
    dr, dw = torch.zeros(R, H), torch.zeros(M, K)
    moe.moe_combine_backward(x, rows32, w, t, drows=dr, dtopk_w=dw, err_word=err, stream=7)
    _holds(rec, "moe_combine_backward", dout=x, dout_stride=300, out_dtype=BF, rows=rows32,
           rows_dtype=FL, topk_w=w, M=M, top_k=K, hidden=H, num_rows=R, drows=dr, dtopk_w=dw,
           err_word=err, **t)
    moe.moe_combine_backward(x, rows32, w, t, dtopk_w=dw, want_drows=False, stream=7)
    _holds(rec, "moe_combine_backward", drows=None, dtopk_w=dw)
    moe.moe_combine_backward(x, None, w, t, drows=dr, want_dtopk_w=False, stream=7)
    _holds(rec, "moe_combine_backward", rows=None, rows_dtype=FL, drows=dr, dtopk_w=None)
    ids, dl = torch.zeros(M, K, dtype=torch.int32), torch.zeros(M, E)
    moe.moe_topk_softmax_backward(ids, w, dw, E, dlogits=dl, err_word=err, stream=7)
    _holds(rec, "moe_topk_softmax_backward", topk_ids=ids, topk_w=w, dtopk_w=dw, M=M,
           num_experts=E, top_k=K, dlogits=dl, err_word=err)
    wt = torch.zeros(H, dtype=bf)
    o = dict(out=torch.zeros(M, H, dtype=bf), sum=torch.zeros(M, H, dtype=bf),
             codes=torch.zeros(M, H, dtype=torch.uint8), scale=torch.zeros(M, 2),
             rstd=torch.zeros(M))
    assert moe.moe_add_rmsnorm(x, wt, 0.5, residual=dx, out=o, stream=7) is o
    _holds(rec, "moe_add_rmsnorm", x=x, x_stride=300, residual=dx, residual_stride=H, weight=wt,
           dtype=BF, weight_dtype=BF, M=M, hidden=H, eps=0.5, sum_out=o["sum"], out=o["out"],
           out_codes=o["codes"], out_scale=o["scale"], rstd=o["rstd"])
    dwt, ws = torch.zeros(H), torch.zeros(5000, dtype=torch.uint8)
    moe.moe_add_rmsnorm_backward(x, o["sum"], wt, o["rstd"], dsum=o["out"], dx=dx, dweight=dwt,
                                 workspace=ws, stream=7)
    _holds(rec, "moe_add_rmsnorm_backward", dout=x, dout_stride=300, sum=o["sum"], sum_stride=H,
           weight=wt, rstd=o["rstd"], dsum=o["out"], dsum_stride=H, dtype=BF, weight_dtype=BF,
           M=M, hidden=H, dx=dx, dweight=dwt, workspace=ws, workspace_bytes=5000)
    moe.moe_add_rmsnorm_backward(x, o["sum"], wt, o["rstd"], dx=dx, want_dweight=False, stream=7)
    _holds(rec, "moe_add_rmsnorm_backward", dsum=None, dweight=None, workspace=None,
           workspace_bytes=0)
    layer = _layer(H=256)
    a, b, c, d = (torch.zeros(M, 256, dtype=bf) for _ in range(4))
    nw = torch.zeros(256, dtype=bf)
    moe.moe_decode_block(layer, a, b, nw, d, ws, eps=0.25, sum_out=b, normed=c, err_word=err,
                         stream=7)
    _holds(rec, "moe_decode_block", x=a, residual=b, norm_weight=nw, eps=0.25, M=M, sum_out=b,
           normed=c, out=d, workspace=ws, workspace_bytes=5000, err_word=err)


def test_one_row_has_no_stride(rec):
    """A single row's stride says nothing: any view of one row is dense."""
    x = torch.zeros(3, 2 * H, dtype=torch.bfloat16)[:1, :H]
    t = _t()
    moe.moe_dispatch(x, t, K, rows=torch.zeros(R, H, dtype=torch.bfloat16), stream=7)
    _holds(rec, "moe_dispatch", x=x, x_stride=H, M=1)


def test_binding_refuses_what_the_entry_points_cannot_read(rec):
    bf = torch.bfloat16
    t, w = _t(), torch.zeros(M, K)
    x, rows = torch.zeros(M, H, dtype=bf), torch.zeros(R, H, dtype=bf)
    x8 = torch.zeros(M, H, dtype=torch.float8_e4m3fn)
    wt, rstd, ids = torch.zeros(H, dtype=bf), torch.zeros(M), torch.zeros(M, K, dtype=torch.int32)
    bad = [
        lambda: moe.moe_dispatch(torch.zeros(M, 2 * H, dtype=bf)[:, ::2], t, K),
        lambda: moe.moe_dispatch(torch.zeros(M, 1, dtype=bf).expand(M, H), t, K),
        lambda: moe.moe_dispatch(x.double(), t, K),
        lambda: moe.moe_dispatch(x, t, K, rows=rows[:5]),
        lambda: moe.moe_dispatch(x, t, K, rows=rows.float()),
        lambda: moe.moe_dispatch(x, t, K, x_scale=torch.zeros(M, 2)),
        lambda: moe.moe_dispatch(x8, t, K),
        lambda: moe.moe_dispatch(x8, t, K, x_scale=torch.zeros(M, 1)),
        lambda: moe.moe_dispatch(x, t, K + 1),                       # tables too short
        lambda: moe.moe_dispatch(x, {**t, "token_to_perm": torch.zeros(M * K)}, K),
        lambda: moe.moe_dispatch(x, t, K, err_word=torch.zeros(1)),
        lambda: moe.moe_dispatch_backward(rows[:, ::2], t, M, K),
        lambda: moe.moe_dispatch_backward(rows[:7], t, M, K),
        lambda: moe.moe_dispatch_backward(rows, t, M, K, dx=x.float()),
        lambda: moe.moe_combine(rows, w.double(), t),
        lambda: moe.moe_combine(rows, w, t, out=x[:2]),
        lambda: moe.moe_combine(rows, w, t, out=x, out_dtype=torch.float32),
        lambda: moe.moe_combine(rows.to(torch.float8_e4m3fn), w, t),
        lambda: moe.moe_combine_backward(x, None, w, t),
        lambda: moe.moe_combine_backward(x, rows, w, t, want_drows=False, want_dtopk_w=False),
        lambda: moe.moe_combine_backward(x, rows, w, t, drows=rows.float()),
        lambda: moe.moe_combine_backward(x, rows, w, t, dtopk_w=torch.zeros(M, K + 1)),
        lambda: moe.moe_combine_backward(x[:2], rows, w, t),
        lambda: moe.moe_topk_softmax_backward(ids.long(), w, w, E),
        lambda: moe.moe_topk_softmax_backward(ids, w, w[:2], E),
        lambda: moe.moe_topk_softmax_backward(ids, w, w, E, dlogits=torch.zeros(M, E + 1)),
        lambda: moe.moe_add_rmsnorm(x, wt[:-1]),
        lambda: moe.moe_add_rmsnorm(x, wt, residual=x.float()),
        lambda: moe.moe_add_rmsnorm(x, wt, residual=x[:2]),
        lambda: moe.moe_add_rmsnorm(x, wt, want=("nothing",)),
        lambda: moe.moe_add_rmsnorm(x, wt, out=dict(out=x.float())),
        lambda: moe.moe_add_rmsnorm(x, wt, out=dict(other=x)),
        lambda: moe.moe_add_rmsnorm(x, wt, out=dict(codes=x8, scale=torch.zeros(M, 1))),
        lambda: moe.moe_add_rmsnorm_backward(x, x.float(), wt, rstd),
        lambda: moe.moe_add_rmsnorm_backward(x, x, wt, rstd[:2]),
        lambda: moe.moe_add_rmsnorm_backward(x, x, wt, rstd, dweight=wt),
        lambda: moe.moe_add_rmsnorm_backward(x, x, wt, rstd, dsum=x[:2]),
        lambda: moe.moe_decode_block(_layer(), x, x, wt, x, torch.zeros(8, dtype=torch.uint8)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    assert not rec.calls


def test_binding_refuses_tensors_off_the_device():
    """CPU tensors are no device buffers: refused before any call."""
    x, t = torch.zeros(M, H, dtype=torch.bfloat16), _t()
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_dispatch(x, t, K)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_add_rmsnorm(x, torch.zeros(H, dtype=torch.bfloat16))


# every table, weight and error word at an odd address and at an even one that
# is not theirs; and the weights' absence where there is no row at all
HALF = ctypes.c_void_p(4096 + 2)
MISPLACED = [
    ("moe_dispatch", DISPATCH, ("token_to_perm", "sorted_token_ids", "num_tokens_post_padded",
                                "err_word")),
    ("moe_dispatch_backward", DISPATCH_BWD, ("token_to_perm", "err_word")),
    ("moe_combine", COMBINE, ("topk_w", "token_to_perm", "err_word")),
    ("moe_combine_backward", COMBINE_BWD, ("topk_w", "token_to_perm", "sorted_token_ids",
                                           "num_tokens_post_padded", "dtopk_w", "err_word")),
    ("moe_topk_softmax_backward", TOPK_BWD, ("topk_ids", "topk_w", "dtopk_w", "dlogits",
                                             "err_word")),
    ("moe_add_rmsnorm", NORM, ("out_scale", "rstd")),
    ("moe_add_rmsnorm_backward", NORM_BWD, ("rstd", "dweight")),
]


@pytest.mark.parametrize("fn,base,names", MISPLACED, ids=[m[0] for m in MISPLACED])
def test_misplaced_tables_and_weights_are_refused(fn, base, names):
    for name in names:
        for at in (ODD, HALF):
            assert call(fn, base, **{name: at}) == EINVAL, (name, at)


def test_combine_gradient_wants_its_weights_whatever_the_rows():
    """Every slot's weight is read for drows, with num_rows = 0 too."""
    for n in (0, 64):
        assert call("moe_combine_backward", COMBINE_BWD, topk_w=None, num_rows=n) == EINVAL
        assert call("moe_combine_backward", COMBINE_BWD, topk_w=None, dtopk_w=None,
                    num_rows=n) == EINVAL


NO_DEVICE = """
import ctypes
import expert_routing_alignment_gb300 as moe
from tests import test_rows_abi as t
for fn, base in (("moe_dispatch", t.DISPATCH), ("moe_dispatch_backward", t.DISPATCH_BWD),
                 ("moe_combine", t.COMBINE), ("moe_combine_backward", t.COMBINE_BWD),
                 ("moe_topk_softmax_backward", t.TOPK_BWD), ("moe_add_rmsnorm", t.NORM),
                 ("moe_add_rmsnorm_backward", t.NORM_BWD)):
    assert t.call(fn, base) == moe.MOE_ECUDA, fn
    assert moe.load().moe_last_cuda_error() != 0, fn
layer = t._layer()
a, b, c, d = (ctypes.c_void_p(4096 * i) for i in (2, 3, 4, 5))
assert moe.load().moe_decode_block(
    ctypes.pointer(layer._struct), a, b, t.F, 1e-6, 4, b, c, d, ctypes.c_void_p(1 << 20),
    moe.workspace_bytes(layer, 4), None, None) == moe.MOE_ECUDA
print("refused")
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="its pointers are no device buffers")
def test_without_a_device_every_call_returns_its_error():
    """In a process of its own, with every device hidden: a call that fails to
    find one must not end the process."""
    p = subprocess.run([sys.executable, "-c", NO_DEVICE], capture_output=True, text=True, cwd=ROOT,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, timeout=300)
    assert p.returncode == 0 and "refused" in p.stdout, (p.returncode, p.stderr[-2000:])


NO_CUDA = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):   # as in a build without CUDA
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import expert_routing_alignment_gb300 as moe
assert moe.moe_align_sizes(16, 8, 16)[0] > 0
assert moe.add_rmsnorm_backward_workspace_bytes(4, 256) > 0
x = torch.zeros(2, 64, dtype=torch.bfloat16)
try:
    moe.moe_add_rmsnorm(x, x[0])
except ValueError as e:
    assert "CUDA" in str(e)
    print("refused")
"""


def test_import_and_host_calls_need_no_cuda_build_of_torch():
    p = subprocess.run([sys.executable, "-c", NO_CUDA], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert p.returncode == 0 and "refused" in p.stdout, (p.returncode, p.stderr[-2000:])
