"""Host side of the four-bit rows and their products, without a GPU: refusals
come before any launch, and the binding passes each argument at the position
the header declares it and refuses what the entry points cannot read."""
from __future__ import annotations

import ctypes

import pytest
import torch

import expert_routing_alignment_gb300 as moe
from tests.test_rows_abi import BF, E4, EINVAL, EUNS, F, FL, HF, ODD, OK, _val, call, header_params

HALF = ctypes.c_void_p(4096 + 8)   # 8-byte aligned
QUANT = dict(x=F, x_stride=256, dtype=BF, groups=4, rows=1, cols=256, given_scale=None,
             sorted_token_ids=None, num_slots=0, codes=F, scale=F, global_scale=F, values=None,
             workspace=None, workspace_bytes=0, stream=None)
GROUPS = dict(QUANT, rows=8, workspace=F, workspace_bytes=1 << 20)
DEQUANT = dict(codes=F, scale=F, global_scale=F, groups=4, rows=8, cols=256, dtype=BF, out=F,
               stream=None)
PRODUCT = dict(weight=(4096, 4096, 4096), num_experts=8, out_dim=128, in_dim=256, codes=F, scale=F,
               global_scale=F, by_token=1, M=4, top_k=2, expert_offsets=F, sorted_token_ids=F,
               num_rows=64, out_dtype=BF, out=F, err_word=None, stream=None)


def proj(p):
    return None if p is None else ctypes.byref(moe._Proj(*p))


def product(fn="moe_grouped_product_nvfp4", **changed):
    args = {**PRODUCT, **changed}
    if fn == "moe_grouped_gate_up_nvfp4":
        up = args.pop("up", args["weight"])
        args["gate"], args["up"] = proj(args.pop("weight")), proj(up)
    else:
        args["weight"] = proj(args["weight"])
    names = header_params(fn)
    assert set(args) == set(names)
    return getattr(moe.load(), fn)(*[args[n] for n in names])


@pytest.mark.parametrize("base,status,changes", [
    (QUANT, EINVAL, [
        dict(x=None), dict(codes=None, scale=None, global_scale=None), dict(groups=-1),
        dict(rows=0), dict(cols=0), dict(x_stride=-1), dict(num_slots=-1), dict(dtype=E4),
        dict(dtype=0), dict(x=ODD), dict(codes=ODD), dict(codes=ctypes.c_void_p(4100)),
        dict(global_scale=ODD), dict(given_scale=ODD), dict(values=ODD),
        dict(sorted_token_ids=ODD), dict(values=F, x_stride=512)]),
    (QUANT, EUNS, [dict(cols=8), dict(cols=250), dict(cols=16400), dict(groups=1 << 30, rows=4),
                   dict(rows=2, sorted_token_ids=F)]),
    (GROUPS, EINVAL, [dict(workspace=None), dict(workspace_bytes=16), dict(workspace=HALF)]),
], ids=["rows-einval", "rows-unsupported", "groups-einval"])
def test_quantize_refuses_before_any_launch(base, status, changes):
    for ch in changes:
        assert call("moe_quantize_nvfp4", base, **ch) == status, ch


def test_dequantize_refuses_before_any_launch():
    for ch in (dict(codes=None), dict(scale=None), dict(global_scale=None), dict(out=None),
               dict(codes=ODD), dict(global_scale=ODD), dict(out=ODD), dict(dtype=E4),
               dict(groups=-1), dict(rows=0), dict(cols=0)):
        assert call("moe_dequantize_nvfp4", DEQUANT, **ch) == EINVAL, ch
    for ch in (dict(cols=24), dict(cols=16400), dict(groups=1 << 30)):
        assert call("moe_dequantize_nvfp4", DEQUANT, **ch) == EUNS, ch


@pytest.mark.parametrize("fn", ["moe_grouped_product_nvfp4", "moe_grouped_gate_up_nvfp4"])
def test_products_refuse_before_any_launch(fn):
    for ch in (dict(weight=None), dict(weight=(0, 4096, 4096)), dict(weight=(4096, 0, 4096)),
               dict(weight=(4096, 4096, 0)), dict(weight=(4104, 4096, 4096)),
               dict(weight=(4096, 4104, 4096)), dict(weight=(4096, 4096, 4097)), dict(codes=None),
               dict(scale=None), dict(global_scale=None), dict(expert_offsets=None),
               dict(sorted_token_ids=None), dict(out=None), dict(codes=HALF), dict(scale=HALF),
               dict(global_scale=ODD), dict(expert_offsets=ODD), dict(sorted_token_ids=ODD),
               dict(out=ODD), dict(err_word=ODD), dict(num_experts=0), dict(out_dim=0),
               dict(in_dim=0), dict(M=-1), dict(top_k=0), dict(num_rows=-1), dict(out_dtype=E4),
               dict(out_dtype=0)):
        assert product(fn, **ch) == EINVAL, ch
    for ch in (dict(num_experts=1025), dict(in_dim=48), dict(in_dim=16416), dict(out_dim=65537),
               dict(top_k=33), dict(M=1 << 20), dict(num_experts=1024, out_dim=65536, in_dim=32,
                                                     M=1 << 20, top_k=1, num_rows=-1)):
        assert product(fn, **ch) == (EINVAL if "num_rows" in ch else EUNS), ch


def test_gate_up_needs_both():
    assert product("moe_grouped_gate_up_nvfp4", up=None) == EINVAL
    assert product("moe_grouped_gate_up_nvfp4", up=(4096, 4104, 4096)) == EINVAL


def test_nothing_to_do_is_a_call_without_work():
    """Returns with nothing launched (there is no device here)."""
    assert call("moe_quantize_nvfp4", QUANT, groups=0, x=None) == OK
    assert call("moe_quantize_nvfp4", QUANT, groups=0, cols=24) == EUNS
    assert call("moe_dequantize_nvfp4", DEQUANT, groups=0, codes=None) == OK
    for fn in ("moe_grouped_product_nvfp4", "moe_grouped_gate_up_nvfp4"):
        assert product(fn, M=0, codes=None, out=None) == OK
        assert product(fn, num_rows=0, out=None) == OK
        assert product(fn, M=0, in_dim=48) == EUNS


def test_quantize_workspace():
    f = moe.load().moe_quantize_nvfp4_workspace_bytes
    assert f(-1, 4, 64) == f(4, 0, 64) == f(4, 4, 24) == f(4, 4, 16400) == 0
    assert 0 < f(0, 1, 16) <= f(1 << 20, 1, 16384) <= f(1, 2, 16) < f(1024, 1536, 2048) < 1 << 20


class _Recorder:
    def __init__(self):
        self.calls = {}

    def moe_quantize_nvfp4_workspace_bytes(self, groups, rows, cols):
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


def _holds(rec, fn, **want):
    names = header_params(fn)
    got = dict(zip(names, rec.calls[fn]))
    assert len(rec.calls[fn]) == len(names)
    for name, v in {**want, "stream": 7}.items():
        exp = v.data_ptr() if isinstance(v, torch.Tensor) else v
        assert _val(got[name]) == exp, name
    return got


U8 = torch.uint8


def packed(*lead, cols):
    return dict(codes=torch.zeros(*lead, cols // 2, dtype=U8),
                scale=torch.zeros(*lead, cols // 16, dtype=U8), global_scale=torch.zeros(lead[0]))


def tables(E, n, rows):
    i32 = dict(dtype=torch.int32)
    return dict(sorted_token_ids=torch.zeros(rows, **i32), token_to_perm=torch.zeros(n, **i32),
                expert_offsets=torch.zeros(E + 1, **i32))


def test_binding_passes_arguments_in_the_headers_order(rec):
    wide = torch.zeros(4, 300, dtype=torch.bfloat16)
    x = wide[:, 8: 8 + 160]
    q = dict(packed(4, cols=160), values=torch.zeros(4, 160, dtype=torch.bfloat16))
    given, t = torch.ones(4), tables(8, 6, 4)
    assert moe.moe_quantize_nvfp4(x, global_scale=given, tables=t, out=q, stream=7) is q
    _holds(rec, "moe_quantize_nvfp4", x=x, x_stride=300, dtype=BF, groups=4, rows=1, cols=160,
           given_scale=given, sorted_token_ids=t["sorted_token_ids"], num_slots=6,
           codes=q["codes"], scale=q["scale"], global_scale=q["global_scale"], values=q["values"],
           workspace=None, workspace_bytes=0)
    m = torch.zeros(3, 5, 64)[:, :, :48]
    q = dict(scale=torch.zeros(3, 5, 3, dtype=torch.float8_e4m3fn))
    ws = torch.zeros(5000, dtype=U8)
    moe.moe_quantize_nvfp4(m, out=q, workspace=ws, stream=7)
    _holds(rec, "moe_quantize_nvfp4", x=m, x_stride=64, dtype=FL, groups=3, rows=5, cols=48,
           given_scale=None, sorted_token_ids=None, codes=None, scale=q["scale"],
           global_scale=None, values=None, workspace=ws, workspace_bytes=5000)
    q, out = packed(3, 5, cols=48), torch.zeros(3, 5, 48, dtype=torch.float16)
    assert moe.moe_dequantize_nvfp4(**q, out=out, stream=7) is out
    _holds(rec, "moe_dequantize_nvfp4", groups=3, rows=5, cols=48, dtype=HF, out=out, **q)
    t, err = tables(8, 8, 64), torch.zeros(1, dtype=torch.int32)
    w, up = (tuple(packed(8, 40, cols=96).values()) for _ in range(2))
    rows, out = packed(4, cols=96), torch.zeros(64, 40)
    assert moe.moe_grouped_product_nvfp4(w, rows, t, 2, out=out, err_word=err, stream=7) is out
    common = dict(num_experts=8, out_dim=40, in_dim=96, M=4, top_k=2, num_rows=64, out_dtype=FL,
                  out=out, err_word=err, expert_offsets=t["expert_offsets"],
                  sorted_token_ids=t["sorted_token_ids"])
    got = _holds(rec, "moe_grouped_product_nvfp4", by_token=1, **rows, **common)
    assert [getattr(got["weight"]._obj, n) for n in ("codes", "scale", "global_scale")] == [
        v.data_ptr() for v in w]
    sorted_rows = packed(64, cols=96)
    moe.moe_grouped_gate_up_nvfp4(w, up, tuple(sorted_rows.values()), t, 2, M=4, out=out,
                                  err_word=err, stream=7)
    got = _holds(rec, "moe_grouped_gate_up_nvfp4", by_token=0, **sorted_rows, **common)
    for name, p in (("gate", w), ("up", up)):
        assert [getattr(got[name]._obj, n) for n in ("codes", "scale", "global_scale")] == [
            v.data_ptr() for v in p]


def test_binding_refuses_what_the_entry_points_cannot_read(rec):
    x = torch.zeros(4, 160, dtype=torch.bfloat16)
    t = tables(8, 8, 64)
    w, rows = packed(8, 40, cols=96), packed(4, cols=96)
    bad = [
        lambda: moe.moe_quantize_nvfp4(x[0]),
        lambda: moe.moe_quantize_nvfp4(x.double()),
        lambda: moe.moe_quantize_nvfp4(x[:, ::2]),
        lambda: moe.moe_quantize_nvfp4(torch.zeros(3, 5, 64)[:, ::2, :]
                                       .transpose(0, 1)),
        lambda: moe.moe_quantize_nvfp4(torch.zeros(3, 5, 64)[:, :3]),
        lambda: moe.moe_quantize_nvfp4(x, want=("code",)),
        lambda: moe.moe_quantize_nvfp4(x, out=dict(codes=torch.zeros(4, 160, dtype=U8))),
        lambda: moe.moe_quantize_nvfp4(x, out=dict(values=torch.zeros(4, 160))),
        lambda: moe.moe_quantize_nvfp4(x, global_scale=torch.ones(3)),
        lambda: moe.moe_quantize_nvfp4(x, global_scale=torch.ones(4).double()),
        lambda: moe.moe_quantize_nvfp4(x, tables=t),
        lambda: moe.moe_dequantize_nvfp4(w["codes"][0, 0], w["scale"], w["global_scale"]),
        lambda: moe.moe_dequantize_nvfp4(w["codes"], w["scale"][:, :, :1], w["global_scale"]),
        lambda: moe.moe_dequantize_nvfp4(**w, dtype=torch.float64),
        lambda: moe.moe_dequantize_nvfp4(**w, out=torch.zeros(8, 40, 95)),
        lambda: moe.moe_grouped_product_nvfp4(w, rows, t, 2, M=4),       # not in expert order
        lambda: moe.moe_grouped_product_nvfp4(w, packed(4, cols=64), t, 2),
        lambda: moe.moe_grouped_product_nvfp4(packed(9, 40, cols=96), rows, t, 2),
        lambda: moe.moe_grouped_product_nvfp4(packed(8, cols=96), rows, t, 2),
        lambda: moe.moe_grouped_product_nvfp4(w, rows, t, 2, out=torch.zeros(64, 41)),
        lambda: moe.moe_grouped_product_nvfp4(w, rows, t, 2, out_dtype=torch.float64),
        lambda: moe.moe_grouped_product_nvfp4(w, rows, t, 2, err_word=torch.zeros(1)),
        lambda: moe.moe_grouped_product_nvfp4(tuple(w.values())[:2], rows, t, 2),
        lambda: moe.moe_grouped_gate_up_nvfp4(w, packed(8, 41, cols=96), rows, t, 2),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(i)
    assert not rec.calls


def test_binding_refuses_tensors_off_the_device():
    x = torch.zeros(4, 160, dtype=torch.bfloat16)
    w, rows = packed(8, 40, cols=96), packed(4, cols=96)
    for f in (lambda: moe.moe_quantize_nvfp4(x), lambda: moe.moe_dequantize_nvfp4(**w),
              lambda: moe.moe_grouped_product_nvfp4(w, rows, tables(8, 8, 64), 2)):
        with pytest.raises(ValueError):
            f()
