"""Measured cases of the operators around the expert products: tokens into
expert order and back (each direction with its gradient), the gradient of the
top-k softmax, and the residual addition with the RMS norm in front of the
router (its 8-bit output and its gradient).

With ``own`` false, ``run`` computes an operator in elementary torch
operations in fp32, rounded once at the end; with ``own`` true it makes the
framework's calls on the same state.  ``exact`` computes the same outputs
from the definitions in float64.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def _tokens(name, op, way, dtype, M, H, E, k, BS, skipped=0.0):
    """skipped: the share of the slots whose expert is not here."""
    return dict(name=name, op=op, way=way, dtype=dtype, M=M, H=H, E=E, k=k, BS=BS,
                skipped=skipped)


def _norm(name, way, dtype, M, H, quantise=False):
    return dict(name=name, op="norm", way=way, dtype=dtype, M=M, H=H, quantise=quantise)


def listed():
    return [
        # a decode step of eight sequences: latency alone counts
        _tokens("dispatch_decode_bf16", "dispatch", "forward", "bf16", 8, 2048, 128, 8, 16),
        # a prefill batch in 8 bits, its scales by 128 columns along with it
        _tokens("dispatch_prefill_e4m3", "dispatch", "forward", "e4m3", 4096, 4096, 256, 8, 64),
        # the gradient of a training batch's tokens
        _tokens("dispatch_grad_bf16", "dispatch", "backward", "bf16", 8192, 2048, 128, 8, 128),
        # a verify batch's expert outputs back to token order
        _tokens("combine_verify_bf16", "combine", "forward", "bf16", 128, 4096, 256, 8, 64),
        # a ragged batch with half of the experts on another device
        _tokens("combine_ragged_f16", "combine", "forward", "f16", 5003, 2880, 32, 4, 64, 0.5),
        # a large training batch: gradients of rows and of weights
        _tokens("combine_grad_bf16", "combine", "backward", "bf16", 16384, 4096, 256, 8, 128),
        # the router trained behind frozen experts: the layer's own fp32 rows,
        # bf16 gradients of its output, the weights' gradients alone
        _tokens("router_grad_f32", "combine", "weights", "f32", 512, 4096, 256, 8, 64),
        # the router's gradient of a decode-sized and of a training batch
        dict(name="topk_grad_small", op="topk", M=8, E=128, k=8),
        dict(name="topk_grad_large", op="topk", M=32768, E=256, k=8),
        # a decode step's residual addition and norm
        _norm("norm_decode_bf16", "forward", "bf16", 8, 2048),
        # a prefill batch's, with the rows that block-scaled products read
        _norm("norm_prefill_e4m3", "forward", "bf16", 4096, 4096, True),
        # a training batch's gradient
        _norm("norm_grad_bf16", "backward", "bf16", 10007, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _hidden(rng):
    h = _log(rng, 64, 8192)
    step = rng.choice([128, 128, 128, 8, 8, 1])   # whole blocks, whole vectors, any
    return max(step, h // step * step)


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["dispatch", "dispatch", "combine", "combine", "combine", "topk", "norm",
                     "norm", "norm"])
    E = _log(rng, 4, 1024)
    k = rng.randint(1, min(8, E))
    M = _log(rng, 1, 16384)
    H = _hidden(rng)
    if op == "topk":
        return dict(op=op, M=_log(rng, 1, 32768), E=E, k=k)
    if op == "norm":
        way = rng.choice(["forward", "forward", "backward"])
        c = _norm("", way, rng.choice(["bf16", "bf16", "f16", "f32"]), M, H,
                  way == "forward" and rng.random() < 0.5)
    else:
        way = rng.choice(["forward", "backward"] + (["weights"] if op == "combine" else []))
        kinds = ["bf16", "bf16", "f16", "f32"]
        if op == "dispatch" and way == "forward":
            kinds += ["e4m3", "e4m3"]
        c = _tokens("", op, way, rng.choice(kinds), M, H, E, k, rng.choice([1, 16, 64, 128]),
                    rng.choice([0.0, 0.0, 0.25, 0.75]))
    c.pop("name")
    while work(c)["bytes"] > most:
        c["M"] = max(1, c["M"] // 2)
    return c


def _kinds(case):
    """The types of the expert rows and of the token rows: fp32 rows of a
    combination meet bf16 tokens, as in the framework's own layer."""
    rows = case["dtype"]
    return rows, "bf16" if rows == "f32" and case["op"] == "combine" else rows


def work(case):
    """Inputs once and outputs once.  The padded length depends on the seed's
    routing: each of the experts expected to have a token ends half a block
    early on average, and has one block at least."""
    M = case["M"]
    if case["op"] == "topk":
        n = M * case["k"]
        return {"bytes": 12 * n + 4 * M * case["E"], "flops": 4 * n}
    H = case["H"]
    if case["op"] == "norm":
        b = BYTES[case["dtype"]]
        if case["way"] == "backward":   # dout, s, dsum -> dx; weight, rstd -> dweight
            return {"bytes": 4 * b * M * H + b * H + 4 * H + 4 * M, "flops": 10 * M * H}
        out = M * H + 4 * M * -(-H // 128) if case["quantise"] else b * M * H
        return {"bytes": 3 * b * M * H + b * H + out + 4 * M, "flops": 6 * M * H}
    E, BS = case["E"], case["BS"]
    n = M * case["k"]
    real = n * (1 - case["skipped"])
    active = E * (1 - (1 - 1 / E) ** real)
    total = max(real + active * (BS - 1) / 2, active * BS)
    rb, tb = (BYTES[d] for d in _kinds(case))
    scale = 4 * -(-H // 128) if case["dtype"] == "e4m3" else 0
    if case["op"] == "dispatch":
        if case["way"] == "forward":
            return {"bytes": M * (H * rb + scale) + total * (H * rb + scale) + 4 * n,
                    "flops": 0}
        return {"bytes": real * H * rb + M * H * tb + 4 * n, "flops": real * H}
    if case["way"] == "forward":
        return {"bytes": real * H * rb + M * H * tb + 8 * n, "flops": 2 * real * H}
    by = M * H * tb + real * H * rb + 12 * n
    if case["way"] == "weights":
        return {"bytes": by, "flops": 2 * real * H}
    return {"bytes": by + total * H * rb, "flops": 3 * real * H}


# --------------------------------------------------------------------------
# the inputs
# --------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(
        0.0, scale, generator=g).to(dtype)


def _route(g, M, E, k):
    """Top-k ids and softmax weights of logits with a bias per expert (some
    experts are busier than others)."""
    logits = _randn(g, M, E) + 0.5 * _randn(g, 1, E)
    v, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(v, dim=1)


def _tables(ids, E, BS):
    """The alignment of the flat ids (ids outside [0, E) are skipped): sorted
    positions in expert order, each expert's run padded to a multiple of BS."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    bound = min(n * BS, n + E * (BS - 1))
    max_total = -(-bound // BS) * BS
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=E + 1)
    start = torch.cumsum(count, 0) - count
    padded = (count[:E] + BS - 1) // BS * BS
    offs = torch.zeros(E + 1, dtype=torch.long, device=flat.device)
    offs[1:] = torch.cumsum(padded, 0)
    sorted_key = key[order]
    rank = torch.arange(n, device=flat.device) - start[sorted_key]
    pos = torch.where(sorted_key < E, offs[sorted_key] + rank, torch.full_like(rank, -1))
    perm = torch.empty(n, dtype=torch.long, device=flat.device)
    perm[order] = pos
    where = torch.full((max_total + 1,), n, dtype=torch.int32, device=flat.device)
    where[torch.where(perm >= 0, perm, torch.full_like(perm, max_total))] = torch.arange(
        n, dtype=torch.int32, device=flat.device)
    return dict(sorted_token_ids=where[:max_total].clone(),
                token_to_perm=perm.to(torch.int32),
                num_tokens_post_padded=offs[E:].to(torch.int32)), max_total


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, op = case["M"], case["op"]
    s = dict(op=op, way=case.get("way"), M=M)
    if op == "topk":
        ids, w = _route(g, M, case["E"], case["k"])
        s.update(ids=ids, w=w, dw=_randn(g, M, case["k"]), E=case["E"])
        return s
    H, dt = case["H"], DTYPES[case["dtype"]]
    if op == "norm":
        w = (1.0 + _randn(g, H, scale=0.1)).to(dt)
        s.update(weight=w, quantise=case["quantise"])
        a = _randn(g, M, H, dtype=dt)
        b = _randn(g, M, H, dtype=dt, scale=4.0)   # the residual stream is the larger one
        if case["way"] == "forward":
            s.update(x=a, residual=b)
        else:
            s.update(dout=a, sum=b, dsum=_randn(g, M, H, dtype=dt),
                     rstd=torch.rsqrt(b.double().square().mean(1) + EPS).float())
        return s
    E, k, BS = case["E"], case["k"], case["BS"]
    ids, w = _route(g, M, E, k)
    if case["skipped"]:
        away = torch.rand(E, generator=g, device="cuda") < case["skipped"]
        ids = torch.where(away[ids.long()], torch.full_like(ids, -1), ids)
    tables, max_total = _tables(ids, E, BS)
    tok = DTYPES[_kinds(case)[1]]
    s.update(tables=tables, k=k, w=w)
    if op == "dispatch" and case["way"] == "forward":
        if case["dtype"] == "e4m3":
            s["x"] = _randn(g, M, H, scale=64.0).clamp(-E4M3_MAX, E4M3_MAX).to(dt)
            s["x_scale"] = torch.rand(M, -(-H // 128), generator=g, device="cuda") * 0.01
            s["rows_scale"] = torch.zeros(max_total, -(-H // 128), device="cuda")
        else:
            s["x"] = _randn(g, M, H, dtype=dt)
        s["rows"] = torch.zeros(max_total, H, dtype=torch.uint8 if case["dtype"] == "e4m3" else dt,
                                device="cuda")
        if case["dtype"] == "e4m3":
            s["rows"] = s["rows"].view(dt)
    elif op == "dispatch":
        s["drows"] = _randn(g, max_total, H, dtype=dt)
    else:
        s["rows"] = _randn(g, max_total, H, dtype=dt)
        if case["way"] == "backward":
            s["drows"] = torch.zeros(max_total, H, dtype=dt, device="cuda")
        if case["way"] != "forward":
            s["dout"] = _randn(g, M, H, dtype=tok)
        s["out_dtype"] = tok
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    op, way = s["op"], s["way"]
    if op == "topk":
        return _topk_plain(s)
    if op == "norm":
        return _norm_plain(s) if way == "forward" else _norm_grad_plain(s)
    if op == "dispatch":
        return _dispatch_plain(s) if way == "forward" else _dispatch_grad_plain(s)
    return _combine_plain(s) if way == "forward" else _combine_grad_plain(s)


def _run_own(s):
    import expert_routing_alignment_gb300 as moe
    op, way = s["op"], s["way"]
    if op == "topk":
        return moe.moe_topk_softmax_backward(s["ids"], s["w"], s["dw"], s["E"])
    if op == "norm":
        if way == "forward":
            want = ("sum", "rstd") + (("codes", "scale") if s["quantise"] else ("out",))
            return moe.moe_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"],
                                       want=want)
        dx, dw = moe.moe_add_rmsnorm_backward(s["dout"], s["sum"], s["weight"], s["rstd"],
                                              dsum=s["dsum"])
        return {"dx": dx, "dweight": dw}
    t = s["tables"]
    if op == "dispatch":
        if way == "forward":
            return moe.moe_dispatch(s["x"], t, s["k"], rows=s["rows"], x_scale=s.get("x_scale"),
                                    rows_scale=s.get("rows_scale"))
        return moe.moe_dispatch_backward(s["drows"], t, s["M"], s["k"])
    if way == "forward":
        return moe.moe_combine(s["rows"], s["w"], t, out_dtype=s["out_dtype"])
    drows, dw = moe.moe_combine_backward(s["dout"], s["rows"], s["w"], t, drows=s.get("drows"),
                                         want_drows=way == "backward")
    return {"drows": drows, "dtopk_w": dw}


def _slots(s):
    perm = s["tables"]["token_to_perm"].long()
    return perm, perm >= 0


def _scattered(s, v):
    """v's rows at their slots' positions, zero everywhere else."""
    perm, real = _slots(s)
    slot = torch.nonzero(real).squeeze(1)
    buf = torch.zeros(s["rows"].shape[0], v.shape[1], dtype=v.dtype, device=v.device)
    return buf.index_copy(0, perm[slot], v[slot // s["k"]])


def _dispatch_plain(s):
    if "x_scale" not in s:
        return _scattered(s, s["x"])
    codes = _scattered(s, s["x"].view(torch.uint8))
    return codes.view(torch.float8_e4m3fn), _scattered(s, s["x_scale"])


def _taken(s, rows):
    """rows by slot [M, k, H] in fp32, zero where the slot is skipped."""
    perm, real = _slots(s)
    v = rows[perm.clamp(min=0)].float()
    v = torch.where(real[:, None], v, torch.zeros((), device=v.device))
    return v.view(s["M"], s["k"], rows.shape[1])


def _dispatch_grad_plain(s):
    return _taken(s, s["drows"]).sum(1).to(s["drows"].dtype)


def _combine_plain(s):
    return (_taken(s, s["rows"]) * s["w"][:, :, None]).sum(1).to(s["out_dtype"])


def _combine_grad_plain(s):
    perm, real = _slots(s)
    d = s["dout"].float()
    out = {"drows": None, "dtopk_w": (_taken(s, s["rows"]) * d[:, None, :]).sum(2)}
    if s["way"] == "backward":
        slot = torch.nonzero(real).squeeze(1)
        g = d[slot // s["k"]] * s["w"].reshape(-1)[slot][:, None]
        buf = torch.zeros_like(s["drows"])
        out["drows"] = buf.index_copy(0, perm[slot], g.to(buf.dtype))
    return out


def _topk_plain(s):
    w, dw = s["w"], s["dw"]
    g = w * (dw - (w * dw).sum(1, keepdim=True))
    return torch.zeros(s["M"], s["E"], device=g.device).scatter_add(1, s["ids"].long(), g)


def _norm_plain(s):
    t = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = t.float()
    rstd = 1.0 / torch.sqrt(f.square().mean(1) + EPS)
    v = f * rstd[:, None] * s["weight"].float()
    if not s["quantise"]:
        return {"sum": t, "rstd": rstd, "out": v.to(t.dtype)}
    M, H = v.shape
    blocks = -(-H // 128)
    p = torch.nn.functional.pad(v, (0, blocks * 128 - H)).view(M, blocks, 128)
    scale = (p.abs().amax(2) / E4M3_MAX).clamp(min=SCALE_MIN)
    codes = (p / scale[:, :, None]).view(M, blocks * 128)[:, :H].to(torch.float8_e4m3fn)
    return {"sum": t, "rstd": rstd, "codes": codes, "scale": scale}


def _norm_grad_plain(s):
    d, f, w, r = s["dout"].float(), s["sum"].float(), s["weight"].float(), s["rstd"][:, None]
    xh = f * r
    g = d * w
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True)) + s["dsum"].float()
    return {"dx": dx.to(s["dout"].dtype), "dweight": (d * xh).sum(0)}


# --------------------------------------------------------------------------
# the same outputs in float64, from the definitions
# --------------------------------------------------------------------------

def _e4m3(q):
    """The E4M3 values nearest to float64 q (|q| <= 448), ties to even."""
    e = (torch.frexp(q)[1].long() - 1).clamp(min=-6) - 3
    step = ((e + 1023) << 52).view(torch.float64)   # 2^e; torch.ldexp is not exact
    return torch.round(q / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op, way = s["op"], s["way"]
    if op == "topk":
        out = torch.zeros(s["M"], s["E"], dtype=torch.float64, device="cuda")
        w, dw = s["w"].double(), s["dw"].double()
        mean = torch.einsum("tj,tj->t", w, dw)
        for j in range(w.shape[1]):
            col = s["ids"][:, j: j + 1].long()
            out.scatter_add_(1, col, (w[:, j] * (dw[:, j] - mean))[:, None])
        return out
    if op == "norm" and way == "forward":
        f = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        H = f.shape[1]
        rstd = (torch.einsum("th,th->t", f, f) / H + EPS) ** -0.5
        v = torch.einsum("th,t,h->th", f, rstd, s["weight"].double())
        if not s["quantise"]:
            return {"sum": f, "rstd": rstd, "out": v}
        # v/scale = 448 s w / max|s w|: without rstd every product is exact, and
        # so are the ties of the rounding to a code
        p, codes, scales = f * s["weight"].double(), [], []
        for c in range(0, H, 128):
            b, most = p[:, c: c + 128], p[:, c: c + 128].abs().max(1).values
            scale = most * rstd / E4M3_MAX
            q = torch.where((scale >= SCALE_MIN)[:, None], b * E4M3_MAX / most[:, None],
                            b * rstd[:, None] / SCALE_MIN)
            codes.append(_e4m3(q))
            scales.append(scale.clamp(min=SCALE_MIN))
        return {"sum": f, "rstd": rstd, "codes": torch.cat(codes, 1),
                "scale": torch.stack(scales, 1)}
    if op == "norm":
        d, f, w = s["dout"].double(), s["sum"].double(), s["weight"].double()
        r = s["rstd"].double()
        dot = torch.einsum("th,th,h->t", d, f, w) * r / f.shape[1]
        dx = s["dsum"].double() + r[:, None] * (d * w) - (dot * r * r)[:, None] * f
        return {"dx": dx, "dweight": torch.einsum("th,th,t->h", d, f, r)}
    perm = s["tables"]["token_to_perm"].view(s["M"], s["k"]).long()
    if op == "dispatch" and way == "forward":
        def scattered(v):
            # behind the last row, one that takes what is skipped
            out = torch.zeros(s["rows"].shape[0] + 1, v.shape[1], dtype=torch.float64,
                              device="cuda")
            for j in range(s["k"]):
                out[perm[:, j]] = v
            return out[:-1]
        x = s["x"].float().double()
        return (scattered(x), scattered(s["x_scale"].double())) if "x_scale" in s else scattered(x)
    src = s["drows"] if op == "dispatch" else s["rows"]
    w = s["w"].double() if op == "combine" else torch.ones_like(s["w"], dtype=torch.float64)
    out = torch.zeros(s["M"], src.shape[1], dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    dr = torch.zeros(src.shape[0] + 1, src.shape[1], dtype=torch.float64,
                     device="cuda") if way == "backward" and op == "combine" else None
    for j in range(s["k"]):
        here = perm[:, j] >= 0
        p = perm[here, j]
        if "dout" not in s:
            out[here] += src[p].double() * w[here, j: j + 1]
            continue
        d = s["dout"][here].double()
        dw[here, j] = torch.einsum("th,th->t", d, src[p].double())
        if dr is not None:
            dr[p] = d * w[here, j: j + 1]
    if "dout" not in s:
        return out
    return {"drows": None if dr is None else dr[:-1], "dtopk_w": dw}
