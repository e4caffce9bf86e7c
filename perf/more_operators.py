"""Measured cases of the four-bit operators: rows and expert weights into NVFP4
(E2M1 codes, an E4M3 scale per 16 elements, an fp32 global scale) and back,
and the grouped products of four-bit rows and four-bit expert weights, plain
and with the SiLU product of gate and up.

With ``own`` false, ``run`` computes an operator in elementary torch
operations in fp32, rounded once at the end; with ``own`` true it makes the
framework's calls on the same state.  ``exact`` computes the same outputs
from the definitions in float64.

The definition of the four-bit form of x, by groups of elements that share a
global scale (a row, or an expert's matrix) and blocks of 16 in a row:

    g = max(max|x| / 2688, 2^-80), the maximum over the blocks without NaN
        and infinity                                          (fp32)
    s = e4m3(min(fl(max|block| / fl(6 g)), 448)), NaN where the block has one
    code = e2m1(fl(x / fl(s g))), ties to even, at most 6;  0 where s is 0
    value = code * fl(s g)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GLOBAL_MIN = 2.0 ** -80
PACKED = 0.5 + 1 / 16   # bytes of an element with its share of the block's scale


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def _pack(name, op, dtype, groups, rows, cols):
    """groups of rows x cols share a global scale: rows = 1 for token rows,
    groups = experts for weights."""
    return dict(name=name, op=op, dtype=dtype, groups=groups, rows=rows, cols=cols)


def _product(name, op, dtype, M, E, k, BS, cols, rows, by_token, skipped=0.0):
    """Weights [E, rows, cols]; by_token: the rows are the M tokens', else they
    are in expert order; skipped: the share of the slots whose expert is not here."""
    return dict(name=name, op=op, dtype=dtype, M=M, E=E, k=k, BS=BS, cols=cols, rows=rows,
                by_token=by_token, skipped=skipped)


def listed():
    return [
        # the tokens of a decode step ahead of their experts: latency alone counts
        _pack("quantize_decode_bf16", "quantize", "bf16", 8, 1, 2048),
        # a prefill batch's tokens
        _pack("quantize_prefill_bf16", "quantize", "bf16", 8192, 1, 4096),
        # a training step's expert weights, one global scale an expert
        _pack("quantize_experts_bf16", "quantize", "bf16", 32, 1536, 2048),
        # expert weights back to bf16, for products of the user's own
        _pack("dequantize_experts_bf16", "dequantize", "bf16", 64, 768, 2048),
        # a ragged batch's rows back to fp32
        _pack("dequantize_rows_f32", "dequantize", "f32", 5003, 1, 2880),
        # one token of a decode step: eight experts' gate and up
        _product("gate_up_one_token_bf16", "gate_up", "bf16", 1, 128, 8, 16, 2048, 768, True),
        # a verify batch: a few rows for each of many experts
        _product("gate_up_verify_bf16", "gate_up", "bf16", 128, 256, 8, 16, 4096, 1536, True),
        # a prefill batch
        _product("gate_up_prefill_bf16", "gate_up", "bf16", 4096, 128, 8, 64, 2048, 768, True),
        # a ragged batch with half of the experts on another device
        _product("gate_up_ragged_f16", "gate_up", "f16", 5003, 32, 4, 64, 2880, 2880, True, 0.5),
        # a decode step's down projection
        _product("product_decode_bf16", "product", "bf16", 8, 128, 8, 16, 768, 2048, False),
        # a large prefill batch's down projection
        _product("product_prefill_bf16", "product", "bf16", 8192, 256, 8, 128, 1536, 4096, False),
        # widths that are no whole tiles, fp32 results: a gradient through a transposed set
        _product("product_odd_f32", "product", "f32", 777, 48, 6, 1, 1120, 1000, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, steps):
    w, step = _log(rng, lo, hi), rng.choice(steps)
    return max(step, w // step * step)


def draw(rng):
    op = rng.choice(["quantize", "quantize", "dequantize", "gate_up", "gate_up", "product",
                     "product"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("quantize", "dequantize"):
        cols = _width(rng, 16, 8192, [128, 128, 32, 16])
        if rng.random() < 0.6:
            c = _pack("", op, dtype, _log(rng, 1, 32768), 1, cols)
        else:
            c = _pack("", op, dtype, _log(rng, 1, 128), _log(rng, 1, 4096), cols)
        most = 1 << 27
        while c["groups"] * c["rows"] * cols > most:
            c["groups"], c["rows"] = max(1, c["groups"] // 2), max(1, c["rows"] * 3 // 4)
    else:
        E = _log(rng, 4, 512)
        c = _product("", op, dtype, _log(rng, 1, 8192), E, rng.randint(1, min(8, E)),
                     rng.choice([1, 16, 64, 128]), _width(rng, 64, 4096, [256, 256, 64, 32]),
                     _width(rng, 32, 4096, [128, 128, 32, 8]), op == "gate_up" or rng.random() < 0.3,
                     rng.choice([0.0, 0.0, 0.25, 0.75]))
        flops = max(work(x)["flops"] for x in listed() if x["op"] == op)
        elements = max(x["E"] * x["rows"] * x["cols"] for x in listed() if x["op"] == op)
        while work(c)["flops"] > flops:
            c["M"] = max(1, c["M"] // 2)
        while c["E"] * c["rows"] * c["cols"] > elements:
            c["E"] = max(c["k"], c["E"] // 2)
            if c["E"] == c["k"]:
                break
    c.pop("name")
    return c


def work(case):
    """Inputs once and outputs once: quantisation writes the codes, scales and
    the values that they stand for; a product reads the weights of the experts
    that the routing is expected to reach."""
    b = BYTES[case["dtype"]]
    if case["op"] in ("quantize", "dequantize"):
        n = case["groups"] * case["rows"] * case["cols"]
        by = n * (PACKED + b) + 4 * case["groups"]
        return {"bytes": by + (n * b if case["op"] == "quantize" else 0), "flops": 2 * n}
    E, n = case["E"], case["M"] * case["k"]
    real = n * (1 - case["skipped"])
    active = E * (1 - case["skipped"]) * (1 - (1 - 1 / E) ** n)
    sets = 2 if case["op"] == "gate_up" else 1
    weights = sets * active * (case["rows"] * case["cols"] * PACKED + 4)
    rows = (case["M"] if case["by_token"] else real) * (case["cols"] * PACKED + 4)
    return {"bytes": weights + rows + real * case["rows"] * b + 4 * n + 4 * E,
            "flops": 2 * sets * real * case["rows"] * case["cols"]}


# --------------------------------------------------------------------------
# the inputs
# --------------------------------------------------------------------------

def _randn(g, *shape, scale=1.0):
    return torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g)


def _token_rows(g, n, cols):
    """Rows as they leave a norm: a few columns are much larger than the rest."""
    col = torch.exp(0.3 * _randn(g, cols))
    col = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 12.0 * col, col)
    return _randn(g, n, cols) * col


def _expert_rows(g, n, cols):
    """Rows as the SiLU product leaves them."""
    a = 1.5 * _randn(g, n, cols)
    return a / (1.0 + torch.exp(-a)) * _randn(g, n, cols, scale=1.5)


def _weights(g, E, rows, cols):
    """A set's (codes, scale, global scale), from normal weights whose spread
    differs by row; eight experts at a time."""
    parts = []
    for e in range(0, E, 8):
        n = min(8, E - e)
        w = _randn(g, n, rows, cols, scale=0.02) * torch.exp(0.3 * _randn(g, n, rows, 1))
        parts.append(_quantize(w)[:3])
    return tuple(torch.cat(p) for p in zip(*parts))


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
    offs = torch.zeros(E + 1, dtype=torch.long, device=flat.device)
    offs[1:] = torch.cumsum((count[:E] + BS - 1) // BS * BS, 0)
    sorted_key = key[order]
    rank = torch.arange(n, device=flat.device) - start[sorted_key]
    pos = torch.where(sorted_key < E, offs[sorted_key] + rank, torch.full_like(rank, -1))
    perm = torch.empty(n, dtype=torch.long, device=flat.device)
    perm[order] = pos
    where = torch.full((max_total + 1,), n, dtype=torch.int32, device=flat.device)
    where[torch.where(perm >= 0, perm, torch.full_like(perm, max_total))] = torch.arange(
        n, dtype=torch.int32, device=flat.device)
    return dict(sorted_token_ids=where[:max_total].clone(),
                expert_offsets=offs.to(torch.int32),
                token_to_perm=perm.to(torch.int32),
                num_tokens_post_padded=offs[E:].to(torch.int32)), max_total, count[:E]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(op=op, dtype=dt, values=torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda"))
    if op in ("quantize", "dequantize"):
        G, R, C = case["groups"], case["rows"], case["cols"]
        if R == 1:
            x = _token_rows(g, G, C).to(dt)
        else:
            x = (_randn(g, G, R, C, scale=0.02) * torch.exp(0.3 * _randn(g, G, R, 1))).to(dt)
        if op == "quantize":
            s["x"] = x
        else:
            s["packed"] = _quantize(x)[:3]
        return s
    M, E, k, R, C = case["M"], case["E"], case["k"], case["rows"], case["cols"]
    logits = _randn(g, M, E) + 0.5 * _randn(g, 1, E)   # some experts are busier than others
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    if case["skipped"]:
        away = torch.rand(E, generator=g, device="cuda") < case["skipped"]
        ids = torch.where(away[ids.long()], torch.full_like(ids, -1), ids)
    tables, max_total, count = _tables(ids, E, case["BS"])
    rows = _token_rows(g, M, C) if case["by_token"] else _expert_rows(g, max_total, C)
    rows = dict(zip(("codes", "scale", "global_scale"), _quantize(rows.to(torch.bfloat16))))
    s.update(tables=tables, M=M, k=k, by_token=case["by_token"], rows=rows, count=count,
             most=max(1, int(count.max())), weight=_weights(g, E, R, C),
             out=torch.zeros(max_total, R, dtype=dt, device="cuda"))
    if op == "gate_up":
        s["up"] = _weights(g, E, R, C)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quantize":
        _, scale, glob, values = _quantize(s["x"])
        return {"values": values.to(s["dtype"]), "scale": scale.view(torch.float8_e4m3fn),
                "global_scale": glob}
    if s["op"] == "dequantize":
        return _values(s, *s["packed"]).to(s["dtype"])
    return _product_plain(s)


def _run_own(s):
    import expert_routing_alignment_gb300 as moe
    op = s["op"]
    if op == "quantize":
        q = moe.moe_quantize_nvfp4(s["x"], want=("codes", "scale", "global_scale", "values"))
        return {"values": q["values"], "scale": q["scale"].view(torch.float8_e4m3fn),
                "global_scale": q["global_scale"]}
    if op == "dequantize":
        return moe.moe_dequantize_nvfp4(*s["packed"], dtype=s["dtype"])
    M = None if s["by_token"] else s["M"]
    if op == "gate_up":
        return moe.moe_grouped_gate_up_nvfp4(s["weight"], s["up"], s["rows"], s["tables"], s["k"],
                                             M=M, out=s["out"])
    return moe.moe_grouped_product_nvfp4(s["weight"], s["rows"], s["tables"], s["k"], M=M,
                                         out=s["out"])


def _quantize(x):
    """(codes, scale bytes, global scale, fp32 values) of x [G, C] or [G, R, C]."""
    f = x.float()
    b = f.reshape(*f.shape[:-1], f.shape[-1] // 16, 16)
    m = b.abs().amax(-1)
    whole = torch.isfinite(m)
    top = torch.where(whole, m, torch.zeros_like(m)).flatten(1).amax(1)
    # by a tensor: torch divides by a number through its rounded reciprocal
    glob = (top / torch.full_like(top, 2688.0)).clamp(min=GLOBAL_MIN)
    g = glob.view(-1, *[1] * (m.dim() - 1))
    scale = torch.where(whole, (m / (6.0 * g)).clamp(max=448.0),
                        torch.full_like(m, math.nan)).to(torch.float8_e4m3fn)
    step = (scale.float() * g)[..., None]
    q = (b / step).abs()
    up = [q > 0.25, q >= 0.75, q > 1.25, q >= 1.75, q > 2.5, q >= 3.5, q > 5.0]
    code = torch.stack([u.to(torch.uint8) for u in up]).sum(0, dtype=torch.uint8)
    mag = torch.where(code < 5, code.float() * 0.5, code.float() - 2.0 + (code == 7).float())
    # codes 0..4 are 0, 0.5, 1, 1.5, 2 and 5, 6, 7 are 3, 4, 6
    zero = step == 0
    mag = torch.where(zero, torch.zeros_like(mag), mag)
    code = torch.where(zero, torch.zeros_like(code), code | (torch.signbit(b).to(torch.uint8) << 3))
    code = code.reshape(f.shape)
    values = (torch.copysign(mag, b) * step).reshape(f.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8), glob, values)


def _values(s, codes, scale, glob):
    """The fp32 values of codes [G, C / 2] or [G, R, C / 2]."""
    c = torch.stack([codes & 15, codes >> 4], -1)
    v = s["values"][c.int()].view(*codes.shape[:-1], -1, 16)
    step = scale.view(torch.float8_e4m3fn).float() * glob.view(-1, *[1] * (codes.dim() - 1))
    return (v * step[..., None]).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _product_plain(s):
    t, most = s["tables"], s["most"]
    slots = torch.arange(most, device="cuda")
    real = slots[None, :] < s["count"][:, None]                       # [E, most]
    pos = t["expert_offsets"][:-1, None].long() + slots[None, :]
    rows = _values(s, *(s["rows"][n] for n in ("codes", "scale", "global_scale")))
    at = torch.where(real, pos, torch.zeros_like(pos))
    if s["by_token"]:
        at = t["sorted_token_ids"][at].long().clamp(max=s["M"] * s["k"] - 1) // s["k"]
    x = rows[at]                                                      # [E, most, C]
    y = torch.bmm(x, _values(s, *s["weight"]).transpose(1, 2))
    if "up" in s:
        y = y / (1.0 + torch.exp(-y)) * torch.bmm(x, _values(s, *s["up"]).transpose(1, 2))
    out = torch.zeros_like(s["out"])
    out[pos[real]] = y[real].to(out.dtype)
    return out


# --------------------------------------------------------------------------
# the same outputs in float64, from the definitions
# --------------------------------------------------------------------------

def _wide(codes, scale, glob):
    """Codes as float64 values, one matrix or one set of rows: [n, C]."""
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64,
                    device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        v[..., half::2] = mag[(c & 7).int()] * (1.0 - 2.0 * (c >> 3).double())
    s = scale.view(torch.float8_e4m3fn).to(torch.float64)
    return v * torch.repeat_interleave(s, 16, dim=-1) * glob


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "dequantize":
        codes, scale, glob = s["packed"]
        return torch.stack([_wide(codes[i], scale[i], glob[i].double())
                            for i in range(codes.shape[0])]) if codes.dim() == 3 else \
            _wide(codes, scale, glob.double()[:, None])
    if op == "quantize":
        values, scales, globs = [], [], []
        x = s["x"]
        step_rows = 1 if x.dim() == 3 else 1024
        for i in range(0, x.shape[0], step_rows):
            part = x[i: i + step_rows].double()
            blocks = part.unflatten(-1, (-1, 16))
            m = blocks.abs().amax(-1)
            top = m.flatten(1).amax(1)
            top = (top / torch.full_like(top, 2688.0)).clamp(min=GLOBAL_MIN)
            g = top.float()
            six = (6.0 * g).double()   # as the definition rounds it
            shape = (-1,) + (1,) * (m.dim() - 1)
            # quotients as the definition rounds them: by a step that is itself
            # rounded, exact ties would otherwise fall to either side
            sc = (m / six.view(shape)).float().double().clamp(max=448.0)
            # the nearest E4M3 number: steps of 2^(e - 3), 2^-9 below 2^-6
            e = (torch.frexp(sc)[1].long() - 1).clamp(min=-6)
            unit = ((e - 3 + 1023) << 52).view(torch.float64)
            sc = torch.round(sc / unit) * unit
            t = (sc * g.double().view(shape)).float().double()[..., None]
            q = torch.where(t > 0, blocks / torch.where(t > 0, t, torch.ones_like(t)),
                            torch.zeros_like(blocks))
            q = q.float().double()
            a = q.abs().clamp(max=6.0)
            # E2M1: steps of 1/2 below 2, of 1 below 4, of 2 up to 6
            half = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
            code = torch.round(a / half) * half
            values.append((torch.sign(q) * code * t).reshape(part.shape))
            scales.append(sc)
            globs.append(top)
        return {"values": torch.cat(values), "scale": torch.cat(scales),
                "global_scale": torch.cat(globs)}
    t = s["tables"]
    offs = t["expert_offsets"].tolist()
    count = s["count"].tolist()
    r = s["rows"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e, n in enumerate(count):
        if not n:
            continue
        p = torch.arange(offs[e], offs[e] + n, device="cuda")
        at = t["sorted_token_ids"][p].long() // s["k"] if s["by_token"] else p
        x = _wide(r["codes"][at], r["scale"][at], r["global_scale"][at].double()[:, None])

        def times(w):
            return x @ _wide(w[0][e], w[1][e], w[2][e].double()).T

        y = times(s["weight"])
        if "up" in s:
            y = y * torch.sigmoid(y) * times(s["up"])
        out[p] = y
    return out
