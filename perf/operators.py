"""Cases of the operators around and inside the expert MLP, each in a plain form and as the library's calls.

Three operators of a mixture-of-experts layer:
  route   the top-k experts of every token from its router logits, their weights, and the logits'
          gradient (`moe_route`, `moe_route_bwd`)
  move    tokens sorted by expert and back: token rows copied into expert order, expert outputs summed
          per token with or without their weights, and the gradients of both (`moe_dispatch`,
          `moe_combine`, `moe_combine_bwd`, `moe_dispatch_bwd`)
  mxfp4   microscaled 4-bit floating point (E2M1 elements, one E8M0 scale per 32): quantisation and
          grouped product, forward with weights kept in 4 bits, or a linear layer's whole step

With `own` false `run` computes them in elementary torch operations; with `own` true it makes the calls
a user of the library makes.  `exact` computes the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 32  # elements per MXFP4 scale
STEP = 128  # elements per K step: the scales of a step are kept together per row


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one decoding step of 16 requests: latency
        dict(name="route_decode", op="route", tokens=16, experts=32, topk=4, score="softmax", renormalize=True,
             dtype="bf16", masked=0.0, grad=False),
        # a training batch over many experts, sigmoid scores in FP32
        dict(name="route_train_wide", op="route", tokens=65536, experts=256, topk=8, score="sigmoid",
             renormalize=True, dtype="f32", masked=0.0, grad=True),
        # odd sizes, experts switched off for some tokens, padding tokens with no expert at all
        dict(name="route_train_masked", op="route", tokens=4099, experts=61, topk=3, score="softmax",
             renormalize=False, dtype="bf16", masked=0.3, grad=True),
        # one decoding step of eight requests, two experts each: latency
        dict(name="move_decode", op="move", tokens=8, topk=2, experts=16, hidden=4096, dtype="bf16",
             weights="combine", dropped=0.0, grad=False),
        # a prompt batch of the 16-expert layer: 32768 rows
        dict(name="move_prefill", op="move", tokens=16384, topk=2, experts=16, hidden=4096, dtype="bf16",
             weights="combine", dropped=0.0, grad=False),
        # backward of the 32-expert layer with 65536 rows; the weights are applied inside the expert
        dict(name="move_train_rows", op="move", tokens=8192, topk=8, experts=32, hidden=7168, dtype="bf16",
             weights="rows", dropped=0.0, grad=True),
        # FP32 rows of an odd width, a quarter of the slots without an expert, weights at the combine
        dict(name="move_train_odd", op="move", tokens=1021, topk=3, experts=61, hidden=1001, dtype="f32",
             weights="combine", dropped=0.25, grad=True),
        # one decoding step of 16 requests, two of 16 experts each: reads the 4-bit weights once
        dict(name="mxfp4_decode", op="mxfp4", rows=32, experts=16, n=4096, k=4096, skew=0.0, step=False),
        # a prompt batch of the 16-expert layer
        dict(name="mxfp4_prefill", op="mxfp4", rows=32768, experts=16, n=4096, k=4096, skew=0.0, step=False),
        # a skewed batch of the 32-expert layer's second linear, some experts empty
        dict(name="mxfp4_skewed", op="mxfp4", rows=16384, experts=32, n=7168, k=2048, skew=1.2, step=False),
        # a linear layer's training step on a small, ragged batch
        dict(name="mxfp4_step_small", op="mxfp4", rows=256, experts=4, n=256, k=512, skew=0.7, step=True),
        # a linear layer's training step at the 16-expert layer's size: output, input and weight gradients
        dict(name="mxfp4_step", op="mxfp4", rows=32768, experts=16, n=4096, k=4096, skew=0.0, step=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "move", "mxfp4"))
    if op == "route":
        experts = _log(rng, 2, 256)
        return dict(op=op, tokens=_log(rng, 1, 65536), experts=experts, topk=rng.randint(1, min(8, experts)),
                    score=rng.choice(("softmax", "sigmoid")), renormalize=rng.random() < 0.5,
                    dtype=rng.choice(("bf16", "f32")), masked=rng.choice((0.0, 0.3)), grad=rng.random() < 0.6)
    if op == "move":
        experts, hidden = _log(rng, 2, 256), _log(rng, 64, 7168)
        if rng.random() < 0.6:
            hidden = -(-hidden // 64) * 64
        topk = rng.randint(1, min(8, experts))
        return dict(op=op, tokens=min(_log(rng, 1, 32768), 65536 // topk), topk=topk, experts=experts, hidden=hidden,
                    dtype=rng.choice(("bf16", "bf16", "f32")) if hidden <= 2048 else "bf16",
                    weights=rng.choice(("combine", "rows")), dropped=rng.choice((0.0, 0.25)), grad=rng.random() < 0.5)
    experts, n, k = _log(rng, 1, 32), 32 * _log(rng, 4, 224), 32 * _log(rng, 4, 224)
    while experts * n * k > 16 * 4096 * 4096:
        experts = max(1, experts // 2)
        n = 32 * max(4, n // 64)
    rows = _log(rng, 1, min(32768, 32768 * 4096 * 4096 // (n * k)))
    return dict(op=op, rows=rows, experts=experts, n=n, k=k, skew=rng.choice((0.0, 0.7, 1.2)), step=rng.random() < 0.5)


def splits_of(case):
    """Rows of each expert: equal shares, or shares that fall off as rank^-skew in a shuffled order with
    the last eighth of the ranks empty.  They go by the case alone."""
    e, m = case["experts"], case["rows"]
    r = np.random.RandomState(e * 1009 + m % 100003)
    if case["skew"] == 0.0:
        return [m * (i + 1) // e - m * i // e for i in r.permutation(e)]
    w = np.arange(1, e + 1, dtype=np.float64) ** -case["skew"]
    if e >= 8:
        w[e - e // 8:] = 0.0
    return [int(v) for v in r.multinomial(m, w[r.permutation(e)] / w.sum())]


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s = 2 if case["dtype"] == "bf16" else 4
        # logits in, experts and weights out; backward: the weights' gradient in, the logits' out
        b = t * (e * s + 8 * k)
        if case["grad"]:
            b += t * (4 * k + e * s)
        return {"bytes": b, "flops": t * e * (4 if not case["grad"] else 8)}
    if case["op"] == "move":
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        s = 2 if case["dtype"] == "bf16" else 4
        m = int(t * k * (1.0 - case["dropped"]))
        if not case["grad"]:
            # token rows in, expert rows out; expert outputs in, tokens out; experts, weights, row numbers
            return {"bytes": 2 * (t + m) * h * s + t * k * (4 + 8 + 4), "flops": 2 * m * h}
        # token gradients in and out, both expert-row gradients; with the weights at the combine the
        # expert outputs too
        b = 2 * (t + m) * h * s + t * k * 12
        if case["weights"] == "combine":
            b += m * h * s
        return {"bytes": b, "flops": (4 if case["weights"] == "combine" else 1) * m * h}
    m, n, k = case["rows"], case["n"], case["k"]
    hit = sum(1 for v in splits_of(case) if v)
    if not case["step"]:
        # rows in BF16, the weights of the experts that have rows in 4 bits, outputs in BF16
        return {"bytes": 2 * m * k + hit * n * k * 17 // 32 + 2 * m * n, "flops": 2 * m * n * k}
    # x, weights and dy in BF16; y, dx and the weight gradient in BF16
    return {"bytes": 2 * (2 * m * k + 2 * m * n) + 2 * 2 * case["experts"] * n * k, "flops": 6 * m * n * k}


# ----------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = {"case": case}

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        logits = normal(t, e, std=1.5, dtype=torch.float32)
        if case["masked"]:
            off = torch.rand((t, e), generator=g, device="cuda") < case["masked"]
            pad = torch.rand((t, 1), generator=g, device="cuda") < 0.1
            logits = logits.masked_fill(off | pad, -math.inf)
        d["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        d["dweights"] = normal(t, k, dtype=torch.float32)
        return d
    if case["op"] == "move":
        t, k, e, h = case["tokens"], case["topk"], case["experts"], case["hidden"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # k distinct experts a token, some of them more popular than others
        score = torch.rand((t, e), generator=g, device="cuda") + torch.rand((1, e), generator=g, device="cuda")
        idx = score.sort(dim=1, descending=True).indices[:, :k].to(torch.int32)
        if case["dropped"]:
            idx = idx.masked_fill(torch.rand((t, k), generator=g, device="cuda") < case["dropped"], -1)
        d["idx"] = idx.contiguous()
        d["weights"] = torch.rand((t, k), generator=g, device="cuda")
        m = t * k
        d["row_of_slot"], _ = _sort_plain(d["idx"], e)
        if not case["grad"]:
            d["x"] = normal(t, h, dtype=dt)
            d["out_rows"] = normal(m, h, dtype=dt)  # what the experts answer
            d["rows"] = torch.zeros((m, h), dtype=dt, device="cuda")  # rows past the last used one stay zeros
            d["row_weights"] = torch.zeros(m, device="cuda")
        else:
            d["dy"] = normal(t, h, dtype=dt)
            d["out_rows"] = normal(m, h, dtype=dt)
            d["dx_rows"] = normal(m, h, dtype=dt)  # gradient that the experts return for their rows
            d["dp_rows"] = normal(m, dtype=torch.float32)  # and for the rows' weights
            d["dout_rows"] = torch.zeros((m, h), dtype=dt, device="cuda")
        return d
    m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    d["splits"] = splits_of(case)
    d["x"] = normal(m, k)
    w = normal(e * n, k, std=0.02)
    if case["step"]:
        d["w"], d["dy"] = w, normal(m, n)
    else:
        # the weights as the library's 4-bit tensor: two codes a byte, and four scales a row and K step
        codes, scales = _codes_plain(w.float())
        steps = -(-k // STEP)
        d["w_codes"] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
        s = torch.zeros((e * n, 4 * steps), dtype=torch.uint8, device="cuda")
        s[:, : k // BLOCK] = scales
        d["w_scales"] = s.view(e * n, steps, 4).permute(1, 0, 2).contiguous()
    return d


# ------------------------------------------------------------------------------------- plain forms


def _route_plain(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["topk"]
    x = s["logits"].float()
    top = torch.sort(x, dim=1, descending=True, stable=True)
    there = top.values[:, :k] > -math.inf
    pick = top.indices[:, :k]
    if c["score"] == "softmax":
        ex = torch.exp(x - top.values[:, :1].clamp_min(-3.0e38))
        p = ex / ex.sum(dim=1, keepdim=True).clamp_min(1e-37)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    w = torch.where(there, p.gather(1, pick), 0.0)
    total = w.sum(dim=1, keepdim=True).clamp_min(1e-37)
    if c["renormalize"]:
        w = w / total
    out = {"experts": torch.where(there, pick, -1).to(torch.int32), "weights": w}
    if c["grad"]:
        # in 64 bits: g_j - sum_i g_i w_i cancels where one weight is near 1
        x = x.double()
        if c["score"] == "softmax":
            ex = torch.exp(x - top.values[:, :1].clamp_min(-3.0e38))
            p = ex / ex.sum(dim=1, keepdim=True).clamp_min(1e-37)
        else:
            p = 1.0 / (1.0 + torch.exp(-x))
        w = torch.where(there, p.gather(1, pick), 0.0)
        gw = torch.where(there, s["dweights"], 0.0).double()
        if c["renormalize"]:
            total = w.sum(dim=1, keepdim=True).clamp_min(1e-37)
            gw = torch.where(there, gw - (gw * w).sum(dim=1, keepdim=True) / total, 0.0) / total
        gp = torch.zeros((t, e), dtype=torch.float64, device="cuda").scatter_(1, pick, gw)
        if c["score"] == "softmax":
            dx = p * (gp - (gp * p).sum(dim=1, keepdim=True))
        else:
            dx = gp * p * (1.0 - p)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _sort_plain(idx, experts):
    """Row of every slot in expert order (-1 where it has no expert), and the rows of each expert."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, experts)
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=idx.device))
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=idx.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    return torch.where(flat >= 0, rows, -1).to(torch.int32).view(idx.shape), counts[:experts]


def _move_plain(s):
    c = s["case"]
    t, k, h = c["tokens"], c["topk"], c["hidden"]
    m = t * k
    if not c["grad"]:
        row, counts = _sort_plain(s["idx"], c["experts"])
        # slots without an expert go to one row past the end
        at = torch.where(row.view(-1) >= 0, row.view(-1), m).long()
        rows = torch.zeros((m + 1, h), dtype=s["x"].dtype, device="cuda")
        rows[at] = s["x"].repeat_interleave(k, dim=0)
        out = {"row_of_slot": row, "splits": counts, "rows": rows[:m]}
        got = s["out_rows"].float()[row.clamp_min(0).long()]
        got = torch.where((row >= 0)[:, :, None], got, 0.0)
        if c["weights"] == "combine":
            got = got * s["weights"][:, :, None]
        else:
            out["row_weights"] = torch.zeros(m + 1, device="cuda").scatter_(0, at, s["weights"].view(-1))[:m]
        out["y"] = got.sum(dim=1).to(s["x"].dtype)
        return out
    row = s["row_of_slot"]
    there = row >= 0
    at = torch.where(there, row, m).view(-1).long()
    dy = s["dy"].float()
    per_slot = dy.repeat_interleave(k, dim=0)
    if c["weights"] == "combine":
        got = s["out_rows"].float()[row.clamp_min(0).long()]
        dw = torch.where(there, (got * dy[:, None, :]).sum(dim=2), 0.0)
        per_slot = per_slot * s["weights"].view(-1, 1)
    else:
        dw = torch.where(there, s["dp_rows"][row.clamp_min(0).long()], 0.0)
    drows = torch.zeros((m + 1, h), dtype=s["dy"].dtype, device="cuda")
    drows[at] = per_slot.to(s["dy"].dtype)
    back = torch.where(there[:, :, None], s["dx_rows"].float()[row.clamp_min(0).long()], 0.0)
    return {"drows": drows[:m], "dweights": dw, "dx": back.sum(dim=1).to(s["dy"].dtype)}


def _scale_plain(code):
    """2^(code - 127) from its bits."""
    return torch.where(code > 0, code << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _grid_plain(x):
    """Values on the E2M1 grid over their block's scale, and the scale codes, of x [rows, width]."""
    b = x.view(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(dim=2)
    code = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 2 + 127, 0).clamp(0, 254).to(torch.int32)
    v = (b / _scale_plain(code)[:, :, None]).clamp(-6.0, 6.0)
    a = v.abs()
    r = torch.where(a < 2.0, torch.round(a * 2.0) * 0.5, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0))
    return torch.copysign(r, v), code


def _quantised_plain(x):
    """x rounded to MXFP4 along its last dimension, as the values it then stands for."""
    q, code = _grid_plain(x)
    return (q * _scale_plain(code)[:, :, None]).view(x.shape)


def _codes_plain(x):
    q, code = _grid_plain(x)
    a = q.abs()
    c = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
    return (c | (torch.signbit(q).to(torch.uint8) << 3)).view(x.shape), code.to(torch.uint8)


def _weights_plain(s):
    """The 4-bit weights as numbers [experts, n, k]."""
    c = s["case"]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    table = torch.cat([table, -table])
    b = s["w_codes"]
    v = torch.stack([table[(b & 15).int()], table[(b >> 4).int()]], dim=2).view(b.shape[0], -1, BLOCK)
    scales = s["w_scales"].permute(1, 0, 2).reshape(b.shape[0], -1)[:, : c["k"] // BLOCK].to(torch.int32)
    return (v * _scale_plain(scales)[:, :, None]).view(c["experts"], c["n"], c["k"])


def _columns(x):
    """One expert's rows as columns, filled up with zeros to whole blocks."""
    return torch.nn.functional.pad(x.t(), (0, -x.shape[0] % BLOCK)).contiguous()


def _mxfp4_plain(s):
    c = s["case"]
    xs = s["x"].float()
    x = _quantised_plain(xs).split(s["splits"])
    if not c["step"]:
        return {"y": torch.cat([a @ w.t() for a, w in zip(x, _weights_plain(s))]).to(torch.bfloat16)}
    dys = s["dy"].float()
    dy = _quantised_plain(dys).split(s["splits"])
    w = s["w"].float()
    wr = _quantised_plain(w).view(c["experts"], c["n"], c["k"])
    wc = _quantised_plain(w.view(c["experts"], c["n"], c["k"]).transpose(1, 2).reshape(-1, c["n"])).view(c["experts"], c["k"], c["n"])
    y = torch.cat([a @ b.t() for a, b in zip(x, wr)])
    dx = torch.cat([a @ b.t() for a, b in zip(dy, wc)])
    xc = [_quantised_plain(_columns(a)) if a.shape[0] else None for a in xs.split(s["splits"])]
    dyc = [_quantised_plain(_columns(a)) if a.shape[0] else None for a in dys.split(s["splits"])]
    empty = torch.zeros((c["n"], c["k"]), device="cuda")
    dw = torch.stack([empty if a is None else b @ a.t() for a, b in zip(xc, dyc)])
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ------------------------------------------------------------------------------ the library's calls


def _route_own(s):
    from moe_grouped_scaled_amd import moe_route, moe_route_bwd

    c = s["case"]
    idx, w = moe_route(s["logits"], c["topk"], score=c["score"], renormalize=c["renormalize"])
    out = {"experts": idx, "weights": w}
    if c["grad"]:
        out["dlogits"] = moe_route_bwd(s["logits"], idx, s["dweights"], score=c["score"], renormalize=c["renormalize"])
    return out


def _move_own(s):
    from moe_grouped_scaled_amd import moe_combine, moe_combine_bwd, moe_dispatch, moe_dispatch_bwd

    c = s["case"]
    at_combine = c["weights"] == "combine"
    if not c["grad"]:
        if at_combine:
            row, splits = moe_dispatch(s["idx"], c["experts"], s["x"], s["rows"])
            y = moe_combine(row, s["out_rows"], weights=s["weights"])
            return {"row_of_slot": row, "splits": splits, "rows": s["rows"], "y": y}
        row, splits = moe_dispatch(s["idx"], c["experts"], s["x"], s["rows"], weights=s["weights"],
                                   row_weights=s["row_weights"])
        y = moe_combine(row, s["out_rows"])
        return {"row_of_slot": row, "splits": splits, "rows": s["rows"], "row_weights": s["row_weights"], "y": y}
    row = s["row_of_slot"]
    if at_combine:
        dw = moe_combine_bwd(row, s["dy"], s["dout_rows"], rows=s["out_rows"], weights=s["weights"])
        dx, _ = moe_dispatch_bwd(row, s["dx_rows"])
    else:
        moe_combine_bwd(row, s["dy"], s["dout_rows"])
        dx, dw = moe_dispatch_bwd(row, s["dx_rows"], drow_weights=s["dp_rows"])
    return {"drows": s["dout_rows"], "dweights": dw, "dx": dx}


def _mxfp4_own(s):
    from moe_grouped_scaled_amd import QBuf, QTensor, grouped_gemm_mx, grouped_mx_quantize

    c = s["case"]
    m, n, k, e, splits = c["rows"], c["n"], c["k"], c["experts"], s["splits"]
    bf16 = torch.bfloat16
    y = torch.empty((m, n), dtype=bf16, device="cuda")
    x_row = QTensor("mxfp4", False, splits, k)
    if not c["step"]:
        grouped_mx_quantize("mxfp4", splits, k, s["x"], x_row)
        w = QBuf(s["w_codes"].data_ptr(), s["w_scales"].data_ptr(), None, 0)
        grouped_gemm_mx("fprop", "mxfp4", splits, m, n, k, x_row, w, y)
        return {"y": y}
    x_col = QTensor("mxfp4", True, splits, k)
    w_row, w_col = QTensor("mxfp4", False, [n] * e, k), QTensor("mxfp4", True, [n] * e, k)
    dy_row, dy_col = QTensor("mxfp4", False, splits, n), QTensor("mxfp4", True, splits, n)
    grouped_mx_quantize("mxfp4", splits, k, s["x"], x_row, x_col)
    grouped_mx_quantize("mxfp4", [n] * e, k, s["w"], w_row, w_col)
    grouped_gemm_mx("fprop", "mxfp4", splits, m, n, k, x_row, w_row, y)
    grouped_mx_quantize("mxfp4", splits, n, s["dy"], dy_row, dy_col)
    dx = torch.empty((m, k), dtype=bf16, device="cuda")
    grouped_gemm_mx("dgrad", "mxfp4", splits, m, k, n, dy_row, w_col, dx)
    dw = torch.empty((e, n, k), dtype=bf16, device="cuda")
    grouped_gemm_mx("wgrad", "mxfp4", splits, n, k, m, dy_col, x_col, dw)
    return {"y": y, "dx": dx, "dw": dw}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _route_own, "move": _move_own, "mxfp4": _mxfp4_own}[op](state)
    return {"route": _route_plain, "move": _move_plain, "mxfp4": _mxfp4_plain}[op](state)


# ------------------------------------------------------------------------- the definitions, 64 bits


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    k = c["topk"]
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    rows = np.arange(x.shape[0])[:, None]
    live = np.isfinite(x[rows, order])
    safe = np.where(np.isfinite(x), x, -1e4)
    if c["score"] == "softmax":
        z = np.exp(safe - safe.max(axis=1, keepdims=True)) * np.isfinite(x)
        p = z / np.maximum(z.sum(axis=1, keepdims=True), 1e-300)
    else:
        p = np.isfinite(x) / (1.0 + np.exp(np.minimum(-safe, 700.0)))
    w = p[rows, order] * live
    norm = np.maximum(w.sum(axis=1, keepdims=True), 1e-300) if c["renormalize"] else 1.0
    out = {"experts": None, "weights": torch.from_numpy(w / norm)}
    if c["grad"]:
        # chain rule through w_j / sum_i w_i, then through the score
        gw = s["dweights"].double().cpu().numpy() * live
        if c["renormalize"]:
            gw = (gw - (gw * w / norm).sum(axis=1, keepdims=True)) / norm * live
        gp = np.zeros_like(p)
        np.put_along_axis(gp, order, gw, axis=1)
        if c["score"] == "softmax":
            dx = p * (gp - (p * gp).sum(axis=1, keepdims=True))
        else:
            dx = gp * p * (1.0 - p)
        out["dlogits"] = torch.from_numpy(dx)
    return out


def _exact_move(s):
    c = s["case"]
    row = s["row_of_slot"].long()
    t, k, h = c["tokens"], c["topk"], c["hidden"]
    w = s["weights"].double() if c["weights"] == "combine" else torch.ones((t, k), dtype=torch.float64, device="cuda")
    live = (row >= 0).double()
    safe = row.clamp_min(0)

    def per_token(values):
        y = torch.zeros((t, h), dtype=torch.float64, device="cuda")
        for j in range(k):
            y += values[safe[:, j]].double() * (w[:, j] * live[:, j])[:, None]
        return y

    if not c["grad"]:
        return {"row_of_slot": None, "splits": None, "rows": None, "row_weights": None, "y": per_token(s["out_rows"])}
    drows = torch.zeros((t * k, h), dtype=torch.float64, device="cuda")
    dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        on = live[:, j] > 0
        drows[row[on, j]] = s["dy"][on].double() * w[on, j][:, None]
        if c["weights"] == "combine":
            dw[on, j] = (s["out_rows"][row[on, j]].double() * s["dy"][on].double()).sum(dim=1)
        else:
            dw[on, j] = s["dp_rows"][row[on, j]].double()
    w = torch.ones_like(w)
    return {"drows": drows, "dweights": dw, "dx": per_token(s["dx_rows"])}


def _exact_grid(x):
    """MXFP4 of x along its last dimension: the nearest E2M1 value by counting the midpoints below."""
    b = x.double().reshape(x.shape[0], -1, BLOCK)
    top = b.abs().amax(dim=2, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2.0)
    a = (b / scale).abs()
    q = torch.zeros_like(a)
    for mid, up, gap in ((0.25, 0, 0.5), (0.75, 1, 0.5), (1.25, 0, 0.5), (1.75, 1, 0.5), (2.5, 0, 1.0), (3.5, 1, 1.0), (5.0, 0, 2.0)):
        q += gap * ((a >= mid) if up else (a > mid)).double()
    return (torch.where(b < 0, -q, q) * scale).reshape(x.shape)


def _exact_mxfp4(s):
    c = s["case"]
    e, n, k = c["experts"], c["n"], c["k"]
    y, dx, dw, lo = [], [], [], 0
    for i, m in enumerate(s["splits"]):
        x = s["x"][lo : lo + m]
        if not c["step"]:
            codes = s["w_codes"][i * n : (i + 1) * n].long()
            codes = torch.stack([codes & 15, codes >> 4], dim=2).view(n, k)
            mag = codes & 7
            v = torch.where(mag < 2, mag.double() * 0.5, (1.0 + 0.5 * (mag & 1).double()) * torch.exp2((mag >> 1).double() - 1.0))
            sc = s["w_scales"][:, i * n : (i + 1) * n].permute(1, 0, 2).reshape(n, -1)[:, : k // BLOCK].double()
            w = torch.where(codes > 7, -v, v) * torch.exp2(sc - 127.0).repeat_interleave(BLOCK, dim=1)
            y.append(_exact_grid(x) @ w.t() if m else torch.zeros((0, n), dtype=torch.float64, device="cuda"))
        else:
            w, dy = s["w"][i * n : (i + 1) * n], s["dy"][lo : lo + m]
            wide = torch.zeros((-(-m // BLOCK) * BLOCK, k + n), dtype=torch.float64, device="cuda")
            wide[:m, :k], wide[:m, k:] = x.double(), dy.double()
            if m:
                y.append(_exact_grid(x) @ _exact_grid(w).t())
                dx.append(_exact_grid(dy) @ _exact_grid(w.t().contiguous()).t())
                both = _exact_grid(wide.t().contiguous())
                dw.append(both[k:] @ both[:k].t())
            else:
                dw.append(torch.zeros((n, k), dtype=torch.float64, device="cuda"))
        lo += m
    out = {"y": torch.cat(y)}
    if c["step"]:
        out.update(dx=torch.cat(dx), dw=torch.stack(dw))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "move": _exact_move, "mxfp4": _exact_mxfp4}[case["op"]](s)
