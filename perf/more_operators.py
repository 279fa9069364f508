"""Cases of the unquantized and the 4-bit expert block and of gradient clipping, in a plain form and as the library's calls.

Three operators next to the quantized expert MLP:
  gated   the gated feed-forward block of every expert in BF16: gate and up projection, activation, product and
          per-row scale, then the second linear; forward, or forward and backward (`GatedMLP`)
  w4      products of few rows with weights held as 4-bit integers with a scale and a zero point per group of
          32, 64 or 128, as one linear (`grouped_gemm_w4`) or as the whole gated block (`W4GatedMLP`)
  clip    the global norm of many gradients, and the gradients scaled down to a largest norm (`clip_grad_norm`)

With `own` false `run` computes them in elementary torch operations; with `own` true it makes the calls
a user of the library makes.  `exact` computes the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

LIMIT, ALPHA, BETA = 7.0, 1.0, 0.0  # of the clamped SwiGLU
EPS = 1e-6  # added to the norm before dividing


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token of one request through a dense (or shared) block: reads the weights once
        dict(name="gated_token", op="gated", rows=1, experts=1, hidden=4096, ffn=4096, kind="swiglu", skew=0.0,
             probs=False, bias=False, grad=False),
        # a decoding step of 16 requests, two of 16 experts each, at the wide layer's sizes
        dict(name="gated_decode", op="gated", rows=32, experts=16, hidden=7168, ffn=2048, kind="swiglu", skew=0.0,
             probs=True, bias=False, grad=False),
        # a prompt batch over 16 experts, some far more popular than others, two empty
        dict(name="gated_prefill", op="gated", rows=8192, experts=16, hidden=4096, ffn=4096, kind="clamped_swiglu",
             skew=1.2, probs=True, bias=True, grad=False),
        # a training step of the dense block
        dict(name="gated_train", op="gated", rows=8192, experts=1, hidden=4096, ffn=4096, kind="swiglu", skew=0.0,
             probs=False, bias=False, grad=True),
        # a training step of the 32-expert layer on a skewed batch
        dict(name="gated_train_experts", op="gated", rows=16384, experts=32, hidden=7168, ffn=2048, kind="swiglu",
             skew=1.2, probs=False, bias=False, grad=True),
        # a small, ragged batch at widths that no tile divides
        dict(name="gated_train_odd", op="gated", rows=1021, experts=5, hidden=1000, ffn=1096, kind="glu", skew=0.7,
             probs=False, bias=False, grad=True),
        # one token through one linear: latency
        dict(name="w4_token", op="w4", rows=1, experts=1, n=4096, k=4096, group=128, zeros=True, skew=0.0, block=False,
             probs=False, bias=False),
        # a decoding step of 16 requests, two of 16 experts each: the block's 4-bit weights once
        dict(name="w4_decode", op="w4", rows=32, experts=16, n=4096, k=4096, group=128, zeros=True, skew=0.0,
             block=True, probs=True, bias=False),
        # ragged rows of a small batch, symmetric weights in groups of 32, a width that no tile divides, bias
        dict(name="w4_rows_odd", op="w4", rows=61, experts=4, n=7160, k=2080, group=32, zeros=False, skew=0.7,
             block=False, probs=False, bias=True),
        # a few layers' small tensors (biases, router weights, norms): latency
        dict(name="clip_small", op="clip", tensors=12, elements=300000, spread=6.0, dtype="mixed", out="same"),
        # the gradients of a deep stack: hundreds of tensors of very different sizes, BF16 and FP32
        dict(name="clip_many", op="clip", tensors=400, elements=400000000, spread=8.0, dtype="mixed", out="same"),
        # the FP32 weight gradients of the 16-expert block, clipped into BF16 copies
        dict(name="clip_experts", op="clip", tensors=2, elements=16 * 12288 * 4096, spread=2.0, dtype="f32", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "gated", "w4", "w4", "clip"))
    if op == "clip":
        tensors = _log(rng, 1, 400)
        return dict(op=op, tensors=tensors, elements=max(tensors, _log(rng, 1000, 16 * 12288 * 4096)),
                    spread=rng.choice((1.0, 3.0, 8.0)), dtype=rng.choice(("bf16", "f32", "mixed")),
                    out=rng.choice(("same", "bf16")))
    experts = _log(rng, 1, 32)
    skew = rng.choice((0.0, 0.7, 1.2))
    if op == "gated":
        hidden, ffn = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 512)
        while experts * hidden * ffn > 32 * 7168 * 2048:
            experts = max(1, experts // 2)
        grad = rng.random() < 0.5
        rows = _log(rng, 1, min(32768, 16384 * 7168 * 2048 // (hidden * ffn)))
        return dict(op=op, rows=rows, experts=experts, hidden=hidden, ffn=ffn, skew=skew, grad=grad,
                    kind=rng.choice(("swiglu", "clamped_swiglu", "glu")), probs=not grad and rng.random() < 0.5,
                    bias=not grad and rng.random() < 0.5)
    group = rng.choice((32, 64, 128))
    block = rng.random() < 0.5
    k = group * _log(rng, max(1, 128 // group), 7168 // group)
    n = group * _log(rng, max(1, 128 // group), 7168 // group) if block else _log(rng, 100, 7168)
    return dict(op=op, rows=_log(rng, 1, 512), experts=experts, n=n, k=k, group=group, zeros=rng.random() < 0.5,
                skew=skew, block=block, probs=block and rng.random() < 0.5, bias=rng.random() < 0.5)


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


def sizes_of(case):
    """Elements and type of each gradient: the largest exp(spread) times the smallest, shuffled.  They go by the
    case alone."""
    n, total = case["tensors"], case["elements"]
    r = np.random.RandomState(n * 7919 + total % 100003)
    w = np.exp(np.linspace(0.0, case["spread"], n))[r.permutation(n)] if n > 1 else np.ones(1)
    sizes = np.maximum(1, (w / w.sum() * total).astype(np.int64))
    kinds = {"bf16": ["bf16"] * n, "f32": ["f32"] * n,
             "mixed": ["f32" if v else "bf16" for v in r.randint(0, 2, n)]}[case["dtype"]]
    return [(int(s), k) for s, k in zip(sizes, kinds)]


def work(case):
    if case["op"] == "clip":
        # every gradient in and every scaled gradient out; a multiplication for the norm and one for the scale
        b = 4
        for s, k in sizes_of(case):
            size = 2 if k == "bf16" else 4
            b += s * (size + (2 if case["out"] == "bf16" else size))
        return {"bytes": b, "flops": 3 * case["elements"]}
    m, e = case["rows"], case["experts"]
    hit = sum(1 for v in splits_of(case) if v)
    if case["op"] == "gated":
        h, f = case["hidden"], case["ffn"]
        b = 2 * (2 * m * h) + 2 * hit * 3 * f * h + (4 * m if case["probs"] else 0)
        if not case["grad"]:
            return {"bytes": b, "flops": 6 * m * h * f}
        # the outputs' gradient in, the inputs' and every weight's gradient out
        return {"bytes": b + 2 * (2 * m * h) + 2 * e * 3 * f * h, "flops": 18 * m * h * f}
    n, k, g = case["n"], case["k"], case["group"]
    per_group = g / 2 + 2 + (1 if case["zeros"] else 0)
    groups = (2 * n * k + k * n if case["block"] else n * k) // g
    out = k if case["block"] else n
    return {"bytes": int(2 * m * k + hit * groups * per_group + 2 * m * out + (4 * m if case["probs"] else 0)),
            "flops": 2 * m * groups * g}


# ----------------------------------------------------------------------------------------- inputs


def _w4_weights(g, e, n, k, case):
    """Random 4-bit weights [e, n, k] as a checkpoint holds them: codes two a byte (the even element in the low
    half), scales in BF16, zero points as whole numbers (8 where there are none)."""
    codes = torch.randint(0, 256, (e, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((e, n, k // case["group"]), generator=g, device="cuda") * 0.006 + 0.001).to(torch.bfloat16)
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(0, 16, scales.shape, generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales, zeros


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = {"case": case}

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    if case["op"] == "clip":
        # gradients live in one buffer for each type, each from a multiple of 64 elements on
        d["flat"], d["grads"], d["out"] = [], [], []
        types = {"bf16": torch.bfloat16, "f32": torch.float32}
        sizes = sizes_of(case)
        for name, dt in types.items():
            mine = [(i, s) for i, (s, k) in enumerate(sizes) if k == name]
            total = sum(-(-s // 64) * 64 for _, s in mine)
            if not total:
                continue
            buf = torch.zeros(total, dtype=dt, device="cuda")
            out = torch.zeros(total, dtype=torch.bfloat16 if case["out"] == "bf16" else dt, device="cuda")
            lo = 0
            for i, s in mine:
                # layers differ in the size of their gradients
                buf[lo : lo + s] = normal(s, std=10.0 ** -(i % 4), dtype=dt)
                d["grads"].append(buf[lo : lo + s])
                d["out"].append(out[lo : lo + s])
                lo += -(-s // 64) * 64
            d["flat"].append((buf, out))
        d["max_norm"] = 1.0
        return d
    m, e = case["rows"], case["experts"]
    d["splits"] = splits_of(case)
    d["probs"] = torch.rand(m, generator=g, device="cuda") if case["probs"] else None
    if case["op"] == "gated":
        h, f = case["hidden"], case["ffn"]
        d["x"] = normal(m, h)
        d["w1"], d["w2"] = normal(e, 2 * f, h, std=0.02), normal(e, h, f, std=0.02)
        d["b1"] = normal(e, 2 * f, std=0.02) if case["bias"] else None
        d["b2"] = normal(e, h, std=0.02) if case["bias"] else None
        if case["grad"]:
            d["dy"] = normal(m, h)
        if own:
            from moe_grouped_scaled_amd import GatedMLP

            need = case["grad"]
            d["mlp"] = GatedMLP(case["kind"], d["w1"], d["w2"], b1=d["b1"], b2=d["b2"], limit=LIMIT, alpha=ALPHA,
                                beta=BETA, grad_x1=need, grad_probs=False, grad_fc1=need, grad_fc2=need,
                                dw_dtype=torch.bfloat16)
        return d
    n, k = case["n"], case["k"]
    d["x"] = normal(m, k)
    if case["block"]:
        d["w1"], d["w2"] = _w4_weights(g, e, 2 * n, k, case), _w4_weights(g, e, k, n, case)
        d["b1"] = normal(e, 2 * n, std=0.02) if case["bias"] else None
        d["b2"] = normal(e, k, std=0.02) if case["bias"] else None
    else:
        d["w1"] = _w4_weights(g, e, n, k, case)
        d["b1"] = normal(e, n, std=0.02) if case["bias"] else None
    if own:
        from moe_grouped_scaled_amd import W4GatedMLP, w4_pack

        d["w1_packed"] = w4_pack(*d["w1"])
        if case["block"]:
            d["mlp"] = W4GatedMLP("swiglu", d["w1_packed"], w4_pack(*d["w2"]), b1=d["b1"], b2=d["b2"])
    return d


# ------------------------------------------------------------------------------------- plain forms


def _act_plain(kind, gate, up):
    """The activation's value and its derivatives by gate and up, in elementary operations."""
    if kind == "glu":
        s = 1.0 / (1.0 + torch.exp(-gate))
        return s * up, s * (1.0 - s) * up, s
    if kind == "swiglu":
        s = 1.0 / (1.0 + torch.exp(-gate))
        return gate * s * up, up * s * (1.0 + gate * (1.0 - s)), gate * s
    g, u = gate.clamp_max(LIMIT), up.clamp(-LIMIT, LIMIT)
    s = 1.0 / (1.0 + torch.exp(-ALPHA * g))
    dg = torch.where(gate <= LIMIT, (u + BETA) * s * (1.0 + ALPHA * g * (1.0 - s)), 0.0)
    du = torch.where((up >= -LIMIT) & (up <= LIMIT), g * s, 0.0)
    return g * s * (u + BETA), dg, du


def _gated_plain(s):
    c = s["case"]
    f = c["ffn"]
    y, dx, dw1, dw2, lo = [], [], [], [], 0
    for i, m in enumerate(s["splits"]):
        if not m:
            if c["grad"]:
                dw1.append(torch.zeros_like(s["w1"][i]))
                dw2.append(torch.zeros_like(s["w2"][i]))
            continue
        x, w1, w2 = s["x"][lo : lo + m].float(), s["w1"][i].float(), s["w2"][i].float()
        pre = x @ w1.t()
        if c["bias"]:
            pre = pre + s["b1"][i].float()
        a, dg, du = _act_plain(c["kind"], pre[:, :f], pre[:, f:])
        if c["probs"]:
            a = a * s["probs"][lo : lo + m, None]
        out = a @ w2.t()
        if c["bias"]:
            out = out + s["b2"][i].float()
        y.append(out.to(torch.bfloat16))
        if c["grad"]:
            dy = s["dy"][lo : lo + m].float()
            da = dy @ w2
            dpre = torch.cat([da * dg, da * du], dim=1)
            dx.append((dpre @ w1).to(torch.bfloat16))
            dw1.append((dpre.t() @ x).to(torch.bfloat16))
            dw2.append((dy.t() @ a).to(torch.bfloat16))
        lo += m
    res = {"y": torch.cat(y)}
    if c["grad"]:
        res.update(dx=torch.cat(dx), dw1=torch.stack(dw1), dw2=torch.stack(dw2))
    return res


def _w4_values(w, i, group):
    codes, scales, zeros = w
    q = torch.stack([codes[i] & 15, codes[i] >> 4], dim=2).view(codes.shape[1], -1, group).float()
    z = zeros[i][:, :, None].float() if zeros is not None else 8.0
    return ((q - z) * scales[i][:, :, None].float()).view(codes.shape[1], -1)


def _w4_plain(s):
    c = s["case"]
    y, lo = [], 0
    for i, m in enumerate(s["splits"]):
        if not m:
            continue
        v = s["x"][lo : lo + m].float() @ _w4_values(s["w1"], i, c["group"]).t()
        if c["bias"]:
            v = v + s["b1"][i].float()
        if c["block"]:
            v, _, _ = _act_plain("swiglu", v[:, : c["n"]], v[:, c["n"] :])
            if c["probs"]:
                v = v * s["probs"][lo : lo + m, None]
            v = v @ _w4_values(s["w2"], i, c["group"]).t()
            if c["bias"]:
                v = v + s["b2"][i].float()
        y.append(v.to(torch.bfloat16))
        lo += m
    return {"y": torch.cat(y)}


def _clip_plain(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        total = total + (t.double() * t.double()).sum()
    norm = total.sqrt()
    scale = (s["max_norm"] / (norm + EPS)).clamp_max(1.0).float()
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * scale)
    return {"norm": norm.float(), "grads": [o for _, o in s["flat"]]}


# ------------------------------------------------------------------------------ the library's calls


def _gated_own(s):
    y = s["mlp"].forward(s["x"], s["probs"], s["splits"])
    if not s["case"]["grad"]:
        return {"y": y}
    g = s["mlp"].backward(s["dy"])
    return {"y": y, "dx": g["dx1"], "dw1": g["dw1"], "dw2": g["dw2"]}


def _w4_own(s):
    if s["case"]["block"]:
        return {"y": s["mlp"].forward(s["x"], s["probs"], s["splits"])}
    from moe_grouped_scaled_amd import grouped_gemm_w4

    return {"y": grouped_gemm_w4(s["splits"], s["x"], s["w1_packed"], bias=s["b1"])}


def _clip_own(s):
    from moe_grouped_scaled_amd import clip_grad_norm

    norm = clip_grad_norm(s["grads"], s["max_norm"], eps=EPS, out=s["out"])
    return {"norm": norm, "grads": [o for _, o in s["flat"]]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gated": _gated_own, "w4": _w4_own, "clip": _clip_own}[op](state)
    return {"gated": _gated_plain, "w4": _w4_plain, "clip": _clip_plain}[op](state)


# ------------------------------------------------------------------------- the definitions, 64 bits


def _exact_act(kind, g, u):
    """(value, by gate, by up) from the definition, written with the hyperbolic tangent."""
    if kind == "clamped_swiglu":
        gc, uc = torch.minimum(g, g.new_tensor(LIMIT)), torch.maximum(torch.minimum(u, u.new_tensor(LIMIT)), u.new_tensor(-LIMIT))
        s = 0.5 + 0.5 * torch.tanh(0.5 * ALPHA * gc)
        ds = ALPHA * s * (1.0 - s)
        return gc * s * (uc + BETA), (s + gc * ds) * (uc + BETA) * (g <= LIMIT), gc * s * (u.abs() <= LIMIT)
    s = 0.5 + 0.5 * torch.tanh(0.5 * g)
    ds = s * (1.0 - s)
    if kind == "glu":
        return s * u, ds * u, s
    return g * s * u, (s + g * ds) * u, g * s


def _exact_gated(s):
    c = s["case"]
    f, h, e, m = c["ffn"], c["hidden"], c["experts"], c["rows"]
    wide = dict(dtype=torch.float64, device="cuda")
    out = {"y": torch.zeros((m, h), **wide)}
    if c["grad"]:
        out.update(dx=torch.zeros((m, h), **wide), dw1=torch.zeros((e, 2 * f, h), **wide), dw2=torch.zeros((e, h, f), **wide))
    ends = np.cumsum(s["splits"])
    for i in range(e):
        at = slice(int(ends[i] - s["splits"][i]), int(ends[i]))
        if at.start == at.stop:
            continue
        x, wg, wu, w2 = s["x"][at].double(), s["w1"][i, :f].double(), s["w1"][i, f:].double(), s["w2"][i].double()
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        if s["b1"] is not None:
            g, u = g + s["b1"][i, :f].double(), u + s["b1"][i, f:].double()
        a, by_g, by_u = _exact_act(c["kind"], g, u)
        p = 1.0 if s["probs"] is None else s["probs"][at].double()[:, None]
        out["y"][at] = torch.mm(a * p, w2.t()) + (0.0 if s["b2"] is None else s["b2"][i].double())
        if c["grad"]:
            dy = s["dy"][at].double()
            da = torch.mm(dy, w2) * p
            dg, du = da * by_g, da * by_u
            out["dx"][at] = torch.mm(dg, wg) + torch.mm(du, wu)
            out["dw1"][i, :f], out["dw1"][i, f:] = torch.mm(dg.t(), x), torch.mm(du.t(), x)
            out["dw2"][i] = torch.mm(dy.t(), a * p)
    return out


def _exact_w4_product(x, w, i, group, bias):
    """x times the transposed weights of one expert: per group, scale * (x . codes - zero * sum of x)."""
    codes, scales, zeros = w
    n, k = codes.shape[1], codes.shape[2] * 2
    y = torch.zeros((x.shape[0], n), dtype=torch.float64, device=x.device)
    q = torch.empty((n, k), dtype=torch.float64, device=x.device)
    q[:, 0::2] = torch.remainder(codes[i].double(), 16.0)
    q[:, 1::2] = torch.floor(codes[i].double() / 16.0)
    for j in range(k // group):
        xs = x[:, j * group : (j + 1) * group]
        z = torch.full((n,), 8.0, dtype=torch.float64, device=x.device) if zeros is None else zeros[i, :, j].double()
        dot = torch.mm(xs, q[:, j * group : (j + 1) * group].t()) - xs.sum(dim=1)[:, None] * z
        y += dot * scales[i, :, j].double()
    return y if bias is None else y + bias[i].double()


def _exact_w4(s):
    c = s["case"]
    ends = np.cumsum(s["splits"])
    y = torch.zeros((c["rows"], c["k"] if c["block"] else c["n"]), dtype=torch.float64, device="cuda")
    for i in range(c["experts"]):
        at = slice(int(ends[i] - s["splits"][i]), int(ends[i]))
        if at.start == at.stop:
            continue
        v = _exact_w4_product(s["x"][at].double(), s["w1"], i, c["group"], s["b1"])
        if c["block"]:
            v = _exact_act("swiglu", v[:, : c["n"]], v[:, c["n"] :])[0]
            if s["probs"] is not None:
                v = v * s["probs"][at].double()[:, None]
            v = _exact_w4_product(v, s["w2"], i, c["group"], s["b2"])
        y[at] = v
    return {"y": y}


def _exact_clip(s):
    # sums of 2^12 elements, their sums over 2^24, and those on the host
    parts = []
    for t in s["grads"]:
        for lo in range(0, t.numel(), 1 << 24):
            v = t[lo : lo + (1 << 24)].double()
            v = torch.nn.functional.pad(v * v, (0, -v.numel() % (1 << 12))).view(-1, 1 << 12).sum(dim=1)
            parts.append(v.sum())
    norm = math.sqrt(math.fsum(torch.stack(parts).cpu().tolist()))
    scale = min(1.0, s["max_norm"] / (norm + EPS))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [t.double() * scale for t, _ in s["flat"]]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "w4": _exact_w4, "clip": _exact_clip}[case["op"]](s)
