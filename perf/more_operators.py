"""An expert layer around layer norm and in 8-bit integers: what is measured, and the operators' plain forms.

Three operators: tokens sorted by expert and back, with the choices' weights
applied (and the gradients of both ways); layer norm with the residual's
addition (and its gradients); and the product of 8-bit integers with a scale
for each token and channel, dense or grouped by expert, from values that are
quantised as they come or from the layer norm's own 8-bit output.

``run`` computes a case in elementary torch operations, in 32 bits, or with
``own`` set by the library's kernels.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
MIN_AMAX = 2.0 ** -100
TOP_CODE = 127.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # One step of decoding for 16 sequences: sorted by expert, handed out, and put together again.
        {"name": "route_decode", "op": "route", "tokens": 16, "top": 4, "experts": 32, "held": 32, "cols": 4096,
         "type": "bf16"},
        # A prefill where this GPU holds half of the experts: the other choices get no row.
        {"name": "route_prefill", "op": "route", "tokens": 8192, "top": 8, "experts": 128, "held": 64, "cols": 2048,
         "type": "bf16"},
        # A training step of the routing around the experts: both ways, and the gradients of both.
        {"name": "route_train_bf16", "op": "route_train", "tokens": 8192, "top": 2, "experts": 8, "held": 8,
         "cols": 4096, "type": "bf16"},
        # The same in fp32 at odd sizes, a small layer.
        {"name": "route_train_f32_odd", "op": "route_train", "tokens": 777, "top": 3, "experts": 12, "held": 12,
         "cols": 257, "type": "f32"},
        # A training step of the norm: forward, then the gradients.
        {"name": "norm_train_bf16", "op": "norm_train", "rows": 8192, "cols": 4096, "type": "bf16"},
        # The same in fp32 at an odd width (no row but the first is 16-byte aligned).
        {"name": "norm_train_f32_odd", "op": "norm_train", "rows": 1000, "cols": 777, "type": "f32"},
        # A linear layer while decoding 16 sequences: norm, 8-bit rows, product.
        {"name": "linear_decode", "op": "linear", "m": 16, "n": 8192, "k": 8192, "weights": "nk", "norm": True},
        # Odd sizes in every direction (rows off 16 bytes), values quantised as they come.
        {"name": "linear_odd", "op": "linear", "m": 1000, "n": 3000, "k": 777, "weights": "nk", "norm": False},
        # Weights stored the other way.
        {"name": "linear_kn", "op": "linear", "m": 2048, "n": 4096, "k": 4096, "weights": "kn", "norm": False},
        # A large prefill: norm and product.
        {"name": "linear_large", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "weights": "nk", "norm": True},
        # 16 tokens, 4 experts each of 32: every expert's weights are read for a few rows.
        {"name": "experts_decode", "op": "experts", "rows": 64, "groups": 32, "n": 4096, "k": 4096},
        # A prefill through 16 experts with uneven loads.
        {"name": "experts_prefill", "op": "experts", "rows": 8192, "groups": 16, "n": 4096, "k": 4096},
    ]


def _spread(rng, low, high, multiple=1):
    """A size between low and high, even over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, v // multiple * multiple))


def draw(rng):
    op = rng.choice(["route", "route_train", "norm_train", "linear", "experts"])
    multiple = rng.choice([1, 8, 128])
    if op in ("route", "route_train"):
        experts = _spread(rng, 2, 256)
        return {"op": op, "tokens": _spread(rng, 1, 8192), "top": rng.randint(1, min(8 if op == "route" else 4, experts)),
                "experts": experts, "held": experts if rng.random() < 0.5 else rng.randint(1, experts),
                "cols": _spread(rng, 64, 4096 if op == "route_train" else 2048, multiple),
                "type": rng.choice(["f32", "bf16"])}
    if op == "norm_train":
        return {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 128, 8192, multiple),
                "type": rng.choice(["f32", "bf16"])}
    if op == "linear":
        return {"op": op, "m": _spread(rng, 1, 8192), "n": _spread(rng, 128, 8192, multiple),
                "k": _spread(rng, 128, 8192, multiple), "weights": rng.choice(["nk", "kn"]),
                "norm": rng.random() < 0.5}
    return {"op": op, "rows": _spread(rng, 1, 8192), "groups": _spread(rng, 1, 64),
            "n": _spread(rng, 128, 4096, multiple), "k": _spread(rng, 128, 4096, multiple)}


def _padded_rows(rows, cols, dtype):
    """rows x cols whose rows start on 16 bytes, as the library's own allocations of codes do."""
    per = 16 // dtype.itemsize
    return torch.empty((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


def _sizes(rows, groups, seed):
    """How many rows each group has: uneven, as a router leaves them, some of them none."""
    g = torch.Generator().manual_seed(seed + 77)
    share = torch.softmax(torch.randn(groups, generator=g) * 0.7, 0)
    return torch.bincount(torch.multinomial(share, rows, replacement=True, generator=g), minlength=groups).tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * scale

    def activations(rows, cols):
        """Normal values with a few channels much larger than the rest, as a residual stream has."""
        channel = torch.ones(cols, device="cuda")
        channel[torch.rand(cols, device="cuda", generator=gen) < 0.01] = 20.0
        return normal(rows, cols) * channel

    def kept(t, dtype):
        out = _padded_rows(*t.shape, dtype)
        out.copy_(t)
        return out

    def weight_codes(rows, cols):
        return (normal(rows, cols, scale=40.0).round_().clamp_(-TOP_CODE, TOP_CODE)).to(torch.int8)

    def channel_scales(*shape, depth):
        """Scales of weights of about depth ** -0.5, a channel's each."""
        return (0.5 + torch.rand(*shape, device="cuda", generator=gen)) * (depth ** -0.5 / 40.0)

    s = dict(case)
    op = case["op"]
    if op in ("route", "route_train"):
        tokens, cols, dtype = case["tokens"], case["cols"], TYPES[case["type"]]
        # Some experts are liked more than others; a token's choices are the largest of its logits.
        logits = normal(tokens, case["experts"]) + normal(case["experts"], scale=0.7)
        value, expert = logits.topk(case["top"], dim=1)
        s["weights"] = value.softmax(dim=1)
        # Experts that other GPUs hold are no group here.
        s["expert"] = torch.where(expert < case["held"], expert, torch.full_like(expert, -1))
        s["x"] = normal(tokens, cols).to(dtype)
        s["residual"] = activations(tokens, cols).to(dtype)
        s["y"] = normal(tokens * case["top"], cols, scale=0.5).to(dtype)
        if op == "route_train":
            s["dout"] = normal(tokens, cols, scale=0.1).to(dtype)
            s["drows"] = normal(tokens * case["top"], cols, scale=0.1).to(dtype)
    elif op == "norm_train":
        rows, cols, dtype = case["rows"], case["cols"], TYPES[case["type"]]
        s["x"] = normal(rows, cols, scale=0.5).to(dtype)
        s["residual"] = (activations(rows, cols) + normal(rows, 1, scale=0.5)).to(dtype)
        s["weight"] = (1.0 + normal(cols, scale=0.1)).to(dtype)
        s["bias"] = normal(cols, scale=0.1).to(dtype)
        s["dy"] = normal(rows, cols, scale=0.1).to(dtype)
        s["dsum"] = normal(rows, cols, scale=0.1).to(dtype)
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"] = activations(m, k).to(torch.bfloat16)
        if case["norm"]:
            s["residual"] = normal(m, k).to(torch.bfloat16)
            s["weight"] = (1.0 + normal(k, scale=0.1)).to(torch.bfloat16)
            s["norm_bias"] = normal(k, scale=0.1).to(torch.bfloat16)
        w = weight_codes(n, k) if case["weights"] == "nk" else weight_codes(k, n)
        s["b"] = kept(w, torch.int8)
        s["b_scales"] = channel_scales(n, depth=k)
        s["bias"] = normal(n, scale=0.1)
    else:
        rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        s["sizes"] = _sizes(rows, groups, seed)
        s["ends"] = torch.tensor(s["sizes"]).cumsum(0).to(device="cuda", dtype=torch.int32)
        s["x"] = activations(rows, k).to(torch.bfloat16)
        s["b"] = torch.empty((groups, n, -(-k // 16) * 16), dtype=torch.int8, device="cuda")[:, :, :k]
        for g in range(groups):
            s["b"][g].copy_(weight_codes(n, k))
        s["b_scales"] = channel_scales(groups, n, depth=k)
    return s


def _plan(expert, held):
    """(order, place, ends): choices in the order of their experts, the row of each choice, where experts end."""
    flat = expert.flatten()
    key = torch.where(flat < 0, torch.full_like(flat, held), flat)
    order = key.argsort(stable=True)
    sizes = (key[:, None] == torch.arange(held, device=key.device)).sum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=key.device)
    ends = sizes.cumsum(0)
    place = torch.where(flat < 0, torch.full_like(flat, -1), place)
    order = torch.where(torch.arange(order.numel(), device=key.device) < ends[-1], order, torch.full_like(order, -1))
    return order.int(), place.int().view(expert.shape), ends.int()


def _handed_out(x, order, top):
    rows = x[order.clamp_min(0).long() // top]
    return torch.where((order >= 0)[:, None], rows, torch.zeros_like(rows))


def _of_choices(rows, place):
    """tokens x top x cols in 32 bits, zero where a choice has no row."""
    each = rows[place.clamp_min(0).long()].float()
    return torch.where((place >= 0)[:, :, None], each, torch.zeros_like(each))


def _layer_norm(x, residual, weight, bias):
    """(sum as it is kept, its norm before the last rounding) in 32 bits."""
    total = (x.float() + residual.float()).to(x.dtype)
    t = total.float()
    c = t - t.mean(dim=1, keepdim=True)
    r = torch.rsqrt(c.square().mean(dim=1, keepdim=True) + EPS)
    return total, c * r * weight.float() + bias.float()


def _layer_norm_grads(dy, total, weight, dsum):
    t, d = total.float(), dy.float()
    c = t - t.mean(dim=1, keepdim=True)
    r = torch.rsqrt(c.square().mean(dim=1, keepdim=True) + EPS)
    n, g = c * r, d * weight.float()
    dx = r * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True)) + dsum.float()
    return dx, (d.double() * n.double()).sum(dim=0), d.double().sum(dim=0)


def _row_codes(v):
    """Whole numbers (as 32-bit values) and scales of rows."""
    amax = v.abs().amax(dim=1).clamp_min(MIN_AMAX)
    return (v * (TOP_CODE / amax)[:, None]).round(), amax / TOP_CODE


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "route":
        order, place, ends = _plan(state["expert"], state["held"])
        rows = _handed_out(state["x"], order, state["top"])
        out = state["residual"].float() + (_of_choices(state["y"], place) * state["weights"][:, :, None]).sum(1)
        return {"order": order, "place": place, "ends": ends, "rows": rows, "out": out.to(rows.dtype)}
    if op == "route_train":
        x, w = state["x"], state["weights"]
        order, place, ends = _plan(state["expert"], state["held"])
        rows = _handed_out(x, order, state["top"])
        each = _of_choices(state["y"], place)
        out = state["residual"].float() + (each * w[:, :, None]).sum(1)
        dw = (each * state["dout"].float()[:, None, :]).sum(2)
        share = w.flatten()[order.clamp_min(0).long()]
        dy = _handed_out(state["dout"], order, state["top"]).float() * share[:, None]
        dx = _of_choices(state["drows"], place).sum(1) + state["dout"].float()
        return {"order": order, "place": place, "ends": ends, "rows": rows, "out": out.to(x.dtype),
                "dy": dy.to(x.dtype), "dweights": dw, "dx": dx.to(x.dtype)}
    if op == "norm_train":
        x, w = state["x"], state["weight"]
        total, y = _layer_norm(x, state["residual"], w, state["bias"])
        dx, dw, db = _layer_norm_grads(state["dy"], total, w, state["dsum"])
        return {"sum": total, "y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.float(), "db": db.float()}
    if op == "linear":
        got = {}
        v = state["x"].float()
        if state["norm"]:
            got["sum"], v = _layer_norm(state["x"], state["residual"], state["weight"], state["norm_bias"])
        code, got["scales"] = _row_codes(v)
        b = state["b"].float()
        y = code @ (b.t() if state["weights"] == "nk" else b)
        got["y"] = (y * got["scales"][:, None] * state["b_scales"] + state["bias"]).to(torch.bfloat16)
        return got
    code, scales = _row_codes(state["x"].float())
    y = torch.cat([p @ q.float().t() * s for p, q, s in zip(code.split(state["sizes"]), state["b"], state["b_scales"])])
    return {"scales": scales, "y": (y * scales[:, None]).to(torch.bfloat16)}


def _run_own(state):
    import tiled_gemm_f32_amd as tg
    op = state["op"]
    if op in ("route", "route_train"):
        w = state["weights"]
        order, place, ends = tg.expert_plan(state["expert"], state["held"])
        rows = tg.dispatch(state["x"], place, ends)
        got = {"order": order, "place": place, "ends": ends, "rows": rows,
               "out": tg.combine(state["y"], place, weights=w, residual=state["residual"])}
        if op == "route_train":
            got["dy"], got["dweights"] = tg.combine_backward(state["dout"], state["y"], place, w, ends)
            got["dx"] = tg.combine(state["drows"], place, residual=state["dout"])
        return got
    if op == "norm_train":
        y, total, _ = tg.layer_norm(state["x"], state["weight"], state["bias"], residual=state["residual"], eps=EPS)
        dx, dw, db = tg.layer_norm_backward(state["dy"], total, state["weight"], dsum=state["dsum"], eps=EPS)
        return {"sum": total, "y": y, "dx": dx, "dw": dw, "db": db}
    if op == "linear":
        got = {}
        if state["norm"]:
            code, got["sum"], got["scales"] = tg.layer_norm(state["x"], state["weight"], state["norm_bias"],
                                                            residual=state["residual"], eps=EPS, out_dtype=torch.int8)
        else:
            code, got["scales"] = tg.quantize_int8(state["x"])
        got["y"] = tg.int8_gemm(code, state["b"], got["scales"], state["b_scales"], bias=state["bias"],
                                op_b="T" if state["weights"] == "nk" else "N")
        return got
    code, scales = tg.quantize_int8(state["x"])
    return {"scales": scales, "y": tg.int8_gemm(code, state["b"], scales, state["b_scales"], ends=state["ends"])}


def work(case):
    op = case["op"]
    if op in ("route", "route_train"):
        t, c, e = case["tokens"], case["cols"], 4 if case["type"] == "f32" else 2
        choices = t * case["top"]
        used = choices * case["held"] / case["experts"]           # choices that have a row, about
        # reads the choices, x, the weights, the residual and the experts' rows; writes the plan, the rows and out
        size = 8 * choices + 8 * choices + 4 * case["held"] + 4 * choices + (3 * t + choices + used) * c * e
        if op == "route":
            return {"bytes": size, "flops": 2 * used * c}
        # reads dout and the rows' gradients; writes the gradients of the experts' rows, of the weights and of x
        return {"bytes": size + (2 * t + used + choices) * c * e + 4 * choices, "flops": 6 * used * c}
    if op == "norm_train":
        r, c, e = case["rows"], case["cols"], 4 if case["type"] == "f32" else 2
        # reads x, residual, dy, dsum, weight, bias; writes sum, y, dx, dw, db
        return {"bytes": 7 * r * c * e + c * (2 * e + 8), "flops": 20 * r * c}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        # reads x (and the residual, and writes the sum), the weights, scales and bias; writes the scales and y
        return {"bytes": m * k * (6 if case["norm"] else 2) + n * k + 4 * m + 8 * n + 2 * m * n, "flops": 2 * m * n * k}
    rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
    # Weights of groups without rows are not needed: about groups * (1 - (1 - 1/groups)^rows) have some.
    used = groups * (1.0 - (1.0 - 1.0 / groups) ** rows) if groups > 1 else 1.0
    return {"bytes": 2 * rows * k + used * n * (k + 4) + 4 * rows + 2 * rows * n, "flops": 2 * rows * n * k}


# 64 bits, from the definitions.

def _exact_rows(v):
    """(codes, scales) of rows in 64 bits."""
    top = torch.clamp(v.abs().max(dim=1).values, min=MIN_AMAX)
    return torch.round(v * TOP_CODE / top[:, None]), top / TOP_CODE


def _exact_norm(s):
    """(sum in 64 bits, as kept, deviation over its size) of rows."""
    t64 = s["x"].to(torch.float64) + s["residual"].to(torch.float64)
    kept = t64.to(s["x"].dtype).to(torch.float64)
    mean = kept.sum(dim=1) / kept.shape[1]
    off = kept - mean[:, None]
    inverse = 1.0 / torch.sqrt((off * off).sum(dim=1) / kept.shape[1] + EPS)
    return t64, off * inverse[:, None], inverse


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("route", "route_train"):
        tokens, top, cols, held = case["tokens"], case["top"], case["cols"], case["held"]
        expert = s["expert"].cpu()
        flat = expert.reshape(-1)
        # Rows go out expert by expert, a token's earlier ones first.
        lists = [torch.nonzero(flat == e).flatten() for e in range(held)]
        ends = torch.tensor([x.numel() for x in lists]).cumsum(0)
        used = int(ends[-1])
        order = torch.full((tokens * top,), -1, dtype=torch.int64)
        order[:used] = torch.cat(lists)
        place = torch.full((tokens * top,), -1, dtype=torch.int64)
        place[order[:used]] = torch.arange(used)
        here, back = order[:used].cuda(), place.view(tokens, top).cuda()
        token = here // top
        rows = torch.zeros((tokens * top, cols), dtype=f64, device="cuda")
        rows[:used] = s["x"].to(f64)[token]
        out = s["residual"].to(f64)
        w = s["weights"].to(f64)
        weight_of_row = w.reshape(-1)[here]
        out.index_add_(0, token, s["y"][:used].to(f64) * weight_of_row[:, None])
        got = {"order": order.int(), "place": back.int(), "ends": ends.int(), "rows": rows, "out": out}
        if op == "route_train":
            d = s["dout"].to(f64)
            dy = torch.zeros((tokens * top, cols), dtype=f64, device="cuda")
            dy[:used] = d[token] * weight_of_row[:, None]
            dw = torch.zeros(tokens * top, dtype=f64, device="cuda")
            dw[here] = (d[token] * s["y"][:used].to(f64)).sum(dim=1)
            got["dy"], got["dweights"] = dy, dw.view(tokens, top)
            got["dx"] = d.clone().index_add_(0, token, s["drows"][:used].to(f64))
        return got
    if op == "norm_train":
        t64, unit, inverse = _exact_norm(s)
        w, dy = s["weight"].to(f64), s["dy"].to(f64)
        y = unit * w[None, :] + s["bias"].to(f64)[None, :]
        up, n = dy * w[None, :], case["cols"]
        along = (up * unit).sum(dim=1) / n
        dx = inverse[:, None] * (up - (up.sum(dim=1) / n)[:, None] - unit * along[:, None]) + s["dsum"].to(f64)
        return {"sum": t64, "y": y, "dx": dx, "dw": (dy * unit).sum(dim=0), "db": dy.sum(dim=0)}
    if op == "linear":
        got, v = {}, s["x"].to(f64)
        if case["norm"]:
            got["sum"], unit, _ = _exact_norm(s)
            v = unit * s["weight"].to(f64)[None, :] + s["norm_bias"].to(f64)[None, :]
        code, scale = _exact_rows(v)
        b = s["b"].to(f64)
        y = code @ (b.t() if case["weights"] == "nk" else b)
        got["scales"], got["y"] = scale, scale[:, None] * y * s["b_scales"].to(f64)[None, :] + s["bias"].to(f64)[None, :]
        return got
    code, scale = _exact_rows(s["x"].to(f64))
    y = torch.empty((case["rows"], case["n"]), dtype=f64, device="cuda")
    first = 0
    for g, size in enumerate(s["sizes"]):
        if size:
            here = slice(first, first + size)
            y[here] = (code[here] @ s["b"][g].to(f64).t()) * scale[here, None] * s["b_scales"][g].to(f64)[None, :]
        first += size
    return {"scales": scale, "y": y}
