"""The operators of a sparse expert layer: what is measured, and their plain forms.

Three operators: the root-mean-square norm that adds the residual and gives
fp8 codes with scales (and its backward pass), the fp8 product with a scale
for each block of 128 (with the quantiser that makes its left operand), and
products grouped by expert with ragged sizes (and their gradients).

``run`` computes a case in elementary torch operations, in 32 bits, or with
``own`` set by the library's kernels.  ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -100
FP8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # One step of decoding for 16 sequences: the norm before a layer's products.
        {"name": "norm_fp8_decode", "op": "norm_fp8", "rows": 16, "cols": 8192},
        # A prefill of 8192 tokens through the same norm.
        {"name": "norm_fp8_prefill", "op": "norm_fp8", "rows": 8192, "cols": 8192},
        # A training step of the norm: forward, then the gradients.
        {"name": "norm_train_bf16", "op": "norm_train", "rows": 8192, "cols": 4096, "type": "bf16"},
        # The same in fp32 at an odd width (no row but the first is 16-byte aligned).
        {"name": "norm_train_f32_odd", "op": "norm_train", "rows": 1000, "cols": 777, "type": "f32"},
        # A linear layer with fp8 weights while decoding 16 sequences: activations are quantised as they come.
        {"name": "block_decode", "op": "block", "m": 16, "n": 8192, "k": 8192, "weights": "nk", "codes": False},
        # Odd sizes in every direction (padded rows, the last scale block cut).
        {"name": "block_odd", "op": "block", "m": 1000, "n": 3000, "k": 777, "weights": "nk", "codes": False},
        # The gradient of a linear layer's input: the stored weights are read the other way.
        {"name": "block_input_grad", "op": "block", "m": 2048, "n": 4096, "k": 4096, "weights": "kn", "codes": False},
        # A large prefill or training product, whose left operand an earlier norm left in fp8.
        {"name": "block_large", "op": "block", "m": 8192, "n": 8192, "k": 8192, "weights": "nk", "codes": True},
        # 16 tokens, 4 experts each of 32: every expert's weights are read for a few rows.
        {"name": "grouped_fp8_decode", "op": "grouped_fp8", "rows": 64, "groups": 32, "n": 4096, "k": 4096},
        # A prefill through 16 experts with uneven loads.
        {"name": "grouped_fp8_prefill", "op": "grouped_fp8", "rows": 8192, "groups": 16, "n": 4096, "k": 4096},
        # A training step of the experts' product: output, input gradient, weight gradients.
        {"name": "grouped_train_bf16", "op": "grouped_train", "rows": 8192, "groups": 8, "n": 4096, "k": 2048,
         "type": "bf16"},
        # fp32 with odd sizes, a small layer.
        {"name": "grouped_train_f32_odd", "op": "grouped_train", "rows": 777, "groups": 12, "n": 1000, "k": 257,
         "type": "f32"},
    ]


def _spread(rng, low, high, multiple=1):
    """A size between low and high, even over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, v // multiple * multiple))


def draw(rng):
    op = rng.choice(["norm_fp8", "norm_train", "block", "grouped_fp8", "grouped_train"])
    multiple = rng.choice([1, 8, 128])
    if op == "norm_fp8":
        return {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 128, 8192, multiple)}
    if op == "norm_train":
        return {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 128, 8192, multiple),
                "type": rng.choice(["f32", "bf16"])}
    if op == "block":
        return {"op": op, "m": _spread(rng, 1, 8192), "n": _spread(rng, 128, 8192, multiple),
                "k": _spread(rng, 128, 8192, multiple), "weights": rng.choice(["nk", "kn"]),
                "codes": rng.random() < 0.5}
    if op == "grouped_fp8":
        return {"op": op, "rows": _spread(rng, 1, 8192), "groups": _spread(rng, 1, 64),
                "n": _spread(rng, 128, 4096, multiple), "k": _spread(rng, 128, 4096, multiple)}
    kind = rng.choice(["f32", "bf16"])
    most = 4096 if kind == "bf16" else 1024
    return {"op": op, "rows": _spread(rng, 1, 8192 if kind == "bf16" else 4096), "groups": _spread(rng, 1, 64),
            "n": _spread(rng, 64, most, multiple), "k": _spread(rng, 64, most, multiple), "type": kind}


def _blocks(n):
    return -(-n // BLOCK)


def _padded_rows(rows, cols, dtype):
    """rows x cols whose rows start on 16 bytes, as the library's own allocations do."""
    per = 16 // dtype.itemsize
    return torch.empty((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


def _row_codes(x, rounded=True):
    """Codes and scales of x, a block of 128 columns of a row each (rounded=False: codes before rounding)."""
    rows, cols = x.shape
    kb = _blocks(cols)
    xp = torch.nn.functional.pad(x, (0, kb * BLOCK - cols)).view(rows, kb, BLOCK)
    finite = torch.where(xp.isfinite(), xp, torch.zeros_like(xp))
    scale = finite.abs().amax(dim=2).clamp_min(MIN_AMAX) / E4M3_MAX
    code = (xp / scale[:, :, None]).view(rows, kb * BLOCK)[:, :cols]
    return (code.to(FP8) if rounded else code), scale


def _tile_codes(w):
    """Codes and scales of a stored weight, a block of 128 x 128 each."""
    rows, cols = w.shape
    rb, cb = _blocks(rows), _blocks(cols)
    wp = torch.nn.functional.pad(w, (0, cb * BLOCK - cols, 0, rb * BLOCK - rows)).view(rb, BLOCK, cb, BLOCK)
    scale = wp.abs().amax(dim=(1, 3)).clamp_min(MIN_AMAX) / E4M3_MAX
    return (wp / scale[:, None, :, None]).view(rb * BLOCK, cb * BLOCK)[:rows, :cols].to(FP8), scale


def _from_rows(code, scale, dtype):
    """Values of codes with a scale for each 128 columns of a row."""
    return code.to(dtype) * scale.to(dtype).repeat_interleave(BLOCK, dim=1)[:, :code.shape[1]]


def _from_tiles(code, scale, dtype):
    """Values of codes with a scale for each 128 x 128 block (any leading dimensions)."""
    s = scale.to(dtype).repeat_interleave(BLOCK, dim=-2)[..., :code.shape[-2], :]
    return code.to(dtype) * s.repeat_interleave(BLOCK, dim=-1)[..., :code.shape[-1]]


def _sizes(rows, groups, seed):
    """How many rows each group has: uneven, as a router leaves them, some of them none."""
    g = torch.Generator().manual_seed(seed + 77)
    share = torch.softmax(torch.randn(groups, generator=g) * 0.7, 0)
    if rows == 0:
        return [0] * groups
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

    s = dict(case)
    op = case["op"]
    if op in ("norm_fp8", "norm_train"):
        rows, cols = case["rows"], case["cols"]
        dtype = torch.bfloat16 if op == "norm_fp8" else TYPES[case["type"]]
        s["x"] = normal(rows, cols, scale=0.5).to(dtype)
        s["residual"] = activations(rows, cols).to(dtype)
        s["weight"] = (1.0 + normal(cols, scale=0.1)).to(dtype)
        if op == "norm_train":
            s["dy"] = normal(rows, cols, scale=0.1).to(dtype)
            s["dsum"] = normal(rows, cols, scale=0.1).to(dtype)
    elif op == "block":
        m, n, k = case["m"], case["n"], case["k"]
        x = activations(m, k).to(torch.bfloat16)
        if case["codes"]:
            code, s["a_scales"] = _row_codes(x.float())
            s["a"] = kept(code, FP8)
        else:
            s["x"] = kept(x, torch.bfloat16)
        w = normal(n, k, scale=k ** -0.5) if case["weights"] == "nk" else normal(k, n, scale=k ** -0.5)
        code, s["b_scales"] = _tile_codes(w)
        s["b"] = kept(code, FP8)
    else:
        rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
        s["sizes"] = _sizes(rows, groups, seed)
        s["ends"] = torch.tensor(s["sizes"]).cumsum(0).to(device="cuda", dtype=torch.int32)
        x = activations(rows, k).to(torch.bfloat16)
        if op == "grouped_fp8":
            code, s["a_scales"] = _row_codes(x.float())
            s["a"] = kept(code, FP8)
            pad = -(-k // 16) * 16
            s["b"] = torch.empty((groups, n, pad), dtype=FP8, device="cuda")[:, :, :k]
            s["b_scales"] = torch.empty((groups, _blocks(n), _blocks(k)), device="cuda")
            for g in range(groups):
                code, s["b_scales"][g] = _tile_codes(normal(n, k, scale=k ** -0.5))
                s["b"][g].copy_(code)
        else:
            dtype = TYPES[case["type"]]
            s["x"] = x.to(dtype)
            s["w"] = normal(groups, n, k, scale=k ** -0.5).to(dtype)
            s["dy"] = normal(rows, n, scale=0.1).to(dtype)
    return s


def _norm(x, residual, weight, wide, eps=EPS):
    """(sum as it is kept, its norm before the last rounding) with the arithmetic in `wide`."""
    total = (x.to(wide) + residual.to(wide)).to(x.dtype)
    t = total.to(wide)
    r = torch.rsqrt(t.square().mean(dim=1, keepdim=True) + eps)
    return total, t * r * weight.to(wide)


def _norm_grads(dy, total, weight, dsum, wide, eps=EPS):
    t, d = total.to(wide), dy.to(wide)
    r = torch.rsqrt(t.square().mean(dim=1, keepdim=True) + eps)
    g = d * weight.to(wide)
    dx = r * (g - t * r.square() * (g * t).mean(dim=1, keepdim=True)) + dsum.to(wide)
    return dx, (d.double() * t.double() * r.double()).sum(dim=0)


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "norm_fp8":
        total, y = _norm(state["x"], state["residual"], state["weight"], torch.float32)
        code, scale = _row_codes(y)
        return {"sum": total, "codes": code, "scales": scale}
    if op == "norm_train":
        x, w = state["x"], state["weight"]
        total, y = _norm(x, state["residual"], w, torch.float32)
        dx, dw = _norm_grads(state["dy"], total, w, state["dsum"], torch.float32)
        return {"sum": total, "y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.float()}
    if op == "block":
        code, scale = (state["a"], state["a_scales"]) if state["codes"] else _row_codes(state["x"].float())
        a, b = _from_rows(code, scale, torch.float32), _from_tiles(state["b"], state["b_scales"], torch.float32)
        y = (a @ (b.t() if state["weights"] == "nk" else b)).to(torch.bfloat16)
        return {"y": y} if state["codes"] else {"codes": code, "scales": scale, "y": y}
    if op == "grouped_fp8":
        a = _from_rows(state["a"], state["a_scales"], torch.float32)
        b = _from_tiles(state["b"], state["b_scales"], torch.float32)
        return {"y": torch.cat([p @ q.t() for p, q in zip(a.split(state["sizes"]), b)]).to(torch.bfloat16)}
    x, w, dy, sizes = state["x"].float(), state["w"].float(), state["dy"].float(), state["sizes"]
    y = torch.cat([p @ q.t() for p, q in zip(x.split(sizes), w)])
    dx = torch.cat([p @ q for p, q in zip(dy.split(sizes), w)])
    dw = torch.stack([p.t() @ q for p, q in zip(dy.split(sizes), x.split(sizes))])
    return {"y": y.to(state["x"].dtype), "dx": dx.to(state["x"].dtype), "dw": dw}


def _run_own(state):
    import tiled_gemm_f32_amd as tg
    op = state["op"]
    if op == "norm_fp8":
        code, total, scale = tg.rms_norm(state["x"], state["weight"], residual=state["residual"], eps=EPS,
                                         out_dtype=FP8)
        return {"sum": total, "codes": code, "scales": scale}
    if op == "norm_train":
        y, total, _ = tg.rms_norm(state["x"], state["weight"], residual=state["residual"], eps=EPS)
        dx, dw = tg.rms_norm_backward(state["dy"], total, state["weight"], dsum=state["dsum"], eps=EPS)
        return {"sum": total, "y": y, "dx": dx, "dw": dw}
    if op == "block":
        code, scale = (state["a"], state["a_scales"]) if state["codes"] else tg.quantize(state["x"])
        y = tg.block_gemm(code, state["b"], scale, state["b_scales"], op_b="T" if state["weights"] == "nk" else "N")
        return {"y": y} if state["codes"] else {"codes": code, "scales": scale, "y": y}
    if op == "grouped_fp8":
        return {"y": tg.grouped_gemm(state["a"], state["b"], state["ends"], a_scales=state["a_scales"],
                                     b_scales=state["b_scales"], op_b="T", out_dtype=torch.bfloat16)}
    x, w, dy, ends = state["x"], state["w"], state["dy"], state["ends"]
    return {"y": tg.grouped_gemm(x, w, ends, op_b="T", out_dtype=x.dtype),
            "dx": tg.grouped_gemm(dy, w, ends, op_b="N", out_dtype=x.dtype),
            "dw": tg.grouped_wgrad(dy, x, ends)}


def work(case):
    op = case["op"]
    if op in ("norm_fp8", "norm_train"):
        r, c = case["rows"], case["cols"]
        if op == "norm_fp8":
            # reads x, residual and weight; writes the sum, the codes and the scales
            return {"bytes": r * c * (2 + 2 + 2 + 1) + 4 * r * _blocks(c) + 2 * c, "flops": 8 * r * c}
        e = 4 if case["type"] == "f32" else 2
        # reads x, residual, dy, dsum, weight; writes sum, y, dx, dw
        return {"bytes": 7 * r * c * e + c * (e + 4), "flops": 16 * r * c}
    if op == "block":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * (m * _blocks(k) + _blocks(n) * _blocks(k))
        # reads the codes, or bf16 values whose codes it writes too
        return {"bytes": m * k * (1 if case["codes"] else 3) + n * k + scales + 2 * m * n, "flops": 2 * m * n * k}
    rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
    if op == "grouped_fp8":
        # Weights of groups without rows are not needed: about groups * (1 - (1 - 1/groups)^rows) have some.
        used = groups * (1.0 - (1.0 - 1.0 / groups) ** rows) if groups > 1 else 1.0
        scales = 4 * (rows * _blocks(k) + used * _blocks(n) * _blocks(k))
        return {"bytes": rows * k + used * n * k + scales + 2 * rows * n, "flops": 2 * rows * n * k}
    e = 4 if case["type"] == "f32" else 2
    # reads x, dy and w; writes y, dx and dw
    return {"bytes": e * (2 * rows * (n + k) + groups * n * k) + 4 * groups * n * k, "flops": 6 * rows * n * k}


# 64 bits, from the definitions.

def _exact_codes(v):
    """(codes before rounding, scales) of v, 128 columns at a time."""
    parts = v.split(BLOCK, dim=1)
    tops = torch.stack([p.masked_fill(~p.isfinite(), 0).abs().max(dim=1).values for p in parts], dim=1)
    scales = torch.clamp(tops, min=MIN_AMAX) / E4M3_MAX
    return torch.cat([p / scales[:, j:j + 1] for j, p in enumerate(parts)], dim=1), scales


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("norm_fp8", "norm_train"):
        t64 = s["x"].to(f64) + s["residual"].to(f64)
        kept = t64.to(s["x"].dtype).to(f64)
        inverse = 1.0 / torch.sqrt((kept * kept).sum(dim=1) / case["cols"] + EPS)
        y = kept * inverse[:, None] * s["weight"].to(f64)[None, :]
        if op == "norm_fp8":
            code, scale = _exact_codes(y)
            return {"sum": t64, "codes": code, "scales": scale}
        up = s["dy"].to(f64) * s["weight"].to(f64)[None, :]
        along = (up * kept).sum(dim=1) / case["cols"] * inverse ** 3
        dx = up * inverse[:, None] - kept * along[:, None] + s["dsum"].to(f64)
        dw = (s["dy"].to(f64) * kept * inverse[:, None]).sum(dim=0)
        return {"sum": t64, "y": y, "dx": dx, "dw": dw}

    def tiles(code, scale):
        i = torch.arange(code.shape[0], device=code.device) // BLOCK
        j = torch.arange(code.shape[1], device=code.device) // BLOCK
        return code.to(f64) * scale.to(f64)[i][:, j]

    def rows_of(code, scale):
        j = torch.arange(code.shape[1], device=code.device) // BLOCK
        return code.to(f64) * scale.to(f64)[:, j]

    if op == "block":
        if case["codes"]:
            code, scale = None, None
            a = rows_of(s["a"], s["a_scales"])
        else:
            code, scale = _exact_codes(s["x"].to(f64))
            scale32 = scale.to(torch.float32)    # scales are kept in 32 bits, codes in 8
            wide = scale32.to(f64).repeat_interleave(BLOCK, dim=1)[:, :case["k"]]
            a = (s["x"].to(f64) / wide).to(torch.float32).to(FP8).to(f64) * wide
        b = tiles(s["b"], s["b_scales"])
        y = a @ (b.t() if case["weights"] == "nk" else b)
        return {"y": y} if case["codes"] else {"codes": code, "scales": scale, "y": y}
    ends = [0]
    for size in s["sizes"]:
        ends.append(ends[-1] + size)
    if op == "grouped_fp8":
        a = rows_of(s["a"], s["a_scales"])
        y = torch.empty((case["rows"], case["n"]), dtype=f64, device="cuda")
        for g in range(case["groups"]):
            if ends[g + 1] > ends[g]:
                y[ends[g]:ends[g + 1]] = a[ends[g]:ends[g + 1]] @ tiles(s["b"][g], s["b_scales"][g]).t()
        return {"y": y}
    y = torch.empty((case["rows"], case["n"]), dtype=f64, device="cuda")
    dx = torch.empty((case["rows"], case["k"]), dtype=f64, device="cuda")
    dw = torch.zeros((case["groups"], case["n"], case["k"]), dtype=f64, device="cuda")
    for g in range(case["groups"]):
        here = slice(ends[g], ends[g + 1])
        if ends[g + 1] > ends[g]:
            x, w, d = s["x"][here].to(f64), s["w"][g].to(f64), s["dy"][here].to(f64)
            y[here], dx[here], dw[g] = x @ w.t(), d @ w, d.t() @ x
    return {"y": y, "dx": dx, "dw": dw}
