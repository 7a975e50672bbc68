"""A sparse expert layer on the library's operators: trained in bf16, then
served in fp8 with block scales or in 8-bit integers.

    python examples/expert_layer.py [--tokens 2048] [--hidden 1024] [--inner 512] [--experts 16] [--steps 30]
                                    [--norm rms|layer] [--codes fp8|int8]

The layer: s = x + residual, h = norm(s), two linear maps with a SiLU between
them in each of the two experts that the router picks for a token, their
results weighted and added to s; then a linear head on the norm of that.
Training uses rms_norm or layer_norm and their gradients, expert_plan,
dispatch and combine (combine_backward) around the experts, grouped_gemm
(forward and input gradient) and grouped_wgrad.  Serving quantises the weights
once.  In fp8 it uses the norm with fp8 output, grouped_gemm and block_gemm
with scales, and quantize between the two maps; in 8-bit integers the layer
norm with their output (or the RMS norm and quantize_int8), int8_gemm and
quantize_int8.  Where a token goes stays on the GPU throughout: no step waits
for the host.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_gemm_f32_amd as tg  # noqa: E402

FP8 = torch.float8_e4m3fn
TOP = 2


class Norm(torch.autograd.Function):
    """(norm(x + residual) * weight, x + residual), x and residual bf16, weight an fp32 master."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        w = weight.to(x.dtype)
        out, summed, _ = tg.rms_norm(x, w, residual=residual)
        ctx.save_for_backward(summed, w)
        return out, summed

    @staticmethod
    def backward(ctx, dout, dsum):
        summed, w = ctx.saved_tensors
        dx, dw = tg.rms_norm_backward(dout, summed, w, dsum=dsum)
        return dx, dx, dw


class LayerNorm(torch.autograd.Function):
    """(layer norm of x + residual, x + residual), weight and bias fp32 masters."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias):
        w = weight.to(x.dtype)
        out, summed, _ = tg.layer_norm(x, w, bias.to(x.dtype), residual=residual)
        ctx.save_for_backward(summed, w)
        return out, summed

    @staticmethod
    def backward(ctx, dout, dsum):
        summed, w = ctx.saved_tensors
        dx, dw, db = tg.layer_norm_backward(dout, summed, w, dsum=dsum)
        return dx, dx, dw, db


class Dispatch(torch.autograd.Function):
    """Each token's row to its experts' rows."""

    @staticmethod
    def forward(ctx, x, place, ends):
        ctx.save_for_backward(place)
        return tg.dispatch(x, place, ends)

    @staticmethod
    def backward(ctx, drows):
        return tg.combine(drows.contiguous(), *ctx.saved_tensors), None, None


class Combine(torch.autograd.Function):
    """residual[t] + the rows of token t's choices, each times its weight."""

    @staticmethod
    def forward(ctx, rows, place, ends, weights, residual):
        ctx.save_for_backward(rows, place, ends, weights)
        return tg.combine(rows, place, weights, residual)

    @staticmethod
    def backward(ctx, dout):
        rows, place, ends, weights = ctx.saved_tensors
        dout = dout.contiguous()
        drows, dweights = tg.combine_backward(dout, rows, place, weights, ends)
        return drows, None, None, dweights, dout


class GroupedLinear(torch.autograd.Function):
    """x[i] @ weight[g].T for each row i of group g, weight (groups x N x K) an fp32 master."""

    @staticmethod
    def forward(ctx, x, weight, ends):
        w = weight.to(x.dtype)
        ctx.save_for_backward(x, w, ends)
        return tg.grouped_gemm(x, w, ends)

    @staticmethod
    def backward(ctx, dy):
        x, w, ends = ctx.saved_tensors
        dy = dy.contiguous()
        return tg.grouped_gemm(dy, w, ends, op_b="N"), tg.grouped_wgrad(dy, x, ends), None


def route(h, router):
    """(place, ends, weights): the rows of each token's choices, sorted by expert, and the choices' weights."""
    value, expert = (h.float() @ router.t()).topk(TOP, dim=1)
    _, place, ends = tg.expert_plan(expert, router.shape[0])
    return place, ends, value.softmax(dim=1)


class ExpertLayer(torch.nn.Module):
    def __init__(self, hidden, inner, experts, out, norm="rms"):
        super().__init__()
        p = torch.nn.Parameter
        self.norm, self.last = p(torch.ones(hidden)), p(torch.ones(hidden))
        if norm == "layer":
            self.norm_bias, self.last_bias = p(torch.zeros(hidden)), p(torch.zeros(hidden))
        self.router = p(torch.randn(experts, hidden) / hidden ** 0.5)
        self.up = p(torch.randn(experts, inner, hidden) / hidden ** 0.5)
        self.down = p(torch.randn(experts, hidden, inner) / inner ** 0.5)
        self.head = p(torch.randn(1, out, hidden) / hidden ** 0.5)

    def normed(self, x, residual, name):
        weight, bias = getattr(self, name), getattr(self, name + "_bias", None)
        return Norm.apply(x, residual, weight) if bias is None else LayerNorm.apply(x, residual, weight, bias)

    def forward(self, x, residual):
        h, summed = self.normed(x, residual, "norm")
        place, ends, weights = route(h, self.router)
        y = GroupedLinear.apply(Dispatch.apply(h, place, ends), self.up, ends)
        y = GroupedLinear.apply(F.silu(y), self.down, ends)
        y = Combine.apply(y, place, ends, weights, summed)
        y, _ = self.normed(y, torch.zeros_like(y), "last")
        whole = torch.full((1,), x.shape[0], dtype=torch.int32, device=x.device)
        return GroupedLinear.apply(y, self.head, whole)       # one group: a dense layer


class Served:
    """What the served layers share: the trained norms and router, and the norms' calls."""

    def __init__(self, layer):
        self.weights = {n: p.detach().bfloat16() for n, p in layer.named_parameters() if p.dim() == 1}
        self.router = layer.router.detach()

    def normed(self, x, name, residual=None, out_dtype=None):
        weight, bias = self.weights[name], self.weights.get(name + "_bias")
        if bias is None:
            return tg.rms_norm(x, weight, residual=residual, out_dtype=out_dtype)
        return tg.layer_norm(x, weight, bias, residual=residual, out_dtype=out_dtype)


class Fp8Layer(Served):
    """The trained layer's weights as E4M3 codes with a scale for every 128 x 128 tile."""

    def __init__(self, layer):
        super().__init__(layer)
        self.up, self.down = self.pack(layer.up), self.pack(layer.down)
        self.head = tg.quantize(layer.head.detach()[0], 128)

    @staticmethod
    def pack(weight):
        pairs = [tg.quantize(w, 128) for w in weight.detach()]
        return torch.stack([q.view(torch.uint8) for q, _ in pairs]).view(FP8), torch.stack([s for _, s in pairs])

    def __call__(self, x, residual):
        q, summed, scales = self.normed(x, "norm", residual, FP8)
        place, ends, weights = route(self.normed(summed, "norm")[0], self.router)
        rows, row_scales = tg.dispatch(q, place, ends, scales=scales)
        y = tg.grouped_gemm(rows, self.up[0], ends, row_scales, self.up[1])
        q, scales = tg.quantize(F.silu(y))
        y = tg.grouped_gemm(q, self.down[0], ends, scales, self.down[1])
        y = tg.combine(y, place, weights, summed)
        q, _, scales = self.normed(y, "last", out_dtype=FP8)
        return tg.block_gemm(q, self.head[0], scales, self.head[1])


class Int8Layer(Served):
    """The trained layer's weights as 8-bit integers with a scale for every output channel."""

    def __init__(self, layer):
        super().__init__(layer)
        self.up, self.down, self.head = (self.pack(w) for w in (layer.up, layer.down, layer.head))

    @staticmethod
    def pack(weight):
        pairs = [tg.quantize_int8(w) for w in weight.detach()]
        return torch.stack([q for q, _ in pairs]), torch.stack([s for _, s in pairs])

    def quantised(self, x, name, residual=None):
        if name + "_bias" in self.weights:
            return self.normed(x, name, residual, torch.int8)
        y, summed, _ = self.normed(x, name, residual)
        q, scales = tg.quantize_int8(y)
        return q, summed, scales

    def __call__(self, x, residual):
        q, summed, scales = self.quantised(x, "norm", residual)
        place, ends, weights = route(self.normed(summed, "norm")[0], self.router)
        rows, row_scales = tg.dispatch(q, place, ends, scales=scales)
        y = tg.int8_gemm(rows, self.up[0], row_scales, self.up[1], ends=ends)
        q, scales = tg.quantize_int8(F.silu(y))
        y = tg.int8_gemm(q, self.down[0], scales, self.down[1], ends=ends)
        y = tg.combine(y, place, weights, summed)
        q, _, scales = self.quantised(y, "last")
        return tg.int8_gemm(q, self.head[0][0], scales, self.head[1][0])


def run(tokens=2048, hidden=1024, inner=512, experts=16, out=256, steps=30, seed=0, say=print, norm="rms", codes="fp8"):
    """(losses, relative error of the served layer's outputs against the bf16 layer's, on the rows of a batch
    and on a batch of 4 rows)."""
    torch.manual_seed(seed)
    layer = ExpertLayer(hidden, inner, experts, out, norm).cuda()
    x = torch.randn(tokens, hidden).bfloat16().cuda()
    residual = torch.randn(tokens, hidden).bfloat16().cuda()
    target = torch.tanh(x.float() @ torch.randn(hidden, out).cuda() / hidden ** 0.5)
    optimiser = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        optimiser.zero_grad(set_to_none=True)
        loss = F.mse_loss(layer(x, residual).float(), target)
        loss.backward()
        optimiser.step()
        losses.append(float(loss.detach()))
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    served, errors = {"fp8": Fp8Layer, "int8": Int8Layer}[codes](layer), []
    with torch.no_grad():
        for rows in (tokens, 4):
            want, got = layer(x[:rows], residual[:rows]).float(), served(x[:rows], residual[:rows]).float()
            errors.append(float((got - want).norm() / want.norm()))
            say(f"{codes} against bf16 on {rows} rows: relative error {errors[-1]:.4f}", flush=True)
    return losses, errors


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("hidden", 1024), ("inner", 512), ("experts", 16), ("steps", 30)):
        parser.add_argument(f"--{name}", type=int, default=value)
    parser.add_argument("--norm", choices=("rms", "layer"), default="rms")
    parser.add_argument("--codes", choices=("fp8", "int8"), default="fp8")
    run(**vars(parser.parse_args()))
