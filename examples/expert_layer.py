"""A sparse expert layer on the library's operators: trained in bf16, then
served in fp8 with block scales.

    python examples/expert_layer.py [--tokens 2048] [--hidden 1024] [--inner 512] [--experts 16] [--steps 30]

The layer: s = x + residual, h = norm(s), two linear maps with a SiLU between
them in each of the two experts that the router picks for a token, their
results weighted and added to s; then a linear head on the norm of that.
Training uses rms_norm / rms_norm_backward, grouped_gemm (forward and input
gradient) and grouped_wgrad; serving quantises the weights once and uses
rms_norm with fp8 output, grouped_gemm and block_gemm with scales, and
quantize between the two maps.  Where a token goes stays on the GPU
throughout: no step waits for the host.
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
    """(order, back, ends, share): the rows token * TOP + choice sorted by
    expert, where each of them went, the experts' ends, the choices' weights."""
    value, expert = (h.float() @ router.t()).topk(TOP, dim=1)
    flat = expert.flatten()
    order = flat.argsort(stable=True)
    sizes = (flat[:, None] == torch.arange(router.shape[0], device=h.device)).sum(0)
    return order, order.argsort(), sizes.cumsum(0).to(torch.int32), value.softmax(dim=1)


def combine(rows, back, share, summed):
    each = rows[back].view(share.shape[0], TOP, -1).float()
    return (summed.float() + (each * share[:, :, None]).sum(1)).to(summed.dtype)


class ExpertLayer(torch.nn.Module):
    def __init__(self, hidden, inner, experts, out):
        super().__init__()
        p = torch.nn.Parameter
        self.norm, self.last = p(torch.ones(hidden)), p(torch.ones(hidden))
        self.router = p(torch.randn(experts, hidden) / hidden ** 0.5)
        self.up = p(torch.randn(experts, inner, hidden) / hidden ** 0.5)
        self.down = p(torch.randn(experts, hidden, inner) / inner ** 0.5)
        self.head = p(torch.randn(1, out, hidden) / hidden ** 0.5)

    def forward(self, x, residual):
        h, summed = Norm.apply(x, residual, self.norm)
        order, back, ends, share = route(h, self.router)
        y = GroupedLinear.apply(h[order // TOP], self.up, ends)
        y = GroupedLinear.apply(F.silu(y), self.down, ends)
        y = combine(y, back, share, summed)
        y, _ = Norm.apply(y, torch.zeros_like(y), self.last)
        whole = torch.full((1,), x.shape[0], dtype=torch.int32, device=x.device)
        return GroupedLinear.apply(y, self.head, whole)       # one group: a dense layer


class Fp8Layer:
    """The trained layer's weights as E4M3 codes with a scale for every 128 x 128 tile."""

    def __init__(self, layer):
        self.norm, self.last = layer.norm.detach().bfloat16(), layer.last.detach().bfloat16()
        self.router = layer.router.detach()
        self.up, self.down = self.pack(layer.up), self.pack(layer.down)
        self.head = tg.quantize(layer.head.detach()[0], 128)

    @staticmethod
    def pack(weight):
        pairs = [tg.quantize(w, 128) for w in weight.detach()]
        return torch.stack([q.view(torch.uint8) for q, _ in pairs]).view(FP8), torch.stack([s for _, s in pairs])

    def __call__(self, x, residual):
        q, summed, scales = tg.rms_norm(x, self.norm, residual=residual, out_dtype=FP8)
        order, back, ends, share = route(tg.rms_norm(summed, self.norm)[0], self.router)
        rows = order // TOP
        y = tg.grouped_gemm(q.view(torch.uint8)[rows].view(FP8), self.up[0], ends, scales[rows], self.up[1])
        q, scales = tg.quantize(F.silu(y))
        y = tg.grouped_gemm(q, self.down[0], ends, scales, self.down[1])
        y = combine(y, back, share, summed)
        q, _, scales = tg.rms_norm(y, self.last, out_dtype=FP8)
        return tg.block_gemm(q, self.head[0], scales, self.head[1])


def run(tokens=2048, hidden=1024, inner=512, experts=16, out=256, steps=30, seed=0, say=print):
    """(losses, relative error of the fp8 layer's outputs against the bf16 layer's, on the rows of a batch
    and on a batch of 4 rows)."""
    torch.manual_seed(seed)
    layer = ExpertLayer(hidden, inner, experts, out).cuda()
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
    served, errors = Fp8Layer(layer), []
    with torch.no_grad():
        for rows in (tokens, 4):
            want, got = layer(x[:rows], residual[:rows]).float(), served(x[:rows], residual[:rows]).float()
            errors.append(float((got - want).norm() / want.norm()))
            say(f"fp8 against bf16 on {rows} rows: relative error {errors[-1]:.4f}", flush=True)
    return losses, errors


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("hidden", 1024), ("inner", 512), ("experts", 16), ("steps", 30)):
        parser.add_argument(f"--{name}", type=int, default=value)
    run(**vars(parser.parse_args()))
