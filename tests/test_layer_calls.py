"""Layer norm, 8-bit products and the routing: the wrappers' two ways, other
streams, captured graphs, and a run of all of them together."""
import math
import os
import sys

import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_torch_calls import same, stream_of

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

F32, BF16, FP8, I8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module")
def calls():
    tg.load()
    from tiled_gemm_f32_amd import _torch_calls
    return _torch_calls


def test_calls_outside_the_common_case_are_left_to_the_wrappers(calls):
    x, w = torch.zeros(4, 8), torch.ones(8)
    q, s, e = torch.zeros(4, 8, dtype=I8), torch.ones(4), torch.zeros(4, 2, dtype=torch.int64)
    place, ends, share = e.int(), torch.tensor([4], dtype=torch.int32), torch.ones(4, 2)
    for got in (calls.layer_norm(x, w, w, None, 1e-5, None, 0, 0), calls.layer_norm(x, w, 1, x, 1e-5, I8, 0, 0),
                calls.layer_norm(None, w, None, x, 1e-5, 7, 0, 0), calls.layer_norm(x, w, None, x, "1", None, 0, 0),
                calls.layer_norm_backward(x, x, w, None, 1e-5, 0, 0), calls.layer_norm_backward(x, 1, w, 2, None, 0, 0),
                calls.quantize_int8(x, 0, 0), calls.quantize_int8(None, 0, 0), calls.quantize_int8(x),
                calls.int8_gemm(q, q, s, s, None, None, "T", None, 0, 0),
                calls.int8_gemm(1, 2, 3, 4, 5, 6, 7, 8, 0, 0), calls.expert_plan(e, 3, 0, 0),
                calls.expert_plan(e, "3", 0, 0), calls.expert_plan(None, 3, 0, 0), calls.expert_plan(e, 1 << 70, 0, 0),
                calls.dispatch(x, place, ends, None, 0, 0), calls.dispatch(1, 2, 3, 4, 0, 0),
                calls.combine(x, place, share, x, 0, 0), calls.combine(x, None, None, None, 0, 0),
                calls.combine_backward(x, x, place, share, ends, 0, 0), calls.combine_backward(1, 2, 3, 4, 5, 0, 0)):
        assert got is None


def inputs(M, N, K, dtype, top=3, groups=5):
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randn(M, K + 3, generator=g).to(dtype).cuda()[:, 1:K + 1]
    w, b = (torch.nn.Parameter(torch.randn(K, generator=g).to(dtype).cuda()) for _ in range(2))
    experts = torch.randint(-1, groups, (M, top), generator=g).cuda()
    weights = torch.rand(M, top, generator=g).cuda()
    codes = torch.randint(-128, 128, (groups, N, K), generator=g, dtype=I8).cuda()
    scales = torch.rand(groups, N, generator=g).cuda()
    return x, w, b, experts, weights, codes, scales, groups


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 40, 24), (5, 1, 130), (33, 257, 1), (48, 256, 384), (1500, 20, 40)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_both_ways_give_the_same(gpu_available, calls, M, N, K, dtype):
    say(f"[calls] {M}x{N}x{K} {dtype}")
    here = torch.cuda.current_stream().cuda_stream        # a stream passed in: the wrapper's own way
    x, w, b, experts, weights, codes, scales, groups = inputs(M, N, K, dtype)
    for residual in (None, x + 1):
        for bias in (None, b):
            for kind in (None, F32, BF16, FP8, I8):
                same(tg.layer_norm(x, w, bias, residual=residual, out_dtype=kind),
                     tg.layer_norm(x, w, bias, residual=residual, out_dtype=kind, stream=here))
        same(tg.layer_norm_backward(x, x, w, dsum=residual), tg.layer_norm_backward(x, x, w, dsum=residual, stream=here))
    q, s = tg.quantize_int8(x)
    same((q, s), tg.quantize_int8(x, stream=here))
    ends = torch.tensor([M // 2] * (groups - 1) + [M], dtype=torch.int32).cuda()
    for op in "TN":
        c = codes if op == "T" else codes.transpose(1, 2).contiguous()
        for kind in (None, F32):
            for bias in (None, scales):
                same(tg.int8_gemm(q, c[1], s, scales[1], bias=bias[0] if bias is not None else None, op_b=op, out_dtype=kind),
                     tg.int8_gemm(q, c[1], s, scales[1], bias=bias[0] if bias is not None else None, op_b=op,
                                  out_dtype=kind, stream=here))
                same(tg.int8_gemm(q, c, s, scales, ends=ends, bias=bias, op_b=op, out_dtype=kind),
                     tg.int8_gemm(q, c, s, scales, ends=ends, bias=bias, op_b=op, out_dtype=kind, stream=here))
    for e in (experts, experts.int()):
        plan = tg.expert_plan(e, groups)
        same(plan, tg.expert_plan(e, groups, stream=here))
    order, place, ends = plan
    for t, sc in ((x, None), (q, s), tg.quantize(x)):
        same(tg.dispatch(t, place, ends, scales=sc), tg.dispatch(t, place, ends, scales=sc, stream=here))
    rows = tg.dispatch(x, place, ends)
    for share in (None, weights):
        for residual in (None, x):
            same(tg.combine(rows, place, weights=share, residual=residual),
                 tg.combine(rows, place, weights=share, residual=residual, stream=here))
    same(tg.combine_backward(x, rows, place, weights, ends), tg.combine_backward(x, rows, place, weights, ends, stream=here))


@pytest.mark.gpu
def test_a_call_on_another_stream_allocates_there(gpu_available, calls):
    x, w, b, experts, weights, codes, scales, groups = inputs(3000, 64, 256, F32)
    order, place, ends = tg.expert_plan(experts, groups)
    rows = tg.dispatch(x, place, ends)
    q, s = tg.quantize_int8(x)
    rows_end = ends.clamp_max(3000)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for name, call in (("layer_norm", lambda h: tg.layer_norm(x, w, b, residual=x, out_dtype=I8, stream=h)),
                       ("backward", lambda h: tg.layer_norm_backward(x, x, w, dsum=x, stream=h)),
                       ("rows", lambda h: tg.quantize_int8(x, stream=h)),
                       ("product", lambda h: (tg.int8_gemm(q, codes, s, scales, ends=rows_end, stream=h),)),
                       ("plan", lambda h: tg.expert_plan(experts, groups, stream=h)),
                       ("dispatch", lambda h: tg.dispatch(q, place, ends, scales=s, stream=h)),
                       ("combine", lambda h: (tg.combine(rows, place, weights, x, stream=h),)),
                       ("combine backward", lambda h: tg.combine_backward(x, rows, place, weights, ends, stream=h))):
        say(f"[calls] another stream: {name}")
        got = call(other.cuda_stream)
        assert [stream_of(t) for t in got] == [other.cuda_stream] * len(got)
        other.synchronize()
        same(got, call(None))


def layer(x, res, w, b, experts, weights, codes, scales, dout):
    """One of everything, as a layer uses them; a tuple of all results."""
    groups = codes.shape[0]
    h, total, _ = tg.layer_norm(x, w, b, residual=res)
    q, _, s = tg.layer_norm(x, w, b, residual=res, out_dtype=I8)
    order, place, ends = tg.expert_plan(experts, groups)
    rows, row_scales = tg.dispatch(q, place, ends, scales=s)
    y = tg.int8_gemm(rows, codes, row_scales, scales, ends=ends)
    out = tg.combine(y, place, weights=weights, residual=total)
    dy, dweights = tg.combine_backward(dout, y, place, weights, ends)
    dh = tg.combine(tg.dispatch(dout, place, ends), place)
    dx, dw, db = tg.layer_norm_backward(dh, total, w, dsum=dout)
    return h, total, q, s, order, place, ends, rows, row_scales, y, out, dy, dweights, dx, dw, db


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [40, 1500])
def test_calls_capture_into_graphs_and_replay(gpu_available, tokens):
    say(f"[calls] graphs of {tokens} tokens")
    x, w, b, experts, weights, codes, scales, groups = inputs(tokens, 384, 384, BF16)
    static = [x.contiguous(), x + 1, w.detach(), b.detach(), experts, weights, codes, scales, x * 0.5]
    layer(*static)
    torch.cuda.synchronize()
    graphs, results = [], []
    for _ in range(2):                                    # two graphs, whose replays take turns
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(layer(*static))
        graphs.append(graph)
    g = torch.Generator().manual_seed(8)
    for turn in range(5):
        static[0].copy_(torch.randn(tokens, 384, generator=g).bfloat16())
        static[4].copy_(torch.randint(-1, groups, (tokens, 3), generator=g))
        static[5].copy_(torch.rand(tokens, 3, generator=g))
        graphs[turn % 2].replay()
        other = (torch.randn(500, 500, device="cuda") @ torch.randn(500, 500, device="cuda")).sum()
        graphs[(turn + 1) % 2].replay()
        assert math.isfinite(float(other))
        want = layer(*static)
        torch.cuda.synchronize()
        for got in results:
            same(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,inner,experts", [(300, 256, 128, 8), (513, 200, 333, 5)])
def test_expert_layer_around_layer_norm_and_in_8_bit_integers(gpu_available, tokens, hidden, inner, experts):
    import expert_layer
    losses, errors = expert_layer.run(tokens, hidden, inner, experts, out=64, steps=3, norm="layer", codes="int8")
    assert all(math.isfinite(v) for v in losses)
    # Each of three products has two quantised operands.  A row's values are off by up to half a step, a step being
    # its largest magnitude over 127: by at most sqrt(cols) / 254 of its norm, and as three products of them.
    cols = max(hidden, inner)
    assert all(e < 6 ** 0.5 * cols ** 0.5 / 254 for e in errors), errors


@pytest.mark.gpu
def test_gradients_of_the_layer_against_plain_torch(gpu_available):
    """The layer's gradients through the operators against the same layer in elementary operations in 64 bits."""
    import expert_layer
    torch.manual_seed(3)
    tokens, hidden, inner, experts = 40, 64, 48, 4
    model = expert_layer.ExpertLayer(hidden, inner, experts, 16, norm="layer").cuda()
    x, res = torch.randn(tokens, hidden).cuda(), torch.randn(tokens, hidden).cuda()
    d = torch.randn(tokens, 16).cuda()
    say("[calls] layer's gradients")
    params = list(model.parameters())
    got = torch.autograd.grad((model(x, res) * d).sum(), params)

    wide = [p.detach().double().cpu().requires_grad_() for p in params]
    p = dict(zip((n for n, _ in model.named_parameters()), wide))
    xs, rs = x.double().cpu(), res.double().cpu()

    def norm(v, w, b):
        c = v - v.mean(dim=1, keepdim=True)
        return c * (c.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * w + b

    s = xs + rs
    h = norm(s, p["norm"], p["norm_bias"])
    value, expert = (h @ p["router"].t()).topk(2, dim=1)
    share = value.softmax(dim=1)
    out = s
    for k in range(2):
        up, down = p["up"][expert[:, k]], p["down"][expert[:, k]]
        y = torch.nn.functional.silu((up * h[:, None, :]).sum(2))
        out = out + share[:, k:k + 1] * (down * y[:, None, :]).sum(2)
    loss = ((norm(out, p["last"], p["last_bias"]) @ p["head"][0].t()) * d.double().cpu()).sum()
    want = torch.autograd.grad(loss, wide)
    # fp32 throughout: some hundred roundings of 2^-24 in a row, on values that cancel by a factor of ten at most
    for (name, _), a, b in zip(model.named_parameters(), got, want):
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off < 1000 * 2.0 ** -24, (name, float(off))
