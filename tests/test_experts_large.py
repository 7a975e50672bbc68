"""The expert layer's operators past 2^31 elements: results at both ends of
operands and outputs whose offsets do not fit 32 bits, against 64-bit
references of those rows.  Tolerances are test_experts.py's.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_experts import BF16, F32, FP8, U16, U32, depth, f64, gen, norm64, plain_codes, product_tol, values, within

pytestmark = pytest.mark.gpu

ROWS, COLS = 262144 + 40, 8192                    # rows from 2^31 elements on


def ends_filled(rows, cols, dtype, seed):
    """rows x cols of zeros on the GPU but for the first and the last 30 rows, and those on the host."""
    t = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    head, tail = (torch.randn(30, cols, generator=gen(seed + i)).to(dtype) for i in (0, 1))
    t[:30].copy_(head)
    t[-30:].copy_(tail)
    return t, (head, tail)


def both(t):
    return t[:30], t[-30:]


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def test_norm_and_quantiser(gpu_available):
    say(f"[large] norm {ROWS}x{COLS}")
    x, xs = ends_filled(ROWS, COLS, BF16, 1)
    r, rs = ends_filled(ROWS, COLS, BF16, 3)
    w = (1 + 0.1 * torch.randn(COLS, generator=gen(5))).bfloat16()
    eps = 1e-5
    out, total, _ = tg.rms_norm(x, w.cuda(), residual=r, eps=eps)
    for o, s, a, b in zip(both(out), both(total), xs, rs):
        want = (a.float() + b.float()).bfloat16()
        assert torch.equal(s.cpu(), want)
        y = norm64(want, w, eps)
        within(o, y, y.abs() * ((depth(COLS) / 2 + 8) * U32 * (1 + U16) + U16), "norm")
    assert not out[30:-30].any()
    say("[large] quantiser")
    del out, total, r
    for rows in (1, 128):
        q, s = tg.quantize(x, rows)
        head, hs = plain_codes(xs[0] if rows == 1 else torch.cat([xs[0], torch.zeros(98, COLS, dtype=BF16)]), rows)
        assert torch.equal(q[:30].cpu().float(), head[:30].float()) and torch.equal(s[:len(hs)].cpu(), hs)
        start = ROWS - 30 if rows == 1 else ROWS // 128 * 128        # 40 rows in the last blocks of 128
        tail = x[start:].cpu()
        code, ts = plain_codes(tail, rows)
        assert torch.equal(q[start:].cpu().float(), code.float()) and torch.equal(s[-len(ts):].cpu(), ts)


def test_norm_gradients(gpu_available):
    say(f"[large] norm gradients {ROWS}x{COLS}")
    s, ss = ends_filled(ROWS, COLS, BF16, 1)
    dy, dys = ends_filled(ROWS, COLS, BF16, 3)
    w = (1 + 0.1 * torch.randn(COLS, generator=gen(5))).bfloat16()
    eps = 1e-5
    dx, dw = tg.rms_norm_backward(dy, s, w.cuda(), eps=eps)
    want_dw, size_dw = torch.zeros(COLS, dtype=torch.float64), torch.zeros(COLS, dtype=torch.float64)
    for got, a, d in zip(both(dx), map(f64, ss), map(f64, dys)):
        rr = (a.square().mean(dim=1, keepdim=True) + eps) ** -0.5
        g = d * f64(w)
        mean = (g * a).mean(dim=1, keepdim=True)
        want = rr * (g - a * rr * rr * mean)
        size = rr * (g.abs() + a.abs() * rr * rr * (g * a).abs().mean(dim=1, keepdim=True))
        within(got, want, size * (2 * depth(COLS) + 16) * U32 + want.abs() * U16 * 1.001, "dx")
        want_dw += (d * a * rr).sum(0)
        size_dw += (d * a * rr).abs().sum(0)
    within(dw, want_dw, size_dw * (60 + depth(COLS) + 20) * U32, "dweight")          # sixty terms, and zeros


def test_norm_gradients_of_long_rows(gpu_available):
    """Rows past 2^27 values: a sum over partial rows for 32 columns a workgroup is more than 2^32 threads."""
    M, N, edge = 2, 2 ** 27 + 40, 256
    say(f"[large] norm gradients {M}x{N}")
    g = gen(11)
    host = [torch.randn(M, 2 * edge, generator=g).bfloat16() for _ in range(2)]
    w0 = (1 + 0.1 * torch.randn(2 * edge, generator=g)).bfloat16()
    s, dy = (torch.zeros(M, N, dtype=BF16, device="cuda") for _ in range(2))
    w = torch.ones(N, dtype=BF16, device="cuda")
    for t, h in ((s, host[0]), (dy, host[1]), (w, w0)):
        t[..., :edge].copy_(h[..., :edge])
        t[..., -edge:].copy_(h[..., edge:])
    eps = 1e-5
    dx, dw = tg.rms_norm_backward(dy, s, w, eps=eps)
    a, d, up = f64(host[0]), f64(host[1]), f64(host[1]) * f64(w0)
    rr = (a.square().sum(dim=1, keepdim=True) / N + eps) ** -0.5
    mean = (up * a).sum(dim=1, keepdim=True) / N
    want, size = rr * (up - a * rr * rr * mean), rr * (up.abs() + a.abs() * rr * rr * (up * a).abs().sum(1, True) / N)
    got = torch.cat([dx[:, :edge], dx[:, -edge:]], dim=1)
    # (A thread adds eight values of each end, zeros between them; then the tree.)
    within(got, want, size * (2 * (16 + 26) + 16) * U32 + want.abs() * U16 * 1.001, "dx")
    within(torch.cat([dw[:edge], dw[-edge:]]), (d * a * rr).sum(0), (d * a * rr).abs().sum(0) * (2 + 16 + 26 + 20) * U32,
           "dweight")
    assert not dx[:, edge:-edge].any() and not dw[edge:-edge].any()


@pytest.mark.parametrize("op", ["T", "N"])
def test_products_of_a_large_output(gpu_available, op):
    M, N, K = 65536 + 70, 32768, 144
    say(f"[large] block op={op} {M}x{N}x{K}")
    x = torch.randn(M, K, generator=gen(1))
    qa, sa = tg.quantize(x.cuda())
    qb, sb = tg.quantize(torch.randn(*((N, K) if op == "T" else (K, N)), generator=gen(2)).cuda(), 128)
    out = tg.block_gemm(qa, qb, sa, sb, op_b=op)
    b = values(qb.cpu(), sb.cpu(), 128)
    b = b.t() if op == "T" else b
    for rows in (slice(0, 20), slice(M - 20, M)):
        a = values(qa[rows].cpu(), sa[rows].cpu(), 1)
        want = a @ b
        within(out[rows], want, product_tol(a, b, want, True, BF16), (op, rows))


def test_weight_gradients_of_a_large_output(gpu_available):
    G, M, N, K = 9, 50, 16384, 16384
    say(f"[large] wgrad {G} groups {N}x{K}")
    dy, x = torch.randn(M, N, generator=gen(1)).bfloat16(), torch.randn(M, K, generator=gen(2)).bfloat16()
    ends = torch.tensor([20] * (G - 1) + [M], dtype=torch.int32).cuda()
    dw = tg.grouped_wgrad(dy.cuda(), x.cuda(), ends)
    for g, (lo, hi) in ((0, (0, 20)), (G - 1, (20, M))):
        for rows in (slice(0, 40), slice(N - 40, N)):
            p, q = f64(dy[lo:hi, rows]), f64(x[lo:hi])
            within(dw[g, rows], p.t() @ q, (p.abs().t() @ q.abs()) * (hi - lo + 4) * U32, (g, rows))
    assert not dw[1:-1].any()
