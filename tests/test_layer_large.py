"""Layer norm, 8-bit products and the routing past 2^31 elements: results whose
offsets do not fit 32 bits."""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_int8 import codes, exact, gen
from test_int8 import within as int8_within
from test_layer_norm import BF16, EPS, F32, I8, U16, gradients, reference, within

pytestmark = pytest.mark.gpu

ROWS, COLS = 262144 + 40, 8192                    # rows from 2^31 elements on


@pytest.fixture(autouse=True)
def freed():
    yield
    torch.cuda.empty_cache()


def ends_filled(rows, cols, dtype, seed):
    """rows x cols of zeros on the GPU but for the first and the last 30 rows, and those on the host."""
    t = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    head, tail = (torch.randn(30, cols, generator=gen(seed + i)).to(dtype) for i in (0, 1))
    t[:30].copy_(head)
    t[-30:].copy_(tail)
    return t, (head, tail)


def both(t):
    return t[:30], t[-30:]


def test_layer_norm(gpu_available):
    say(f"[large] layer norm {ROWS}x{COLS}")
    x, xs = ends_filled(ROWS, COLS, BF16, 1)
    r, rs = ends_filled(ROWS, COLS, BF16, 3)
    w, b = (1 + 0.1 * torch.randn(COLS, generator=gen(5))).bfloat16(), torch.randn(COLS, generator=gen(6)).bfloat16()
    for out_dtype in (BF16, I8):
        out, total, scales = tg.layer_norm(x, w.cuda(), b.cuda(), residual=r, eps=EPS, out_dtype=out_dtype)
        for i, (o, s, p, q) in enumerate(zip(both(out), both(total), xs, rs)):
            want = (p.float() + q.float()).bfloat16()
            assert torch.equal(s.cpu(), want)
            y, tol = reference(want, w, b)
            if out_dtype is BF16:
                within(o, y, tol + U16 * (y.abs() + tol), "y")
            else:
                step = both(scales)[i].cpu().double()[:, None]
                within(o.cpu().double() * step, y, 0.5 * step * (1 + 2.0 ** -10) + tol + 2.0 ** -22 * y.abs(), "codes")
        del out, total
    say(f"[large] layer norm gradients {ROWS}x{COLS}")
    dx, dw, db = tg.layer_norm_backward(r, x, w.cuda(), eps=EPS)
    parts = [gradients(dy, s, w, None) for dy, s in zip(rs, xs)]
    for got, (want, tol) in zip(both(dx), parts):
        within(got, want[0], tol[0] + U16 * (want[0].abs() + tol[0]), "dx")
    # sixty terms and zeros, which add nothing
    within(dw, parts[0][0][1] + parts[1][0][1], 2 * (parts[0][1][1] + parts[1][1][1]), "dw")
    within(db, parts[0][0][2] + parts[1][0][2], 2 * (parts[0][1][2] + parts[1][1][2]), "db")


def test_rows_and_products(gpu_available):
    say(f"[large] int8 rows {ROWS}x{COLS}")
    x, xs = ends_filled(ROWS, COLS, BF16, 1)
    q, s = tg.quantize_int8(x)
    for got, scale, want in zip(both(q), both(s), xs):
        top = want.float().abs().amax(dim=1)
        assert torch.equal(scale.cpu(), top / 127)
        assert torch.equal(got.cpu(), (want.float() * (torch.tensor(127.0) / top)[:, None]).round().to(I8))
    assert not q[30:-30].any()
    del x, q
    M, N, K = 65536 + 70, 32768, 144
    for op in "TN":
        say(f"[large] int8 op={op} {M}x{N}x{K}")
        a, b = codes(1, M, K), codes(2, *((N, K) if op == "T" else (K, N)))
        sa, sb = torch.rand(M, generator=gen(1)), torch.rand(N, generator=gen(2))
        out = tg.int8_gemm(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), op_b=op)
        for rows in (slice(0, 20), slice(M - 20, M)):
            int8_within(out[rows], *exact(a[rows], b, sa[rows], sb, None, op, BF16), (op, rows))
        del out


def test_routing(gpu_available):
    tokens, top, cols = 33000, 8, 8192                    # 2.16e9 values handed out
    say(f"[large] routing {tokens} x {top} x {cols}")
    experts = torch.randn(tokens, 64, generator=gen(1)).topk(top, dim=1)[1].cuda()
    order, place, ends = tg.expert_plan(experts, 64)
    x = torch.randn(tokens, cols, generator=gen(2)).bfloat16().cuda()
    rows = tg.dispatch(x, place, ends)
    assert rows.numel() > 2 ** 31
    for lo in range(0, tokens * top, 50000):
        here = order[lo:lo + 50000].long()
        assert torch.equal(rows[lo:lo + 50000], x[here // top])
    out = tg.combine(rows, place)
    assert torch.equal(out, (8 * x.float()).bfloat16())            # eight equal terms: exact
    weights = torch.full((tokens, top), 0.5, device="cuda")
    drows, dw = tg.combine_backward(x, rows, place, weights, ends)
    for lo in range(0, tokens * top, 50000):
        assert torch.equal(drows[lo:lo + 50000], (0.5 * rows[lo:lo + 50000].float()).bfloat16())
    want = x.double().square().sum(dim=1, keepdim=True).expand(tokens, top)
    within(dw, want.cpu(), want.cpu() * (8 * 16 + 26) * 2.0 ** -24, "dweights")
    last = torch.tensor([tokens * top - 3], dtype=torch.int32, device="cuda")
    tg.dispatch(x, place, last, out=rows)
    assert not rows[-3:].any() and rows[-4].any()
