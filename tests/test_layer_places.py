"""Layer norm in place at every shape of a row, and the passes over 32 MB and more (which use non-temporal
accesses) at widths and addresses off their 8 values."""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_layer_norm import BF16, EPS, F32, FP8, HALF, I8, SIZES, gen, gradients, inputs, within
from test_routing import case

pytestmark = pytest.mark.gpu

LARGE = 32 << 20


def same(p, q):
    return torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [300, 1500, 3000, 4104, 8192, 9001, 16384, 20001])
def test_sum_in_place(gpu_available, dtype, N):
    M = 6
    x, res, w, b = (t.cuda() for t in inputs(M, N, dtype))
    for kind in (None, BF16, I8, FP8):
        want = tg.layer_norm(x, w, b, residual=res, eps=EPS, out_dtype=kind)
        for into in ("x", "residual"):
            say(f"[places] {dtype} {M}x{N} sum over {into}, out {kind}")
            xd, rd = x.clone(), res.clone()
            got = tg.layer_norm(xd, w, b, residual=rd, eps=EPS, out_dtype=kind, summed=xd if into == "x" else rd)
            assert got[1] is (xd if into == "x" else rd) and same(got[1], want[1]) and same(got[0], want[0])
            assert (got[2] is None and want[2] is None) or same(got[2], want[2])
            assert same(rd, res) if into == "x" else same(xd, x)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,pad,offset", SIZES)
def test_gradient_in_place(gpu_available, dtype, M, N, pad, offset):
    dy, s, w, _ = (t.cuda() for t in inputs(M, N, dtype))
    ds = (torch.randn(M, N, generator=gen(5)) * 0.5).to(dtype).cuda()
    want = tg.layer_norm_backward(dy, s, w, dsum=ds, eps=EPS)
    for into in ("dy", "dsum"):
        say(f"[places] {dtype} {M}x{N} gradient over {into}")
        d, e = shifted(dy, pad, offset), shifted(ds, pad, offset)
        got = tg.layer_norm_backward(d, s, w, dsum=e, eps=EPS, dx=d if into == "dy" else e)
        assert got[0] is (d if into == "dy" else e) and all(same(p, q) for p, q in zip(got, want))
        assert same(e, ds) if into == "dy" else same(d, dy)


def shifted(t, pad, offset):
    """A copy whose rows are `pad` values further apart and start `offset` values into their memory."""
    rows, cols = t.shape
    buf = torch.zeros(rows * (cols + pad) + offset, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


WIDE = [777, 1001, 2047, 4095, 8191, 16383]


def rows_for(N, dtype):
    return LARGE // (N * dtype.itemsize) + 9


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", WIDE)
def test_large_layer_norm(gpu_available, dtype, N):
    """Rows' results are those of the same rows in calls below 32 MB, to the bit; sums within their tolerance."""
    M = rows_for(N, dtype)
    x, res, w, b = inputs(M, N, dtype)
    wd, bd, half, off = w.cuda(), b.cuda(), M // 2, None
    halves = (slice(half), slice(half, M))
    for pad, offset in ((0, 0), (5, 3)):
        say(f"[places] layer norm {dtype} {M}x{N} pad={pad} offset={offset}")
        xd, rd = shifted(x.cuda(), pad, offset), shifted(res.cuda(), pad, offset)

        def room():
            return shifted(torch.zeros(M, N, dtype=dtype, device="cuda"), pad, offset)

        for kind in (I8, None):
            want = [tg.layer_norm(xd[i], wd, bd, residual=rd[i], eps=EPS, out_dtype=kind) for i in halves]
            got = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS, out_dtype=kind, summed=room(),
                                out=None if kind else room())
            for p, q in zip(got, zip(*want)):
                assert (p is None and q[0] is None) or same(p, torch.cat(q))
        dx, dw, db = tg.layer_norm_backward(xd, got[1], wd, dsum=rd, eps=EPS, dx=room())
        assert same(dx, torch.cat([tg.layer_norm_backward(xd[i], got[1][i], wd, dsum=rd[i], eps=EPS)[0] for i in halves]))
        if off is None:
            first = dx.clone(), dw, db
            want, off = gradients(x, got[1].cpu(), w, res)
            # a team takes M / 512 rows and more, one after the other
            more = 1 + M / 512 / 96
            within(dx, want[0], off[0] + HALF[dtype] * (want[0].abs() + off[0]), "dx")
            within(dw, want[1], off[1] * more, "dw")
            within(db, want[2], off[2] * more, "db")
        else:
            assert all(same(p, q) for p, q in zip(first, (dx, dw, db)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 3)])
@pytest.mark.parametrize("N", WIDE + [20001])
def test_large_routing(gpu_available, dtype, N, pad, offset):
    """Rows handed out, together again and their gradients in one call of 32 MB and more, and in calls of a few
    hundred columns: to the bit but for the sums over columns."""
    top, groups = 2, 5
    tokens = rows_for(N, dtype) // top + 1
    say(f"[places] routing {dtype} {tokens}x{top}x{N} pad={pad} offset={offset}")
    _, place, ends = tg.expert_plan(case(tokens, top, groups, 0.1), groups)
    g = torch.Generator(device="cuda").manual_seed(N)

    def some(rows):
        return shifted(torch.randn(rows, N, device="cuda", generator=g).to(dtype), pad, offset)

    x, d, y, w = some(tokens), some(tokens), some(tokens * top), torch.rand(tokens, top, device="cuda", generator=g)
    cuts = [slice(a, min(a + 600, N)) for a in range(0, N, 600)]
    assert tokens * top * 600 * dtype.itemsize < LARGE
    out = some(tokens * top)
    tg.dispatch(x, place, ends, out=out)
    assert same(out, torch.cat([tg.dispatch(x[:, c], place, ends) for c in cuts], dim=1))
    out = some(tokens)
    tg.combine(y, place, w, d, out=out)
    assert same(out, torch.cat([tg.combine(y[:, c], place, w, d[:, c]) for c in cuts], dim=1))
    out = some(tokens * top)
    _, dw = tg.combine_backward(d, y, place, w, ends, drows=out)
    parts = [tg.combine_backward(d[:, c], y[:, c], place, w, ends) for c in cuts]
    assert same(out, torch.cat([p[0] for p in parts], dim=1))
    # sums of N products in two orders, each off by at most a chunk's, a team's and the tree's additions
    products = torch.where((place >= 0)[:, :, None], y.double()[place.clamp_min(0).long()], 0.0) * d.double()[:, None, :]
    off = (8 * -(-N // 512) + 26) * 2.0 ** -24 * products.abs().sum(dim=2)
    assert ((dw.double() - products.sum(dim=2)).abs() <= off).all()


@pytest.mark.parametrize("tokens", [1, 16])
def test_few_tokens_into_many_rows(gpu_available, tokens):
    """A buffer of a fixed number of rows: those from the last end on are cleared, and nothing else is touched."""
    rows, N, top = 3000, 1000, 2
    say(f"[places] {tokens} tokens into {rows} rows")
    _, place, ends = tg.expert_plan(torch.arange(tokens * top, device="cuda").view(tokens, top) % 7, 7)
    x, scales = torch.randn(tokens, N, device="cuda").bfloat16(), torch.rand(tokens, device="cuda")
    buf = torch.full((rows + 2, N), 5.0, device="cuda").bfloat16()
    moved = torch.full((rows,), 5.0, device="cuda")
    tg.dispatch(x, place, ends, scales=scales, out=buf[1:-1], out_scales=moved)
    assert (buf[0] == 5).all() and (buf[-1] == 5).all()
    for t in range(tokens):
        for k in range(top):
            assert same(buf[1 + int(place[t, k])], x[t]) and moved[int(place[t, k])] == scales[t]
    assert (buf[1 + tokens * top:-1] == 0).all() and (moved[tokens * top:] == 0).all()
    drows = torch.full((rows, N), 5.0, device="cuda").bfloat16()
    weights = torch.rand(tokens, top, device="cuda")
    tg.combine_backward(x, buf[1:-1], place, weights, ends, drows=drows)
    assert (drows[tokens * top:] == 0).all() and (drows[:tokens * top] != 5).any(dim=1).all()
