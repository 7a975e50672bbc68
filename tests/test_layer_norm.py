"""Layer norm on the GPU against 64 bits.

Tolerances count roundings.  A sum of n fp32 terms in a tree of depth d is off
by at most d * 2^-24 of the sum of magnitudes; a rounding to bf16 by 2^-8 of
the value, to e4m3 by 2^-4 of it.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U32, U16, U8 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
FP8, BF16, F32, I8 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int8
HALF = {F32: 0.0, BF16: U16}
EPS = 1e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def padded(t, pad=0, offset=0):
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset + 1,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def f64(t):
    return t.detach().to(device="cpu").to(torch.float64)


def within(got, want, tol, what):
    got, want = f64(got), f64(want)
    off = (got - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300))[bad].max()))


def depth(N):
    """Additions in a row's sum, at most: 8 values a chunk, a chunk for each 512 columns, then the tree."""
    return 8 * -(-N // 512) + 26


def parts(s):
    """(s - mean, r, error of s - mean, relative error of r) of rows in 64 bits."""
    s, N = f64(s), s.shape[1]
    mean = s.mean(dim=1, keepdim=True)
    c = s - mean
    var = c.square().mean(dim=1, keepdim=True)
    r = (var + EPS).rsqrt()
    # the mean: a sum and a quotient; the difference: one rounding more
    off = (depth(N) + 2) * U32 * s.abs().mean(dim=1, keepdim=True) + U32 * c.abs()
    # the variance: 2 |c| off a term (the mean's own part of off cancels to first order, and is counted all the
    # same), a square and the sum; r: half of that and a quotient, a sum, a root and a reciprocal
    var_off = (2 * c.abs() * off + off.square()).mean(dim=1, keepdim=True) + (depth(N) + 2) * U32 * var
    return c, r, off, 0.5 * var_off / (var + EPS) + 4 * U32


SIZES = [(1, 1, 0, 0), (3, 7, 1, 0), (5, 128, 0, 0), (2, 777, 0, 1), (4, 1024, 8, 0), (3, 1025, 0, 0), (2, 4096, 0, 0),
         (3, 4104, 8, 8), (2, 8192, 0, 0), (2, 8193, 3, 0), (1, 16384, 0, 0), (2, 20001, 0, 0), (1030, 33, 0, 0)]


def inputs(M, N, dtype, seed=0):
    g = gen(M * 7 + N + seed)
    x = torch.randn(M, N, generator=g).to(dtype)
    res = (torch.randn(M, N, generator=g) * 2 + torch.randn(M, 1, generator=g) * 3).to(dtype)
    w = (1 + 0.2 * torch.randn(N, generator=g)).to(dtype)
    b = (0.3 * torch.randn(N, generator=g)).to(dtype)
    return x, res, w, b


def reference(s, w, b):
    """(y, how far off fp32 may be) in 64 bits."""
    c, r, off, rel = parts(s)
    w = f64(w)
    unit = c * r
    y = unit * w + (f64(b) if b is not None else 0.0)
    tol = ((off * r + unit.abs() * (rel + 2 * U32)) * w.abs() + U32 * y.abs()) * (1 + 2.0 ** -10) + 1e-30
    return y, tol


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,pad,offset", SIZES)
def test_forward(gpu_available, dtype, M, N, pad, offset):
    x, res, w, b = inputs(M, N, dtype)
    xd, rd, wd, bd = padded(x, pad, offset), padded(res, pad, offset), w.cuda(), b.cuda()
    for with_res, with_bias, out_dtype in ((True, True, dtype), (False, True, F32), (True, False, BF16)):
        say(f"[layer norm] {dtype} {M}x{N} pad={pad} residual={with_res} bias={with_bias} out={out_dtype}")
        out, summed, none = tg.layer_norm(xd, wd, bd if with_bias else None, residual=rd if with_res else None,
                                          eps=EPS, out_dtype=out_dtype)
        assert none is None and out.dtype == out_dtype
        s = (x.float() + res.float()).to(dtype) if with_res else x
        assert torch.equal(summed.cpu(), s) and (with_res or summed is xd)
        y, tol = reference(s, w, b if with_bias else None)
        within(out, y, tol + HALF[out_dtype] * (y.abs() + tol), "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,pad,offset", SIZES)
def test_codes(gpu_available, dtype, M, N, pad, offset):
    x, res, w, b = inputs(M, N, dtype)
    xd, rd, wd, bd = padded(x, pad, offset), padded(res, pad, offset), w.cuda(), b.cuda()
    s = (x.float() + res.float()).to(dtype)
    y, tol = reference(s, w, b)
    say(f"[layer norm] int8 {dtype} {M}x{N} pad={pad}")
    codes, summed, scales = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS, out_dtype=I8)
    assert torch.equal(summed.cpu(), s) and codes.dtype == I8 and scales.shape == (M,)
    top = y.abs().amax(dim=1)
    within(scales, top / 127, (tol.amax(dim=1) + 2 * U32 * top) / 127, "int8 scales")
    # a code is off by half of a step, y by its tolerance, and the scale by its own
    step = f64(scales)[:, None]
    within(f64(codes) * step, y, 0.5 * step * (1 + 2.0 ** -10) + tol + 4 * U32 * y.abs(), "int8 values")
    assert f64(codes).abs().amax(dim=1).eq(127).all()
    say(f"[layer norm] fp8 {dtype} {M}x{N} pad={pad}")
    codes, summed, scales = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS, out_dtype=FP8)
    assert codes.dtype == FP8 and scales.shape == (M, -(-N // 128))
    wide = f64(scales).repeat_interleave(128, dim=1)[:, :N]
    within(f64(codes.float()) * wide, y, U8 * (y.abs() + tol) + 2.0 ** -10 * wide + tol + 4 * U32 * y.abs(), "fp8 values")


def test_large_mean(gpu_available):
    """A mean a thousand times the deviation: a difference of squares would lose it."""
    for N in (100, 1000, 4000, 8000, 16000, 20000):
        say(f"[layer norm] large mean {N}")
        s = 1000.0 + torch.randn(3, N, generator=gen(N))
        out, _, _ = tg.layer_norm(s.cuda(), torch.ones(N).cuda(), eps=EPS)
        y, tol = reference(s, torch.ones(N), None)
        within(out, y, tol, "y")
        assert float(tol.max()) < 0.05 * float(y.abs().max())


def test_in_place_and_special_rows(gpu_available):
    M, N = 5, 300
    x, res, w, b = inputs(M, N, F32)
    x[1], res[1] = 3.0, 0.0                 # no deviation: y is the bias
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    for dtype in (F32, BF16):
        for into in ("x", "residual", "scales"):
            say(f"[layer norm] in place {dtype} {into}")
            xd, rd, wd, bd = (t.to(dtype).cuda() for t in (x, res, w, b))
            want = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS)
            got = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS, summed={"x": xd, "residual": rd}.get(into),
                                out=torch.empty_like(xd))
            for p, q in zip(want[:2], got[:2]):
                assert torch.equal(p.nan_to_num(9.0), q.nan_to_num(9.0)) and torch.equal(p.isnan(), q.isnan())
            assert torch.equal(got[0][1], bd) and got[0][2:4].isnan().all() and got[0][[0, 4]].isfinite().all()
        codes, _, scales = tg.layer_norm(x.to(dtype).cuda(), w.to(dtype).cuda(), b.to(dtype).cuda(),
                                         residual=res.to(dtype).cuda(), out_dtype=I8)
        assert scales[2:4].isnan().all() and (codes[2:4] == 0).all() and scales[[0, 1, 4]].isfinite().all()


def gradients(dy, s, w, ds):
    """(dx, dw, db) and how far off fp32 may be, in 64 bits."""
    M, N = s.shape
    c, r, off, rel = parts(s)
    dy, w = f64(dy), f64(w)
    ds = f64(ds) if ds is not None else torch.zeros(M, N, dtype=torch.float64)
    n, g = c * r, dy * w
    n_off = off * r + n.abs() * (rel + U32)
    gm, gn = g.mean(dim=1, keepdim=True), (g * n).mean(dim=1, keepdim=True)
    dx = r * (g - gm - n * gn) + ds
    D = depth(N) + 4
    gm_off = D * U32 * g.abs().mean(dim=1, keepdim=True)
    gn_off = (g.abs() * n_off).mean(dim=1, keepdim=True) + gn.abs() * rel + D * U32 * (g * n).abs().mean(dim=1, keepdim=True)
    inner = U32 * 3 * (g.abs() + gm.abs() + (n * gn).abs()) + gm_off + n.abs() * gn_off + n_off * gn.abs()
    dx_off = r * (inner + (rel + U32) * (g - gm - n * gn).abs()) + U32 * dx.abs()
    # sums over rows: at most as many additions as rows, and those of the tree over partial sums
    R = min(M, 32) + 64
    dw_off = (dy.abs() * n_off).sum(dim=0) + R * U32 * (dy * n).abs().sum(dim=0)
    db_off = R * U32 * dy.abs().sum(dim=0)
    return (dx, (dy * n).sum(dim=0), dy.sum(dim=0)), (2 * dx_off + 1e-30, 2 * dw_off + 1e-30, db_off + 1e-30)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,pad,offset", SIZES + [(2600, 40, 0, 0), (2200, 1100, 0, 0), (1600, 2100, 0, 0), (1100, 4100, 0, 0),
                                                    (9, 2048, 0, 0), (3, 2049, 1, 1),
                                                    (1030, 8200, 0, 0)])
def test_backward(gpu_available, dtype, M, N, pad, offset):
    x, s, w, _ = inputs(M, N, dtype)
    dy, ds = x, (torch.randn(M, N, generator=gen(5)) * 0.5).to(dtype)
    for with_ds in (True, False):
        say(f"[layer norm] backward {dtype} {M}x{N} pad={pad} ds={with_ds}")
        args = padded(dy, pad, offset), padded(s, pad, offset), w.cuda()
        dsd = padded(ds, pad, offset) if with_ds else None
        got = tg.layer_norm_backward(*args, dsum=dsd, eps=EPS)
        want, tol = gradients(dy, s, w, ds if with_ds else None)
        half = HALF[dtype]
        within(got[0], want[0], tol[0] + half * (want[0].abs() + tol[0]), "dx")
        within(got[1], want[1], tol[1], "dw")
        within(got[2], want[2], tol[2], "db")
        again = tg.layer_norm_backward(*args, dsum=dsd, eps=EPS)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
    # one gradient without the other, and in place of dy and of dsum
    only = tg.layer_norm_backward(*args, eps=EPS, want_dweight=False)
    assert only[1] is None and torch.equal(only[0], got[0]) and torch.equal(only[2], got[2])
    only = tg.layer_norm_backward(*args, eps=EPS, want_dbias=False)
    assert only[2] is None and torch.equal(only[0], got[0]) and torch.equal(only[1], got[1])
    none = tg.layer_norm_backward(*args, eps=EPS, want_dweight=False, want_dbias=False, dx=args[0])
    assert none[1] is None and none[2] is None and torch.equal(none[0], got[0]) and none[0] is args[0]


# Operands of 32 MB and more, in every shape of a row: passes that go past the L2.
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [1000, 1024, 2048, 4000, 8192, 16384])
def test_large_passes(gpu_available, dtype, N):
    M = 2 ** 25 // (4 if dtype == F32 else 2) // N + 70
    say(f"[layer norm] large {dtype} {M}x{N}")
    x, res, w, b = inputs(M, N, dtype)
    xd, rd, wd, bd = x.cuda(), res.cuda(), w.cuda(), b.cuda()
    s = (x.float() + res.float()).to(dtype)
    y, tol = reference(s, w, b)
    out, summed, _ = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS)
    assert torch.equal(summed.cpu(), s)
    within(out, y, tol + HALF[dtype] * (y.abs() + tol), "y")
    codes, summed, scales = tg.layer_norm(xd, wd, bd, residual=rd, eps=EPS, out_dtype=I8)
    assert torch.equal(summed.cpu(), s)
    step = f64(scales)[:, None]
    within(f64(codes) * step, y, 0.5 * step * (1 + 2.0 ** -10) + tol + 4 * U32 * y.abs(), "int8 values")
    want, off = gradients(x, s, w, res)
    got = tg.layer_norm_backward(xd, summed, wd, dsum=rd, eps=EPS)
    # a team takes M / 512 rows and more, one after the other
    more = 1 + M / 512 / 96
    within(got[0], want[0], off[0] + HALF[dtype] * (want[0].abs() + off[0]), "dx")
    within(got[1], want[1], off[1] * more, "dw")
    within(got[2], want[2], off[2] * more, "db")


def test_gradients_against_differences(gpu_available):
    M, N, h = 4, 37, 1e-2
    x, _, w, b = (t.double() for t in inputs(M, N, F32))
    x = x.float().double()
    d = torch.randn(M, N, generator=gen(3)).double().float().double()

    def loss(x, w, b):
        c = x - x.mean(dim=1, keepdim=True)
        return ((c * (c.square().mean(dim=1, keepdim=True) + EPS).rsqrt() * w + b) * d).sum()

    say("[layer norm] against differences")
    dx, dw, db = tg.layer_norm_backward(d.float().cuda(), x.float().cuda(), w.float().cuda(), eps=EPS)
    for got, at in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w.float().double(), b]
        for i in range(0, args[at].numel(), 5):
            step = torch.zeros(args[at].numel(), dtype=torch.float64)
            step[i] = h
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + step.view_as(args[at]), args[at] - step.view_as(args[at])
            far, near = (float(loss(*up) - loss(*down)) / (2 * h), None)
            half_up, half_down = list(args), list(args)
            half_up[at], half_down[at] = args[at] + step.view_as(args[at]) / 2, args[at] - step.view_as(args[at]) / 2
            near = float(loss(*half_up) - loss(*half_down)) / h
            # the quotient at half the step is off by about a third of how far the two are apart
            assert abs(float(got.flatten()[i]) - near) <= abs(far - near) + 1e-4 * (1 + abs(near)), (at, i)


def test_empty_and_refused(gpu_available):
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    say("[layer norm] empty calls")
    out, summed, _ = tg.layer_norm(f(0, 8), f(8), f(8))
    assert out.shape == (0, 8)
    dx, dw, db = tg.layer_norm_backward(f(0, 8), f(0, 8), f(8))
    assert dx.shape == (0, 8) and (dw == 0).all() and (db == 0).all()
    assert tg.layer_norm(f(4, 0), f(0))[0].shape == (4, 0)
    for error, call in [
            (TypeError, lambda: tg.layer_norm(f(4, 8).half(), f(8))), (ValueError, lambda: tg.layer_norm(f(8), f(8))),
            (ValueError, lambda: tg.layer_norm(f(4, 8), f(7))), (TypeError, lambda: tg.layer_norm(f(4, 8), f(8).bfloat16())),
            (ValueError, lambda: tg.layer_norm(f(4, 8), f(8), f(9))), (ValueError, lambda: tg.layer_norm(f(4, 8), f(16)[::2])),
            (ValueError, lambda: tg.layer_norm(f(4, 8), f(8), f(16)[::2])),
            (ValueError, lambda: tg.layer_norm(f(4, 8), f(8), residual=f(4, 9))),
            (ValueError, lambda: tg.layer_norm(f(8, 4).t(), f(8))), (ValueError, lambda: tg.layer_norm(f(4, 8).cpu(), f(8))),
            (ValueError, lambda: tg.layer_norm(f(4, 8), f(8), scales=f(4))),
            (ValueError, lambda: tg.layer_norm(f(4, 8), f(8), out_dtype=I8, scales=f(4, 1))),
            (TypeError, lambda: tg.layer_norm(f(4, 8), f(8), out_dtype=torch.int32)),
            (TypeError, lambda: tg.layer_norm(f(4, 8), f(8), out=f(4, 8), out_dtype=BF16)),
            (tg.GemmError, lambda: tg.layer_norm(f(4, 8), f(8), eps=-1.0)),
            (ValueError, lambda: tg.layer_norm_backward(f(4, 8), f(4, 9), f(8))),
            (TypeError, lambda: tg.layer_norm_backward(f(4, 8), f(4, 8).bfloat16(), f(8))),
            (ValueError, lambda: tg.layer_norm_backward(f(4, 8), f(4, 8), f(8), dsum=f(3, 8)))]:
        with pytest.raises(error):
            call()
