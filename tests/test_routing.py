"""Tokens sorted by expert and back, on the GPU against plain forms.

The plan and the rows handed out are exact.  A combined value is off by at most
(top + 1) * 2^-24 of the sum of its terms' magnitudes, a weight's gradient by
the additions in a row's sum, a rounding to bf16 by 2^-8 of the value.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
FP8, BF16, F32, I8 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int8
HALF = {F32: 0.0, BF16: U16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().to(device="cpu").to(torch.float64)


def within(got, want, tol, what):
    off = (f64(got) - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def padded(t, pad=0, offset=0):
    rows, cols = t.shape
    raw = t.view(torch.uint8) if t.dtype == FP8 else t
    fill = float("nan") if raw.is_floating_point() else 0x7F
    buf = torch.full((rows * (cols + pad) + offset + 1,), fill, dtype=raw.dtype, device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(raw)
    return view.view(t.dtype) if t.dtype == FP8 else view


def plain_plan(experts, groups):
    flat = experts.flatten().tolist()
    order = [i for g in range(groups) for i in [j for j, e in enumerate(flat) if e == g]] if len(flat) * groups < 3e6 else None
    if order is None:
        key = torch.tensor([e if 0 <= e < groups else groups for e in flat])
        used = int((key < groups).sum())
        order = key.argsort(stable=True)[:used].tolist()
    place = [-1] * len(flat)
    for row, i in enumerate(order):
        place[i] = row
    counts = [0] * groups
    for e in flat:
        if 0 <= e < groups:
            counts[e] += 1
    ends = torch.tensor(counts).cumsum(0).to(torch.int32)
    order = order + [-1] * (len(flat) - len(order))
    return torch.tensor(order, dtype=torch.int32), torch.tensor(place, dtype=torch.int32).view(experts.shape), ends


PLANS = [(1, 1, 1), (1, 3, 5), (3, 1, 2), (16, 4, 32), (64, 1, 64), (65, 2, 65), (100, 8, 128), (1000, 3, 7), (1024, 8, 8),
         (1025, 8, 8), (5000, 2, 256), (777, 11, 769), (3000, 4, 1500), (2000, 5, 4096), (20000, 8, 16), (70001, 1, 300),
         (40, 70, 3000)]


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,top,groups", PLANS)
def test_plan(gpu_available, dtype, tokens, top, groups):
    for kind in ("spread", "dropped", "one", "none"):
        say(f"[plan] {tokens} x {top} of {groups} {dtype} {kind}")
        experts = torch.randint(0, groups, (tokens, top), generator=gen(tokens + top), dtype=dtype)
        if kind == "dropped":
            gone = torch.rand(tokens, top, generator=gen(1))
            experts[gone < 0.2] = -1
            experts[gone > 0.8] = groups
            experts[(gone > 0.4) & (gone < 0.45)] = torch.iinfo(dtype).max
            experts[(gone > 0.5) & (gone < 0.55)] = torch.iinfo(dtype).min
            if dtype is torch.int64:
                experts[(gone > 0.6) & (gone < 0.65)] = 1 << 32          # whose lower half is a group
        elif kind == "one":
            experts[:] = groups - 1
        elif kind == "none":
            experts[:] = -7
        wide = torch.full((tokens, top + 3), 0, dtype=dtype, device="cuda")
        wide[:, 1:top + 1] = experts.cuda()
        want = plain_plan(experts, groups)
        for arg in (experts.cuda(), wide[:, 1:top + 1]):
            got = tg.expert_plan(arg, groups)
            for g, w, what in zip(got, want, ("order", "place", "ends")):
                assert g.dtype == torch.int32 and torch.equal(g.cpu(), w), (what, kind)


COLS = [1, 3, 8, 15, 16, 33, 257, 512, 1000, 1024, 1025, 2048, 4096, 4100, 8192, 8200, 16400]


def case(tokens, top, groups, dropped=0.3, seed=0):
    experts = torch.randint(0, groups, (tokens, top), generator=gen(tokens + seed))
    experts[torch.rand(tokens, top, generator=gen(seed + 9)) < dropped] = -1
    return experts.cuda()


@pytest.mark.parametrize("dtype", [F32, BF16, FP8, I8])
@pytest.mark.parametrize("cols", COLS)
def test_dispatch(gpu_available, dtype, cols):
    for tokens, top, groups, pad, offset in ((1, 1, 1, 0, 0), (37, 3, 5, 3, 1), (300, 8, 16, 16, 0)):
        say(f"[dispatch] {dtype} {tokens} x {cols} top={top} pad={pad}")
        x = torch.randint(0, 256, (tokens, cols * torch.empty(0, dtype=dtype).element_size()), generator=gen(cols),
                          dtype=torch.uint8).view(dtype)         # any bits, NaN among them
        _, place, ends = tg.expert_plan(case(tokens, top, groups), groups)
        xd = padded(x, pad, offset)
        rows = tg.dispatch(xd, place, ends)
        assert rows.shape == (tokens * top, cols) and rows.dtype == dtype
        want = torch.zeros(tokens * top, cols, dtype=dtype)
        bits = lambda t: t.cpu().contiguous().view(torch.uint8)  # noqa: E731
        flat = place.cpu().flatten()
        have = flat >= 0
        token = torch.arange(tokens).repeat_interleave(top)
        want.view(torch.uint8)[flat[have].long()] = x.view(torch.uint8)[token[have]]
        assert torch.equal(bits(rows), bits(want))
        # into the caller's tensor: fewer and more rows than choices, its padding left alone; scales along
        for n in (max(1, tokens * top // 2), tokens * top + 5):
            out = padded(torch.ones(n, cols).to(dtype), 5, 0)
            back = out.as_strided((n, cols + 5), (cols + 5, 1)).view(torch.uint8).view(n, -1)
            for shape in ((tokens,), (tokens, 3)):
                scales = torch.rand(shape, generator=gen(2))
                got, moved = tg.dispatch(xd, place, ends, scales=scales.cuda(), out=out)
                assert got is out and moved.shape == (n, *shape[1:])
                both = min(n, tokens * top)
                assert torch.equal(bits(out)[:both], bits(want)[:both])
                assert (bits(out)[int(ends[-1]):] == 0).all() and (moved[int(ends[-1]):] == 0).all()
                sent = torch.zeros(tokens * top, *shape[1:])
                sent[flat[have].long()] = scales[token[have]]
                assert torch.equal(moved.cpu()[:both], sent[:both])
            wide = cols * x.element_size()
            assert torch.equal(back[:, wide:].cpu(), bits(padded(torch.zeros(n, cols).to(dtype), 5, 0).as_strided(
                (n, cols + 5), (cols + 5, 1)))[:, wide:])


def of_choices(rows, place):
    each = f64(rows)[place.cpu().clamp_min(0).long()]
    return torch.where((place.cpu() >= 0)[:, :, None], each, torch.zeros((), dtype=torch.float64))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", COLS)
def test_combine(gpu_available, dtype, cols):
    for tokens, top, groups, pad, offset in ((1, 1, 1, 0, 0), (37, 3, 5, 3, 1), (130, 9, 16, 8, 0), (7, 131, 16, 0, 0)):
        _, place, ends = tg.expert_plan(case(tokens, top, groups), groups)
        g = gen(cols + tokens)
        rows = torch.randn(tokens * top, cols, generator=g).to(dtype)
        rows[int(ends[-1]):] = float("nan")                        # no choice reads these
        weights = torch.rand(tokens, top, generator=g)
        weights[place.cpu() < 0] = float("nan")                    # nor are these used
        res = torch.randn(tokens, cols, generator=g).to(dtype)
        for with_w, with_res in ((True, True), (False, False), (True, False), (False, True)):
            say(f"[combine] {dtype} {tokens} x {cols} top={top} pad={pad} weights={with_w} residual={with_res}")
            resd = padded(res, pad, offset) if with_res else None
            out = tg.combine(padded(rows, pad, offset), place, weights=padded(weights, 2) if with_w else None,
                             residual=resd)
            terms = of_choices(rows, place) * (f64(weights).nan_to_num(0.0)[:, :, None] if with_w else 1.0)
            start = f64(res) if with_res else torch.zeros(tokens, cols, dtype=torch.float64)
            want = start + terms.sum(dim=1)
            tol = (top + 1) * U32 * (start.abs() + terms.abs().sum(dim=1)) * (1 + U16)
            within(out, want, tol + HALF[dtype] * (want.abs() + tol), "out")
            if with_res:
                again = tg.combine(padded(rows, pad, offset), place, weights=padded(weights, 2) if with_w else None,
                                   residual=resd, out=resd)
                assert again is resd and torch.equal(again, out)


def depth(N):
    return 8 * -(-N // 512) + 26


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", COLS)
def test_combine_backward(gpu_available, dtype, cols):
    for tokens, top, groups, pad, offset in ((1, 1, 1, 0, 0), (37, 3, 5, 3, 1), (60, 67, 16, 8, 0)):
        say(f"[combine backward] {dtype} {tokens} x {cols} top={top} pad={pad}")
        _, place, ends = tg.expert_plan(case(tokens, top, groups), groups)
        g = gen(cols + tokens)
        rows = torch.randn(tokens * top, cols, generator=g).to(dtype)
        rows[int(ends[-1]):] = float("nan")
        weights, dout = torch.rand(tokens, top, generator=g), torch.randn(tokens, cols, generator=g).to(dtype)
        args = padded(dout, pad, offset), padded(rows, pad, offset), place, padded(weights, 2), ends
        drows, dweights = tg.combine_backward(*args)
        each = of_choices(rows, place)
        products = each * f64(dout)[:, None, :]
        tol = depth(cols) * U32 * products.abs().sum(dim=2) * (1 + U16)
        within(dweights, products.sum(dim=2), tol, "dweights")
        assert (dweights.cpu()[place.cpu() < 0] == 0).all()
        want = torch.zeros(tokens * top, cols, dtype=torch.float64)
        flat, have = place.cpu().flatten().long(), place.cpu().flatten() >= 0
        value = (f64(weights)[:, :, None] * f64(dout)[:, None, :]).view(tokens * top, cols)
        want[flat[have]] = value[have]
        within(drows, want, (U32 + HALF[dtype] * (1 + U16)) * want.abs() * (1 + U16) + 1e-45, "drows")
        assert (drows[int(ends[-1]):] == 0).all()
        only, none = tg.combine_backward(*args, want_dweights=False)
        assert none is None and torch.equal(only, drows)
        again, dw = tg.combine_backward(*args, drows=args[1])                  # over the rows themselves
        assert again is args[1] and torch.equal(again, drows) and torch.equal(dw, dweights)


# Rows of 32 MB and more in all, which go past the L2, and of less in as many waves.
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,top,cols", [(5000, 1, 1000), (9000, 2, 1000), (2500, 2, 4000), (1300, 2, 8000), (700, 3, 16400)])
def test_many_rows(gpu_available, dtype, tokens, top, cols):
    say(f"[routing] many rows {dtype} {tokens} x {top} x {cols}")
    order, place, ends = tg.expert_plan(case(tokens, top, 20, 0.1), 20)
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, d = (torch.randn(tokens, cols, device="cuda", generator=g).to(dtype) for _ in range(2))
    w = torch.rand(tokens, top, device="cuda", generator=g)
    rows = tg.dispatch(x, place, ends)
    token, have = order.clamp_min(0).long() // top, (order >= 0)[:, None]
    assert torch.equal(rows, torch.where(have, x[token], torch.zeros((), dtype=dtype, device="cuda")))
    each = torch.where((place >= 0)[:, :, None], rows[place.clamp_min(0).long()].double(), torch.zeros((), device="cuda").double())
    terms = each * w.double()[:, :, None]
    want = d.double() + terms.sum(dim=1)
    tol = (top + 1) * U32 * (d.double().abs() + terms.abs().sum(dim=1)) * (1 + U16)
    got = tg.combine(rows, place, w, d)
    assert ((got.double() - want).abs() <= tol + HALF[dtype] * (want.abs() + tol)).all()
    drows, dw = tg.combine_backward(d, rows, place, w, ends)
    value = torch.where(have, w.flatten()[order.clamp_min(0).long()].double()[:, None] * d[token].double(), 0.0)
    assert ((drows.double() - value).abs() <= (U32 + HALF[dtype] * (1 + U16)) * value.abs() * (1 + U16) + 1e-45).all()
    products = each * d.double()[:, None, :]
    assert ((dw.double() - products.sum(dim=2)).abs() <= depth(cols) * U32 * products.abs().sum(dim=2) * (1 + U16)).all()


def test_gradients_against_differences(gpu_available):
    """combine(f(dispatch(x))) with f one weight a row, its gradients through the operators against differences."""
    tokens, top, groups, cols, h = 6, 3, 4, 20, 0.25
    experts = case(tokens, top, groups, 0.2)
    _, place, ends = tg.expert_plan(experts, groups)
    g = gen(4)
    x, w = torch.randn(tokens, cols, generator=g), torch.rand(tokens, top, generator=g)
    gain, d = torch.rand(tokens * top, 1, generator=g) + 0.5, torch.randn(tokens, cols, generator=g)

    def loss(x, w):
        p = place.cpu()
        each = x[:, None, :] * gain.double()[p.clamp_min(0).long()] * w[:, :, None]
        out = x + torch.where((p >= 0)[:, :, None], each, torch.zeros((), dtype=torch.float64)).sum(dim=1)
        return (out * d.double()).sum()

    say("[routing] against differences")
    xd, wd, dd = x.cuda(), w.cuda(), d.cuda()
    y = tg.dispatch(xd, place, ends) * gain.cuda()
    dy, dw = tg.combine_backward(dd, y, place, wd, ends)
    dx = tg.combine(dy * gain.cuda(), place, residual=dd)
    for got, at in ((dx, 0), (dw, 1)):
        args = [x.double(), w.double()]
        for i in range(args[at].numel()):
            step = torch.zeros(args[at].numel(), dtype=torch.float64)
            step[i] = h
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + step.view_as(args[at]), args[at] - step.view_as(args[at])
            # linear in x and in w: the quotient is the gradient but for fp32's roundings
            want = float(loss(*up) - loss(*down)) / (2 * h)
            assert abs(float(got.flatten()[i]) - want) <= 1e-5 * (1 + abs(want)), (at, i)


def test_bad_places_touch_nothing(gpu_available):
    """Places past the rows, and past the last end, are no rows."""
    tokens, top, cols, n = 8, 2, 40, 10
    place = torch.tensor([[0, 10], [1, -5], [2, 1 << 30], [3, 11], [-(1 << 31), 4], [9, 5], [6, 2 ** 31 - 1], [7, 8]],
                         dtype=torch.int32).cuda()
    x = torch.randn(tokens, cols, generator=gen(1)).cuda()
    for last in (10, 6, 0, -3, 1000):
        say(f"[routing] bad places, last end {last}")
        ends = torch.tensor([last], dtype=torch.int32).cuda()
        used = min(max(last, 0), n)
        buf = torch.full((n + 2, cols), 5.0).cuda()
        tg.dispatch(x, place, ends, out=buf[1:n + 1])
        assert (buf[0] == 5).all() and (buf[n + 1] == 5).all() and (buf[1 + used:n + 1] == 0).all()
        for t in range(tokens):
            for k in range(top):
                r = int(place[t, k])
                if 0 <= r < used:
                    assert torch.equal(buf[1 + r], x[t])
        buf = torch.full((n + 2, cols), 5.0).cuda()
        _, dw = tg.combine_backward(x, torch.ones(n, cols).cuda(), place, torch.ones(tokens, top).cuda(), ends,
                                    drows=buf[1:n + 1])
        assert (buf[0] == 5).all() and (buf[n + 1] == 5).all() and (buf[1 + used:n + 1] == 0).all()
        fine = (place.cpu() >= 0) & (place.cpu() < used)
        assert (dw.cpu()[~fine] == 0).all()
    rows = torch.randn(n, cols, generator=gen(2)).cuda()
    out = tg.combine(rows, place)
    for t in range(tokens):
        want = sum((f64(rows[int(r)]) for r in place[t].tolist() if 0 <= r < n), torch.zeros(cols, dtype=torch.float64))
        within(out[t], want, 1e-6 * (1 + want.abs()), "out")


def test_rows_without_a_name_stay(gpu_available):
    """Before the last end, rows that no place names are left as they were."""
    place = torch.tensor([[0], [3]], dtype=torch.int32).cuda()
    ends = torch.tensor([2, 5], dtype=torch.int32).cuda()
    x = torch.ones(2, 8).cuda()
    say("[routing] rows without a name")
    out = torch.full((7, 8), 5.0).cuda()
    tg.dispatch(x, place, ends, out=out)
    assert out[:, 0].tolist() == [1, 5, 5, 1, 5, 0, 0]
    out = torch.full((7, 8), 5.0).cuda()
    tg.combine_backward(x, out.clone(), place, torch.full((2, 1), 2.0).cuda(), ends, drows=out)
    assert out[:, 0].tolist() == [2, 5, 5, 2, 5, 0, 0]


def test_empty_calls(gpu_available):
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    say("[routing] empty calls")
    order, place, ends = tg.expert_plan(torch.zeros(0, 3, dtype=torch.int64, device="cuda"), 4)
    assert order.shape == (0,) and place.shape == (0, 3) and (ends == 0).all()
    assert tg.dispatch(f(0, 8), place, ends).shape == (0, 8)
    out = f(5, 8)
    tg.dispatch(f(0, 8), place, ends, out=out)
    assert (out == 0).all()
    assert tg.combine(f(0, 8), place, weights=f(0, 3)).shape == (0, 8)
    drows, dw = tg.combine_backward(f(0, 8), f(4, 8), place, f(0, 3), ends)
    assert (drows == 0).all() and dw.shape == (0, 3)
    place = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(tg.combine(f(0, 8), place, residual=2 * f(2, 8)), 2 * f(2, 8))
    drows, dw = tg.combine_backward(f(2, 8), f(0, 8), place, f(2, 3), ends)
    assert drows.shape == (0, 8) and (dw == 0).all()
    drows, dw = tg.combine_backward(f(2, 0), f(6, 0), place, f(2, 3), ends)
    assert (dw == 0).all()
    assert tg.dispatch(f(2, 0), place, ends).shape == (6, 0)


def test_refusals(gpu_available):
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    e = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    place, ends = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for error, call in [
            (TypeError, lambda: tg.expert_plan(f(4, 2), 3)), (ValueError, lambda: tg.expert_plan(e[0], 3)),
            (ValueError, lambda: tg.expert_plan(e.cpu(), 3)), (ValueError, lambda: tg.expert_plan(e, 0)),
            (ValueError, lambda: tg.expert_plan(e[:, :0], 3)), (tg.GemmError, lambda: tg.expert_plan(e, 4097)),
            (ValueError, lambda: tg.expert_plan(e.t(), 3)),
            (TypeError, lambda: tg.dispatch(f(4, 8).half(), place, ends)),
            (ValueError, lambda: tg.dispatch(f(5, 8), place, ends)), (TypeError, lambda: tg.dispatch(f(4, 8), e, ends)),
            (ValueError, lambda: tg.dispatch(f(2, 8), place.t(), ends)),
            (ValueError, lambda: tg.dispatch(f(4, 8), place, ends[:0])),
            (TypeError, lambda: tg.dispatch(f(4, 8), place, ends.long())),
            (ValueError, lambda: tg.dispatch(f(4, 8), place, ends.cpu())),
            (ValueError, lambda: tg.dispatch(f(4, 8), place, ends, scales=f(5))),
            (TypeError, lambda: tg.dispatch(f(4, 8), place, ends, scales=f(4).bfloat16())),
            (ValueError, lambda: tg.dispatch(f(4, 8), place, ends, out=f(8, 9))),
            (TypeError, lambda: tg.dispatch(f(4, 8), place, ends, out=f(8, 8).bfloat16())),
            (ValueError, lambda: tg.dispatch(f(4, 8), place, ends, out_scales=f(8))),
            (TypeError, lambda: tg.combine(f(8, 8).half(), place)), (TypeError, lambda: tg.combine(f(8, 8), e)),
            (ValueError, lambda: tg.combine(f(8, 8), place, weights=f(4, 3))),
            (TypeError, lambda: tg.combine(f(8, 8), place, weights=f(4, 2).bfloat16())),
            (ValueError, lambda: tg.combine(f(8, 8), place, residual=f(5, 8))),
            (TypeError, lambda: tg.combine(f(8, 8), place, residual=f(4, 8).bfloat16())),
            (ValueError, lambda: tg.combine(f(8, 8), place, out=f(4, 9))),
            (ValueError, lambda: tg.combine_backward(f(5, 8), f(8, 8), place, f(4, 2), ends)),
            (ValueError, lambda: tg.combine_backward(f(4, 8), f(8, 9), place, f(4, 2), ends)),
            (TypeError, lambda: tg.combine_backward(f(4, 8), f(8, 8).bfloat16(), place, f(4, 2), ends)),
            (ValueError, lambda: tg.combine_backward(f(4, 8), f(8, 8), place, f(4, 3), ends)),
            (ValueError, lambda: tg.combine_backward(f(4, 8), f(8, 8), place, f(4, 2), ends, drows=f(7, 8)))]:
        with pytest.raises(error):
            call()
