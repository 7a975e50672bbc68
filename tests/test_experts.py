"""The sparse expert layer's operators on the GPU against 64-bit references.

Tolerances count roundings.  A sum of n fp32 terms in any order is off by at
most n * 2^-24 of the sum of magnitudes; a rounding to bf16 by 2^-8 of the
value, to e4m3 by 2^-4 of it (2^-10 among the subnormals).  The fp8 matrix
core sums each run of 8 products to 2^-10 of its largest (include/gemm.h).
"""
import itertools

import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say

pytestmark = pytest.mark.gpu

U32, U16, U8 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
FP8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
HALF = {F32: 0.0, BF16: U16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def padded(t, pad=0, offset=0):
    """Device copy of a matrix (or of a stack of them) inside a wider buffer of NaN, `offset` elements in."""
    raw = t.dtype == FP8
    src = t.view(torch.uint8) if raw else t
    lead, rows, cols = (1, *src.shape) if src.dim() == 2 else src.shape
    ld = cols + pad
    buf = torch.full((lead * rows * ld + offset + 1,), 0x7F if raw else float("nan"), dtype=src.dtype, device="cuda")
    view = buf[offset:offset + lead * rows * ld].view(lead, rows, ld)[:, :, :cols]
    view.copy_(src)
    view = view if src.dim() == 3 else view[0]
    return view.view(FP8) if raw else view


def f64(t):
    return t.detach().to(device="cpu").to(torch.float64)


def within(got, want, tol, what):
    got, want = f64(got), f64(want)
    assert torch.equal(got.isnan(), want.isnan()), what
    off = (got - want).abs()
    bad = ~((off <= tol) | want.isnan() | (got == want))
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300))[bad].max()))


# ---------------------------------------------------------------- quantiser

def plain_codes(x, block_rows):
    """The header's formula, in fp32 as it says, on the host."""
    M, K = x.shape
    rb, kb = -(-M // block_rows), -(-K // 128)
    xp = torch.zeros(rb * block_rows, kb * 128)
    xp[:M, :K] = x.float()
    t = xp.view(rb, block_rows, kb, 128)
    amax = torch.where(t.isfinite(), t.abs(), torch.zeros(())).amax(dim=(1, 3)).clamp_min(2.0 ** -100)
    inv = torch.tensor(448.0) / amax
    c = (t * inv[:, None, :, None]).reshape(rb * block_rows, kb * 128)[:M, :K]
    c = torch.where(x.float().isfinite(), c.clamp(-448, 448), torch.tensor(float("nan")))
    return c.to(FP8), amax / 448.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,K,pad,offset", [(1, 1, 0, 0), (3, 127, 1, 1), (5, 128, 0, 0), (130, 129, 7, 3),
                                            (129, 777, 0, 0), (256, 1024, 8, 8), (300, 2000, 16, 0)])
def test_quantize(gpu_available, dtype, block_rows, M, K, pad, offset):
    say(f"[quantize] {dtype} block_rows={block_rows} {M}x{K} pad={pad} offset={offset}")
    x = (torch.randn(M, K, generator=gen(M + K)) * torch.logspace(-3, 3, K)).to(dtype)
    q, s = tg.quantize(padded(x, pad, offset), block_rows)
    want, scale = plain_codes(x, block_rows)
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(q.cpu().float(), want.float())
    assert q.stride(0) % 16 == 0 or M == 1
    # into the caller's tensors, whose padding stays as it was
    out = padded(torch.zeros(M, K).to(FP8), 5, 0)
    back = out.as_strided((M, K + 5), (K + 5, 1)).view(torch.uint8)
    q2, s2 = tg.quantize(padded(x, pad, offset), block_rows, out=out, scales=torch.empty_like(s))
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    assert (back[:, K:] == 0x7F).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(gpu_available, block_rows):
    x = torch.zeros(130, 400)
    x[0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0])
    x[1, 128:256] = float("nan")
    x[2, 256:] = 1e-35
    x[3, 5] = 3.4e38
    x[4, 130] = 1e-45
    for dtype in (F32, BF16):
        say(f"[quantize] special values {dtype} {block_rows}")
        q, s = tg.quantize(x.to(dtype).cuda(), block_rows)
        want, scale = plain_codes(x.to(dtype), block_rows)
        assert torch.equal(s.cpu(), scale)
        got = q.cpu().float()
        assert torch.equal(got.isnan(), want.float().isnan())
        assert torch.equal(got.nan_to_num(7.0), want.float().nan_to_num(7.0))


# --------------------------------------------------------------------- norm

def depth(N):
    """Additions in a row's sum of squares, at most: 8 values a chunk, a chunk for each 512 columns, then the tree."""
    return 8 * -(-N // 512) + 26


def norm64(s, w, eps):
    s, w = f64(s), f64(w)
    return s / (s.square().mean(dim=1, keepdim=True) + eps).sqrt() * w


NORM_SIZES = [(1, 1, 0, 0), (3, 7, 1, 0), (5, 128, 0, 0), (2, 777, 0, 1), (4, 1024, 8, 0), (3, 1025, 0, 0),
              (2, 4096, 0, 0), (3, 4104, 8, 8), (2, 8192, 0, 0), (2, 8193, 3, 0), (1, 16384, 0, 0), (2, 20001, 0, 0),
              (1, 40960, 0, 0), (1500, 264, 0, 0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N,pad,offset", NORM_SIZES)
def test_rms_norm(gpu_available, dtype, residual, M, N, pad, offset):
    say(f"[norm] {dtype} residual={residual} {M}x{N} pad={pad} offset={offset}")
    g = gen(N + M)
    x, r = torch.randn(M, N, generator=g).to(dtype), (3 * torch.randn(M, N, generator=g)).to(dtype)
    w = (1 + 0.2 * torch.randn(N, generator=g)).to(dtype)
    s = (x.float() + r.float()).to(dtype) if residual else x
    xd, wd, rd = padded(x, pad, offset), w.cuda(), padded(r, pad, offset) if residual else None
    eps = 1e-5
    want = norm64(s, w, eps)
    rel = (depth(N) / 2 + 8) * U32
    for kind in (F32, BF16, FP8):
        out, total, scales = tg.rms_norm(xd, wd, residual=rd, eps=eps, out_dtype=kind)
        assert torch.equal(total.cpu(), s)
        if kind == FP8:
            top = torch.nn.functional.pad(want.abs(), (0, -N % 128)).view(M, -1, 128).amax(dim=2).clamp_min(2.0 ** -100)
            within(scales, top / 448, top / 448 * (rel + 2 * U32), "scales")
            wide = f64(scales).repeat_interleave(128, dim=1)[:, :N]
            within(f64(out) * wide, want, want.abs() * (U8 + 2 * rel) + wide * 2.0 ** -10, "codes")
        else:
            assert scales is None
            within(out, want, want.abs() * (rel + HALF[kind] * (1 + rel)), kind)


def test_rms_norm_in_place_and_rows_of_zeros(gpu_available):
    say("[norm] in place")
    x, r = torch.randn(6, 520, generator=gen(1)).bfloat16(), torch.randn(6, 520, generator=gen(2)).bfloat16()
    x[3], r[3] = 0, 0
    w = torch.ones(520).bfloat16().cuda()
    want, s, sc = tg.rms_norm(x.cuda(), w, residual=r.cuda(), out_dtype=FP8)
    for target in (0, 1):
        xd, rd = x.cuda(), r.cuda()
        out, total, scales = tg.rms_norm(xd, w, residual=rd, summed=(xd, rd)[target], out_dtype=FP8)
        assert total.data_ptr() == (xd, rd)[target].data_ptr()
        assert torch.equal(total, s) and torch.equal(scales, sc)
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))
    assert (want[3].float() == 0).all() and (s[3] == 0).all()
    assert torch.equal(sc[3].cpu(), torch.full((5,), 2.0 ** -100) / 448)
    # an infinity or a NaN spoils its own row only
    x[1, 7], x[4, 9] = float("inf"), float("nan")
    out, _, _ = tg.rms_norm(x.cuda(), w, residual=r.cuda(), out_dtype=F32)
    ok = [0, 2, 3, 5]
    again, _, _ = tg.rms_norm(x.cuda()[ok], w, residual=r.cuda()[ok], out_dtype=F32)
    assert torch.equal(out[ok], again)
    assert out[4].isnan().all() and out[1, 7].isnan()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("with_ds", [False, True])
@pytest.mark.parametrize("M,N,pad,offset", NORM_SIZES + [(3000, 64, 0, 0)])
def test_rms_norm_backward(gpu_available, dtype, with_ds, M, N, pad, offset):
    say(f"[norm grad] {dtype} ds={with_ds} {M}x{N} pad={pad} offset={offset}")
    g = gen(N + M + 5)
    dy, s, ds = (torch.randn(M, N, generator=g).to(dtype) for _ in range(3))
    w = (1 + 0.2 * torch.randn(N, generator=g)).to(dtype)
    eps = 1e-5
    dx, dw = tg.rms_norm_backward(padded(dy, pad, offset), padded(s, pad, offset), w.cuda(),
                                  dsum=padded(ds, pad, offset) if with_ds else None, eps=eps)
    dy6, s6, w6 = f64(dy), f64(s), f64(w)
    d6 = f64(ds) if with_ds else torch.zeros(M, N, dtype=torch.float64)
    r = (s6.square().mean(dim=1, keepdim=True) + eps).rsqrt()
    up = dy6 * w6
    want = r * (up - s6 * r * r * (up * s6).mean(dim=1, keepdim=True)) + d6
    size = r * up.abs() + s6.abs() * r ** 3 * (up * s6).abs().mean(dim=1, keepdim=True) + d6.abs()
    within(dx, want, size * (2 * depth(N) + 16) * U32 + HALF[dtype] * want.abs() * 1.001, "dx")
    terms = dy6 * s6 * r
    within(dw, terms.sum(dim=0), terms.abs().sum(dim=0) * (M + depth(N) + 20) * U32, "dw")
    # dx may be dy or dsum itself
    for k in range(2 if with_ds else 1):
        a, b = padded(dy, pad, offset), padded(ds, pad, offset) if with_ds else None
        dx2, none = tg.rms_norm_backward(a, padded(s, pad, offset), w.cuda(), dsum=b, eps=eps, dx=(a, b)[k],
                                         want_dweight=False)
        assert none is None and torch.equal(dx2, dx)


def test_rms_norm_gradients_against_differences(gpu_available):
    say("[norm grad] differences")
    M, N, eps, h = 3, 40, 1e-3, 1e-5
    g = gen(9)
    x, w, dy = torch.randn(M, N, generator=g), torch.rand(N, generator=g) + 0.5, torch.randn(M, N, generator=g)
    dx, dw = tg.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=eps)

    def loss(x6, w6):
        return float((norm64(x6, w6, eps) * f64(dy)).sum())

    # Central differences of a smooth function of size ~10: h^2 (1e-10) of truncation, 1e-15 / h of rounding.
    for i, j in itertools.product(range(M), range(N)):
        e = torch.zeros(M, N, dtype=torch.float64)
        e[i, j] = h
        assert abs((loss(f64(x) + e, w) - loss(f64(x) - e, w)) / (2 * h) - float(dx[i, j])) < 1e-5
    for j in range(N):
        e = torch.zeros(N, dtype=torch.float64)
        e[j] = h
        assert abs((loss(x, f64(w) + e) - loss(x, f64(w) - e)) / (2 * h) - float(dw[j])) < 1e-5


def test_norm_gradient_without_rows_is_zero(gpu_available):
    dx, dw = tg.rms_norm_backward(torch.empty(0, 96, device="cuda"), torch.empty(0, 96, device="cuda"),
                                  torch.ones(96, device="cuda"))
    assert dx.shape == (0, 96) and (dw == 0).all()


# ----------------------------------------------------------------- products

def fp8_matrix(rows, cols, seed, block_rows):
    return plain_codes(torch.randn(rows, cols, generator=gen(seed)) * torch.logspace(-1, 1, cols), block_rows)


def values(code, scale, block_rows):
    s = f64(scale).repeat_interleave(128, dim=-1)[..., :code.shape[-1]]
    return f64(code) * (s.repeat_interleave(block_rows, dim=-2)[..., :code.shape[-2], :] if block_rows > 1 else s)


def product_tol(a, b, want, fp8, kind, alpha=1.0):
    size = a.abs() @ b.abs() * abs(alpha)
    K = a.shape[1]
    tol = size * ((K + 6) * U32 + (2.0 ** -10 if fp8 else 0.0))
    return tol * (1 + HALF[kind]) + HALF[kind] * want.abs()


BLOCK_SIZES = [  # M, N, K, pad (bytes a row past the next multiple of 16), offset
    (1, 1, 1, 0, 0), (1, 256, 128, 0, 0), (3, 130, 257, 0, 0), (16, 512, 4096, 0, 0), (17, 129, 1000, 0, 0),
    (64, 300, 777, 0, 0), (128, 128, 128, 16, 16), (129, 257, 384, 0, 0), (256, 256, 1024, 0, 0),
    (300, 520, 264, 32, 0), (513, 384, 1040, 0, 0), (70, 90, 129, 3, 1), (1000, 1111, 300, 0, 0),
    (2100, 2304, 256, 0, 0), (4, 5000, 640, 0, 0), (33, 64, 8192, 0, 0)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K,pad,offset", BLOCK_SIZES)
def test_block_gemm(gpu_available, op, M, N, K, pad, offset):
    say(f"[block] op={op} {M}x{N}x{K} pad={pad} offset={offset}")
    qa, sa = fp8_matrix(M, K, M + K, 1)
    qb, sb = fp8_matrix(*((N, K) if op == "T" else (K, N)), N + K, 128)
    a, b = values(qa, sa, 1), values(qb, sb, 128)
    b = b.t() if op == "T" else b
    want = a @ b
    Ad, Bd = padded(qa, -K % 16 + pad, offset), padded(qb, -qb.shape[1] % 16 + pad, offset)
    for kind, alpha in ((BF16, 1.0), (F32, -0.5)):
        out = padded(torch.zeros(M, N).to(kind), 3, 1)
        back = out.as_strided((M, N + 3), (N + 3, 1))
        got = tg.block_gemm(Ad, Bd, sa.cuda(), sb.cuda(), op_b=op, alpha=alpha, out=out)
        within(got, alpha * want, product_tol(a, b, alpha * want, True, kind, alpha), kind)
        assert back[:-1, N:].isnan().all()
    # scales stored the other way around
    got = tg.block_gemm(Ad, Bd, sa.cuda().t().contiguous().t(), sb.cuda().t().contiguous().t(), op_b=op, out_dtype=F32)
    assert torch.equal(got, tg.block_gemm(Ad, Bd, sa.cuda(), sb.cuda(), op_b=op, out_dtype=F32))


@pytest.mark.parametrize("op", ["T", "N"])
def test_block_gemm_special_values_stay_in_their_rows(gpu_available, op):
    """A NaN code spoils its row (or column) of the product only, and the bytes past K never count."""
    M, N, K = 70, 140, 200
    say(f"[block] special values op={op}")
    qa, sa = fp8_matrix(M, K, 1, 1)
    qb, sb = fp8_matrix(*((N, K) if op == "T" else (K, N)), 2, 128)
    want = tg.block_gemm(padded(qa, 8), padded(qb, -qb.shape[1] % 16), sa.cuda(), sb.cuda(), op_b=op, out_dtype=F32)
    qa.view(torch.uint8)[5, 199] = 0x7F
    (qb.view(torch.uint8)[7] if op == "T" else qb.view(torch.uint8)[:, 7])[3] = 0xFF
    got = tg.block_gemm(padded(qa, 8), padded(qb, -qb.shape[1] % 16), sa.cuda(), sb.cuda(), op_b=op, out_dtype=F32)
    assert got[5].isnan().all() and got[:, 7].isnan().all()
    keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
    keep[5], keep[:, 7] = False, False
    assert torch.equal(got[keep], want[keep]) and not want.isnan().any()


def test_block_gemm_without_depth_gives_zeros(gpu_available):
    a, b = torch.empty(5, 0, dtype=FP8, device="cuda"), torch.empty(7, 0, dtype=FP8, device="cuda")
    got = tg.block_gemm(a, b, torch.empty(5, 0, device="cuda"), torch.empty(1, 0, device="cuda"), out_dtype=F32)
    assert got.shape == (5, 7) and (got == 0).all()
    qa, sa = fp8_matrix(5, 64, 3, 1)
    qa.view(torch.uint8)[0, 0] = 0x7F
    got = tg.block_gemm(padded(qa), padded(qa), sa.cuda(), sa.cuda()[:1], alpha=0.0, out_dtype=F32)
    assert (got == 0).all()


def ends_of(sizes):
    return torch.tensor(list(itertools.accumulate(sizes)), dtype=torch.int32)


GROUPINGS = [  # rows of each group, rows past the last end
    ([5], 0), ([0], 3), ([0, 0, 4, 0], 0), ([1, 1, 1], 1), ([16, 17, 0, 33, 64], 2), ([128, 0, 129, 255], 0),
    ([300, 1, 40, 0, 260], 70), ([2] * 70 + [0] * 60 + [3] * 5, 1), ([600], 0)]
DEPTHS = [(64, 32), (130, 257), (256, 512)]     # N, K


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
@pytest.mark.parametrize("sizes,rest", GROUPINGS)
@pytest.mark.parametrize("N,K", DEPTHS)
def test_grouped_gemm(gpu_available, op, dtype, sizes, rest, N, K):
    say(f"[grouped] {dtype} op={op} sizes={str(sizes)[:40]} rest={rest} N={N} K={K}")
    G, M = len(sizes), sum(sizes) + rest
    shape = (N, K) if op == "T" else (K, N)
    extra = {}
    if dtype == FP8:
        x, sa = fp8_matrix(M, K, 11, 1)
        pairs = [fp8_matrix(*shape, 100 + g, 128) for g in range(G)]
        w = torch.stack([q.view(torch.uint8) for q, _ in pairs]).view(FP8)
        sb = torch.stack([s for _, s in pairs])
        extra = {"a_scales": sa.cuda(), "b_scales": sb.cuda()}
        a, b = values(x, sa, 1), values(w, sb, 128)
    else:
        x = torch.randn(M, K, generator=gen(1)).to(dtype)
        w = torch.randn(G, *shape, generator=gen(2)).to(dtype)
        a, b = f64(x), f64(w)
    b = b.transpose(1, 2) if op == "T" else b
    ends = ends_of(sizes)
    for pad in (0, 1):
        unit = 16 if dtype == FP8 else 8
        xd, wd = padded(x, -K % unit + pad), padded(w, -shape[1] % unit + pad)
        for kind in (F32, BF16):
            got = tg.grouped_gemm(xd, wd, ends.cuda(), op_b=op, alpha=0.5, out=padded(torch.ones(M, N).to(kind), 2),
                                  **extra)
            at = 0
            for g, size in enumerate(sizes):
                if size:
                    p = a[at:at + size]
                    want = 0.5 * (p @ b[g])
                    within(got[at:at + size], want, product_tol(p, b[g], want, dtype == FP8, kind, 0.5), (g, kind))
                at += size
            assert (got[at:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
def test_grouped_ends_out_of_range_touch_nothing_else(gpu_available, dtype):
    """Ends that run backwards, below zero or past M count as their running maximum, within 0 .. M."""
    say(f"[grouped] ends out of range {dtype}")
    M, N, K, G = 90, 64, 128, 6
    x, w = torch.randn(M, K, generator=gen(1)), torch.randn(G, N, K, generator=gen(2))
    extra = {}
    if dtype == FP8:
        x, sa = plain_codes(x, 1)
        pairs = [plain_codes(w[g], 128) for g in range(G)]
        w = torch.stack([q.view(torch.uint8) for q, _ in pairs]).view(FP8)
        extra = {"a_scales": sa.cuda(), "b_scales": torch.stack([s for _, s in pairs]).cuda()}
    else:
        x, w = x.to(dtype), w.to(dtype)
    out = padded(torch.zeros(M + 60, N), 0)
    for bad, good in (([10, 5, -3, 50, 1000, 70], [10, 10, 10, 50, 90, 90]), ([-5, 2, 1, 0, 3, 80], [0, 2, 2, 2, 3, 80])):
        out.fill_(7.0)
        got = tg.grouped_gemm(padded(x), padded(w), torch.tensor(bad, dtype=torch.int32).cuda(), out=out[30:30 + M], **extra)
        want = tg.grouped_gemm(padded(x), padded(w), torch.tensor(good, dtype=torch.int32).cuda(), out_dtype=F32, **extra)
        assert torch.equal(got, want)
        assert (out[:30] == 7).all() and (out[30 + M:] == 7).all()
        if dtype != FP8:
            dy = torch.randn(M, N, generator=gen(3)).to(dtype)
            a = tg.grouped_wgrad(padded(dy), padded(x), torch.tensor(bad, dtype=torch.int32).cuda())
            b = tg.grouped_wgrad(padded(dy), padded(x), torch.tensor(good, dtype=torch.int32).cuda())
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes,rest", GROUPINGS)
@pytest.mark.parametrize("N,K", [(64, 32), (130, 257), (264, 520)])
def test_grouped_wgrad(gpu_available, dtype, sizes, rest, N, K):
    say(f"[wgrad] {dtype} sizes={str(sizes)[:40]} rest={rest} N={N} K={K}")
    G, M = len(sizes), sum(sizes) + rest
    dy, x = torch.randn(M, N, generator=gen(4)).to(dtype), torch.randn(M, K, generator=gen(5)).to(dtype)
    dy[M - rest:], x[M - rest:] = float("nan"), float("nan")       # rows of no group are not read
    c0 = torch.randn(G, N, K, generator=gen(6))
    ends = ends_of(sizes).cuda()
    for pad in (0, 1):
        dyd, xd = padded(dy, -N % 8 + pad), padded(x, -K % 8 + pad)
        for alpha, beta in ((1.0, 0.0), (0.5, -2.0)):
            out = padded(c0 if beta else torch.full((G, N, K), float("nan")), 3)
            got = tg.grouped_wgrad(dyd, xd, ends, alpha=alpha, beta=beta, out=out)
            at = 0
            for g, size in enumerate(sizes):
                p, q = f64(dy[at:at + size]), f64(x[at:at + size])
                old = beta * f64(c0[g]) if beta else torch.zeros(N, K, dtype=torch.float64)
                want = alpha * (p.t() @ q) + old
                tol = ((p.abs().t() @ q.abs()) * abs(alpha) + old.abs()) * (size + 4) * U32
                within(got[g], want, tol, g)
                at += size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,K", [(70, 33), (300, 256), (1, 40), (40, 3)])
def test_weight_gradients_into_rows_in_turn(gpu_available, dtype, N, K):
    """out as N x groups x K in memory: a row of every group after the other, with a gap that stays as it was."""
    say(f"[wgrad] rows in turn {dtype} {N}x{K}")
    G, M = 3, 100
    dy, x = torch.randn(M, N, generator=gen(1)).to(dtype).cuda(), torch.randn(M, K, generator=gen(2)).to(dtype).cuda()
    ends = ends_of([30, 0, 70]).cuda()
    buf = torch.full((N, G, K + 5), 7.0, device="cuda")
    out = buf[:, :, :K].transpose(0, 1)
    want = tg.grouped_wgrad(dy, x, ends)
    assert tg.grouped_wgrad(dy, x, ends, out=out) is out and torch.equal(out, want)
    tg.grouped_wgrad(dy, x, ends, beta=1.0, out=out)
    assert torch.equal(out, tg.grouped_wgrad(dy, x, ends, beta=1.0, out=want))
    assert (buf[:, :, K:] == 7.0).all()


def test_grouped_gradients_against_differences(gpu_available):
    """The three products of a training step, as gradients of one loss."""
    say("[grouped] differences")
    sizes, N, K, h = [3, 0, 4], 6, 5, 1e-3
    M, G = sum(sizes), len(sizes)
    x, w, dy = (torch.randn(*s, generator=gen(i)) for i, s in enumerate([(M, K), (G, N, K), (M, N)]))
    ends = ends_of(sizes).cuda()
    dx = tg.grouped_gemm(dy.cuda(), w.cuda(), ends, op_b="N")
    dw = tg.grouped_wgrad(dy.cuda(), x.cuda(), ends)
    owner = torch.repeat_interleave(torch.arange(G), torch.tensor(sizes))

    def loss(x6, w6):
        return float((torch.stack([w6[owner[i]] @ x6[i] for i in range(M)]) * f64(dy)).sum())

    # The loss is linear in each, so central differences have rounding only: 1e-13 / h.
    for i, k in itertools.product(range(M), range(K)):
        e = torch.zeros(M, K, dtype=torch.float64)
        e[i, k] = h
        assert abs((loss(f64(x) + e, f64(w)) - loss(f64(x) - e, f64(w))) / (2 * h) - float(dx[i, k])) < 1e-5
    for g, n, k in itertools.product(range(G), range(N), range(K)):
        e = torch.zeros(G, N, K, dtype=torch.float64)
        e[g, n, k] = h
        assert abs((loss(f64(x), f64(w) + e) - loss(f64(x), f64(w) - e)) / (2 * h) - float(dw[g, n, k])) < 1e-5


def layer_inputs():
    g = gen(21)
    x, r = torch.randn(200, 384, generator=g).bfloat16().cuda(), torch.randn(200, 384, generator=g).bfloat16().cuda()
    w = torch.ones(384).bfloat16().cuda()
    ups = [tg.quantize((torch.randn(256, 384, generator=g) / 20).cuda(), 128) for _ in range(5)]
    up = torch.stack([q.view(torch.uint8) for q, _ in ups]).view(FP8)
    return x, r, w, up, torch.stack([s for _, s in ups]), ends_of([60, 0, 100, 7, 30]).cuda()


def sequence(x, r, w, up, up_s, ends):
    """Every operator once: what a training step with fp8 products would call."""
    q, s, sc = tg.rms_norm(x, w, residual=r, out_dtype=FP8)
    y = tg.grouped_gemm(q, up, ends, a_scales=sc, b_scales=up_s)
    qy, sy = tg.quantize(y)
    dx = tg.grouped_gemm(qy, up, ends, a_scales=sy, b_scales=up_s, op_b="N")
    one = tg.block_gemm(qy, up[2], sy, up_s[2], op_b="N", out_dtype=F32)
    dw = tg.grouped_wgrad(y, s, ends)
    gx, gw = tg.rms_norm_backward(dx, s, w, dsum=x)
    return [q.float(), s, sc, y, qy.float(), sy, dx, one, dw, gx, gw]


def test_calls_capture_into_a_graph_and_replay(gpu_available):
    inputs = layer_inputs()
    say("[experts] eager reference")
    want = [t.clone() for t in sequence(*inputs)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        sequence(*inputs)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("[experts] capture")
    with torch.cuda.graph(graph):
        got = sequence(*inputs)
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        again = sequence(*inputs)                       # eager work between replays
        torch.cuda.synchronize()
        say(f"[experts] replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b, c) in enumerate(zip(got, want, again)):
            assert torch.equal(a, b) and torch.equal(c, b), (rep, i)


def test_calls_on_another_stream(gpu_available):
    """A stream handle other than torch's current one: results and the memory they were allocated in are whole."""
    inputs = layer_inputs()
    want = [t.clone() for t in sequence(*inputs)]
    x, r, w, up, up_s, ends = inputs
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    h = other.cuda_stream
    say("[experts] other stream")
    for _ in range(3):
        q, s, sc = tg.rms_norm(x, w, residual=r, out_dtype=FP8, stream=h)
        y = tg.grouped_gemm(q, up, ends, a_scales=sc, b_scales=up_s, stream=h)
        qy, sy = tg.quantize(y, stream=h)
        dx = tg.grouped_gemm(qy, up, ends, a_scales=sy, b_scales=up_s, op_b="N", stream=h)
        one = tg.block_gemm(qy, up[2], sy, up_s[2], op_b="N", out_dtype=F32, stream=h)
        dw = tg.grouped_wgrad(y, s, ends, stream=h)
        gx, gw = tg.rms_norm_backward(dx, s, w, dsum=x, stream=h)
        other.synchronize()
        for a, b in zip([q.float(), s, sc, y, qy.float(), sy, dx, one, dw, gx, gw], want):
            assert torch.equal(a, b)


def test_shared_weights_and_per_tensor_scales(gpu_available):
    """Strides of zero: one matrix for every group, one scale for a whole operand."""
    x = torch.randn(40, 128, generator=gen(1)).bfloat16().cuda()
    w = torch.randn(96, 128, generator=gen(2)).bfloat16().cuda()
    ends = torch.tensor([10, 10, 40], dtype=torch.int32).cuda()
    one = tg.grouped_gemm(x, w[None], ends[-1:], out_dtype=F32)
    assert torch.equal(tg.grouped_gemm(x, w.expand(3, 96, 128), ends, out_dtype=F32), one)
    qa, qb = x.to(FP8), w.to(FP8)
    s = torch.full((1, 1), 0.25, device="cuda")
    got = tg.block_gemm(qa, qb, s.expand(40, 1), s, out_dtype=F32)
    plain = tg.block_gemm(qa, qb, torch.ones(40, 1, device="cuda"), torch.ones(1, 1, device="cuda"), out_dtype=F32)
    assert torch.equal(got, plain * 0.0625)


def test_a_short_call_of_a_large_cache_of_weights(gpu_available):
    """Groups whose weights start past 2^31 bytes (and elements): offsets are 64-bit."""
    say("[grouped] weights past 2^31 elements")
    G, N, K = 18, 4096, 32768                         # 2.4e9 elements of fp8
    w = torch.zeros((G, N, K), dtype=torch.uint8, device="cuda").view(FP8)
    last, s = tg.quantize(torch.randn(N, K, generator=gen(1)).cuda(), 128)
    w[-1].view(torch.uint8).copy_(last.view(torch.uint8))
    qa, sa = tg.quantize(torch.randn(5, K, generator=gen(2)).cuda())
    ends = torch.zeros(G, dtype=torch.int32)
    ends[-1] = 5
    got = tg.grouped_gemm(qa, w, ends.cuda(), a_scales=sa, b_scales=s.expand(G, -1, -1), out_dtype=F32)
    want = tg.block_gemm(qa, last, sa, s, out_dtype=F32)
    assert torch.equal(got, want) and float(want.abs().max()) > 1
