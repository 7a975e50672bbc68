"""8-bit integer rows and products on the GPU against exact sums.

Sums of 8-bit products are exact.  A result is x = round(round(sum) * b), then
round(x * a + bias), then for bf16 one rounding more: x is made on the host in
fp32, and the rest is off by at most 2^-24 (fp32) and 2^-8 (bf16) of the value.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say

pytestmark = pytest.mark.gpu

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8
U32, U16 = 2.0 ** -24, 2.0 ** -8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def padded(t, pad=0, offset=0, fill=113):
    """Device copy of a matrix (or of a stack of them) inside a wider buffer, `offset` elements in."""
    lead, rows, cols = (1, *t.shape) if t.dim() == 2 else t.shape
    ld = cols + pad
    buf = torch.full((lead * rows * ld + offset + 1,), fill, dtype=t.dtype, device="cuda")
    view = buf[offset:offset + lead * rows * ld].view(lead, rows, ld)[:, :, :cols]
    view.copy_(t)
    return view if t.dim() == 3 else view[0]


def plain_rows(x):
    """The header's formula in fp32 on the host: (codes, scales)."""
    x = x.float()
    fine = x.isfinite().all(dim=1)
    amax = torch.where(x.isfinite(), x.abs(), torch.zeros(())).amax(dim=1).clamp_min(2.0 ** -100)
    codes = (x * (torch.tensor(127.0) / amax)[:, None]).round()
    codes = torch.where(fine[:, None], codes, torch.zeros(())).to(I8)
    return codes, torch.where(fine, amax / 127.0, torch.tensor(float("nan")))


def same_scales(got, want):
    return torch.equal(got.cpu().isnan(), want.isnan()) and torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


ROW_SIZES = [(1, 1, 0, 0), (3, 7, 1, 1), (5, 128, 0, 0), (9, 777, 0, 1), (4, 1024, 8, 0), (6, 1025, 0, 0), (2, 4096, 0, 0),
             (3, 4104, 8, 8), (2, 8192, 0, 0), (2, 8193, 3, 0), (1, 16384, 0, 0), (3, 20001, 0, 1), (4099, 40, 0, 0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K,pad,offset", ROW_SIZES)
def test_rows(gpu_available, dtype, M, K, pad, offset):
    say(f"[int8 rows] {dtype} {M}x{K} pad={pad} offset={offset}")
    x = (torch.randn(M, K, generator=gen(M + K)) * torch.logspace(-2, 2, K)).to(dtype)
    codes, scales = tg.quantize_int8(padded(x, pad, offset, 1e30))
    want, scale = plain_rows(x)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(codes.cpu(), want)
    assert codes.stride(0) % 16 == 0 or M == 1
    # into the caller's tensors, whose padding stays as it was
    out = padded(torch.zeros(M, K, dtype=I8), 5)
    q, s = tg.quantize_int8(padded(x, pad, offset, 1e30), out=out, scales=torch.empty_like(scales))
    assert torch.equal(q.cpu(), want) and torch.equal(s, scales) and q.data_ptr() == out.data_ptr()
    assert (out.as_strided((M, K + 5), (K + 5, 1))[:, K:] == 113).all()


@pytest.mark.parametrize("K", [5, 300, 3000, 6000, 12000, 20000])
def test_rows_of_special_values(gpu_available, K):
    x = torch.randn(8, K, generator=gen(K))
    x[0] = 0.0
    x[1, K // 2] = float("inf")
    x[2, K - 1] = float("nan")
    x[3, 0] = -float("inf")
    x[4] = 1e-35
    x[5, K // 3] = 3.3e38
    x[6] = -2.0
    x[7, 0], x[7, 1:] = 2.0, 1.0          # 63.5: a tie
    for dtype in (F32, BF16):
        say(f"[int8 rows] special values {K} {dtype}")
        codes, scales = tg.quantize_int8(x.to(dtype).cuda())
        want, scale = plain_rows(x.to(dtype))
        assert same_scales(scales, scale) and scales.cpu().isnan().sum() == 3
        assert torch.equal(codes.cpu(), want)


def exact(a, b, ascale, bscale, bias, op, out_dtype):
    """(value in 64 bits, how far off it may be) of one group."""
    total = (a.double() @ (b.double().t() if op == "T" else b.double())).float()       # whole numbers below 2^53: exact
    x = total * bscale
    v = x.double() * ascale.double()[:, None] + (bias.double() if bias is not None else 0.0)
    return v, v.abs() * U32 * (1 + U32) + (v.abs() * U16 * (1 + U32) if out_dtype is BF16 else 0.0)


def within(got, want, tol, what):
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def codes(seed, *shape):
    return torch.randint(-128, 128, shape, generator=gen(seed), dtype=I8)


SIZES = [(1, 1, 1), (1, 40, 24), (3, 5, 7), (16, 64, 64), (17, 33, 65), (5, 1, 130), (33, 257, 1), (64, 128, 128),
         (48, 256, 384), (100, 130, 15), (129, 127, 129), (130, 300, 257), (256, 256, 256), (200, 1000, 513),
         (300, 200, 2049), (257, 513, 1023), (64, 1000, 4096), (16, 4096, 512), (1, 3000, 3000), (700, 900, 640)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(gpu_available, op, M, N, K):
    a, b = codes(M + K, M, K), codes(N + K, *((N, K) if op == "T" else (K, N)))
    ascale, bscale = torch.rand(M, generator=gen(1)) * 0.1, torch.rand(N, generator=gen(2)) * 0.1
    bias = torch.randn(N, generator=gen(3)) * 10
    for pad, offset, out_dtype, with_bias in ((0, 0, BF16, True), (16 - K % 16, 0, F32, False), (3, 1, F32, True),
                                              (0, 5, BF16, False)):
        say(f"[int8] {M}x{N}x{K} op={op} pad={pad} offset={offset} {out_dtype} bias={with_bias}")
        out = tg.int8_gemm(padded(a, pad, offset), padded(b, pad, offset), ascale.cuda(), bscale.cuda(),
                           bias=bias.cuda() if with_bias else None, op_b=op, out_dtype=out_dtype)
        want, tol = exact(a, b, ascale, bscale, bias if with_bias else None, op, out_dtype)
        within(out, want, tol, (pad, offset, out_dtype))


def ends_of(sizes):
    return torch.tensor(sizes).cumsum(0).to(torch.int32)


GROUPS = [([4], 4), ([0, 3, 0, 5], 8), ([1, 1, 1, 1], 9), ([33, 0, 64, 31], 140), ([300, 0, 17], 317), ([0, 0], 5),
          ([128, 128], 256), ([700, 1, 90], 800), (list(range(70)), 2500), ([2] * 200, 400)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("sizes,M", GROUPS, ids=lambda v: str(v)[:20])
@pytest.mark.parametrize("N,K", [(40, 24), (130, 257), (256, 384)])
def test_grouped_product(gpu_available, op, sizes, M, N, K):
    G = len(sizes)
    a, b = codes(M + K, M, K), codes(N + K, G, *((N, K) if op == "T" else (K, N)))
    ascale, bscale = torch.rand(M, generator=gen(1)), torch.rand(G, N, generator=gen(2)) + 0.1
    bias = torch.randn(G, N, generator=gen(3)) * 100
    ends = ends_of(sizes)
    for pad, offset, out_dtype, with_bias in ((-K % 16, 0, BF16, True), (3, 1, F32, False)):
        say(f"[int8 grouped] {sizes} of {M} x {N} x {K} op={op} pad={pad} {out_dtype}")
        out = torch.full((M, N + 3), 7.0, dtype=out_dtype, device="cuda")
        tg.int8_gemm(padded(a, pad, offset), padded(b, pad, offset), ascale.cuda(), bscale.cuda(), ends=ends.cuda(),
                     bias=bias.cuda() if with_bias else None, op_b=op, out=out[:, :N])
        first = 0
        for g, end in enumerate(ends.tolist()):
            if end > first:
                want, tol = exact(a[first:end], b[g], ascale[first:end], bscale[g], bias[g] if with_bias else None, op,
                                  out_dtype)
                within(out[first:end, :N], want, tol, (g, pad))
            first = end
        assert (out[first:, :N] == 0).all() and (out[:, N:] == 7.0).all()


def test_sums_are_exact_to_the_largest_depth(gpu_available):
    K = 131071
    a, b = torch.full((3, K), -128, dtype=I8), torch.full((2, K), -128, dtype=I8)
    b[1] = 127
    a[2, 1::2] = 127
    one = torch.ones(3).cuda()
    for pad in (1, 0):
        say(f"[int8] K={K} pad={pad}")
        out = tg.int8_gemm(padded(a, pad), padded(b, pad), one, one[:2], out_dtype=F32)
        want = a.double() @ b.double().t()
        assert want.abs().max() == 128 * 128 * K and torch.equal(out.cpu(), want.float())


def test_scales_shared_and_special(gpu_available):
    M, N, K = 40, 70, 300
    a, b = codes(1, M, K), codes(2, N, K)
    one = torch.full((1,), 0.5).cuda()
    say("[int8] one scale for all rows and columns")
    out = tg.int8_gemm(a.cuda(), b.cuda(), one.expand(M), one.expand(N), out_dtype=F32)
    assert torch.equal(out.cpu().double(), 0.25 * (a.double() @ b.double().t()))
    ascale = torch.ones(M)
    ascale[3], ascale[4] = float("nan"), float("inf")
    say("[int8] NaN and infinite scales stay in their rows")
    out = tg.int8_gemm(a.cuda(), b.cuda(), ascale.cuda(), torch.ones(N).cuda(), out_dtype=F32).cpu()
    assert out[3].isnan().all() and not out[4].isfinite().any() and out[5:].isfinite().all() and out[:3].isfinite().all()


def test_empty_calls(gpu_available):
    z = lambda *s: torch.zeros(s, dtype=I8, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    say("[int8] empty calls")
    assert tg.int8_gemm(z(0, 8), z(5, 8), f(0), f(5)).shape == (0, 5)
    assert tg.int8_gemm(z(4, 8), z(0, 8), f(4), f(0)).shape == (4, 0)
    out = tg.int8_gemm(z(4, 0), z(5, 0), f(4), f(5), bias=2 * f(5))
    assert (out == 2).all()
    ends = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    out = tg.int8_gemm(z(4, 0), z(2, 5, 0), f(4), f(2, 5), ends=ends, bias=2 * f(2, 5))
    assert (out[:3] == 2).all() and (out[3:] == 0).all()
    out = tg.int8_gemm(z(4, 8), z(0, 5, 8), f(4), f(0, 5), ends=ends[:0])
    assert out.shape == (4, 5) and (out == 0).all()
    q, s = tg.quantize_int8(f(0, 8))
    assert q.shape == (0, 8) and s.shape == (0,)


def test_refusals(gpu_available):
    z = lambda *s: torch.zeros(s, dtype=I8, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    ends = torch.tensor([1, 4], dtype=torch.int32, device="cuda")
    for error, call in [
            (TypeError, lambda: tg.int8_gemm(f(4, 8), z(5, 8), f(4), f(5))),
            (TypeError, lambda: tg.int8_gemm(z(4, 8), f(5, 8), f(4), f(5))),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 9), f(4), f(5))),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(5), f(5))),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(4))),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), bias=f(4))),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), bias=f(10)[::2])),
            (TypeError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5).bfloat16())),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5).cpu())),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(2, 5, 8), f(4), f(2, 5))),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), ends=ends)),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(3, 5, 8), f(4), f(3, 5), ends=ends)),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), op_b="X")),
            (ValueError, lambda: tg.int8_gemm(z(8, 4).t(), z(5, 8), f(4), f(5))),
            (TypeError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), out_dtype=torch.float8_e4m3fn)),
            (TypeError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), out_dtype=I8)),
            (ValueError, lambda: tg.int8_gemm(z(4, 8), z(5, 8), f(4), f(5), out=f(4, 4))),
            (tg.GemmError, lambda: tg.int8_gemm(z(1, 131072), z(1, 131072), f(1), f(1))),
            (TypeError, lambda: tg.quantize_int8(z(4, 8))), (ValueError, lambda: tg.quantize_int8(f(4, 8).cpu())),
            (ValueError, lambda: tg.quantize_int8(f(8))), (TypeError, lambda: tg.quantize_int8(f(4, 8), out=f(4, 8))),
            (ValueError, lambda: tg.quantize_int8(f(4, 8), scales=f(5))),
            (ValueError, lambda: tg.quantize_int8(f(4, 8), scales=f(8)[::2]))]:
        with pytest.raises(error):
            call()
