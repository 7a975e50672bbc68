"""The expert layer's products at sizes that reach each tile, each depth of
staging and each way of loading, and the skinny and general kernels around
their limits, against 64-bit references.

Tolerances are test_experts.py's: (K + 6) roundings of 2^-24 of the sum of
magnitudes, 2^-10 of it for fp8, and half a step of the stored type.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_experts import BF16, F32, FP8, U32, ends_of, f64, fp8_matrix, gen, padded, product_tol, values, within

pytestmark = pytest.mark.gpu

UNIT = {F32: 4, BF16: 8, FP8: 16}                    # elements in 16 bytes
# A row this long (bytes) puts a panel of 256 rows past 2^31.
FAR = 2 ** 31 // 256


def operands(dtype, M, N, K, op, seed, groups=0):
    """A (M x K), B (as stored), their values in 64 bits (B's as K x N) and the scales."""
    shape = (N, K) if op == "T" else (K, N)
    if dtype == FP8:
        q, sa = fp8_matrix(M, K, seed, 1)
        pairs = [fp8_matrix(*shape, seed + 1 + g, 128) for g in range(max(groups, 1))]
        w = torch.stack([p.view(torch.uint8) for p, _ in pairs]).view(FP8)
        sb = torch.stack([s for _, s in pairs])
        a, b = values(q, sa, 1), values(w, sb, 128)
    else:
        q = torch.randn(M, K, generator=gen(seed)).to(dtype)
        w = torch.randn(max(groups, 1), *shape, generator=gen(seed + 1)).to(dtype)
        sa = sb = None
        a, b = f64(q), f64(w)
    b = b.transpose(1, 2) if op == "T" else b
    return q, w, a, b, sa, sb


def run(dtype, op, x, w, sa, sb, ends, kind, M, N, alpha=0.5):
    extra = {"a_scales": sa.cuda(), "b_scales": sb.cuda()} if dtype == FP8 else {}
    out = padded(torch.ones(M, N).to(kind), 3)
    back = out.as_strided((M, N + 3), (N + 3, 1))
    got = tg.grouped_gemm(x, w, ends, op_b=op, alpha=alpha, out=out, **extra)
    assert back[:-1, N:].isnan().all()
    return got


def check_one(dtype, op, M, N, K, pads=(0, 1), kinds=(F32, BF16)):
    q, w, a, b, sa, sb = operands(dtype, M, N, K, op, M + N + K)
    want = 0.5 * (a @ b[0])
    ends = ends_of([M]).cuda()
    for pad in pads:
        x, y = padded(q, -K % UNIT[dtype] + pad), padded(w, -w.shape[2] % UNIT[dtype] + pad)
        for kind in kinds:
            got = run(dtype, op, x, y, sa, sb, ends, kind, M, N)
            within(got, want, product_tol(a, b[0], want, dtype == FP8, kind, 0.5), (pad, kind))


# The last slab whole, cut at 16 bytes, cut inside 16 bytes.
TILES = [(3500, 3500, 256), (3500, 3490, 131), (3000, 2900, 144), (1500, 2900, 201), (1500, 2901, 256),
         (1300, 2500, 521), (520, 4000, 528), (1300, 2500, 200), (400, 2500, 1101), (400, 2500, 2100),
         (400, 2500, 207), (100, 500, 200), (129, 515, 77), (2500, 2900, 193)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
@pytest.mark.parametrize("M,N,K", TILES)
def test_tiles_of_every_size(gpu_available, dtype, op, M, N, K):
    say(f"[tiles] {dtype} op={op} {M}x{N}x{K}")
    check_one(dtype, op, M, N, K)


# Few tiles and a long k: its slabs shared out among a workgroup's waves, unevenly.
@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
@pytest.mark.parametrize("M,N,K", [(100, 520, 2111), (40, 2001, 4096), (250, 1000, 1043), (65, 129, 9000),
                                   (70, 4000, 528), (1, 7000, 1500), (90, 90, 300)])
def test_few_tiles_of_a_long_product(gpu_available, dtype, op, M, N, K):
    say(f"[few tiles] {dtype} op={op} {M}x{N}x{K}")
    check_one(dtype, op, M, N, K)


# 256 x 256 tiles: one whole turn of 256 compute units and 64 tiles more (four workgroups to each), 121
# (two to each), 144 (left whole); and the same at sizes that leave rows and columns of the parts empty.
@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("M,N,K", [(5000, 4096, 300), (3300, 7400, 272), (6400, 4096, 300), (4900, 3968, 256),
                                   (3201, 7300, 390)])
def test_tiles_past_the_last_whole_turn(gpu_available, dtype, op, M, N, K):
    say(f"[last turn] {dtype} op={op} {M}x{N}x{K}")
    check_one(dtype, op, M, N, K, pads=(0,), kinds=(F32,))


def uneven(M, groups):
    """Rows of each group: the first of every four empty, the second a single row, the rest unlike each other."""
    part = [0 if g % 4 == 0 else 1 if g % 4 == 1 else 3 + 5 * g for g in range(groups)]
    part[-1] += M - 7 - sum(part)
    return part


GROUPS = [(1000, 2900, 520, 16), (3000, 2900, 520, 32), (2000, 2890, 521, 32), (4000, 2000, 520, 32), (500, 1500, 527, 16),
          (8192, 2048, 600, 8), (9000, 2496, 304, 70)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
@pytest.mark.parametrize("M,N,K,groups", GROUPS)
def test_tiles_of_groups(gpu_available, dtype, op, M, N, K, groups):
    say(f"[tiles] {dtype} op={op} {M}x{N}x{K} in {groups} groups")
    sizes = uneven(M, groups)
    q, w, a, b, sa, sb = operands(dtype, M, N, K, op, 7, groups)
    ends = ends_of(sizes).cuda()
    for pad in (0, 1):
        x, y = padded(q, -K % UNIT[dtype] + pad), padded(w, -w.shape[2] % UNIT[dtype] + pad)
        got = run(dtype, op, x, y, sa, sb, ends, F32, M, N)
        at = 0
        for g, size in enumerate(sizes):
            want = 0.5 * (a[at:at + size] @ b[g])
            within(got[at:at + size], want, product_tol(a[at:at + size], b[g], want, dtype == FP8, F32, 0.5), (pad, g))
            at += size
        assert (got[at:] == 0).all() and at == M - 7


# Rows in one tile of 16, 32 and 64; columns enough for one workgroup of 32 on each compute unit, and for two.
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(1, 64), (49, 1024), (50, 1037), (8200, 130), (8201, 647), (16400, 128), (16385, 517)])
def test_few_rows(gpu_available, dtype, M, N, K):
    say(f"[few rows] {dtype} {M}x{N}x{K}")
    check_one(dtype, "T", M, N, K, pads=(0,))


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (65, 130, 1), (70, 129, 3), (3, 2, 40), (130, 3, 200), (64, 64, 7),
                                   (200, 70, 15)])
def test_rows_shorter_than_a_load(gpu_available, dtype, op, M, N, K):
    say(f"[short] {dtype} op={op} {M}x{N}x{K}")
    check_one(dtype, op, M, N, K)


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("dtype", [F32, BF16, FP8])
@pytest.mark.parametrize("side", ["A", "B"])
def test_rows_far_apart(gpu_available, dtype, op, side):
    M, N, K = 67, 33, 65
    say(f"[far] {dtype} op={op} {side}")
    size = dtype.itemsize
    q, w, a, b, sa, sb = operands(dtype, M, N, K, op, 5)
    want = 0.5 * (a @ b[0])
    t = q if side == "A" else w[0]
    rows, cols = t.shape
    raw = torch.uint8 if dtype == FP8 else dtype
    far = torch.empty(((rows - 1) * FAR) // size + cols, dtype=raw, device="cuda")
    far = far.as_strided((rows, cols), (FAR // size, 1))
    far.copy_(t.view(raw))
    far = far.view(FP8) if dtype == FP8 else far
    x = far if side == "A" else padded(q, -K % UNIT[dtype])
    y = far[None] if side == "B" else padded(w, -w.shape[2] % UNIT[dtype])
    got = run(dtype, op, x, y, sa, sb, ends_of([M]).cuda(), F32, M, N)
    within(got, want, product_tol(a, b[0], want, dtype == FP8, F32, 0.5), side)


WGRADS = [(100, 8, 2000, 520), (100, 8, 2990, 520), (301, 3, 1500, 1111), (100, 8, 256, 1500), (100, 8, 130, 3001),
          (2500, 8, 128, 1000), (4000, 3, 130, 264), (9000, 7, 65, 96), (50000, 64, 24, 40), (3200, 65, 40, 72),
          (100, 2, 128, 128), (1000, 8, 1500, 520), (77, 2, 1, 300), (77, 2, 300, 3)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,groups,N,K", WGRADS)
def test_weight_gradients_of_every_tile(gpu_available, dtype, M, groups, N, K):
    say(f"[wgrad tiles] {dtype} {groups} groups of {M} rows {N}x{K}")
    sizes = [0] * groups
    sizes[0], sizes[-1] = M // 3, M - M // 3 - 5 * (groups > 2)
    if groups > 2:
        sizes[1] = 1
    dy, x = torch.randn(M, N, generator=gen(4)).to(dtype), torch.randn(M, K, generator=gen(5)).to(dtype)
    used = sum(sizes)
    dy[used:], x[used:] = float("nan"), float("nan")
    ends = ends_of(sizes).cuda()
    c0 = torch.randn(groups, N, K, generator=gen(6))
    for pad in (0, 1):
        dyd, xd = padded(dy, -N % 8 + pad), padded(x, -K % 8 + pad)
        for beta in (0.0, 1.0):
            out = padded(c0 if beta else torch.full((groups, N, K), float("nan")), 1)
            got = tg.grouped_wgrad(dyd, xd, ends, alpha=0.5, beta=beta, out=out)
            at = 0
            for g, size in enumerate(sizes):
                old = beta * f64(c0[g])
                if size == 0:
                    assert torch.equal(got[g].cpu(), beta * c0[g]), g
                    continue
                p, q = f64(dy[at:at + size]), f64(x[at:at + size])
                want = 0.5 * (p.t() @ q) + old
                within(got[g], want, (0.5 * (p.abs().t() @ q.abs()) + old.abs()) * (size + 4) * U32, (pad, beta, g))
                at += size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,groups,N,K", [(1800, 3, 632, 2136), (300, 8, 256, 1912)])
def test_weight_gradients_of_128_x_128_tiles(gpu_available, dtype, M, groups, N, K):
    test_weight_gradients_of_every_tile(gpu_available, dtype, M, groups, N, K)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weight_gradients_of_rows_far_apart(gpu_available, dtype):
    M, N, K = 35, 70, 65
    say(f"[wgrad far] {dtype}")
    dy, x = torch.randn(M, N, generator=gen(4)).to(dtype), torch.randn(M, K, generator=gen(5)).to(dtype)
    ld = FAR // dtype.itemsize
    far = torch.empty((M - 1) * ld + K, dtype=dtype, device="cuda").as_strided((M, K), (ld, 1))
    far.copy_(x)
    got = tg.grouped_wgrad(dy.cuda(), far, ends_of([M]).cuda())
    want = f64(dy).t() @ f64(x)
    within(got[0], want, (f64(dy).abs().t() @ f64(x).abs()) * (M + 4) * U32, "far")
