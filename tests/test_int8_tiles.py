"""Products of 8-bit integers at sizes that reach each tile, each depth of
staging and each way of loading, the kernels for few rows and few tiles, and
the general kernel around their limits, against exact sums (test_int8.py).
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_int8 import BF16, F32, codes, ends_of, exact, gen, padded, within

pytestmark = pytest.mark.gpu

# A row this long (bytes) puts a panel of 256 rows past 2^31.
FAR = 2 ** 31 // 256


def check(op, M, N, K, sizes=None, pads=(0, 1), kinds=(F32, BF16)):
    """`sizes`: rows of each group (None: one product without groups)."""
    G = len(sizes or [0])
    a, b = codes(M + K, M, K), codes(N + K, G, *((N, K) if op == "T" else (K, N)))
    ascale, bscale, bias = torch.rand(M, generator=gen(1)), torch.rand(G, N, generator=gen(2)), torch.randn(G, N, generator=gen(3))
    ends = None if sizes is None else ends_of(sizes).cuda()
    pick = (lambda t: t) if sizes is not None else (lambda t: t[0])
    want = []
    first = 0
    for g, n in enumerate(sizes or [M]):
        rows = slice(first, first + n)
        want.append((rows, [exact(a[rows], b[g], ascale[rows], bscale[g], bias[g], op, k) for k in kinds]))
        first += n
    for pad in pads:
        x, w = padded(a, -K % 16 + pad), padded(b, -b.shape[2] % 16 + pad)
        for i, kind in enumerate(kinds):
            back = torch.full((M, N + 3), 7.0, dtype=kind, device="cuda")
            tg.int8_gemm(x, pick(w), ascale.cuda(), pick(bscale).cuda(), ends=ends, bias=pick(bias).cuda(), op_b=op,
                         out=back[:, :N])
            got = back.cpu()
            assert (got[:, N:] == 7.0).all() and (got[first:, :N] == 0).all()
            for rows, pairs in want:
                within(got[rows, :N], *pairs[i], (rows, pad, kind))


# The last slab whole, cut at 16 bytes, cut inside 16 bytes.
TILES = [(3500, 3500, 256), (3500, 3490, 131), (3000, 2900, 144), (1500, 2900, 201), (1500, 2901, 256),
         (1300, 2500, 521), (520, 4000, 528), (1300, 2500, 200), (400, 2500, 1101), (400, 2500, 2100),
         (400, 2500, 207), (100, 500, 200), (129, 515, 77), (2500, 2900, 193)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K", TILES)
def test_tiles_of_every_size(gpu_available, op, M, N, K):
    say(f"[int8 tiles] op={op} {M}x{N}x{K}")
    check(op, M, N, K)


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K", [(100, 520, 2111), (40, 2001, 4096), (250, 1000, 1043), (65, 129, 9000),
                                   (70, 4000, 528), (1, 7000, 1500), (90, 90, 300), (33, 40, 50000)])
def test_few_tiles_of_a_long_product(gpu_available, op, M, N, K):
    say(f"[int8 few tiles] op={op} {M}x{N}x{K}")
    check(op, M, N, K)


# 256 x 256 tiles: one whole turn of 256 compute units and 64 tiles more, 121, 144; and parts left empty.
@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K", [(5000, 4096, 300), (3300, 7400, 272), (6400, 4096, 300), (4900, 3968, 256),
                                   (3201, 7300, 390)])
def test_tiles_past_the_last_whole_turn(gpu_available, op, M, N, K):
    say(f"[int8 last turn] op={op} {M}x{N}x{K}")
    check(op, M, N, K, pads=(0,), kinds=(F32,))


def uneven(M, groups):
    """Rows of each group: the first of every four empty, the second a single row, the rest unlike each other."""
    part = [0 if g % 4 == 0 else 1 if g % 4 == 1 else 3 + 5 * g for g in range(groups)]
    part[-1] += M - 7 - sum(part)
    return part


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K,groups", [(1000, 2900, 520, 16), (3000, 2900, 520, 32), (2000, 2890, 521, 32),
                                          (500, 1500, 527, 16), (8192, 2048, 600, 8), (9000, 2496, 304, 70)])
def test_tiles_of_groups(gpu_available, op, M, N, K, groups):
    say(f"[int8 tiles] op={op} {M}x{N}x{K} in {groups}")
    check(op, M, N, K, sizes=uneven(M, groups), pads=(0, 3), kinds=(BF16,))


# Few rows in all, in every shape of the streaming kernel, and one row past its tiles.
@pytest.mark.parametrize("M,N,K,groups", [(1, 300, 1000, 0), (16, 4100, 2048, 0), (17, 9000, 336, 0), (33, 700, 1041, 0),
                                          (64, 20000, 160, 0), (65, 512, 640, 0), (3, 100, 16, 0), (16, 16, 33000, 0),
                                          (64, 500, 700, 32), (200, 1000, 512, 13), (900, 300, 272, 20), (5, 4096, 144, 64)])
def test_few_rows(gpu_available, M, N, K, groups):
    say(f"[int8 few rows] {M}x{N}x{K} in {groups}")
    if groups:
        order = torch.randperm(M, generator=gen(M)) % groups
        check("T", M, N, K, sizes=torch.bincount(order, minlength=groups).tolist())
    else:
        check("T", M, N, K)


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("far", ["a", "b"])
def test_rows_far_apart(gpu_available, op, far):
    M, N, K = 40, 24, 48
    say(f"[int8 far] op={op} {far}")
    a, b = codes(1, M, K), codes(2, *((N, K) if op == "T" else (K, N)))
    ascale, bscale = torch.rand(M, generator=gen(1)), torch.rand(N, generator=gen(2))
    move = lambda t, long: padded(t, FAR + 5 - t.shape[1]) if long else t.cuda()  # noqa: E731
    out = tg.int8_gemm(move(a, far == "a"), move(b, far == "b"), ascale.cuda(), bscale.cuda(), op_b=op, out_dtype=F32)
    within(out, *exact(a, b, ascale, bscale, None, op, F32), far)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M,N,K", [(70, 90, 15), (70, 15, 90), (300, 7, 3), (1, 1, 131071), (64, 64, 16)])
def test_short_rows(gpu_available, op, M, N, K):
    say(f"[int8 short] op={op} {M}x{N}x{K}")
    check(op, M, N, K)
    check(op, M, N, K, sizes=[M // 2, 0, M - M // 2])


def test_rows_do_not_depend_on_the_others(gpu_available):
    """A row's result is the same in any call that holds it."""
    N, K = 500, 900
    a, b = codes(1, 600, K).cuda(), codes(2, N, K).cuda()
    s, t = torch.rand(600, generator=gen(1)).cuda(), torch.rand(N, generator=gen(2)).cuda()
    say("[int8] rows alone and together")
    whole = tg.int8_gemm(a, b, s, t, out_dtype=F32)
    for lo, hi in ((0, 1), (3, 20), (100, 164), (5, 505), (0, 600)):
        assert torch.equal(tg.int8_gemm(a[lo:hi], b, s[lo:hi], t, out_dtype=F32), whole[lo:hi])
