"""Norm gradients of more rows than the backward pass has teams, so that a team
takes three rows or more: the turns of the sums' two sets of slots, the weight
gradient over a team's rows (in registers, and in the workspace where rows are
long), and the last sum over all partial rows.  Every shape that a row is
shared out in, against test_experts.py's 64-bit reference.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_experts import BF16, F32, gen, padded, test_rms_norm_backward as check

pytestmark = pytest.mark.gpu

# One wave a row (2048 teams), four (768), sixteen with one and two chunks a lane (512), longer rows (512).
ROWS = [(6500, 264, 0, 0), (4200, 777, 1, 1), (1700, 1100, 3, 0), (2000, 4096, 0, 0), (1100, 5000, 8, 8),
        (1100, 8192, 0, 0), (1100, 12000, 1, 0), (1030, 16384, 0, 0), (1100, 17000, 0, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,pad,offset", ROWS)
def test_teams_of_several_rows(gpu_available, dtype, M, N, pad, offset):
    assert M > 2 * tg.gemm_rms_norm_workspace_size(M, N) // (4 * N) * (4 if N <= 1024 else 1)
    check(gpu_available, dtype, True, M, N, pad, offset)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N", [(9000, 520), (3100, 2500), (2100, 6001), (2100, 9000), (1600, 18000)])
def test_results_repeat(gpu_available, dtype, M, N):
    """The same bits in every call, with other work of other shapes between them."""
    say(f"[norm grad] repeats {dtype} {M}x{N}")
    g = torch.Generator(device="cuda").manual_seed(M + N)
    dy, s, ds = (torch.randn(M, N, device="cuda", generator=g).to(dtype) for _ in range(3))
    w = (1 + 0.2 * torch.randn(N, generator=gen(1))).to(dtype).cuda()
    small = padded(torch.randn(40, 300, generator=gen(2)).to(dtype))
    first = tg.rms_norm_backward(dy, s, w, dsum=ds)
    for _ in range(4):
        tg.rms_norm_backward(small, small, w[:300])
        again = tg.rms_norm_backward(dy, s, w, dsum=ds)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
