"""Layer norm's weight and bias gradients add rows that cancel without losing the rest.

A team of threads sums the rows that it takes in fp32; the teams' sums are added in 64 bits.  Here every team
takes one row, whose dy * n (n is 1 or -1) and dy are exact, and so are the sums of a workgroup's four teams: the
sum over all of them is below 2^53 and whole, so it is exact, and so is the result, below 2^24.
"""
import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say

pytestmark = pytest.mark.gpu

BIG = 2.0 ** 27            # fp32 holds multiples of 16 from here on
WIDTHS = [64, 1024, 2048, 4096, 8192, 16384, 32768]          # every shape of a row


def gradients(column, N, dtype):
    """(dweight, dbias) where every column of dy is `column` and the norm's rows are 1, -1, 1, ..."""
    sign = torch.ones(N).index_fill_(0, torch.arange(1, N, 2), -1.0)
    dy = torch.tensor(column)[:, None].expand(-1, N).to(dtype).cuda().contiguous()
    s = sign.expand(len(column), -1).to(dtype).cuda().contiguous()
    _, dw, db = tg.layer_norm_backward(dy, s, torch.ones(N, dtype=dtype, device="cuda"), eps=0.0)
    return dw.cpu() * sign, db.cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", WIDTHS)
def test_sums_over_teams(gpu_available, dtype, N):
    M = 512
    column = [0.0, 1.0, 0.0, 0.0] * (M // 4)
    column[:4], column[-4:] = [BIG, 0.0, 0.0, 0.0], [0.0, 0.0, 0.0, -BIG]
    say(f"[layer norm] sums over teams {dtype} {M}x{N}")
    for got in gradients(column, N, dtype):
        assert (got == M // 4 - 2).all(), got[:4]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", WIDTHS)
def test_sums_over_a_workgroups_teams(gpu_available, dtype, N):
    say(f"[layer norm] sums over a workgroup's teams {dtype} {N}")
    for column, want in (([BIG, 3.0, -BIG, 0.0], 3), ([3.0, BIG, 5.0, -BIG], 8), ([-BIG, 1.0, 1.0, BIG], 2)):
        for got in gradients(column, N, dtype):
            assert (got == want).all(), (column, got[:4])
