"""Sizes next to 2^31 and past it in the calls around the experts.  Nothing here runs a kernel: the calls
are refused."""
import ctypes

import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_experts_abi import grouped, wgrad
from test_layer_abi import INVALID, PA, PB, PD, UNSUP, back, combine, dispatch, plan, product

MOST = 2 ** 31 - 64          # the last count that a 32-bit number walks 64 at a time


@pytest.mark.parametrize("count", [MOST + 1, 2 ** 31 - 1])
def test_counts_that_a_32_bit_walk_would_pass_are_unsupported(count):
    assert combine(tokens=1, top=count, ldw=count) == UNSUP
    assert combine(tokens=1, top=count, w=0, ldw=0) == UNSUP
    assert back(tokens=1, top=count, ldw=count, lddw=count) == UNSUP
    assert back(tokens=1, top=count, ldw=count, dw=0, lddw=0) == UNSUP
    assert dispatch(tokens=1, top=count) == UNSUP
    assert dispatch(tokens=1, top=1, cols=count, s=PA, lds=count, t=PB, ldt=count) == UNSUP
    assert dispatch(tokens=0, top=1, cols=count, s=PA, lds=count, t=PB, ldt=count) == UNSUP


# Counts of groups and of a token's choices whose lower 32 bits are a small one.
@pytest.mark.parametrize("count", [2 ** 32 + 2, 2 ** 31, 2 ** 40 + 1, 2 ** 63 + 1])
def test_counts_past_32_bits_are_not_cut_to_them(count):
    assert plan(top=count, ld=count) == UNSUP
    assert plan(groups=count) == UNSUP
    assert dispatch(top=count) == UNSUP
    assert combine(top=count, ldw=2 ** 31 - 1) == UNSUP
    assert back(top=count, ldw=2 ** 31 - 1, lddw=2 ** 31 - 1) == UNSUP
    assert product(groups=count, ends=PD) == UNSUP
    assert grouped(groups=count) == UNSUP and wgrad(groups=count) == UNSUP
    assert tg.gemm_expert_plan_workspace_size(100000, 8, count) == 0
    assert tg.gemm_expert_plan_workspace_size(1, count, 8) == 0


@pytest.mark.parametrize("count", [-2 ** 32 + 2, -2 ** 31 - 1, -2 ** 40 + 1])
def test_negative_counts_past_32_bits_are_invalid(count):
    assert plan(top=count) == plan(groups=count) == dispatch(top=count) == combine(top=count) == INVALID
    assert back(top=count) == product(groups=count, ends=PD) == INVALID
    assert grouped(groups=count) == wgrad(groups=count) == INVALID
    assert tg.gemm_expert_plan_workspace_size(100000, 8, count) == 0


def test_counts_may_be_ctypes_values():
    two = ctypes.c_int32(2)
    assert tg.gemm_expert_plan_workspace_size(100000, two, ctypes.c_int32(64)) == \
        tg.gemm_expert_plan_workspace_size(100000, 2, 64) > 0
    assert plan(top=two, ld=1) == dispatch(top=two, ldx=1) == combine(top=two, ldr=1) == back(top=two, lddo=1) == INVALID
    assert grouped(groups=two, lda=1) == wgrad(groups=two, lddy=1) == product(groups=two, ends=PD, lda=1) == INVALID


@pytest.mark.gpu
def test_torch_calls_with_counts_past_32_bits(gpu_available):
    many = 2 ** 32 + 2
    say(f"[limits] {many} choices and groups")
    wide = torch.empty(1, many, dtype=torch.int32, device="cuda")          # 17 GB, never read
    ends, share = wide[0], wide.view(torch.float32)
    x, code = torch.ones(1, 1, device="cuda"), torch.ones(1, 1, dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    here = torch.cuda.current_stream().cuda_stream
    for way in ({}, {"stream": here}):
        for call in (lambda: tg.expert_plan(wide, 3, **way), lambda: tg.combine(x, wide, **way),
                     lambda: tg.combine(x, wide, share, **way),
                     lambda: tg.int8_gemm(code, code.expand(many, 1, 1), one, share.view(many, 1), ends=ends, **way),
                     lambda: tg.grouped_gemm(x, share.view(many, 1, 1), ends, **way)):
            with pytest.raises(tg.GemmError) as refused:
                call()
            assert refused.value.status == UNSUP
    del wide, ends, share
    torch.cuda.empty_cache()
