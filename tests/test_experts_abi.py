"""Argument checks of the sparse expert layer's entry points (CPU only: they
come back before any HIP call), and the bound on the row tiles of a grouped
launch."""
import itertools
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

import tiled_gemm_f32_amd as tg
from tiled_gemm_f32_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, FP8 = tg.GEMM_DTYPE_F32, tg.GEMM_DTYPE_BF16F32, tg.GEMM_DTYPE_FP8F32
N_, T_ = tg.GEMM_OP_N, tg.GEMM_OP_T
OK, INVALID, UNSUP, SCRATCH = tg.GEMM_OK, tg.GEMM_ERR_INVALID_ARG, tg.GEMM_ERR_UNSUPPORTED, tg.GEMM_ERR_SCRATCH
# Well-aligned stand-in device addresses: only inspected.
PA, PB, PC, PD = 0x7f0000000000, 0x7f1000000000, 0x7f2000000000, 0x7f3000000000
BIG = 2 ** 31


def scales(a=PA, a_row=1, a_block=1, b=PB, b_n=1, b_k=1, b_group=1):
    return tg.BlockScales(a, a_row, a_block, b, b_n, b_k, b_group)


def quant(dtype=F32, block=1, M=4, K=256, X=PA, ldx=256, Q=PB, ldq=256, s=PC, lds=2):
    return tg.gemm_quantize(dtype, block, M, K, X, ldx, Q, ldq, s, lds)


def norm(dtype=BF16, M=4, N=256, X=PA, ldx=256, res=0, ldr=0, w=PB, eps=1e-6, total=0, ldt=0, kind=tg.GEMM_OUT_BF16,
         out=PC, ldo=256, s=0, lds=0):
    return tg.gemm_rms_norm(dtype, M, N, X, ldx, res, ldr, w, eps, total, ldt, kind, out, ldo, s, lds)


def grad(dtype=BF16, M=4, N=256, dY=PA, lddy=256, S=PB, lds=256, w=PC, eps=1e-6, dS=0, ldds=0, dX=PD, lddx=256, dw=0,
         ws=0, nbytes=0):
    return tg.gemm_rms_norm_backward(dtype, M, N, dY, lddy, S, lds, w, eps, dS, ldds, dX, lddx, dw, ws, nbytes)


def block(op=T_, M=4, N=256, K=128, alpha=1.0, A=PA, lda=128, B=PB, ldb=None, sc="fine", kind=tg.GEMM_OUT_BF16, out=PC,
          ldo=256):
    ldb = (K if op == T_ else N) if ldb is None else ldb
    return tg.gemm_block_scaled(op, M, N, K, alpha, A, lda, B, ldb, scales() if sc == "fine" else sc, kind, out, ldo)


def grouped(dtype=BF16, op=T_, groups=3, ends=PD, M=4, N=256, K=128, alpha=1.0, A=PA, lda=128, B=PB, ldb=None,
            stride=1 << 16, sc=None, kind=tg.GEMM_OUT_BF16, out=PC, ldo=256):
    ldb = (K if op == T_ else N) if ldb is None else ldb
    return tg.gemm_grouped(dtype, op, groups, ends, M, N, K, alpha, A, lda, B, ldb, stride, sc, kind, out, ldo)


def wgrad(dtype=BF16, groups=3, ends=PD, M=4, N=256, K=128, alpha=1.0, dY=PA, lddy=256, X=PB, ldx=128, beta=0.0, dW=PC,
          ldw=128, stride=256 * 128):
    return tg.gemm_grouped_wgrad(dtype, groups, ends, M, N, K, alpha, dY, lddy, X, ldx, beta, dW, ldw, stride)


REFUSED = [
    (quant, dict(dtype=FP8)), (quant, dict(dtype=9)), (quant, dict(block=2)), (quant, dict(block=0)),
    (quant, dict(M=-1)), (quant, dict(K=-1)), (quant, dict(ldx=255)), (quant, dict(ldq=255)), (quant, dict(lds=1)),
    (quant, dict(X=0)), (quant, dict(Q=0)), (quant, dict(s=0)), (quant, dict(X=PA + 2)), (quant, dict(s=PC + 2)),
    (quant, dict(dtype=BF16, X=PA + 1)),
    (norm, dict(dtype=FP8)), (norm, dict(kind=3)), (norm, dict(kind=-1)), (norm, dict(M=-1)), (norm, dict(N=-1)),
    (norm, dict(ldx=255)), (norm, dict(ldo=255)), (norm, dict(res=PD, ldr=255)), (norm, dict(total=PD, ldt=255)),
    (norm, dict(eps=-1e-6)), (norm, dict(eps=float("nan"))), (norm, dict(eps=float("inf"))), (norm, dict(X=0)),
    (norm, dict(w=0)), (norm, dict(out=0)), (norm, dict(X=PA + 1)), (norm, dict(res=PD + 1, ldr=256)),
    (norm, dict(total=PD + 1, ldt=256)), (norm, dict(out=PC + 1)), (norm, dict(kind=tg.GEMM_OUT_FP8)),
    (norm, dict(kind=tg.GEMM_OUT_FP8, s=PD, lds=1)), (norm, dict(kind=tg.GEMM_OUT_FP8, s=PD + 2, lds=2)),
    (grad, dict(dtype=FP8)), (grad, dict(M=-1)), (grad, dict(N=-1)), (grad, dict(lddy=255)), (grad, dict(lds=255)),
    (grad, dict(lddx=255)), (grad, dict(dS=PD, ldds=255)), (grad, dict(eps=-1.0)), (grad, dict(dY=0)),
    (grad, dict(S=0)), (grad, dict(w=0)), (grad, dict(dX=0)), (grad, dict(dY=PA + 1)), (grad, dict(nbytes=-1)),
    (grad, dict(dw=PA + 2, ws=PA, nbytes=1 << 30)), (grad, dict(dw=PA, ws=PA + 2, nbytes=1 << 30)),
    (block, dict(op=2)), (block, dict(M=-1)), (block, dict(N=-1)), (block, dict(K=-1)), (block, dict(lda=127)),
    (block, dict(ldb=127)), (block, dict(op=N_, ldb=255)), (block, dict(ldo=255)), (block, dict(A=0)),
    (block, dict(B=0)), (block, dict(out=0)), (block, dict(out=PC + 1)), (block, dict(kind=5)),
    (block, dict(sc=None)), (block, dict(sc=scales(a=0))), (block, dict(sc=scales(b=0))),
    (block, dict(sc=scales(a=PA + 2))), (block, dict(sc=scales(a_row=-1))), (block, dict(sc=scales(b_n=-1))),
    (block, dict(sc=scales(b_k=-1))), (block, dict(sc=scales(a_block=-1))), (block, dict(sc=scales(b_group=-1))),
    (grouped, dict(dtype=9)), (grouped, dict(op=-1)), (grouped, dict(groups=-1)), (grouped, dict(ends=0)),
    (grouped, dict(ends=PD + 2)), (grouped, dict(M=-1)), (grouped, dict(lda=127)), (grouped, dict(stride=-1)),
    (grouped, dict(sc=scales())), (grouped, dict(dtype=FP8)), (grouped, dict(A=PA + 1)), (grouped, dict(B=0)),
    (grouped, dict(dtype=F32, B=PB + 2)), (grouped, dict(kind=tg.GEMM_OUT_F32, out=PC + 2)),
    (wgrad, dict(dtype=9)), (wgrad, dict(groups=-1)), (wgrad, dict(ends=0)), (wgrad, dict(N=-1)),
    (wgrad, dict(lddy=255)), (wgrad, dict(ldx=127)), (wgrad, dict(ldw=127)), (wgrad, dict(stride=256 * 128 - 1)),
    (wgrad, dict(stride=-1)), (wgrad, dict(dW=0)), (wgrad, dict(dW=PC + 2)), (wgrad, dict(X=0)), (wgrad, dict(dY=0)),
    (wgrad, dict(dY=PA + 1)),
]


@pytest.mark.parametrize("fn,kwargs", REFUSED, ids=lambda v: v.__name__ if callable(v) else str(sorted(v))[:40])
def test_invalid_calls_are_refused(fn, kwargs):
    assert fn(**kwargs) == INVALID


@pytest.mark.parametrize("fn,kwargs", [
    (quant, dict(M=BIG)), (quant, dict(ldx=BIG)), (norm, dict(M=BIG)), (norm, dict(ldo=BIG)), (grad, dict(lddx=BIG)),
    (block, dict(M=BIG)), (block, dict(lda=BIG)), (block, dict(kind=tg.GEMM_OUT_FP8)),
    (grouped, dict(groups=65536)), (grouped, dict(kind=tg.GEMM_OUT_FP8)),
    (grouped, dict(M=BIG - 1, N=BIG - 1, ldo=BIG - 1)), (wgrad, dict(groups=65536)), (wgrad, dict(dtype=FP8)),
    (wgrad, dict(N=BIG - 1, K=BIG - 1, lddy=BIG - 1, ldx=BIG - 1, ldw=BIG - 1, stride=(BIG - 1) * (BIG - 1))),
])
def test_calls_outside_what_the_kernels_index_are_unsupported(fn, kwargs):
    assert fn(**kwargs) == UNSUP


@pytest.mark.parametrize("ldw,stride,fine", [
    (128, 256 * 128, True), (3 * 128, 128, True), (400, 130, True), (128, 255 * 128 + 127, False), (3 * 128 - 1, 128, False),
    (400, 127, False), (128, 128, False), (128, 0, False), (2 ** 31 - 1, 2 ** 30, False), (128, 2 ** 62, True),
    (400, 2 ** 47, True)])
def test_results_of_groups_may_take_turns_but_not_overlap(ldw, stride, fine):
    assert (wgrad(ldw=ldw, stride=stride) == INVALID) == (not fine)


@pytest.mark.parametrize("fn,kwargs", [
    (quant, dict(M=0, X=0, Q=0, s=0)), (quant, dict(K=0, X=0, Q=0, s=0)), (norm, dict(M=0, X=0, w=0, out=0)),
    (norm, dict(N=0, X=0, w=0, out=0)), (grad, dict(M=0, dY=0, S=0, w=0, dX=0)), (grad, dict(N=0, dY=0, S=0, dX=0)),
    (block, dict(M=0, A=0, out=0)), (block, dict(N=0, B=0, out=0)), (grouped, dict(M=0, A=0, out=0, ends=0)),
    (grouped, dict(N=0, B=0, out=0, ends=0)), (wgrad, dict(groups=0, dW=0, ends=0)), (wgrad, dict(N=0, dW=0)),
    (wgrad, dict(K=0, dW=0)),
])
def test_empty_calls_do_nothing(fn, kwargs):
    assert fn(**kwargs) == OK


def test_workspace_of_the_norm_gradient():
    assert tg.gemm_rms_norm_workspace_size(0, 128) == 0 == tg.gemm_rms_norm_workspace_size(128, 0)
    assert tg.gemm_rms_norm_workspace_size(-1, 5) == 0
    need = tg.gemm_rms_norm_workspace_size(100, 256)
    assert need > 0 and need % (4 * 256) == 0
    assert grad(M=100, dw=PA, ws=0, nbytes=need) == SCRATCH
    assert grad(M=100, dw=PA, ws=PB, nbytes=need - 1) == SCRATCH
    # never more partial rows than rows (up to a workgroup's four), nor an unbounded number of them
    for M, N in itertools.product([1, 3, 100, 5000, 10 ** 6], [1, 777, 4096, 8192, 16384, 50000]):
        rows = tg.gemm_rms_norm_workspace_size(M, N) // (4 * N)
        assert 1 <= rows <= min(2048, M + 3)


def test_torch_wrappers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 128)
    ends = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        tg.quantize(x)
    with pytest.raises(TypeError):
        tg.quantize(x.double())
    with pytest.raises(ValueError):
        tg.rms_norm(x, torch.ones(128))
    with pytest.raises(ValueError):
        tg.rms_norm_backward(x, x, torch.ones(128))
    with pytest.raises(ValueError):
        tg.block_gemm(x.to(torch.float8_e4m3fn), x.to(torch.float8_e4m3fn), x, x, op_b="X")
    with pytest.raises(ValueError):
        tg.grouped_gemm(x, torch.zeros(2, 8, 128), ends)
    with pytest.raises(TypeError):
        tg.grouped_gemm(x.half(), torch.zeros(2, 8, 128).half(), ends)
    with pytest.raises(ValueError):
        tg.grouped_wgrad(x, x, ends)


def test_row_tile_bound_holds_for_every_division():
    """most_row_tiles against the largest count over divisions of M rows."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tempfile.mkdtemp(prefix="tiles_")
    try:
        src = os.path.join(d, "t.cpp")
        with open(src, "w") as f:
            f.write("#include <cstdint>\n#include <cstdio>\n")
            text = open(os.path.join(ROOT, "tiled_gemm_f32_amd", "csrc", "gemm_grouped.hpp")).read()
            at = text.index("inline int64_t most_row_tiles")
            f.write(text[at:text.index("\n}\n", at) + 3])
            f.write("int main(){long m,g,t;while(scanf(\"%ld %ld %ld\",&m,&g,&t)==3)"
                    "printf(\"%ld\\n\",(long)most_row_tiles(m,g,t,true));}\n")
        exe = os.path.join(d, "t")
        subprocess.run(["g++", "-O1", "-o", exe, src], check=True)
        asked = [(m, g, t) for m in range(1, 14) for g in range(0, 4) for t in (1, 2, 4)]
        out = subprocess.run([exe], input="\n".join("%d %d %d" % a for a in asked), capture_output=True, text=True,
                             check=True).stdout.split()
        for (m, g, t), got in zip(asked, map(int, out)):
            most = 0
            for cut in itertools.combinations_with_replacement(range(m + 1), g):
                edges = (0,) + cut + (m,)
                most = max(most, sum(-(-(b - a) // t) for a, b in zip(edges, edges[1:])))
            assert got == most, (m, g, t, got, most)
    finally:
        shutil.rmtree(d, ignore_errors=True)


def test_every_new_entry_point_is_bound():
    for name in ("gemm_quantize", "gemm_rms_norm", "gemm_rms_norm_backward", "gemm_block_scaled", "gemm_grouped",
                 "gemm_grouped_wgrad", "gemm_rms_norm_workspace_size"):
        assert name in _lib.EXPORTED and hasattr(tg, name)
