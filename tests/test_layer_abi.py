"""Argument checks of layer norm, the 8-bit products and the routing (CPU only:
they come back before any HIP call), and the plan's workspace."""
import itertools

import pytest
import torch

import tiled_gemm_f32_amd as tg
from tiled_gemm_f32_amd import _lib

F32, BF16, FP8 = tg.GEMM_DTYPE_F32, tg.GEMM_DTYPE_BF16F32, tg.GEMM_DTYPE_FP8F32
N_, T_ = tg.GEMM_OP_N, tg.GEMM_OP_T
OK, INVALID, UNSUP, SCRATCH = tg.GEMM_OK, tg.GEMM_ERR_INVALID_ARG, tg.GEMM_ERR_UNSUPPORTED, tg.GEMM_ERR_SCRATCH
O32, O16, O8, OI = tg.GEMM_OUT_F32, tg.GEMM_OUT_BF16, tg.GEMM_OUT_FP8, tg.GEMM_OUT_INT8
# Well-aligned stand-in device addresses: only inspected.
PA, PB, PC, PD = 0x7f0000000000, 0x7f1000000000, 0x7f2000000000, 0x7f3000000000
BIG = 2 ** 31


def norm(dtype=BF16, M=4, N=256, X=PA, ldx=256, res=0, ldr=0, w=PB, b=0, eps=1e-5, total=0, ldt=0, kind=O16, out=PC,
         ldo=256, s=0, lds=0):
    return tg.gemm_layer_norm(dtype, M, N, X, ldx, res, ldr, w, b, eps, total, ldt, kind, out, ldo, s, lds)


def grad(dtype=BF16, M=4, N=256, dY=PA, lddy=256, S=PB, lds=256, w=PC, eps=1e-5, dS=0, ldds=0, dX=PD, lddx=256, dw=0,
         db=0, ws=0, nbytes=0):
    return tg.gemm_layer_norm_backward(dtype, M, N, dY, lddy, S, lds, w, eps, dS, ldds, dX, lddx, dw, db, ws, nbytes)


def quant(dtype=F32, M=4, K=256, X=PA, ldx=256, Q=PB, ldq=256, s=PC):
    return tg.gemm_quantize_int8(dtype, M, K, X, ldx, Q, ldq, s)


def scales(a=PA, a_row=1, b=PB, b_col=1, b_group=1, bias=0, bias_group=0):
    return tg.Int8Scales(a, a_row, b, b_col, b_group, bias, bias_group)


def product(op=T_, groups=1, ends=0, M=4, N=256, K=128, A=PA, lda=128, B=PB, ldb=None, stride=0, sc="fine", kind=O16,
            out=PC, ldo=256):
    ldb = (K if op == T_ else N) if ldb is None else ldb
    return tg.gemm_int8(op, groups, ends, M, N, K, A, lda, B, ldb, stride, scales() if sc == "fine" else sc, kind, out, ldo)


def plan(size=8, tokens=4, top=2, groups=3, experts=PA, ld=2, order=PB, place=PC, ends=PD, ws=0, nbytes=0):
    return tg.gemm_expert_plan(size, tokens, top, groups, experts, ld, order, place, ends, ws, nbytes)


def dispatch(size=2, tokens=4, top=2, N=256, X=PA, ldx=256, place=PB, last=PC, rows=8, out=PD, ldo=256, cols=0, s=0, lds=0,
             t=0, ldt=0):
    return tg.gemm_dispatch(size, tokens, top, N, X, ldx, place, last, rows, out, ldo, cols, s, lds, t, ldt)


def combine(dtype=BF16, tokens=4, top=2, N=256, rows=PA, ldr=256, n=8, place=PB, w=PC, ldw=2, res=0, ldres=0, out=PD,
            ldo=256):
    return tg.gemm_combine(dtype, tokens, top, N, rows, ldr, n, place, w, ldw, res, ldres, out, ldo)


def back(dtype=BF16, tokens=4, top=2, N=256, dout=PA, lddo=256, rows=PA, ldr=256, n=8, place=PB, last=PC, w=PC, ldw=2,
         drows=PD, lddr=256, dw=PB, lddw=2):
    return tg.gemm_combine_backward(dtype, tokens, top, N, dout, lddo, rows, ldr, n, place, last, w, ldw, drows, lddr, dw, lddw)


REFUSED = [
    (norm, dict(dtype=FP8)), (norm, dict(kind=4)), (norm, dict(kind=-1)), (norm, dict(M=-1)), (norm, dict(N=-1)),
    (norm, dict(ldx=255)), (norm, dict(ldo=255)), (norm, dict(res=PD, ldr=255)), (norm, dict(total=PD, ldt=255)),
    (norm, dict(eps=-1e-6)), (norm, dict(eps=float("nan"))), (norm, dict(eps=float("inf"))), (norm, dict(X=0)),
    (norm, dict(w=0)), (norm, dict(out=0)), (norm, dict(X=PA + 1)), (norm, dict(w=PB + 1)), (norm, dict(b=PB + 1)),
    (norm, dict(dtype=F32, b=PB + 2)), (norm, dict(res=PD + 1, ldr=256)), (norm, dict(total=PD + 1, ldt=256)),
    (norm, dict(out=PC + 1)), (norm, dict(kind=O32, out=PC + 2)), (norm, dict(kind=O8)), (norm, dict(kind=O8, s=PD, lds=1)),
    (norm, dict(kind=O8, s=PD + 2, lds=2)), (norm, dict(kind=OI)), (norm, dict(kind=OI, s=PD, lds=0)),
    (norm, dict(kind=OI, s=PD + 2, lds=1)),
    (grad, dict(dtype=FP8)), (grad, dict(M=-1)), (grad, dict(N=-1)), (grad, dict(lddy=255)), (grad, dict(lds=255)),
    (grad, dict(lddx=255)), (grad, dict(dS=PD, ldds=255)), (grad, dict(eps=-1.0)), (grad, dict(dY=0)),
    (grad, dict(S=0)), (grad, dict(w=0)), (grad, dict(dX=0)), (grad, dict(dY=PA + 1)), (grad, dict(nbytes=-1)),
    (grad, dict(dw=PA + 2, ws=PA, nbytes=1 << 30)), (grad, dict(db=PA + 2, ws=PA, nbytes=1 << 30)),
    (grad, dict(dw=PA, ws=PA + 2, nbytes=1 << 30)),
    (quant, dict(dtype=FP8)), (quant, dict(dtype=9)), (quant, dict(M=-1)), (quant, dict(K=-1)), (quant, dict(ldx=255)),
    (quant, dict(ldq=255)), (quant, dict(X=0)), (quant, dict(Q=0)), (quant, dict(s=0)), (quant, dict(X=PA + 2)),
    (quant, dict(s=PC + 2)), (quant, dict(dtype=BF16, X=PA + 1)),
    (product, dict(op=2)), (product, dict(M=-1)), (product, dict(N=-1)), (product, dict(K=-1)), (product, dict(lda=127)),
    (product, dict(ldb=127)), (product, dict(op=N_, ldb=255)), (product, dict(ldo=255)), (product, dict(A=0)),
    (product, dict(B=0)), (product, dict(out=0)), (product, dict(out=PC + 1)), (product, dict(kind=O32, out=PC + 2)),
    (product, dict(kind=5)), (product, dict(sc=None)), (product, dict(sc=scales(a=0))), (product, dict(sc=scales(b=0))),
    (product, dict(sc=scales(a=PA + 2))), (product, dict(sc=scales(b=PA + 2))), (product, dict(sc=scales(bias=PA + 2))),
    (product, dict(sc=scales(a_row=-1))), (product, dict(sc=scales(b_col=-1))), (product, dict(sc=scales(b_group=-1))),
    (product, dict(sc=scales(bias_group=-1))), (product, dict(groups=-1, ends=PD)), (product, dict(groups=2)),
    (product, dict(groups=2, ends=PD + 2)), (product, dict(groups=2, ends=PD, stride=-1)),
    (plan, dict(size=2)), (plan, dict(tokens=-1)), (plan, dict(top=0)), (plan, dict(groups=0)), (plan, dict(ld=1)),
    (plan, dict(experts=0)), (plan, dict(experts=PA + 4)), (plan, dict(size=4, experts=PA + 2)), (plan, dict(place=0)),
    (plan, dict(ends=0)), (plan, dict(ends=PD + 2)), (plan, dict(order=PB + 2)), (plan, dict(place=PC + 1)),
    (plan, dict(nbytes=-1)), (plan, dict(ws=PA + 2, nbytes=1 << 20)),
    (dispatch, dict(size=3)), (dispatch, dict(size=8)), (dispatch, dict(tokens=-1)), (dispatch, dict(top=0)),
    (dispatch, dict(N=-1)), (dispatch, dict(rows=-1)), (dispatch, dict(cols=-1)), (dispatch, dict(ldx=255)),
    (dispatch, dict(ldo=255)), (dispatch, dict(X=0)), (dispatch, dict(X=PA + 1)), (dispatch, dict(place=0)),
    (dispatch, dict(place=PB + 2)), (dispatch, dict(last=PC + 2)), (dispatch, dict(out=0)), (dispatch, dict(out=PD + 1)),
    (dispatch, dict(cols=3, s=PA, lds=2, t=PB, ldt=3)), (dispatch, dict(cols=3, s=PA, lds=3, t=PB, ldt=2)),
    (dispatch, dict(cols=1, s=0, lds=1, t=PB, ldt=1)), (dispatch, dict(cols=1, s=PA, lds=1, t=0, ldt=1)),
    (dispatch, dict(cols=1, s=PA + 2, lds=1, t=PB, ldt=1)),
    (combine, dict(dtype=FP8)), (combine, dict(tokens=-1)), (combine, dict(top=0)), (combine, dict(N=-1)),
    (combine, dict(n=-1)), (combine, dict(ldr=255)), (combine, dict(ldo=255)), (combine, dict(ldw=1)),
    (combine, dict(res=PA, ldres=255)), (combine, dict(rows=0)), (combine, dict(rows=PA + 1)), (combine, dict(place=0)),
    (combine, dict(w=PC + 2)), (combine, dict(res=PA + 1, ldres=256)), (combine, dict(out=0)), (combine, dict(out=PD + 1)),
    (back, dict(dtype=FP8)), (back, dict(tokens=-1)), (back, dict(top=0)), (back, dict(N=-1)), (back, dict(n=-1)),
    (back, dict(lddo=255)), (back, dict(ldr=255)), (back, dict(lddr=255)), (back, dict(ldw=1)), (back, dict(lddw=1)),
    (back, dict(dout=0)), (back, dict(dout=PA + 1)), (back, dict(rows=0)), (back, dict(place=0)), (back, dict(w=0)),
    (back, dict(last=PC + 2)), (back, dict(drows=0)), (back, dict(drows=PD + 1)), (back, dict(dw=PB + 2)),
    (back, dict(n=0, place=0)), (back, dict(n=0, w=0)),
]


@pytest.mark.parametrize("fn,kwargs", REFUSED, ids=lambda v: v.__name__ if callable(v) else str(sorted(v))[:40])
def test_invalid_calls_are_refused(fn, kwargs):
    assert fn(**kwargs) == INVALID


@pytest.mark.parametrize("fn,kwargs", [
    (norm, dict(M=BIG)), (norm, dict(ldo=BIG)), (norm, dict(kind=OI, s=PD, lds=BIG)), (grad, dict(lddx=BIG)),
    (quant, dict(M=BIG)), (quant, dict(ldx=BIG)), (product, dict(M=BIG)), (product, dict(lda=BIG)),
    (product, dict(K=131072, lda=131072)), (product, dict(kind=O8)), (product, dict(kind=OI)),
    (product, dict(groups=65536, ends=PD)), (product, dict(M=BIG - 1, N=BIG - 1, ldo=BIG - 1)),
    (plan, dict(groups=4097)), (plan, dict(tokens=BIG)), (plan, dict(tokens=2 ** 29 + 1)), (plan, dict(ld=BIG)),
    (dispatch, dict(tokens=BIG)), (dispatch, dict(tokens=2 ** 30, top=2)), (dispatch, dict(rows=BIG)),
    (dispatch, dict(ldo=BIG)), (dispatch, dict(cols=1, s=PA, lds=BIG, t=PB, ldt=1)), (combine, dict(N=BIG, ldr=BIG, ldo=BIG)),
    (combine, dict(tokens=2 ** 30)), (combine, dict(ldw=BIG)), (combine, dict(n=BIG)), (back, dict(n=BIG)),
    (back, dict(lddw=BIG)), (back, dict(tokens=2 ** 30)),
])
def test_calls_outside_what_the_kernels_index_are_unsupported(fn, kwargs):
    assert fn(**kwargs) == UNSUP


@pytest.mark.parametrize("fn,kwargs", [
    (norm, dict(M=0, X=0, w=0, out=0)), (norm, dict(N=0, X=0, w=0, out=0)), (norm, dict(M=0, X=0, w=0, out=0, kind=OI, lds=1)),
    (grad, dict(M=0, dY=0, S=0, w=0, dX=0)), (grad, dict(N=0, dY=0, S=0, dX=0)), (quant, dict(M=0, X=0, Q=0, s=0)),
    (quant, dict(K=0, X=0, Q=0, s=0)), (product, dict(M=0, A=0, out=0)), (product, dict(N=0, B=0, out=0)),
    (dispatch, dict(rows=0, out=0)), (dispatch, dict(N=0, X=0, out=0)), (dispatch, dict(tokens=0, X=0, place=0, last=0)),
    (combine, dict(tokens=0, out=0)), (combine, dict(N=0, rows=0, out=0)), (back, dict(tokens=0, last=0)),
    (back, dict(n=0, dw=0, drows=0, place=0, w=0)), (back, dict(tokens=0, n=0, drows=0)),
])
def test_empty_calls_do_nothing(fn, kwargs):
    assert fn(**kwargs) == OK


def test_workspaces():
    for M, N in ((0, 128), (128, 0), (-1, 5), (BIG, 5)):
        assert tg.gemm_layer_norm_workspace_size(M, N) == 0
    need = tg.gemm_layer_norm_workspace_size(100, 256)
    assert need > 0 and need % (8 * 256) == 0
    for wanted in (dict(dw=PA), dict(db=PA), dict(dw=PA, db=PB)):
        assert grad(M=100, ws=0, nbytes=need, **wanted) == SCRATCH
        assert grad(M=100, ws=PB, nbytes=need - 1, **wanted) == SCRATCH
    # never more partial rows than rows (up to a workgroup's four), nor an unbounded number of them
    for M, N in itertools.product([1, 3, 100, 5000, 10 ** 6], [1, 777, 4096, 8192, 16384, 50000]):
        rows = tg.gemm_layer_norm_workspace_size(M, N) // (8 * N)
        assert 1 <= rows <= min(2048, M + 3)
    for tokens, top, groups in ((0, 2, 3), (4, 0, 3), (4, 2, 0), (-1, 2, 3), (4, 2, 4097), (BIG, 2, 3), (16, 4, 32)):
        assert tg.gemm_expert_plan_workspace_size(tokens, top, groups) == 0
    need = tg.gemm_expert_plan_workspace_size(100000, 8, 64)
    assert 0 < need <= 128 * 64 * 4 and need % (64 * 4) == 0
    assert plan(tokens=100000, top=8, ld=8, groups=64, ws=0, nbytes=need) == SCRATCH
    assert plan(tokens=100000, top=8, ld=8, groups=64, ws=PA, nbytes=need - 1) == SCRATCH


def test_torch_wrappers_refuse_host_tensors_and_wrong_types():
    x, q = torch.zeros(4, 128), torch.zeros(4, 128, dtype=torch.int8)
    e = torch.zeros(4, 2, dtype=torch.int64)
    place, ends, w = e.int(), torch.zeros(2, dtype=torch.int32), torch.ones(4, 2)
    for error, call in [
            (ValueError, lambda: tg.layer_norm(x, torch.ones(128))), (TypeError, lambda: tg.layer_norm(x.double(), x[0])),
            (ValueError, lambda: tg.layer_norm_backward(x, x, torch.ones(128))), (ValueError, lambda: tg.quantize_int8(x)),
            (TypeError, lambda: tg.quantize_int8(x.half())), (ValueError, lambda: tg.int8_gemm(q, q, x[:, 0], x[:, 0])),
            (ValueError, lambda: tg.int8_gemm(q, q, x[:, 0], x[:, 0], op_b="X")), (ValueError, lambda: tg.expert_plan(e, 3)),
            (TypeError, lambda: tg.expert_plan(w, 3)), (ValueError, lambda: tg.dispatch(x, place, ends)),
            (TypeError, lambda: tg.dispatch(x.half(), place, ends)), (ValueError, lambda: tg.combine(x, place)),
            (TypeError, lambda: tg.combine(x.half(), place)),
            (ValueError, lambda: tg.combine_backward(x, x, place, w, ends)),
            (TypeError, lambda: tg.combine_backward(x.half(), x, place, w, ends))]:
        with pytest.raises(error):
            call()


def test_every_new_entry_point_is_bound():
    for name in ("gemm_layer_norm", "gemm_layer_norm_workspace_size", "gemm_layer_norm_backward", "gemm_quantize_int8",
                 "gemm_int8", "gemm_expert_plan", "gemm_expert_plan_workspace_size", "gemm_dispatch", "gemm_combine",
                 "gemm_combine_backward"):
        assert name in _lib.EXPORTED and hasattr(tg, name)
