"""The operators of a sparse expert layer over torch tensors: block
quantisation to fp8, RMS norm with the residual's addition (and its
gradients), the fp8 product with a scale for each block of 128, and products
grouped by expert (and their weight gradients).

Like ``gemm``, these only read shapes, strides and pointers, allocate what
is not passed in, and forward to the C entry points of include/gemm.h, which
states each operator's formula.  Tensors are 2-D (or 3-D: a group's matrix
each) with unit stride along their last dimension; rows may be padded.  Work
goes to ``stream`` (an integer handle; None: torch's current stream) and no
call waits for the device.  What a call allocates belongs to the stream that
it runs on, so that the memory's earlier uses are over when the call writes
it; results made on another stream than torch's current one are recorded on
that one too, so that they may be used and dropped there once the caller has
ordered the two.
"""
from __future__ import annotations

from ._lib import (
    GEMM_DTYPE_BF16F32, GEMM_DTYPE_F32, GEMM_DTYPE_FP8F32, GEMM_OK, GEMM_OP_N, GEMM_OP_T, GEMM_OUT_BF16, GEMM_OUT_F32,
    GEMM_OUT_FP8, GEMM_SCALE_BLOCK, BlockScales, GemmError, gemm_block_scaled, gemm_grouped, gemm_grouped_wgrad,
    gemm_quantize, gemm_rms_norm, gemm_rms_norm_backward, gemm_rms_norm_workspace_size)


# A call costs the host about as long as a small kernel runs.  The common ones
# (outputs allocated here, the current device and stream) therefore go through
# _torch_calls, which checks, allocates and forwards them without Python in
# between, and answers None to anything else: that is done below, where the
# checks read each attribute of a tensor once, compare devices as numbers, and
# make messages only when something is wrong.

class _NoCalls:
    """Stands in for _torch_calls where it has not been built."""

    def __getattr__(self, name):
        return lambda *args: None


_calls = _device_of_calls = _stream_of_calls = None


def _common(name: str, *args):
    """The call in _torch_calls on the current device and stream; None if it is not one for it."""
    global _calls, _device_of_calls, _stream_of_calls
    if _calls is None:
        import torch
        from ._lib import load
        load()
        _device_of_calls, _stream_of_calls = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        try:
            from . import _torch_calls
            _calls = _torch_calls
        except ImportError:
            _calls = _NoCalls()
    device = _device_of_calls()
    got = getattr(_calls, name)(*args, device, _stream_of_calls(device))
    if type(got) is int:
        raise GemmError(got, name)
    return got


def _elsewhere(stream: int, like, fn, *args):
    """fn(*args) with `stream` as torch's current one, or None if it is that already (or `like` not on a GPU)."""
    import torch
    if not like.is_cuda:
        return None
    device = like.get_device()
    if stream == torch._C._cuda_getCurrentRawStream(device):
        return None
    caller = torch.cuda.current_stream(device)
    # (torch takes a handle of 0, the default stream, for none given, and makes a stream.)
    other = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(other):
        got = fn(*args)
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None and not any(t is a for a in args):
            t.record_stream(caller)
    return got


def _float_type(t, what: str) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return GEMM_DTYPE_BF16F32
    if t.dtype is torch.float32:
        return GEMM_DTYPE_F32
    raise TypeError(f"{what} must be float32 or bfloat16 (got {t.dtype})")


def _out_type(dtype, what: str) -> int:
    import torch
    if dtype is torch.bfloat16:
        return GEMM_OUT_BF16
    if dtype is torch.float8_e4m3fn:
        return GEMM_OUT_FP8
    if dtype is torch.float32:
        return GEMM_OUT_F32
    raise TypeError(f"{what} must be float32, bfloat16 or float8_e4m3fn (got {dtype})")


def _ld(t, what: str) -> int:
    """Leading dimension of a matrix (or of each matrix of a 3-D tensor)."""
    strides = t.stride()
    rows, cols = t.shape[-2:]
    if rows > 1 and cols > 1 and strides[-1] == 1 and strides[-2] >= cols:
        return strides[-2]
    if t.numel() == 0:
        return max(cols, 1)
    if cols > 1 and strides[-1] != 1:
        raise ValueError(f"{what} must have unit stride along its rows; got strides {strides}")
    if rows > 1 and strides[-2] < max(cols, 1):
        raise ValueError(f"{what} must be row-major with rows that do not overlap; got strides {strides}")
    return strides[-2] if rows > 1 else max(cols, 1)


def _device(t, what: str) -> int:
    """Number of the GPU a tensor is on."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a tensor on the GPU")
    return t.get_device()


def _check(t, what: str, device: int, shape=None, dtype=None, dim: int = 2):
    if t.get_device() != device or not t.is_cuda:
        raise ValueError(f"{what} must be a tensor on cuda:{device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype} (got {t.dtype})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if shape is None and t.dim() != dim:
        raise ValueError(f"{what} must be {dim}-D, got shape {tuple(t.shape)}")


def _blocks(n: int) -> int:
    return -(-n // GEMM_SCALE_BLOCK)


def _new(rows: int, cols: int, dtype, device, unit: int = 1):
    """(tensor, leading dimension): an uninitialised rows x cols matrix whose rows start on multiples of `unit`."""
    import torch
    ld = max(-(-cols // unit) * unit, 1)
    return torch.empty_strided((rows, cols), (ld, 1), dtype=dtype, device=device), ld


def _call(name: str, device: int, fn, *args):
    """fn(*args, stream) on GPU `device`, on its current stream."""
    import torch
    stream = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != GEMM_OK:
        raise GemmError(st, name)


def quantize(x, block_rows: int = 1, out=None, scales=None, stream=None):
    """(codes, scales) of a float32 or bfloat16 matrix in float8_e4m3fn.

    ``block_rows`` 1: a scale for every 128 columns of a row (activations;
    scales is rows x ceil(cols / 128)); 128: a scale for every 128 x 128 tile
    (weights).  ``x`` is about ``codes * scale`` of each block.  Codes
    allocated here have rows padded to 16 bytes."""
    import torch
    if out is None and scales is None and stream is None and x.is_cuda:
        got = _common("quantize", x, block_rows)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, x, quantize, x, block_rows, out, scales)
        if got is not None:
            return got
    dt = _float_type(x, "x")
    device = _device(x, "x")
    _check(x, "x", device)
    if block_rows not in (1, GEMM_SCALE_BLOCK):
        raise ValueError(f"block_rows is 1 or {GEMM_SCALE_BLOCK} (got {block_rows})")
    M, K = x.shape
    if out is None:
        out, ldq = _new(M, K, torch.float8_e4m3fn, x.device, 16)
    else:
        _check(out, "out", device, (M, K), torch.float8_e4m3fn)
        ldq = _ld(out, "out")
    if scales is None:
        scales, lds = _new(-(-M // block_rows), _blocks(K), torch.float32, x.device)
    else:
        _check(scales, "scales", device, (-(-M // block_rows), _blocks(K)), torch.float32)
        lds = _ld(scales, "scales")
    _call("quantize", device, gemm_quantize, dt, block_rows, M, K, x.data_ptr(), _ld(x, "x"),
          out.data_ptr(), ldq, scales.data_ptr(), lds)
    return out, scales


def rms_norm(x, weight, residual=None, eps: float = 1e-6, out_dtype=None, out=None, summed=None, scales=None,
             stream=None):
    """(out, summed, scales) of a row-wise RMS norm of ``x`` (+ ``residual``).

    x, residual (the same shape) and weight (one value a column) share a type,
    float32 or bfloat16.  ``summed`` is x + residual rounded to that type, the
    next residual (x itself without one); it may be passed as x or residual to
    update them in place.  ``out`` is float32, bfloat16 or float8_e4m3fn
    (``out_dtype``, by default x's type); with float8_e4m3fn ``scales`` holds
    a scale for every 128 columns of a row, otherwise it is None."""
    import torch
    if out is None and summed is None and scales is None and stream is None and x.is_cuda:
        got = _common("rms_norm", x, weight, residual, eps, out_dtype)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, x, rms_norm, x, weight, residual, eps, out_dtype, out, summed, scales)
        if got is not None:
            return got
    dt = _float_type(x, "x")
    device = _device(x, "x")
    _check(x, "x", device)
    M, N = x.shape
    _check(weight, "weight", device, (N,), x.dtype)
    if N > 1 and weight.stride(0) != 1:
        raise ValueError("weight must be contiguous")
    r_ptr = s_ptr = c_ptr = ldr = ld_sum = ld_scales = 0
    if residual is not None:
        _check(residual, "residual", device, (M, N), x.dtype)
        r_ptr, ldr = residual.data_ptr(), _ld(residual, "residual")
    if summed is not None:
        _check(summed, "summed", device, (M, N), x.dtype)
        s_ptr, ld_sum = summed.data_ptr(), _ld(summed, "summed")
    elif residual is not None:
        summed, ld_sum = _new(M, N, x.dtype, x.device)
        s_ptr = summed.data_ptr()
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        kind = _out_type(out.dtype, "out")
        _check(out, "out", device, (M, N))
        ldo = _ld(out, "out")
    else:
        kind = _out_type(out_dtype or x.dtype, "out")
        out, ldo = _new(M, N, out_dtype or x.dtype, x.device, 16 if kind == GEMM_OUT_FP8 else 1)
    if kind == GEMM_OUT_FP8:
        if scales is None:
            scales, ld_scales = _new(M, _blocks(N), torch.float32, x.device)
        else:
            _check(scales, "scales", device, (M, _blocks(N)), torch.float32)
            ld_scales = _ld(scales, "scales")
        c_ptr = scales.data_ptr()
    elif scales is not None:
        raise ValueError("scales go with a float8_e4m3fn output")
    _call("rms_norm", device, gemm_rms_norm, dt, M, N, x.data_ptr(), _ld(x, "x"), r_ptr, ldr,
          weight.data_ptr(), float(eps), s_ptr, ld_sum, kind, out.data_ptr(), ldo, c_ptr, ld_scales)
    return out, summed if summed is not None else x, scales


def rms_norm_backward(dy, summed, weight, dsum=None, eps: float = 1e-6, dx=None, want_dweight: bool = True,
                      stream=None):
    """(dx, dweight) of ``rms_norm``, from the gradient ``dy`` of its output.

    ``summed`` is what the forward pass returned; ``dsum`` the gradient that
    reaches it past the norm.  dx is the gradient of x and of the residual
    alike (it may be passed as dy or dsum); dweight is float32, or None if it
    is not wanted."""
    import torch
    if dx is None and want_dweight and stream is None and dy.is_cuda:
        got = _common("rms_norm_backward", dy, summed, weight, dsum, eps)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, dy, rms_norm_backward, dy, summed, weight, dsum, eps, dx, want_dweight)
        if got is not None:
            return got
    dt = _float_type(dy, "dy")
    device = _device(dy, "dy")
    _check(dy, "dy", device)
    M, N = dy.shape
    _check(summed, "summed", device, (M, N), dy.dtype)
    _check(weight, "weight", device, (N,), dy.dtype)
    if N > 1 and weight.stride(0) != 1:
        raise ValueError("weight must be contiguous")
    if dsum is not None:
        _check(dsum, "dsum", device, (M, N), dy.dtype)
    if dx is None:
        dx, lddx = _new(M, N, dy.dtype, dy.device)
    else:
        _check(dx, "dx", device, (M, N), dy.dtype)
        lddx = _ld(dx, "dx")
    dweight = None
    dw_ptr = ws_ptr = need = 0
    if want_dweight:
        need = gemm_rms_norm_workspace_size(M, N)
        dweight = torch.empty_strided((N,), (1,), dtype=torch.float32, device=dy.device)
        ws = torch.empty_strided((max(need, 4),), (1,), dtype=torch.uint8, device=dy.device)
        dw_ptr, ws_ptr = dweight.data_ptr(), ws.data_ptr()
    _call("rms_norm_backward", device, gemm_rms_norm_backward, dt, M, N, dy.data_ptr(), _ld(dy, "dy"),
          summed.data_ptr(), _ld(summed, "summed"), weight.data_ptr(), float(eps),
          dsum.data_ptr() if dsum is not None else 0, _ld(dsum, "dsum") if dsum is not None else 0, dx.data_ptr(), lddx,
          dw_ptr, ws_ptr, need)
    return dx, dweight


def _strides(scales, lead: int, shape, what: str):
    """Strides of a scale tensor's last two dimensions, after checking its shape."""
    if scales.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(scales.shape)}")
    strides = scales.stride()
    return strides[lead], strides[lead + 1]


def _block_scales(A, B, a_scales, b_scales, op_b: str, M: int, N: int, K: int, device: int):
    """The gemm_block_scales of a call.  b_scales follows B as it is stored:
    [group,] blocks of B's rows, blocks of its columns."""
    import torch
    for t, what in ((a_scales, "a_scales"), (b_scales, "b_scales")):
        if t is None:
            raise ValueError(f"float8_e4m3fn operands need {what}")
        if t.get_device() != device or t.dtype is not torch.float32:
            _check(t, what, device, t.shape, torch.float32)
    a_row, a_block = _strides(a_scales, 0, (M, _blocks(K)), "a_scales")
    lead = B.dim() - 2
    shape = tuple(B.shape[:lead]) + (_blocks(B.shape[-2]), _blocks(B.shape[-1]))
    rows, cols = _strides(b_scales, lead, shape, "b_scales")
    b_n, b_k = (rows, cols) if op_b == "T" else (cols, rows)
    return BlockScales(a_scales.data_ptr(), a_row, a_block, b_scales.data_ptr(), b_n, b_k,
                       b_scales.stride(0) if lead else 0)


def _product_out(M: int, N: int, out, out_dtype, default, like, device: int):
    """(out, its leading dimension, its type) of a product."""
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    kind = _out_type(out.dtype if out is not None else out_dtype or default, "out")
    if kind == GEMM_OUT_FP8:
        raise TypeError("out must be float32 or bfloat16")
    if out is not None:
        _check(out, "out", device, (M, N))
        return out, _ld(out, "out"), kind
    out, ldo = _new(M, N, out_dtype or default, like.device)
    return out, ldo, kind


def block_gemm(A, B, a_scales, b_scales, op_b: str = "T", alpha: float = 1.0, out=None, out_dtype=None, stream=None):
    """out = alpha * A @ op(B) of float8_e4m3fn operands with block scales.

    A is M x K with a_scales M x ceil(K / 128).  ``op_b`` "T": B is N x K, "N":
    K x N; b_scales has a scale for each 128 x 128 tile of B as it is stored,
    so a layer's weights and their scales serve its forward product ("T") and
    the gradient of its input ("N") alike.  ``out`` is bfloat16 by default,
    or float32."""
    import torch
    if out is None and stream is None and A.is_cuda:
        got = _common("block_gemm", A, B, a_scales, b_scales, op_b, alpha, out_dtype)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, A, block_gemm, A, B, a_scales, b_scales, op_b, alpha, out, out_dtype)
        if got is not None:
            return got
    if op_b not in ("N", "T"):
        raise ValueError("op_b is 'N' or 'T'")
    device = _device(A, "A")
    _check(A, "A", device, dtype=torch.float8_e4m3fn)
    _check(B, "B", device, dtype=torch.float8_e4m3fn)
    M, K = A.shape
    N, K2 = B.shape if op_b == "T" else (B.shape[1], B.shape[0])
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A {tuple(A.shape)}, op_b={op_b} {tuple(B.shape)}")
    sc = _block_scales(A, B, a_scales, b_scales, op_b, M, N, K, device)
    out, ldo, kind = _product_out(M, N, out, out_dtype, torch.bfloat16, A, device)
    _call("block_gemm", device, gemm_block_scaled, GEMM_OP_T if op_b == "T" else GEMM_OP_N, M, N, K,
          float(alpha), A.data_ptr(), _ld(A, "A"), B.data_ptr(), _ld(B, "B"), sc, kind, out.data_ptr(), ldo)
    return out


def _check_ends(ends, device: int, groups: int):
    import torch
    _check(ends, "ends", device, (groups,), torch.int32)
    if groups > 1 and ends.stride(0) != 1:
        raise ValueError("ends must be contiguous")


def grouped_gemm(A, B, ends, a_scales=None, b_scales=None, op_b: str = "T", alpha: float = 1.0, out=None,
                 out_dtype=None, stream=None):
    """out[i] = alpha * A[i] @ op(B[g]) for each row i of group g.

    A's rows are sorted by group; ``ends`` (int32, on the GPU) holds the row
    each group ends before, and is read there.  B is groups x N x K (``op_b``
    "T") or groups x K x N ("N").  Operands are float32, bfloat16, or
    float8_e4m3fn with scales as in ``block_gemm`` (b_scales with a leading
    dimension of groups).  Rows past the last end become zero.  ``out`` is
    float32 or bfloat16: by default A's type, bfloat16 for fp8."""
    import torch
    if out is None and stream is None and A.is_cuda:
        got = _common("grouped_gemm", A, B, ends, a_scales, b_scales, op_b, alpha, out_dtype)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, A, grouped_gemm, A, B, ends, a_scales, b_scales, op_b, alpha, out, out_dtype)
        if got is not None:
            return got
    if op_b not in ("N", "T"):
        raise ValueError("op_b is 'N' or 'T'")
    fp8 = A.dtype == torch.float8_e4m3fn
    dt = GEMM_DTYPE_FP8F32 if fp8 else _float_type(A, "A")
    device = _device(A, "A")
    _check(A, "A", device)
    _check(B, "B", device, dtype=A.dtype, dim=3)
    M, K = A.shape
    groups = B.shape[0]
    N, K2 = B.shape[1:] if op_b == "T" else (B.shape[2], B.shape[1])
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A {tuple(A.shape)}, op_b={op_b} {tuple(B.shape)}")
    _check_ends(ends, device, groups)
    sc = None
    if fp8:
        sc = _block_scales(A, B, a_scales, b_scales, op_b, M, N, K, device)
    elif a_scales is not None or b_scales is not None:
        raise ValueError("scales go with float8_e4m3fn operands")
    out, ldo, kind = _product_out(M, N, out, out_dtype, torch.bfloat16 if fp8 else A.dtype, A, device)
    _call("grouped_gemm", device, gemm_grouped, dt, GEMM_OP_T if op_b == "T" else GEMM_OP_N, groups,
          ends.data_ptr(), M, N, K, float(alpha), A.data_ptr(), _ld(A, "A"), B.data_ptr(), _ld(B, "B"),
          B.stride(0) if groups > 1 else 0, sc, kind, out.data_ptr(), ldo)
    return out


def grouped_wgrad(dy, x, ends, alpha: float = 1.0, beta: float = 0.0, out=None, stream=None):
    """out[g] = alpha * dy_g^T @ x_g + beta * out[g], over the rows of each group.

    dy is M x N and x M x K, both float32 or bfloat16, rows sorted by group as
    in ``grouped_gemm``; ``out`` is float32, groups x N x K (allocated when
    None; then beta must be 0).  A group without rows gives beta * out[g]."""
    import torch
    if out is None and beta == 0.0 and stream is None and dy.is_cuda:
        got = _common("grouped_wgrad", dy, x, ends, alpha)
        if got is not None:
            return got
    if stream is not None:
        got = _elsewhere(stream, dy, grouped_wgrad, dy, x, ends, alpha, beta, out)
        if got is not None:
            return got
    dt = _float_type(dy, "dy")
    device = _device(dy, "dy")
    _check(dy, "dy", device)
    _check(x, "x", device, dtype=dy.dtype)
    if x.shape[0] != dy.shape[0]:
        raise ValueError(f"dy and x differ in rows: {tuple(dy.shape)}, {tuple(x.shape)}")
    M, N = dy.shape
    K = x.shape[1]
    if ends.dim() != 1:
        raise ValueError(f"ends must be 1-D, got shape {tuple(ends.shape)}")
    groups = ends.shape[0]
    _check_ends(ends, device, groups)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input out")
        out = torch.empty((groups, N, K), dtype=torch.float32, device=dy.device)
    _check(out, "out", device, (groups, N, K), torch.float32)
    _call("grouped_wgrad", device, gemm_grouped_wgrad, dt, groups, ends.data_ptr(), M, N, K,
          float(alpha), dy.data_ptr(), _ld(dy, "dy"), x.data_ptr(), _ld(x, "x"), float(beta), out.data_ptr(),
          _ld(out, "out"), out.stride(0) if groups > 1 else 0)
    return out
