"""The torch wrappers' two ways: _torch_calls for the common case, Python for
the rest.  Both give the same results, and _torch_calls answers None (so that
the wrapper takes the call) to whatever it does not take."""
import pytest
import torch

import tiled_gemm_f32_amd as tg

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def calls():
    tg.load()
    from tiled_gemm_f32_amd import _torch_calls
    return _torch_calls


def test_calls_outside_the_common_case_are_left_to_the_wrappers(calls):
    x, w = torch.zeros(4, 8), torch.ones(8)
    q, s = torch.zeros(4, 8, dtype=FP8), torch.ones(4, 1)
    ends = torch.tensor([4], dtype=torch.int32)
    for got in (calls.quantize(x, 1, 0, 0), calls.quantize(x, 7, 0, 0), calls.quantize(x, "1", 0, 0),
                calls.quantize(None, 1, 0, 0), calls.quantize(x, 1), calls.quantize(x, 1, "0", 0),
                calls.rms_norm(x, w, None, 1e-5, None, 0, 0), calls.rms_norm(x, None, x, 1e-5, FP8, 0, 0),
                calls.rms_norm(x, w, None, "1e-5", 3, 0, 0), calls.rms_norm_backward(x, x, w, None, 1e-5, 0, 0),
                calls.rms_norm_backward(x, x, w, 1, None, 0, 0), calls.block_gemm(q, q, s, s, "T", 1.0, None, 0, 0),
                calls.block_gemm(q, q, None, None, "X", None, None, 0, 0),
                calls.grouped_gemm(x, x[None], ends, None, None, "T", 1.0, None, 0, 0),
                calls.grouped_gemm(1, 2, 3, 4, 5, 6, 7, 8, 0, 0), calls.grouped_wgrad(x, x, ends, 1.0, 0, 0),
                calls.grouped_wgrad(x, x, None, None, 0, 0)):
        assert got is None


def same(a, b):
    for p, q in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
        assert (p is None) == (q is None)
        if p is not None:
            assert p.dtype == q.dtype and p.shape == q.shape and p.stride() == q.stride() and p.device == q.device
            assert torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 40, 24), (5, 1, 130), (33, 257, 1), (48, 256, 384)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_both_ways_give_the_same(gpu_available, calls, M, N, K, dtype):
    print(f"[calls] {M}x{N}x{K} {dtype}", flush=True)
    g = torch.Generator().manual_seed(M + N + K)
    here = torch.cuda.current_stream().cuda_stream        # a stream passed in: the wrapper's own way
    x = torch.randn(M, K + 3, generator=g).to(dtype).cuda()[:, 1:K + 1]
    w = torch.nn.Parameter(torch.randn(K, generator=g).to(dtype).cuda())
    for rows in (1, 128):
        same(tg.quantize(x, rows), tg.quantize(x, rows, stream=here))
    for residual in (None, x + 1):
        for kind in (None, F32, BF16, FP8):
            same(tg.rms_norm(x, w, residual=residual, out_dtype=kind),
                 tg.rms_norm(x, w, residual=residual, out_dtype=kind, stream=here))
        same(tg.rms_norm_backward(x, x, w, dsum=residual), tg.rms_norm_backward(x, x, w, dsum=residual, stream=here))
    qa, sa = tg.quantize(x)
    ends = torch.tensor([M // 2, M // 2, M], dtype=torch.int32).cuda()
    for op in "TN":
        b = torch.randn(3, *((N, K) if op == "T" else (K, N)), generator=g).to(dtype).cuda()
        codes, scales = zip(*(tg.quantize(m, 128) for m in b))
        qb, sb = torch.stack([c.view(torch.uint8) for c in codes]).view(FP8), torch.stack(scales)
        for kind in (None, F32):
            same(tg.block_gemm(qa, qb[1], sa, sb[1], op_b=op, out_dtype=kind),
                 tg.block_gemm(qa, qb[1], sa, sb[1], op_b=op, out_dtype=kind, stream=here))
            same(tg.grouped_gemm(x, b, ends, op_b=op, alpha=0.5, out_dtype=kind),
                 tg.grouped_gemm(x, b, ends, op_b=op, alpha=0.5, out_dtype=kind, stream=here))
            same(tg.grouped_gemm(qa, qb, ends, a_scales=sa, b_scales=sb, op_b=op, out_dtype=kind),
                 tg.grouped_gemm(qa, qb, ends, a_scales=sa, b_scales=sb, op_b=op, out_dtype=kind, stream=here))
    dy = torch.randn(M, N, generator=g).to(dtype).cuda()
    same(tg.grouped_wgrad(dy, x, ends), tg.grouped_wgrad(dy, x, ends, stream=here))


@pytest.mark.gpu
def test_refusals_are_the_wrappers(gpu_available, calls):
    x = torch.zeros(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    with pytest.raises(TypeError):
        tg.quantize(x.half())
    with pytest.raises(ValueError):
        tg.quantize(x.t())
    with pytest.raises(ValueError):
        tg.rms_norm(x, w[:7])
    with pytest.raises(TypeError):
        tg.rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        tg.rms_norm(x, w, residual=x[:3])
    with pytest.raises(TypeError):
        tg.rms_norm(x, w, out_dtype=torch.float16)
    with pytest.raises(tg.GemmError):
        tg.rms_norm(x, w, eps=-1.0)
    q, s = tg.quantize(x)
    with pytest.raises(ValueError):
        tg.block_gemm(q, q, s, None)
    with pytest.raises(ValueError):
        tg.block_gemm(q, q, s[:3], s[:1])
    with pytest.raises(ValueError):
        tg.grouped_gemm(x, x[None], torch.tensor([4, 4], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        tg.grouped_wgrad(x, x[:3], torch.tensor([4], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        tg.grouped_wgrad(x, x, torch.tensor([4], dtype=torch.int32, device="cuda"), beta=1.0)


def stream_of(t):
    """The stream whose memory a tensor's is."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= t.data_ptr() < segment["address"] + segment["total_size"]:
            return segment["stream"]


@pytest.mark.gpu
def test_a_call_on_another_stream_allocates_there(gpu_available, calls):
    """Memory of the current stream may still be in use there when the other stream writes it."""
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(96, 256, generator=g).cuda(), torch.ones(256, device="cuda")
    qa, sa = tg.quantize(x)
    qb, sb = tg.quantize(x, 128)
    ends = torch.tensor([40, 96], dtype=torch.int32).cuda()
    b = torch.randn(2, 64, 256, generator=g).cuda()
    dy = torch.randn(96, 64, generator=g).cuda()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for call in (lambda h: tg.quantize(x, stream=h), lambda h: tg.quantize(x, 128, stream=h),
                 lambda h: tg.rms_norm(x, w, residual=x, out_dtype=FP8, stream=h),
                 lambda h: tg.rms_norm_backward(x, x, w, dsum=x, stream=h),
                 lambda h: (tg.block_gemm(qa, qb, sa, sb, stream=h),),
                 lambda h: (tg.grouped_gemm(x, b, ends, stream=h),),
                 lambda h: (tg.grouped_wgrad(dy, x, ends, stream=h),)):
        got = call(other.cuda_stream)
        assert [stream_of(t) for t in got] == [other.cuda_stream] * len(got)
        other.synchronize()
        same(got, call(None) if len(got) > 1 else (call(None)[0],))
    # the caller's own tensors stay its own
    out, kept = torch.empty(96, 256, device="cuda"), torch.empty(96, 256, device="cuda")
    got = tg.rms_norm(x, w, residual=x, out=out, summed=kept, stream=other.cuda_stream)
    assert got[0] is out and got[1] is kept and got[2] is None
    other.synchronize()
    same(got[:2], tg.rms_norm(x, w, residual=x)[:2])


@pytest.mark.gpu
def test_results_of_another_stream_may_be_dropped_on_the_current_one(gpu_available, calls):
    """While the current stream still has work, memory of a result that was dropped is not given to the other stream."""
    x = torch.ones(1024, 1024, device="cuda")
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    q, s = tg.quantize(x, stream=other.cuda_stream)
    other.synchronize()
    where = q.data_ptr()
    torch.cuda._sleep(20_000_000)
    use = q.view(torch.uint8).clone()
    del q
    with torch.cuda.stream(other):
        again = torch.empty(1024, 1024, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != where
    torch.cuda.synchronize()
    assert (use == use[0, 0]).all()


@pytest.mark.gpu
def test_the_default_streams_handle_is_the_default_stream(gpu_available, calls):
    """Handle 0 while another stream is the current one: the call runs behind the default stream's work."""
    x = torch.zeros(512, 512, device="cuda")
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        with torch.cuda.stream(default):
            torch.cuda._sleep(20_000_000)
            x.fill_(3.0)
        q, s = tg.quantize(x, stream=default.cuda_stream)
        torch.cuda.current_stream().wait_stream(default)
        assert stream_of(q) == stream_of(s) == default.cuda_stream == 0
        assert (q.float() == 448.0).all()
        # (Divided on the host: torch on the GPU multiplies by the rounded reciprocal.)
        assert (s.cpu() == torch.tensor(3.0) / 448.0).all()
