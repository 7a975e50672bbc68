"""What the torch wrappers allocate is seen by torch: dispatch modes, the filling of uninitialised memory in
deterministic mode, the profiler, inference mode."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import tiled_gemm_f32_amd as tg

from gpu_helpers import say

pytestmark = pytest.mark.gpu

FP8, BF16, I8 = torch.float8_e4m3fn, torch.bfloat16, torch.int8


class Seen(TorchDispatchMode):
    """Addresses of the tensors that were made while it was on."""

    def __init__(self):
        super().__init__()
        self.made = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor) and "empty" in str(func):
            self.made.add(out.data_ptr())
        return out


def cases():
    x = torch.randn(8, 256, device="cuda")
    w, one = torch.ones(256, device="cuda"), torch.ones(8, device="cuda")
    (q, s), (qb, sb) = tg.quantize(x), tg.quantize(x, 128)
    c, cs = tg.quantize_int8(x)
    experts = torch.arange(16, device="cuda").view(8, 2) % 3
    _, place, ends = tg.expert_plan(experts, 3)
    share, rows = torch.rand(8, 2, device="cuda"), torch.randn(16, 256, device="cuda")
    whole = torch.tensor([8], dtype=torch.int32, device="cuda")
    return {
        "quantize": lambda: tg.quantize(x), "rms_norm": lambda: tg.rms_norm(x, w, residual=x, out_dtype=FP8),
        "rms_norm_backward": lambda: tg.rms_norm_backward(x, x, w), "block_gemm": lambda: tg.block_gemm(q, qb, s, sb),
        "grouped_gemm": lambda: tg.grouped_gemm(x, x[None], whole), "grouped_wgrad": lambda: tg.grouped_wgrad(x, x, whole),
        "layer_norm": lambda: tg.layer_norm(x, w, w, residual=x, out_dtype=I8),
        "layer_norm_backward": lambda: tg.layer_norm_backward(x, x, w), "quantize_int8": lambda: tg.quantize_int8(x),
        "int8_gemm": lambda: tg.int8_gemm(c, c, cs, cs), "expert_plan": lambda: tg.expert_plan(experts, 3),
        "dispatch": lambda: tg.dispatch(x, place, ends, scales=one), "combine": lambda: tg.combine(rows, place, share, x),
        "combine_backward": lambda: tg.combine_backward(x, rows, place, share, ends),
    }


NAMES = ["quantize", "rms_norm", "rms_norm_backward", "block_gemm", "grouped_gemm", "grouped_wgrad", "layer_norm",
         "layer_norm_backward", "quantize_int8", "int8_gemm", "expert_plan", "dispatch", "combine", "combine_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_a_dispatch_mode_sees_what_is_allocated(gpu_available, name):
    say(f"[allocations] {name}")
    call = cases()[name]
    want = call()
    with Seen() as seen:
        got = call()
    for p, q in zip(*(t if isinstance(t, tuple) else (t,) for t in (want, got))):
        assert q.data_ptr() in seen.made
        assert torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))
    assert torch.equal(call()[0].float(), want[0].float())                    # and without it again


@pytest.mark.parametrize("name", NAMES)
def test_results_of_inference_mode_are_inference_tensors(gpu_available, name):
    say(f"[allocations] inference {name}")
    call = cases()[name]
    with torch.inference_mode():
        got = call()
    for t in got if isinstance(got, tuple) else (got,):
        assert t.is_inference()
    got = call()
    for t in got if isinstance(got, tuple) else (got,):
        assert not t.is_inference()


@pytest.mark.parametrize("dtype", [torch.float32, BF16, I8])
def test_deterministic_mode_fills_uninitialised_memory(gpu_available, dtype):
    """Rows that no place names are left as they were: as torch leaves new memory."""
    x = torch.ones(8, 256, device="cuda").to(dtype)
    place = torch.full((8, 2), -1, dtype=torch.int32, device="cuda")
    ends, one = torch.tensor([16], dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda")
    say(f"[allocations] deterministic {dtype}")
    for _ in range(3):              # memory that these results may get again
        kept = [torch.zeros(16, 256, device="cuda").to(dtype), torch.zeros(16, device="cuda")]
        del kept
        was = torch.are_deterministic_algorithms_enabled()
        torch.use_deterministic_algorithms(True)
        try:
            rows, scales = tg.dispatch(x, place, ends, scales=one)
        finally:
            torch.use_deterministic_algorithms(was)
        assert (rows == 127).all() if dtype is I8 else rows.isnan().all()
        assert scales.isnan().all()
        del rows, scales


@pytest.mark.parametrize("name", ["rms_norm", "expert_plan"])
def test_the_profiler_sees_what_is_allocated(gpu_available, name):
    say(f"[allocations] profiler {name}")
    call = cases()[name]
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU], acc_events=True) as seen:
        got = call()
    made = sum(e.count for e in seen.key_averages() if e.key == "aten::empty_strided")
    assert made >= len(got)
