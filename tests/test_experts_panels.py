"""Operands walked down k whose rows do not start on 16 bytes, past 2^31 bytes
from the first row to the last: the bound on a slab's loads (on the CPU), and
products and weight gradients against 64-bit references.

Tolerances are test_experts.py's: a sum of n fp32 terms is off by at most
(n + 6) * 2^-24 of the sum of magnitudes, an fp8 product by 2^-10 more.
"""
import os
import random
import shutil
import subprocess

import pytest
import torch

import tiled_gemm_f32_amd as tg

from gpu_helpers import say
from test_experts import BF16, F32, FP8, U32, ends_of, f64, fp8_matrix, gen, product_tol, values, within
from test_experts_large import ends_filled

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GROUPED = os.path.join(ROOT, "tiled_gemm_f32_amd", "csrc", "gemm_grouped.hpp")


def host_program(tmp_path, names, main):
    """A program of gemm_grouped.hpp's functions `names` (compiled with signed overflow trapped) and `main`."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    text = open(GROUPED).read()
    source = "#include <cstdint>\n#include <cstdio>\n"
    for name in names:
        at = text.index(name)
        at = text.rindex("\n", 0, at) + 1
        line = text[at:text.index("\n", at) + 1]
        source += line if line.endswith("}\n") else text[at:text.index("\n}\n", at) + 3]
    (tmp_path / "t.cpp").write_text(source + main)
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-o", exe, str(tmp_path / "t.cpp")], check=True)
    return exe


def answers(exe, asked):
    out = subprocess.run([exe], input="\n".join(" ".join(map(str, a)) for a in asked), capture_output=True, text=True,
                         check=True).stdout.split()
    return [int(v) for v in out]


# Rows of the panel, bytes a row, k of a slab, bytes of a tile's columns.
PANELS = [(300000, 8194, 64, 256), (262144, 8194, 64, 256), (131072, 16388, 32, 512), (16384, 256514, 64, 130),
          (49152, 65537, 128, 128), (2 ** 31 - 1, 16, 64, 16), (1200, 2 ** 23 - 257, 128, 64), (700, 4000012, 32, 512),
          (5, 16, 64, 2), (64, 18, 64, 18), (65, 18, 64, 4), (1, 100, 128, 1)]


def test_a_slabs_loads_are_bounded_within_its_panel(tmp_path):
    exe = host_program(tmp_path, ["constexpr int slab_limit"],
                       "int main(){int a,b,c,d;while(scanf(\"%d %d %d %d\",&a,&b,&c,&d)==4)"
                       "printf(\"%d\\n\",slab_limit(a,b,c,d));}\n")
    rng = random.Random(1)
    panels = list(PANELS)
    for _ in range(400):
        step = rng.choice([rng.randrange(16, 400), rng.randrange(16, 2 ** 23 - 256)])
        wide = rng.randrange(1, min(step, 1024) + 1)
        panels.append((rng.randrange(1, rng.choice([300, 2 ** 31 - 1])), step, rng.choice([32, 64, 128]), wide))
    asked = []
    for rows, step, bk, wide in panels:
        slabs = -(-rows // bk)
        for t in sorted({0, slabs // 3, slabs // 2, max(slabs - 2, 0), slabs - 1}):
            asked.append((rows - t * bk, bk, step, wide))
    for (left, bk, step, wide), limit in zip(asked, answers(exe, asked)):
        end = (left - 1) * step + wide                     # of the panel
        assert -16 < limit <= end - 16
        if left <= bk:
            assert limit == end - 16                       # the last slab's only clamped load is its last one
        else:                                              # no load of valid columns is clamped in another
            assert (bk - 1) * step + (wide - 1) // 16 * 16 <= limit


def test_slabs_of_a_depth_near_2_to_the_31(tmp_path):
    """Their number, the first row of each (and of the few that are sent for past the last), and the rows left."""
    exe = host_program(tmp_path, ["constexpr int slabs_of", "constexpr int slab_first", "constexpr int slab_left"],
                       "int main(){int t,b,l;while(scanf(\"%d %d %d\",&t,&b,&l)==3)"
                       "printf(\"%d %d %d\\n\",slabs_of(l,b),slab_first(t,b,l),slab_left(t,b,l));}\n")
    asked = []
    for bk in (32, 64, 128):
        for depth in (1, bk - 1, bk, bk + 1, 5 * bk, 10 ** 6 + 3, 2 ** 31 - 129, 2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 1):
            slabs = -(-depth // bk)
            asked += [(t, bk, depth) for t in {0, slabs // 2, slabs - 1, *range(slabs, slabs + 6)}]
    got = answers(exe, asked)
    for i, (t, bk, depth) in enumerate(asked):
        assert got[3 * i:3 * i + 3] == [-(-depth // bk), min(t * bk, depth - 1), depth - t * bk], (t, bk, depth)


def wide_rows(rows, cols, ld, dtype, seed):
    """rows x cols at odd addresses, ld elements apart, and their values on the host."""
    t = torch.randn(rows, cols, generator=gen(seed)).to(dtype)
    buf = torch.empty((rows - 1) * ld + cols + 1, dtype=dtype, device="cuda")
    view = buf.as_strided((rows, cols), (ld, 1), 1)
    view.copy_(t)
    return view, t


@pytest.fixture
def freed():
    yield
    torch.cuda.empty_cache()


LD = 1000003                                               # elements: 2 or 4 MB


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows", [(F32, 700), (BF16, 1300)])
@pytest.mark.parametrize("side", ["dy", "x"])
@pytest.mark.parametrize("sizes", [[1], [0.3, 0.0, 0.7]])
def test_weight_gradients_of_deep_panels(gpu_available, freed, dtype, rows, side, sizes):
    N, K = 70, 140
    say(f"[panels] wgrad {dtype} {side} {rows} rows in {len(sizes)} groups")
    sizes = [int(f * rows) for f in sizes]
    sizes[-1] = rows - sum(sizes[:-1])
    dy, dy0 = wide_rows(rows, N, LD if side == "dy" else N + 1, dtype, 1)
    x, x0 = wide_rows(rows, K, LD if side == "x" else K + 1, dtype, 2)
    got = tg.grouped_wgrad(dy, x, ends_of(sizes).cuda())
    at = 0
    for g, size in enumerate(sizes):
        p, q = f64(dy0[at:at + size]), f64(x0[at:at + size])
        within(got[g], p.t() @ q, (p.abs().t() @ q.abs()) * (size + 4) * U32, g)
        at += size


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,depth", [(F32, 700), (BF16, 1300)])
@pytest.mark.parametrize("M,N", [(40, 70), (3000, 300)])
def test_products_with_weights_walked_down_deep_panels(gpu_available, freed, dtype, depth, M, N):
    say(f"[panels] op N {dtype} {M}x{N}x{depth}")
    w, w0 = wide_rows(depth, N, LD, dtype, 1)
    x, x0 = wide_rows(M, depth, depth + 1, dtype, 2)
    got = tg.grouped_gemm(x, w[None], ends_of([M]).cuda(), op_b="N", out_dtype=F32)
    a, b = f64(x0), f64(w0)
    want = a @ b
    within(got, want, product_tol(a, b, want, False, F32), (M, N))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(40, 70), (1000, 300)])
def test_fp8_products_with_weights_walked_down_deep_panels(gpu_available, freed, M, N):
    depth, ld = 1300, 1900001
    say(f"[panels] fp8 op N {M}x{N}x{depth}")
    qa, sa = fp8_matrix(M, depth, 1, 1)
    qb, sb = fp8_matrix(depth, N, 2, 128)
    buf = torch.empty((depth - 1) * ld + N + 1, dtype=torch.uint8, device="cuda")
    w = buf.as_strided((depth, N), (ld, 1), 1)
    w.copy_(qb.view(torch.uint8))
    got = tg.block_gemm(qa.cuda(), w.view(FP8), sa.cuda(), sb.cuda(), op_b="N", out_dtype=F32)
    a, b = values(qa, sa, 1), values(qb, sb, 128)
    want = a @ b
    within(got, want, product_tol(a, b, want, True, F32), (M, N))


@pytest.mark.gpu
def test_weight_gradients_of_many_rows(gpu_available, freed):
    """A group of 300000 rows of 4097 bf16 values, 2.5 GB: all zeros but the first and the last 30 rows."""
    M, N, K = 300000, 4097, 40
    say(f"[panels] wgrad {M} rows of {N}")
    dy, dys = ends_filled(M, N, BF16, 1)
    x, xs = ends_filled(M, K, BF16, 3)
    x[30:-30] = 1                                          # (counts whatever is read in place of the zeros)
    got = tg.grouped_wgrad(dy, x, ends_of([M]).cuda())
    pairs = [(f64(p), f64(q)) for p, q in zip(dys, xs)]
    want = sum(p.t() @ q for p, q in pairs)
    within(got[0], want, sum(p.abs().t() @ q.abs() for p, q in pairs) * (60 + 4) * U32, "many rows")
