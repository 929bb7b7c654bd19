"""The layer's training step: sizes at its limits and the tilings that sizes reach, checked without a GPU."""
import ctypes
import os
import subprocess

import pytest

import routed_expert_ffn_04_amd as moe
from experts_plan_cases import EXPERTS, spread
from test_dense_limits import Shape

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")
P, BIG = 0x1000, 1 << 62


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 4])
def test_sizes_that_an_int32_does_not_hold_are_refused(size):
    t = Shape(size, 16)
    for call in (lambda: moe.quant_i8x16(t), lambda: moe.dequant_i8x16(t, None), lambda: moe.dispatch(t, None, 1),
                 lambda: moe.dispatch_backward(t, None, 1), lambda: moe.combine_backward(t, None, None, None),
                 lambda: moe.experts_ffn(t, None, None), lambda: moe.experts_ffn_backward(t, t, None, None),
                 lambda: moe.dispatch((t, None), None, 1)):
        with pytest.raises(ValueError, match=str(2 ** 31 - 1)):
            call()
    w = Shape(3, size, 16)
    with pytest.raises(ValueError, match=str(2 ** 31 - 1)):
        moe._experts_bank(moe.Experts(w, w, w), 16, 0)


def test_products_that_no_grid_holds_are_refused():
    L, most = moe.lib(), 1 << 30
    bank = moe.ExpertsT(8, 64, 1 << 21, moe.BF16, P, P, P, None, None, None)
    b = ctypes.byref(bank)
    assert L.moe_experts_ffn(P, moe.BF16, P, most, b, P, moe.BF16, None, moe.F32, None, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_experts_ffn_workspace_size(most, 8, 64, 1 << 21) == 0
    assert L.moe_experts_ffn_backward(P, P, moe.BF16, None, P, most, b, None, moe.F32, None, P, P, P, P, P, BIG,
                                      None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_experts_ffn_backward_workspace_size(most, 8, 64, 1 << 21, 0, moe.BF16) == 0
    # 1024 experts whose gradients alone are more tiles than a grid holds
    assert L.moe_experts_ffn_backward_workspace_size(64, 1024, 1 << 21, 1 << 21, 0, moe.BF16) == 0


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """The tiling of a product, from the library's own header."""
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text('''#include "experts_plan.h"
using namespace moe::gemm;
extern "C" int rows_plan(int R, int n, long cols, int K, int* ring) {
    const int e = rows_edge(R, n, cols, K, 64);
    *ring = e ? ring_of(e, even_tiles(R, n, e) * ((cols + e - 1) / e)) : 0;
    return e;
}
extern "C" int grads_plan(int R, int n, int H, int I, int cus, int* ring) {
    const GroupSize p[3] = {{0, H, (I + 63) / 64 * 64 + I, false}, {2 * I, H, 0, true}, {H, I, 0, true}};
    if (stream_tiles(p, 3, n) >= cus) return 0;
    const int e = group_edge(p, 3, R, n, 64);
    long tiles = 0;
    for (const GroupSize& s : p) tiles += group_tiles(s, R, n, e);
    *ring = ring_of(e, tiles);
    return e;
}
extern "C" long grid(int R, int n, int edge, long nt) { return rows_grid(R, n, edge, nt); }
''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan.so")],
                   check=True)
    L = ctypes.CDLL(str(d / "plan.so"))
    L.rows_plan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_long, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.grid.argtypes, L.grid.restype = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_long], ctypes.c_long
    return L


@pytest.mark.parametrize("product,tiling,sizes", EXPERTS)
def test_the_sizes_tested_on_a_gpu_reach_their_tilings(plan, product, tiling, sizes):
    R, n, H, I = sizes
    ring = ctypes.c_int()
    if product == "grads":
        edge = plan.grads_plan(R, n, H, I, 256, ctypes.byref(ring))
    else:
        cols, K = {"gateup": (2 * I, H), "down": (H, I), "dh": (I, H), "dx": (H, -(-I // 64) * 64 + I)}[product]
        edge = plan.rows_plan(R, n, cols, K, ctypes.byref(ring))
    assert (f"{edge}r{ring.value}" if edge else "stream") == tiling


@pytest.mark.parametrize("rows", [[1], [0, 0, 7], [64, 64], [65, 1, 64], [257, 255, 0, 1], [1] * 100, [300] * 3 + [0] * 50])
def test_grids_have_room_for_every_spread_of_the_rows(plan, rows):
    for edge in (64, 128, 256):
        for nt in (1, 3, 28):
            assert plan.grid(sum(rows), len(rows), edge, nt) >= sum(-(-m // edge) for m in rows) * nt


@pytest.mark.parametrize("product,tiling,sizes", EXPERTS)
def test_spread(product, tiling, sizes):
    R, n, _, _ = sizes
    rows = spread(R, n)
    assert sum(rows) == R and len(rows) == n and (n == 1 or 0 in rows)


def test_rows_longer_than_their_columns_count_are_refused():
    """Columns are counted in 32 bits, a few thousand past the row's end."""
    L, wide = moe.lib(), (1 << 31) - 8
    assert L.moe_dispatch(P, moe.BF16, None, 1, wide, P, 1, 1, P, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_dispatch_backward(P, moe.BF16, 1, P, 1, 1, wide, None, 0, P, moe.BF16, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_combine_backward(P, moe.BF16, P, moe.BF16, None, 1, P, P, 1, 1, wide, P, moe.BF16, P,
                                  None) == moe.MOE_ERR_UNSUPPORTED
