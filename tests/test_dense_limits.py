"""Sizes at the limits of the operators around the MoE layer, checked without a GPU."""
import ctypes
import os
import subprocess

import pytest

import routed_expert_ffn_04_amd as moe
from dense_plan_cases import FFN, I8


class Shape:
    """Stands for a tensor on a GPU; only its sizes are looked at."""
    device = "cuda:0"

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 4])
def test_sizes_that_an_int32_does_not_hold_are_refused(size):
    """They would reach the library as their low 32 bits: 2^32 + 4 rows as 4."""
    t = Shape(size, 16)
    for call in (lambda: moe.quant_i8(t), lambda: moe.norm(t), lambda: moe.norm_backward(t, None, t, t),
                 lambda: moe.linear_i8(t, None, t, None), lambda: moe.ffn(t, None), lambda: moe.ffn_backward(t, t, None),
                 lambda: moe.quant_i8(Shape(4, size))):
        with pytest.raises(ValueError, match=str(2 ** 31 - 1)):
            call()
    w = Shape(1, size, 16)
    with pytest.raises(ValueError, match=str(2 ** 31 - 1)):
        moe._dense_bank(moe.Experts(w, w, w), 16, 0)


# ---------------------------------------------------------------- grids

P, BIG = 0x1000, 1 << 62   # a non-null dummy: validation ends before any use
CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")


def test_products_that_no_grid_holds_are_refused():
    """Before anything is launched, and with a workspace size of 0."""
    L, most = moe.lib(), 1 << 30
    assert L.moe_linear_i8(P, P, most, 16, P, P, None, most, P, moe.F32, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_linear_i8_workspace_size(most, 16, most) == 0
    # 2^22 x 2 tiles of 256 x 256, one more than a grid of 512 threads each holds
    assert L.moe_linear_i8(P, P, most, 131056, P, P, None, 500, P, moe.F32, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
    bank = moe.ExpertsT(1, 64, 1 << 21, moe.BF16, P, P, P, None, None, None)
    assert L.moe_ffn(P, moe.BF16, most, ctypes.byref(bank), P, moe.BF16, None, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_ffn_workspace_size(most, 64, 1 << 21) == 0
    assert L.moe_ffn_backward(P, P, moe.BF16, most, ctypes.byref(bank), None, P, P, P, P, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_ffn_backward_workspace_size(most, 64, 1 << 21, 0) == 0


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan_tiles(M, mma_cols, K, stage_elems, rows) -> dict, from the library's own header."""
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text('''#include "tile_plan.h"
extern "C" int plan_tiles(long M, long cols, int K, int stage, int rows, int* out) {
    const moe::gemm::Plan p = moe::gemm::plan_tiles(M, cols, K, stage, rows != 0);
    out[0] = p.few; out[1] = p.edge; out[2] = p.splits; out[3] = p.kspan; out[4] = p.workgroups;
    return moe::gemm::fits(p);
}
extern "C" int plan_together(const int* sizes, int n, int stage) {   // of products with operands by columns
    double apart = 0;
    moe::gemm::Size s[3];
    for (int i = 0; i < n; ++i) {
        s[i] = {sizes[3 * i], sizes[3 * i + 1], sizes[3 * i + 2]};
        apart += moe::gemm::plan_tiles(s[i].M, s[i].N, s[i].K, stage, false).us + 2;
    }
    return moe::gemm::plan_together(s, n, stage, apart);
}
''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan.so")],
                   check=True)
    L = ctypes.CDLL(str(d / "plan.so"))
    f = L.plan_tiles
    f.argtypes = [ctypes.c_long, ctypes.c_long, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    def call(M, cols, K, stage, rows):
        out = (ctypes.c_int * 5)()
        ok = f(M, cols, K, stage, rows, out)
        return dict(zip(("few", "edge", "splits", "kspan", "workgroups"), out), fits=bool(ok))
    call.together = lambda sizes: L.plan_together((ctypes.c_int * 9)(*(v for s in sizes for v in s)), len(sizes), 64)
    return call


MOST_FEW = 16 * ((2 ** 32 - 1) // 512)   # columns that the few-row kernel's grid holds


@pytest.mark.parametrize("T,K,N", [(1, 16, MOST_FEW), (1, 16, MOST_FEW + 1), (16, 64, MOST_FEW + 16), (1, 16, 1 << 30),
                                   (40, 7168, 1 << 30), (1 << 30, 16, 8), (1 << 30, 131056, 250), (1 << 20, 64, 1 << 18)])
def test_plans_take_kernels_whose_grid_holds_the_product(plan, T, K, N):
    p = plan(T, N, K, 128, 1)
    assert p["fits"] and bool(p["few"]) == (T <= 16 and N <= MOST_FEW)
    if p["few"]:
        assert (N + 15) // 16 * 512 < 2 ** 32
    else:
        tiles = -(-T // p["edge"]) * -(-N // p["edge"])
        assert p["workgroups"] == tiles * p["splits"]
        assert p["workgroups"] * (512 if p["edge"] == 256 else 256) < 2 ** 32


@pytest.mark.parametrize("product,tiling,sizes", FFN + I8)
def test_the_sizes_tested_on_a_gpu_reach_their_tilings(plan, product, tiling, sizes):
    """As launch_tiling and launch_products choose."""
    if product == "i8":
        p = plan(sizes[0], sizes[2], sizes[1], 128, 1)
    else:
        T, H, I = sizes
        K = -(-I // 64) * 64 + I                # of dx: du's half begins on a stage
        if product == "grads":
            edge = plan.together([(T, H, K), (2 * I, H, T), (H, I, T)])
            assert (f"joint{edge}" if edge else "apart") == tiling
            return
        M, cols, k, rows = {"gateup": (T, 2 * I, H, 1), "down": (T, H, I, 1), "dh": (T, I, H, 0), "dx": (T, H, K, 0),
                            "dwgu": (2 * I, H, T, 0), "dw1": (I, H, T, 0), "dwd": (H, I, T, 0)}[product]
        p = plan(M, cols, k, 64, rows)
    assert not p["few"]
    deep = p["edge"] < 256 and p["workgroups"] <= (512 if p["edge"] == 64 else 256)
    assert f"{p['edge']}r{10 if deep else 5}{'/k' if p['splits'] > 1 else ''}" == tiling
