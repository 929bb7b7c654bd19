"""The experts' products: which workgroup takes which rows, from the library's own header, without a GPU."""
import ctypes
import os
import random
import subprocess

import pytest

import routed_expert_ffn_04_amd as moe
from experts_cut_cases import CUTS
from experts_plan_cases import spread

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("cuts")
    (d / "cuts.cpp").write_text('''#include <vector>
#include "experts_plan.h"
using namespace moe::gemm;
extern "C" int edge(int R, int n, long cols, int K) { return rows_edge(R, n, cols, K, 64); }
// Every workgroup of a product of 256-row tiles over these rows.  count: whole tiles, upper and lower halves with rows, and
// halves that follow a full round.  Returns how many blocks of 128 rows and 256 columns are not taken exactly once.
extern "C" int tiles(const int* rows, int n, int nt, int cus, int* count) {
    int R = 0, total = 0;
    for (int e = 0; e < n; ++e) R += rows[e], total += (rows[e] + 255) / 256 * nt;
    std::vector<int> taken(2 * total);
    const long grid = R ? rows_grid(R, n, 256, nt) : 0;
    for (long b = 0; b < grid; ++b) {
        const Cut c = cut_of((int)b, total, cus);
        int t = in_die_order(c.block, total), first = 0, e = 0, tm, tn;
        if (t < 0) continue;
        for (int own; t >= (own = (rows[e] + 255) / 256 * nt); ++e) t -= own, first += own;
        band_of(t, (rows[e] + 255) / 256, nt, tm, tn);
        const int m = rows[e] - tm * 256;
        if (c.half == 2 && m <= 128) continue;   // a workgroup without rows
        int* at = &taken[2 * (first + tm * nt + tn)];
        if (c.half != 2) ++at[0];
        if (c.half != 1 || m <= 128) ++at[1];
        ++count[c.half];
        count[3] += c.half && b / kDies >= cus;
    }
    int wrong = 0;
    for (int v : taken) wrong += v != 1;
    return wrong;
}
''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "cuts.cpp"), "-o", str(d / "cuts.so")],
                   check=True)
    L = ctypes.CDLL(str(d / "cuts.so"))
    L.edge.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_long, ctypes.c_int]

    def tiles(rows, nt, cus):
        count = (ctypes.c_int * 4)()
        wrong = L.tiles((ctypes.c_int * len(rows))(*rows), len(rows), nt, cus, count)
        return wrong, list(count)
    return L.edge, tiles


@pytest.mark.parametrize("product,sizes", CUTS)
def test_both_halves_of_cut_tiles_have_rows(plan, product, sizes):
    """The sizes tested on a GPU reach what they are listed for."""
    edge, tiles = plan
    R, n, H, I = sizes
    cols, K = {"gateup": (2 * I, H), "down": (H, I), "dh": (I, H), "dx": (H, -(-I // 64) * 64 + I)}[product]
    assert edge(R, n, cols, K) == 256
    wrong, (whole, upper, lower, later) = tiles(spread(R, n), -(-cols // 256), 32)
    assert wrong == 0 and whole > 0 and upper > 0 and lower > 0 and later > 0


def test_sizes_have_odd_and_even_stages():
    for product in ("gateup", "down", "dh"):
        assert {-(-(I if product == "down" else H) // 64) % 2 for p, (_, _, H, I) in CUTS if p == product} == {0, 1}


@pytest.mark.parametrize("cus", [1, 4, 30, 32, 38])
def test_every_row_is_taken_once(plan, cus):
    _, tiles = plan
    r = random.Random(cus)
    spreads = [[1], [256], [257, 0, 255], [0, 0, 0, 129], [128] * 9, [300] * 70, [0] * 65 + [1000], [4000, 1, 0, 130]]
    spreads += [[r.choice([0, 1, r.randint(0, 700)]) for _ in range(r.randint(1, 80))] for _ in range(40)]
    halves = 0
    for rows in spreads:
        for nt in (1, 3, 16, 28):
            wrong, (whole, upper, lower, _) = tiles(rows, nt, cus)
            assert wrong == 0, (rows, nt)
            halves += lower
    assert halves > 0 or cus == 1
