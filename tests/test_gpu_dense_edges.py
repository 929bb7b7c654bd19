"""The operators around the MoE layer at the edges of what their boundary
allows, against their formulas in 64 bits; inputs, formulas and bounds are those
of test_gpu_dense.py."""
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from test_gpu_dense import BF, F32, HALF, norm_case, norm_grad_ref, norm_ref, within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm

# T that leaves the last run of rows short where a row takes 64 (4097, 1500 rows), 128, 256, 512 and 1024
# threads, and some that do not
EPS_SHAPES = [(4097, 64), (1500, 264), (777, 1001), (520, 1032), (1100, 2003), (600, 4104), (517, 8200), (1024, 512),
              (521, 1032), (601, 4104)]


@pytest.mark.parametrize("eps", [0.0, 1e-2])
@pytest.mark.parametrize("T,H", EPS_SHAPES)
def test_norm_with_another_eps(T, H, eps):
    """eps = 0 is allowed for rows that are not all zero: whatever the number of rows, every
    gradient is finite and right."""
    for gate_div in (None, 37):
        c = norm_case(T, H, 21, gate_div=gate_div)
        kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=c["gate_div"], res_scale=0.75, pre_w=c["pre_w"], eps=eps)
        r, x = moe.norm(c["y"], c["res"], x_dtype=F32, **kw)
        rr, xx, er, ex = norm_ref(c, eps=eps)
        within(r, rr, er + HALF[BF] * (rr.abs() + er), "r")
        within(x, xx, ex + HALF[F32] * (xx.abs() + ex), "x")
        got = moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], **kw)
        ref = norm_grad_ref(c, 0.75, eps)
        assert {k for k, v in got.items() if v is not None} == set(ref)
        for k, (v, e) in ref.items():
            within(got[k], v, e + HALF[got[k].dtype] * (v.abs() + e), f"{k} gate_div={gate_div}")
