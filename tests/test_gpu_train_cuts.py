"""The experts' products where the last round of tiles is cut into halves."""
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from experts_cut_cases import CUTS
from experts_plan_cases import spread
from test_gpu_dense import BF, F32, outbuf
from test_gpu_train import I8, U8, Experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,n,H,I", sorted({s for _, s in CUTS}))
def test_cut_tiles(R, n, H, I):
    """Both kinds of checkpoints, forward and back, against the formulas in 64 bits."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256    # what the sizes were found for
    c = Experts(spread(R, n), H, I, 4)
    y, guard = outbuf((R, H), BF)
    gu, guard_gu = outbuf((R, 2 * I), F32)
    moe.experts_ffn(c.x, c.offsets, c.bank, want_gu=True, out=y, gu=gu)
    c.check_forward(y, gu, False)
    q, guard_q = outbuf((R, 2 * I), I8)
    e, guard_e = outbuf((R, 2 * -(-I // 16)), U8)
    y8, guard_y8 = outbuf((R, H), F32)
    moe.experts_ffn(c.x, c.offsets, c.bank, out=y8, gu=(q, e))
    c.check_forward(y8, (q, e), True)
    assert torch.equal(y8.to(BF), y)
    for check in (guard, guard_gu, guard_q, guard_e, guard_y8):
        check()
    for need in (("dx",), ("dx", "dw_gate", "dw_up", "dw_down")):
        c.check_backward(moe.experts_ffn_backward(c.dy, c.x, c.offsets, c.bank, gu, need=need))
        c.check_backward(moe.experts_ffn_backward(c.dy, c.x, c.offsets, c.bank, (q, e), need=need), (q, e))
