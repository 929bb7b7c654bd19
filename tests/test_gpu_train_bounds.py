"""The layer's training step at the edges of its contract: alignment, what is not read, workspaces and outputs of exactly
their size."""
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from test_gpu_train import I8, Experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dense", [False, True])
def test_rows_of_a_checkpoint_on_8_bytes(dense):
    """Rows sliced from a checkpoint 264 wide, so that their codes begin on 8 bytes, are as good as a copy on 16."""
    c = Experts([71] if dense else [30, 0, 41], 264, 136)
    q, e = moe.quant_i8x16(torch.cat([c.x[:1], c.x]))
    kept = q[1:], e[1:]
    copy = tuple(t.clone() for t in kept)
    assert kept[0].data_ptr() % 16 == 8 and copy[0].data_ptr() % 16 == 0

    def back(x, gu):
        return moe.ffn_backward(c.dy, x, c.bank, gu) if dense else moe.experts_ffn_backward(c.dy, x, c.offsets, c.bank, gu)

    _, gu = moe.experts_ffn(c.x, c.offsets, c.bank, want_gu=True, gu_dtype=I8)
    for saved in (gu, None):
        for a, b in zip(back(kept, saved), back(copy, saved)):
            assert torch.equal(a, b)
    assert torch.equal(moe.dequant_i8x16(*kept), moe.dequant_i8x16(*copy))
    dest = torch.arange(c.R, dtype=torch.int32, device="cuda").flip(0)
    assert torch.equal(moe.dispatch(kept, dest, 1), moe.dispatch(copy, dest, 1))
