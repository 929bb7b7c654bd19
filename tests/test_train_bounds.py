"""The layer's training step: what the boundary takes at the edges of its contract, checked without a GPU.
A call that passes the checks on its tensors ends at the workspace, which is too small here."""
import ctypes

import routed_expert_ffn_04_amd as moe

P = 0x1000
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
BF, I8 = moe.BF16, moe.I8


def experts_back(x=P, x_dt=BF, xe=None, gu=P, dx=P, dwg=P, dwu=P, dwd=P):
    bank = moe.ExpertsT(3, 72, 32, BF, P, P, P, None, None, None)
    return moe.lib().moe_experts_ffn_backward(P, x, x_dt, xe, P, 5, ctypes.byref(bank), gu, moe.F32, None, dx, dwg, dwu, dwd,
                                              P, 16, None)


def ffn_back(x=P, x_dt=BF, xe=None, gu=P, dx=P, dwg=P, dwu=P, dwd=P):
    bank = moe.ExpertsT(1, 72, 32, BF, P, P, P, None, None, None)
    return moe.lib().moe_ffn_ckpt_backward(P, x, x_dt, xe, 5, ctypes.byref(bank), gu, moe.F32, None, dx, dwg, dwu, dwd, P, 16, None)


def test_codes_of_x_are_aligned_like_their_pieces():
    """Rows of a checkpoint whose width is 8 mod 16 begin on 8 bytes."""
    for call in (experts_back, ffn_back):
        assert call(x=P + 8, x_dt=I8, xe=P) == WORKSPACE
        assert call(x=P + 8, x_dt=I8, xe=P + 1) == WORKSPACE
        assert call(x=P + 4, x_dt=I8, xe=P) == INVALID
        assert call(x=P + 8) == INVALID


def test_x_is_asked_for_where_it_is_read():
    """With g and u saved, x is read for the gradients of the gate and up weights alone."""
    def dense(x=None, x_dt=BF, xe=None, gu=P, dx=P, dwg=None, dwu=None, dwd=P):
        bank = moe.ExpertsT(1, 72, 32, BF, P, P, P, None, None, None)
        return moe.lib().moe_ffn_backward(P, x, x_dt, 5, ctypes.byref(bank), gu, dx, dwg, dwu, dwd, P, 16, None)
    for call in (experts_back, ffn_back, dense):
        assert call(x=None, dwg=None, dwu=None) == WORKSPACE
        assert call(x=None, dx=None, dwg=None, dwu=None) == WORKSPACE
        assert call(x=None, dwg=P, dwu=None) == INVALID
        assert call(x=None, dwg=None, dwu=P) == INVALID
        assert call(x=None, dwg=None, dwu=None, gu=None) == INVALID     # g and u are computed again
