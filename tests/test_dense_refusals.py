"""Operators around the MoE layer: arguments that the boundary refuses, and
calls with nothing to do, checked without a GPU."""
import ctypes

import pytest

import routed_expert_ffn_04_amd as moe

P, Q = 0x1000, 0x1004   # non-null dummies, 16-byte aligned and not; validation fails before any use
BIG = 1 << 40


def _bank(n=1, H=64, I=32, dt=moe.BF16, w=P):
    return moe.ExpertsT(n, H, I, dt, w, w, w, None, None, None)


def _ffn(T=4, bank=None, x=P, y=P, x_dt=moe.BF16, y_dt=moe.BF16, gu=None, ws=P, nbytes=BIG):
    bank = _bank() if bank is None else bank
    return moe.lib().moe_ffn(x, x_dt, T, ctypes.byref(bank), y, y_dt, gu, ws, nbytes, None)


def test_ffn_refusals():
    assert _ffn(T=-1) == moe.MOE_ERR_INVALID
    assert moe.lib().moe_ffn(P, moe.BF16, 4, None, P, moe.BF16, None, P, BIG, None) == moe.MOE_ERR_INVALID
    assert _ffn(bank=_bank(n=2)) == moe.MOE_ERR_INVALID
    assert _ffn(bank=_bank(dt=moe.F32)) == moe.MOE_ERR_UNSUPPORTED
    assert _ffn(bank=_bank(dt=moe.E4M3)) == moe.MOE_ERR_UNSUPPORTED
    assert _ffn(bank=_bank(H=60)) == moe.MOE_ERR_UNSUPPORTED
    assert _ffn(bank=_bank(I=36)) == moe.MOE_ERR_UNSUPPORTED
    assert _ffn(bank=_bank(H=0)) == moe.MOE_ERR_INVALID
    assert _ffn(bank=_bank(w=None)) == moe.MOE_ERR_INVALID
    assert _ffn(bank=_bank(w=Q)) == moe.MOE_ERR_INVALID
    assert _ffn(x_dt=moe.F32) == moe.MOE_ERR_UNSUPPORTED
    assert _ffn(y_dt=moe.E4M3) == moe.MOE_ERR_UNSUPPORTED
    assert _ffn(x=None) == moe.MOE_ERR_INVALID
    assert _ffn(y=Q) == moe.MOE_ERR_INVALID
    assert _ffn(gu=Q) == moe.MOE_ERR_INVALID
    assert _ffn(nbytes=16) == moe.MOE_ERR_WORKSPACE
    assert _ffn(ws=None) == moe.MOE_ERR_WORKSPACE
    assert _ffn(ws=P + 16) == moe.MOE_ERR_WORKSPACE
    assert moe.lib().moe_last_error().decode() != ""


def test_ffn_backward_refusals():
    def call(T=4, bank=None, dy=P, x=P, dt=moe.BF16, gu=P, out=P, ws=P, nbytes=BIG):
        bank = _bank() if bank is None else bank
        return moe.lib().moe_ffn_backward(dy, x, dt, T, ctypes.byref(bank), gu, out, out, out, out, ws, nbytes, None)
    assert call(T=-1) == moe.MOE_ERR_INVALID
    assert call(bank=_bank(n=3)) == moe.MOE_ERR_INVALID
    assert call(bank=_bank(dt=moe.MXFP4)) == moe.MOE_ERR_UNSUPPORTED
    assert call(dt=moe.F32) == moe.MOE_ERR_UNSUPPORTED
    assert call(dy=None) == moe.MOE_ERR_INVALID
    assert call(x=Q) == moe.MOE_ERR_INVALID
    assert call(out=Q) == moe.MOE_ERR_INVALID
    assert call(nbytes=16) == moe.MOE_ERR_WORKSPACE
    need = moe.lib().moe_ffn_backward_workspace_size
    assert need(4, 64, 32, 0) > need(4, 64, 32, 1) > 0
    assert call(gu=None, nbytes=need(4, 64, 32, 1)) == moe.MOE_ERR_WORKSPACE   # without gu the workspace holds it
    assert call(out=None) == moe.MOE_OK                                        # nothing wanted


def _norm(T=4, H=64, y=P, res=P, y_dt=0, r_dt=0, w_dt=0, gate=None, gate_div=1, scale=1.0, eps=1e-6, r=P, x=P, x_dt=0,
          xs=None, pre=P):
    return moe.lib().moe_norm(y, y_dt, res, r_dt, T, H, None, gate, gate_div, pre, w_dt, scale, eps, r, x, x_dt, xs, None)


def test_norm_refusals():
    assert _norm(T=-1) == moe.MOE_ERR_INVALID
    assert _norm(H=0) == moe.MOE_ERR_INVALID
    assert _norm(H=16385) == moe.MOE_ERR_UNSUPPORTED
    assert _norm(y_dt=moe.E4M3) == moe.MOE_ERR_UNSUPPORTED
    assert _norm(r_dt=moe.I8) == moe.MOE_ERR_UNSUPPORTED
    assert _norm(w_dt=moe.MXFP8) == moe.MOE_ERR_UNSUPPORTED
    assert _norm(x_dt=moe.E4M3) == moe.MOE_ERR_UNSUPPORTED
    assert _norm(gate=P, gate_div=0) == moe.MOE_ERR_INVALID
    assert _norm(scale=float("nan")) == moe.MOE_ERR_INVALID
    assert _norm(eps=-1.0) == moe.MOE_ERR_INVALID
    assert _norm(y=None) == moe.MOE_ERR_INVALID
    assert _norm(r=None, x=None) == moe.MOE_ERR_INVALID
    assert _norm(x_dt=moe.I8) == moe.MOE_ERR_INVALID           # no scales
    assert _norm(y=P + 2) == moe.MOE_ERR_INVALID               # not aligned to its elements
    assert _norm(T=0, y=None, res=None, r=None, x=None) == moe.MOE_OK


def test_norm_backward_refusals():
    def call(T=4, H=64, dx=P, dr=P, y=P, r=P, post=P, gate=P, gate_div=2, pre=P, dpost=P, dgate=P, dpre=P, nbytes=BIG, x_dt=0):
        return moe.lib().moe_norm_backward(dx, x_dt, dr, y, 0, r, 0, T, H, post, gate, gate_div, pre, 0, 1.0, 1e-6,
                                           P, P, dpost, dgate, dpre, P, nbytes, None)
    assert call(T=-1) == moe.MOE_ERR_INVALID
    assert call(H=20000) == moe.MOE_ERR_UNSUPPORTED
    assert call(x_dt=moe.I8) == moe.MOE_ERR_UNSUPPORTED
    assert call(dx=None, dr=None) == moe.MOE_ERR_INVALID
    assert call(r=None) == moe.MOE_ERR_INVALID
    assert call(dx=None) == moe.MOE_ERR_INVALID                # dpre_w without dx
    assert call(y=None) == moe.MOE_ERR_INVALID
    assert call(post=None) == moe.MOE_ERR_INVALID              # dpost_w without post_w
    assert call(gate=None) == moe.MOE_ERR_INVALID
    assert call(gate_div=0) == moe.MOE_ERR_INVALID
    assert call(nbytes=16) == moe.MOE_ERR_WORKSPACE


def test_i8_refusals():
    L = moe.lib()
    assert L.moe_quant_i8(P, 0, 4, 40, P, P, None) == moe.MOE_ERR_UNSUPPORTED      # cols % 16
    assert L.moe_quant_i8(P, 2, 4, 64, P, P, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_quant_i8(P, 0, 4, 64, None, P, None) == moe.MOE_ERR_INVALID
    assert L.moe_quant_i8(Q, 0, 4, 64, P, P, None) == moe.MOE_ERR_INVALID
    assert L.moe_quant_i8(None, 0, 0, 64, None, None, None) == moe.MOE_OK

    def call(T=4, K=64, N=5, q=P, xs=P, w=P, wsc=P, out=P, out_dt=0, ws=P, nbytes=BIG):
        return L.moe_linear_i8(q, xs, T, K, w, wsc, None, N, out, out_dt, ws, nbytes, None)
    assert call(T=-1) == moe.MOE_ERR_INVALID
    assert call(N=0) == moe.MOE_ERR_INVALID
    assert call(K=72) == moe.MOE_ERR_UNSUPPORTED
    assert call(K=131072) == moe.MOE_ERR_UNSUPPORTED           # an int32 sum could overflow
    assert call(out_dt=moe.I8) == moe.MOE_ERR_UNSUPPORTED
    assert call(w=None) == moe.MOE_ERR_INVALID
    assert call(q=P + 8) == moe.MOE_ERR_INVALID
    assert call(T=0, q=None, out=None) == moe.MOE_OK
    assert L.moe_linear_i8_workspace_size(4, 72, 8) == 0
    need = L.moe_linear_i8_workspace_size(1, 7168, 4096)
    if need:
        assert call(T=1, K=7168, N=4096, nbytes=need - 1) == moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (128, 7168, 2048), (16384, 7168, 2048), (1000, 2056, 1336)])
def test_workspace_sizes_grow_with_the_call(T, H, I):
    L = moe.lib()
    assert L.moe_ffn_workspace_size(T, H, I) >= T * I * 2
    assert L.moe_ffn_backward_workspace_size(T, H, I, 1) >= T * I * 6
    assert L.moe_norm_backward_workspace_size(T, H, 0) > 0
    assert L.moe_ffn_workspace_size(0, H, I) == 0
    assert L.moe_ffn_workspace_size(T, H + 1, I) == 0


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 16)
    for call in (lambda: moe.quant_i8(x), lambda: moe.norm(x), lambda: moe.norm_backward(x, None, x, x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("size", [dict(H=1 << 22), dict(I=1 << 22)])
def test_ffn_refuses_rows_beyond_the_tile_offsets(size):
    assert _ffn(bank=_bank(**size)) == moe.MOE_ERR_UNSUPPORTED
    bank = _bank(**size)
    assert moe.lib().moe_ffn_backward(P, P, moe.BF16, 4, ctypes.byref(bank), P, P, P, P, P, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED


def test_row_counts_beyond_32_bit_tiles_are_refused():
    most = (1 << 31) - 1
    assert _ffn(T=most) == moe.MOE_ERR_UNSUPPORTED
    assert moe.lib().moe_ffn_workspace_size(most, 64, 32) == 0
    bank = _bank()
    assert moe.lib().moe_ffn_backward(P, P, moe.BF16, most, ctypes.byref(bank), P, P, P, P, P, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
    for T, N in ((most, 8), (4, most)):
        assert moe.lib().moe_linear_i8(P, P, T, 64, P, P, None, N, P, moe.F32, P, BIG, None) == moe.MOE_ERR_UNSUPPORTED
        assert moe.lib().moe_linear_i8_workspace_size(T, 64, N) == 0
