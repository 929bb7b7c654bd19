"""The layer's training step: arguments that the boundary refuses, and calls with
nothing to do, checked without a GPU."""
import ctypes

import pytest

import routed_expert_ffn_04_amd as moe

P, Q = 0x1000, 0x1004   # non-null dummies, 16-byte aligned and not; validation fails before any use
BIG = 1 << 40
MOST = (1 << 31) - 1
OK, INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_OK, moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def _bank(n=3, H=64, I=32, dt=moe.BF16, w=P):
    return moe.ExpertsT(n, H, I, dt, w, w, w, None, None, None)


def test_i8x16_refusals():
    def quant(x=P, dt=moe.BF16, rows=4, cols=24, q=P, e=P):
        return moe.lib().moe_quant_i8x16(x, dt, rows, cols, q, e, None)

    def dequant(q=P, e=P, rows=4, cols=24, out=P, dt=moe.F32):
        return moe.lib().moe_dequant_i8x16(q, e, rows, cols, out, dt, None)
    for call in (quant, dequant):
        assert call(rows=-1) == INVALID
        assert call(cols=0) == INVALID
        assert call(cols=20) == UNSUPPORTED
        assert call(dt=moe.I8) == UNSUPPORTED
        assert call(q=None) == INVALID
        assert call(e=None) == INVALID
        assert call(q=Q) == INVALID
        assert call(rows=MOST) == UNSUPPORTED
        assert call(rows=1 << 30, cols=1 << 20) == UNSUPPORTED      # more lanes than a grid holds
        assert call(rows=0, q=None, e=None) == OK
    assert quant(x=None) == INVALID
    assert quant(x=P + 8) == INVALID
    assert dequant(out=None) == INVALID
    assert dequant(out=P + 8) == INVALID


def test_dispatch_refusals():
    def call(x=P, dt=moe.BF16, e=None, T=4, H=64, dest=P, k=2, R=8, xs=P):
        return moe.lib().moe_dispatch(x, dt, e, T, H, dest, k, R, xs, None)
    assert call(T=-1) == INVALID
    assert call(k=0) == INVALID
    assert call(H=0) == INVALID
    assert call(R=-1) == INVALID
    assert call(H=60) == UNSUPPORTED
    assert call(dt=moe.E4M3) == UNSUPPORTED
    assert call(dt=moe.I8) == INVALID                               # no exponents
    assert call(x=None) == INVALID
    assert call(dest=None) == INVALID
    assert call(xs=None) == INVALID
    assert call(x=Q) == INVALID
    assert call(xs=P + 8) == INVALID
    assert call(dt=moe.I8, e=P, x=Q) == INVALID
    assert call(dest=P + 2) == INVALID
    assert call(T=MOST) == UNSUPPORTED
    assert call(T=1 << 29, k=4) == UNSUPPORTED
    assert call(R=MOST) == UNSUPPORTED
    assert call(T=1 << 28, H=1 << 20) == UNSUPPORTED                # more workgroups than a grid holds
    assert call(T=0, x=None, dest=None, xs=None) == OK
    assert call(R=0, x=None, dest=None, xs=None) == OK


def test_dispatch_backward_refusals():
    def call(dxs=P, dt=moe.BF16, R=8, dest=P, T=4, k=2, H=64, add=None, add_dt=0, dx=P, dx_dt=moe.BF16):
        return moe.lib().moe_dispatch_backward(dxs, dt, R, dest, T, k, H, add, add_dt, dx, dx_dt, None)
    assert call(T=-1) == INVALID
    assert call(k=-2) == INVALID
    assert call(H=12) == UNSUPPORTED
    assert call(dt=moe.I8) == UNSUPPORTED
    assert call(dx_dt=moe.E4M3) == UNSUPPORTED
    assert call(add=P + 64, add_dt=moe.I8) == UNSUPPORTED
    assert call(add=P, add_dt=moe.F32) == INVALID                   # dx is add in another dtype
    assert call(dxs=None) == INVALID
    assert call(dx=None) == INVALID
    assert call(dest=None) == INVALID
    assert call(dxs=Q) == INVALID
    assert call(add=Q, add_dt=moe.BF16) == INVALID
    assert call(dx=P + 8) == INVALID
    assert call(T=MOST) == UNSUPPORTED
    assert call(T=0, dxs=None, dest=None, dx=None) == OK


def test_combine_backward_refusals():
    def call(dout=P, d_dt=moe.BF16, y=P, y_dt=moe.BF16, ys=None, R=8, dest=P, w=P, T=4, k=2, H=128, dy=P, dy_dt=moe.BF16, dw=P):
        return moe.lib().moe_combine_backward(dout, d_dt, y, y_dt, ys, R, dest, w, T, k, H, dy, dy_dt, dw, None)
    assert call(T=-1) == INVALID
    assert call(H=36) == UNSUPPORTED
    assert call(d_dt=moe.E4M3) == UNSUPPORTED
    assert call(dy_dt=moe.I8) == UNSUPPORTED
    assert call(y_dt=moe.MXFP4) == UNSUPPORTED
    assert call(y_dt=moe.E4M3) == INVALID                           # no scales
    assert call(y_dt=moe.E4M3, ys=P, H=136) == UNSUPPORTED
    assert call(dout=None) == INVALID
    assert call(dest=None) == INVALID
    assert call(w=None) == INVALID
    assert call(y=None) == INVALID
    assert call(y=Q) == INVALID
    assert call(dy=P + 8) == INVALID
    assert call(dw=P + 2) == INVALID
    assert call(T=MOST) == UNSUPPORTED
    assert call(dy=None, dw=None) == OK
    assert call(T=0, dout=None, y=None, dest=None, w=None) == OK


def _experts(bank=None, R=5, x=P, dt=moe.BF16, off=P, y=P, y_dt=moe.BF16, gu=None, g_dt=moe.F32, ge=None, ws=P, nbytes=BIG):
    bank = _bank() if bank is None else bank
    return moe.lib().moe_experts_ffn(x, dt, off, R, ctypes.byref(bank), y, y_dt, gu, g_dt, ge, ws, nbytes, None)


def _experts_back(bank=None, R=5, dy=P, x=P, x_dt=moe.BF16, xe=None, off=P, gu=P, g_dt=moe.F32, ge=None, out=P, ws=P, nbytes=BIG):
    bank = _bank() if bank is None else bank
    return moe.lib().moe_experts_ffn_backward(dy, x, x_dt, xe, off, R, ctypes.byref(bank), gu, g_dt, ge, out, out, out, out, ws,
                                              nbytes, None)


@pytest.mark.parametrize("call", [_experts, _experts_back])
def test_experts_refusals(call):
    assert call(R=-1) == INVALID
    assert call(R=MOST) == UNSUPPORTED
    assert call(bank=_bank(n=0)) == INVALID
    assert call(bank=_bank(n=1025)) == UNSUPPORTED
    assert call(bank=_bank(dt=moe.F32)) == UNSUPPORTED
    assert call(bank=_bank(H=60)) == UNSUPPORTED
    assert call(bank=_bank(I=-8)) == INVALID
    assert call(bank=_bank(H=1 << 22)) == UNSUPPORTED
    assert call(bank=_bank(w=None)) == INVALID
    assert call(bank=_bank(w=Q)) == INVALID
    assert call(x=None) == INVALID
    assert call(off=None) == INVALID
    assert call(x=Q) == INVALID
    assert call(off=P + 2) == INVALID
    assert call(gu=Q) == INVALID
    assert call(gu=P, g_dt=moe.BF16) == UNSUPPORTED
    assert call(gu=P, g_dt=moe.I8) == INVALID                       # no exponents
    assert call(nbytes=16) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    assert call(ws=P + 16) == WORKSPACE
    assert moe.lib().moe_last_error().decode() != ""


def test_experts_refusals_of_each():
    L = moe.lib()
    assert _experts(dt=moe.F32) == UNSUPPORTED
    assert _experts(y_dt=moe.E4M3) == UNSUPPORTED
    assert _experts(y=Q) == INVALID
    assert _experts(R=0, x=None, off=None, y=None, ws=None, nbytes=0) == OK
    assert _experts_back(x_dt=moe.F32) == UNSUPPORTED
    assert _experts_back(x_dt=moe.I8) == INVALID                    # no exponents
    assert _experts_back(dy=None) == INVALID
    assert _experts_back(out=Q) == INVALID
    assert _experts_back(out=None) == OK                            # nothing wanted
    assert L.moe_experts_ffn(P, moe.BF16, P, 5, None, P, moe.BF16, None, 0, None, P, BIG, None) == INVALID
    need = L.moe_experts_ffn_backward_workspace_size
    assert need(5, 3, 64, 32, 0, moe.BF16) > need(5, 3, 64, 32, 1, moe.BF16) > 0
    assert need(5, 3, 64, 32, 1, moe.I8) > need(5, 3, 64, 32, 1, moe.BF16)
    assert _experts_back(gu=None, nbytes=need(5, 3, 64, 32, 1, moe.BF16)) == WORKSPACE    # without gu the workspace holds it
    assert _experts_back(x_dt=moe.I8, xe=P, nbytes=need(5, 3, 64, 32, 1, moe.BF16)) == WORKSPACE
    assert need(0, 3, 64, 32, 1, moe.BF16) == 0 and need(5, 0, 64, 32, 1, moe.BF16) == 0 and need(5, 3, 60, 32, 1, moe.BF16) == 0
    assert L.moe_experts_ffn_workspace_size(5, 3, 64, 32) > 0
    assert L.moe_experts_ffn_workspace_size(5, 1025, 64, 32) == 0


def test_ffn_ckpt_refusals():
    L = moe.lib()

    def ahead(T=4, n=1, x=P, gu=P, ge=P, dt=moe.BF16, nbytes=BIG):
        bank = _bank(n=n)
        return L.moe_ffn_ckpt(x, dt, T, ctypes.byref(bank), P, moe.BF16, gu, ge, P, nbytes, None)

    def back(T=4, n=1, x=P, x_dt=moe.I8, xe=P, gu=P, g_dt=moe.I8, ge=P, nbytes=BIG, out=P):
        bank = _bank(n=n)
        return L.moe_ffn_ckpt_backward(P, x, x_dt, xe, T, ctypes.byref(bank), gu, g_dt, ge, out, out, out, out, P, nbytes, None)
    for call in (ahead, back):
        assert call(T=-1) == INVALID
        assert call(T=MOST) == UNSUPPORTED
        assert call(n=2) == INVALID
        assert call(x=None) == INVALID
        assert call(x=Q) == INVALID
        assert call(gu=Q) == INVALID
        assert call(ge=None) == INVALID
        assert call(nbytes=16) == WORKSPACE
    assert ahead(gu=None) == INVALID
    assert ahead(dt=moe.I8) == UNSUPPORTED
    assert ahead(T=0, x=None, gu=None, ge=None) == OK
    assert back(xe=None) == INVALID
    assert back(x_dt=moe.F32) == UNSUPPORTED
    assert back(g_dt=moe.E4M3) == UNSUPPORTED
    assert back(out=None) == OK
    need = L.moe_ffn_ckpt_backward_workspace_size
    assert need(4, 64, 32, 1, moe.I8) > need(4, 64, 32, 1, moe.BF16) > 0
    assert back(nbytes=need(4, 64, 32, 1, moe.BF16)) == WORKSPACE
    assert L.moe_ffn_ckpt_workspace_size(4, 64, 32) > 0 and L.moe_ffn_ckpt_workspace_size(4, 64, 36) == 0


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    d = torch.zeros(2, dtype=torch.int32)
    off = torch.zeros(2, dtype=torch.int32)
    bank = moe.Experts(x.view(1, 2, 16), x.view(1, 2, 16), x.view(1, 16, 2))
    for call in (lambda: moe.quant_i8x16(x), lambda: moe.dequant_i8x16(x.to(torch.int8), x[:, :1].to(torch.uint8)),
                 lambda: moe.dispatch(x, d, 1), lambda: moe.dispatch_backward(x, d, 1),
                 lambda: moe.combine_backward(x, x, d, torch.ones(2, 1)), lambda: moe.experts_ffn(x, off, bank),
                 lambda: moe.experts_ffn_backward(x, x, off, bank)):
        with pytest.raises(ValueError):
            call()
