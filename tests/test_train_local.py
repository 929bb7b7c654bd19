"""Combine where only some rows are here: arguments that the boundary refuses, checked without a GPU."""
import routed_expert_ffn_04_amd as moe

P = 0x1000
INVALID, UNSUPPORTED, OK = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


def test_combine_rows_refusals():
    def call(y=P, dt=moe.BF16, ys=None, R=5, sh=None, sh_dt=0, dest=P, w=P, T=4, k=2, H=128, out=P, out_dt=moe.F32):
        return moe.lib().moe_combine_rows(y, dt, ys, R, sh, sh_dt, dest, w, T, k, H, out, out_dt, None)
    assert call(R=-1) == INVALID
    assert call(T=-1) == INVALID
    assert call(k=0) == INVALID
    assert call(H=136) == UNSUPPORTED
    assert call(dt=moe.MXFP4) == UNSUPPORTED
    assert call(sh=P, sh_dt=moe.E4M3) == UNSUPPORTED
    assert call(out_dt=moe.E4M3) == UNSUPPORTED
    assert call(y=None) == INVALID
    assert call(y=P + 8) == INVALID
    assert call(dt=moe.E4M3) == INVALID                             # no scales
    assert call(dest=None) == INVALID
    assert call(w=None) == INVALID
    assert call(out=None) == INVALID
    assert call(R=0, y=None, dest=None) == INVALID
    assert call(T=0, y=None, dest=None, w=None, out=None) == OK
    assert "combine_rows" in _error(call)


def _error(call):
    call(R=-7)
    return moe.lib().moe_last_error().decode()
