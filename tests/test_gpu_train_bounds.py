"""The layer's training step at the edges of its contract: alignment, what is not read, workspaces and outputs of exactly
their size."""
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from test_gpu_dense import BF, F32
from test_gpu_train import I8, NAMES, Experts

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


@pytest.mark.parametrize("dense", [False, True])
def test_backward_without_x(dense):
    """Frozen gate and up weights: the other gradients without x, with either kind of saved g and u."""
    c = Experts([71] if dense else [30, 0, 41], 264, 136)
    for dtype in (F32, I8):
        if dense:
            _, gu = moe.ffn(c.x, c.bank, want_gu=True, gu_dtype=dtype)
            back = lambda x, need: moe.ffn_backward(c.dy, x, c.bank, gu, need=need)
        else:
            _, gu = moe.experts_ffn(c.x, c.offsets, c.bank, want_gu=True, gu_dtype=dtype)
            back = lambda x, need: moe.experts_ffn_backward(c.dy, x, c.offsets, c.bank, gu, need=need)
        for need in (("dx",), ("dw_down",), ("dx", "dw_down")):
            got = back(None, need)
            assert [t is not None for t in got] == [name in need for name in NAMES]
            c.check_backward(got, gu if dtype is I8 else None)
            assert all(torch.equal(a, b) for a, b in zip(got, back(c.x, need)) if a is not None)
        with pytest.raises(moe.MoeError):
            back(None, ("dw_up",))
    with pytest.raises(moe.MoeError):
        moe.ffn_backward(c.dy, None, c.bank) if dense else moe.experts_ffn_backward(c.dy, None, c.offsets, c.bank)


def test_checkpoint_of_more_lanes_than_a_grid_holds():
    """2^30 rows of 24 columns are 2^32 lanes, which go out in two launches: the rows around the seam, the first and the
    last (the others hold whatever the memory held)."""
    rows, cols, n = 1 << 30, 24, 50
    seam = (2 ** 32 - 256) // 4
    assert seam + n <= rows                                              # (the second launch has the last 64 rows)
    x = torch.empty((rows, cols), dtype=BF, device="cuda")
    q, e = torch.empty((rows, cols), dtype=I8, device="cuda"), torch.empty((rows, 2), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(1)
    some = {}
    for a in (0, seam - n, seam, rows - n):
        some[a] = torch.randn((n, cols), generator=g).to("cuda", BF)
        if a == rows - n:                                                # overlaps the rows behind the seam
            some[seam] = some[seam][:a - seam]
        x[a:a + n] = some[a]
    moe.quant_i8x16(x, out=(q, e))
    for a, v in some.items():
        rq, re = moe.quant_i8x16(v)
        assert torch.equal(q[a:a + len(v)], rq) and torch.equal(e[a:a + len(v)], re)
        x[a:a + len(v)] = 0
    moe.dequant_i8x16(q, e, out=x)
    for a, v in some.items():
        assert torch.equal(x[a:a + len(v)], moe.dequant_i8x16(*moe.quant_i8x16(v)))
    del x, q, e
    torch.cuda.empty_cache()
