"""The layer's training step at the edges of its contract: alignment, what is not read, workspaces and outputs of exactly
their size."""
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from test_gpu_dense import BF, F32, outbuf, rand
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


def test_rows_of_more_workgroups_than_a_grid_holds():
    """2^24 workgroups of 256 threads are one more than a grid holds: tokens of one workgroup each, in two launches.  The
    tokens that have a row here lie around the seam and at both ends."""
    H, R, seam = 1032, 8, (2 ** 32 - 1) // 256
    T = seam + 9
    at = [0, 1, seam - 1, seam, seam + 1, T - 2, T - 1]
    dest = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    x = torch.empty((T, H), dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(2)
    for i, t in enumerate(at):
        dest[t] = i
        x[t] = torch.randn(H, generator=g).to("cuda", BF)
    xs, guard = outbuf((R, H), BF)
    moe.dispatch(x, dest, 1, out=xs)
    guard()
    assert bool((xs[len(at):] == 77).all())
    for i, t in enumerate(at):
        assert torch.equal(xs[i], x[t])
    rows = rand(g, (R, H), 1.0, BF)
    moe.dispatch_backward(rows, dest, 1, out=x)
    for i, t in enumerate(at):
        assert torch.equal(x[t], rows[i])
    for t in (2, seam - 2, seam + 2, T - 3):
        assert bool((x[t] == 0).all())
    moe.dispatch_backward(rows, dest, 1, add=x, out=x)
    for i, t in enumerate(at):
        assert torch.equal(x[t], (2 * rows[i].float()).to(BF))
    # 8-bit checkpoints of the same many tokens: codes and exponents move on together
    del x
    q, e = torch.empty((T, H), dtype=I8, device="cuda"), torch.empty((T, 65), dtype=torch.uint8, device="cuda")
    kept, exps = moe.quant_i8x16(rows)
    for i, t in enumerate(at):
        q[t], e[t] = kept[i], exps[i]
    moe.dispatch((q, e), dest, 1, out=xs)
    assert torch.equal(xs[:len(at)], moe.dequant_i8x16(kept, exps)[:len(at)])
    guard()
    del q, e
    torch.cuda.empty_cache()


def test_assignments_of_more_waves_than_a_grid_holds():
    """2^26 assignments and more, four a workgroup, in two launches."""
    H, R, k, seam = 8, 8, 2, (2 ** 32 - 1) // 256 * 4
    T = seam // k + 5
    at = [0, 1, seam - 1, seam, seam + 1, T * k - 2, T * k - 1]
    dest = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    dout = torch.ones((T, H), dtype=BF, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    for i, f in enumerate(at):
        dest[f] = i
        dout[f // k] = f % 11 + 1
    y = torch.arange(R, device="cuda", dtype=torch.float32).add(1).unsqueeze(1).expand(R, H).to(BF).contiguous()
    buf, guard = outbuf((R, H), BF)
    dy, dw = moe.combine_backward(dout, y, dest, w, dy=buf)
    guard()
    for i, f in enumerate(at):
        assert torch.equal(dy[i], 0.5 * dout[f // k]) and float(dw.view(-1)[f]) == 8 * float(dout[f // k, 0]) * (i + 1)
    assert bool((dy[len(at):] == 77).all()) and int((dw != 0).sum()) == len(at)
    del dw, dout, w, dest
    torch.cuda.empty_cache()
