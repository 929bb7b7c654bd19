"""The layer's routed half where only some experts are here: assignments to the others have
no row (dest outside [0, R)), from dispatch to combine and back."""
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from test_gpu_dense import BF, F32, HALF, gamma, outbuf, rand, within
from test_gpu_train import Rows, U8, check_grads, order, step_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("absent", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 128), (5, 3, 7, 256), (50, 9, 12, 384), (300, 8, 256, 2048), (70001, 2, 4, 128)])
def test_combine(T, k, E, H, absent):
    """Against the sum over the rows that are here, in 64 bits; the weights of the others, NaN here, reach nothing."""
    if absent == 1.0:
        R = 0
        dest = torch.tensor([-1, 0, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(T * k)[:T * k].cuda()
    else:
        dest, R = order(T, k, E, T + H, absent)
    g = torch.Generator().manual_seed(T + H)
    here = ((dest >= 0) & (dest < R)).view(T, k)
    w = rand(g, (T, k), 1.0, F32)
    w[~here] = float("nan")
    kinds = [(F32, None, F32), (BF, BF, BF), (BF, F32, F32), (U8, None, BF), (U8, BF, F32)]
    for y_t, sh_t, out_t in kinds:
        y_scale = None
        if y_t is U8:
            y = torch.randn((R, H), generator=g).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(U8).cuda()
            y_scale = (torch.rand((R, H // 128), generator=g) + 0.01).cuda()
            yd = y.view(torch.float8_e4m3fn).double() * y_scale.double().repeat_interleave(128, 1)
        else:
            y = rand(g, (max(R, 1), H), 1.0, y_t)[:R]
            yd = y.double()
        sh = None if sh_t is None else rand(g, (T, H), 1.0, sh_t)
        rows = torch.zeros((T, k, H), dtype=torch.float64, device="cuda")
        rows[here] = yd[dest.view(T, k)[here].long()] * w[here].double().unsqueeze(1)
        ref, mag = rows.sum(1), rows.abs().sum(1)
        if sh is not None:
            ref, mag = ref + sh.double(), mag + sh.double().abs()
        out, guard = outbuf((T, H), out_t)
        moe.combine(y, sh, dest, w, y_scale=y_scale, out=out)
        # k fused products and sums; an e4m3 value times its scale rounds once more
        e = gamma(k + 1) * mag
        within(out, ref, e + HALF[out_t] * (ref.abs() + e), "out")
        guard()


@pytest.mark.parametrize("first,count", [(0, 3), (2, 4), (5, 3), (7, 1)])
def test_training_step_of_some_experts(first, count):
    """A step with experts [first, first + count) of 8: every operator on what the one before it gave, and the
    tokens' sums over the parts of all GPUs' experts would be those of the whole layer."""
    T, H, E, k, I = 150, 256, 8, 3, 136
    x, w_router, bank, dout = step_inputs(T, H, E, I)
    ids, w = moe.route(x, w_router, None, k, "softmax")
    _, offsets, _, dest = moe.permute(ids, E)
    a, b = offsets[first].item(), offsets[first + count].item()
    R = b - a
    mine = (dest - a).to(torch.int32)                                   # rows before come out negative, those behind past R
    off = (offsets[first:first + count + 1] - a).to(torch.int32)
    part = moe.Experts(*(t[first:first + count] for t in (bank.w_gate, bank.w_up, bank.w_down)))
    here = ((mine >= 0) & (mine < R)).view(T, k)
    at = mine.view(T, k)[here].long()
    assert 0 < R < T * k
    xs = moe.dispatch(x, mine, k, R=R)
    y, gu = moe.experts_ffn(xs, off, part, want_gu=True)
    out, guard = outbuf((T, H), BF)
    moe.combine(y, None, mine, w, out=out)
    guard()
    rows = torch.zeros((T, k, H), dtype=torch.float64, device="cuda")
    rows[here] = y.double()[at] * w[here].double().unsqueeze(1)
    ref, mag = rows.sum(1), gamma(k + 1) * rows.abs().sum(1)
    within(out, ref, mag + HALF[BF] * (ref.abs() + mag), "out")
    dy, dw = moe.combine_backward(dout, y, mine, w)
    assert bool((dw[~here] == 0).all()) and dy.shape == (R, H)
    dxs, *grads = moe.experts_ffn_backward(dy, xs, off, part, gu)
    ends = off.tolist()
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        r = Rows(xs[lo:hi], dy[lo:hi], part.w_gate[e], part.w_up[e], part.w_down[e])
        within(y[lo:hi], r.y, r.ey + HALF[BF] * (r.y.abs() + r.ey), "y")
        check_grads(r, (dxs, *grads), lo, hi, e)
    dx = moe.dispatch_backward(dxs, mine, k)
    back = torch.zeros((T, k, H), dtype=torch.float64, device="cuda")
    back[here] = dxs.double()[at]
    ref, mag = back.sum(1), gamma(k) * back.abs().sum(1)
    within(dx, ref, mag + HALF[BF] * (ref.abs() + mag), "dx")


def test_combine_in_range_is_unchanged():
    """With every row here, both calls of the boundary give the same bits."""
    T, k, E, H = 333, 5, 16, 640
    dest, R = order(T, k, E, 1)
    g = torch.Generator().manual_seed(1)
    y, sh, w = rand(g, (R, H), 1.0, BF), rand(g, (T, H), 1.0, BF), rand(g, (T, k), 1.0, F32)
    one = moe.combine(y, sh, dest, w)
    two = torch.empty_like(one)
    moe._check(moe.lib().moe_combine(y.data_ptr(), moe.BF16, None, sh.data_ptr(), moe.BF16, dest.data_ptr(), w.data_ptr(),
                                     T, k, H, two.data_ptr(), moe.F32, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(one, two)
