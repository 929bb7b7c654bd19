"""The products of the training step through the C ABI, every output and a workspace of exactly the size asked for between
guard bytes: nothing around them is written, and what a workspace held before does not matter."""
import ctypes

import pytest
import torch

import routed_expert_ffn_04_amd as moe
from experts_cut_cases import CUTS
from experts_plan_cases import spread
from test_gpu_dense import BF, F32
from test_gpu_train import I8, U8, Experts

pytestmark = pytest.mark.gpu

AROUND = 1 << 18   # guard bytes on each side, a multiple of 256
FILL = 77


class Guarded:
    """Device buffers between guard bytes; the outputs hold FILL in every element, workspaces bits of NaN."""

    def __init__(self):
        self.all = []

    def raw(self, nbytes):
        whole = torch.full((nbytes + 2 * AROUND,), 0xA5, dtype=U8, device="cuda")
        self.all.append((whole, nbytes))
        assert whole.data_ptr() % 256 == 0
        return whole[AROUND:AROUND + nbytes]

    def out(self, shape, dtype):
        t = torch.full(shape, FILL, dtype=dtype, device="cuda")
        place = self.raw(t.numel() * t.element_size())
        got = place.view(dtype).view(shape)
        got.copy_(t)
        return got

    def ws(self, nbytes):
        t = self.raw(nbytes)
        t.fill_(0xFF)
        return t

    def check(self):
        for whole, nbytes in self.all:
            assert bool((whole[:AROUND] == 0xA5).all()) and bool((whole[AROUND + nbytes:] == 0xA5).all()), "written out of range"


def ptr(t):
    return None if t is None or not t.numel() else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def forward(c, bank, i8, offsets):
    """(y, gu, guards) of moe_experts_ffn, or without offsets of moe_ffn_ckpt and moe_ffn."""
    L, g, R, H, I, n = moe.lib(), Guarded(), c.R, c.H, c.I, bank.n
    y = g.out((R, H), BF)
    gu, ge = (g.out((R, 2 * I), I8), g.out((R, 2 * -(-I // 16)), U8)) if i8 else (g.out((R, 2 * I), F32), None)
    b = ctypes.byref(bank)
    if offsets is not None:
        ws = g.ws(L.moe_experts_ffn_workspace_size(R, n, H, I))
        moe._check(L.moe_experts_ffn(ptr(c.x), moe.BF16, ptr(offsets), R, b, ptr(y), moe.BF16, ptr(gu),
                                     moe.I8 if i8 else moe.F32, ptr(ge), ptr(ws), ws.numel(), stream()))
    elif i8:
        ws = g.ws(L.moe_ffn_ckpt_workspace_size(R, H, I))
        moe._check(L.moe_ffn_ckpt(ptr(c.x), moe.BF16, R, b, ptr(y), moe.BF16, ptr(gu), ptr(ge), ptr(ws), ws.numel(), stream()))
    else:
        ws = g.ws(L.moe_ffn_workspace_size(R, H, I))
        moe._check(L.moe_ffn(ptr(c.x), moe.BF16, R, b, ptr(y), moe.BF16, ptr(gu), ptr(ws), ws.numel(), stream()))
    g.check()
    return y, (gu, ge) if i8 else gu


def backward(c, bank, x, gu, offsets, need=(1, 1, 1, 1)):
    """The gradients of moe_experts_ffn_backward, or without offsets of moe_ffn_ckpt_backward."""
    L, g, R, H, I, n = moe.lib(), Guarded(), c.R, c.H, c.I, bank.n
    shapes = ((R, H), (n, I, H), (n, I, H), (n, H, I))
    o = [g.out(s, BF) if wanted else None for s, wanted in zip(shapes, need)]
    q, e = x if isinstance(x, tuple) else (x, None)
    s, se = gu if isinstance(gu, tuple) else (gu, None)
    x_dt, g_dt = moe.I8 if e is not None else moe.BF16, moe.I8 if se is not None else moe.F32
    b, has = ctypes.byref(bank), int(gu is not None)
    if offsets is not None:
        ws = g.ws(L.moe_experts_ffn_backward_workspace_size(R, n, H, I, has, x_dt))
        moe._check(L.moe_experts_ffn_backward(ptr(c.dy), ptr(q), x_dt, ptr(e), ptr(offsets), R, b, ptr(s), g_dt, ptr(se),
                                              *map(ptr, o), ptr(ws), ws.numel(), stream()))
    else:
        ws = g.ws(L.moe_ffn_ckpt_backward_workspace_size(R, H, I, has, x_dt))
        moe._check(L.moe_ffn_ckpt_backward(ptr(c.dy), ptr(q), x_dt, ptr(e), R, b, ptr(s), g_dt, ptr(se), *map(ptr, o), ptr(ws),
                                           ws.numel(), stream()))
    g.check()
    return o


# gradients in one launch with dx (64- and 128-row tiles) and streamed; ragged everywhere
CASES = [([70, 0, 9], 264, 136), ([1], 8, 8), ([129, 300, 1], 1032, 520), ([700, 20, 0, 300], 1000, 1000),
         ([(37 * e) % 101 for e in range(24)], 264, 264), ([(311 * e) % 700 for e in range(23)], 520, 264),
         ([0, 4000, 0], 520, 264)]


@pytest.mark.parametrize("around", [(0, 0), (5, 130)])
@pytest.mark.parametrize("sizes,H,I", CASES)
def test_experts(sizes, H, I, around):
    c = Experts(sizes, H, I, 6, *around)
    bank = c.bank.struct()
    a, b = around[0], c.R - around[1]

    def outside(t):
        return t is None or bool((t[:a] == FILL).all()) and bool((t[b:] == FILL).all())

    for i8 in (False, True):
        y, gu = forward(c, bank, i8, c.offsets)
        c.check_forward(y, gu, i8)
        assert outside(y) and all(outside(t) for t in (gu if i8 else (gu,)))
        xs = [c.x, moe.quant_i8x16(c.x)]
        for x in xs:
            held = x if isinstance(x, tuple) else None
            got = backward(c, bank, x, gu, c.offsets)
            assert outside(got[0])
            c.check_backward(got, gu if i8 else None, held)
        for k in range(4):
            one = backward(c, bank, c.x, gu, c.offsets, [int(i == k) for i in range(4)])
            assert outside(one[0])
            c.check_backward(one, gu if i8 else None)
    again = backward(c, bank, c.x, None, c.offsets)
    assert outside(again[0])
    c.check_backward(again)


@pytest.mark.parametrize("R,n,H,I", sorted({s for _, s in CUTS} | {(1464, 3, 2712, 200), (68, 58, 8, 296), (93, 69, 1680, 368)}))
def test_experts_in_large_tiles(R, n, H, I):
    """256-row tiles of every product, whole, half and cut, and of the gradients in one launch and streamed: the guards
    (the values are checked where these sizes come from)."""
    c = Experts(spread(R, n), H, I, 6)
    bank = c.bank.struct()
    for i8 in (False, True):
        _, gu = forward(c, bank, i8, c.offsets)
        for need in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 1)):
            backward(c, bank, moe.quant_i8x16(c.x) if i8 else c.x, gu, c.offsets, need)
    backward(c, bank, c.x, None, c.offsets)


@pytest.mark.parametrize("sizes,H,I", [([40, 50, 30], 264, 136), ([30] * 30, 264, 264), ([400, 500], 520, 264),
                                       ([400, 0, 500, 600, 300, 241, 300, 400], 200, 2320)])
def test_offsets_past_the_rows(sizes, H, I):
    """Offsets that are not what they should be are cut to the rows there are, in every product forward and back."""
    c = Experts(sizes, H, I, 8)
    bank, n = c.bank.struct(), len(sizes)
    far = 2 ** 31 - 1
    for bad in ([0] + [40] * (n - 1) + [far], [-5] + [c.R + 10] * (n - 1) + [90], [far] + [0] * n, [-far - 1] * n + [far],
                [(c.R if e % 2 else 0) for e in range(n + 1)]):
        offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for i8 in (False, True):
            _, gu = forward(c, bank, i8, offsets)
            for need in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 1, 1)):
                backward(c, bank, c.x, gu, offsets, need)
        backward(c, bank, moe.quant_i8x16(c.x), None, offsets)


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (17, 264, 136), (129, 1032, 520), (515, 2056, 1336), (700, 264, 8), (1000, 1000, 1000)])
def test_dense(T, H, I):
    c = Experts([T], H, I, 3)
    bank = c.bank.struct()
    for i8 in (False, True):
        y, gu = forward(c, bank, i8, None)
        c.check_forward(y, gu, i8)
        kept = moe.quant_i8x16(c.x)
        c.check_backward(backward(c, bank, kept, gu, None), gu if i8 else None, kept)
        for k in range(4):
            c.check_backward(backward(c, bank, c.x, gu, None, [int(i == k) for i in range(4)]), gu if i8 else None)
    c.check_backward(backward(c, bank, c.x, None, None))
