"""The operators around the MoE layer at the edges of what their boundary
allows, against their formulas in 64 bits; inputs, formulas and bounds are those
of test_gpu_dense.py."""
import numpy as np
import pytest
import torch

import routed_expert_ffn_04_amd as moe
from dense_plan_cases import FFN as FFN_TILINGS, I8 as I8_TILINGS
from test_gpu_dense import (BF, F32, Ffn, HALF, I8, check_norm_grads, codes_of, norm_case, norm_grad_ref, norm_ref, outbuf,
                            rand, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm

# T that leaves the last run of rows short where a row takes 64 (4097, 1500 rows), 128, 256, 512 and 1024
# threads, and some that do not
EPS_SHAPES = [(4097, 64), (1500, 264), (777, 1001), (520, 1032), (1100, 2003), (600, 4104), (517, 8200), (1024, 512),
              (521, 1032), (601, 4104)]


@pytest.mark.parametrize("eps", [0.0, 1e-2])
@pytest.mark.parametrize("T,H", EPS_SHAPES)
def test_norm_with_another_eps(T, H, eps):
    """eps = 0 is allowed for rows that are not all zero: whatever the number of rows, every
    gradient is finite and right."""
    for gate_div in (None, 37):
        c = norm_case(T, H, 21, gate_div=gate_div)
        kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=c["gate_div"], res_scale=0.75, pre_w=c["pre_w"], eps=eps)
        r, x = moe.norm(c["y"], c["res"], x_dtype=F32, **kw)
        rr, xx, er, ex = norm_ref(c, eps=eps)
        within(r, rr, er + HALF[BF] * (rr.abs() + er), "r")
        within(x, xx, ex + HALF[F32] * (xx.abs() + ex), "x")
        got = moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], **kw)
        ref = norm_grad_ref(c, 0.75, eps)
        assert {k for k, v in got.items() if v is not None} == set(ref)
        for k, (v, e) in ref.items():
            within(got[k], v, e + HALF[got[k].dtype] * (v.abs() + e), f"{k} gate_div={gate_div}")


# rows that 64, 128, 256 (one and two chunks), 512 and 1024 threads hold; more rows than workers in the
# forward step, so that a worker takes several: the next row in flight, both LDS sets of the row sums
LONG_RUNS = [(9001, 264), (5001, 1001), (5003, 1024), (2501, 2003), (2500, 2048), (1201, 4104), (1200, 8192), (603, 8200),
             (600, 16383)]
TYPES = [(BF, BF, F32), (F32, F32, BF), (BF, F32, F32)]


@pytest.mark.parametrize("T,H", LONG_RUNS)
@pytest.mark.parametrize("y,r,w", TYPES)
def test_norm_with_several_rows_a_worker(T, H, y, r, w):
    """Forward, with gates that change inside a run of rows and one gate for all."""
    for gate_div, off in ((5, 0), (T, 0), (1, 1)):
        c = norm_case(T, H, 27, y, r, w, gate_div, off=off)
        kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=gate_div, res_scale=0.75, pre_w=c["pre_w"])
        ro, guard = outbuf((T, H), r)
        got_r, got_x = moe.norm(c["y"], c["res"], r=ro, x_dtype=F32, **kw)
        rr, xx, er, ex = norm_ref(c)
        within(got_r, rr, er + HALF[r] * (rr.abs() + er), "r")
        within(got_x, xx, ex + HALF[F32] * (xx.abs() + ex), "x")
        guard()
        _, (q, s) = moe.norm(c["y"], c["res"], x_dtype=I8, **kw)
        rq, rs = codes_of(got_x)
        assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("T,H", [(777, 1001), (1500, 1024), (1100, 2003), (1025, 2048), (600, 4104), (1031, 7168), (520, 8200),
                                 (513, 16384)])
@pytest.mark.parametrize("y,r,w", TYPES)
def test_norm_gradients_with_several_rows_a_run(T, H, y, r, w):
    """Runs of two to five rows, the last one short: gates that end inside a run, that are whole
    runs, that span runs, and none; with and without post_w and the gradient of x or r."""
    for gate_div in (None, 1, 2, 3, 37, T):
        check_norm_grads(norm_case(T, H, 28, y, r, w, gate_div))
    check_norm_grads(norm_case(T, H, 29, y, r, w, 37, post=False))
    c = norm_case(T, H, 30, y, r, w, 5)
    check_norm_grads(c, use_dx=False)
    check_norm_grads(c, use_dr=False)
    check_norm_grads(norm_case(T, H, 31, y, r, w, 7, off=1))


# ---------------------------------------------------------------- int8

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [16, 2064, 9008, 20000])
def test_a_nan_keeps_its_row_through_int8(cols, dtype):
    """One NaN (of either sign, anywhere in the row): the row's scale is NaN, and so is its row
    of the product; an infinity makes the scale infinite.  Other rows are as without them."""
    g = torch.Generator().manual_seed(cols)
    x = rand(g, (7, cols), 1.0, dtype)
    w = torch.randint(-127, 128, (24, cols), generator=g).to(I8).cuda()
    ws = torch.rand(24, generator=g).cuda()
    q0, s0 = moe.quant_i8(x)
    good = moe.linear_i8(q0, s0, w, ws, out_dtype=F32)
    bad = x.clone()
    nan = torch.tensor(float("nan"), dtype=dtype, device="cuda")
    bad[1, 0], bad[2, cols - 1], bad[4, cols // 2], bad[5] = nan, torch.copysign(nan, -torch.ones_like(nan)), nan, nan
    bad[4, 1], bad[6, 3] = float("inf"), -float("inf")
    q, s = moe.quant_i8(bad)
    y = moe.linear_i8(q, s, w, ws, out_dtype=F32)
    for t in (1, 2, 4, 5):
        assert bool(torch.isnan(s[t])) and bool(torch.isnan(y[t]).all()), t
    assert bool(torch.isinf(s[6]))
    for t in (0, 3):
        assert torch.equal(q[t], q0[t]) and torch.equal(s[t], s0[t]) and torch.equal(y[t], good[t])


@pytest.mark.parametrize("H", [264, 1001, 2560, 7168, 16384])
def test_a_nan_keeps_its_row_through_the_norm_to_int8(H):
    c = norm_case(9, H, 23, gate_div=3)
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=3, pre_w=c["pre_w"], x_dtype=I8)
    _, (q0, s0) = moe.norm(c["y"], c["res"], **kw)
    y, res = c["y"].clone(), c["res"].clone()
    y[4, H // 2], res[7, H - 1] = float("nan"), float("nan")
    _, (q, s) = moe.norm(y, res, **kw)
    assert torch.isnan(s).nonzero().flatten().tolist() == [4, 7]
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])


def test_quant_i8_of_the_longest_row():
    """2^31 - 16 columns, the most that the boundary takes: the steps of a thread pass 2^31."""
    cols = (1 << 31) - 16
    x = torch.empty(1, cols, dtype=BF, device="cuda")
    step = 1 << 28
    value = lambda at: (torch.arange(at, min(at + step, cols), device="cuda") % 251 - 125).to(BF)
    for at in range(0, cols, step):
        x[0, at:at + step] = value(at)
    x[0, cols - 1] = 127
    q, s = moe.quant_i8(x)
    assert s.tolist() == [1.0]
    for at in range(0, cols, step):
        want = value(at).to(I8)
        if at + step >= cols:
            want[-1] = 127
        assert torch.equal(q[0, at:at + step], want), at


# ---------------------------------------------------------------- sizes beyond an int32

def test_norm_of_more_rows_than_an_int32_holds_is_refused():
    y = torch.empty((1 << 32) + 4, 1, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        moe.norm(y)
    with pytest.raises(ValueError):
        moe.norm_backward(y, None, y, y)


@pytest.mark.parametrize("gate_div", [9, 10, 2 ** 31, 2 ** 32 + 1, 2 ** 40])
def test_one_gate_for_more_rows_than_there_are(gate_div):
    """However large gate_div is: the one gate applies to every row."""
    c = norm_case(9, 264, 25, gate_div=9)
    kw = dict(post_w=c["post_w"], gate=c["gate"], res_scale=0.75, pre_w=c["pre_w"])
    want = moe.norm(c["y"], c["res"], gate_div=9, **kw)
    got = moe.norm(c["y"], c["res"], gate_div=gate_div, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], gate_div=9, **kw)
    got = moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], gate_div=gate_div, **kw)
    assert all(torch.equal(got[k], want[k]) for k in want)


# ---------------------------------------------------------------- arguments that contradict each other

def test_dtypes_that_contradict_a_tensor_are_refused():
    """An output's dtype is the given tensor's; another one asked for beside it is an error."""
    f, c = Ffn(4, 64, 32), norm_case(4, 64, 26)
    new = lambda dtype, *shape: torch.empty(shape or (4, 64), dtype=dtype, device="cuda")
    q, w, one = new(I8), new(I8, 8, 64), new(F32, 4)
    for call in (lambda: moe.norm(c["y"], c["res"], r_dtype=F32),                     # r is kept like res
                 lambda: moe.norm(c["y"], r=new(BF), r_dtype=F32),
                 lambda: moe.norm(c["y"], c["res"], r=new(F32)),
                 lambda: moe.norm(c["y"], c["res"], x=new(BF), x_dtype=F32),
                 lambda: moe.norm(c["y"], c["res"], x=(q, one), x_dtype=BF),
                 lambda: moe.norm(c["y"], c["res"], x=(new(BF), one)),                # scales go with int8 codes
                 lambda: moe.norm(c["y"], c["res"], x=(None, one)),
                 lambda: moe.ffn(f.x, f.bank, out=new(BF), y_dtype=F32),
                 lambda: moe.linear_i8(q, one, w, new(F32, 8), out=new(F32, 4, 8), out_dtype=BF)):
        with pytest.raises(TypeError):
            call()
    # the same dtype again is no contradiction
    assert moe.norm(c["y"], c["res"], r_dtype=BF, x=new(F32), x_dtype=F32)[0].dtype is BF
    assert moe.norm(c["y"], r_dtype=F32)[0].dtype is F32
    assert moe.norm(c["y"], c["res"], x=(q, one), x_dtype=I8)[1][0] is q
    assert moe.norm(c["y"], c["res"], x=(None, one), x_dtype=I8)[1][1] is one
    assert moe.ffn(f.x, f.bank, out=new(F32), y_dtype=F32).dtype is F32


# ---------------------------------------------------------------- grids

def test_linear_i8_of_more_columns_than_the_few_row_grid_holds():
    """One token and 2^27 + 16 output channels: beyond the grid of the kernel for a few rows."""
    N, K = (1 << 27) + 16, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randint(-127, 128, (N, K), generator=gen, dtype=I8, device="cuda")
    ws = torch.rand(N, generator=gen, device="cuda")
    q = torch.randint(-127, 128, (1, K), generator=gen, dtype=I8, device="cuda")
    qs = torch.tensor([0.37], device="cuda")
    out = moe.linear_i8(q, qs, w, ws, out_dtype=F32)
    step = 1 << 24
    for at in range(0, N, step):
        total = (w[at:at + step].int() * q.int()).sum(1)       # exact, and so is its conversion: below 2^24
        assert torch.equal(out[0, at:at + step], total.float() * (qs * ws[at:at + step])), at


def test_gradients_of_no_tokens_are_zero_in_large_matrices():
    H, I = 4096, 4104
    bank = moe.Experts(*(torch.zeros(s, dtype=BF, device="cuda") for s in ((1, I, H), (1, I, H), (1, H, I))))
    none = torch.empty(0, H, dtype=BF, device="cuda")
    torch.full((3 * H * I,), float("nan"), dtype=BF, device="cuda")      # what the outputs' memory may hold
    for g in moe.ffn_backward(none, none, bank)[1:]:
        assert bool((g == 0).all())


# ---------------------------------------------------------------- every tiling of the products

FORWARD = sorted({sizes for product, _, sizes in FFN_TILINGS if product in ("gateup", "down")})
BACKWARD = sorted({(product, sizes) for product, _, sizes in FFN_TILINGS if product not in ("gateup", "down")})
NEED = {"dh": ("dw_up",), "dx": ("dx",), "dwgu": ("dw_gate", "dw_up"), "dw1": ("dw_up",), "dwd": ("dw_down",),
        "grads": ("dx", "dw_gate", "dw_up", "dw_down")}


@pytest.mark.parametrize("T,H,I", FORWARD)
def test_ffn_tilings(T, H, I):
    c = Ffn(T, H, I, 31)
    out, guard = outbuf((T, H), BF)
    gu, guard_gu = outbuf((T, 2 * I), F32)
    y, gu = moe.ffn(c.x, c.bank, want_gu=True, out=out, gu=gu)
    c.check_y(y)
    c.check_gu(gu)
    guard()
    guard_gu()
    assert torch.equal(moe.ffn(c.x, c.bank), y)
    c.check_y(moe.ffn(c.x, c.bank, y_dtype=F32), "fp32 y")


@pytest.mark.parametrize("product,sizes", BACKWARD)
def test_ffn_gradient_tilings(product, sizes):
    c = Ffn(*sizes, 32)
    _, gu = moe.ffn(c.x, c.bank, want_gu=True)
    grads = moe.ffn_backward(c.dy, c.x, c.bank, gu, need=NEED[product])
    assert [g is not None for g in grads] == [n in NEED[product] for n in NEED["grads"]]
    c.check_grads(grads)
    if product == "dw1":
        c.check_grads(moe.ffn_backward(c.dy, c.x, c.bank, gu, need=("dw_gate",)))


@pytest.mark.parametrize("T,K,N", [sizes for _, _, sizes in I8_TILINGS])
def test_linear_i8_tilings(T, K, N):
    """The sum is exact and its three fp32 roundings are those of the formula, so fp32 outputs are equal bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(T + K + N)
    q, w = (torch.randint(-128, 128, s, generator=gen, dtype=I8, device="cuda") for s in ((T, K), (N, K)))
    qs, ws, b = (torch.randn(n, generator=gen, device="cuda") for n in (T, N, N))
    total = (q.double() @ w.double().t()).float()                # exact in 64 bits
    ref = total * (qs[:, None] * ws)
    for bias, out in ((None, F32), (b, F32), (None, BF), (b, BF)):
        o, guard = outbuf((T, N), out)
        moe.linear_i8(q, qs, w, ws, bias, out=o)
        want = ref if bias is None else ref + bias
        assert torch.equal(o, want.to(out)), (bias is not None, out)
        guard()


# ---------------------------------------------------------------- tensors of more than 2^31 elements

def test_ffn_of_more_elements_than_an_int32_counts():
    """Only the last rows are not zero, so everything, the weights' gradients too, is as for them alone."""
    T, H, I, n = 524400, 4104, 264, 400
    assert (T - n) * H > 1 << 31
    c = Ffn(n, H, I, 33)
    x, dy = (torch.zeros(T, H, dtype=BF, device="cuda") for _ in range(2))
    x[-n:], dy[-n:] = c.x, c.dy
    y, gu = moe.ffn(x, c.bank, want_gu=True)
    c.check_y(y[-n:])
    c.check_gu(gu[-n:])
    assert not bool(y[:-n].any())
    dx, *dw = moe.ffn_backward(dy, x, c.bank, gu)
    c.check_grads([dx[-n:], *dw])
    assert not bool(dx[:-n].any())


def test_norm_of_more_elements_than_an_int32_counts():
    """Rows do not depend on each other: the last ones are as in a call of their own."""
    T, H, n = 262400, 8192, 200
    assert (T - n) * H > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(5)
    y, res, dx = (torch.empty(T, H, dtype=BF, device="cuda").normal_(generator=gen) for _ in range(3))
    w = torch.rand(H, generator=gen, device="cuda") + 0.5
    kw = dict(post_w=w, pre_w=w, res_scale=0.75)
    for x_dtype in (BF, I8):
        r, x = moe.norm(y, res, x_dtype=x_dtype, **kw)
        r1, x1 = moe.norm(y[-n:], res[-n:], x_dtype=x_dtype, **kw)
        assert torch.equal(r[-n:], r1)
        for a, b in zip(x, x1) if x_dtype is I8 else ((x, x1),):
            assert torch.equal(a[-n:], b)
    g = moe.norm_backward(dx, res, y, r, **kw)
    g1 = moe.norm_backward(dx[-n:], res[-n:], y[-n:], r1, **kw)
    assert torch.equal(g["dy"][-n:], g1["dy"]) and torch.equal(g["dres"][-n:], g1["dres"])


@pytest.mark.parametrize("T,K,N", [(131200, 16400, 72), (3, 16400, 131200), (40, 16400, 131200), (131200, 16, 16500)])
def test_linear_i8_of_more_elements_than_an_int32_counts(T, K, N):
    """Codes, weights (few rows and tiles) and outputs: the last rows and columns, bit for bit."""
    assert max(T * K, N * K, T * N) > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, w = (torch.randint(-128, 128, s, generator=gen, dtype=I8, device="cuda") for s in ((T, K), (N, K)))
    qs, ws = torch.rand(T, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    out = moe.linear_i8(q, qs, w, ws, out_dtype=F32)
    t, n = slice(max(0, T - 150), T), slice(max(0, N - 150), N)
    total = (q[t].double() @ w[n].double().t()).float()
    assert torch.equal(out[t, n], total * (qs[t, None] * ws[n]))


# ---------------------------------------------------------------- streams

def test_norm_and_int8_on_streams_of_their_own():
    """Two streams at once, each call's scratch and outputs its own."""
    c = norm_case(1500, 520, 34, gate_div=37)
    w = torch.randint(-127, 128, (130, 512), dtype=I8, device="cuda")
    ws = torch.rand(130, device="cuda")
    x = c["y"][:, :512].contiguous()
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=37, pre_w=c["pre_w"])

    def calls(stream=None):
        q, s = moe.quant_i8(x, stream=stream)
        return [*moe.norm(c["y"], c["res"], stream=stream, **kw),
                *moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], stream=stream, **kw).values(),
                q, s, moe.linear_i8(q, s, w, ws, stream=stream)]
    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [calls(s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, want))
