"""The operators around the MoE layer against their formulas in 64 bits.

Tolerances are elementwise bounds: a rounding to a type is off by at most half
a step of the value (bf16 2^-8, fp32 2^-24 relative), a sum of n terms in fp32 by
at most n 2^-23 of the sum of magnitudes (the matrix cores may truncate where a
CPU would round), and errors of what goes into a step are carried through it with
the magnitudes of its other factors."""
import numpy as np
import pytest
import torch

import routed_expert_ffn_04_amd as moe

pytestmark = pytest.mark.gpu

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def gamma(n):
    return (n + 4) * 2.0 ** -23


def rand(g, shape, scale, dtype, mean=0.0):
    """A tensor inside a larger buffer of NaN (int8: -128), so that reads past either end show."""
    n = int(np.prod(shape))
    v = torch.randn(n, generator=g, dtype=torch.float32) * scale + mean
    big = torch.full((n + 2048,), float("nan"), dtype=dtype, device="cuda")
    big[1024:1024 + n] = v.to(device="cuda", dtype=dtype)
    return big[1024:1024 + n].view(shape)


def outbuf(shape, dtype):
    """(tensor to write, check): the bytes around it keep their pattern."""
    n = int(np.prod(shape))
    raw = torch.full((n + 2048,), 77, dtype=dtype, device="cuda")

    def check():
        assert bool((raw[:1024] == 77).all()) and bool((raw[1024 + n:] == 77).all()), "written out of range"
    return raw[1024:1024 + n].view(shape), check


def within(got, ref, tol, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = ((got - ref).abs() - tol).max().item() if got.numel() else -1.0
    assert over <= 0, f"{what}: off by {over} more than its bound (largest bound {tol.max().item()})"


# ---------------------------------------------------------------- dense FFN

class Ffn:
    """Inputs, the formulas in 64 bits and their error bounds."""

    def __init__(self, T, H, I, seed=0):
        g = torch.Generator().manual_seed(1000 * seed + T + H + I)
        self.x, self.dy = rand(g, (T, H), 1.0, BF), rand(g, (T, H), 1.0, BF)
        self.wg, self.wu = rand(g, (1, I, H), H ** -0.5, BF), rand(g, (1, I, H), H ** -0.5, BF)
        self.wd = rand(g, (1, H, I), I ** -0.5, BF)
        self.bank = moe.Experts(self.wg, self.wu, self.wd)
        x, dy, wg, wu, wd = (t.double() for t in (self.x, self.dy, self.wg[0], self.wu[0], self.wd[0]))
        self.g, self.u = x @ wg.t(), x @ wu.t()
        s = torch.sigmoid(self.g)
        a = self.g * s
        h = a * self.u
        # bounds of g and u, and of h before and after its rounding; hardware exp and reciprocal: 2^-20
        self.eg, self.eu = gamma(H) * (x.abs() @ wg.abs().t()), gamma(H) * (x.abs() @ wu.abs().t())
        eh = 1.1 * self.u.abs() * self.eg + a.abs() * self.eu + 2.0 ** -20 * h.abs()
        eh = eh + HALF[BF] * (h.abs() + eh)
        self.y = h @ wd.t()
        self.ey = eh @ wd.abs().t() + gamma(I) * (h.abs() @ wd.abs().t())
        dh = dy @ wd
        edh = gamma(H) * (dy.abs() @ wd.abs())
        slope = s * (1 + self.g * (1 - s))
        dg, du = dh * self.u * slope, dh * a
        # |slope| <= 1.1, its derivative <= 0.5 in magnitude
        edg = (self.u * slope).abs() * edh + (dh * slope).abs() * self.eu + 0.5 * (dh * self.u).abs() * self.eg
        edg = edg + 2.0 ** -20 * (dh * self.u).abs() * (s + (a * (1 - s)).abs())
        edg = edg + HALF[BF] * (dg.abs() + edg)
        edu = a.abs() * edh + 1.1 * dh.abs() * self.eg + 2.0 ** -20 * du.abs()
        edu = edu + HALF[BF] * (du.abs() + edu)
        self.dx = dg @ wg + du @ wu
        mag = dg.abs() @ wg.abs() + du.abs() @ wu.abs()
        self.edx = edg @ wg.abs() + edu @ wu.abs() + gamma(2 * I) * mag
        self.dwg, self.dwu, self.dwd = dg.t() @ x, du.t() @ x, dy.t() @ h
        self.edwg = edg.t() @ x.abs() + gamma(T) * (dg.abs().t() @ x.abs())
        self.edwu = edu.t() @ x.abs() + gamma(T) * (du.abs().t() @ x.abs())
        self.edwd = dy.abs().t() @ eh + gamma(T) * (dy.abs().t() @ h.abs())

    def check_y(self, y, what="y"):
        within(y, self.y, self.ey + HALF[y.dtype] * (self.y.abs() + self.ey), what)

    def check_gu(self, gu):
        I = self.g.shape[1]
        within(gu[:, :I], self.g, self.eg, "g")
        within(gu[:, I:], self.u, self.eu, "u")

    def check_grads(self, grads):
        for name, got, ref, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, (self.dx, self.dwg, self.dwu, self.dwd),
                                     (self.edx, self.edwg, self.edwu, self.edwd)):
            if got is not None:
                within(got.view(ref.shape), ref, e + HALF[BF] * (ref.abs() + e), name)


# token counts around the tiles (16, 128, 256), hidden sizes below, at and off a stage (32) and a tile
FFN_SHAPES = [(1, 8, 8), (1, 256, 512), (2, 7168, 2048), (3, 264, 136), (16, 1024, 512), (17, 1032, 520), (33, 40, 1000),
              (64, 256, 512), (65, 512, 264), (127, 256, 128), (128, 7168, 2048), (129, 136, 264), (255, 512, 512),
              (257, 2056, 1336), (515, 264, 8), (1000, 8, 264), (2049, 1024, 512), (4096, 2048, 1024)]


@pytest.mark.parametrize("T,H,I", FFN_SHAPES)
def test_ffn_forward(T, H, I):
    c = Ffn(T, H, I)
    out, guard = outbuf((T, H), BF)
    gu, guard_gu = outbuf((T, 2 * I), F32)
    y, gu = moe.ffn(c.x, c.bank, want_gu=True, out=out, gu=gu)
    c.check_y(y)
    c.check_gu(gu)
    guard()
    guard_gu()
    assert torch.equal(moe.ffn(c.x, c.bank), y)                       # without gu: the same
    c.check_y(moe.ffn(c.x, c.bank, y_dtype=F32), "fp32 y")


@pytest.mark.parametrize("T,H,I", FFN_SHAPES)
def test_ffn_backward(T, H, I):
    c = Ffn(T, H, I, 1)
    _, gu = moe.ffn(c.x, c.bank, want_gu=True)
    grads = moe.ffn_backward(c.dy, c.x, c.bank, gu)
    c.check_grads(grads)
    again = moe.ffn_backward(c.dy, c.x, c.bank)                       # g and u computed again
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    for k, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):  # each one alone
        one = moe.ffn_backward(c.dy, c.x, c.bank, gu, need=(name,))
        assert [t is None for t in one] == [i != k for i in range(4)]
        c.check_grads(one)


def test_ffn_large_values():
    """g far in both tails of the sigmoid: exp overflows to infinity on one side."""
    c = Ffn(40, 64, 64, 2)
    x = (c.x.float() * 300).to(BF)
    y, gu = moe.ffn(x, c.bank, want_gu=True)
    assert gu.abs().max().item() > 200
    g, u = (gu[:, :64].double(), gu[:, 64:].double())
    s = torch.sigmoid(g)
    dh = c.dy.double() @ c.wd[0].double()
    dx, dwg, dwu, dwd = moe.ffn_backward(c.dy, x, c.bank, gu)
    for t in (y, dx, dwg, dwu, dwd):
        assert bool(torch.isfinite(t).all())
    dg = dh * u * (s + g * s * (1 - s))
    ref = dg.t() @ x.double()
    # dg's own rounding and dh's sum, through the product
    e = (HALF[BF] + 2.0 ** -19) * (dg.abs().t() @ x.double().abs())
    e = e + gamma(64) * (((c.dy.double().abs() @ c.wd[0].double().abs()) * u.abs() * 1.1).t() @ x.double().abs())
    e = e + gamma(40) * (dg.abs().t() @ x.double().abs())
    within(dwg[0], ref, e + HALF[BF] * (ref.abs() + e), "dw_gate")


def test_ffn_gradients_against_differences():
    """dx and dw against central differences of the fp32-output forward pass along random directions."""
    T, H, I = 48, 96, 80
    c = Ffn(T, H, I, 3)
    _, gu = moe.ffn(c.x, c.bank, want_gu=True)
    grads = moe.ffn_backward(c.dy, c.x, c.bank, gu)
    t64 = lambda x, wg, wu, wd: (((x @ wg.t()) * torch.sigmoid(x @ wg.t()) * (x @ wu.t())) @ wd.t() * c.dy.double()).sum()
    base = [c.x.double(), c.wg[0].double(), c.wu[0].double(), c.wd[0].double()]
    bounds = [c.edx, c.edwg, c.edwu, c.edwd]
    gen = torch.Generator(device="cuda").manual_seed(9)
    for k in range(4):
        d = torch.randn(base[k].shape, generator=gen, dtype=torch.float64, device="cuda")
        eps = 1e-5
        hi, lo = list(base), list(base)
        hi[k], lo[k] = base[k] + eps * d, base[k] - eps * d
        diff = (t64(*hi) - t64(*lo)) / (2 * eps)
        got = grads[k].view(d.shape).double()
        tol = ((bounds[k] + HALF[BF] * (got.abs() + bounds[k])) * d.abs()).sum() + 1e-4 * diff.abs()
        assert (got * d).sum().sub(diff).abs() <= tol


def test_ffn_no_tokens():
    c = Ffn(4, 64, 32)
    assert moe.ffn(c.x[:0], c.bank).shape == (0, 64)
    dx, dwg, dwu, dwd = moe.ffn_backward(c.dy[:0], c.x[:0], c.bank)
    assert dx.shape == (0, 64)
    for t in (dwg, dwu, dwd):
        assert bool((t == 0).all())


# ---------------------------------------------------------------- norm

def norm_case(T, H, seed=0, y=BF, r=BF, w=F32, gate_div=None, post=True, pre=True, off=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + H)

    def cut(shape, scale, dtype, mean=0.0):
        if not off:
            return rand(g, shape, scale, dtype, mean)
        n = int(np.prod(shape))   # element offset `off`: not 16-byte aligned
        return rand(g, (n + off,), scale, dtype, mean)[off:].view(shape)
    return {"y": cut((T, H), 0.5, y), "res": cut((T, H), 2.0, r), "post_w": cut((H,), 0.1, w, 1.0) if post else None,
            "pre_w": cut((H,), 0.1, w, 1.0) if pre else None, "gate_div": gate_div or 1,
            "gate": cut((-(-T // gate_div), H), 0.25, w, 0.5) if gate_div else None,
            "dx": cut((T, H), 1.0, BF), "dr": cut((T, H), 1.0, r)}


def norm_ref(c, a=0.75, eps=1e-6, res=True):
    """(r, x, bound of r, bound of x before their last rounding) in 64 bits."""
    y = c["y"].double()
    H = y.shape[1]
    rel = 80 * 2.0 ** -24   # a row's mean (at most 64 terms a thread, then a tree), the root and the products
    n = y
    if c["post_w"] is not None:
        n = y / (y.square().mean(1, keepdim=True) + eps).sqrt() * c["post_w"].double()
    if c["gate"] is not None:
        n = n * c["gate"].double().repeat_interleave(c["gate_div"], 0)[:y.shape[0]]
    base = a * c["res"].double() if res else torch.zeros_like(y)
    r = base + n
    er = rel * n.abs() + 2.0 ** -23 * (base.abs() + n.abs())
    inv = 1 / (r.square().mean(1, keepdim=True) + eps).sqrt()
    w = c["pre_w"].double() if c["pre_w"] is not None else torch.ones(H, dtype=torch.float64, device=y.device)
    x = r * inv * w
    # rms(r) moves by at most the rms of er
    ex = er * inv * w.abs() + x.abs() * (rel + inv * er.square().mean(1, keepdim=True).sqrt())
    return r, x, er, ex


NORM_SHAPES = [(1, 1), (1, 7168), (2, 8), (3, 7), (5, 63), (4, 512), (7, 520), (130, 65), (9, 1001), (33, 2048), (17, 2056),
               (6, 4096), (5, 4104), (3, 8192), (2, 8200), (2, 16384), (2, 16383), (3, 4097), (700, 128)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("y,r,x,w", [(BF, BF, BF, F32), (F32, F32, F32, F32), (BF, F32, BF, BF), (F32, BF, F32, BF)])
def test_norm_forward(T, H, y, r, x, w):
    for gate_div, post in ((None, True), (1, False), (T, True), (max(1, T // 3), True)):
        c = norm_case(T, H, 1, y, r, w, gate_div, post)
        ro, guard_r = outbuf((T, H), r)
        xo, guard_x = outbuf((T, H), x)
        got = moe.norm(c["y"], c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=c["gate_div"], res_scale=0.75,
                       pre_w=c["pre_w"], r=ro, x=xo)
        rr, xx, er, ex = norm_ref(c)
        within(got[0], rr, er + HALF[r] * (rr.abs() + er), "r")
        within(got[1], xx, ex + HALF[x] * (xx.abs() + ex), "x")
        guard_r()
        guard_x()


def test_norm_variants():
    c = norm_case(9, 264, 2, gate_div=4)
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=4, pre_w=c["pre_w"])
    r, x = moe.norm(c["y"], c["res"], **kw)
    assert moe.norm(c["y"], c["res"], want_x=False, **kw)[1] is None
    only_x = moe.norm(c["y"], c["res"], want_r=False, **kw)
    assert only_x[0] is None and torch.equal(only_x[1], x)
    # no residual, no weights
    d = dict(c, post_w=None, pre_w=None, gate=None)
    rr, xx, er, ex = norm_ref(d, res=False)
    r0, x0 = moe.norm(c["y"])
    within(r0, rr, er + HALF[BF] * (rr.abs() + er), "r without residual")
    within(x0, xx, ex + HALF[BF] * (xx.abs() + ex), "x without weights")
    # in place on the residual stream
    res = c["res"].clone()
    r1, x1 = moe.norm(c["y"], res, r=res, **kw)
    assert r1.data_ptr() == res.data_ptr() and torch.equal(r1, r) and torch.equal(x1, x)
    # rows of zeros: rms is sqrt(eps), everything is 0
    z = torch.zeros_like(c["y"])
    r2, x2 = moe.norm(z, torch.zeros_like(c["res"]), **kw)
    assert bool((r2 == 0).all()) and bool((x2 == 0).all())
    assert moe.norm(c["y"][:0], c["res"][:0], pre_w=c["pre_w"])[0].shape == (0, 264)


@pytest.mark.parametrize("T,H", [(5, 264), (3, 7168), (2, 96)])
def test_norm_unaligned_rows_equal_aligned_ones(T, H):
    """One element off a 16-byte boundary takes the narrow loads: within the same bounds."""
    c = norm_case(T, H, 3, gate_div=2, off=1)
    assert c["y"].data_ptr() % 16 != 0
    r, x = moe.norm(c["y"], c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=2, res_scale=0.75, pre_w=c["pre_w"])
    rr, xx, er, ex = norm_ref(c)
    within(r, rr, er + HALF[BF] * (rr.abs() + er), "r")
    within(x, xx, ex + HALF[BF] * (xx.abs() + ex), "x")
    check_norm_grads(c)


def norm_grad_ref(c, a, eps=1e-6, use_dx=True, use_dr=True):
    """{name: (value, bound before its last rounding)} in 64 bits; c["res"] is the stored r."""
    rel = 120 * 2.0 ** -24
    y, r = c["y"].double(), c["res"].double()
    T, H = y.shape
    dr = c["dr"].double() if use_dr else torch.zeros_like(r)
    d, ed = dr, torch.zeros_like(dr)
    out = {}
    if use_dx:
        dx = c["dx"].double()
        w = c["pre_w"].double() if c["pre_w"] is not None else torch.ones(H, dtype=torch.float64, device=y.device)
        inv = 1 / (r.square().mean(1, keepdim=True) + eps).sqrt()
        xh, t = r * inv, dx * w
        m, mm = (t * xh).mean(1, keepdim=True), (t * xh).abs().mean(1, keepdim=True)
        d = dr + inv * (t - xh * m)
        ed = rel * (dr.abs() + inv * (t.abs() + xh.abs() * mm))
        if c["pre_w"] is not None:
            out["dpre_w"] = ((dx * xh).sum(0), (rel + gamma(T)) * (dx * xh).abs().sum(0))
    out["dres"] = (a * d, abs(a) * (ed + 2.0 ** -23 * d.abs()))
    has_post, has_gate = c["post_w"] is not None, c["gate"] is not None
    p = 1 / (y.square().mean(1, keepdim=True) + eps).sqrt()
    yh = y * p
    n = yh * c["post_w"].double() if has_post else y
    dn, edn = d, ed
    if has_gate:
        gd = c["gate_div"]
        G = c["gate"].shape[0]
        at = torch.arange(T, device=y.device) // gd
        gr = c["gate"].double()[at]
        val = torch.zeros((G, H), dtype=torch.float64, device=y.device).index_add_(0, at, d * n)
        err = (ed * n.abs()) + (rel + gamma(min(gd, T))) * (d * n).abs()
        out["dgate"] = (val, torch.zeros_like(val).index_add_(0, at, err))
        dn, edn = d * gr, ed * gr.abs() + 2.0 ** -24 * (d * gr).abs()
    if has_post:
        w = c["post_w"].double()
        out["dpost_w"] = ((dn * yh).sum(0), ((edn * yh.abs()) + (rel + gamma(T)) * (dn * yh).abs()).sum(0))
        t, et = dn * w, edn * w.abs()
        m = (t * yh).mean(1, keepdim=True)
        em = (et * yh.abs() + rel * (t * yh).abs()).mean(1, keepdim=True)
        edn = p * (et + yh.abs() * em + rel * (t.abs() + yh.abs() * (t * yh).abs().mean(1, keepdim=True)))
        dn = p * (t - yh * m)
    out["dy"] = (dn, edn + 2.0 ** -23 * dn.abs())
    return out


def check_norm_grads(c, a=0.75, use_dx=True, use_dr=True, **kw):
    got = moe.norm_backward(c["dx"] if use_dx else None, c["dr"] if use_dr else None, c["y"], c["res"], post_w=c["post_w"],
                            gate=c["gate"], gate_div=c["gate_div"], res_scale=a, pre_w=c["pre_w"], **kw)
    ref = norm_grad_ref(c, a, use_dx=use_dx, use_dr=use_dr)
    assert {k for k, v in got.items() if v is not None} == set(ref)
    for k, (v, e) in ref.items():
        within(got[k], v, e + HALF[got[k].dtype] * (v.abs() + e), k)
    return got


@pytest.mark.parametrize("T,H", NORM_SHAPES + [(1500, 264), (4097, 64)])
@pytest.mark.parametrize("y,r,w", [(BF, BF, F32), (F32, F32, BF), (BF, F32, F32)])
def test_norm_backward(T, H, y, r, w):
    for gate_div, post in ((None, True), (1, True), (T, False), (T, True), (max(1, T // 3), True), (3, True), (37, True)):
        check_norm_grads(norm_case(T, H, 4, y, r, w, gate_div, post))


def test_norm_backward_parts():
    c = norm_case(50, 264, 5, gate_div=7)
    check_norm_grads(c, use_dx=False)
    check_norm_grads(c, use_dr=False)
    check_norm_grads(dict(c, pre_w=None))
    check_norm_grads(dict(c, post_w=None, gate=None))
    full = check_norm_grads(c)
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=7, res_scale=0.75, pre_w=c["pre_w"])
    for name in full:
        one = moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], need=(name,), **kw)
        assert [k for k, v in one.items() if v is not None] == [name]
        assert torch.equal(one[name], full[name])
    none = moe.norm_backward(c["dx"][:0], c["dr"][:0], c["y"][:0], c["res"][:0], post_w=c["post_w"], pre_w=c["pre_w"])
    assert bool((none["dpost_w"] == 0).all()) and bool((none["dpre_w"] == 0).all()) and none["dy"].shape == (0, 264)


def test_norm_gradients_against_differences():
    T, H, a, eps = 12, 40, 0.75, 1e-6
    c = norm_case(T, H, 6, F32, F32, F32, 5, True)
    # loss = <x, dx> + <r, dr> at the forward step's own r
    y, res, pw, g, w = (c[k].double() for k in ("y", "res", "post_w", "gate", "pre_w"))
    dx, dr = c["dx"].double(), c["dr"].double()

    def loss(y, res, pw, g, w):
        n = y / (y.square().mean(1, keepdim=True) + eps).sqrt() * pw * g.repeat_interleave(5, 0)[:T]
        r = a * res + n
        x = r / (r.square().mean(1, keepdim=True) + eps).sqrt() * w
        return (x * dx).sum() + (r * dr).sum()
    r, _ = moe.norm(c["y"], c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=5, res_scale=a, pre_w=c["pre_w"])
    got = moe.norm_backward(c["dx"], c["dr"], c["y"], r, post_w=c["post_w"], gate=c["gate"], gate_div=5, res_scale=a,
                            pre_w=c["pre_w"])
    base = [y, res, pw, g, w]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for k, name in enumerate(("dy", "dres", "dpost_w", "dgate", "dpre_w")):
        d = torch.randn(base[k].shape, generator=gen, dtype=torch.float64, device="cuda")
        hi, lo = list(base), list(base)
        hi[k], lo[k] = base[k] + 1e-5 * d, base[k] - 1e-5 * d
        diff = (loss(*hi) - loss(*lo)) / 2e-5
        dot = (got[name].double() * d)
        assert (dot.sum() - diff).abs() <= 1e-5 * dot.abs().sum()


# ---------------------------------------------------------------- int8

def codes_of(x):
    x = x.float().cpu().numpy()
    amax = np.abs(x).max(axis=1)
    s = (amax / np.float32(127)).astype(np.float32)
    s[s == 0] = 1
    return np.clip(np.rint(x / s[:, None]), -127, 127).astype(np.int8), s


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 2048), (2, 2064), (130, 7168), (7, 16384)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quant_i8_equals_the_rule(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = rand(g, (rows, cols), 1.0, dtype)
    x[0] = 0                                                 # a row of zeros
    if rows > 1:
        x[1, 0] = 4.0
        x[1, 1:] = x[1, 1:].clamp(-4, 4)
        x[1, 1], x[1, 2] = 2.0, -2.0                         # exactly half of the maximum: 63.5, a tie
    if rows > 2:
        x[2] = x[2] * 1e-38                                  # subnormal scale
    out = (outbuf((rows, cols), I8), outbuf((rows,), F32))
    q, s = moe.quant_i8(x, out=(out[0][0], out[1][0]))
    rq, rs = codes_of(x)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    out[0][1]()
    out[1][1]()


I8_SHAPES = [(1, 16, 1), (1, 64, 17), (2, 7168, 4096), (3, 80, 129), (16, 2064, 1501), (17, 48, 255), (33, 1024, 512),
             (64, 512, 1000), (127, 144, 128), (128, 7168, 512), (129, 4096, 130), (257, 272, 257), (333, 2064, 1501),
             (1025, 512, 264), (2048, 1024, 8), (2049, 2048, 2056)]


@pytest.mark.parametrize("T,K,N", I8_SHAPES)
@pytest.mark.parametrize("out,bias", [(F32, True), (BF, False), (BF, True)])
def test_linear_i8(T, K, N, out, bias):
    g = torch.Generator().manual_seed(T + K + N)

    def codes(shape):
        n = int(np.prod(shape))
        big = torch.full((n + 2048,), -128, dtype=I8, device="cuda")
        big[1024:1024 + n] = torch.randint(-128, 128, (n,), generator=g).to(I8).cuda()
        return big[1024:1024 + n].view(shape)
    q, w = codes((T, K)), codes((N, K))
    qs, wsc = rand(g, (T,), 1.0, F32), rand(g, (N,), 1.0, F32)
    b = rand(g, (N,), 100.0, F32) if bias else None
    o, guard = outbuf((T, N), out)
    y = moe.linear_i8(q, qs, w, wsc, b, out=o)
    ref = (q.double() @ w.double().t()) * (qs.double()[:, None] * wsc.double())
    tol = 3 * 2.0 ** -24 * ref.abs()      # the sum to fp32, the product of the scales, their product
    if bias:
        ref = ref + b.double()
        tol = tol + 2.0 ** -24 * (ref.abs() + tol)
    within(y, ref, tol + HALF[out] * (ref.abs() + tol), "out")
    guard()


def test_linear_i8_extreme_sums():
    """The largest K: the int32 sum reaches 128 * 128 * K, just below 2^31."""
    K = 131056
    q = torch.full((3, K), -128, dtype=I8, device="cuda")
    w = torch.full((5, K), -128, dtype=I8, device="cuda")
    w[1] = 127
    one = torch.ones(3, device="cuda")
    out = moe.linear_i8(q, one, w, torch.ones(5, device="cuda"), out_dtype=F32)
    assert bool((out[:, 0] == float(128 * 128 * K)).all())
    assert bool((out[:, 1].double() == float(np.float32(-128 * 127 * K))).all())


def test_linear_i8_unaligned_output():
    g = torch.Generator().manual_seed(5)
    q, w = (torch.randint(-128, 128, s, generator=g).to(I8).cuda() for s in ((9, 64), (24, 64)))
    one, ones = torch.ones(9, device="cuda"), torch.ones(24, device="cuda")
    buf = torch.zeros(9 * 24 + 3, dtype=F32, device="cuda")
    o = buf[3:].view(9, 24)
    moe.linear_i8(q, one, w, ones, out=o)
    assert torch.equal(o.double(), q.double() @ w.double().t()) and bool((buf[:3] == 0).all())


@pytest.mark.parametrize("T,H,N", [(1, 256, 40), (5, 7168, 64), (40, 272, 33)])
def test_norm_to_i8_product(T, H, N):
    """The norm step writing codes: they are the quantised fp32 x, up to its own error at a rounding border."""
    c = norm_case(T, H, 8, gate_div=2)
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=2, res_scale=0.75, pre_w=c["pre_w"])
    r, (q, s) = moe.norm(c["y"], c["res"], x_dtype=I8, **kw)
    r2, x32 = moe.norm(c["y"], c["res"], x_dtype=F32, **kw)
    assert torch.equal(r, r2)
    rq, rs = codes_of(x32)            # the same fp32 x, quantised by the rule
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    g = torch.Generator().manual_seed(N)
    w = torch.randint(-127, 128, (N, H), generator=g).to(I8).cuda()
    wsc = torch.rand(N, generator=g).cuda()
    y = moe.linear_i8(q, s, w, wsc, out_dtype=F32)
    ref = (q.double() @ w.double().t()) * (s.double()[:, None] * wsc.double())
    within(y, ref, 4 * 2.0 ** -24 * ref.abs(), "out")


# ---------------------------------------------------------------- as they are used

def test_refusals_on_the_gpu():
    c = Ffn(4, 64, 32)
    with pytest.raises(ValueError):
        moe.ffn(c.x.t(), c.bank)                                   # shape
    with pytest.raises(ValueError):
        moe.ffn(torch.zeros(4, 128, dtype=BF, device="cuda")[:, ::2], c.bank)      # strides
    with pytest.raises(TypeError):
        moe.ffn(c.x.float(), c.bank)
    with pytest.raises(ValueError):
        moe.ffn_backward(c.dy[:3], c.x, c.bank)
    with pytest.raises(moe.MoeError):
        moe.ffn(c.x, c.bank, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.norm(c.x, gate=torch.ones(3, 64, device="cuda"), gate_div=2)           # 2 rows wanted
    with pytest.raises(TypeError):
        moe.norm(c.x, gate=torch.ones(4, 64, device="cuda"), pre_w=torch.ones(64, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        moe.linear_i8(torch.zeros(2, 32, dtype=I8, device="cuda"), torch.ones(2, device="cuda"),
                      torch.zeros(3, 16, dtype=I8, device="cuda"), torch.ones(3, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.quant_i8(torch.zeros(2, 24, device="cuda"))            # columns not a multiple of 16


def block(x_res, y, c, moe_args, i8w):
    """Norm step -> MoE layer -> norm step -> dense FFN -> norm step with int8 codes -> int8 product."""
    r, x = moe.norm(y, x_res, post_w=c["post_w"], gate=c["gate"], gate_div=c["gate_div"], pre_w=c["pre_w"])
    wr, routed, shared, bank = moe_args
    m = moe.layer(x, wr, None, 2, "sigmoid", routed, shared, out_dtype=BF)
    r, x = moe.norm(m, r, gate=c["gate"], gate_div=c["gate_div"], pre_w=c["pre_w"])
    f = moe.ffn(x, bank)
    r, (q, s) = moe.norm(f, r, pre_w=c["pre_w"], x_dtype=I8)
    return r, moe.linear_i8(q, s, *i8w, out_dtype=F32)


def block_setup(T=40, H=256, I=128, E=8):
    g = torch.Generator().manual_seed(77)
    c = norm_case(T, H, 9, gate_div=16)
    mk = lambda n, a, b: (torch.randn(n, a, b, generator=g) * 0.05).to(BF).cuda()
    routed = moe.Experts(mk(E, I, H), mk(E, I, H), mk(E, H, I))
    shared = moe.Experts(mk(1, I, H), mk(1, I, H), mk(1, H, I))
    bank = moe.Experts(mk(1, 264, H), mk(1, 264, H), mk(1, H, 264))
    wr = (torch.randn(H, E, generator=g) / 16).cuda()
    i8w = (torch.randint(-127, 128, (100, H), generator=g).to(I8).cuda(), torch.rand(100, generator=g).cuda() * 1e-3)
    return c, (wr, routed, shared, bank), i8w


def test_block_of_them_together():
    c, args, i8w = block_setup()
    r, out = block(c["res"], c["y"], c, args, i8w)
    # the same from the parts' own plain forms in 64 bits, on the parts' stored inputs
    d = dict(c)
    rr, xx, _, _ = norm_ref(d, a=1.0)
    wr, routed, shared, bank = args
    x = xx.to(BF)
    logits = x.double() @ wr.double()
    top = logits.topk(2, dim=1)
    w = torch.sigmoid(top.values)
    w = w / w.sum(1, keepdim=True)

    def swiglu(v, b, e):
        wg, wu, wd = (t[e].double() for t in (b.w_gate, b.w_up, b.w_down))
        g = v @ wg.t()
        return (g * torch.sigmoid(g) * (v @ wu.t())) @ wd.t()
    every = torch.stack([swiglu(x.double(), routed, e) for e in range(8)], 1)
    m = swiglu(x.double(), shared, 0) + (every.gather(1, top.indices[..., None].expand(-1, -1, 256)) * w[..., None]).sum(1)
    rr, xx, _, _ = norm_ref(dict(c, y=m.to(BF), res=rr.to(BF), post_w=None), a=1.0)
    f = swiglu(xx.to(BF).double(), bank, 0)
    rr, xx, _, _ = norm_ref(dict(c, y=f.to(BF), res=rr.to(BF), post_w=None, gate=None), a=1.0)
    ref = (xx @ i8w[0].double().t()) * i8w[1].double()
    # several bf16 roundings in a row (2^-8 each) and the int8 step (at most half of amax / 127 an element)
    assert (r.double() - rr).norm() / rr.norm() <= 6 * 2.0 ** -8
    assert (out.double() - ref).norm() / ref.norm() <= 6 * 2.0 ** -8 + xx.abs().max(1).values.max() / 254 / xx.abs().mean()


def test_captured_and_replayed():
    c, args, i8w = block_setup()
    f = Ffn(40, 256, 264, 4)

    def step(y, dy):
        r, out = block(c["res"], y, c, args, i8w)
        yy, gu = moe.ffn(f.x, f.bank, want_gu=True)
        g = moe.ffn_backward(dy, f.x, f.bank, gu)
        n = moe.norm_backward(c["dx"], c["dr"], y, c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=16,
                              pre_w=c["pre_w"])
        return [r, out, yy, *g, *n.values()]
    y, dy = c["y"].clone(), f.dy.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(y, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(y, dy)
    for k in range(3):
        y.copy_(c["y"] * (1 + k))
        dy.copy_(f.dy * (2 - k))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step(y, dy)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_on_a_stream_of_its_own():
    f = Ffn(300, 512, 264, 5)
    want = moe.ffn(f.x, f.bank, want_gu=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [moe.ffn(f.x, f.bank, want_gu=True, stream=s) for s in streams for _ in range(3)]   # two streams at once
    grads = [moe.ffn_backward(f.dy, f.x, f.bank, g[1], stream=streams[k // 3]) for k, g in enumerate(got)]
    torch.cuda.synchronize()
    ref = moe.ffn_backward(f.dy, f.x, f.bank, want[1])
    for g, d in zip(got, grads):
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
        assert all(torch.equal(a, b) for a, b in zip(d, ref))


def test_runs_are_bitwise_equal():
    f = Ffn(700, 1032, 520, 6)
    c = norm_case(900, 1032, 10, gate_div=70)
    _, gu = moe.ffn(f.x, f.bank, want_gu=True)

    def both():
        n = moe.norm_backward(c["dx"], c["dr"], c["y"], c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=70,
                              pre_w=c["pre_w"])
        return [moe.ffn(f.x, f.bank), *moe.ffn_backward(f.dy, f.x, f.bank, gu), *n.values()]
    a, b = both(), both()
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("T,H,off", [(3, 1001, 0), (2, 264, 1), (70, 33, 0), (2, 9000, 0)])
def test_norm_int8_rows_of_any_width(T, H, off):
    c = norm_case(T, H, 11, gate_div=2, off=off)
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=2, res_scale=0.75, pre_w=c["pre_w"])
    q, gq = outbuf((T, H), I8)
    s, gs = outbuf((T,), F32)
    moe.norm(c["y"], c["res"], x=(q, s), **kw)
    _, x32 = moe.norm(c["y"], c["res"], x_dtype=F32, **kw)
    rq, rs = codes_of(x32)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    gq()
    gs()


def test_norm_gradients_in_place():
    """dres over dr and dy over dx, as the boundary allows for dres: every element is read before it is written."""
    c = norm_case(70, 520, 12, gate_div=9)
    want = check_norm_grads(c)
    L, p = moe.lib(), lambda t: t.data_ptr()
    dr = c["dr"].clone()
    dy = torch.empty_like(c["y"])
    ws = torch.empty(L.moe_norm_backward_workspace_size(70, 520, 9), dtype=torch.uint8, device="cuda")
    st = L.moe_norm_backward(p(c["dx"]), 1, p(dr), p(c["y"]), 1, p(c["res"]), 1, 70, 520, p(c["post_w"]), p(c["gate"]), 9,
                             p(c["pre_w"]), 0, 0.75, 1e-6, p(dy), p(dr), None, None, None, p(ws), ws.numel(),
                             torch.cuda.current_stream().cuda_stream)
    assert st == moe.MOE_OK
    assert torch.equal(dr, want["dres"]) and torch.equal(dy, want["dy"])


def test_one_bad_token_stays_alone():
    """Inf and NaN in one token's row reach no other token's output."""
    c = Ffn(70, 264, 136, 7)
    good = moe.ffn(c.x, c.bank)
    x = c.x.clone()
    x[33] = float("inf")
    x[33, 5] = float("nan")
    y = moe.ffn(x, c.bank)
    keep = torch.arange(70, device="cuda") != 33
    assert torch.equal(y[keep], good[keep])
    n = norm_case(9, 264, 13, gate_div=3)
    r0, x0 = moe.norm(n["y"], n["res"], post_w=n["post_w"], gate=n["gate"], gate_div=3, pre_w=n["pre_w"])
    yy = n["y"].clone()
    yy[4] = float("nan")
    r1, x1 = moe.norm(yy, n["res"], post_w=n["post_w"], gate=n["gate"], gate_div=3, pre_w=n["pre_w"])
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(r0[keep], r1[keep]) and torch.equal(x0[keep], x1[keep])


def test_two_graphs_with_one_workspace():
    """Two captured calls that were given the same workspace, replayed in turn on one stream."""
    a, b = Ffn(300, 264, 136, 8), Ffn(70, 520, 264, 9)
    L = moe.lib()
    ws = torch.empty(max(L.moe_ffn_workspace_size(300, 264, 136), L.moe_ffn_workspace_size(70, 520, 264)), dtype=torch.uint8,
                     device="cuda")
    want = [moe.ffn(c.x, c.bank) for c in (a, b)]
    graphs, outs = [], []
    for c in (a, b):
        out = torch.empty_like(c.x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.ffn(c.x, c.bank, out=out, ws=ws)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("T,H,I", [(20, 264, 72), (64, 512, 2504), (300, 264, 1000), (70, 1024, 2056), (600, 1032, 1144)])
def test_ffn_dx_with_ragged_halves(T, H, I):
    """dx sums over the gate's and the up's columns, whose last stages are not whole; alone it is split along k."""
    c = Ffn(T, H, I, 11)
    _, gu = moe.ffn(c.x, c.bank, want_gu=True)
    c.check_grads(moe.ffn_backward(c.dy, c.x, c.bank, gu, need=("dx",)))
    c.check_grads(moe.ffn_backward(c.dy, c.x, c.bank, gu, need=("dx", "dw_up")))


@pytest.mark.parametrize("T,H,gate_div", [(4100, 72, 4100), (9000, 40, 7), (16500, 16, 300), (33000, 8, 33000)])
def test_norm_backward_of_many_short_rows(T, H, gate_div):
    """More and longer runs of rows: the parameter gradients against 64 bits, twice the same."""
    c = norm_case(T, H, 5, gate_div=gate_div)
    r, _ = moe.norm(c["y"], c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=gate_div, pre_w=c["pre_w"], want_x=False)
    call = lambda: moe.norm_backward(c["dx"], c["dr"], c["y"], r, post_w=c["post_w"], gate=c["gate"], gate_div=gate_div,
                                     pre_w=c["pre_w"])
    one, two = call(), call()
    assert all(torch.equal(one[k], two[k]) for k in one)
    y, rr, dx, dr = (t.double() for t in (c["y"], r, c["dx"], c["dr"]))
    gate = c["gate"].double().repeat_interleave(gate_div, 0)[:T]
    q = 1 / (rr.square().mean(1, keepdim=True) + 1e-6).sqrt()
    p = 1 / (y.square().mean(1, keepdim=True) + 1e-6).sqrt()
    g = dx * c["pre_w"].double()
    d = dr + q * (g - rr * q * (g * rr * q).mean(1, keepdim=True))
    # every term of a sum over the rows is off by its own few roundings (those of the row's
    # sums, the root and the products: 40 at these widths), relative to the sizes of d's parts;
    # the sums over the rows (runs of at most 64, then slices of the runs) by gamma of their depth
    size = dr.abs() + q * (g.abs() + (rr * q).abs() * (g * rr * q).abs().mean(1, keepdim=True))
    rel = 40 * 2.0 ** -24 + gamma(64 + 2048)
    for name, ref, terms in (("dpre_w", (dx * rr * q).sum(0), (dx * rr * q).abs().sum(0)),
                             ("dpost_w", (gate * d * y * p).sum(0), (gate.abs() * size * (y * p).abs()).sum(0))):
        within(one[name], ref, rel * terms, name)
    n = y * p * c["post_w"].double()
    which = torch.arange(T, device="cuda") // gate_div
    G = c["gate"].shape[0]
    ref = torch.zeros(G, H, dtype=torch.float64, device="cuda").index_add_(0, which, d * n)
    bound = torch.zeros(G, H, dtype=torch.float64, device="cuda").index_add_(0, which, size * n.abs())
    within(one["dgate"], ref, rel * bound, "dgate")


def test_workspace_in_pieces_is_refused():
    """A workspace whose elements are not one piece of memory: more bytes than it has would be written."""
    c = Ffn(40, 64, 64, 4)
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20),
               torch.empty(1 << 11, 1 << 10, dtype=torch.uint8, device="cuda")[:, :1 << 9]):
        with pytest.raises(ValueError, match="contiguous"):
            moe.ffn(c.x, c.bank, ws=ws)
        with pytest.raises(ValueError, match="contiguous"):
            moe.ffn_backward(c.dy, c.x, c.bank, ws=ws)


def test_quant_i8_of_more_rows_than_a_grid_holds():
    rows, cols = (1 << 24) + 3, 16
    x = (torch.arange(rows, device="cuda", dtype=torch.int32)[:, None] % 251 - 125).to(BF) * torch.ones(cols, dtype=BF, device="cuda")
    x[:, 0] = 127
    q, s = moe.quant_i8(x)
    assert bool((s == 1).all())
    assert torch.equal(q[:, 0], torch.full((rows,), 127, dtype=torch.int8, device="cuda"))
    assert torch.equal(q[:, 15].to(torch.int32), torch.arange(rows, device="cuda", dtype=torch.int32) % 251 - 125)


@pytest.mark.parametrize("T,H", [(1, 1024), (5, 520), (131, 1001), (700, 768), (9, 1023)])
@pytest.mark.parametrize("y,r,w", [(BF, BF, F32), (F32, F32, BF)])
def test_norm_of_medium_rows(T, H, y, r, w):
    """Rows of two waves: both directions against the 64-bit form, with a gate that ends inside a run."""
    c = norm_case(T, H, 7, y=y, r=r, w=w, gate_div=3)
    ref_r, ref_x, er, ex = norm_ref(c)
    got_r, got_x = moe.norm(c["y"], c["res"], post_w=c["post_w"], gate=c["gate"], gate_div=3, res_scale=0.75,
                            pre_w=c["pre_w"], x_dtype=F32)
    within(got_r, ref_r, er + HALF[r] * (ref_r.abs() + er), "r")
    within(got_x, ref_x, ex + HALF[F32] * (ref_x.abs() + ex), "x")


@pytest.mark.parametrize("T,H", [(1, 2056), (37, 2560), (1100, 4096), (300, 4095), (3, 2049)])
@pytest.mark.parametrize("y,r,w", [(BF, BF, F32), (F32, F32, BF), (BF, F32, F32)])
def test_norm_of_rows_of_two_chunks(T, H, y, r, w):
    """Rows that a thread holds in two chunks, with runs of more than one row."""
    c = norm_case(T, H, 8, y=y, r=r, w=w, gate_div=5)
    ref_r, ref_x, er, ex = norm_ref(c)
    kw = dict(post_w=c["post_w"], gate=c["gate"], gate_div=5, res_scale=0.75, pre_w=c["pre_w"])
    got_r, got_x = moe.norm(c["y"], c["res"], x_dtype=F32, **kw)
    within(got_r, ref_r, er + HALF[r] * (ref_r.abs() + er), "r")
    within(got_x, ref_x, ex + HALF[F32] * (ref_x.abs() + ex), "x")
    _, (q, s) = moe.norm(c["y"], c["res"], x_dtype=torch.int8, **kw)
    off = (q.double() * s.double()[:, None] - ref_x).abs()   # half a step, and x's own error
    assert bool((off <= 0.5 * s.double()[:, None] * (1 + 2.0 ** -16) + 2 * ex).all())
