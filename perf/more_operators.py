"""The operators of a training step of the mixture-of-experts layer as cases to measure.

Four groups of calls, each in two forms: `own` False computes the plain form
from elementary torch operations in 32 bits, `own` True makes the library's
calls.

  dispatch      rows of the tokens sorted by expert, xs[dest[t k + j]] = x[t], and the gradient of that,
                dx[t] = sum_j dxs[dest[t k + j]]
  combine_grad  gradients of out[t] = sum_j w[t, j] y[dest[t k + j]]: dy and dw
  experts       the experts' gated FFN on their sorted rows and the gradients of rows and weights;
                what the backward pass needs of the forward one kept in fp32, or in blocks of 16
                columns with 8-bit codes and a shared exponent (rows and pre-activations)
  ffn_ckpt      the dense gated FFN with its gradients from such 8-bit checkpoints

H = 7168, I = 2048, 256 experts and 8 per token are the sizes of the large
layer, 32 experts an eighth of it; T = 64, H = 256, 8 experts and 2 per token
those of the tiny one.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16   # columns that share an exponent


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the tiny workload's layer in fp32: launches count
        {"name": "dispatch_tiny", "op": "dispatch", "T": 64, "k": 2, "E": 8, "H": 256, "x": "f32"},
        # a backward pass that makes the sorted rows again from an 8-bit checkpoint of the tokens
        {"name": "dispatch_ckpt", "op": "dispatch", "T": 4096, "k": 8, "E": 256, "H": 7168, "x": "i8"},
        # the large layer on a full batch
        {"name": "dispatch_large", "op": "dispatch", "T": 16384, "k": 8, "E": 256, "H": 7168, "x": "bf16"},
        # a small batch of the large layer
        {"name": "combine_grad_small", "op": "combine_grad", "T": 128, "k": 8, "E": 256, "H": 7168, "d": "bf16", "y": "bf16"},
        # rows of an odd width, an odd number of tokens and of experts, all in fp32
        {"name": "combine_grad_ragged", "op": "combine_grad", "T": 5003, "k": 6, "E": 61, "H": 2056, "d": "f32", "y": "f32"},
        # expert outputs that came back in fp8
        {"name": "combine_grad_fp8", "op": "combine_grad", "T": 8192, "k": 8, "E": 256, "H": 7168, "d": "bf16", "y": "e4m3"},
        # the tiny workload's layer, one training step
        {"name": "experts_tiny", "op": "experts", "R": 128, "E": 8, "H": 256, "I": 512, "skew": 0.0, "save": "f32"},
        # many small experts, few rows, some experts without any
        {"name": "experts_few", "op": "experts", "R": 777, "E": 64, "H": 2048, "I": 1408, "skew": 1.2, "save": "i8"},
        # the nine experts of one GPU of an expert-parallel group, each with its own number of rows
        {"name": "experts_share", "op": "experts", "R": 19663, "E": 9, "H": 7168, "I": 2048, "skew": 0.5, "save": "f32"},
        # an eighth of the large layer, a micro-batch, checkpoints in 8 bits
        {"name": "experts_step", "op": "experts", "R": 16384, "E": 32, "H": 7168, "I": 2048, "skew": 0.3, "save": "i8"},
        # a ragged batch of a small model
        {"name": "ffn_ckpt_ragged", "op": "ffn_ckpt", "T": 515, "H": 2056, "I": 1336},
        # the large layer's shared expert on a training micro-batch
        {"name": "ffn_ckpt_step", "op": "ffn_ckpt", "T": 4096, "H": 7168, "I": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine_grad", "experts", "experts", "ffn_ckpt"])
    if op in ("dispatch", "combine_grad"):
        k = rng.randint(1, 8)
        c = {"op": op, "T": _log(rng, 1, 16384), "k": k, "E": _log(rng, max(k, 4), 256), "H": 8 * _log(rng, 16, 896)}
        if op == "dispatch":
            return {**c, "x": rng.choice(["bf16", "bf16", "f32", "i8"])}
        y = rng.choice(["bf16", "bf16", "f32", "e4m3"])
        if y == "e4m3":   # scales are held for 128 columns
            c["H"] = 128 * rng.randint(1, 56)
        return {**c, "d": "f32" if y == "f32" else "bf16", "y": y}
    if op == "ffn_ckpt":
        return {"op": op, "T": _log(rng, 1, 4096), "H": 8 * _log(rng, 16, 896), "I": 8 * _log(rng, 16, 256)}
    H, I = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 256)
    E = _log(rng, 1, min(64, 32 * 7168 * 2048 // (H * I)))
    return {"op": op, "R": _log(rng, 1, 16384), "E": E, "H": H, "I": I, "skew": rng.choice([0.0, 0.4, 1.2]),
            "save": rng.choice(["f32", "i8"])}


# ---------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, scale, dtype):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=g).to(dtype)


def _rows_of(case, seed):
    """Rows of each expert: one draw of R rows over experts of falling popularity, in random order."""
    r = np.random.RandomState(seed % (1 << 32))
    p = np.arange(1, case["E"] + 1, dtype=np.float64) ** -case["skew"]
    return r.multinomial(case["R"], r.permutation(p / p.sum()))


def _sorted(s, g, case):
    """A token's k experts, all different, and the sorted order of the assignments."""
    T, k, E = case["T"], case["k"], case["E"]
    ids = torch.rand((T, E), device="cuda", generator=g).topk(k, dim=1).indices.reshape(-1)
    src = torch.sort(ids, stable=True).indices
    dest = torch.empty_like(src)
    dest[src] = torch.arange(T * k, device="cuda")
    s["src"], s["dest"] = src.to(torch.int32), dest.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    bf = torch.bfloat16
    if op == "dispatch":
        T, R, H = case["T"], case["T"] * case["k"], case["H"]
        _sorted(s, g, case)
        s["x"] = _normal(g, (T, H), 1.0, _DT[case["x"]])      # rows come out of a norm
        if case["x"] == "i8":
            s["x"] = _plain_i8(s["x"].float())                # the checkpoint that is in hand
        s["dxs"] = _normal(g, (R, H), 1.0, _DT[case["x"]])
    elif op == "combine_grad":
        T, R, H = case["T"], case["T"] * case["k"], case["H"]
        _sorted(s, g, case)
        s["dout"] = _normal(g, (T, H), 1.0, _DT[case["d"]])
        w = torch.rand((T, case["k"]), device="cuda", generator=g) + 0.05
        s["w"] = w / w.sum(dim=1, keepdim=True)
        s["y_scale"] = None
        if case["y"] == "e4m3":
            s["y"] = _normal(g, (R, H), 100.0, torch.float32).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s["y_scale"] = torch.empty((R, H // 128), device="cuda").uniform_(0.002, 0.02, generator=g)
        else:
            s["y"] = _normal(g, (R, H), 1.0, _DT[case["y"]])
    else:
        H, I = case["H"], case["I"]
        E, R = (case["E"], case["R"]) if op == "experts" else (1, case["T"])
        s["x"] = _normal(g, (R, H), 1.0, bf)
        s["w_gate"] = _normal(g, (E, I, H), 0.02, bf)
        s["w_up"] = _normal(g, (E, I, H), 0.02, bf)
        s["w_down"] = _normal(g, (E, H, I), 0.02, bf)
        s["dy"] = _normal(g, (R, H), 1.0, bf)
        if op == "experts":
            n = _rows_of(case, seed)
            s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
            s["most"] = int(n.max())
    return s


# ---------------------------------------------------------------- plain forms (32 bits, rounded once at the end)

def _plain_i8(v):
    """(codes [rows][cols] int8, exponents [rows][blocks] uint8) of the blocks of 16 columns."""
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    p = torch.zeros((rows, nb * BLOCK), dtype=torch.float32, device=v.device)
    p[:, :cols] = v
    p = p.view(rows, nb, BLOCK)
    top = torch.frexp(p.abs().amax(dim=2)).exponent - 1      # floor(log2)
    e = torch.where((p != 0).any(dim=2), top - 6 + 127, torch.ones_like(top)).clamp(min=1)
    code = torch.round(torch.ldexp(p, 127 - e.unsqueeze(2))).clamp(-127, 127).to(torch.int8)
    return code.view(rows, -1)[:, :cols].contiguous(), e.to(torch.uint8)


def _plain_value(q):
    code, e = q
    cols = code.shape[1]
    return torch.ldexp(code.float(), e.to(torch.int32).repeat_interleave(BLOCK, dim=1)[:, :cols] - 127)


def _held(v):
    return _plain_value(_plain_i8(v))


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _plain_dispatch(s):
    c = s["case"]
    x = _plain_value(s["x"]) if c["x"] == "i8" else s["x"].float()
    dx = s["dxs"].float()[s["dest"].long()].view(c["T"], c["k"], c["H"]).sum(dim=1)
    return {"xs": x[s["src"].long() // c["k"]].to(_DT[c["x"]]), "dx": dx.to(_DT[c["x"]])}


def _plain_combine_grad(s):
    c = s["case"]
    T, k, H = c["T"], c["k"], c["H"]
    dout, src = s["dout"].float(), s["src"].long()
    if c["y"] == "e4m3":
        y = s["y"].view(torch.float8_e4m3fn).float() * s["y_scale"].repeat_interleave(128, dim=1)
    else:
        y = s["y"].float()
    dy = dout[src // k] * s["w"].view(-1)[src].unsqueeze(1)
    dw = (y[s["dest"].long()].view(T, k, H) * dout.unsqueeze(1)).sum(dim=2)
    return {"dy": dy.to(_DT[c["d"]]), "dw": dw}


def _plain_grads(x, held_x, wg, wu, wd, dy, held):
    """Products of a batch of experts, rows padded with zeros: y, dx and the weights' gradients."""
    g, u = torch.matmul(x, wg.transpose(1, 2)), torch.matmul(x, wu.transpose(1, 2))
    y = torch.matmul(g * _sigmoid(g) * u, wd.transpose(1, 2))
    g, u = held(g), held(u)
    sg = _sigmoid(g)
    a = g * sg
    dh = torch.matmul(dy, wd)
    dg = dh * u * sg * (1.0 + g * (1.0 - sg))
    du = dh * a
    return {"y": y, "dx": torch.matmul(dg, wg) + torch.matmul(du, wu), "dw_gate": torch.matmul(dg.transpose(1, 2), held_x),
            "dw_up": torch.matmul(du.transpose(1, 2), held_x), "dw_down": torch.matmul(dy.transpose(1, 2), a * u)}


def _plain_experts(s):
    c = s["case"]
    bf = torch.bfloat16
    x, dy = s["x"].float(), s["dy"].float()
    wg, wu, wd = (s[k].float() for k in ("w_gate", "w_up", "w_down"))
    i8 = c["op"] == "ffn_ckpt" or c["save"] == "i8"
    held_x = _held(x) if i8 else x

    def held(v):
        return _held(v.reshape(-1, v.shape[2])).view(v.shape) if i8 else v

    if c["op"] == "ffn_ckpt":
        out = _plain_grads(x[None], held_x[None], wg, wu, wd, dy[None], held)
        return {k: (v[0] if k in ("y", "dx") else v).to(bf) for k, v in out.items()}
    E, R, n = c["E"], c["R"], max(s["most"], 1)
    row = torch.arange(R, device=x.device)
    off = s["offsets"].long()
    expert = torch.searchsorted(off[1:].contiguous(), row, right=True)
    at = expert * n + row - off[expert]

    def padded(v):
        p = torch.zeros((E * n, v.shape[1]), dtype=torch.float32, device=v.device)
        p[at] = v
        return p.view(E, n, -1)

    out = _plain_grads(padded(x), padded(held_x), wg, wu, wd, padded(dy), held)
    return {k: (v.view(E * n, -1)[at] if k in ("y", "dx") else v).to(bf) for k, v in out.items()}


# ---------------------------------------------------------------- one pass

def _moe():
    import routed_expert_ffn_04_amd as moe
    return moe


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if op == "dispatch":
        if own:
            moe = _moe()
            return {"xs": moe.dispatch(s["x"], s["dest"], c["k"]), "dx": moe.dispatch_backward(s["dxs"], s["dest"], c["k"])}
        return _plain_dispatch(s)
    if op == "combine_grad":
        if own:
            dy, dw = _moe().combine_backward(s["dout"], s["y"], s["dest"], s["w"], y_scale=s["y_scale"])
            return {"dy": dy, "dw": dw}
        return _plain_combine_grad(s)
    if own:
        moe = _moe()
        bank = moe.Experts(s["w_gate"], s["w_up"], s["w_down"])
        i8 = op == "ffn_ckpt" or c["save"] == "i8"
        kept = torch.int8 if i8 else torch.float32
        if op == "ffn_ckpt":
            y, gu = moe.ffn(s["x"], bank, want_gu=True, gu_dtype=kept)
        else:
            y, gu = moe.experts_ffn(s["x"], s["offsets"], bank, want_gu=True, gu_dtype=kept)
        x = moe.quant_i8x16(s["x"]) if i8 else s["x"]
        if op == "ffn_ckpt":
            grads = moe.ffn_backward(s["dy"], x, bank, gu)
        else:
            grads = moe.experts_ffn_backward(s["dy"], x, s["offsets"], bank, gu)
        return {"y": y, **dict(zip(("dx", "dw_gate", "dw_up", "dw_down"), grads))}
    return _plain_experts(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    e = {"bf16": 2, "f32": 4, "i8": 1 + 1 / BLOCK, "e4m3": 1 + 4 / 128}
    if op in ("dispatch", "combine_grad"):
        T, k, H = case["T"], case["k"], case["H"]
        R = T * k
        if op == "dispatch":
            rows = 2 if case["x"] == "i8" else e[case["x"]]
            # x and dxs read, xs and dx written, the order read twice
            return {"bytes": int(T * H * (e[case["x"]] + rows) + 2 * R * H * rows + 8 * R), "flops": R * H}
        # dout and y read, dy written; the order, w and dw
        return {"bytes": int((T + R) * H * e[case["d"]] + R * H * e[case["y"]] + 12 * R), "flops": 3 * R * H}
    H, I = case["H"], case["I"]
    E, R = (case["E"], case["R"]) if op == "experts" else (1, case["T"])
    # weights of the experts that have rows read, all gradients written; x and dy read, y and dx written
    return {"bytes": 6 * (min(E, R) + E) * H * I + 8 * R * H, "flops": 18 * R * H * I}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_held(v):
    """v as blocks of 16 columns hold it: multiples of 2^(floor(log2 max) - 6), at most 127 of them."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    full = cols // BLOCK * BLOCK
    for lo, hi in ((0, full), (full, cols)):
        if lo == hi or rows == 0:
            continue
        b = v[:, lo:hi].reshape(rows, -1, min(BLOCK, hi - lo))
        big = b.abs().max(2, keepdim=True).values
        power = torch.floor(torch.log2(torch.where(big > 0, big, torch.ones_like(big))))
        step = torch.exp2(torch.clamp(power - 6, min=-126))
        out[:, lo:hi] = (torch.round(b / step).clamp(-127, 127) * step).reshape(rows, -1)
    return out


def _exact_ffn(x, kept_x, wg, wu, wd, dy, i8):
    g, u = x @ wg.T, x @ wu.T
    sig = torch.sigmoid(g)
    y = (g * sig * u) @ wd.T
    if i8:
        # held as the fp32 value that is formed rounds
        g, u = _exact_held(g.float().double()), _exact_held(u.float().double())
        sig = torch.sigmoid(g)
    dh = dy @ wd
    dg = dh * u * (sig + g * sig * (1.0 - sig))
    du = dh * g * sig
    return y, dg @ wg + du @ wu, dg.T @ kept_x, du.T @ kept_x, dy.T @ (g * sig * u)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        if case["x"] == "i8":
            code, e = s["x"]
            step = torch.exp2(e.double() - 127.0)
            x = code.double() * step.unsqueeze(2).expand(-1, -1, BLOCK).reshape(case["T"], -1)[:, :case["H"]]
        else:
            x = s["x"].double()
        token = torch.div(s["src"], case["k"], rounding_mode="floor").long()
        dx = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        return {"xs": x.index_select(0, token), "dx": dx.index_add_(0, token, s["dxs"].double())}
    if op == "combine_grad":
        token = torch.div(s["src"], case["k"], rounding_mode="floor").long()
        d = s["dout"].double().index_select(0, token)
        if case["y"] == "e4m3":
            y = s["y"].view(torch.float8_e4m3fn).double().view(d.shape[0], -1, 128) * s["y_scale"].double().unsqueeze(2)
            y = y.view(d.shape)
        else:
            y = s["y"].double()
        dw = torch.empty(d.shape[0], dtype=torch.float64, device="cuda")
        dw[s["src"].long()] = y.mul_(d).sum(1)
        return {"dy": d.mul_(s["w"].double().flatten()[s["src"].long()].unsqueeze(1)), "dw": dw.view(case["T"], case["k"])}
    x, dy = s["x"].double(), s["dy"].double()
    i8 = op == "ffn_ckpt" or case["save"] == "i8"
    kept = _exact_held(x) if i8 else x
    ends = [0, case["T"]] if op == "ffn_ckpt" else s["offsets"].tolist()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw = {k: torch.empty(s[k].shape, dtype=torch.float64, device="cuda") for k in ("w_gate", "w_up", "w_down")}
    for n, (a, b) in enumerate(zip(ends, ends[1:])):
        w = [s[k][n].double() for k in dw]
        y[a:b], dx[a:b], dw["w_gate"][n], dw["w_up"][n], dw["w_down"][n] = _exact_ffn(
            x[a:b], kept[a:b], *w, dy[a:b], i8)
    return {"y": y, "dx": dx, **{"d" + k: v for k, v in dw.items()}}
