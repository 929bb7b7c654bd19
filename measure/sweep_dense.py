"""Times of the operators around the MoE layer over sizes.

Each line is one call of an entry point (or the quantisation alone) at one
size: the mean over a captured graph of calls that take inputs and weights in
turn from sets of more than 600 MB together, so that they come from HBM and not
from the 256 MB cache, the least of three replays.  GB/s counts each input read
once and each output written once, TFLOP/s the products' operations.

    python -m measure.sweep_dense [--only ffn grad norm norm_grad i8] [--out FILE]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import routed_expert_ffn_04_amd as moe  # noqa: E402

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
SETS_BYTES = 600 << 20

FFN = ([(T, 7168, 2048) for T in (1, 4, 16, 17, 64, 128, 256, 512, 1024, 2048, 4096, 16384)]
       + [(T, H, I) for H, I in ((1024, 512), (2048, 1408), (4096, 1024)) for T in (1, 16, 17)]
       + [(64, 256, 512), (515, 2056, 1336), (1024, 2048, 1024)])
GRAD = [(64, 256, 512), (515, 2056, 1336), (1024, 2048, 1024), (4096, 2048, 1024)] + [(T, 7168, 2048) for T in (64, 512, 2048, 4096)]
# T, H, y, r and x (in the gradients dx), rows of a gate
NORM = [(128, 7168, BF, BF, 128), (4096, 7168, BF, BF, 4096), (16384, 7168, BF, F32, 512), (16384, 1024, BF, BF, 16384),
        (8192, 2560, BF, BF, 8192), (2048, 16384, BF, BF, 2048)]
NORM_GRAD = [(777, 1001, F32, F32, 37), (5000, 2003, F32, F32, 37), (2048, 512, BF, BF, 2048), (8192, 256, BF, BF, 8192),
             (16384, 512, BF, BF, 16384), (65536, 128, BF, BF, 65536), (16384, 1024, BF, BF, 16384), (4096, 7168, BF, BF, 4096),
             (2048, 16384, BF, BF, 2048)]
LINEAR = [(T, 7168, 4096) for T in (1, 16, 17, 64, 512, 1024, 8192)] + [(333, 2064, 1501)]
QUANT = [(128, 7168), (333, 2064), (8192, 7168), (16384, 4096)]
NORM_I8 = [(16, 7168), (8192, 7168), (16384, 4096)]


def graph_us(call, sets: int) -> float:
    n = max(12, 2 * sets)
    for i in range(sets):
        call(i)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(n):
            call(i % sets)
    g.replay()
    best = float("inf")
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


def sets_of(nbytes: int) -> int:
    return max(3, min(200, SETS_BYTES // nbytes + 1))


def normal(shape, dtype, scale=1.0):
    return torch.randn(shape, device="cuda").mul_(scale).to(dtype)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--only", nargs="*", default=["ffn", "grad", "norm", "norm_grad", "i8"])
    ap.add_argument("--out", default=None, help="also write the table to this file")
    args = ap.parse_args()
    moe.lib()
    lines = []

    def say(line):
        lines.append(line)
        print(line, flush=True)

    def point(what, size, call, sets, nbytes, flops=0):
        us = graph_us(call, sets)
        say(f"{what:<28} {size:<24} {us:>9.2f} {nbytes / us * 1e-3:>8.0f} {flops / us * 1e-6 if flops else 0:>8.1f}")

    say(f"# operators around the MoE layer, weights from HBM, one graph of calls (python -m measure.sweep_dense {' '.join(sys.argv[1:])})")
    say(f"{'call':<28} {'size':<24} {'us':>9} {'GB/s':>8} {'TFLOP/s':>8}")

    def bank(H, I):
        return moe.Experts(normal((1, I, H), BF, 0.02), normal((1, I, H), BF, 0.02), normal((1, H, I), BF, 0.02))

    for name, sizes in (("ffn", FFN), ("grad", GRAD)):
        for T, H, I in sizes if name in args.only else ():
            n = sets_of(6 * H * I + 2 * T * H)
            s = [(normal((T, H), BF), bank(H, I), normal((T, H), BF)) for _ in range(n)]
            if name == "ffn":
                point("ffn", f"{T} x {H} x {I}", lambda i: moe.ffn(s[i][0], s[i][1]), n, 6 * H * I + 4 * T * H, 6 * T * H * I)
            else:
                gu = [moe.ffn(x, b, want_gu=True)[1] for x, b, _ in s]
                point("ffn_backward", f"{T} x {H} x {I}", lambda i: moe.ffn_backward(s[i][2], s[i][0], s[i][1], gu[i]), n,
                      12 * H * I + 6 * T * H + 8 * T * I, 12 * T * H * I)
                del gu
            del s
    kind = lambda t: "f32" if t is F32 else "bf16"
    for name, sizes in (("norm", NORM), ("norm_grad", NORM_GRAD)):
        for T, H, y, r, div in sizes if name in args.only else ():
            w, gate = normal((H,), F32), normal((-(-T // div), H), F32)
            kw = dict(post_w=w, gate=gate, gate_div=div, pre_w=w)
            row = T * H
            if name == "norm":
                nbytes = row * (2 * y.itemsize + 2 * r.itemsize)
                n = sets_of(nbytes)
                s = [(normal((T, H), y), normal((T, H), r)) for _ in range(n)]
                point(f"norm {kind(y)}, r {kind(r)}", f"{T} x {H}", lambda i: moe.norm(*s[i], **kw), n, nbytes)
            else:
                nbytes = row * (3 * y.itemsize + 3 * r.itemsize)
                n = sets_of(nbytes)
                s = [(normal((T, H), y), normal((T, H), r), normal((T, H), y), normal((T, H), r)) for _ in range(n)]
                point(f"norm_backward {kind(y)}, r {kind(r)}", f"{T} x {H}", lambda i: moe.norm_backward(*s[i], **kw), n, nbytes)
            del s
    if "i8" in args.only:
        for T, K, N in LINEAR:
            n = sets_of(N * K + T * K)
            s = [tuple(torch.randint(-127, 128, m, dtype=I8, device="cuda") for m in ((T, K), (N, K))) for _ in range(n)]
            a, b = normal((T,), F32), normal((N,), F32)
            point("linear_i8", f"{T} x {K} x {N}", lambda i: moe.linear_i8(s[i][0], a, s[i][1], b), n,
                  N * K + T * K + 2 * T * N, 2 * T * K * N)
            del s
        for T, H in QUANT:
            n = sets_of(2 * T * H)
            s = [normal((T, H), BF) for _ in range(n)]
            point("quant_i8 bf16", f"{T} x {H}", lambda i: moe.quant_i8(s[i]), n, 3 * T * H)
            del s
        for T, H in NORM_I8:
            n = sets_of(4 * T * H)
            s = [(normal((T, H), BF), normal((T, H), BF)) for _ in range(n)]
            w = normal((H,), F32)
            point("norm to int8, bf16", f"{T} x {H}", lambda i: moe.norm(*s[i], pre_w=w, x_dtype=I8), n, 7 * T * H)
            del s
    if args.out:
        with open(args.out, "w") as f:
            f.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    main()
