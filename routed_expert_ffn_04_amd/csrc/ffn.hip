// Dense gated FFN block and its gradients in bf16 (moe_ffn, moe_ffn_backward; with
// checkpoints in 8 bits: moe_ffn_ckpt, moe_ffn_ckpt_backward).
//   g = x Wg^T, u = x Wu^T, h = silu(g) u, y = h Wd^T      (weights output-major)
// One kernel forms both projections of the same columns side by side, applies
// the activation and the product in its epilogue and writes h once.
// Backward, with the fp32 g and u that the forward pass saved:
//   dh = dy Wd        -> epilogue: dg = dh u s (1 + g (1 - s)), du = dh g s, h again   (s = sigmoid(g))
//   dx = [dg du] [Wg; Wu]       one product over 2 I
//   [dWg; dWu] = [dg du]^T x    one product with 2 I rows
//   dWd = dy^T h
// The matrices are met in the layout they have: products over the contiguous
// index read rows, the others read columns (gemm_tile.h), nothing is
// transposed in memory.
//
// Roundings: h, dg and du go into the next product as bf16 (nearest even), as
// the matrix cores take them; g and u are kept in fp32, because rounding them
// as well would put a second error of the same size on dx and the gate and up
// gradients.  All sums are fp32.
//
// Checkpoints in 8 bits (i8x16.h), where the caller asks for them: the gate/up epilogue
// writes the codes of g and u instead of their fp32 values, and that of dh reads them.  x
// is restored once for the weight gradients, whose tiles load straight into LDS: 16 us
// for 4096 x 7168, of 950 for the block forward and back (7168 x 2048).
#include <algorithm>
#include <utility>

#include "gemm_plan.h"

namespace moe {
using namespace gemm;

namespace {

constexpr int kKE = kStage / 2;

Operand rows(const void* p, long ld, int n, const void* p2 = nullptr) {
    return Operand{(const uint8_t*)p, (const uint8_t*)p2, (size_t)ld * 2, n};
}
Operand cols(const void* p, long ld, int n, const void* p2 = nullptr) {
    return Operand{(const uint8_t*)p, (const uint8_t*)p2, (size_t)ld * 2, n};
}

Args base(int M, int N, int K) {
    Args G{};
    G.M = M; G.N = N; G.K = K; G.vec = 1; G.msplit = M;
    return G;
}

size_t max2(size_t a, size_t b) { return a > b ? a : b; }

struct Forward {
    Plan gateup, down;
    size_t h, part, total;   // workspace
};
Plan gateup_plan(int T, int H, int I, bool tiles) { return plan_tiles(T, 2L * I, H, kKE, !tiles); }
// tiles: not the kernel for a few rows, whose waves hold eight gate columns, half of an i8x16 block
Forward forward(int T, int H, int I, bool tiles) {
    Forward f;
    f.gateup = gateup_plan(T, H, I, tiles);
    f.down = plan_tiles(T, H, I, kKE, true);
    f.h = 0;
    f.part = align256((size_t)T * I * 2);
    f.total = f.part + max2(part_bytes(f.gateup, T, 2L * I), part_bytes(f.down, T, H));
    if (!fits(f.gateup) || !fits(f.down)) f.total = kUnfit;
    return f;
}

// k of dx = dg Wg + du Wu: dg's, and du's from the next stage on
int turn_of(int I) { return (I + kKE - 1) / kKE * kKE; }

struct Backward {
    Plan gateup, dh, dx, dwgu, dw1, dwd;   // dw1: one of the gate and up gradients alone
    size_t gu, dgu, h, x, part, total;
};
Backward backward(int T, int H, int I, bool has_gu, bool x_i8) {
    Backward w;
    w.gateup = gateup_plan(T, H, I, false);
    w.dh = plan_tiles(T, I, H, kKE, false);
    w.dx = plan_tiles(T, H, turn_of(I) + I, kKE, false);
    w.dwgu = plan_tiles(2L * I, H, T, kKE, false);
    w.dw1 = plan_tiles(I, H, T, kKE, false);
    w.dwd = plan_tiles(H, I, T, kKE, false);
    size_t o = 0;
    w.gu = o;
    o += has_gu ? 0 : align256((size_t)T * I * 8);
    w.dgu = o;
    o += align256((size_t)T * I * 4);
    w.h = o;
    o += align256((size_t)T * I * 2);
    w.x = o;
    o += x_i8 ? align256((size_t)T * H * 2) : 0;
    w.part = o;
    size_t most = max2(part_bytes(w.dh, T, I), part_bytes(w.dx, T, H));
    most = max2(most, max2(part_bytes(w.dwgu, 2L * I, H), part_bytes(w.dw1, I, H)));
    most = max2(most, part_bytes(w.dwd, H, I));
    if (!has_gu) most = max2(most, part_bytes(w.gateup, T, 2L * I));
    w.total = o + most;
    if ((!has_gu && !fits(w.gateup)) || !fits(w.dh) || !fits(w.dx) || !fits(w.dwgu) || !fits(w.dw1) || !fits(w.dwd))
        w.total = kUnfit;
    return w;
}

hipError_t gateup(const FfnProblem& p, const Plan& plan, void* h, float* gu, float* part, hipStream_t s) {
    Args G = base(p.T, p.I, p.H);
    G.A = rows(p.x, p.H, p.T);
    G.B = rows(p.wg, p.H, p.I, p.wu);
    G.out = h;
    G.out2 = gu;
    return run<kBf16, kRow, kRow, kEpiGateUp>(G, plan, part, s);
}

// The same, g and u kept as i8x16 blocks.
hipError_t gateup8(const FfnProblem& p, const Plan& plan, void* h, float* part, hipStream_t s) {
    Args G = base(p.T, p.I, p.H);
    G.A = rows(p.x, p.H, p.T);
    G.B = rows(p.wg, p.H, p.I, p.wu);
    G.out = h;
    G.q = p.gu8;
    G.qe = p.gu8_e;
    return run<kBf16, kRow, kRow, kEpiGateUp8>(G, plan, part, s);
}

// The last products of the backward pass, which do not depend on each other:
// one launch whose workgroups take the tiles of all of them, the longest tiles
// first.  The tiles of one product rarely fill their last round of CUs (4096 x 7168
// x 2048: 1.75, 1.75 and 0.875 rounds, 4.375 together), and small products are
// mostly launches.
struct Product {
    Args G;
    Plan plan;   // its tiling if it runs alone
    int weight;  // a weight gradient (both operands by columns), else dx
};
struct Products {
    Args G[3];
    int first[4];   // first workgroup of each
    int weight[3];
};

template <int EDGE>
__global__ __launch_bounds__(tile_threads(EDGE)) __attribute__((amdgpu_waves_per_eu(tile_waves(EDGE, 5)))) void products_kernel(
    Products P) {
    const int b = blockIdx.x;
    const int i = (b >= P.first[1]) + (b >= P.first[2]);
    const int block = b - P.first[i], blocks = P.first[i + 1] - P.first[i];
    if (P.weight[i]) tile<kBf16, kCol, kCol, kEpiOut, false, EDGE, EDGE, 5>(P.G[i], block, blocks);
    else tile<kBf16, kRow, kCol, kEpiOut, false, EDGE, EDGE, 5>(P.G[i], block, blocks);
}

template <int EDGE>
hipError_t launch_together(const Product* todo, int n, hipStream_t s) {
    Products P{};
    long total = 0;
    for (int i = 0; i < n; ++i) {
        P.G[i] = todo[i].G;
        P.G[i].splits = 1;
        P.G[i].kspan = (P.G[i].K + kKE - 1) / kKE * kKE;
        P.weight[i] = todo[i].weight;
        P.first[i] = (int)total;
        total += count_tiles(P.G[i], EDGE, EDGE);
        if (!grid_fits(total, tile_threads(EDGE))) return hipErrorInvalidValue;
    }
    for (int i = n; i < 4; ++i) P.first[i] = (int)total;
    static DeviceCache ready;
    if (!allow_lds(ready, products_kernel<EDGE>, tile_lds(EDGE, 5))) return hipErrorInvalidValue;
    products_kernel<EDGE><<<dim3((unsigned)total), dim3(tile_threads(EDGE)), tile_lds(EDGE, 5), s>>>(P);
    return hipGetLastError();
}

hipError_t launch_products(Product* todo, int n, float* part, hipStream_t s) {
    // longest reduction first
    for (int i = 1; i < n; ++i)
        for (int j = i; j > 0 && todo[j].G.K > todo[j - 1].G.K; --j) std::swap(todo[j], todo[j - 1]);
    double apart = 0;
    Size sizes[3];
    for (int i = 0; i < n; ++i) {
        apart += todo[i].plan.us + 2;
        sizes[i] = {todo[i].G.M, todo[i].G.N, todo[i].G.K};
    }
    const int best = plan_together(sizes, n, kKE, apart);
    if (best == 256) return launch_together<256>(todo, n, s);
    if (best == 128) return launch_together<128>(todo, n, s);
    if (best == 64) return launch_together<64>(todo, n, s);
    hipError_t e = hipSuccess;
    for (int i = 0; i < n && e == hipSuccess; ++i)
        e = todo[i].weight ? run<kBf16, kCol, kCol, kEpiOut>(todo[i].G, todo[i].plan, part, s)
                           : run<kBf16, kRow, kCol, kEpiOut>(todo[i].G, todo[i].plan, part, s);
    return e;
}

__global__ __launch_bounds__(256) void zero_kernel(uint4* out, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) out[i] = uint4{0, 0, 0, 0};
}

}  // namespace

hipError_t launch_zero_bf16(void* out, size_t values, hipStream_t s) {
    const size_t n = values / 8;
    zero_kernel<<<dim3((unsigned)std::min((n + 255) / 256, (size_t)4096)), dim3(256), 0, s>>>((uint4*)out, n);
    return hipGetLastError();
}

size_t ffn_ws_bytes(int T, int H, int I, int gu8) { return T > 0 ? forward(T, H, I, gu8 != 0).total : 0; }
size_t ffn_backward_ws_bytes(int T, int H, int I, int has_gu, int x_i8) {
    return T > 0 ? backward(T, H, I, has_gu != 0, x_i8 != 0).total : 0;
}

hipError_t launch_ffn(const FfnProblem& p, void* ws, hipStream_t s) {
    const Forward w = forward(p.T, p.H, p.I, p.gu8 != nullptr);
    uint8_t* b = (uint8_t*)ws;
    float* part = (float*)(b + w.part);
    hipError_t e = p.gu8 ? gateup8(p, w.gateup, b + w.h, part, s) : gateup(p, w.gateup, b + w.h, p.gu, part, s);
    if (e != hipSuccess) return e;
    Args G = base(p.T, p.H, p.I);
    G.A = rows(b + w.h, p.I, p.T);
    G.B = rows(p.wd, p.I, p.H);
    G.out = p.y;
    G.out_f32 = p.y_f32;
    return run<kBf16, kRow, kRow, kEpiOut>(G, w.down, part, s);
}

hipError_t launch_ffn_backward(const FfnProblem& q, void* ws, hipStream_t s) {
    FfnProblem p = q;
    hipError_t e = hipSuccess;
    if (p.T == 0) {
        const size_t n = (size_t)p.I * p.H;
        if (p.dwg) e = launch_zero_bf16(p.dwg, n, s);
        if (e == hipSuccess && p.dwu) e = launch_zero_bf16(p.dwu, n, s);
        if (e == hipSuccess && p.dwd) e = launch_zero_bf16(p.dwd, n, s);
        return e;
    }
    const int T = p.T, H = p.H, I = p.I;
    const bool has_gu = p.gu_in || p.gu8;
    const Backward w = backward(T, H, I, has_gu, p.x_e != nullptr);
    uint8_t* b = (uint8_t*)ws;
    float* part = (float*)(b + w.part);
    uint8_t* dgu = b + w.dgu;
    uint8_t* h = b + w.h;
    const float* gu = p.gu_in;
    if (p.x_e && (!has_gu || p.dwg || p.dwu)) {
        e = launch_dequant_i8x16((const int8_t*)p.x, p.x_e, T, H, b + w.x, 0, s);
        if (e != hipSuccess) return e;
        p.x = b + w.x;
    }
    if (!has_gu) {
        gu = (const float*)(b + w.gu);
        e = gateup(p, w.gateup, h, (float*)(b + w.gu), part, s);
        if (e != hipSuccess) return e;
    }
    {
        Args G = base(T, I, H);
        G.A = rows(p.dy, H, T);
        G.B = cols(p.wd, I, I);
        G.gu = gu;
        G.q = p.gu8;
        G.qe = p.gu8_e;
        G.out = dgu;
        G.out2 = h;
        e = p.gu8 ? run<kBf16, kRow, kCol, kEpiGrad8>(G, w.dh, part, s) : run<kBf16, kRow, kCol, kEpiGrad>(G, w.dh, part, s);
    }
    if (e != hipSuccess) return e;
    // the products that are wanted: dx, the gate and up gradients (both at once, or
    // one with its half of dgu), the down gradient
    Product todo[3];
    int n = 0;
    if (p.dx) {
        Args G = base(T, H, turn_of(I) + I);
        G.turn = turn_of(I);
        G.len = I;
        G.A = rows(dgu, 2L * I, T, dgu + (size_t)I * 2);
        G.B = cols(p.wg, H, H, p.wu);
        G.out = p.dx;
        todo[n++] = {G, w.dx, 0};
    }
    if (p.dwg || p.dwu) {
        const bool both = p.dwg && p.dwu;
        Args G = base(both ? 2 * I : I, H, T);
        G.A = cols(dgu + (p.dwg ? 0 : (size_t)I * 2), 2L * I, both ? 2 * I : I);
        G.B = cols(p.x, H, H);
        G.out = p.dwg ? p.dwg : p.dwu;
        G.out2 = p.dwu;
        G.msplit = I;
        todo[n++] = {G, both ? w.dwgu : w.dw1, 1};
    }
    if (p.dwd) {
        Args G = base(H, I, T);
        G.A = cols(p.dy, H, H);
        G.B = cols(h, I, I);
        G.out = p.dwd;
        todo[n++] = {G, w.dwd, 1};
    }
    return launch_products(todo, n, part, s);
}

}  // namespace moe
