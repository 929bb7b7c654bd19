// The gated FFN of n experts on rows sorted by expert, and its gradients, in bf16
// (moe_experts_ffn, moe_experts_ffn_backward).  Rows [offsets[e], offsets[e + 1])
// belong to expert e; the offsets are read on the device only.
//   g = x Wg^T, u = x Wu^T, h = silu(g) u, y = h Wd^T          with the expert's weights
//   dh = dy Wd -> dg, du, h    dx = dg Wg + du Wu    [dWg; dWu] = [dg du]^T x    dWd = dy^T h
// The tiles are those of the dense block (gemm_tile.h; roundings: ffn.hip).  A
// product whose rows are the expert's (kRows) has as many row tiles as they fill, a
// weight gradient (kSum) sums over them: its tiles are the same for every expert, its
// reduction has the expert's length, and zeros without rows.  Every workgroup finds its
// expert and tile by a prefix sum over the offsets, which its first wave-wide loads
// bring: no list is made beforehand, and nothing about the rows has to reach the host.
//
// 16384 rows, 32 experts of 7168 x 2048, shares that differ, g and u in 8 bits: gate/up 1001 us,
// down 544, dh 535, dx 957 (0.9 to 1.0 PFLOP/s: experts' last tiles are 13 to 15 % more of a tile's time
// than their rows need, and weights come from HBM meanwhile), weight gradients 1690
// (gemm_stream.h); a large product reaches 1.4.  Few rows,
// 64 experts of 2048 x 1408: the weights' bytes, 5.2 TB/s over the whole step.
#include <algorithm>

#include "experts_plan.h"
#include "gemm_half.h"
#include "gemm_plan.h"
#include "gemm_stream.h"

namespace moe {
using namespace gemm;

namespace {

constexpr int kKE = kStage / 2;
static_assert(kDies == kXcds && kStreamEdge == kStreamM && kStreamEdge == kStreamN, "what the plans count with");

// One product for all experts: G as for expert 0 from row 0 on, and the steps
// from expert to expert.
struct Grouped {
    Args G;
    size_t wstep;          // kRows: bytes of an expert's weights (B); kSum: of its gradient
    const int32_t* offsets;
    int n, R;              // experts; rows there are
    int nt;                // kRows: column tiles; kSum: tiles of an expert
    int cus;               // kRows, 256-row tiles: CUs of a die
};

// Workgroup `block`'s among all experts' row tiles: the expert, the tile within it and
// the expert's rows; false past the last one.  Every wave does this by itself.
// cuts: with the halves of the last round (cut_of, half_tile).
struct Place {
    int e, t, first, m;
    int half;   // as in Cut
};
__device__ __forceinline__ bool find_rows(const Grouped& P, int edge, int block, bool cuts, Place& at) {
    const int lane = threadIdx.x % kWave;
    auto tiles = [&](int e) {
        if (e >= P.n) return 0;
        const int a = rows_before(P.offsets, e, P.R), b = rows_before(P.offsets, e + 1, P.R);
        return (max(b - a, 0) + edge - 1) / edge * P.nt;
    };
    auto scan = [&](int v) {
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(v, d, kWave);
            if (lane >= d) v += o;
        }
        return v;
    };
    int total = 0;
    for (int e0 = 0; e0 < P.n; e0 += kWave) total += __builtin_amdgcn_readlane(scan(tiles(e0 + lane)), kWave - 1);
    at.half = 0;
    if (cuts) {
        const Cut c = cut_of(block, total, P.cus);
        block = c.block;
        at.half = c.half;
    }
    int t = in_die_order(block, total);
    if (t < 0) return false;
    for (int e0 = 0; e0 < P.n; e0 += kWave) {
        const int own = tiles(e0 + lane), upto = scan(own);
        const uint64_t past = __ballot(t < upto);
        if (past) {
            const int l = __builtin_ctzll(past);
            at.e = e0 + l;
            at.t = t - __builtin_amdgcn_readlane(upto - own, l);
            // (offsets that do not ascend can name more tiles than 32 bits count)
            if ((unsigned)at.t >= (unsigned)__builtin_amdgcn_readlane(own, l)) return false;
            at.first = __builtin_amdgcn_readfirstlane(rows_before(P.offsets, at.e, P.R));
            at.m = __builtin_amdgcn_readfirstlane(rows_before(P.offsets, at.e + 1, P.R)) - at.first;
            return true;
        }
        t -= __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    return false;
}

// The product of one expert.
template <int EPI>
__device__ __forceinline__ Args rows_of(const Grouped& P, const Place& at) {
    Args G = P.G;
    const size_t r = (size_t)at.first, N = (size_t)G.N;
    G.M = G.A.n = G.msplit = at.m;
    G.A.p += r * G.A.ld;
    G.A.p2 += r * G.A.ld;
    G.B.p += at.e * P.wstep;
    G.B.p2 += at.e * P.wstep;
    const size_t nb = 2 * (size_t)i8x16_blocks(G.N);
    if constexpr (EPI == kEpiOut) {
        G.out = (uint8_t*)G.out + r * N * (G.out_f32 ? 4 : 2);
    } else if constexpr (EPI == kEpiGateUp || EPI == kEpiGateUp8) {
        G.out = (uint8_t*)G.out + r * N * 2;
        if (G.out2) G.out2 = (uint8_t*)G.out2 + r * N * 8;
    } else {
        G.out = (uint8_t*)G.out + r * N * 4;
        G.out2 = (uint8_t*)G.out2 + r * N * 2;
        G.gu += r * 2 * N;
    }
    if constexpr (EPI == kEpiGateUp8 || EPI == kEpiGrad8) {
        G.q += r * 2 * N;
        G.qe += r * nb;
    }
    return G;
}

// Workgroups of weight gradients of `nt` tiles an expert.  The dies share out every
// expert's tiles, so that none has the long experts for itself.
__device__ __forceinline__ bool find_sum(int nt, int block, int& e, int& t) {
    const int per = die_share(nt);
    e = block / kXcds / per;
    const int x = (block + e) % kXcds, j = block / kXcds % per;   // the dies with a tile more take turns
    const int base = nt / kXcds, extra = nt % kXcds;
    t = x * base + min(x, extra) + j;
    return j < base + (x < extra ? 1 : 0);
}

// Weight gradient of expert e, its tile t.
__device__ __forceinline__ Args sum_of(const Grouped& P, int e, int t, int& tm, int& tn) {
    Args G = P.G;
    const int first = __builtin_amdgcn_readfirstlane(rows_before(P.offsets, e, P.R));
    G.K = G.kspan = max(__builtin_amdgcn_readfirstlane(rows_before(P.offsets, e + 1, P.R)) - first, 0);
    G.A.p += (size_t)first * G.A.ld;
    G.B.p += (size_t)first * G.B.ld;
    G.out = (uint8_t*)G.out + (size_t)e * P.wstep;
    if (G.out2) G.out2 = (uint8_t*)G.out2 + (size_t)e * P.wstep;
    band_of(t, G.mt, G.nt, tm, tn);
    return G;
}

template <int LB, int EPI, int EDGE, int R>
__global__ __launch_bounds__(tile_threads(EDGE)) __attribute__((amdgpu_waves_per_eu(tile_waves(EDGE, R)))) void rows_kernel(
    Grouped P) {
    constexpr bool GU = EPI == kEpiGateUp || EPI == kEpiGateUp8;
    Place at;
    if (!find_rows(P, EDGE, blockIdx.x, EDGE == 256, at)) return;
    const Args G = rows_of<EPI>(P, at);
    int tm, tn;
    band_of(at.t, (at.m + EDGE - 1) / EDGE, P.nt, tm, tn);
    if constexpr (EDGE == 256) {
        const int m0 = tm * EDGE + (at.half == 2 ? EDGE / 2 : 0);
        if (m0 >= at.m) return;
        if (at.half || at.m - m0 <= EDGE / 2) {
            half_tile<LB, EPI, GU>(G, m0, tn);
            return;
        }
    }
    tile_at<kBf16, kRow, LB, EPI, GU, EDGE, EDGE, R>(G, tm, tn, 0);
}

// The last products of the backward pass, which do not depend on each other: one launch.
struct Products {
    Grouped P[3];
    int first[4];   // first workgroup of each
    int sum[3];     // a weight gradient, else dx
};
template <int EDGE, int R>
__global__ __launch_bounds__(tile_threads(EDGE)) __attribute__((amdgpu_waves_per_eu(tile_waves(EDGE, R)))) void products_kernel(
    Products Q) {
    const int b = blockIdx.x;
    const int i = (b >= Q.first[1]) + (b >= Q.first[2]);
    const Grouped& P = Q.P[i];
    int tm, tn;
    if (Q.sum[i]) {
        int e, t;
        if (!find_sum(P.nt, b - Q.first[i], e, t)) return;
        const Args G = sum_of(P, e, t, tm, tn);
        tile_at<kBf16, kCol, kCol, kEpiOut, false, EDGE, EDGE, R>(G, tm, tn, 0);
    } else {
        Place at;
        if (!find_rows(P, EDGE, b - Q.first[i], false, at)) return;
        const Args G = rows_of<kEpiOut>(P, at);
        band_of(at.t, (at.m + EDGE - 1) / EDGE, P.nt, tm, tn);
        tile_at<kBf16, kRow, kCol, kEpiOut, false, EDGE, EDGE, R>(G, tm, tn, 0);
    }
}

__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void stream_kernel(Stream S) { stream(S); }

// ---------------------------------------------------------------- host

Operand rows(const void* p, long ld, int n, const void* p2 = nullptr) {
    return Operand{(const uint8_t*)p, (const uint8_t*)p2, (size_t)ld * 2, n};
}

Grouped base(const ExpertsProblem& p, int N, int K) {
    Grouped P{};
    P.G.N = N;
    P.G.K = P.G.kspan = K;
    P.G.splits = 1;
    P.G.vec = 1;
    P.offsets = p.offsets;
    P.n = p.n;
    P.R = p.R;
    return P;
}

template <int LB, int EPI, int EDGE, int R>
hipError_t launch_rows_ring(const Grouped& P, long grid, hipStream_t s) {
    auto* k = rows_kernel<LB, EPI, EDGE, R>;
    static DeviceCache ready;
    if (!allow_lds(ready, k, tile_lds(EDGE, R))) return hipErrorInvalidValue;
    k<<<dim3((unsigned)grid), dim3(tile_threads(EDGE)), tile_lds(EDGE, R), s>>>(P);
    return hipGetLastError();
}

template <int LB, int EPI, int EDGE>
hipError_t launch_rows_edge(Grouped P, hipStream_t s) {
    constexpr bool GU = EPI == kEpiGateUp || EPI == kEpiGateUp8;
    P.nt = (P.G.N + (GU ? EDGE / 2 : EDGE) - 1) / (GU ? EDGE / 2 : EDGE);
    P.cus = std::max(device_cu_count() / kXcds, 1);
    const long grid = rows_grid(P.R, P.n, EDGE, P.nt);
    if (!grid_fits(grid, tile_threads(EDGE))) return hipErrorInvalidValue;
    if constexpr (EDGE < 256) {
        if (ring_of(EDGE, even_tiles(P.R, P.n, EDGE) * P.nt) == 10) return launch_rows_ring<LB, EPI, EDGE, 10>(P, grid, s);
    }
    return launch_rows_ring<LB, EPI, EDGE, 5>(P, grid, s);
}

template <int LB, int EPI>
hipError_t launch_rows(const Grouped& P, hipStream_t s) {
    constexpr bool GU = EPI == kEpiGateUp || EPI == kEpiGateUp8;
    switch (rows_edge(P.R, P.n, GU ? 2L * P.G.N : P.G.N, P.G.K, kKE)) {
        case 64: return launch_rows_edge<LB, EPI, 64>(P, s);
        case 128: return launch_rows_edge<LB, EPI, 128>(P, s);
        case 256: return launch_rows_edge<LB, EPI, 256>(P, s);
        default: return hipErrorInvalidValue;
    }
}

// k of dx = dg Wg + du Wu: dg's, and du's from the next stage on
int turn_of(int I) { return (I + kKE - 1) / kKE * kKE; }

struct Forward {
    size_t h, total;
};
Forward forward(int R, int I) {
    Forward f;
    f.h = 0;
    f.total = align256((size_t)R * I * 2);
    return f;
}
struct Backward {
    size_t gu, dgu, h, x, total;
};
Backward backward(int R, int H, int I, bool has_gu, bool x_i8) {
    Backward w;
    size_t o = 0;
    w.gu = o;
    o += has_gu ? 0 : align256((size_t)R * I * 8);
    w.dgu = o;
    o += align256((size_t)R * I * 4);
    w.h = o;
    o += align256((size_t)R * I * 2);
    w.x = o;
    o += x_i8 ? align256((size_t)R * H * 2) : 0;
    w.total = o;
    return w;
}

template <int EDGE, int R>
hipError_t launch_products_ring(const Products& Q, long total, hipStream_t s) {
    auto* k = products_kernel<EDGE, R>;
    static DeviceCache ready;
    if (!allow_lds(ready, k, tile_lds(EDGE, R))) return hipErrorInvalidValue;
    k<<<dim3((unsigned)total), dim3(tile_threads(EDGE)), tile_lds(EDGE, R), s>>>(Q);
    return hipGetLastError();
}

template <int EDGE>
hipError_t launch_products(Products Q, const GroupSize* sizes, int m, hipStream_t s) {
    long total = 0, tiles = 0;
    for (int i = 0; i < m; ++i) {
        Grouped& P = Q.P[i];
        Q.first[i] = (int)total;
        P.G.mt = (sizes[i].M + EDGE - 1) / EDGE;
        P.G.nt = (sizes[i].N + EDGE - 1) / EDGE;
        P.nt = Q.sum[i] ? P.G.mt * P.G.nt : P.G.nt;
        total += group_grid(sizes[i], P.R, P.n, EDGE);
        tiles += group_tiles(sizes[i], P.R, P.n, EDGE);
        if (!grid_fits(total, tile_threads(EDGE))) return hipErrorInvalidValue;
    }
    for (int i = m; i < 4; ++i) Q.first[i] = (int)total;
    if constexpr (EDGE < 256) {
        if (ring_of(EDGE, tiles) == 10) return launch_products_ring<EDGE, 10>(Q, total, s);
    }
    return launch_products_ring<EDGE, 5>(Q, total, s);
}

hipError_t launch_stream(const Grouped* todo, int m, hipStream_t s) {
    Stream S{};
    S.offsets = todo[0].offsets;
    S.n = todo[0].n;
    S.R = todo[0].R;
    long total = 0;
    for (int i = 0; i < m; ++i) {
        const Grouped& P = todo[i];
        const Args& G = P.G;
        SumProduct& D = S.P[i];
        D.A = G.A.p; D.B = G.B.p;
        D.lda = (uint32_t)G.A.ld; D.ldb = (uint32_t)G.B.ld;
        D.M = G.out2 ? G.msplit : G.M; D.N = G.N;
        D.half = (D.M + kStreamM - 1) / kStreamM;
        D.mt = G.out2 ? 2 * D.half : D.half;
        D.nt = (D.N + kStreamN - 1) / kStreamN;
        D.skip = (uint32_t)G.msplit * 2;
        D.out = (uint8_t*)G.out; D.out2 = (uint8_t*)G.out2;
        D.step = P.wstep;
        D.per = die_share(D.mt * D.nt);
        total += (long)S.n * D.per;
        if (total > 0x7fffffffL) return hipErrorInvalidValue;
        if (i == 0) S.first = (int)total;
    }
    S.total = (int)total;
    const int grid = std::max(device_cu_count() / kXcds, 1) * kXcds;
    static DeviceCache ready;
    if (!allow_lds(ready, stream_kernel, kStreamLds)) return hipErrorInvalidValue;
    stream_kernel<<<dim3(grid), dim3(512), kStreamLds, s>>>(S);
    return hipGetLastError();
}

hipError_t gateup(const ExpertsProblem& p, const void* x, void* h, float* gu, bool i8, hipStream_t s) {
    Grouped P = base(p, p.I, p.H);
    P.G.A = rows(x, p.H, 0);
    P.G.B = rows(p.wg, p.H, p.I, p.wu);
    P.wstep = (size_t)p.I * p.H * 2;
    P.G.out = h;
    if (i8) {
        P.G.q = p.gu8;
        P.G.qe = p.gu8_e;
        return launch_rows<kRow, kEpiGateUp8>(P, s);
    }
    P.G.out2 = gu;
    return launch_rows<kRow, kEpiGateUp>(P, s);
}

// Whether every product has a tiling whose grid holds it.
bool fits(int R, int n, int H, int I, bool grads) {
    if (R == 0) return true;
    if (!rows_edge(R, n, 2L * I, H, kKE)) return false;
    if (!grads) return rows_edge(R, n, H, I, kKE) != 0;
    const GroupSize all[3] = {{0, H, turn_of(I) + I, false}, {2 * I, H, 0, true}, {H, I, 0, true}};
    return rows_edge(R, n, I, H, kKE) && rows_edge(R, n, H, turn_of(I) + I, kKE) && group_edge(all, 3, R, n, kKE);
}

}  // namespace

size_t experts_ws_bytes(int R, int n, int H, int I) {
    return R == 0 ? 0 : fits(R, n, H, I, false) ? forward(R, I).total : kUnfit;
}
size_t experts_backward_ws_bytes(int R, int n, int H, int I, int has_gu, int x_i8) {
    return R == 0 ? 0 : fits(R, n, H, I, true) ? backward(R, H, I, has_gu != 0, x_i8 != 0).total : kUnfit;
}

hipError_t launch_experts(const ExpertsProblem& p, void* ws, hipStream_t s) {
    uint8_t* h = (uint8_t*)ws + forward(p.R, p.I).h;
    const hipError_t e = gateup(p, p.x, h, p.gu, p.gu8 != nullptr, s);
    if (e != hipSuccess) return e;
    Grouped P = base(p, p.H, p.I);
    P.G.A = rows(h, p.I, 0);
    P.G.B = rows(p.wd, p.I, p.H);
    P.wstep = (size_t)p.I * p.H * 2;
    P.G.out = p.y;
    P.G.out_f32 = p.y_f32;
    return launch_rows<kRow, kEpiOut>(P, s);
}

hipError_t launch_experts_backward(const ExpertsProblem& p, void* ws, hipStream_t s) {
    const int R = p.R, H = p.H, I = p.I;
    const size_t one = (size_t)I * H;
    hipError_t e = hipSuccess;
    if (R == 0) {
        if (p.dwg) e = launch_zero_bf16(p.dwg, p.n * one, s);
        if (e == hipSuccess && p.dwu) e = launch_zero_bf16(p.dwu, p.n * one, s);
        if (e == hipSuccess && p.dwd) e = launch_zero_bf16(p.dwd, p.n * one, s);
        return e;
    }
    const bool has_gu = p.gu || p.gu8;
    const Backward w = backward(R, H, I, has_gu, p.x_e != nullptr);
    uint8_t* b = (uint8_t*)ws;
    uint8_t* dgu = b + w.dgu;
    uint8_t* h = b + w.h;
    const void* x = p.x;
    if (p.x_e && (!has_gu || p.dwg || p.dwu)) {
        e = launch_dequant_i8x16((const int8_t*)p.x, p.x_e, R, H, b + w.x, 0, s);
        if (e != hipSuccess) return e;
        x = b + w.x;
    }
    const float* gu = p.gu;
    if (!has_gu) {
        e = gateup(p, x, h, (float*)(b + w.gu), false, s);
        if (e != hipSuccess) return e;
        gu = (const float*)(b + w.gu);
    }
    {
        Grouped P = base(p, I, H);
        P.G.A = rows(p.dy, H, 0);
        P.G.B = rows(p.wd, I, I);
        P.wstep = one * 2;
        P.G.gu = gu;
        P.G.q = p.gu8;
        P.G.qe = p.gu8_e;
        P.G.out = dgu;
        P.G.out2 = h;
        e = p.gu8 ? launch_rows<kCol, kEpiGrad8>(P, s) : launch_rows<kCol, kEpiGrad>(P, s);
        if (e != hipSuccess) return e;
    }
    Products Q{};
    GroupSize sizes[3];
    int m = 0;
    if (p.dx) {
        Grouped P = base(p, H, turn_of(I) + I);
        P.G.turn = turn_of(I);
        P.G.len = I;
        P.G.A = rows(dgu, 2L * I, 0, dgu + (size_t)I * 2);
        P.G.B = rows(p.wg, H, H, p.wu);
        P.wstep = one * 2;
        P.G.out = p.dx;
        sizes[m] = {0, P.G.N, P.G.K, false};
        Q.P[m++] = P;
    }
    const auto weight = [&](const Operand& A, const Operand& B, int M, int N, void* out, void* out2, int msplit) {
        Grouped P = base(p, N, 0);
        P.G.M = M;
        P.G.A = A;
        P.G.B = B;
        P.wstep = one * 2;
        P.G.out = out;
        P.G.out2 = out2;
        P.G.msplit = msplit;
        Q.sum[m] = 1;
        sizes[m] = {M, N, 0, true};
        Q.P[m++] = P;
    };
    if (p.dwg || p.dwu) {
        const bool both = p.dwg && p.dwu;
        const int M = both ? 2 * I : I;
        weight(rows(dgu + (p.dwg ? 0 : (size_t)I * 2), 2L * I, M), rows(x, H, H), M, H, p.dwg ? p.dwg : p.dwu, both ? p.dwu : nullptr, I);
    }
    if (p.dwd) weight(rows(p.dy, H, H), rows(h, I, I), H, I, p.dwd, nullptr, H);
    if (m == 0) return hipSuccess;
    if (m == 1 && p.dx) return launch_rows<kCol, kEpiOut>(Q.P[0], s);
    const int sums = p.dx ? 1 : 0;   // the weight gradients follow
    if (stream_tiles(sizes, m, p.n) >= device_cu_count()) {
        if (p.dx) e = launch_rows<kCol, kEpiOut>(Q.P[0], s);
        return e == hipSuccess ? launch_stream(&Q.P[sums], m - sums, s) : e;
    }
    switch (group_edge(sizes, m, R, p.n, kKE)) {
        case 64: return launch_products<64>(Q, sizes, m, s);
        case 128: return launch_products<128>(Q, sizes, m, s);
        case 256: return launch_products<256>(Q, sizes, m, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace moe
