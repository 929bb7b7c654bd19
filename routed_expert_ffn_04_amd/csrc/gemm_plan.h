// Tile size and k-splits of a product, and the kernel that sums the splits.
#pragma once
#include "dense.h"
#include "gemm_tile.h"

namespace moe {
namespace gemm {

struct Plan {
    int big;             // 256 x 256 tiles, else 128 x 128
    int splits, kspan;
};

// mma_cols: MFMA columns of the product (gate/up: both matrices' columns).
inline Plan plan_tiles(long M, long mma_cols, int K, int stage_elems) {
    Plan p;
    const long big = ((M + 255) / 256) * ((mma_cols + 255) / 256);
    p.big = big >= 192;
    const int stages = (K + stage_elems - 1) / stage_elems;
    p.splits = 1;
    p.kspan = stages * stage_elems;
    if (!p.big) {
        const long tiles = ((M + 127) / 128) * ((mma_cols + 127) / 128);
        if (tiles < 256) {
            const int want = (int)((511 + tiles) / tiles);
            const int most = stages / 4 > 1 ? stages / 4 : 1;
            const int s = want < most ? want : most;
            const int span = (stages + s - 1) / s;
            p.kspan = span * stage_elems;
            p.splits = (stages + span - 1) / span;
        }
    }
    return p;
}

// bytes of the partial sums
inline size_t part_bytes(const Plan& p, long M, long cols) { return p.splits > 1 ? align256((size_t)p.splits * M * cols * 4) : 0; }

// Sums the k-splits in their order and applies the product's epilogue.  A
// thread takes eight consecutive columns of one row.  splits = 0: the
// outputs of an empty sum.
template <int EPI>
__global__ __launch_bounds__(256) void reduce_kernel(Args G, const float* __restrict__ part, int splits) {
    const int groups = (G.N + 7) / 8;
    const long at = (long)blockIdx.x * 256 + threadIdx.x;
    if (at >= (long)G.M * groups) return;
    const int m = (int)(at / groups), n = (int)(at % groups) * 8;
    constexpr bool GU = EPI == kEpiGateUp;
    const size_t cols = GU ? 2 * (size_t)G.N : (size_t)G.N;
    const size_t plane = (size_t)G.M * cols;
    const float* p = part + (size_t)m * cols + n;
    const bool whole = (G.N & 3) == 0 && n + 8 <= G.N;
    auto load = [&](const float* q, float(&v)[8]) {
        if (whole) {
            const float4 a = *(const float4*)q, b = *(const float4*)(q + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = n + e < G.N ? q[e] : 0.0f;
        }
    };
    auto total = [&](const float* q, float(&sum)[8]) {
        int acc[8] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
        for (int s = 0; s < splits; ++s) {
            float v[8];
            load(q + s * plane, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (EPI == kEpiI8) acc[e] += __float_as_int(v[e]);   // the splits of an int8 product are int32
                else sum[e] += v[e];
            }
        }
        if (EPI == kEpiI8)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = (float)acc[e];
    };
    float v[8];
    total(p, v);
    if constexpr (EPI == kEpiGateUp) {
        float u[8], h[8];
        total(p + G.N, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = silu_mul(v[e], u[e]);
        *(uint4*)((uint16_t*)G.out + (size_t)m * G.N + n) = pack8(h);
        if (G.out2) {
            float* o = (float*)G.out2 + (size_t)m * cols + n;
            *(float4*)o = make_float4(v[0], v[1], v[2], v[3]);
            *(float4*)(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
            o += G.N;
            *(float4*)o = make_float4(u[0], u[1], u[2], u[3]);
            *(float4*)(o + 4) = make_float4(u[4], u[5], u[6], u[7]);
        }
    } else if constexpr (EPI == kEpiGrad) {
        float g[8], u[8], dg[8], du[8], h[8];
        const float* gp = G.gu + (size_t)m * (2 * (size_t)G.N) + n;
        load(gp, g);
        load(gp + G.N, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) swiglu_grad(g[e], u[e], v[e], dg[e], du[e], h[e]);
        uint16_t* d = (uint16_t*)G.out + (size_t)m * (2 * (size_t)G.N) + n;
        *(uint4*)d = pack8(dg);
        *(uint4*)(d + G.N) = pack8(du);
        *(uint4*)((uint16_t*)G.out2 + (size_t)m * G.N + n) = pack8(h);
    } else if constexpr (EPI == kEpiI8) {
        const float xs = G.xs[m];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int ne = min(n + e, G.N - 1);
            v[e] *= xs * G.ws[ne];
            if (G.bias) v[e] += G.bias[ne];
        }
        store8(G, (uint8_t*)G.out + (size_t)m * G.N * (G.out_f32 ? 4 : 2), n, v, G.out_f32);
    } else {
        const size_t row_bytes = (size_t)G.N * (G.out_f32 ? 4 : 2);
        uint8_t* o = m < G.msplit ? (uint8_t*)G.out + (size_t)m * row_bytes
                                  : (uint8_t*)G.out2 + (size_t)(m - G.msplit) * row_bytes;
        store8(G, o, n, v, G.out_f32);
    }
}

template <int EPI>
hipError_t launch_reduce(const Args& G, const float* part, int splits, hipStream_t s) {
    const long threads = (long)G.M * ((G.N + 7) / 8);
    const long blocks = (threads + 255) / 256;
    if (blocks > 0x7fffffffL) return hipErrorInvalidValue;
    if (blocks == 0) return hipSuccess;
    reduce_kernel<EPI><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(G, part, splits);
    return hipGetLastError();
}

// The product with its epilogue: one launch, or the k-splits' partial sums
// into `part` and a second launch that joins them.
template <int E, int LA, int LB, int EPI>
hipError_t run(Args G, const Plan& p, float* part, hipStream_t s) {
    constexpr bool GU = EPI == kEpiGateUp;
    G.splits = p.splits;
    G.kspan = p.kspan;
    if (p.big) return launch_tiles<E, LA, LB, EPI, GU, 256, 256>(G, s);
    if (p.splits == 1) return launch_tiles<E, LA, LB, EPI, GU, 128, 128>(G, s);
    Args P = G;
    P.out = part;
    P.vec = (G.N & 3) == 0;
    const hipError_t e = launch_tiles<E, LA, LB, kEpiPart, GU, 128, 128>(P, s);
    return e != hipSuccess ? e : launch_reduce<EPI>(G, part, p.splits, s);
}

}  // namespace gemm
}  // namespace moe
