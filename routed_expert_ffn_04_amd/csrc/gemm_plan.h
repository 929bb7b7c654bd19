// A product by its plan: the launch of its tiles, and the kernel that sums the k-splits.
#pragma once
#include <algorithm>

#include "dense.h"
#include "gemm_few.h"
#include "gemm_tile.h"
#include "tile_plan.h"

namespace moe {
namespace gemm {

// bytes of the partial sums
inline size_t part_bytes(const Plan& p, long M, long cols) { return p.splits > 1 ? align256((size_t)p.splits * M * cols * 4) : 0; }

// Sums the k-splits in their order and applies the product's epilogue.  A
// thread takes eight consecutive columns of one row.
template <int EPI>
__global__ __launch_bounds__(256) void reduce_kernel(Args G, const float* __restrict__ part, int splits) {
    // kEpiGateUp8: whole blocks of 16 columns, whose halves meet in neighbouring lanes
    const int groups = EPI == kEpiGateUp8 ? 2 * i8x16_blocks(G.N) : (G.N + 7) / 8;
    const long at = (long)blockIdx.x * 256 + threadIdx.x;
    if (at >= (long)G.M * groups) return;
    const int m = (int)(at / groups), n = (int)(at % groups) * 8;
    constexpr bool GU = EPI == kEpiGateUp || EPI == kEpiGateUp8;
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
        for (int s0 = 0; s0 < splits; s0 += 4) {   // four splits' loads in flight
            float v[4][8];
#pragma unroll
            for (int s = 0; s < 4; ++s) load(q + min(s0 + s, splits - 1) * plane, v[s]);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s0 + s < splits)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (EPI == kEpiI8) acc[e] += __float_as_int(v[s][e]);   // the splits of an int8 product are int32
                        else sum[e] += v[s][e];
                    }
        }
        if (EPI == kEpiI8)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = (float)acc[e];
    };
    float v[8];
    total(p, v);
    if constexpr (GU) {
        float u[8], h[8];
        total(p + G.N, u);
        if constexpr (EPI == kEpiGateUp8) {
            store_gu8(G, m, n, v, u);
            if (n >= G.N) return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = silu_mul(v[e], u[e]);
        *(uint4*)((uint16_t*)G.out + (size_t)m * G.N + n) = pack8(h);
        if (EPI == kEpiGateUp && G.out2) {
            float* o = (float*)G.out2 + (size_t)m * cols + n;
            *(float4*)o = make_float4(v[0], v[1], v[2], v[3]);
            *(float4*)(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
            o += G.N;
            *(float4*)o = make_float4(u[0], u[1], u[2], u[3]);
            *(float4*)(o + 4) = make_float4(u[4], u[5], u[6], u[7]);
        }
    } else if constexpr (EPI == kEpiGrad || EPI == kEpiGrad8) {
        float g[8], u[8], dg[8], du[8], h[8];
        if constexpr (EPI == kEpiGrad8) {
            const size_t nb = (size_t)i8x16_blocks(G.N), at8 = (size_t)m * (2 * (size_t)G.N) + n;
            const uint8_t* e = G.qe + (size_t)m * (2 * nb) + n / kI8Block;
            i8x16_values(*(const uint2*)(G.q + at8), e[0], g);
            i8x16_values(*(const uint2*)(G.q + at8 + G.N), e[nb], u);
        } else {
            const float* gp = G.gu + (size_t)m * (2 * (size_t)G.N) + n;
            load(gp, g);
            load(gp + G.N, u);
        }
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
    const long threads = (long)G.M * (EPI == kEpiGateUp8 ? 2 * i8x16_blocks(G.N) : (G.N + 7) / 8);
    const long blocks = (threads + 255) / 256;
    if (blocks == 0) return hipSuccess;
    if (!grid_fits(blocks, 256)) return hipErrorInvalidValue;
    reduce_kernel<EPI><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(G, part, splits);
    return hipGetLastError();
}

// 128-row tiles: with one workgroup per CU a ring of ten half-stages (1024 x 4096
// gate/up: 77 us against 108 with five), with more two per CU and five each
// (4096 x 2048 dh: 146 us against 193 with ten).
template <int E, int LA, int LB, int EPI, bool GU>
hipError_t launch_tiling(const Args& G, const Plan& p, hipStream_t s) {
    if (p.edge == 256) return launch_tiles<E, LA, LB, EPI, GU, 256, 256, 5>(G, s);
    if (p.edge == 64) {
        if (p.workgroups <= 512) return launch_tiles<E, LA, LB, EPI, GU, 64, 64, 10>(G, s);
        return launch_tiles<E, LA, LB, EPI, GU, 64, 64, 5>(G, s);
    }
    if (p.workgroups <= 256) return launch_tiles<E, LA, LB, EPI, GU, 128, 128, 10>(G, s);
    return launch_tiles<E, LA, LB, EPI, GU, 128, 128, 5>(G, s);
}

// The product with its epilogue: one launch, or the k-splits' partial sums
// into `part` and a second launch that joins them.
template <int E, int LA, int LB, int EPI>
hipError_t run(Args G, const Plan& p, float* part, hipStream_t s) {
    constexpr bool GU = EPI == kEpiGateUp || EPI == kEpiGateUp8;
    G.splits = p.splits;
    G.kspan = p.kspan;
    if constexpr (LA == kRow && LB == kRow && EPI != kEpiGateUp8) {
        if (p.few) return launch_few<E, EPI>(G, s);
    }
    Args P = G;
    if (p.splits > 1) {
        P.out = part;
        P.vec = (G.N & 3) == 0;
    }
    const hipError_t e = p.splits > 1 ? launch_tiling<E, LA, LB, kEpiPart, GU>(P, p, s) : launch_tiling<E, LA, LB, EPI, GU>(G, p, s);
    return e != hipSuccess || p.splits == 1 ? e : launch_reduce<EPI>(G, part, p.splits, s);
}

}  // namespace gemm
}  // namespace moe
