// The products for a few rows of A (decode: one to 16 tokens), both operands
// with k contiguous: their time is reading B once, so nothing is tiled and
// nothing passes through LDS.
//
// A workgroup takes 16 weight rows (gate/up: 8 gate rows and the 8 up rows of
// the same columns) for all tokens, its waves share out k in blocks of 128
// bytes (whole cache lines), and every wave loads its MFMA operands straight
// into registers, one block ahead.  Lane l holds weight row l % 16 and bytes [16
// (l / 16), +16) of the block's two halves, for two MFMAs; tokens are laid out the
// same way, so both sides agree on which k a piece holds.  More blocks in flight a
// wave cost more than they bring (four together, unpipelined: 7.4 us against 6.4 for
// a token of 1024 x 512, 9.2 against 8.9 of 2048 x 1408, in one run).  The
// waves' sums meet in LDS in a fixed order and the epilogue follows, with no
// second launch: k is split eight ways, and 16 rows a workgroup give enough
// workgroups for every CU.  One token of the 7168 x 2048 block: 22 us and two
// launches for 88 MB from HBM, 4.0 TB/s; two launches of next to nothing (256 x 512)
// take 5.1.  With 16 tokens as many bytes of x as of weights pass through a wave
// (from L2): 30 us.
#pragma once
#include "gemm_tile.h"
#include "tile_plan.h"

namespace moe {
namespace gemm {

// Four consecutive outputs n .. n + 3 of a row.
__device__ __forceinline__ void store4(const Args& G, uint8_t* row, int n, const float (&v)[4], bool f32) {
    if (G.vec && n + 4 <= G.N) {
        if (f32) *(float4*)((float*)row + n) = make_float4(v[0], v[1], v[2], v[3]);
        else *(uint2*)((uint16_t*)row + n) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < G.N) {
                if (f32) ((float*)row)[n + e] = v[e];
                else ((uint16_t*)row)[n + e] = (uint16_t)f32_to_bf16_bits(v[e]);
            }
    }
}

template <int E, int EPI, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void few_kernel(Args G) {
    constexpr bool GU = EPI == kEpiGateUp;
    constexpr int EB = E == kI8 ? 1 : 2;
    __shared__ __attribute__((aligned(16))) uint8_t sums[WAVES * 1024];
    const int lane = threadIdx.x % 64, r = lane % 16, c = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int n0 = blockIdx.x * (GU ? 8 : 16);
    const int kbytes = G.K * EB;
    const int blocks = (kbytes + 127) / 128;

    const bool up = GU && r >= 8;
    const int wrow = min(n0 + (GU ? r % 8 : r), G.B.n - 1);
    const uint8_t* wp = (up ? G.B.p2 : G.B.p) + (size_t)wrow * G.B.ld + c * 16;
    const uint8_t* xp = G.A.p + (size_t)min(r, G.A.n - 1) * G.A.ld + c * 16;
    const int left = kbytes - c * 16;   // bytes of the row from the lane's first piece on

    typename Acc<E>::type acc{};
    struct Block { i32x4 w[2], x[2]; };
    auto load = [&](int b, Block& t) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int off = b * 128 + h * 64;
            const bool in = off < left;
            t.w[h] = *(const i32x4*)(in ? wp + off : (const uint8_t*)kZeros);
            t.x[h] = i32x4{};
            if (in && r < G.M) t.x[h] = *(const i32x4*)(xp + off);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto mma = [&](const Block& t) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) acc = Acc<E>::mma(t.w[h], t.x[h], acc);
        __builtin_amdgcn_sched_barrier(0);
    };
    Block even, odd;
    int b = wave;
    load(b, even);
    for (; b + WAVES < blocks; b += 2 * WAVES) {
        load(b + WAVES, odd);
        mma(even);
        if (b + 2 * WAVES < blocks) load(b + 2 * WAVES, even);
        mma(odd);
    }
    if (b < blocks) mma(even);
    *(typename Acc<E>::type*)(sums + threadIdx.x * 16) = acc;
    __syncthreads();
    if (wave > 0) return;

    // lane l has n = 4 (l / 16) + v of token l % 16
    typename Acc<E>::type total = acc;
#pragma unroll
    for (int i = 1; i < WAVES; ++i) total += *(const typename Acc<E>::type*)(sums + (i * 64 + lane) * 16);
    const int m = r;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)total[e];
    if constexpr (GU) {
        // rows 0..7 (lanes 0..31) gate, rows 8..15 (lanes 32..63) up
        float u[4], h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = __shfl(v[e], lane % 32 + 32, kWave);
        const int n = n0 + 4 * (c % 2);
        if (m >= G.M || n >= G.N) return;
        if (G.out2) {   // g and u, each from the lanes that hold it
            float* o = (float*)G.out2 + (size_t)m * (2 * (size_t)G.N) + (lane < 32 ? 0 : G.N) + n;
            *(float4*)o = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (lane >= 32) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = silu_mul(v[e], u[e]);
        *(uint2*)((uint16_t*)G.out + (size_t)m * G.N + n) = make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
    } else {
        const int n = n0 + 4 * c;
        if (m >= G.M || n >= G.N) return;
        if constexpr (EPI == kEpiI8) {
            const float xs = G.xs[m];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ne = min(n + e, G.N - 1);
                v[e] *= xs * G.ws[ne];
                if (G.bias) v[e] += G.bias[ne];
            }
        }
        store4(G, (uint8_t*)G.out + (size_t)m * G.N * (G.out_f32 ? 4 : 2), n, v, G.out_f32);
    }
}

template <int E, int EPI>
hipError_t launch_few(const Args& G, hipStream_t s) {
    constexpr int cols = EPI == kEpiGateUp ? 8 : 16;
    const long blocks = ((long)G.N + cols - 1) / cols;
    if (!grid_fits(blocks, kFewThreads)) return hipErrorInvalidValue;
    few_kernel<E, EPI, kFewThreads / 64><<<dim3((unsigned)blocks), dim3(kFewThreads), 0, s>>>(G);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace moe
