// What the norm kernels share: a row held in registers by TPR consecutive
// threads, eight (or one) neighbouring elements at a time, and sums over a row.
#pragma once
#include "common.h"
#include "dense.h"

namespace moe {
namespace norm {

// VEC consecutive elements of an fp32 or bf16 array as loaded: 16 or 32 bytes.
// Loading and unpacking are apart so that many loads can be in flight.
template <int VEC>
struct Raw {
    uint32_t w[VEC];   // VEC = 8: bf16 in w[0..3]
};

template <int VEC>
__device__ __forceinline__ Raw<VEC> load(const void* p, int f32, size_t at, bool in) {
    Raw<VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; ++e) r.w[e] = 0;
    if (!in) return r;
    if constexpr (VEC == 8) {
        if (f32) {
            const uint4* q = (const uint4*)((const float*)p + at);
            const uint4 a = q[0], b = q[1];
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w; r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
        } else {
            const uint4 a = *(const uint4*)((const uint16_t*)p + at);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        }
    } else {
        r.w[0] = f32 ? ((const uint32_t*)p)[at] : (uint32_t)((const uint16_t*)p)[at];
    }
    return r;
}

template <int VEC>
__device__ __forceinline__ void unpack(const Raw<VEC>& r, int f32, float (&v)[VEC]) {
    if (f32) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = __uint_as_float(r.w[e]);
    } else if constexpr (VEC == 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = bf16_bits_to_f32(r.w[e] & 0xFFFFu);
            v[2 * e + 1] = __uint_as_float(r.w[e] & 0xFFFF0000u);
        }
    } else {
        v[0] = bf16_bits_to_f32(r.w[0]);
    }
}

template <int VEC>
__device__ __forceinline__ void store(void* p, int f32, size_t at, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        if (f32) {
            float4* q = (float4*)((float*)p + at);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = f32_to_bf16_bits(v[2 * e]) | (f32_to_bf16_bits(v[2 * e + 1]) << 16);
            *(uint4*)((uint16_t*)p + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        if (f32) ((float*)p)[at] = v[0];
        else ((uint16_t*)p)[at] = (uint16_t)f32_to_bf16_bits(v[0]);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
    return v;
}

// Sums (or maxima) over the TPR threads of a row, the same value in all of
// them.  slot: LDS of TPR / 64 floats a row of the workgroup, two sets used in
// turn so that one barrier a call is enough.
template <int TPR, int N, bool MAX = false>
__device__ __forceinline__ void row_reduce(float (&v)[N], float* slot, int& turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = MAX ? wave_max(v[i]) : wave_sum(v[i]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wave = threadIdx.x / 64, first = wave / W * W;
        const int waves = blockDim.x / 64;
        float* set = slot + (turn & 1) * waves * 2;
        turn ^= 1;
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) set[i * waves + wave] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = set[i * waves + first];
#pragma unroll
            for (int w = 1; w < W; ++w) t = MAX ? fmaxf(t, set[i * waves + first + w]) : t + set[i * waves + first + w];
            v[i] = t;
        }
    }
}

inline bool rows16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace norm
}  // namespace moe
