// What the norm kernels share: a row held in registers by TPR consecutive
// threads, eight (or one) neighbouring elements at a time, and sums over a row.
#pragma once
#include <type_traits>

#include "common.h"
#include "dense.h"

namespace moe {
namespace norm {

// VEC consecutive elements of an fp32 or bf16 array as loaded: 16 or 32 bytes
// (WIDE: either, else bf16 only, in half the registers).  Loading and unpacking
// are apart so that many loads can be in flight.
template <int VEC, bool WIDE>
struct Raw {
    static constexpr int kWords = VEC == 8 ? (WIDE ? 8 : 4) : 1;
    uint32_t w[kWords];
};

template <int VEC, bool WIDE>
__device__ __forceinline__ Raw<VEC, WIDE> load(const void* p, int f32, size_t at, bool in) {
    Raw<VEC, WIDE> r;
#pragma unroll
    for (int e = 0; e < r.kWords; ++e) r.w[e] = 0;
    if (!in) return r;
    if constexpr (VEC == 8) {
        if (WIDE && f32) {
            const uint4* q = (const uint4*)((const float*)p + at);
            const uint4 a = q[0], b = q[1];
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            if constexpr (WIDE) { r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w; }
        } else {
            const uint4 a = *(const uint4*)((const uint16_t*)p + at);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        }
    } else {
        r.w[0] = f32 ? ((const uint32_t*)p)[at] : (uint32_t)((const uint16_t*)p)[at];
    }
    return r;
}

template <int VEC, bool WIDE>
__device__ __forceinline__ void unpack(const Raw<VEC, WIDE>& r, int f32, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        if constexpr (WIDE) {
            if (f32) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = __uint_as_float(r.w[e]);
                return;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = bf16_bits_to_f32(r.w[e] & 0xFFFFu);
            v[2 * e + 1] = __uint_as_float(r.w[e] & 0xFFFF0000u);
        }
    } else {
        v[0] = f32 ? __uint_as_float(r.w[0]) : bf16_bits_to_f32(r.w[0]);
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
            for (int e = 0; e < 4; ++e) w[e] = f32x2_to_bf16x2(v[2 * e], v[2 * e + 1]);
            *(uint4*)((uint16_t*)p + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        if (f32) ((float*)p)[at] = v[0];
        else ((uint16_t*)p)[at] = (uint16_t)f32_to_bf16_bits(v[0]);
    }
}

// VEC weights as floats; ones where there are none.
template <int VEC>
__device__ __forceinline__ void weights(const void* p, int f32, size_t at, bool in, float (&w)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = 1.0f;
    if (p && in) unpack(load<VEC, true>(p, f32, at, true), f32, w);
}

template <bool MAX>
__device__ __forceinline__ float join(float a, float b) { return MAX ? fmaxf(a, b) : a + b; }

// Sum (maximum) over the 16 lanes of a DPP row, in all of them.
template <bool MAX>
__device__ __forceinline__ float row16(float v) {
    auto other = [](float x, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    v = join<MAX>(v, other(v, std::integral_constant<int, 0xB1>{}));    // lane ^ 1
    v = join<MAX>(v, other(v, std::integral_constant<int, 0x4E>{}));    // lane ^ 2
    v = join<MAX>(v, other(v, std::integral_constant<int, 0x141>{}));   // mirrored in 8
    return join<MAX>(v, other(v, std::integral_constant<int, 0x140>{}));   // mirrored in 16
}

// Sums (or maxima) over the TPR threads of a row, the same value in all of
// them: 16 lanes by DPP, the rest through LDS (slot: 2 sets of 2 values for
// every 16 threads of the workgroup, used in turn so that one barrier a call is
// enough).
template <int TPR, int N, bool MAX = false>
__device__ __forceinline__ void row_reduce(float (&v)[N], float* slot, int& turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row16<MAX>(v[i]);
    if constexpr (TPR == 64) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = join<MAX>(v[i], __shfl_xor(v[i], 16, kWave));
            v[i] = join<MAX>(v[i], __shfl_xor(v[i], 32, kWave));
        }
    } else {
        constexpr int W = TPR / 16;
        const int part = threadIdx.x / 16, first = part / W * W, parts = blockDim.x / 16;
        float* set = slot + (turn & 1) * parts * 2;
        turn ^= 1;
        if (threadIdx.x % 16 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) set[i * parts + part] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float4 t = *(const float4*)(set + i * parts + first);
#pragma unroll
            for (int w = 4; w < W; w += 4) {
                const float4 o = *(const float4*)(set + i * parts + first + w);
                t.x = join<MAX>(t.x, o.x); t.y = join<MAX>(t.y, o.y); t.z = join<MAX>(t.z, o.z); t.w = join<MAX>(t.w, o.w);
            }
            v[i] = join<MAX>(join<MAX>(t.x, t.y), join<MAX>(t.z, t.w));
        }
    }
}

inline bool rows16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace norm
}  // namespace moe
