// What the norm kernels share: a row held in registers by TPR consecutive
// threads, eight neighbouring elements at a time, and sums over a row.
#pragma once
#include <type_traits>

#include "common.h"
#include "dense.h"

namespace moe {
namespace norm {

// A thread's chunk: eight neighbouring elements of an fp32 or bf16 row.  RAGGED:
// rows that do not begin on 16 bytes (the vector accesses then carry their
// elements' alignment only, which global memory allows) and whose last chunk is
// shorter (element by element).
constexpr int kVec = 8;

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;

// The chunk as loaded: 16 or 32 bytes (WIDE: either, else bf16 only, in half the
// registers).  Loading and unpacking are apart so that many loads can be in flight.
template <bool WIDE>
struct Raw {
    static constexpr int kWords = WIDE ? 8 : 4;
    uint32_t w[kWords];
};

template <bool RAGGED>
__device__ __forceinline__ u32x4 get16(const void* p) {
    if constexpr (RAGGED) return *(const u32x4_any*)p;
    else return *(const u32x4*)p;
}
template <bool RAGGED, bool STREAM>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
    if constexpr (RAGGED) *(u32x4_any*)p = v;
    else if constexpr (STREAM) __builtin_nontemporal_store(v, (u32x4*)p);
    else *(u32x4*)p = v;
}

// n: elements from `at` to the end of the row (zero or less: none, the rest of the chunk is zero).
template <bool WIDE, bool RAGGED>
__device__ __forceinline__ Raw<WIDE> load(const void* p, int f32, size_t at, int n) {
    Raw<WIDE> r;
#pragma unroll
    for (int e = 0; e < r.kWords; ++e) r.w[e] = 0;
    if (n <= 0) return r;
    if (WIDE && f32) {
        const float* q = (const float*)p + at;
        if (!RAGGED || n >= kVec) {
            const u32x4 a = get16<RAGGED>(q), b = get16<RAGGED>(q + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r.w[e] = a[e];
                if constexpr (WIDE) r.w[4 + e] = b[e];
            }
        } else if constexpr (WIDE) {
#pragma unroll
            for (int e = 0; e < kVec - 1; ++e)
                if (e < n) r.w[e] = __float_as_uint(q[e]);
        }
    } else {
        const uint16_t* q = (const uint16_t*)p + at;
        if (!RAGGED || n >= kVec) {
            const u32x4 a = get16<RAGGED>(q);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.w[e] = a[e];
        } else {
#pragma unroll
            for (int e = 0; e < kVec - 1; ++e)
                if (e < n) r.w[e / 2] |= (uint32_t)q[e] << (16 * (e % 2));
        }
    }
    return r;
}

template <bool WIDE>
__device__ __forceinline__ void unpack(const Raw<WIDE>& r, int f32, float (&v)[kVec]) {
    if constexpr (WIDE) {
        if (f32) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] = __uint_as_float(r.w[e]);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = bf16_bits_to_f32(r.w[e] & 0xFFFFu);
        v[2 * e + 1] = __uint_as_float(r.w[e] & 0xFFFF0000u);
    }
}

// n as in load, above zero.  STREAM: past the caches.
template <bool RAGGED, bool STREAM = false>
__device__ __forceinline__ void store(void* p, int f32, size_t at, const float (&v)[kVec], int n) {
    if (f32) {
        float* q = (float*)p + at;
        if (!RAGGED || n >= kVec) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                put16<RAGGED, STREAM>(q + 4 * h, u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                               __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])});
        } else {
#pragma unroll
            for (int e = 0; e < kVec - 1; ++e)
                if (e < n) q[e] = v[e];
        }
    } else {
        uint16_t* q = (uint16_t*)p + at;
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = f32x2_to_bf16x2(v[2 * e], v[2 * e + 1]);
        if (!RAGGED || n >= kVec) {
            put16<RAGGED, STREAM>(q, w);
        } else {
#pragma unroll
            for (int e = 0; e < kVec - 1; ++e)
                if (e < n) q[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
        }
    }
}

// Weights as floats; ones where there are none.
template <bool RAGGED>
__device__ __forceinline__ void weights(const void* p, int f32, size_t at, int n, float (&w)[kVec]) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] = 1.0f;
    if (p && n > 0) unpack(load<true, RAGGED>(p, f32, at, n), f32, w);
}

template <bool MAX>
__device__ __forceinline__ float join(float a, float b) { return MAX ? max_magnitude(a, b) : a + b; }

// Sum (largest magnitude) over the 16 lanes of a DPP row, in all of them.
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

// Sums (or largest magnitudes) over the TPR threads of a row, the same value in all of
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
