// C consecutive values of a row in fp32 or bf16.
#pragma once
#include "common.h"

namespace moe {

// As loaded, so that many can be under way in few registers.  NT: past the caches' usual
// order, for what is read once; worth it where a wave reads whole lines (16 bytes a
// lane side by side, rows of whole lines), a loss where it does not.
template <bool F32, int C>
struct Raw {
    static constexpr int kWords = F32 ? C : C / 2;
    typedef __attribute__((ext_vector_type(kWords < 4 ? kWords : 4))) int Vec;
    Vec w[kWords < 4 ? 1 : kWords / 4];
    template <bool NT = false>
    __device__ __forceinline__ void load(const void* p, size_t at) {
        const Vec* q = (const Vec*)((const uint8_t*)p + at * (F32 ? 4 : 2));
#pragma unroll
        for (size_t i = 0; i < sizeof(w) / sizeof(Vec); ++i) w[i] = NT ? __builtin_nontemporal_load(q + i) : q[i];
    }
    __device__ __forceinline__ void values(float (&v)[C]) const {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (F32) v[i] = __int_as_float(w[i / 4][i % 4]);
            else v[i] = i % 2 ? __uint_as_float((uint32_t)w[i / 8][i / 2 % 4] & 0xFFFF0000u) : bf16_bits_to_f32((uint32_t)w[i / 8][i / 2 % 4]);
        }
    }
};

template <bool F32, int C>
__device__ __forceinline__ void load_row(const void* p, size_t at, float (&v)[C]) {
    Raw<F32, C> r;
    r.load(p, at);
    r.values(v);
}

template <bool NT = false, class V>
__device__ __forceinline__ void put(V* p, V v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

template <bool F32, int C, bool NT = false>
__device__ __forceinline__ void store_row(void* p, size_t at, const float (&v)[C]) {
    typedef typename Raw<F32, C>::Vec Vec;
    constexpr int kLanes = sizeof(Vec) / 4;
    Vec* q = (Vec*)((uint8_t*)p + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < Raw<F32, C>::kWords / kLanes; ++i) {
        Vec o;
#pragma unroll
        for (int e = 0; e < kLanes; ++e) {
            if constexpr (F32) o[e] = __float_as_int(v[i * kLanes + e]);
            else o[e] = (int)f32x2_to_bf16x2(v[2 * (i * kLanes + e)], v[2 * (i * kLanes + e) + 1]);
        }
        put<NT>(q + i, o);
    }
}

}  // namespace moe
