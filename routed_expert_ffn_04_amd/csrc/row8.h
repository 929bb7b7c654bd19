// Eight consecutive values of a row in fp32 or bf16, 16-byte aligned.
#pragma once
#include "common.h"

namespace moe {

template <bool F32>
__device__ __forceinline__ void load_row8(const void* p, size_t at, float (&v)[8]) {
    if constexpr (F32) {
        const float4 a = *(const float4*)((const float*)p + at), b = *(const float4*)((const float*)p + at + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *(const uint4*)((const uint16_t*)p + at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
            v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store_row8(void* p, size_t at, const float (&v)[8]) {
    if constexpr (F32) {
        float4* o = (float4*)((float*)p + at);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *(uint4*)((uint16_t*)p + at) = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                                  f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
    }
}

}  // namespace moe
