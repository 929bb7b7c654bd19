// Activation checkpoints in 8 bits: blocks of 16 consecutive values of a row, int8
// codes with one power of two.
//   E = max(exponent field of max|v| - 6, 1), 255 where the block holds an infinity or a NaN
//   code = rne(v * 2^(127 - E)), clamped to [-127, 127];  value = code * 2^(E - 127)
// max|v| * 2^(127 - E) lies in [64, 128), so a value is off by at most half a step,
// 1/128 of max|v| (one step where 127.5 and more is clamped to 127), and where E is
// at its least by 2^-127.  v * 2^(127 - E) is exact, and so is the value both in fp32 and in
// bf16 (seven bits times a power of two): a product on the matrix cores takes exactly
// what is held.  A power of two costs up to one bit against a scale of max|v| / 127,
// but a quarter of its storage, and no division.  16 values, because a wave of the
// smallest product tiles holds 16 columns of a row: every tile size writes the same
// blocks.  E = 255 (whose codes are zeros) gives NaN for the whole block.
#pragma once
#include "common.h"

namespace moe {

constexpr int kI8Block = 16;
__host__ __device__ constexpr int i8x16_blocks(int cols) { return (cols + kI8Block - 1) / kI8Block; }

__device__ __forceinline__ uint32_t i8x16_exponent(float amax) {
    const uint32_t f = __float_as_uint(amax) >> 23;   // amax has no sign
    return f == 255u ? 255u : f < 7u ? 1u : f - 6u;
}

// Largest magnitude of the lane's eight values and its neighbour's (lane ^ 1).
__device__ __forceinline__ float i8x16_pair_max(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_magnitude(m, fabsf(v[e]));
    return max_magnitude(m, __shfl_xor(m, 1, kWave));
}

// Eight codes, the first in the lowest byte.
__device__ __forceinline__ uint2 i8x16_codes(const float (&v)[8], uint32_t E) {
    if (E == 255u) return make_uint2(0, 0);
    const float f = __uint_as_float((254u - E) << 23);   // 2^(127 - E)
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (int)fminf(fmaxf(rintf(v[e] * f), -127.0f), 127.0f);
        w[e / 4] |= ((uint32_t)c & 0xFFu) << (8 * (e % 4));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void i8x16_values(uint2 q, uint32_t E, float (&v)[8]) {
    const float f = __uint_as_float(E << 23);   // 2^(E - 127); E = 255: infinity, and 0 * infinity is NaN
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)(int)(int8_t)(w[e / 4] >> (8 * (e % 4))) * f;
}

}  // namespace moe
