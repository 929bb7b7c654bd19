// int8 product with a scale per token and per output channel (moe_linear_i8),
// and the per-token quantisation that feeds it (moe_quant_i8).
//   q[t][k] = rne(x[t][k] / s_t),  s_t = amax_t / 127 (IEEE divisions; 1 where that is 0, NaN with a NaN in the row)
//   out[t][n] = (sum_k q[t][k] w[n][k]) * (s_t * w_scale[n]) + bias[n]
// The sum is exact in int32 (K <= 131071 keeps 128 * 128 * K below 2^31); it is
// converted to fp32 once (nearest even) and scaled.
#include "gemm_plan.h"

namespace moe {
using namespace gemm;

namespace {

// One row per workgroup of 256 threads, held in registers between the row's
// maximum and its codes (NV chunks of eight a thread); wider rows are read a
// second time, from L2.  8192 x 7168 in bf16: 40 us, 4.4 TB/s (46 us reading every
// row twice and dividing every element).
template <bool F32, int NV>
__global__ __launch_bounds__(256) void quant_i8_kernel(const void* __restrict__ x, size_t first, int cols,
                                                       int8_t* __restrict__ q, float* __restrict__ scale) {
    const size_t row = first + blockIdx.x;
    const int tid = threadIdx.x;
    __shared__ float part[4];
    constexpr int kWide = 2048 * NV;   // columns held; the steps past the last column of 2^31 - 16 leave an int's range
    auto load = [&](uint32_t c, float(&v)[8]) __attribute__((always_inline)) {
        if (F32) {
            const float4* p = (const float4*)((const float*)x + row * cols + c);
            const float4 a = p[0], b = p[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 u = *(const uint4*)((const uint16_t*)x + row * cols + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
                v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
            }
        }
    };
    float held[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 256 + tid) * 8;
        if (c < cols) load(c, held[i]);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) held[i][e] = 0.0f;
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_magnitude(amax, fabsf(held[i][e]));
    for (uint32_t c = kWide + tid * 8; c < (uint32_t)cols; c += 2048) {
        float v[8];
        load(c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_magnitude(amax, fabsf(v[e]));
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) amax = max_magnitude(amax, __shfl_xor(amax, m, kWave));
    if (tid % 64 == 0) part[tid / 64] = amax;
    __syncthreads();
    amax = max_magnitude(max_magnitude(part[0], part[1]), max_magnitude(part[2], part[3]));
    const float s = i8_scale(amax), inv = 1.0f / s;
    if (tid == 0) scale[row] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * 256 + tid) * 8;
        if (c < cols) *(uint2*)(q + row * cols + c) = i8_codes8(held[i], s, inv);
    }
    for (uint32_t c = kWide + tid * 8; c < (uint32_t)cols; c += 2048) {
        float v[8];
        load(c, v);
        *(uint2*)(q + row * cols + c) = i8_codes8(v, s, inv);
    }
}

constexpr size_t kRowsALaunch = (size_t)1 << 23;   // a grid holds fewer than 2^32 threads

}  // namespace

hipError_t launch_quant_i8(const void* x, int x_f32, int rows, int cols, int8_t* q, float* scale, hipStream_t s) {
    const dim3 block(256);
    for (size_t first = 0; first < (size_t)rows; first += kRowsALaunch) {
        const dim3 grid((unsigned)std::min(rows - first, kRowsALaunch));
        if (x_f32) {
            if (cols <= 2048) quant_i8_kernel<true, 1><<<grid, block, 0, s>>>(x, first, cols, q, scale);
            else quant_i8_kernel<true, 4><<<grid, block, 0, s>>>(x, first, cols, q, scale);
        } else {
            if (cols <= 2048) quant_i8_kernel<false, 1><<<grid, block, 0, s>>>(x, first, cols, q, scale);
            else quant_i8_kernel<false, 4><<<grid, block, 0, s>>>(x, first, cols, q, scale);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

size_t linear_i8_ws_bytes(int T, int K, int N) {
    if (T == 0) return 0;
    const Plan p = plan_tiles(T, N, K, kStage, true);
    return fits(p) ? part_bytes(p, T, N) : kUnfit;
}

hipError_t launch_linear_i8(const LinearI8Problem& p, void* ws, hipStream_t s) {
    Args G{};
    G.M = p.T; G.N = p.N; G.K = p.K; G.msplit = p.T;
    G.A = Operand{(const uint8_t*)p.q, nullptr, (size_t)p.K, p.T};
    G.B = Operand{(const uint8_t*)p.w, nullptr, (size_t)p.K, p.N};
    G.xs = p.xs; G.ws = p.ws; G.bias = p.bias;
    G.out = p.out;
    G.out_f32 = p.out_f32;
    G.vec = p.N % (p.out_f32 ? 4 : 8) == 0 && ((uintptr_t)p.out & 15u) == 0;
    return run<kI8, kRow, kRow, kEpiI8>(G, plan_tiles(p.T, p.N, p.K, kStage, true), (float*)ws, s);
}

}  // namespace moe
