// Activation checkpoints in 8 bits (format: i8x16.h): moe_quant_i8x16 and
// moe_dequant_i8x16.  Memory-bound: a lane takes eight consecutive columns of a
// row (one 16-byte bf16 load, or two fp32 ones; one 8-byte access of the codes), two
// neighbouring lanes a block.  16384 x 7168 from bf16 67 us (5.3 TB/s), back 65 (5.5).
#include "dense.h"
#include "gffn_common.h"
#include "i8x16.h"
#include "row_io.h"

namespace moe {

namespace {

// Lane -> row and first column.  Rows are whole blocks (lanes past the end of a ragged
// last block only take part in the exchange).
struct At {
    long row;
    int c;
    bool valid;
};
__device__ __forceinline__ At place(long rows, int cols) {
    const int per = 2 * i8x16_blocks(cols);
    const long at = (long)blockIdx.x * 256 + threadIdx.x;
    At a;
    a.row = at / per;
    a.c = (int)(at - a.row * per) * 8;
    a.valid = a.row < rows && a.c < cols;
    return a;
}

template <bool F32>
__global__ __launch_bounds__(256) void quant_kernel(const void* __restrict__ x, long rows, int cols,
                                                    int8_t* __restrict__ q, uint8_t* __restrict__ e8) {
    const At a = place(rows, cols);
    float v[8] = {};
    if (a.valid) load_row<F32, 8>(x, (size_t)a.row * cols + a.c, v);
    const uint32_t E = i8x16_exponent(i8x16_pair_max(v));
    if (!a.valid) return;
    *(uint2*)(q + (size_t)a.row * cols + a.c) = i8x16_codes(v, E);
    if (a.c % kI8Block == 0) e8[(size_t)a.row * i8x16_blocks(cols) + a.c / kI8Block] = (uint8_t)E;
}

template <bool F32>
__global__ __launch_bounds__(256) void dequant_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e8,
                                                      long rows, int cols, void* __restrict__ out) {
    const At a = place(rows, cols);
    if (!a.valid) return;
    float v[8];
    i8x16_values(*(const uint2*)(q + (size_t)a.row * cols + a.c),
                 e8[(size_t)a.row * i8x16_blocks(cols) + a.c / kI8Block], v);
    store_row<F32, 8>(out, (size_t)a.row * cols + a.c, v);
}

// A grid holds fewer than 2^32 threads: rows with more lanes go out in several launches.
template <class Launch>
hipError_t launch_pieces(long rows, int cols, Launch&& launch) {
    const long per = 2L * i8x16_blocks(cols), most = 0xffffff00L / per;
    for (long r = 0; r < rows; r += most) {
        const long n = rows - r < most ? rows - r : most;
        launch(r, n, dim3((unsigned)((n * per + 255) / 256)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_quant_i8x16(const void* x, int x_f32, long rows, int cols, int8_t* q, uint8_t* e8, hipStream_t s) {
    return launch_pieces(rows, cols, [&](long r, long n, dim3 grid) {
        const uint8_t* from = (const uint8_t*)x + (size_t)r * cols * (x_f32 ? 4 : 2);
        int8_t* codes = q + (size_t)r * cols;
        uint8_t* e = e8 + (size_t)r * i8x16_blocks(cols);
        if (x_f32) quant_kernel<true><<<grid, dim3(256), 0, s>>>(from, n, cols, codes, e);
        else quant_kernel<false><<<grid, dim3(256), 0, s>>>(from, n, cols, codes, e);
    });
}

hipError_t launch_dequant_i8x16(const int8_t* q, const uint8_t* e8, long rows, int cols, void* out, int out_f32,
                                hipStream_t s) {
    return launch_pieces(rows, cols, [&](long r, long n, dim3 grid) {
        const int8_t* codes = q + (size_t)r * cols;
        const uint8_t* e = e8 + (size_t)r * i8x16_blocks(cols);
        uint8_t* to = (uint8_t*)out + (size_t)r * cols * (out_f32 ? 4 : 2);
        if (out_f32) dequant_kernel<true><<<grid, dim3(256), 0, s>>>(codes, e, n, cols, to);
        else dequant_kernel<false><<<grid, dim3(256), 0, s>>>(codes, e, n, cols, to);
    });
}

}  // namespace moe
