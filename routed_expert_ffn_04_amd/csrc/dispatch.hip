// The tokens' rows sorted by expert, and the gradients around them (moe_dispatch,
// moe_dispatch_backward, moe_combine_backward).  dest[t k + j] is the sorted row of
// token t's j-th expert (moe_permute); a value outside [0, R) has no row here.
//   dispatch            xs[dest[t k + j]] = x[t]
//   its gradient        dx[t] = add[t] + sum_j dxs[dest[t k + j]]               (fp32, in this order)
//   combine's gradient  dy[dest[t k + j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[dest[t k + j]]>
// Memory-bound, no arithmetic to speak of.  Each runs over the tokens, so a token's row
// is read once from HBM and every sorted row once (read or written): a kernel
// that ran over the sorted rows instead would read the tokens' rows k times.
#include "dense.h"
#include "gffn_common.h"
#include "i8x16.h"
#include "row8.h"

namespace moe {

namespace {

// ---- dispatch: a lane takes 16 bytes of a token's row (of the row as it is written) and stores them k times.
// A workgroup takes 256 pieces of one token, or several tokens with shorter rows.
struct Piece {
    long t;
    int c;
    bool valid;
};
__device__ __forceinline__ Piece piece_of(int T, int pieces, int slabs, int per) {
    Piece p;
    if (per == 1) {
        const uint32_t b = blockIdx.x;
        const uint32_t t = b / (uint32_t)slabs;
        p.t = t;
        p.c = (int)(b - t * slabs) * 256 + (int)threadIdx.x;
        p.valid = p.c < pieces;
    } else {
        const int r = (int)threadIdx.x / pieces;
        p.t = (long)blockIdx.x * per + r;
        p.c = (int)threadIdx.x - r * pieces;
        p.valid = r < per && p.t < T;
    }
    return p;
}

enum { kCopy = 0, kFromI8 = 1 };

template <int KIND>
__global__ __launch_bounds__(256) void dispatch_kernel(const uint8_t* __restrict__ x, const uint8_t* __restrict__ xe,
                                                       int T, int pieces, int slabs, int per,
                                                       const int32_t* __restrict__ dest, int k, int R,
                                                       uint4* __restrict__ xs) {
    const Piece p = piece_of(T, pieces, slabs, per);
    if (!p.valid) return;
    uint4 v;
    if constexpr (KIND == kFromI8) {
        const int blocks = (pieces + 1) / 2;
        float f[8];
        i8x16_values(*(const uint2*)(x + ((size_t)p.t * pieces + p.c) * 8), xe[(size_t)p.t * blocks + p.c / 2], f);
        v = make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                       f32x2_to_bf16x2(f[6], f[7]));
    } else {
        v = ((const uint4*)x)[(size_t)p.t * pieces + p.c];
    }
    const int32_t* d = dest + (size_t)p.t * k;
    for (int j = 0; j < k; ++j) {
        const int r = d[j];
        if ((unsigned)r < (unsigned)R) xs[(size_t)r * pieces + p.c] = v;
    }
}

// ---- gradient of dispatch: a lane takes eight columns of a token, the rows of up to eight experts in flight
constexpr int kRows = 8;

template <bool F32, bool ADD_F32, bool OUT_F32>
__global__ __launch_bounds__(256) void gather_kernel(const void* __restrict__ dxs, const void* __restrict__ add, int T,
                                                     int pieces, int slabs, int per, const int32_t* __restrict__ dest,
                                                     int k, int R, void* __restrict__ dx) {
    const Piece p = piece_of(T, pieces, slabs, per);
    if (!p.valid) return;
    const size_t at = ((size_t)p.t * pieces + p.c) * 8;
    float sum[8] = {};
    if (add) load_row8<ADD_F32>(add, at, sum);
    const int32_t* d = dest + (size_t)p.t * k;
    for (int j0 = 0; j0 < k; j0 += kRows) {
        float v[kRows][8];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int r = j0 + j < k ? d[j0 + j] : -1;
            if ((unsigned)r < (unsigned)R) {
                load_row8<F32>(dxs, ((size_t)r * pieces + p.c) * 8, v[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += v[j][e];
    }
    store_row8<OUT_F32>(dx, at, sum);
}

// ---- gradients of combine: a wave takes one assignment, so the sum over its row stays in the wave
enum { kYNone = 0, kYF32 = 1, kYBf16 = 2, kYE4m3 = 3 };

template <int Y, bool D_F32, bool DY_F32>
__global__ __launch_bounds__(256) void combine_grad_kernel(const void* __restrict__ dout, const void* __restrict__ y,
                                                           const float* __restrict__ y_scale,
                                                           const int32_t* __restrict__ dest, const float* __restrict__ w,
                                                           long n, int k, int H, int R, void* __restrict__ dy,
                                                           float* __restrict__ dw) {
    const int lane = threadIdx.x % kWave;
    const long f = (long)blockIdx.x * 4 + threadIdx.x / kWave;
    if (f >= n) return;
    const long t = f / k;
    const int r = dest[f];
    const bool here = (unsigned)r < (unsigned)R;
    float sum = 0.0f;
    if (here) {
        const float wf = w[f];
        const size_t from = (size_t)t * H, to = (size_t)r * H;
        for (int c = lane * 8; c < H; c += kWave * 8) {
            float d[8];
            load_row8<D_F32>(dout, from + c, d);
            if constexpr (Y != kYNone) {
                float v[8];
                if constexpr (Y == kYE4m3) {
                    const uint2 q = *(const uint2*)((const uint8_t*)y + to + c);
                    const float sc = y_scale[(size_t)r * (H / 128) + c / 128];
                    const uint32_t word[2] = {q.x, q.y};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)word[i], false);
                        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)word[i], true);
                        v[4 * i] = lo[0] * sc;
                        v[4 * i + 1] = lo[1] * sc;
                        v[4 * i + 2] = hi[0] * sc;
                        v[4 * i + 3] = hi[1] * sc;
                    }
                } else {
                    load_row8<Y == kYF32>(y, to + c, v);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(d[e], v[e], sum);
            }
            if (dy) {
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] *= wf;
                store_row8<DY_F32>(dy, to + c, d);
            }
        }
    }
    if constexpr (Y != kYNone) {
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, kWave);
        if (lane == 0) dw[f] = sum;
    }
}

// Launch shape of the kernels over the tokens' pieces of 16 bytes (or eight columns).
struct Shape {
    int slabs, per;
    long blocks;
};
Shape shape_of(int T, int pieces) {
    Shape s;
    s.per = pieces >= 256 ? 1 : 256 / pieces;
    s.slabs = (pieces + 255) / 256;
    s.blocks = s.per == 1 ? (long)T * s.slabs : ((long)T + s.per - 1) / s.per;
    return s;
}
bool fits(long blocks) { return blocks <= 0xffffffffL / 256; }

}  // namespace

bool dispatch_fits(int T, int H, int k) { return fits(shape_of(T, H / 4).blocks) && fits(((long)T * k + 3) / 4); }

hipError_t launch_dispatch(const DispatchProblem& p, hipStream_t s) {
    const int pieces = p.x_f32 ? p.H / 4 : p.H / 8;
    const Shape g = shape_of(p.T, pieces);
    if (!fits(g.blocks)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)g.blocks), block(256);
    const auto run = [&](auto* kernel) {
        kernel<<<grid, block, 0, s>>>((const uint8_t*)p.x, p.xe, p.T, pieces, g.slabs, g.per, p.dest, p.k, p.R, (uint4*)p.xs);
        return hipGetLastError();
    };
    return p.xe ? run(dispatch_kernel<kFromI8>) : run(dispatch_kernel<kCopy>);
}

hipError_t launch_dispatch_backward(const DispatchProblem& p, hipStream_t s) {
    const int pieces = p.H / 8;
    const Shape g = shape_of(p.T, pieces);
    if (!fits(g.blocks)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)g.blocks), block(256);
    const auto run = [&](auto* kernel) {
        kernel<<<grid, block, 0, s>>>(p.dxs, p.add, p.T, pieces, g.slabs, g.per, p.dest, p.k, p.R, p.dx);
        return hipGetLastError();
    };
    if (p.dxs_f32) {
        if (p.add_f32) return p.dx_f32 ? run(gather_kernel<true, true, true>) : run(gather_kernel<true, true, false>);
        return p.dx_f32 ? run(gather_kernel<true, false, true>) : run(gather_kernel<true, false, false>);
    }
    if (p.add_f32) return p.dx_f32 ? run(gather_kernel<false, true, true>) : run(gather_kernel<false, true, false>);
    return p.dx_f32 ? run(gather_kernel<false, false, true>) : run(gather_kernel<false, false, false>);
}

namespace {

template <int Y>
hipError_t combine_grad(const CombineGradProblem& p, hipStream_t s) {
    const long n = (long)p.T * p.k, blocks = (n + 3) / 4;
    if (!fits(blocks)) return hipErrorInvalidValue;
    const auto run = [&](auto* kernel) {
        kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(p.dout, p.y, p.y_scale, p.dest, p.w, n, p.k, p.H, p.R, p.dy, p.dw);
        return hipGetLastError();
    };
    if (p.dout_f32) return p.dy_f32 ? run(combine_grad_kernel<Y, true, true>) : run(combine_grad_kernel<Y, true, false>);
    return p.dy_f32 ? run(combine_grad_kernel<Y, false, true>) : run(combine_grad_kernel<Y, false, false>);
}

}  // namespace

hipError_t launch_combine_backward(const CombineGradProblem& p, hipStream_t s) {
    if (!p.dw) return combine_grad<kYNone>(p, s);
    if (p.y_mode == 0) return combine_grad<kYF32>(p, s);
    if (p.y_mode == 1) return combine_grad<kYBf16>(p, s);
    return combine_grad<kYE4m3>(p, s);
}

}  // namespace moe
