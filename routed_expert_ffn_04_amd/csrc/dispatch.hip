// The tokens' rows sorted by expert, and the gradients around them (moe_dispatch,
// moe_dispatch_backward, moe_combine_backward).  dest[t k + j] is the sorted row of
// token t's j-th expert (moe_permute); a value outside [0, R) has no row here.
//   dispatch            xs[dest[t k + j]] = x[t]
//   its gradient        dx[t] = add[t] + sum_j dxs[dest[t k + j]]               (fp32, in this order)
//   combine's gradient  dy[dest[t k + j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[dest[t k + j]]>
// Memory-bound, no arithmetic to speak of.  Dispatch and its gradient run over the tokens, so
// a token's row is read or written once, and every sorted row once.  Combine's gradient runs
// over a token's assignments one after the other, a wave for each: it loads the token's row k
// times, of which the caches answer all but the first.
//
// Sorted rows are met once, and there are many more of them than the caches hold, so
// they go past the caches' usual order (NT) where a row is whole lines: dispatch of 16384
// tokens to 8 of 7168 columns in bf16 437 -> 355 us for the same tokens again, which the caches
// hold; for others every time 415 to 419 by itself (5.1 TB/s written and read) and 442 in
// turn with its gradient; the gradient 420 -> 376 (5.6).  Rows of other lengths keep the usual
// one, which joins the pieces of a line (2056 columns: 45 us, against 63).  Row numbers that
// are the same in a whole wave are read through the scalar cache: the gradient took 532 us with
// vector loads of them.
#include <algorithm>

#include "dense.h"
#include "gffn_common.h"
#include "i8x16.h"
#include "row_io.h"

namespace moe {

namespace {

// Workgroup's place where every die takes one contiguous run of the `blocks` there are, so that the
// workgroups of a token share its row in one L2 (workgroups go to the dies in turn).  Tokens' pieces:
// 16384 tokens to 8 rows of 7168, inputs in turn, 415 us against 428 (its gradient 375 either way).
// Assignments, where rows are whole lines: e4m3 rows 311 against 318 us (fp32 rows of 2056 110.7
// against 109.2, so not there).
__device__ __forceinline__ uint32_t in_die_order(uint32_t block, uint32_t blocks) {
    const uint32_t x = block % kXcds, base = blocks / kXcds, extra = blocks % kXcds;
    return x * base + min(x, extra) + block / kXcds;
}

// Pieces of a token's row: 16 bytes of what is written or summed.  Long rows (LONG): a
// workgroup takes U * 256 pieces of one token, so that the token and with it its rows' numbers
// are uniform.  Short ones: one piece a lane, several tokens a workgroup.
template <bool LONG, int U>
struct Piece {
    int t, c;
    __device__ __forceinline__ Piece(int pieces, int slabs, int per) {
        if constexpr (LONG) {
            const uint32_t b = in_die_order(blockIdx.x, gridDim.x);
            t = (int)(b / (uint32_t)slabs);
            c = (int)(b - (uint32_t)t * slabs) * (U * 256) + (int)threadIdx.x;
        } else {
            const int r = (int)threadIdx.x / pieces;
            t = r < per ? (int)(blockIdx.x * per + r) : 0x7fffffff;
            c = (int)threadIdx.x - r * pieces;
        }
    }
};

// ---- dispatch: a token's piece is read once and stored k times
template <bool FROM_I8, bool LONG, int U, bool NT>
__global__ __launch_bounds__(256) void dispatch_kernel(const uint8_t* __restrict__ x, const uint8_t* __restrict__ xe,
                                                       int T, int pieces, int slabs, int per,
                                                       const int32_t* __restrict__ dest, int k, int R,
                                                       i32x4* __restrict__ xs) {
    const Piece<LONG, U> p(pieces, slabs, per);
    if (p.t >= T) return;
    i32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = p.c + u * 256;
        if (c >= pieces) continue;
        if constexpr (FROM_I8) {
            float f[8];
            i8x16_values(*(const uint2*)(x + ((size_t)p.t * pieces + c) * 8), xe[(size_t)p.t * ((pieces + 1) / 2) + c / 2], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[u][e] = (int)f32x2_to_bf16x2(f[2 * e], f[2 * e + 1]);
        } else {
            v[u] = ((const i32x4*)x)[(size_t)p.t * pieces + c];
        }
    }
    const int32_t* d = dest + (size_t)p.t * k;
    for (int j = 0; j < k; ++j) {
        const int r = d[j];
        if ((unsigned)r >= (unsigned)R) continue;
        i32x4* row = xs + (size_t)r * pieces;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (p.c + u * 256 < pieces) put<NT>(row + p.c + u * 256, v[u]);
    }
}

// ---- gradient of dispatch: the rows of up to eight experts in flight
constexpr int kRows = 8;

template <bool F32, bool ADD_F32, bool OUT_F32, bool LONG, bool NT>
__global__ __launch_bounds__(256) void gather_kernel(const void* __restrict__ dxs, const void* add, int T,
                                                     int pieces, int slabs, int per, const int32_t* __restrict__ dest,
                                                     int k, int R, void* dx) {   // dx may be add
    constexpr int C = F32 ? 4 : 8;
    const Piece<LONG, 1> p(pieces, slabs, per);
    if (p.t >= T || p.c >= pieces) return;
    const size_t at = ((size_t)p.t * pieces + p.c) * C;
    float sum[C] = {};
    if (add) load_row<ADD_F32, C>(add, at, sum);
    const int32_t* d = dest + (size_t)p.t * k;
    for (int j0 = 0; j0 < k; j0 += kRows) {
        Raw<F32, C> v[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int r = j0 + j < k ? d[j0 + j] : -1;
            v[j] = Raw<F32, C>{};
            if ((unsigned)r < (unsigned)R) v[j].template load<NT>(dxs, ((size_t)r * pieces + p.c) * C);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            float f[C];
            v[j].values(f);
#pragma unroll
            for (int e = 0; e < C; ++e) sum[e] += f[e];
        }
    }
    store_row<OUT_F32, C>(dx, at, sum);
}

// ---- gradients of combine: a wave takes one assignment, so the sum over its row stays in
// the wave; the waves of a workgroup share their tokens' rows in the caches.  S = 2: two
// waves take one, where these are no more than the SIMDs and a wave would go over its row twice (device time,
// rows of 7168 bf16, 128 / 512 / 1024 / 2048 of them: 3.9 / 4.9 / 7.0 / 14.2 us against 5.0 / 6.3 / 8.0 / 13.4).
enum { kYNone = 0, kYF32 = 1, kYBf16 = 2, kYE4m3 = 3 };
// kAhead pieces of 64 lanes have their loads out together.  Eight of them and four waves a
// workgroup, against four and eight: 30018 fp32 rows of 2056 110.7 us against 114.5 (4.8 TB/s), e4m3 rows
// 317 against 323 us, 128 tokens of 8 bf16 rows 9.0 against 10.1.
constexpr int kGradWaves = 4, kAhead = 8;

template <int Y, bool D_F32, bool DY_F32, bool NT, int S>
__global__ __launch_bounds__(kGradWaves * 64) void combine_grad_kernel(
    const void* __restrict__ dout, const void* __restrict__ y, const float* __restrict__ y_scale,
    const int32_t* __restrict__ dest, const float* __restrict__ w, long first, long n, int k, int H, int R,
    void* __restrict__ dy, float* __restrict__ dw) {
    constexpr int C = D_F32 || DY_F32 || Y == kYF32 ? 4 : 8;   // 16 bytes a lane of the wider ones
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const long f = first + (long)(NT ? in_die_order(blockIdx.x, gridDim.x) : blockIdx.x) * (kGradWaves / S) + wave / S;
    if (S == 1 && f >= n) return;
    const long t = f / k;
    const int r = f < n ? dest[f] : -1;
    float sum = 0.0f;
    if ((unsigned)r < (unsigned)R) {
        const float wf = w[f];
        const size_t from = (size_t)t * H, to = (size_t)r * H;
        for (int c0 = (wave % S * (kAhead * kWave) + lane) * C; c0 < H; c0 += S * kAhead * kWave * C) {
            Raw<D_F32, C> d[kAhead];
            Raw<Y == kYF32, C> v[kAhead];   // e4m3: the first word or two of it
            float scale[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int c = c0 + a * kWave * C;
                if (c >= H) break;
                d[a].load(dout, from + c);
                if constexpr (Y == kYE4m3) {
                    const uint8_t* q = (const uint8_t*)y + to + c;
                    if constexpr (C == 8) {
                        const uint2 two = *(const uint2*)q;
                        v[a].w[0][0] = (int)two.x;
                        v[a].w[0][1] = (int)two.y;
                    } else {
                        v[a].w[0][0] = *(const int*)q;
                    }
                    scale[a] = y_scale[(size_t)r * (H / 128) + c / 128];
                } else if constexpr (Y != kYNone) {
                    v[a].template load<NT>(y, to + c);
                }
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int c = c0 + a * kWave * C;
                if (c >= H) break;
                float g[C];
                d[a].values(g);
                if constexpr (Y != kYNone) {
                    float b[C];
                    if constexpr (Y == kYE4m3) {
#pragma unroll
                        for (int i = 0; i < C / 4; ++i) {
                            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(v[a].w[0][i], false);
                            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(v[a].w[0][i], true);
                            b[4 * i] = lo[0] * scale[a];
                            b[4 * i + 1] = lo[1] * scale[a];
                            b[4 * i + 2] = hi[0] * scale[a];
                            b[4 * i + 3] = hi[1] * scale[a];
                        }
                    } else {
                        v[a].values(b);
                    }
#pragma unroll
                    for (int e = 0; e < C; ++e) sum = __builtin_fmaf(g[e], b[e], sum);
                }
                if (dy) {
#pragma unroll
                    for (int e = 0; e < C; ++e) g[e] *= wf;
                    store_row<DY_F32, C, NT>(dy, to + c, g);
                }
            }
        }
    }
    if constexpr (Y != kYNone) {
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, kWave);
        if constexpr (S == 1) {
            if (lane == 0) dw[f] = sum;
        } else {
            __shared__ float part[kGradWaves];
            if (lane == 0) part[wave] = sum;
            __syncthreads();
            if (lane == 0 && wave % S == 0 && f < n) {
                for (int i = 1; i < S; ++i) sum += part[wave + i];
                dw[f] = sum;
            }
        }
    }
}

// Launch shape of the kernels over the tokens' pieces.  A grid holds fewer than 2^32 threads: tokens
// (of combine's gradient: assignments) that need more go out in several launches.
constexpr long kMostBlocks = 0xffffffffL / 256;
struct Shape {
    int slabs, per;
    bool rows;      // LONG
    long most;      // tokens of a launch
    long blocks(long T) const { return rows ? T * slabs : (T + per - 1) / per; }
};
Shape shape_of(int pieces, int u) {
    Shape s;
    s.rows = pieces > 128;   // up to 128 pieces two tokens and more fit a workgroup
    s.per = s.rows ? 1 : 256 / pieces;
    s.slabs = (pieces + u * 256 - 1) / (u * 256);
    s.most = s.rows ? kMostBlocks / s.slabs : kMostBlocks * s.per;
    return s;
}

// Whether the rows of a matrix are whole lines.
bool whole_lines(const void* p, size_t row_bytes) { return ((uintptr_t)p | row_bytes) % 128 == 0; }

constexpr int kU = 2;   // 512 pieces a workgroup: 415 us against 424 with 256 and 417 with 1024 (see in_die_order)

}  // namespace

hipError_t launch_dispatch(const DispatchProblem& p, hipStream_t s) {
    const int pieces = p.x_f32 ? p.H / 4 : p.H / 8;
    const Shape g = shape_of(pieces, kU);
    const auto run = [&](auto* kernel) {
        for (long t = 0; t < p.T; t += g.most) {
            const long n = std::min(g.most, p.T - t);
            kernel<<<dim3((unsigned)g.blocks(n)), dim3(256), 0, s>>>(
                (const uint8_t*)p.x + (size_t)t * pieces * (p.xe ? 8 : 16), p.xe ? p.xe + (size_t)t * i8x16_blocks(p.H) : nullptr,
                (int)n, pieces, g.slabs, g.per, p.dest + (size_t)t * p.k, p.k, p.R, (i32x4*)p.xs);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    if (!g.rows) return p.xe ? run(dispatch_kernel<true, false, 1, false>) : run(dispatch_kernel<false, false, 1, false>);
    if (whole_lines(p.xs, (size_t)pieces * 16))
        return p.xe ? run(dispatch_kernel<true, true, kU, true>) : run(dispatch_kernel<false, true, kU, true>);
    return p.xe ? run(dispatch_kernel<true, true, kU, false>) : run(dispatch_kernel<false, true, kU, false>);
}

namespace {

template <bool F32, bool ADD_F32, bool OUT_F32>
hipError_t gather(const DispatchProblem& p, hipStream_t s) {
    const int pieces = p.H / (F32 ? 4 : 8);
    const Shape g = shape_of(pieces, 1);
    const auto run = [&](auto* kernel) {
        for (long t = 0; t < p.T; t += g.most) {
            const long n = std::min(g.most, p.T - t);
            const size_t at = (size_t)t * p.H;
            kernel<<<dim3((unsigned)g.blocks(n)), dim3(256), 0, s>>>(
                p.dxs, p.add ? (const uint8_t*)p.add + at * (ADD_F32 ? 4 : 2) : nullptr, (int)n, pieces, g.slabs, g.per,
                p.dest + (size_t)t * p.k, p.k, p.R, (uint8_t*)p.dx + at * (OUT_F32 ? 4 : 2));
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    if (!g.rows) return run(gather_kernel<F32, ADD_F32, OUT_F32, false, false>);
    if (whole_lines(p.dxs, (size_t)pieces * 16)) return run(gather_kernel<F32, ADD_F32, OUT_F32, true, true>);
    return run(gather_kernel<F32, ADD_F32, OUT_F32, true, false>);
}

}  // namespace

hipError_t launch_dispatch_backward(const DispatchProblem& p, hipStream_t s) {
    if (p.dxs_f32) {
        if (p.add_f32) return p.dx_f32 ? gather<true, true, true>(p, s) : gather<true, true, false>(p, s);
        return p.dx_f32 ? gather<true, false, true>(p, s) : gather<true, false, false>(p, s);
    }
    if (p.add_f32) return p.dx_f32 ? gather<false, true, true>(p, s) : gather<false, true, false>(p, s);
    return p.dx_f32 ? gather<false, false, true>(p, s) : gather<false, false, false>(p, s);
}

namespace {

template <int Y, bool D_F32, bool DY_F32>
hipError_t combine_grad(const CombineGradProblem& p, hipStream_t s) {
    const long n = (long)p.T * p.k;
    constexpr int C = D_F32 || DY_F32 || Y == kYF32 ? 4 : 8;   // as in the kernel
    const int split = n <= 4L * device_cu_count() && p.H > kAhead * kWave * C ? 2 : 1;
    static_assert(kGradWaves * 64 == 256, "kMostBlocks counts such workgroups");
    const auto run = [&](auto* kernel) {
        for (long f = 0; f < n; f += kMostBlocks * kGradWaves / split) {
            const long blocks = std::min(((n - f) * split + kGradWaves - 1) / kGradWaves, kMostBlocks);
            kernel<<<dim3((unsigned)blocks), dim3(kGradWaves * 64), 0, s>>>(p.dout, p.y, p.y_scale, p.dest, p.w, f, n, p.k, p.H,
                                                                           p.R, p.dy, p.dw);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    const bool nt = (!p.dy || whole_lines(p.dy, (size_t)p.H * (DY_F32 ? 4 : 2))) &&
                    (Y == kYNone || Y == kYE4m3 || whole_lines(p.y, (size_t)p.H * (Y == kYF32 ? 4 : 2)));
    if (split == 2) return run(nt ? combine_grad_kernel<Y, D_F32, DY_F32, true, 2> : combine_grad_kernel<Y, D_F32, DY_F32, false, 2>);
    return run(nt ? combine_grad_kernel<Y, D_F32, DY_F32, true, 1> : combine_grad_kernel<Y, D_F32, DY_F32, false, 1>);
}

template <int Y>
hipError_t combine_grad(const CombineGradProblem& p, hipStream_t s) {
    if (p.dout_f32) return p.dy_f32 ? combine_grad<Y, true, true>(p, s) : combine_grad<Y, true, false>(p, s);
    return p.dy_f32 ? combine_grad<Y, false, true>(p, s) : combine_grad<Y, false, false>(p, s);
}

}  // namespace

hipError_t launch_combine_backward(const CombineGradProblem& p, hipStream_t s) {
    if (!p.dw) return combine_grad<kYNone>(p, s);
    if (p.y_mode == 0) return combine_grad<kYF32>(p, s);
    if (p.y_mode == 1) return combine_grad<kYBf16>(p, s);
    return combine_grad<kYE4m3>(p, s);
}

}  // namespace moe
