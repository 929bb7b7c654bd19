// The norm step between two blocks of a layer (moe_norm):
//   n = rmsnorm(y) * post_w   (n = y without post_w)
//   r = res_scale * res + gate * n
//   x = rmsnorm(r) * pre_w, as fp32, bf16 or int8 codes with one scale per row
// Memory-bound: y and res are read once, r and x written once.  A row stays in
// the registers of its threads between the two norms (both means are sums
// over the whole row), in fp32; r enters the second norm before it is rounded to
// its stored type.  A worker (the threads that share a row) takes a run of
// consecutive rows: the weights are read once a run (at 7168 columns of fp32 they
// are as many bytes as a row's own), and the next row's y and res are on their way
// while a row is reduced.  16384 x 7168 with fp32 r: 282 us, 5.0 TB/s (half of the bytes
// are writes; a copy reaches 4.9).  128 rows: 5 us, the latency of one row.
#include "norm_row.h"

namespace moe {
namespace norm {

template <int TPR, int NV, bool WIDE, bool RAGGED>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormProblem P, int rows_per_worker) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kWorkers = kThreads / TPR;
    typedef Raw<WIDE> Row;
    __shared__ __attribute__((aligned(16))) float slot[kThreads / 16 * 4];
    int turn = 0;
    const int t = threadIdx.x % TPR;
    const int H = P.H;
    const long first = ((long)blockIdx.x * kWorkers + threadIdx.x / TPR) * rows_per_worker;
    auto col = [&](int v) { return (v * TPR + t) * kVec; };
    auto fetch = [&](long row, Row(&y)[NV], Row(&r)[NV]) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int in = row < P.T ? H - col(v) : 0;
            const size_t at = (size_t)(row < P.T ? row : 0) * H + col(v);
            y[v] = load<WIDE, RAGGED>(P.y, P.y_f32, at, in);
            r[v] = load<WIDE, RAGGED>(P.res, P.r_f32, at, P.res ? in : 0);
        }
    };

    Row yr[NV], rr[NV];
    float pw[NV][kVec], gw[NV][kVec], xw[NV][kVec];
    fetch(first, yr, rr);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        weights<RAGGED>(P.post_w, P.w_f32, col(v), H - col(v), pw[v]);
        weights<RAGGED>(P.pre_w, P.w_f32, col(v), H - col(v), xw[v]);
        weights<RAGGED>(nullptr, 0, 0, 0, gw[v]);
    }
    // every worker of the workgroup makes the same number of turns (barriers)
    for (int i = 0; i < rows_per_worker; ++i) {
        const long row = first + i;
        const bool live = row < P.T;
        if (TPR == 64 && !live) return;   // a wave alone: no barriers
        const size_t at0 = (size_t)(live ? row : 0) * H;
        if (P.gate && live && (i == 0 || row % P.gate_div == 0)) {
            const size_t g0 = (size_t)(row / P.gate_div) * H;
#pragma unroll
            for (int v = 0; v < NV; ++v) weights<RAGGED>(P.gate, P.w_f32, g0 + col(v), H - col(v), gw[v]);
        }
        float n[NV][kVec], r[NV][kVec];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            unpack(yr[v], P.y_f32, n[v]);
            unpack(rr[v], P.r_f32, r[v]);
        }
        if (i + 1 < rows_per_worker) fetch(row + 1, yr, rr);
        float p = 1.0f;
        if (P.post_w) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < kVec; ++e) ss[0] = __builtin_fmaf(n[v][e], n[v][e], ss[0]);
            row_reduce<TPR, 1>(ss, slot, turn);
            p = 1.0f / sqrtf(ss[0] / (float)H + P.eps);
        }
        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                n[v][e] = __builtin_fmaf(P.res_scale, r[v][e], n[v][e] * p * pw[v][e] * gw[v][e]);
                ss[0] = __builtin_fmaf(n[v][e], n[v][e], ss[0]);
            }
            if (P.r_out && live && col(v) < H) store<RAGGED>(P.r_out, P.r_f32, at0 + col(v), n[v], H - col(v));
        }
        if (!P.x_out) continue;
        row_reduce<TPR, 1>(ss, slot, turn);
        const float q = 1.0f / sqrtf(ss[0] / (float)H + P.eps);
        float amax[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                n[v][e] = n[v][e] * q * xw[v][e];
                if (P.x_scale) amax[0] = max_magnitude(amax[0], fabsf(n[v][e]));
            }
            if (!P.x_scale && live && col(v) < H) store<RAGGED>(P.x_out, P.x_f32, at0 + col(v), n[v], H - col(v));
        }
        if (!P.x_scale) continue;
        row_reduce<TPR, 1, true>(amax, slot, turn);
        const float s = i8_scale(amax[0]), inv = 1.0f / s;
        if (live && t == 0) P.x_scale[row] = s;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!live || col(v) >= H) continue;
            int8_t* o = (int8_t*)P.x_out + at0 + col(v);
            if (!RAGGED) {
                *(uint2*)o = i8_codes8(n[v], s, inv);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (col(v) + e < H) o[e] = (int8_t)i8_code(n[v][e], s);
            }
        }
    }
}

}  // namespace norm

hipError_t launch_norm(const NormProblem& p, hipStream_t s) {
    using namespace norm;
    const bool ragged = p.H % kVec || !rows16(p.y) || !rows16(p.res) || !rows16(p.post_w) || !rows16(p.gate) ||
                        !rows16(p.pre_w) || !rows16(p.r_out) || ((uintptr_t)p.x_out & (p.x_scale ? 7u : 15u));
    const bool wide = p.y_f32 || (p.res && p.r_f32);
    const int units = (p.H + kVec - 1) / kVec;
    // The narrowest shape that holds a row; runs that give every CU PERCU workgroups, or one row each.
    // Half-empty shapes cost: 16384 x 1024 in bf16 26 us in 128 threads a row and 37.5 in 256,
    // 8192 x 2560 31 in 256 threads of two chunks and 50 in 512.
#define Y(TPR, NV, WIDE, RAGGED, PERCU)                                                                  \
    if (ragged == RAGGED && wide == WIDE && units <= TPR * NV) {                                         \
        constexpr int threads = TPR < 256 ? 256 : TPR, workers = threads / TPR;                          \
        const long most = (long)PERCU * 256 * workers;                                                   \
        const int run = (int)((p.T + most - 1) / most);                                                  \
        const unsigned grid = (unsigned)(((long)p.T + (long)run * workers - 1) / ((long)run * workers)); \
        norm_kernel<TPR, NV, WIDE, RAGGED><<<dim3(grid), dim3(threads), 0, s>>>(p, run);                 \
        return hipGetLastError();                                                                        \
    }
#define X(TPR, NV, PERCU) \
    Y(TPR, NV, false, false, PERCU) Y(TPR, NV, true, false, PERCU) Y(TPR, NV, false, true, PERCU) Y(TPR, NV, true, true, PERCU)
    X(64, 1, 8) X(128, 1, 8) X(256, 1, 8) X(256, 2, 4) X(512, 2, 2) X(1024, 2, 1)
#undef X
#undef Y
    return hipErrorInvalidValue;
}

}  // namespace moe
