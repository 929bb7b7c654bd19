// The norm step between two blocks of a layer (moe_norm):
//   n = rmsnorm(y) * post_w   (n = y without post_w)
//   r = res_scale * res + gate * n
//   x = rmsnorm(r) * pre_w, as fp32, bf16 or int8 codes with one scale per row
// Memory-bound: y and res are read once, r and x written once.  A row stays in
// the registers of its threads between the two norms (both means are sums
// over the whole row), in fp32; r enters the second norm before it is rounded to
// its stored type.
#include "norm_row.h"

namespace moe {
namespace norm {

template <int TPR, int NV, int VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormProblem P) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
    __shared__ float slot[kThreads / 64 * 4];
    int turn = 0;
    const int t = threadIdx.x % TPR;
    const long row = (long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = row < P.T;   // rows past the end take part in the barriers only
    const int H = P.H;
    const size_t at0 = (size_t)(live ? row : 0) * H;
    auto col = [&](int v) { return (v * TPR + t) * VEC; };

    Raw<VEC> yr[NV], rr[NV], pw[NV], gw[NV], xw[NV];
    const size_t gate0 = P.gate ? (size_t)((live ? row : 0) / P.gate_div) * H : 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const bool in = live && col(v) < H;
        yr[v] = load<VEC>(P.y, P.y_f32, at0 + col(v), in);
        rr[v] = load<VEC>(P.res, P.r_f32, at0 + col(v), in && P.res);
        pw[v] = load<VEC>(P.post_w, P.w_f32, col(v), in && P.post_w);
        gw[v] = load<VEC>(P.gate, P.w_f32, gate0 + col(v), in && P.gate);
        xw[v] = load<VEC>(P.pre_w, P.w_f32, col(v), in && P.pre_w);
    }
    float n[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) unpack<VEC>(yr[v], P.y_f32, n[v]);
    if (P.post_w) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss[0] = __builtin_fmaf(n[v][e], n[v][e], ss[0]);
        row_reduce<TPR, 1>(ss, slot, turn);
        const float q = 1.0f / sqrtf(ss[0] / (float)H + P.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w[VEC];
            unpack<VEC>(pw[v], P.w_f32, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) n[v][e] = n[v][e] * q * w[e];
        }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float r[VEC], g[VEC];
        unpack<VEC>(rr[v], P.r_f32, r);
        unpack<VEC>(gw[v], P.w_f32, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            n[v][e] = __builtin_fmaf(P.res_scale, r[e], P.gate ? g[e] * n[v][e] : n[v][e]);
            ss[0] = __builtin_fmaf(n[v][e], n[v][e], ss[0]);
        }
        if (P.r_out && live && col(v) < H) store<VEC>(P.r_out, P.r_f32, at0 + col(v), n[v]);
    }
    if (!P.x_out) return;
    row_reduce<TPR, 1>(ss, slot, turn);
    const float q = 1.0f / sqrtf(ss[0] / (float)H + P.eps);
    float amax[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float w[VEC];
        unpack<VEC>(xw[v], P.w_f32, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            n[v][e] = n[v][e] * q * (P.pre_w ? w[e] : 1.0f);
            amax[0] = fmaxf(amax[0], fabsf(n[v][e]));
        }
        if (!P.x_scale && live && col(v) < H) store<VEC>(P.x_out, P.x_f32, at0 + col(v), n[v]);
    }
    if (!P.x_scale) return;
    row_reduce<TPR, 1, true>(amax, slot, turn);
    const float s = i8_scale(amax[0]);
    if (live && t == 0) P.x_scale[row] = s;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (!live || col(v) >= H) continue;
        int8_t* o = (int8_t*)P.x_out + at0 + col(v);
        if constexpr (VEC == 8) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e / 4] |= i8_code(n[v][e], s) << (8 * (e % 4));
            *(uint2*)o = make_uint2(w[0], w[1]);
        } else {
            *o = (int8_t)i8_code(n[v][0], s);
        }
    }
}

}  // namespace norm

hipError_t launch_norm(const NormProblem& p, hipStream_t s) {
    using namespace norm;
    const bool vec = p.H % 8 == 0 && rows16(p.y) && rows16(p.res) && rows16(p.post_w) && rows16(p.gate) &&
                     rows16(p.pre_w) && rows16(p.r_out) && ((uintptr_t)p.x_out & (p.x_scale ? 7u : 15u)) == 0;
    const int units = vec ? p.H / 8 : p.H;
    // the narrowest shape that holds a row
#define X(TPR, NV, VEC)                                                                                    \
    if (vec == (VEC == 8) && units <= TPR * NV) {                                                          \
        constexpr int threads = TPR < 256 ? 256 : TPR, rows = threads / TPR;                               \
        const unsigned grid = (unsigned)(((long)p.T + rows - 1) / rows);                                   \
        norm_kernel<TPR, NV, VEC><<<dim3(grid), dim3(threads), 0, s>>>(p);                                 \
        return hipGetLastError();                                                                          \
    }
    X(64, 1, 8) X(256, 1, 8) X(256, 2, 8) X(256, 4, 8) X(1024, 2, 8)
    X(64, 1, 1) X(256, 1, 1) X(256, 4, 1) X(1024, 4, 1) X(1024, 16, 1)
#undef X
    return hipErrorInvalidValue;
}

}  // namespace moe
