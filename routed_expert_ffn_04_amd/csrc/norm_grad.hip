// Gradients of the norm step (moe_norm_backward).  With r the stored output of
// the forward step, xh = r / rms(r), yh = y / rms(y):
//   d   = dr + (dx pre_w - xh mean(dx pre_w xh)) / rms(r)         gradient of r
//   dres = res_scale d,   dpre_w = sum_t dx xh
//   dn  = gate d,         dgate  = sum over the gate's rows of d n,   n = yh post_w (or y)
//   dy  = (dn post_w - yh mean(dn post_w yh)) / rms(y)   (dn without post_w),   dpost_w = sum_t dn yh
// Memory-bound: dx, dr, y and r are read once, dy and dres written once.  Each
// worker (the threads that share a row) takes a run of consecutive rows and
// keeps its columns' parameter gradients in fp32 registers; the runs' sums go
// to the workspace and a second kernel adds them in a fixed order, so results
// do not depend on timing.  A run never crosses the end of a gate's rows unless
// it holds whole gates, whose gradients it then writes itself.
#include "norm_row.h"

namespace moe {
namespace norm {

struct Runs {
    int rows;       // rows of a run
    int per_gate;   // runs of one gate's rows; 0: a run holds whole gates
    int workers;
};

// At least `least` rows a run keep the workspace's traffic (three fp32 values
// per column and run, written and read) below that of the rows themselves.
inline Runs runs_of(int T, int gate_div, int want_workers) {
    Runs r;
    const int least = 4;
    int c = (int)(((long)T + want_workers - 1) / want_workers);
    if (c < least) c = least;
    if (gate_div >= c) {
        r.per_gate = (int)(((long)gate_div + c - 1) / c);
        r.rows = (int)(((long)gate_div + r.per_gate - 1) / r.per_gate);
        const long gates = ((long)T + gate_div - 1) / gate_div;
        // the last gate may be short: its runs end with T
        const long tail = T - (gates - 1) * gate_div;
        r.workers = (int)((gates - 1) * r.per_gate + (tail + r.rows - 1) / r.rows);
    } else {
        r.per_gate = 0;
        r.rows = c / gate_div * gate_div;
        r.workers = (int)(((long)T + r.rows - 1) / r.rows);
    }
    return r;
}

template <int TPR, int NV, int VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_grad_kernel(NormProblem P, Runs R, float* __restrict__ part_pre,
                                                                          float* __restrict__ part_post,
                                                                          float* __restrict__ part_gate) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kWorkers = kThreads / TPR;
    __shared__ float slot[kThreads / 64 * 4];
    int turn = 0;
    const int t = threadIdx.x % TPR;
    const long wk = (long)blockIdx.x * kWorkers + threadIdx.x / TPR;
    const int H = P.H;
    auto col = [&](int v) { return (v * TPR + t) * VEC; };
    // the worker's rows [first, end)
    long first = P.T, end = P.T;
    if (wk < R.workers) {
        if (R.per_gate) {
            const long g = wk / R.per_gate;
            first = g * P.gate_div + (wk % R.per_gate) * (long)R.rows;
            end = min(min(first + R.rows, (g + 1) * (long)P.gate_div), (long)P.T);
        } else {
            first = wk * R.rows;
            end = min(first + R.rows, (long)P.T);
        }
    }
    float pre[NV][VEC], post[NV][VEC], gate[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) pre[v][e] = post[v][e] = gate[v][e] = 0.0f;

    Raw<VEC> pw[NV], xw[NV], gw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const bool in = col(v) < H;
        pw[v] = load<VEC>(P.post_w, P.w_f32, col(v), in && P.post_w);
        xw[v] = load<VEC>(P.pre_w, P.w_f32, col(v), in && P.pre_w);
    }
    const float inv_h = 1.0f / (float)H;

    // every worker of the workgroup makes the same number of turns (barriers)
    for (int i = 0; i < R.rows; ++i) {
        const long row = first + i;
        const bool live = row < end;
        const size_t at0 = (size_t)(live ? row : 0) * H;
        if (P.gate && live && (i == 0 || row % P.gate_div == 0)) {
            const size_t g0 = (size_t)(row / P.gate_div) * H;
#pragma unroll
            for (int v = 0; v < NV; ++v) gw[v] = load<VEC>(P.gate, P.w_f32, g0 + col(v), col(v) < H);
        }
        Raw<VEC> dxr[NV], drr[NV], yr[NV], rr[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool in = live && col(v) < H;
            dxr[v] = load<VEC>(P.dx, P.x_f32, at0 + col(v), in && P.dx);
            rr[v] = load<VEC>(P.r, P.r_f32, at0 + col(v), in && P.dx);
            drr[v] = load<VEC>(P.dr, P.r_f32, at0 + col(v), in && P.dr);
            yr[v] = load<VEC>(P.y, P.y_f32, at0 + col(v), in && P.y);
        }
        float d[NV][VEC], y[NV][VEC];
        float sum[2] = {0.0f, 0.0f};   // r r, dx pre_w r
        if (P.dx) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float dx[VEC], r[VEC], w[VEC];
                unpack<VEC>(dxr[v], P.x_f32, dx);
                unpack<VEC>(rr[v], P.r_f32, r);
                unpack<VEC>(xw[v], P.w_f32, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    sum[0] = __builtin_fmaf(r[e], r[e], sum[0]);
                    sum[1] = __builtin_fmaf(dx[e] * (P.pre_w ? w[e] : 1.0f), r[e], sum[1]);
                }
            }
            row_reduce<TPR, 2>(sum, slot, turn);
        }
        const float q = 1.0f / sqrtf(sum[0] * inv_h + P.eps);
        const float c = sum[1] * inv_h * q * q * q;
        float sy[2] = {0.0f, 0.0f};   // y y, dn post_w y
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            unpack<VEC>(drr[v], P.r_f32, d[v]);
            if (P.dx) {
                float dx[VEC], r[VEC], w[VEC];
                unpack<VEC>(dxr[v], P.x_f32, dx);
                unpack<VEC>(rr[v], P.r_f32, r);
                unpack<VEC>(xw[v], P.w_f32, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    pre[v][e] = __builtin_fmaf(dx[e], r[e] * q, pre[v][e]);
                    d[v][e] += q * (dx[e] * (P.pre_w ? w[e] : 1.0f)) - c * r[e];
                }
            }
            if (P.dres && live && col(v) < H) {
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = P.res_scale * d[v][e];
                store<VEC>(P.dres, P.r_f32, at0 + col(v), o);
            }
            float g[VEC], w[VEC];
            unpack<VEC>(yr[v], P.y_f32, y[v]);
            unpack<VEC>(gw[v], P.w_f32, g);
            unpack<VEC>(pw[v], P.w_f32, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // d n without the row's 1 / rms(y): joined below
                if (P.gate && !P.post_w) gate[v][e] = __builtin_fmaf(d[v][e], y[v][e], gate[v][e]);
                if (P.post_w) {
                    const float dn = P.gate ? g[e] * d[v][e] : d[v][e];
                    sy[0] = __builtin_fmaf(y[v][e], y[v][e], sy[0]);
                    sy[1] = __builtin_fmaf(dn * w[e], y[v][e], sy[1]);
                }
            }
        }
        float p = 1.0f, b = 0.0f;
        if (P.post_w) {
            row_reduce<TPR, 2>(sy, slot, turn);
            p = 1.0f / sqrtf(sy[0] * inv_h + P.eps);
            b = sy[1] * inv_h * p * p * p;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float g[VEC], w[VEC], o[VEC];
            unpack<VEC>(gw[v], P.w_f32, g);
            unpack<VEC>(pw[v], P.w_f32, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float dn = P.gate ? g[e] * d[v][e] : d[v][e];
                if (P.post_w) {
                    const float yh = y[v][e] * p;
                    if (P.gate) gate[v][e] = __builtin_fmaf(d[v][e], yh * w[e], gate[v][e]);
                    post[v][e] = __builtin_fmaf(dn, yh, post[v][e]);
                    o[e] = p * (dn * w[e]) - b * y[v][e];
                } else {
                    o[e] = dn;
                }
            }
            if (P.dy && live && col(v) < H) store<VEC>(P.dy, P.y_f32, at0 + col(v), o);
            // the last row of a gate that lies within the run
            if (P.dgate && !R.per_gate && live && ((row + 1) % P.gate_div == 0 || row + 1 == P.T)) {
                if (col(v) < H) store<VEC>(P.dgate, 1, (size_t)(row / P.gate_div) * H + col(v), gate[v]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) gate[v][e] = 0.0f;
            }
        }
    }
    if (wk < R.workers)
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (col(v) < H) {
                const size_t at = (size_t)wk * H + col(v);
                if (part_pre) store<VEC>(part_pre, 1, at, pre[v]);
                if (part_post) store<VEC>(part_post, 1, at, post[v]);
                if (part_gate) store<VEC>(part_gate, 1, at, gate[v]);
            }
}

// Sums of the runs: blockIdx.y = 0 the pre weights (all runs), 1 the post
// weights, 2 + g the runs of gate g.  32 columns x 8 slices of runs a workgroup.
__global__ __launch_bounds__(256) void norm_sum_kernel(int H, Runs R, const float* __restrict__ part_pre,
                                                       const float* __restrict__ part_post,
                                                       const float* __restrict__ part_gate, float* __restrict__ dpre,
                                                       float* __restrict__ dpost, float* __restrict__ dgate) {
    __shared__ float sums[8][33];
    const int c = threadIdx.x % 32, sl = threadIdx.x / 32;
    const long col = (long)blockIdx.x * 32 + c;
    const int what = blockIdx.y;
    const float* part = what == 0 ? part_pre : what == 1 ? part_post : part_gate;
    float* out = what == 0 ? dpre : what == 1 ? dpost : dgate + (size_t)(what - 2) * H;
    if (!part) return;   // the same in the whole workgroup
    const int w0 = what < 2 ? 0 : (what - 2) * R.per_gate;
    const int w1 = what < 2 ? R.workers : min(w0 + R.per_gate, R.workers);
    float s = 0.0f;
    if (col < H)
        for (int w = w0 + sl; w < w1; w += 8) s += part[(size_t)w * H + col];
    sums[sl][c] = s;
    __syncthreads();
    if (sl == 0 && col < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][c];
        out[col] = s;
    }
}

// Runs to aim for: one for each of the 256 CUs where a row takes 1024 threads,
// else two.
inline int want_workers(int threads_per_row) { return threads_per_row >= 1024 ? 256 : 512; }

// Threads per row, chunks per thread and elements per chunk: the row, the
// weights and the gradients of its columns all stay in registers.
struct Shape {
    int tpr, nv;
    bool vec;
};
inline Shape shape_of(int H, bool vec) {
    const int units = vec ? H / 8 : H;
    if (units <= 64) return {64, 1, vec};
    if (units <= 256) return {256, 1, vec};
    if (units <= 1024) return {1024, 1, vec};
    if (vec) return {1024, 2, vec};
    return {1024, units <= 4096 ? 4 : 16, vec};
}

inline int gate_rows(const NormProblem& p) { return p.gate ? (p.gate_div < p.T ? p.gate_div : p.T) : (p.T > 0 ? p.T : 1); }

// the workers of the widest launch that these sizes may get, whatever the alignment
inline long most_workers(int T, int H, int gate_div) {
    long most = 0;
    for (int vec = 0; vec < 2; ++vec) {
        if (vec && H % 8) continue;
        const Runs r = runs_of(T, gate_div, want_workers(shape_of(H, vec).tpr));
        most = r.workers > most ? r.workers : most;
    }
    return most;
}

}  // namespace norm

size_t norm_backward_ws_bytes(int T, int H, int gate_div) {
    if (T <= 0) return 0;
    const int gd = gate_div > 0 && gate_div < T ? gate_div : T;
    return 3 * align256((size_t)norm::most_workers(T, H, gd) * H * 4);
}

hipError_t launch_norm_backward(const NormProblem& p0, void* ws, hipStream_t s) {
    using namespace norm;
    NormProblem p = p0;
    const int gd = gate_rows(p);
    p.gate_div = gd;
    const bool vec = p.H % 8 == 0 && rows16(p.dx) && rows16(p.dr) && rows16(p.y) && rows16(p.r) && rows16(p.post_w) &&
                     rows16(p.gate) && rows16(p.pre_w) && rows16(p.dy) && rows16(p.dres) && rows16(p.dgate);
    const Shape sh = shape_of(p.H, vec);
    Runs R{0, 1, 0};
    float *pre = nullptr, *post = nullptr, *gate = nullptr;
    if (p.T > 0) {
        R = runs_of(p.T, gd, want_workers(sh.tpr));
        const size_t step = align256((size_t)most_workers(p.T, p.H, gd) * p.H * 4);
        if (p.dpre_w) pre = (float*)ws;
        if (p.dpost_w) post = (float*)((uint8_t*)ws + step);
        if (p.dgate && R.per_gate) gate = (float*)((uint8_t*)ws + 2 * step);
        const int threads = sh.tpr < 256 ? 256 : sh.tpr, per = threads / sh.tpr;
        const unsigned grid = (unsigned)((R.workers + per - 1) / per);
#define X(TPR, NV, VEC)                                                                                \
    if (sh.tpr == TPR && sh.nv == NV && (sh.vec ? 8 : 1) == VEC)                                       \
        norm_grad_kernel<TPR, NV, VEC><<<dim3(grid), dim3(threads), 0, s>>>(p, R, pre, post, gate);
        X(64, 1, 8) X(256, 1, 8) X(1024, 1, 8) X(1024, 2, 8)
        X(64, 1, 1) X(256, 1, 1) X(1024, 1, 1) X(1024, 4, 1) X(1024, 16, 1)
#undef X
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else {
        // no rows: the parameter gradients are zero
        pre = p.dpre_w;
        post = p.dpost_w;
    }
    const int gates = gate ? (int)(((long)p.T + gd - 1) / gd) : 0;
    if (!pre && !post && !gate) return hipSuccess;
    norm_sum_kernel<<<dim3((p.H + 31) / 32, 2 + gates), dim3(256), 0, s>>>(p.H, R, pre, post, gate, p.dpre_w, p.dpost_w,
                                                                           p.dgate);
    return hipGetLastError();
}

}  // namespace moe
