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

inline Runs runs_of(int T, int gate_div, int want_workers) {
    Runs r;
    const int c = (int)(((long)T + want_workers - 1) / want_workers);
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

template <int TPR, int NV, int VEC, bool WIDE>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_grad_kernel(NormProblem P, Runs R, float* __restrict__ part_pre,
                                                                          float* __restrict__ part_post,
                                                                          float* __restrict__ part_gate) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kWorkers = kThreads / TPR;
    __shared__ __attribute__((aligned(16))) float slot[kThreads / 16 * 4];
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
    // sums over the rows: dx xh; and d yh of the rows since the gate last changed,
    // from which both dgate (times post_w) and dpost_w (times the gate) follow
    float pre[NV][VEC], post[NV][VEC], dyh[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) pre[v][e] = post[v][e] = dyh[v][e] = 0.0f;

    // the next row's loads go out once this row's registers are free, where the
    // registers suffice
    constexpr bool kAhead = !(WIDE && NV * VEC > 8);
    typedef Raw<VEC, WIDE> Row;
    float pw[NV][VEC], gw[NV][VEC], xw[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const bool in = col(v) < H;
        weights<VEC>(P.post_w, P.w_f32, col(v), in, pw[v]);
        weights<VEC>(P.pre_w, P.w_f32, col(v), in, xw[v]);
        weights<VEC>(nullptr, 0, 0, false, gw[v]);
    }
    const float inv_h = 1.0f / (float)H;
    Row dxr[NV], rr[NV], drr[NV], yr[NV];
    auto fetch = [&](long row) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool in = row < end && col(v) < H;
            const size_t at = (size_t)(in ? row : 0) * H + col(v);
            dxr[v] = load<VEC, WIDE>(P.dx, P.x_f32, at, in && P.dx);
            rr[v] = load<VEC, WIDE>(P.r, P.r_f32, at, in && P.dx);
            drr[v] = load<VEC, WIDE>(P.dr, P.r_f32, at, in && P.dr);
            yr[v] = load<VEC, WIDE>(P.y, P.y_f32, at, in && P.y);
        }
    };
    if (kAhead) fetch(first);
    // every worker of the workgroup makes the same number of turns (barriers)
    for (int i = 0; i < R.rows; ++i) {
        const long row = first + i;
        const bool live = row < end;
        if (!kAhead) fetch(row);
        const size_t at0 = (size_t)(live ? row : 0) * H;
        if (P.gate && live && (i == 0 || row % P.gate_div == 0)) {
            const size_t g0 = (size_t)(row / P.gate_div) * H;
#pragma unroll
            for (int v = 0; v < NV; ++v) weights<VEC>(P.gate, P.w_f32, g0 + col(v), col(v) < H, gw[v]);
        }
        // absent weights are ones, absent gradients and rows zeros: one formula for all
        float d[NV][VEC], y[NV][VEC];
        float q = 0.0f, c = 0.0f;   // 1 / rms(r), mean(dx pre_w r) / rms(r)^3
        if (P.dx) {
            float sum[2] = {0.0f, 0.0f};   // r r, dx pre_w r
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float dx[VEC], r[VEC];
                unpack(dxr[v], P.x_f32, dx);
                unpack(rr[v], P.r_f32, r);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    sum[0] = __builtin_fmaf(r[e], r[e], sum[0]);
                    sum[1] = __builtin_fmaf(dx[e] * xw[v][e], r[e], sum[1]);
                }
            }
            row_reduce<TPR, 2>(sum, slot, turn);
            q = 1.0f / sqrtf(sum[0] * inv_h + P.eps);
            c = sum[1] * inv_h * q * q * q;
        }
        float sy[2] = {0.0f, 0.0f};   // y y, dn post_w y
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float dx[VEC], r[VEC];
            unpack(dxr[v], P.x_f32, dx);
            unpack(rr[v], P.r_f32, r);
            unpack(drr[v], P.r_f32, d[v]);
            unpack(yr[v], P.y_f32, y[v]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                pre[v][e] = __builtin_fmaf(dx[e] * q, r[e], pre[v][e]);
                d[v][e] = __builtin_fmaf(q, dx[e] * xw[v][e], __builtin_fmaf(-c, r[e], d[v][e]));
                sy[0] = __builtin_fmaf(y[v][e], y[v][e], sy[0]);
                sy[1] = __builtin_fmaf(gw[v][e] * d[v][e] * pw[v][e], y[v][e], sy[1]);
            }
            if (P.dres && live && col(v) < H) {
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = P.res_scale * d[v][e];
                store<VEC>(P.dres, P.r_f32, at0 + col(v), o);
            }
        }
        if (kAhead && i + 1 < R.rows) fetch(row + 1);
        float p = 1.0f, b = 0.0f;   // 1 / rms(y), mean(dn post_w y) / rms(y)^3
        if (P.post_w) {
            row_reduce<TPR, 2>(sy, slot, turn);
            p = 1.0f / sqrtf(sy[0] * inv_h + P.eps);
            b = sy[1] * inv_h * p * p * p;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                dyh[v][e] = __builtin_fmaf(d[v][e], y[v][e] * p, dyh[v][e]);
                o[e] = __builtin_fmaf(p, gw[v][e] * d[v][e] * pw[v][e], -b * y[v][e]);
            }
            if (P.dy && live && col(v) < H) store<VEC>(P.dy, P.y_f32, at0 + col(v), o);
        }
        if (live && (row + 1 == end || (P.gate && (row + 1) % P.gate_div == 0))) {
            // the gate's last row here: its gradient, or this run's share of it
            float* to = !P.dgate ? nullptr : R.per_gate ? part_gate + (size_t)wk * H : P.dgate + (size_t)(row / P.gate_div) * H;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    o[e] = pw[v][e] * dyh[v][e];
                    post[v][e] = __builtin_fmaf(gw[v][e], dyh[v][e], post[v][e]);
                    dyh[v][e] = 0.0f;
                }
                if (to && col(v) < H) store<VEC>(to, 1, (size_t)col(v), o);
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
                if (part_gate && first >= end) store<VEC>(part_gate, 1, at, post[v]);   // no rows: zeros
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
#pragma unroll 8
        for (int w = w0 + sl; w < w1; w += 8) s += part[(size_t)w * H + col];
    sums[sl][c] = s;
    __syncthreads();
    if (sl == 0 && col < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][c];
        out[col] = s;
    }
}

// Runs to aim for: one for each of the 256 CUs where a row takes 512 threads or more,
// else two.
inline int want_workers(int threads_per_row) { return threads_per_row >= 512 ? 256 : 512; }

// Threads per row, chunks per thread and elements per chunk: the row, the
// weights and the gradients of its columns all stay in registers.
struct Shape {
    int tpr, nv;
    bool vec, wide;
};
inline Shape shape_of(int H, bool vec, bool wide) {
    const int units = vec ? H / 8 : H;
    if (units <= 64) return {64, 1, vec, wide};
    if (units <= 256) return {256, 1, vec, wide};
    if (vec) return {units <= 1024 ? 512 : 1024, 2, vec, wide};
    if (units <= 1024) return {1024, 1, vec, wide};
    return {1024, units <= 4096 ? 4 : 16, vec, wide};
}

inline int gate_rows(const NormProblem& p) { return p.gate ? (p.gate_div < p.T ? p.gate_div : p.T) : (p.T > 0 ? p.T : 1); }

// the workers of the widest launch that these sizes may get, whatever the alignment
inline long most_workers(int T, int H, int gate_div) {
    long most = 0;
    for (int vec = 0; vec < 2; ++vec) {
        if (vec && H % 8) continue;
        for (int wide = 0; wide < 2; ++wide) {
            const Runs r = runs_of(T, gate_div, want_workers(shape_of(H, vec, wide).tpr));
            most = r.workers > most ? r.workers : most;
        }
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
    const bool wide = !vec || p.y_f32 || p.r_f32 || p.x_f32;
    const Shape sh = shape_of(p.H, vec, wide);
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
#define X(TPR, NV, VEC, WIDE)                                                                          \
    if (sh.tpr == TPR && sh.nv == NV && (sh.vec ? 8 : 1) == VEC && sh.wide == WIDE)                    \
        norm_grad_kernel<TPR, NV, VEC, WIDE><<<dim3(grid), dim3(threads), 0, s>>>(p, R, pre, post, gate);
        X(64, 1, 8, false) X(64, 1, 8, true) X(256, 1, 8, false) X(256, 1, 8, true)
        X(512, 2, 8, false) X(512, 2, 8, true) X(1024, 2, 8, false) X(1024, 2, 8, true)
        X(64, 1, 1, true) X(256, 1, 1, true) X(1024, 1, 1, true) X(1024, 4, 1, true) X(1024, 16, 1, true)
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
