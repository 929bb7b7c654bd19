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
// do not depend on timing.  Gates shorter than a run lie within one run, which
// writes their gradients itself.
//
// dy and dres are stored past the caches, where they would push out rows that
// are still to be read: 4096 x 7168 in bf16, 80 us against 87 (the forward step is
// 41 us against 49 with such stores and does without).
#include <algorithm>

#include "norm_row.h"

namespace moe {
namespace norm {

struct Runs {
    int rows;       // rows of a run
    int workers;
    int gate_div;
    int shared;     // gates longer than a run: summed over the runs; else a run holds whole gates
};

inline Runs runs_of(int T, int gate_div, int want_workers) {
    Runs r;
    r.gate_div = gate_div;
    r.rows = (int)(((long)T + want_workers - 1) / want_workers);
    r.shared = gate_div >= r.rows;
    if (!r.shared) r.rows = r.rows / gate_div * gate_div;
    r.workers = (int)(((long)T + r.rows - 1) / r.rows);
    return r;
}

template <int TPR, int NV, bool WIDE, bool RAGGED>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_grad_kernel(NormProblem P, Runs R, float* __restrict__ part_pre,
                                                                          float* __restrict__ part_post,
                                                                          float* __restrict__ part_gate) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kWorkers = kThreads / TPR;
    __shared__ __attribute__((aligned(16))) float slot[kThreads / 16 * 4];
    int turn = 0;
    const int t = threadIdx.x % TPR;
    const long wk = (long)blockIdx.x * kWorkers + threadIdx.x / TPR;
    const int H = P.H;
    auto col = [&](int v) { return (v * TPR + t) * kVec; };
    // the worker's rows [first, end)
    const long first = wk * R.rows, end = min(first + R.rows, (long)P.T);
    // sums over the rows: dx xh; and d yh of the rows since the gate last changed,
    // from which both dgate (times post_w) and dpost_w (times the gate) follow
    float pre[NV][kVec], post[NV][kVec], dyh[NV][kVec];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < kVec; ++e) pre[v][e] = post[v][e] = dyh[v][e] = 0.0f;

    // the next row's loads go out once this row's registers are free, where the
    // registers suffice
    constexpr bool kAhead = !(WIDE && NV > 1);
    typedef Raw<WIDE> Row;
    float pw[NV][kVec], gw[NV][kVec], xw[NV][kVec];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        weights<RAGGED>(P.post_w, P.w_f32, col(v), H - col(v), pw[v]);
        weights<RAGGED>(P.pre_w, P.w_f32, col(v), H - col(v), xw[v]);
        weights<RAGGED>(nullptr, 0, 0, 0, gw[v]);
    }
    const float inv_h = 1.0f / (float)H;
    Row dxr[NV], rr[NV], drr[NV], yr[NV];
    auto fetch = [&](long row) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int in = row < end ? H - col(v) : 0;
            const size_t at = (size_t)(row < end ? row : 0) * H + col(v);
            dxr[v] = load<WIDE, RAGGED>(P.dx, P.x_f32, at, P.dx ? in : 0);
            rr[v] = load<WIDE, RAGGED>(P.r, P.r_f32, at, P.dx ? in : 0);
            drr[v] = load<WIDE, RAGGED>(P.dr, P.r_f32, at, P.dr ? in : 0);
            yr[v] = load<WIDE, RAGGED>(P.y, P.y_f32, at, P.y ? in : 0);
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
            for (int v = 0; v < NV; ++v) weights<RAGGED>(P.gate, P.w_f32, g0 + col(v), H - col(v), gw[v]);
        }
        // absent weights are ones, absent gradients and rows zeros: one formula for all.
        // The rows that a run lacks at its end take an eps of their own: with P.eps = 0 their
        // 1 / rms would be infinite, and its products with their zeros NaN in the sums
        const float eps = live ? P.eps : 1.0f;
        float d[NV][kVec], y[NV][kVec];
        float q = 0.0f, c = 0.0f;   // 1 / rms(r), mean(dx pre_w r) / rms(r)^3
        if (P.dx) {
            float sum[2] = {0.0f, 0.0f};   // r r, dx pre_w r
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float dx[kVec], r[kVec];
                unpack(dxr[v], P.x_f32, dx);
                unpack(rr[v], P.r_f32, r);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    sum[0] = __builtin_fmaf(r[e], r[e], sum[0]);
                    sum[1] = __builtin_fmaf(dx[e] * xw[v][e], r[e], sum[1]);
                }
            }
            row_reduce<TPR, 2>(sum, slot, turn);
            q = 1.0f / sqrtf(sum[0] * inv_h + eps);
            c = sum[1] * inv_h * q * q * q;
        }
        float sy[2] = {0.0f, 0.0f};   // y y, dn post_w y
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float dx[kVec], r[kVec];
            unpack(dxr[v], P.x_f32, dx);
            unpack(rr[v], P.r_f32, r);
            unpack(drr[v], P.r_f32, d[v]);
            unpack(yr[v], P.y_f32, y[v]);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                pre[v][e] = __builtin_fmaf(dx[e] * q, r[e], pre[v][e]);
                d[v][e] = __builtin_fmaf(q, dx[e] * xw[v][e], __builtin_fmaf(-c, r[e], d[v][e]));
                sy[0] = __builtin_fmaf(y[v][e], y[v][e], sy[0]);
                sy[1] = __builtin_fmaf(gw[v][e] * d[v][e] * pw[v][e], y[v][e], sy[1]);
            }
            if (P.dres && live && col(v) < H) {
                float o[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) o[e] = P.res_scale * d[v][e];
                store<RAGGED, true>(P.dres, P.r_f32, at0 + col(v), o, H - col(v));
            }
        }
        if (kAhead && i + 1 < R.rows) fetch(row + 1);
        float p = 1.0f, b = 0.0f;   // 1 / rms(y), mean(dn post_w y) / rms(y)^3
        if (P.post_w) {
            row_reduce<TPR, 2>(sy, slot, turn);
            p = 1.0f / sqrtf(sy[0] * inv_h + eps);
            b = sy[1] * inv_h * p * p * p;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float o[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                dyh[v][e] = __builtin_fmaf(d[v][e], y[v][e] * p, dyh[v][e]);
                o[e] = __builtin_fmaf(p, gw[v][e] * d[v][e] * pw[v][e], -b * y[v][e]);
            }
            if (P.dy && live && col(v) < H) store<RAGGED, true>(P.dy, P.y_f32, at0 + col(v), o, H - col(v));
        }
        if (live && (row + 1 == end || (P.gate && (row + 1) % P.gate_div == 0))) {
            // the gate's last row here: its gradient, or this run's share of it
            // (a run meets at most two gates that are longer than itself)
            float* to = !P.dgate ? nullptr
                        : R.shared ? part_gate + (size_t)(2 * wk + (row / P.gate_div != first / P.gate_div)) * H
                                   : P.dgate + (size_t)(row / P.gate_div) * H;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float o[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    o[e] = pw[v][e] * dyh[v][e];
                    post[v][e] = __builtin_fmaf(gw[v][e], dyh[v][e], post[v][e]);
                    dyh[v][e] = 0.0f;
                }
                if (to && col(v) < H) store<RAGGED>(to, 1, (size_t)col(v), o, H - col(v));
            }
        }
    }
    if (wk < R.workers)
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (col(v) < H) {
                const size_t at = (size_t)wk * H + col(v);
                if (part_pre) store<RAGGED>(part_pre, 1, at, pre[v], H - col(v));
                if (part_post) store<RAGGED>(part_post, 1, at, post[v], H - col(v));
            }
}

// Sums of the runs, in an order that depends on the sizes alone: for each
// column of the pre weights and of the post weights all runs, for each column of
// a gate the runs that meet it.  A workgroup takes 512 / slices columns, its
// slices share out the runs: 16 for the weights and for gates of many runs, one
// for gates of a few (32 gates of 128 rows in 7168 columns would otherwise be 7168
// workgroups with one load a thread).
constexpr int kSumThreads = 512, kSlices = 16;
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(int T, int H, Runs R, int gate_slices,
                                                               const float* __restrict__ part_pre,
                                                               const float* __restrict__ part_post,
                                                               const float* __restrict__ part_gate,
                                                               float* __restrict__ dpre, float* __restrict__ dpost,
                                                               float* __restrict__ dgate) {
    __shared__ float sums[kSumThreads];
    const int weight_blocks = (H + kSumThreads / kSlices - 1) / (kSumThreads / kSlices);
    const bool is_gate = (int)blockIdx.x >= 2 * weight_blocks;
    const int slices = is_gate ? gate_slices : kSlices, cols = kSumThreads / slices;
    const int blocks = (H + cols - 1) / cols;
    const int at = is_gate ? blockIdx.x - 2 * weight_blocks : blockIdx.x;
    const int what = at / blocks;   // gate, or 0 pre weights, 1 post weights
    const int c = threadIdx.x % cols, sl = threadIdx.x / cols;
    const int col = at % blocks * cols + c;
    const float* part = is_gate ? part_gate : what == 0 ? part_pre : part_post;
    if (!part) return;   // the same in the whole workgroup
    float* out = is_gate ? dgate + (size_t)what * H : what == 0 ? dpre : dpost;
    const long lo = is_gate ? (long)what * R.gate_div : 0, hi = is_gate ? min(lo + R.gate_div, (long)T) : T;
    const int w0 = (int)(lo / R.rows), w1 = (int)((hi + R.rows - 1) / R.rows);
    float s = 0.0f;
    if (col < H)
#pragma unroll 8
        for (int w = w0 + sl; w < w1; w += slices) {
            // a run that begins before the gate holds it in its second place
            const size_t place = is_gate ? (size_t)2 * w + ((long)w * R.rows < lo) : (size_t)w;
            s += part[place * H + col];
        }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (sl == 0 && col < H) {
        for (int i = 1; i < slices; ++i) s += sums[i * cols + c];
        out[col] = s;
    }
}

// Runs to aim for: one for each of the 256 CUs where a row takes 512 threads or more,
// two where it takes 256.  Where it takes a wave or two, their own time for a row
// (1.5 us) counts: four runs a CU and up to eight of 16 rows or more, as far as the
// sums of that many runs (as many bytes as two rows each) cost less.  bf16: 16384 x 512
// 35 us with 1024 runs and 52 with 512, 2048 x 512 16.7 and 15.0, 65536 x 128 98 and 178,
// 67 with 2048; 16384 x 1024 52 with 1024 and 63 with 512 (75 in 256 threads a row, half of
// them idle).
inline int want_workers(int threads_per_row, int T) {
    if (threads_per_row > 128) return threads_per_row >= 512 ? 256 : 512;
    return std::max(512, std::min({T / 4, std::max(1024, T / 16), 2048}));
}

// Threads per row and chunks per thread: the row, the weights and the gradients
// of its columns stay in registers up to 8192 columns.  Beyond, 1024 threads have 128
// registers each, which do not hold them, and the rest goes through scratch memory:
// 2048 x 16384 in bf16 315 us, 1.3 TB/s, where 4096 x 7168 has 4.2.
struct Shape {
    int tpr, nv;
};
inline Shape shape_of(int H) {
    const int units = (H + kVec - 1) / kVec;
    return units <= 64 ? Shape{64, 1} : units <= 128 ? Shape{128, 1} : units <= 256 ? Shape{256, 1} : units <= 1024 ? Shape{512, 2} : Shape{1024, 2};
}

inline int gate_rows(const NormProblem& p) { return p.gate ? (p.gate_div < p.T ? p.gate_div : p.T) : (p.T > 0 ? p.T : 1); }

}  // namespace norm

size_t norm_backward_ws_bytes(int T, int H, int gate_div) {
    using namespace norm;
    if (T <= 0) return 0;
    const Runs r = runs_of(T, gate_div > 0 && gate_div < T ? gate_div : T, want_workers(shape_of(H).tpr, T));
    return 4 * align256((size_t)r.workers * H * 4);   // pre, post, two places for gates
}

hipError_t launch_norm_backward(const NormProblem& p0, void* ws, hipStream_t s) {
    using namespace norm;
    NormProblem p = p0;
    const int gd = gate_rows(p);
    p.gate_div = gd;
    Runs R{1, 0, 1, 0};
    float *pre = nullptr, *post = nullptr, *gate = nullptr;
    if (p.T > 0) {
        const bool ragged = p.H % kVec || !rows16(p.dx) || !rows16(p.dr) || !rows16(p.y) || !rows16(p.r) ||
                            !rows16(p.post_w) || !rows16(p.gate) || !rows16(p.pre_w) || !rows16(p.dy) || !rows16(p.dres) ||
                            !rows16(p.dgate);
        const bool wide = p.y_f32 || p.r_f32 || (p.dx && p.x_f32);
        const Shape sh = shape_of(p.H);
        R = runs_of(p.T, gd, want_workers(sh.tpr, p.T));
        const size_t step = align256((size_t)R.workers * p.H * 4);
        if (p.dpre_w) pre = (float*)ws;
        if (p.dpost_w) post = (float*)((uint8_t*)ws + step);
        if (p.dgate && R.shared) gate = (float*)((uint8_t*)ws + 2 * step);
        const int threads = sh.tpr < 256 ? 256 : sh.tpr, per = threads / sh.tpr;
        const unsigned grid = (unsigned)((R.workers + per - 1) / per);
#define Y(TPR, NV, WIDE, RAGGED)                                      \
    if (sh.tpr == TPR && wide == WIDE && ragged == RAGGED)            \
        norm_grad_kernel<TPR, NV, WIDE, RAGGED><<<dim3(grid), dim3(threads), 0, s>>>(p, R, pre, post, gate);
#define X(TPR, NV) Y(TPR, NV, false, false) Y(TPR, NV, true, false) Y(TPR, NV, false, true) Y(TPR, NV, true, true)
        X(64, 1) X(128, 1) X(256, 1) X(512, 2) X(1024, 2)
#undef X
#undef Y
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else {
        // no rows: the parameter gradients are zero
        pre = p.dpre_w;
        post = p.dpost_w;
    }
    if (!pre && !post && !gate) return hipSuccess;
    const long gates = gate ? ((long)p.T + gd - 1) / gd : 0;
    const int slices = gd / R.rows > 32 ? kSlices : 1;
    auto blocks = [&](int sl) { return ((long)p.H + kSumThreads / sl - 1) / (kSumThreads / sl); };
    const long grid = 2 * blocks(kSlices) + gates * blocks(slices);
    norm_sum_kernel<<<dim3((unsigned)grid), dim3(kSumThreads), 0, s>>>(p.T, p.H, R, slices, pre, post, gate, p.dpre_w,
                                                                       p.dpost_w, p.dgate);
    return hipGetLastError();
}

}  // namespace moe
