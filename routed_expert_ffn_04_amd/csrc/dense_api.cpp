// C ABI of the operators around the mixture-of-experts layer (declarations and
// contracts: include/moe.h): validation and launches; no allocation, no host
// synchronisation.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "api_check.h"
#include "dense.h"
#include "internal.h"

namespace {

using namespace moe::api;

constexpr int kMaxNormH = 16384;
constexpr int kMaxI8K = 131071;   // 128 * 128 * K stays below 2^31

moe_status_t check_norm(const char* name, int32_t T, int32_t H, int32_t y_dt, int32_t r_dt, int32_t w_dt,
                        const void* gate, int32_t gate_div, float res_scale, float eps) {
    if (T < 0 || H <= 0) return fail(MOE_ERR_INVALID, "%s: T=%d H=%d", name, T, H);
    if (H > kMaxNormH) return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d > %d", name, H, kMaxNormH);
    if (!is_float(y_dt) || !is_float(r_dt) || !is_float(w_dt))
        return fail(MOE_ERR_UNSUPPORTED, "%s: dtypes y %d, r %d, weights %d", name, y_dt, r_dt, w_dt);
    if (gate && gate_div <= 0) return fail(MOE_ERR_INVALID, "%s: gate_div=%d", name, gate_div);
    if (!std::isfinite(res_scale) || !std::isfinite(eps) || eps < 0.0f)
        return fail(MOE_ERR_INVALID, "%s: res_scale=%g eps=%g", name, (double)res_scale, (double)eps);
    return MOE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ dense FFN
size_t moe_ffn_workspace_size(int32_t T, int32_t H, int32_t I) {
    if (!dense_sizes(T, H, I)) return 0;
    return or_zero(moe::ffn_ws_bytes(T, H, I));
}

moe_status_t moe_ffn(const void* x, int32_t x_dt, int32_t T, const moe_experts_t* bank, void* y, int32_t y_dt,
                     float* gu, void* ws, size_t ws_bytes, void* stream) {
    moe_status_t st = check_dense(bank, "ffn");
    if (st) return st;
    if (T < 0) return fail(MOE_ERR_INVALID, "ffn: T=%d", T);
    if (T > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "ffn: T=%d > %d", T, kMaxRows);
    if (x_dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "ffn: x dtype %d", x_dt);
    if (!is_float(y_dt)) return fail(MOE_ERR_UNSUPPORTED, "ffn: y dtype %d", y_dt);
    if (T == 0) return MOE_OK;
    if (!x || !y) return fail(MOE_ERR_INVALID, "%s", "ffn: null x or y");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gu, 16))
        return fail(MOE_ERR_INVALID, "%s", "ffn: x, y and gu must be 16-byte aligned");
    const size_t need = moe::ffn_ws_bytes(T, bank->H, bank->I);
    if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "ffn: T=%d H=%d I=%d", T, bank->H, bank->I);
    if (!ws || !aligned(ws, 256) || ws_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "%s", "ffn: workspace");
    moe::FfnProblem p{};
    p.x = x; p.wg = bank->w_gate; p.wu = bank->w_up; p.wd = bank->w_down;
    p.T = T; p.H = bank->H; p.I = bank->I;
    p.y = y; p.y_f32 = y_dt == MOE_F32; p.gu = gu;
    return done(moe::launch_ffn(p, ws, (hipStream_t)stream), "moe_ffn");
}

size_t moe_ffn_backward_workspace_size(int32_t T, int32_t H, int32_t I, int32_t has_gu) {
    if (!dense_sizes(T, H, I)) return 0;
    return or_zero(moe::ffn_backward_ws_bytes(T, H, I, has_gu));
}

moe_status_t moe_ffn_backward(const void* dy, const void* x, int32_t dt, int32_t T, const moe_experts_t* bank,
                              const float* gu, void* dx, void* dw_gate, void* dw_up, void* dw_down, void* ws,
                              size_t ws_bytes, void* stream) {
    moe_status_t st = check_dense(bank, "ffn_backward");
    if (st) return st;
    if (T < 0) return fail(MOE_ERR_INVALID, "ffn_backward: T=%d", T);
    if (T > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "ffn_backward: T=%d > %d", T, kMaxRows);
    if (dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "ffn_backward: dtype %d", dt);
    if (!aligned(dx, 16) || !aligned(dw_gate, 16) || !aligned(dw_up, 16) || !aligned(dw_down, 16) || !aligned(dy, 16) ||
        !aligned(x, 16) || !aligned(gu, 16))
        return fail(MOE_ERR_INVALID, "%s", "ffn_backward: tensors must be 16-byte aligned");
    if (!dx && !dw_gate && !dw_up && !dw_down) return MOE_OK;
    if (T > 0) {
        if (!dy || (!x && reads_x(gu, dw_gate, dw_up))) return fail(MOE_ERR_INVALID, "%s", "ffn_backward: null dy or x");
        const size_t need = moe::ffn_backward_ws_bytes(T, bank->H, bank->I, gu != nullptr);
        if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "ffn_backward: T=%d H=%d I=%d", T, bank->H, bank->I);
        if (!ws || !aligned(ws, 256) || ws_bytes < need)
            return fail(MOE_ERR_WORKSPACE, "%s", "ffn_backward: workspace");
    }
    moe::FfnProblem p{};
    p.x = x; p.wg = bank->w_gate; p.wu = bank->w_up; p.wd = bank->w_down;
    p.T = T; p.H = bank->H; p.I = bank->I;
    p.dy = dy; p.gu_in = gu; p.dx = dx; p.dwg = dw_gate; p.dwu = dw_up; p.dwd = dw_down;
    return done(moe::launch_ffn_backward(p, ws, (hipStream_t)stream), "moe_ffn_backward");
}

// ------------------------------------------------------------------ norm
moe_status_t moe_norm(const void* y, int32_t y_dt, const void* res, int32_t r_dt, int32_t T, int32_t H,
                      const void* post_w, const void* gate, int32_t gate_div, const void* pre_w, int32_t w_dt,
                      float res_scale, float eps, void* r_out, void* x_out, int32_t x_dt, float* x_scale,
                      void* stream) {
    moe_status_t st = check_norm("norm", T, H, y_dt, r_dt, w_dt, gate, gate_div, res_scale, eps);
    if (st) return st;
    if (x_out && !is_float(x_dt) && x_dt != MOE_I8) return fail(MOE_ERR_UNSUPPORTED, "norm: x dtype %d", x_dt);
    if (T == 0) return MOE_OK;
    if (!y || (!r_out && !x_out)) return fail(MOE_ERR_INVALID, "%s", "norm: null y, or neither r nor x wanted");
    const bool i8 = x_out && x_dt == MOE_I8;
    if (i8 && !x_scale) return fail(MOE_ERR_INVALID, "%s", "norm: int8 x without x_scale");
    if (!aligned(y, size_of(y_dt)) || !aligned(res, size_of(r_dt)) || !aligned(r_out, size_of(r_dt)) ||
        (x_out && !i8 && !aligned(x_out, size_of(x_dt))) || !aligned(post_w, size_of(w_dt)) ||
        !aligned(gate, size_of(w_dt)) || !aligned(pre_w, size_of(w_dt)) || (i8 && !aligned(x_scale, 4)))
        return fail(MOE_ERR_INVALID, "%s", "norm: a tensor is not aligned to its elements");
    moe::NormProblem p{};
    p.y = y; p.y_f32 = y_dt == MOE_F32; p.res = res; p.r_f32 = r_dt == MOE_F32; p.T = T; p.H = H;
    p.post_w = post_w; p.gate = gate; p.gate_div = gate ? gate_div : 1; p.pre_w = pre_w; p.w_f32 = w_dt == MOE_F32;
    p.res_scale = res_scale; p.eps = eps;
    p.r_out = r_out; p.x_out = x_out; p.x_f32 = x_dt == MOE_F32; p.x_scale = i8 ? x_scale : nullptr;
    return done(moe::launch_norm(p, (hipStream_t)stream), "moe_norm");
}

size_t moe_norm_backward_workspace_size(int32_t T, int32_t H, int32_t gate_div) {
    if (T < 0 || H <= 0 || H > kMaxNormH) return 0;
    return moe::norm_backward_ws_bytes(T, H, gate_div);
}

moe_status_t moe_norm_backward(const void* dx, int32_t x_dt, const void* dr, const void* y, int32_t y_dt,
                               const void* r, int32_t r_dt, int32_t T, int32_t H, const void* post_w,
                               const void* gate, int32_t gate_div, const void* pre_w, int32_t w_dt, float res_scale,
                               float eps, void* dy, void* dres, float* dpost_w, float* dgate, float* dpre_w, void* ws,
                               size_t ws_bytes, void* stream) {
    moe_status_t st = check_norm("norm_backward", T, H, y_dt, r_dt, w_dt, gate, gate_div, res_scale, eps);
    if (st) return st;
    if (dx && !is_float(x_dt)) return fail(MOE_ERR_UNSUPPORTED, "norm_backward: dx dtype %d", x_dt);
    if (dpost_w && !post_w) return fail(MOE_ERR_INVALID, "%s", "norm_backward: dpost_w without post_w");
    if (dgate && !gate) return fail(MOE_ERR_INVALID, "%s", "norm_backward: dgate without gate");
    if (!aligned(dy, size_of(y_dt)) || !aligned(y, size_of(y_dt)) || !aligned(dres, size_of(r_dt)) ||
        !aligned(dr, size_of(r_dt)) || !aligned(r, size_of(r_dt)) || (dx && !aligned(dx, size_of(x_dt))) ||
        !aligned(post_w, size_of(w_dt)) || !aligned(gate, size_of(w_dt)) || !aligned(pre_w, size_of(w_dt)) ||
        !aligned(dpost_w, 4) || !aligned(dgate, 4) || !aligned(dpre_w, 4))
        return fail(MOE_ERR_INVALID, "%s", "norm_backward: a tensor is not aligned to its elements");
    if (!dy && !dres && !dpost_w && !dgate && !dpre_w) return MOE_OK;
    if (T > 0) {
        if (!dx && !dr) return fail(MOE_ERR_INVALID, "%s", "norm_backward: neither dx nor dr");
        if (dx && !r) return fail(MOE_ERR_INVALID, "%s", "norm_backward: dx without r");
        if (dpre_w && !dx) return fail(MOE_ERR_INVALID, "%s", "norm_backward: dpre_w without dx");
        if ((post_w || gate) && !y) return fail(MOE_ERR_INVALID, "%s", "norm_backward: post_w or gate without y");
        if (!ws || !aligned(ws, 256) || ws_bytes < moe::norm_backward_ws_bytes(T, H, gate ? gate_div : 0))
            return fail(MOE_ERR_WORKSPACE, "%s", "norm_backward: workspace");
    }
    moe::NormProblem p{};
    p.y = y; p.y_f32 = y_dt == MOE_F32; p.r = r; p.r_f32 = r_dt == MOE_F32; p.T = T; p.H = H;
    p.post_w = post_w; p.gate = gate; p.gate_div = gate ? gate_div : 1; p.pre_w = pre_w; p.w_f32 = w_dt == MOE_F32;
    p.res_scale = res_scale; p.eps = eps;
    p.dx = dx; p.x_f32 = x_dt == MOE_F32; p.dr = dr;
    p.dy = dy; p.dres = dres; p.dpost_w = dpost_w; p.dgate = dgate; p.dpre_w = dpre_w;
    return done(moe::launch_norm_backward(p, ws, (hipStream_t)stream), "moe_norm_backward");
}

// ------------------------------------------------------------------ int8
moe_status_t moe_quant_i8(const void* x, int32_t x_dt, int32_t rows, int32_t cols, int8_t* q, float* scale,
                          void* stream) {
    if (rows < 0 || cols <= 0) return fail(MOE_ERR_INVALID, "quant_i8: rows=%d cols=%d", rows, cols);
    if (cols % 16) return fail(MOE_ERR_UNSUPPORTED, "quant_i8: cols=%d not a multiple of 16", cols);
    if (!is_float(x_dt)) return fail(MOE_ERR_UNSUPPORTED, "quant_i8: x dtype %d", x_dt);
    if (rows == 0) return MOE_OK;
    if (!x || !q || !scale) return fail(MOE_ERR_INVALID, "%s", "quant_i8: null pointer");
    if (!aligned(x, 16) || !aligned(q, 8) || !aligned(scale, 4))
        return fail(MOE_ERR_INVALID, "%s", "quant_i8: misaligned x, q or scale");
    return done(moe::launch_quant_i8(x, x_dt == MOE_F32, rows, cols, q, scale, (hipStream_t)stream), "moe_quant_i8");
}

size_t moe_linear_i8_workspace_size(int32_t T, int32_t K, int32_t N) {
    if (T < 0 || K <= 0 || N <= 0 || K % 16 || K > kMaxI8K || T > kMaxRows || N > kMaxRows) return 0;
    return or_zero(moe::linear_i8_ws_bytes(T, K, N));
}

moe_status_t moe_linear_i8(const int8_t* q, const float* q_scale, int32_t T, int32_t K, const int8_t* w,
                           const float* w_scale, const float* bias, int32_t N, void* out, int32_t out_dt, void* ws,
                           size_t ws_bytes, void* stream) {
    if (T < 0 || K <= 0 || N <= 0) return fail(MOE_ERR_INVALID, "linear_i8: T=%d K=%d N=%d", T, K, N);
    if (K % 16 || K > kMaxI8K)
        return fail(MOE_ERR_UNSUPPORTED, "linear_i8: K=%d must be a multiple of 16, at most %d", K, kMaxI8K);
    if (T > kMaxRows || N > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "linear_i8: T=%d N=%d > %d", T, N, kMaxRows);
    if (!is_float(out_dt)) return fail(MOE_ERR_UNSUPPORTED, "linear_i8: out dtype %d", out_dt);
    if (T == 0) return MOE_OK;
    if (!q || !q_scale || !w || !w_scale || !out) return fail(MOE_ERR_INVALID, "%s", "linear_i8: null pointer");
    if (!aligned(q, 16) || !aligned(w, 16) || !aligned(q_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(out, size_of(out_dt)))
        return fail(MOE_ERR_INVALID, "%s", "linear_i8: misaligned tensor");
    const size_t need = moe::linear_i8_ws_bytes(T, K, N);
    if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "linear_i8: T=%d K=%d N=%d", T, K, N);
    if (need && (!ws || !aligned(ws, 256) || ws_bytes < need)) return fail(MOE_ERR_WORKSPACE, "%s", "linear_i8: workspace");
    moe::LinearI8Problem p{};
    p.q = q; p.xs = q_scale; p.w = w; p.ws = w_scale; p.bias = bias; p.T = T; p.K = K; p.N = N;
    p.out = out; p.out_f32 = out_dt == MOE_F32;
    return done(moe::launch_linear_i8(p, ws, (hipStream_t)stream), "moe_linear_i8");
}

}  // extern "C"
