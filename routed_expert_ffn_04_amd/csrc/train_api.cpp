// C ABI of the layer's training step (declarations and contracts: include/moe.h):
// validation and launches; no allocation, no host synchronisation.
#include "moe.h"

#include <hip/hip_runtime.h>

#include "api_check.h"
#include "dense.h"
#include "internal.h"

namespace {

using namespace moe::api;

// What the checkpoint of a row matrix is: codes and exponents, or values.
bool is_i8(int dt) { return dt == MOE_I8; }

moe_status_t check_rows(const char* name, int32_t T, int32_t k, int32_t H, int32_t R) {
    if (T < 0 || k <= 0 || H <= 0 || R < 0) return fail(MOE_ERR_INVALID, "%s: T=%d k=%d H=%d R=%d", name, T, k, H, R);
    if (H % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d not a multiple of 8", name, H);
    if (T > kMaxRows || R > kMaxRows || H > kMaxRows || (int64_t)T * k > kMaxRows || (int64_t)T * H > kMaxValues)
        return fail(MOE_ERR_UNSUPPORTED, "%s: T=%d k=%d H=%d R=%d is too large", name, T, k, H, R);
    return MOE_OK;
}

// The bank of the experts' products: bf16, H and I multiples of 8.
moe_status_t check_experts(const moe_experts_t* b, int32_t R, const char* name) {
    if (!b) return fail(MOE_ERR_INVALID, "%s: null bank", name);
    if (b->n < 1) return fail(MOE_ERR_INVALID, "%s: n = %d", name, b->n);
    if (b->n > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "%s: n = %d > %d", name, b->n, kMaxExperts);
    if (moe_status_t st = check_ffn_bank(b, name)) return st;
    if (R < 0) return fail(MOE_ERR_INVALID, "%s: R=%d", name, R);
    if (R > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "%s: R=%d > %d", name, R, kMaxRows);
    return MOE_OK;
}

moe_status_t check_gu(const char* name, const void* gu, int32_t gu_dt, const void* gu_e8) {
    if (!gu) return MOE_OK;
    if (gu_dt != MOE_F32 && gu_dt != MOE_I8) return fail(MOE_ERR_UNSUPPORTED, "%s: gu dtype %d", name, gu_dt);
    if (is_i8(gu_dt) && !gu_e8) return fail(MOE_ERR_INVALID, "%s: int8 gu without exponents", name);
    if (!aligned(gu, 16)) return fail(MOE_ERR_INVALID, "%s: gu must be 16-byte aligned", name);
    return MOE_OK;
}

moe_status_t check_x(const char* name, const void* x, int32_t x_dt, const void* x_e8) {
    if (x_dt != MOE_BF16 && x_dt != MOE_I8) return fail(MOE_ERR_UNSUPPORTED, "%s: x dtype %d", name, x_dt);
    if (x && is_i8(x_dt) && !x_e8) return fail(MOE_ERR_INVALID, "%s: int8 x without exponents", name);
    if (!aligned(x, is_i8(x_dt) ? 8 : 16)) return fail(MOE_ERR_INVALID, "%s: misaligned x", name);
    return MOE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ checkpoints in 8 bits
static moe_status_t check_i8x16(const char* name, int32_t rows, int32_t cols, int32_t dt) {
    if (rows < 0 || cols <= 0) return fail(MOE_ERR_INVALID, "%s: rows=%d cols=%d", name, rows, cols);
    if (cols % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: cols=%d not a multiple of 8", name, cols);
    if (!is_float(dt)) return fail(MOE_ERR_UNSUPPORTED, "%s: dtype %d", name, dt);
    if (rows > kMaxRows || cols > kMaxRows || (int64_t)rows * cols > kMaxValues)
        return fail(MOE_ERR_UNSUPPORTED, "%s: rows=%d cols=%d is too large", name, rows, cols);
    return MOE_OK;
}

moe_status_t moe_quant_i8x16(const void* x, int32_t x_dt, int32_t rows, int32_t cols, int8_t* q, uint8_t* e8,
                             void* stream) {
    if (moe_status_t st = check_i8x16("quant_i8x16", rows, cols, x_dt)) return st;
    if (rows == 0) return MOE_OK;
    if (!x || !q || !e8) return fail(MOE_ERR_INVALID, "%s", "quant_i8x16: null pointer");
    if (!aligned(x, 16) || !aligned(q, 8)) return fail(MOE_ERR_INVALID, "%s", "quant_i8x16: misaligned x or q");
    return done(moe::launch_quant_i8x16(x, x_dt == MOE_F32, rows, cols, q, e8, (hipStream_t)stream), "moe_quant_i8x16");
}

moe_status_t moe_dequant_i8x16(const int8_t* q, const uint8_t* e8, int32_t rows, int32_t cols, void* out,
                               int32_t out_dt, void* stream) {
    if (moe_status_t st = check_i8x16("dequant_i8x16", rows, cols, out_dt)) return st;
    if (rows == 0) return MOE_OK;
    if (!out || !q || !e8) return fail(MOE_ERR_INVALID, "%s", "dequant_i8x16: null pointer");
    if (!aligned(out, 16) || !aligned(q, 8)) return fail(MOE_ERR_INVALID, "%s", "dequant_i8x16: misaligned out or q");
    return done(moe::launch_dequant_i8x16(q, e8, rows, cols, out, out_dt == MOE_F32, (hipStream_t)stream),
                "moe_dequant_i8x16");
}

// ------------------------------------------------------------------ rows sorted by expert
moe_status_t moe_dispatch(const void* x, int32_t x_dt, const uint8_t* x_e8, int32_t T, int32_t H, const int32_t* dest,
                          int32_t k, int32_t R, void* xs, void* stream) {
    if (moe_status_t st = check_rows("dispatch", T, k, H, R)) return st;
    if (!is_float(x_dt) && !is_i8(x_dt)) return fail(MOE_ERR_UNSUPPORTED, "dispatch: x dtype %d", x_dt);
    if (T == 0 || R == 0) return MOE_OK;
    if (!x || !dest || !xs) return fail(MOE_ERR_INVALID, "%s", "dispatch: null x, dest or xs");
    if (is_i8(x_dt) && !x_e8) return fail(MOE_ERR_INVALID, "%s", "dispatch: int8 x without exponents");
    if (!aligned(x, is_i8(x_dt) ? 8 : 16) || !aligned(xs, 16) || !aligned(dest, 4))
        return fail(MOE_ERR_INVALID, "%s", "dispatch: misaligned x, xs or dest");
    moe::DispatchProblem p{};
    p.T = T; p.k = k; p.H = H; p.R = R; p.dest = dest;
    p.x = x; p.x_f32 = x_dt == MOE_F32; p.xe = is_i8(x_dt) ? x_e8 : nullptr; p.xs = xs;
    return done(moe::launch_dispatch(p, (hipStream_t)stream), "moe_dispatch");
}

moe_status_t moe_dispatch_backward(const void* dxs, int32_t dxs_dt, int32_t R, const int32_t* dest, int32_t T,
                                   int32_t k, int32_t H, const void* add, int32_t add_dt, void* dx, int32_t dx_dt,
                                   void* stream) {
    if (moe_status_t st = check_rows("dispatch_backward", T, k, H, R)) return st;
    if (!is_float(dxs_dt) || !is_float(dx_dt) || (add && !is_float(add_dt)))
        return fail(MOE_ERR_UNSUPPORTED, "dispatch_backward: dtypes dxs %d, add %d, dx %d", dxs_dt, add_dt, dx_dt);
    if (T == 0) return MOE_OK;
    if ((!dxs && R > 0) || !dest || !dx) return fail(MOE_ERR_INVALID, "%s", "dispatch_backward: null dxs, dest or dx");
    if (add == dx && add_dt != dx_dt) return fail(MOE_ERR_INVALID, "%s", "dispatch_backward: dx is add in another dtype");
    if (!aligned(dxs, 16) || !aligned(add, 16) || !aligned(dx, 16) || !aligned(dest, 4))
        return fail(MOE_ERR_INVALID, "%s", "dispatch_backward: misaligned tensor");
    moe::DispatchProblem p{};
    p.T = T; p.k = k; p.H = H; p.R = R; p.dest = dest;
    p.dxs = dxs; p.dxs_f32 = dxs_dt == MOE_F32; p.add = add; p.add_f32 = add_dt == MOE_F32; p.dx = dx;
    p.dx_f32 = dx_dt == MOE_F32;
    return done(moe::launch_dispatch_backward(p, (hipStream_t)stream), "moe_dispatch_backward");
}

moe_status_t moe_combine_backward(const void* dout, int32_t dout_dt, const void* y, int32_t y_dt, const float* y_scale,
                                  int32_t R, const int32_t* dest, const float* topk_w, int32_t T, int32_t k, int32_t H,
                                  void* dy, int32_t dy_dt, float* dw, void* stream) {
    if (moe_status_t st = check_rows("combine_backward", T, k, H, R)) return st;
    if (!is_float(dout_dt) || (dy && !is_float(dy_dt)) || (dw && !is_float(y_dt) && y_dt != MOE_E4M3))
        return fail(MOE_ERR_UNSUPPORTED, "combine_backward: dtypes dout %d, y %d, dy %d", dout_dt, y_dt, dy_dt);
    const bool e4m3 = dw && y_dt == MOE_E4M3;
    if (e4m3 && H % 128) return fail(MOE_ERR_UNSUPPORTED, "combine_backward: H=%d not a multiple of 128 with e4m3 y", H);
    if (T == 0 || (!dy && !dw)) return MOE_OK;
    if (!dout || !dest || !topk_w) return fail(MOE_ERR_INVALID, "%s", "combine_backward: null dout, dest or topk_w");
    if (dw && ((!y && R > 0) || (e4m3 && !y_scale && R > 0)))
        return fail(MOE_ERR_INVALID, "%s", "combine_backward: dw without y or its scales");
    if (!aligned(dout, 16) || (dw && !aligned(y, e4m3 ? 8 : 16)) || !aligned(dy, 16) || !aligned(dest, 4) ||
        !aligned(topk_w, 4) || !aligned(dw, 4) || (e4m3 && !aligned(y_scale, 4)))
        return fail(MOE_ERR_INVALID, "%s", "combine_backward: misaligned tensor");
    moe::CombineGradProblem p{};
    p.T = T; p.k = k; p.H = H; p.R = R; p.dest = dest; p.w = topk_w;
    p.dout = dout; p.dout_f32 = dout_dt == MOE_F32;
    p.y = y; p.y_mode = e4m3 ? 2 : y_dt == MOE_BF16 ? 1 : 0; p.y_scale = y_scale;
    p.dy = dy; p.dy_f32 = dy_dt == MOE_F32; p.dw = dw;
    return done(moe::launch_combine_backward(p, (hipStream_t)stream), "moe_combine_backward");
}

// ------------------------------------------------------------------ the experts' products
static bool experts_sizes(int32_t R, int32_t n, int32_t H, int32_t I) {
    return n >= 1 && n <= kMaxExperts && dense_sizes(R, H, I);
}

size_t moe_experts_ffn_workspace_size(int32_t R, int32_t n, int32_t H, int32_t I) {
    if (!experts_sizes(R, n, H, I)) return 0;
    return or_zero(moe::experts_ws_bytes(R, n, H, I));
}

moe_status_t moe_experts_ffn(const void* xs, int32_t x_dt, const int32_t* offsets, int32_t R, const moe_experts_t* bank,
                             void* y, int32_t y_dt, void* gu, int32_t gu_dt, uint8_t* gu_e8, void* ws, size_t ws_bytes,
                             void* stream) {
    if (moe_status_t st = check_experts(bank, R, "experts_ffn")) return st;
    if (x_dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "experts_ffn: x dtype %d", x_dt);
    if (!is_float(y_dt)) return fail(MOE_ERR_UNSUPPORTED, "experts_ffn: y dtype %d", y_dt);
    if (moe_status_t st = check_gu("experts_ffn", gu, gu_dt, gu_e8)) return st;
    if (R == 0) return MOE_OK;
    if (!xs || !y || !offsets) return fail(MOE_ERR_INVALID, "%s", "experts_ffn: null xs, y or offsets");
    if (!aligned(xs, 16) || !aligned(y, 16) || !aligned(offsets, 4))
        return fail(MOE_ERR_INVALID, "%s", "experts_ffn: misaligned xs, y or offsets");
    const size_t need = moe::experts_ws_bytes(R, bank->n, bank->H, bank->I);
    if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "experts_ffn: R=%d H=%d I=%d", R, bank->H, bank->I);
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s", "experts_ffn: workspace");
    moe::ExpertsProblem p{};
    p.offsets = offsets; p.n = bank->n; p.R = R; p.x = xs; p.H = bank->H; p.I = bank->I;
    p.wg = bank->w_gate; p.wu = bank->w_up; p.wd = bank->w_down;
    p.y = y; p.y_f32 = y_dt == MOE_F32;
    if (gu && is_i8(gu_dt)) { p.gu8 = (int8_t*)gu; p.gu8_e = gu_e8; }
    else p.gu = (float*)gu;
    return done(moe::launch_experts(p, ws, (hipStream_t)stream), "moe_experts_ffn");
}

size_t moe_experts_ffn_backward_workspace_size(int32_t R, int32_t n, int32_t H, int32_t I, int32_t has_gu,
                                               int32_t x_dt) {
    if (!experts_sizes(R, n, H, I)) return 0;
    return or_zero(moe::experts_backward_ws_bytes(R, n, H, I, has_gu, is_i8(x_dt)));
}

moe_status_t moe_experts_ffn_backward(const void* dy, const void* xs, int32_t x_dt, const uint8_t* x_e8,
                                      const int32_t* offsets, int32_t R, const moe_experts_t* bank, const void* gu,
                                      int32_t gu_dt, const uint8_t* gu_e8, void* dx, void* dw_gate, void* dw_up,
                                      void* dw_down, void* ws, size_t ws_bytes, void* stream) {
    const char* name = "experts_ffn_backward";
    if (moe_status_t st = check_experts(bank, R, name)) return st;
    if (moe_status_t st = check_x(name, xs, x_dt, x_e8)) return st;
    if (moe_status_t st = check_gu(name, gu, gu_dt, gu_e8)) return st;
    if (!aligned(dx, 16) || !aligned(dw_gate, 16) || !aligned(dw_up, 16) || !aligned(dw_down, 16) || !aligned(dy, 16) ||
        !aligned(offsets, 4))
        return fail(MOE_ERR_INVALID, "%s: misaligned tensor", name);
    if (!dx && !dw_gate && !dw_up && !dw_down) return MOE_OK;
    if (R > 0) {
        if (!dy || !offsets || (!xs && reads_x(gu, dw_gate, dw_up)))
            return fail(MOE_ERR_INVALID, "%s: null dy, xs or offsets", name);
        const size_t need = moe::experts_backward_ws_bytes(R, bank->n, bank->H, bank->I, gu != nullptr, is_i8(x_dt));
        if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "%s: R=%d H=%d I=%d", name, R, bank->H, bank->I);
        if (!ws || !aligned(ws, 256) || ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace", name);
    }
    moe::ExpertsProblem p{};
    p.offsets = offsets; p.n = bank->n; p.R = R; p.x = xs; p.x_e = is_i8(x_dt) ? x_e8 : nullptr;
    p.H = bank->H; p.I = bank->I;
    p.wg = bank->w_gate; p.wu = bank->w_up; p.wd = bank->w_down;
    if (gu && is_i8(gu_dt)) { p.gu8 = (int8_t*)gu; p.gu8_e = (uint8_t*)gu_e8; }
    else p.gu = (float*)gu;
    p.dy = dy; p.dx = dx; p.dwg = dw_gate; p.dwu = dw_up; p.dwd = dw_down;
    return done(moe::launch_experts_backward(p, ws, (hipStream_t)stream), "moe_experts_ffn_backward");
}

// ------------------------------------------------------------------ the dense block with checkpoints in 8 bits
size_t moe_ffn_ckpt_workspace_size(int32_t T, int32_t H, int32_t I) {
    if (!dense_sizes(T, H, I)) return 0;
    return or_zero(moe::ffn_ws_bytes(T, H, I, 1));
}

moe_status_t moe_ffn_ckpt(const void* x, int32_t x_dt, int32_t T, const moe_experts_t* bank, void* y, int32_t y_dt,
                          int8_t* gu, uint8_t* gu_e8, void* ws, size_t ws_bytes, void* stream) {
    if (moe_status_t st = check_dense(bank, "ffn_ckpt")) return st;
    if (T < 0) return fail(MOE_ERR_INVALID, "ffn_ckpt: T=%d", T);
    if (T > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "ffn_ckpt: T=%d > %d", T, kMaxRows);
    if (x_dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "ffn_ckpt: x dtype %d", x_dt);
    if (!is_float(y_dt)) return fail(MOE_ERR_UNSUPPORTED, "ffn_ckpt: y dtype %d", y_dt);
    if (T == 0) return MOE_OK;
    if (!x || !y || !gu || !gu_e8) return fail(MOE_ERR_INVALID, "%s", "ffn_ckpt: null x, y or gu");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gu, 16))
        return fail(MOE_ERR_INVALID, "%s", "ffn_ckpt: x, y and gu must be 16-byte aligned");
    const size_t need = moe::ffn_ws_bytes(T, bank->H, bank->I, 1);
    if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "ffn_ckpt: T=%d H=%d I=%d", T, bank->H, bank->I);
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s", "ffn_ckpt: workspace");
    moe::FfnProblem p{};
    p.x = x; p.wg = bank->w_gate; p.wu = bank->w_up; p.wd = bank->w_down;
    p.T = T; p.H = bank->H; p.I = bank->I;
    p.y = y; p.y_f32 = y_dt == MOE_F32; p.gu8 = gu; p.gu8_e = gu_e8;
    return done(moe::launch_ffn(p, ws, (hipStream_t)stream), "moe_ffn_ckpt");
}

size_t moe_ffn_ckpt_backward_workspace_size(int32_t T, int32_t H, int32_t I, int32_t has_gu, int32_t x_dt) {
    if (!dense_sizes(T, H, I)) return 0;
    return or_zero(moe::ffn_backward_ws_bytes(T, H, I, has_gu, is_i8(x_dt)));
}

moe_status_t moe_ffn_ckpt_backward(const void* dy, const void* x, int32_t x_dt, const uint8_t* x_e8, int32_t T,
                                   const moe_experts_t* bank, const void* gu, int32_t gu_dt, const uint8_t* gu_e8,
                                   void* dx, void* dw_gate, void* dw_up, void* dw_down, void* ws, size_t ws_bytes,
                                   void* stream) {
    const char* name = "ffn_ckpt_backward";
    if (moe_status_t st = check_dense(bank, name)) return st;
    if (T < 0) return fail(MOE_ERR_INVALID, "%s: T=%d", name, T);
    if (T > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "%s: T=%d > %d", name, T, kMaxRows);
    if (moe_status_t st = check_x(name, x, x_dt, x_e8)) return st;
    if (moe_status_t st = check_gu(name, gu, gu_dt, gu_e8)) return st;
    if (!aligned(dx, 16) || !aligned(dw_gate, 16) || !aligned(dw_up, 16) || !aligned(dw_down, 16) || !aligned(dy, 16))
        return fail(MOE_ERR_INVALID, "%s: tensors must be 16-byte aligned", name);
    if (!dx && !dw_gate && !dw_up && !dw_down) return MOE_OK;
    if (T > 0) {
        if (!dy || (!x && reads_x(gu, dw_gate, dw_up))) return fail(MOE_ERR_INVALID, "%s: null dy or x", name);
        const size_t need = moe::ffn_backward_ws_bytes(T, bank->H, bank->I, gu != nullptr, is_i8(x_dt));
        if (need == moe::kUnfit) return fail(MOE_ERR_UNSUPPORTED, "%s: T=%d H=%d I=%d", name, T, bank->H, bank->I);
        if (!ws || !aligned(ws, 256) || ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace", name);
    }
    moe::FfnProblem p{};
    p.x = x; p.x_e = is_i8(x_dt) ? x_e8 : nullptr; p.wg = bank->w_gate; p.wu = bank->w_up; p.wd = bank->w_down;
    p.T = T; p.H = bank->H; p.I = bank->I;
    if (gu && is_i8(gu_dt)) { p.gu8 = (int8_t*)gu; p.gu8_e = (uint8_t*)gu_e8; }
    else p.gu_in = (const float*)gu;
    p.dy = dy; p.dx = dx; p.dwg = dw_gate; p.dwu = dw_up; p.dwd = dw_down;
    return done(moe::launch_ffn_backward(p, ws, (hipStream_t)stream), "moe_ffn_ckpt_backward");
}

}  // extern "C"
