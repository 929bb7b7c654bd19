// Host-side launchers of the operators around the mixture-of-experts layer:
// the dense gated FFN with its gradients (ffn.hip), the norm step with its
// gradients (norm.hip, norm_grad.hip) and the int8 product (linear_i8.hip).
// Arguments are validated by dense_api.cpp; the launchers only enqueue.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// What the workspace sizes below return for a product that no kernel's grid holds.
constexpr size_t kUnfit = ~(size_t)0;

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct FfnProblem {
    const void* x;                              // bf16 [T][H]
    const void* wg; const void* wu; const void* wd;
    int T, H, I;
    void* y; int y_f32;                         // [T][H]
    float* gu;                                  // [T][2 I] or null
    // backward
    const void* dy;                             // bf16 [T][H]
    const float* gu_in;                         // [T][2 I] or null: recomputed
    void* dx; void* dwg; void* dwu; void* dwd;  // bf16, each may be null
};
size_t ffn_ws_bytes(int T, int H, int I);
size_t ffn_backward_ws_bytes(int T, int H, int I, int has_gu);
hipError_t launch_ffn(const FfnProblem& p, void* ws, hipStream_t s);
hipError_t launch_ffn_backward(const FfnProblem& p, void* ws, hipStream_t s);

struct NormProblem {
    const void* y; int y_f32;
    const void* res; int r_f32;                 // res null: 0
    int T, H;
    const void* post_w; const void* gate; int gate_div; const void* pre_w; int w_f32;
    float res_scale, eps;
    void* r_out; void* x_out; int x_f32;        // either may be null
    float* x_scale;                             // non-null: x_out holds int8 codes
    // backward
    const void* dx; const void* dr; const void* r;
    void* dy; void* dres; float* dpost_w; float* dgate; float* dpre_w;
};
hipError_t launch_norm(const NormProblem& p, hipStream_t s);
size_t norm_backward_ws_bytes(int T, int H, int gate_div);
hipError_t launch_norm_backward(const NormProblem& p, void* ws, hipStream_t s);

hipError_t launch_quant_i8(const void* x, int x_f32, int rows, int cols, int8_t* q, float* scale, hipStream_t s);

struct LinearI8Problem {
    const int8_t* q; const float* xs;           // [T][K], [T]
    const int8_t* w; const float* ws; const float* bias;   // [N][K], [N], [N] or null
    int T, K, N;
    void* out; int out_f32;
};
size_t linear_i8_ws_bytes(int T, int K, int N);
hipError_t launch_linear_i8(const LinearI8Problem& p, void* ws, hipStream_t s);

}  // namespace moe
