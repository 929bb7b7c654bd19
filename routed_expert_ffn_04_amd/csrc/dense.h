// Host-side launchers of the operators around the mixture-of-experts layer:
// the dense gated FFN with its gradients (ffn.hip), the norm step with its
// gradients (norm.hip, norm_grad.hip) and the int8 product (linear_i8.hip); and of
// the layer's training step: the experts' products with their gradients
// (experts.hip), rows sorted by expert and back (dispatch.hip), checkpoints in 8
// bits (ckpt.hip).  Arguments are validated by dense_api.cpp and train_api.cpp;
// the launchers only enqueue.
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
    int8_t* gu8; uint8_t* gu8_e;                // the same in i8x16 blocks, or null (backward: read)
    // backward
    const void* dy;                             // bf16 [T][H]
    const uint8_t* x_e;                         // x holds i8x16 codes with these exponents, or null
    const float* gu_in;                         // [T][2 I] or null: recomputed, unless gu8 is there
    void* dx; void* dwg; void* dwu; void* dwd;  // bf16, each may be null
};
size_t ffn_ws_bytes(int T, int H, int I, int gu8 = 0);
size_t ffn_backward_ws_bytes(int T, int H, int I, int has_gu, int x_i8 = 0);
hipError_t launch_ffn(const FfnProblem& p, void* ws, hipStream_t s);
hipError_t launch_ffn_backward(const FfnProblem& p, void* ws, hipStream_t s);
// Zeros (the weight gradients of no tokens): a multiple of 8 values, 16-byte aligned.
hipError_t launch_zero_bf16(void* out, size_t values, hipStream_t s);

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

// ckpt.hip
hipError_t launch_quant_i8x16(const void* x, int x_f32, long rows, int cols, int8_t* q, uint8_t* e8, hipStream_t s);
hipError_t launch_dequant_i8x16(const int8_t* q, const uint8_t* e8, long rows, int cols, void* out, int out_f32,
                                hipStream_t s);

// dispatch.hip
struct DispatchProblem {
    int T, k, H, R;
    const int32_t* dest;                        // [T][k]
    const void* x; int x_f32; const uint8_t* xe;   // xe non-null: x holds i8x16 codes
    void* xs;                                   // x's type (i8x16: bf16)
    // backward
    const void* dxs; int dxs_f32;
    const void* add; int add_f32;               // or null
    void* dx; int dx_f32;
};
hipError_t launch_dispatch(const DispatchProblem& p, hipStream_t s);
hipError_t launch_dispatch_backward(const DispatchProblem& p, hipStream_t s);

struct CombineGradProblem {
    int T, k, H, R;
    const int32_t* dest; const float* w;        // [T][k]
    const void* dout; int dout_f32;             // [T][H]
    const void* y; int y_mode; const float* y_scale;   // [R][H]: 0 fp32, 1 bf16, 2 e4m3 codes with scales [R][H / 128]
    void* dy; int dy_f32;                       // [R][H] or null
    float* dw;                                  // [T][k] or null
};
hipError_t launch_combine_backward(const CombineGradProblem& p, hipStream_t s);

// experts.hip: the FFN of n experts on rows sorted by expert
struct ExpertsProblem {
    const int32_t* offsets; int n, R;           // device [n + 1]; rows there are
    const void* x; const uint8_t* x_e;          // bf16 [R][H]; backward also i8x16 codes
    const void* wg; const void* wu; const void* wd;
    int H, I;
    void* y; int y_f32;
    float* gu; int8_t* gu8; uint8_t* gu8_e;     // [R][2 I], either or none
    // backward (gu, gu8 read; neither: recomputed)
    const void* dy;
    void* dx; void* dwg; void* dwu; void* dwd;  // each may be null
};
size_t experts_ws_bytes(int R, int n, int H, int I);
size_t experts_backward_ws_bytes(int R, int n, int H, int I, int has_gu, int x_i8);
hipError_t launch_experts(const ExpertsProblem& p, void* ws, hipStream_t s);
hipError_t launch_experts_backward(const ExpertsProblem& p, void* ws, hipStream_t s);

}  // namespace moe
