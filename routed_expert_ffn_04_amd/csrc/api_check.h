// Argument checks shared by the entry points around the layer (dense_api.cpp,
// train_api.cpp).
#pragma once
#include "moe.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense.h"
#include "internal.h"

namespace moe {
namespace api {

using moe::set_error;

template <class... A>
inline moe_status_t fail(moe_status_t st, const char* fmt, A... a) {
    return (moe_status_t)set_error(st, fmt, a...);
}

inline moe_status_t done(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return (moe_status_t)set_error(MOE_OK, "%s", "");
}

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool is_float(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline unsigned size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }

constexpr int kMaxFfn = 1 << 21;    // a tile's 256 rows of 2 I bf16 stay below 2^31 bytes
constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = 1 << 30;   // rows and tiles are counted in 32 bits
constexpr int64_t kMaxValues = (int64_t)1 << 40;   // of a matrix by itself: more than a GPU's memory holds

// A bank of the FFN that is trained: bf16, H and I multiples of 8.
inline moe_status_t check_ffn_bank(const moe_experts_t* b, const char* name) {
    if (b->dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "%s: weight dtype %d", name, b->dt);
    if (b->H <= 0 || b->I <= 0) return fail(MOE_ERR_INVALID, "%s: H=%d I=%d", name, b->H, b->I);
    if (b->H % 8 || b->I % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d I=%d must be multiples of 8", name, b->H, b->I);
    if (b->H > kMaxFfn || b->I > kMaxFfn)
        return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d I=%d > %d", name, b->H, b->I, kMaxFfn);
    if (!b->w_gate || !b->w_up || !b->w_down) return fail(MOE_ERR_INVALID, "%s: null weight pointer", name);
    if (!aligned(b->w_gate, 16) || !aligned(b->w_up, 16) || !aligned(b->w_down, 16))
        return fail(MOE_ERR_INVALID, "%s: weights must be 16-byte aligned", name);
    return MOE_OK;
}

// The bank of the dense block: n = 1.
inline moe_status_t check_dense(const moe_experts_t* b, const char* name) {
    if (!b) return fail(MOE_ERR_INVALID, "%s: null bank", name);
    if (b->n != 1) return fail(MOE_ERR_INVALID, "%s: n = %d, expected 1", name, b->n);
    return check_ffn_bank(b, name);
}

// Whether the backward pass reads x: for g and u where they were not saved, and for the gradients of their weights.
inline bool reads_x(const void* gu, const void* dw_gate, const void* dw_up) { return !gu || dw_gate || dw_up; }

inline bool dense_sizes(int T, int H, int I) {
    return T >= 0 && T <= kMaxRows && H > 0 && I > 0 && H % 8 == 0 && I % 8 == 0 && H <= kMaxFfn && I <= kMaxFfn;
}

inline size_t or_zero(size_t bytes) { return bytes == moe::kUnfit ? 0 : bytes; }

}  // namespace api
}  // namespace moe
