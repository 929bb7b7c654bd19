// Tiled matrix product C[m][n] = sum_k A(m, k) B(n, k) on the matrix cores,
// with the epilogues of the dense gated FFN (forward and backward) and of the
// int8 product.  Used by ffn.hip (bf16) and linear_i8.hip (int8).
//
// Operands.  Each of A and B is stored either with k contiguous (kRow: row m
// holds its k values, like an activation or an output-major weight) or with m
// contiguous (kCol: row k holds the values of all m, which is how the gradient
// products meet the same matrices).  Neither is ever transposed in memory: a
// kCol tile goes into LDS as it is and its fragments are read with the
// transposing LDS read (ds_read_b64_tr_b16: 16 lanes read 4 k-rows x 16
// columns, each lane gets the 4 k values of one column).
//
// Tile.  BM x BN outputs per workgroup, 128 bytes of k per stage (64 bf16 or
// 128 int8).  LDS is a ring of R half-stages (the A part or the B part of a
// stage) filled by direct global->LDS 16-byte loads.
//   256 x 256: 8 waves (2 x 4) of 128 x 64; R = 5, 160 KiB, one workgroup per CU
//   128 x 128: 4 waves (2 x 2) of 64 x 64;  R = 5, 80 KiB, two per CU, or R = 10, 160 KiB, one
//    64 x 64:  4 waves (2 x 2) of 32 x 32;  R = 5, 40 KiB, four per CU, or R = 10, 80 KiB, two
// The rings of ten are for products with few workgroups (launch_tiling).  Each
// wave's product is formed transposed (the n side is the MFMA row operand), so a
// lane holds four consecutive n of one row m.  Four waves of 128 x 128 for the
// 256-row tiles read a third less from LDS but have nothing to run while they
// wait: T = 16384 FFN 1187 us against 1179, T = 4096 gradients 729 against 664.
//
// What binds: the largest products the matrix cores at the clock the power limit
// leaves (FFN of 16384 tokens, 7168 x 2048, 1110 us = 1.30 PFLOP/s; int8 8192 x 7168 x
// 4096 200 us = 2.4 Pop/s; with every load from the same few lines 10 % less), small
// tiles the loads into LDS (0.21 us a stage of 64 rows, 16 KiB).
//
// Row pieces of 128 bytes, whole cache lines: a kernel that only loads moves 32
// KiB per CU into LDS in 0.36 us with 128-byte pieces and in 0.5 to 0.75 us
// with 64-byte ones, and the loads are what limits a stage first.
//
// One barrier per stage.  R = 5: after the last fragments of a stage have been
// read and before its last quarter (256-row tiles) or half multiplies: after it
// both halves of the stage are free and take the B half one stage and the A half
// two stages ahead, which leaves at least a whole stage of products for every load
// to land in.  R = 10: a stage's fragments are all in registers before it
// multiplies, so its halves are free by then and take the stage five further on,
// while the next stage's fragments are read.
//
// Bounds.  m and n past the end re-read the last row (last 16-byte chunk) and
// are never stored; k past the end (the ragged last stage, and the stages that
// the ring prefetches past it) is loaded as zeros, so it adds exactly nothing.
#pragma once
#include "common.h"
#include "gffn_common.h"
#include "i8x16.h"
#include "tile_plan.h"

namespace moe {
namespace gemm {

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum { kRow = 0, kCol = 1 };
enum { kBf16 = 0, kI8 = 1 };

// what becomes of the accumulators
enum Epi {
    kEpiGateUp = 0,    // B tile: BN/2 gate columns then BN/2 up columns; h = silu(g) u (bf16), optionally g and u (fp32)
    kEpiOut = 1,       // bf16 or fp32 matrix
    kEpiGrad = 2,      // acc = dh; with the saved g, u: dg, du (bf16 [M][2 N]) and h (bf16 [M][N])
    kEpiPart = 3,      // 32-bit accumulators of one k-split, [split][M][N] (gate/up: [split][M][2 I])
    kEpiI8 = 4,        // acc * x_scale[m] * w_scale[n] + bias[n], bf16 or fp32
    kEpiGateUp8 = 5,   // kEpiGateUp with g and u as blocks of 16 columns (i8x16.h): codes in q, exponents in qe
    kEpiGrad8 = 6,     // kEpiGrad with g and u from such blocks
};

constexpr uint32_t kFar = 1u << 31;   // past every byte of a tile: 256 rows of at most 2^23 bytes

struct Operand {
    const uint8_t* p;    // element (row 0, k 0)
    const uint8_t* p2;   // gate/up B: the up matrix; with turn: element (row 0, k = turn)
    size_t ld;           // bytes from row to row (kRow: of m; kCol: of k)
    int n;               // rows m (kRow), columns m (kCol); gate/up B: I
};

struct Args {
    Operand A, B;
    int M, N, K;         // N: output columns (gate/up: I)
    int mt, nt;          // tiles
    int splits, kspan;   // k-splits; k elements per split (a multiple of the stage)
    int turn, len;       // a sum of two products (kRow A, kCol B; 0: none): k in [0, len) of p, k in [turn, K) of p2,
                         // turn = len rounded up to the stage, so no stage has rows of both
    int vec;             // rows of the outputs allow 16-byte accesses
    void* out;           // kEpiOut / kEpiI8 / kEpiPart: [M][N]; kEpiGateUp: h; kEpiGrad: dgu
    void* out2;          // kEpiOut: rows m >= msplit, as if they began at row msplit; kEpiGrad: h; kEpiGateUp: gu (or null)
    int msplit;
    int out_f32;
    const float* gu;     // kEpiGrad: saved pre-activations [M][2 N]
    int8_t* q;           // kEpiGateUp8 (written), kEpiGrad8 (read): codes [M][2 N]
    uint8_t* qe;         // and exponents [M][2 ceil(N / 16)]
    const float* xs; const float* ws; const float* bias;   // kEpiI8
};

// k past the end reads this.
static __device__ __align__(16) const uint32_t kZeros[4] = {0, 0, 0, 0};

// Chunk key of row r of a kRow half-stage (128-byte rows): chunk c sits at
// position c ^ key, which spreads the fragment reads over all banks.
__device__ __forceinline__ int row_key(int r) { return (r & 7) ^ ((r >> 3) & 1); }
// The same of row k of a kCol half-stage (2 BM-byte rows): the 32 bytes that a
// half-wave reads of rows 8 g + 0 .. 3, g = 0, 1, fall into different banks.
template <int BM>
__device__ __forceinline__ int col_key(int r) {
    return (BM == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2) | (((r >> 3) & 1) << 1);
}

template <int N>
__device__ __forceinline__ void barrier_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Orders a wave's LDS accesses for its other lanes (they complete in order in
// hardware; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_sync() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// MFMA operands of the 16-row blocks of a wave, one k-step (32 bf16 or 64 int8),
// 16 bytes a lane: lane l holds row l % 16, k values [8 (l / 16), +8) (int8: 16).
// kRow: one 16-byte LDS read.  kCol: two transposing reads of 4 k-rows each; a
// half-wave reads 32 bytes of eight k-rows, which col_key puts into eight
// different parts of the banks.
template <int LAYOUT, int BMN>
struct Frag {
    int off[LAYOUT == kRow ? 2 : 1];   // kRow: by k-step
    __device__ __forceinline__ Frag(int block0, int lane) {
        const int g = lane / 16, j = lane % 16;
        if constexpr (LAYOUT == kRow) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) off[ks] = (block0 * 16 + j) * kStage + (((4 * ks + g) ^ row_key(j)) << 4);
        } else {
            const int row = 8 * g + j / 4;
            off[0] = row * (BMN * 2) + (block0 >> 3) * 256 + ((2 * (block0 & 7) + (j % 4) / 2) ^ col_key<BMN>(row)) * 16 + (j & 1) * 8;
        }
    }
    // b: block within the wave's part (kCol: block0 is a multiple of the part's blocks, so
    // the block's offset is an exclusive or on the chunk bits)
    __device__ __forceinline__ i32x4 read(const uint8_t* half, int b, int ks) const {
        if constexpr (LAYOUT == kRow) {
            return *(const i32x4*)(half + off[ks] + b * 16 * kStage);
        } else {
            const uint8_t* q = half + (off[0] ^ (b * 32)) + ks * 32 * (BMN * 2);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)q);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(q + 4 * (BMN * 2)));
            return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// The 16 x 16 forms: on random operands the chip's power limit lets a
// register-only loop of 16x16x32 bf16 products run at 2.21 PFLOP/s and one of
// 32x32x16 at 1.89 (2.45 and 2.50 on zeros).
template <int E> struct Acc;
template <> struct Acc<kBf16> {
    typedef f32x4 type;
    __device__ static type mma(i32x4 a, i32x4 b, type c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
};
template <> struct Acc<kI8> {
    typedef i32x4 type;
    __device__ static type mma(i32x4 a, i32x4 b, type c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }
};

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                      f32x2_to_bf16x2(v[6], v[7]));
}

// The gated activation's derivative: with s = sigmoid(g), a = g s, h = a u:
//   dg = dh u s (1 + g (1 - s)),  du = dh a.
// 1 - s is formed as e^-g / (1 + e^-g) so that it keeps its digits for large g;
// for g so negative that e^-g overflows, s = 0 makes every term exactly 0.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dh, float& dg, float& du, float& h) {
    const float e = __expf(-g);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    const float a = g * s;
    const float t = s == 0.0f ? 0.0f : a * (e * s);
    dg = dh * u * (s + t);
    du = dh * a;
    h = a * u;
}

// The gate and up columns n .. n + 7 of row m as i8x16 blocks: the lane and its
// neighbour (lane ^ 1: the columns before or after) hold the two halves of a block.
// Called by both, also past the end (values there count as zeros, nothing is stored).
__device__ __forceinline__ void store_gu8(const Args& G, int m, int n, const float (&g)[8], const float (&u)[8]) {
    const bool in = n < G.N;
    float gv[8], uv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        gv[e] = in ? g[e] : 0.0f;
        uv[e] = in ? u[e] : 0.0f;
    }
    const uint32_t ge = i8x16_exponent(i8x16_pair_max(gv)), ue = i8x16_exponent(i8x16_pair_max(uv));
    if (m >= G.M || !in) return;
    const size_t nb = (size_t)i8x16_blocks(G.N);
    int8_t* q = G.q + (size_t)m * (2 * (size_t)G.N) + n;
    *(uint2*)q = i8x16_codes(gv, ge);
    *(uint2*)(q + G.N) = i8x16_codes(uv, ue);
    if (n % kI8Block == 0) {
        uint8_t* e = G.qe + (size_t)m * (2 * nb) + n / kI8Block;
        e[0] = (uint8_t)ge;
        e[nb] = (uint8_t)ue;
    }
}

// Eight consecutive outputs (m, n .. n + 7) of a kEpiOut / kEpiI8 / kEpiPart matrix.
__device__ __forceinline__ void store8(const Args& G, uint8_t* row, int n, const float (&v)[8], bool f32) {
    if (G.vec && n + 8 <= G.N) {
        if (f32) {
            float4* o = (float4*)((float*)row + n);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *(uint4*)((uint16_t*)row + n) = pack8(v);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n + e < G.N) {
                if (f32) ((float*)row)[n + e] = v[e];
                else ((uint16_t*)row)[n + e] = (uint16_t)f32_to_bf16_bits(v[e]);
            }
    }
}

// Workgroup b of `total` -> tile.  Workgroups go to the eight dies round robin,
// each die with an L2 of its own: every die takes one contiguous run of tiles,
// ordered in bands (band_of).
__device__ __forceinline__ void tile_of(int b, int mt, int nt, int total, int& tm, int& tn, int& split) {
    const int x = b % kXcds, j = b / kXcds;
    const int base = total / kXcds, extra = total % kXcds;
    int t = x * base + min(x, extra) + j;
    const int per = mt * nt;
    split = t / per;
    t -= split * per;
    band_of(t, mt, nt, tm, tn);
}

// Epilogue of a wave whose part of the product begins at row mw and column nw.  Every wave has
// left the ring, which becomes the scratch.
template <int E, int EPI, bool GU, int IB, int JB>
__device__ __forceinline__ void finish(const Args& G, const typename Acc<E>::type (&acc)[IB][JB], uint8_t* smem, int wave,
                                       int lane, int mw, int nw, int split) {
    // acc[i][j][v]: m = 16 i + l % 16, n = 16 j + 4 (l / 16) + v of the wave's part.  32 rows at a time pass through the wave's own piece of LDS
    // (rows padded by 16 bytes, free of bank conflicts both ways), so that global
    // accesses are whole row pieces.
    constexpr int WC = JB * 16;                          // MFMA columns of a wave
    constexpr int RS = WC * 4 + 16;
    constexpr int RL = (GU ? WC / 2 : WC) / 8;           // lanes a row, eight outputs each
    constexpr int RP = 64 / RL, kPass = 32 / RP;         // rows a pass
    uint8_t* piece = smem + wave * 32 * RS;
    // A lane's eight columns are the same in every pass: their scales are read once.
    const int nl = nw + (lane % RL) * 8;
    float wsv[8], bv[8], xsv[IB / 2][kPass];
    if constexpr (EPI == kEpiI8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int ne = min(nl + e, G.N - 1);
            wsv[e] = G.ws[ne];
            bv[e] = G.bias ? G.bias[ne] : 0.0f;
        }
#pragma unroll
        for (int ib = 0; ib < IB / 2; ++ib)
#pragma unroll
            for (int p = 0; p < kPass; ++p)
                xsv[ib][p] = G.xs[min(mw + ib * 32 + p * RP + lane / RL, G.M - 1)];
    }
#pragma unroll
    for (int ib = 0; ib < IB / 2; ++ib) {
        const int mb = mw + ib * 32;
        if (mb >= G.M) break;
        // the saved pre-activations of the 32 rows, read while the accumulators pass through LDS
        float4 gv[kPass][2], uv[kPass][2];
        uint2 gq[kPass], uq[kPass];
        uint32_t ge[kPass], ue[kPass];
        if constexpr (EPI == kEpiGrad8) {
            const size_t nb = (size_t)i8x16_blocks(G.N);
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                const size_t m = (size_t)min(mb + p * RP + lane / RL, G.M - 1);
                const int n = min(nl, G.N - 8);
                gq[p] = *(const uint2*)(G.q + m * (2 * (size_t)G.N) + n);
                uq[p] = *(const uint2*)(G.q + m * (2 * (size_t)G.N) + G.N + n);
                ge[p] = G.qe[m * (2 * nb) + n / kI8Block];
                ue[p] = G.qe[m * (2 * nb) + nb + n / kI8Block];
            }
        }
        if constexpr (EPI == kEpiGrad) {
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                const size_t at = (size_t)min(mb + p * RP + lane / RL, G.M - 1) * (2 * (size_t)G.N) + min(nl, G.N - 8);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    gv[p][e] = *(const float4*)(G.gu + at + 4 * e);
                    uv[p][e] = *(const float4*)(G.gu + at + G.N + 4 * e);
                }
            }
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < JB; ++j)
                *(typename Acc<E>::type*)(piece + (i * 16 + lane % 16) * RS + (16 * j + 4 * (lane / 16)) * 4) = acc[ib * 2 + i][j];
        wave_sync();
        auto words = [&](int row, int n, float(&v)[8]) {
            const float4 lo = *(const float4*)(piece + row * RS + n * 4);
            const float4 hi = *(const float4*)(piece + row * RS + n * 4 + 16);
            v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w; v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
        };
        if constexpr (GU) {
            // WC / 2 gate columns, then as many up columns
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                const int row = p * RP + lane / RL, c = (lane % RL) * 8;
                const int m = mb + row, n = nw + c;
                float g[8], u[8], h[8];
                words(row, c, g);
                words(row, WC / 2 + c, u);
                if constexpr (EPI == kEpiGateUp8) store_gu8(G, m, n, g, u);
                if (m < G.M && n < G.N) {
                    if constexpr (EPI == kEpiPart) {
                        float* o = (float*)G.out + ((size_t)split * G.M + m) * (2 * (size_t)G.N) + n;
                        *(float4*)o = make_float4(g[0], g[1], g[2], g[3]);
                        *(float4*)(o + 4) = make_float4(g[4], g[5], g[6], g[7]);
                        o += G.N;
                        *(float4*)o = make_float4(u[0], u[1], u[2], u[3]);
                        *(float4*)(o + 4) = make_float4(u[4], u[5], u[6], u[7]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = silu_mul(g[e], u[e]);
                        *(uint4*)((uint16_t*)G.out + (size_t)m * G.N + n) = pack8(h);
                        if (EPI == kEpiGateUp && G.out2) {
                            float* o = (float*)G.out2 + (size_t)m * (2 * (size_t)G.N) + n;
                            *(float4*)o = make_float4(g[0], g[1], g[2], g[3]);
                            *(float4*)(o + 4) = make_float4(g[4], g[5], g[6], g[7]);
                            o += G.N;
                            *(float4*)o = make_float4(u[0], u[1], u[2], u[3]);
                            *(float4*)(o + 4) = make_float4(u[4], u[5], u[6], u[7]);
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                const int row = p * RP + lane / RL, c = (lane % RL) * 8;
                const int m = mb + row, n = nw + c;
                float v[8];
                words(row, c, v);
                if (m < G.M && n < G.N) {
                    if constexpr (EPI == kEpiGrad || EPI == kEpiGrad8) {
                        float g[8], u[8], dg[8], du[8], h[8];
                        if constexpr (EPI == kEpiGrad8) {
                            i8x16_values(gq[p], ge[p], g);
                            i8x16_values(uq[p], ue[p], u);
                        } else {
                            const float4 ga = gv[p][0], gb = gv[p][1], ua = uv[p][0], ub = uv[p][1];
                            g[0] = ga.x; g[1] = ga.y; g[2] = ga.z; g[3] = ga.w; g[4] = gb.x; g[5] = gb.y; g[6] = gb.z; g[7] = gb.w;
                            u[0] = ua.x; u[1] = ua.y; u[2] = ua.z; u[3] = ua.w; u[4] = ub.x; u[5] = ub.y; u[6] = ub.z; u[7] = ub.w;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) swiglu_grad(g[e], u[e], v[e], dg[e], du[e], h[e]);
                        uint16_t* d = (uint16_t*)G.out + (size_t)m * (2 * (size_t)G.N) + n;
                        *(uint4*)d = pack8(dg);
                        *(uint4*)(d + G.N) = pack8(du);
                        *(uint4*)((uint16_t*)G.out2 + (size_t)m * G.N + n) = pack8(h);
                    } else if constexpr (EPI == kEpiPart) {
                        store8(G, (uint8_t*)((float*)G.out + ((size_t)split * G.M + m) * G.N), n, v, true);
                    } else if constexpr (EPI == kEpiI8) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            v[e] = (float)__float_as_int(v[e]) * (xsv[ib][p] * wsv[e]);
                            if (G.bias) v[e] += bv[e];
                        }
                        store8(G, (uint8_t*)G.out + (size_t)m * G.N * (G.out_f32 ? 4 : 2), n, v, G.out_f32);
                    } else {
                        const size_t row_bytes = (size_t)G.N * (G.out_f32 ? 4 : 2);
                        uint8_t* o = m < G.msplit ? (uint8_t*)G.out + (size_t)m * row_bytes
                                                  : (uint8_t*)G.out2 + (size_t)(m - G.msplit) * row_bytes;
                        store8(G, o, n, v, G.out_f32);
                    }
                }
            }
        }
    }
}

// Launch shape of the tiles: LDS, and waves per SIMD by it.
constexpr int tile_lds(int edge, int ring) { return ring * edge * kStage; }
constexpr int tile_waves(int edge, int ring) { return edge == 256 ? 2 : 163840 / tile_lds(edge, ring); }   // per SIMD

// Tile (tm, tn) of the k-split `split` of G.
template <int E, int LA, int LB, int EPI, bool GU, int BM, int BN, int R>
__device__ __forceinline__ void tile_at(const Args& G, int tm, int tn, int split) {
    constexpr int kThreads = tile_threads(BM);
    constexpr int EB = E == kI8 ? 1 : 2;
    constexpr int KE = kStage / EB;                            // k elements per stage
    constexpr int WN = BM == 256 ? 4 : 2, WM = 2;              // waves along n and m
    constexpr int IB = BM / WM / 16, JB = BN / WN / 16;        // 16 x 16 blocks of a wave
    constexpr int LD = BM * 8 / kThreads;                      // direct loads per lane and half-stage
    constexpr int kHalf = BM * kStage;                         // bytes of a half-stage
    static_assert(BM == BN && LD % 2 == 0, "square tiles");
    constexpr int kTileN = GU ? BN / 2 : BN;                   // output columns per tile
    static_assert(E == kBf16 || (LA == kRow && LB == kRow), "the transposing read is for 16-bit elements");
    static_assert(WM * WN * 64 == kThreads, "waves cover the tile");

    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wm = wave / WN, wn = wave % WN;

    const int m0 = tm * BM, n0 = tn * kTileN;
    const int k0 = split * G.kspan;
    const int kn = min(G.K - k0, G.kspan);                     // k elements of this split
    const int nst = (kn + KE - 1) / KE;

    // ---- the lane's share of the direct loads: LD 16-byte slots in each
    // half-stage, at fixed offsets from a base that is the same in the whole wave
    // (in scalar registers) and moves on by a stage
    uint32_t offa[LD], offb[LD];
    auto place = [&](int layout, const Operand& O, int r0, int half, uint32_t(&off)[LD]) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < LD; ++q) {
            const int at = (wave * LD + q) * 64 + lane;
            if (layout == kRow) {
                const int r = at / 8, c = (at % 8) ^ row_key(r);
                off[q] = (uint32_t)(min(r0 + r - half, O.n - 1) - r0) * (uint32_t)O.ld + c * 16;
            } else {
                constexpr int per = BM * 2 / 16;                       // slots per k row
                const int r = at / per, c = (at % per) ^ col_key<BM>(r);
                off[q] = (uint32_t)r * (uint32_t)O.ld + (min(r0 + c * 8, O.n - 8) - r0) * 2;
            }
        }
    };
    auto origin = [&](int layout, const Operand& O, const uint8_t* p, int r0) __attribute__((always_inline)) {
        return layout == kRow ? p + (size_t)r0 * O.ld + (size_t)k0 * EB : p + (size_t)k0 * O.ld + (size_t)r0 * 2;
    };
    // gate/up: the waves that load the second half of the B rows take the up matrix
    const bool up = GU && wave * LD * 8 >= BN / 2;
    place(LA, G.A, m0, 0, offa);
    place(LB, G.B, n0, up ? BN / 2 : 0, offb);
    const uint8_t* pa = origin(LA, G.A, G.A.p, m0);
    const uint8_t* pb = origin(LB, G.B, up ? G.B.p2 : G.B.p, n0);
    // k of a slot within its stage: kRow its chunk's first, kCol its row
    const int kr = ((lane % 8) ^ (lane / 8)) * (16 / EB);             // q even; q odd: the neighbouring chunk
    const int kc = wave * LD * (64 / (BM / 8)) + lane / (BM / 8);     // q = 0
    auto k_of = [&](int layout, int q) __attribute__((always_inline)) {
        return layout == kRow ? kr ^ ((q & 1) * (16 / EB)) : kc + q * (64 / (BM / 8));
    };
    // from where p would continue to p2, for the stages past the turn
    constexpr bool TWO = LA == kRow && LB == kCol;
    const int turn = TWO && G.turn ? G.turn - k0 : 0x7fffffff;
    const ptrdiff_t past_a = TWO && G.turn ? G.A.p2 - (G.A.p + (size_t)G.turn * EB) : 0;
    const ptrdiff_t past_b = TWO && G.turn ? G.B.p2 - (G.B.p + (size_t)G.turn * G.B.ld) : 0;
    const int end1 = TWO && G.turn ? min(G.len - k0, kn) : kn;   // end of the stages before the turn

    // Loads [q0, q1) of the half-stage that begins at k.  Buffer loads: base and
    // bound in scalar registers, one 32-bit offset a lane, and slots past the end take
    // an offset past the bound, which reads zero.
    auto issue = [&](uint8_t* half, const uint8_t* p, ptrdiff_t past, const uint32_t(&off)[LD], int layout,
                     int k, int q0, int q1) __attribute__((always_inline)) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know the resource's type
        const int left = (TWO && k >= turn ? kn : end1) - k;
        auto rows = __builtin_amdgcn_make_buffer_rsrc((void*)(TWO && k >= turn ? p + past : p), 0, (int)kFar, 0x00027000);
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            const uint32_t at = k_of(layout, q) >= left ? kFar : off[q];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (lds_void*)(half + (wave * LD + q) * 1024), 16, at, 0, 0, 0);
        }
#endif
    };
    int ka = 0, kb = 0;   // first k of the next half-stages to load
    auto issueA = [&](uint8_t* half, int q0, int q1) __attribute__((always_inline)) {
        issue(half, pa, past_a, offa, LA, ka, q0, q1);
        if (q1 == LD) {
            ka += KE;
            pa += LA == kRow ? (size_t)kStage : (size_t)KE * G.A.ld;
        }
    };
    auto issueB = [&](uint8_t* half, int q0, int q1) __attribute__((always_inline)) {
        issue(half, pb, past_b, offb, LB, kb, q0, q1);
        if (q1 == LD) {
            kb += KE;
            pb += LB == kRow ? (size_t)kStage : (size_t)KE * G.B.ld;
        }
    };

    typename Acc<E>::type acc[IB][JB];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j] = typename Acc<E>::type{};

    const Frag<LA, BM> fa(wm * IB, lane);
    const Frag<LB, BN> fb(wn * (GU ? JB / 2 : JB), lane);
    if constexpr (R == 10) {
        // One or two workgroups per CU: a stage's fragments are read while the
        // stage before multiplies (two register sets), since a wave alone on its
        // SIMD has nothing else to do meanwhile: FFN of 1024 x 2048 x 1024 25 us
        // against 28, int8 333 x 2064 x 1501 8.3 against 9.9.
        i32x4 a[2][2][IB], b[2][2][JB];   // [set][k-step]
        auto read = [&](const uint8_t* ha, const uint8_t* hb, int set, int ks) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < JB; ++j)
                b[set][ks][j] = fb.read(hb + (GU && j >= JB / 2 ? BN / 2 * kStage : 0), GU ? j % (JB / 2) : j, ks);
#pragma unroll
            for (int i = 0; i < IB; ++i) a[set][ks][i] = fa.read(ha, i, ks);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto mma = [&](int set, int ks) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < IB; ++i)
#pragma unroll
                for (int j = 0; j < JB; ++j) acc[i][j] = Acc<E>::mma(b[set][ks][j], a[set][ks][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        };
        // The products of the stage in `set` while the next stage is read from
        // rA and rB into the other one; everybody has read this stage's halves,
        // w0 and w1 (see below for the restrict qualifiers).
        auto turn = [&](int set, uint8_t* __restrict__ w0, uint8_t* __restrict__ w1, const uint8_t* __restrict__ rA,
                        const uint8_t* __restrict__ rB) __attribute__((always_inline)) {
            read(rA, rB, set ^ 1, 0);
            mma(set, 0);
            issueA(w0, 0, LD);
            __builtin_amdgcn_sched_barrier(0);
            read(rA, rB, set ^ 1, 1);
            mma(set, 1);
            issueB(w1, 0, LD);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto start = [&](uint8_t* __restrict__ w, const uint8_t* __restrict__ rA, const uint8_t* __restrict__ rB)
                         __attribute__((always_inline)) {
#pragma unroll
            for (int h = 2; h < R; ++h)
                if (h % 2) issueB(w + (h - 2) * kHalf, 0, LD);
                else issueA(w + (h - 2) * kHalf, 0, LD);
            barrier_vm<(R - 2) * LD>();   // the first two halves
            read(rA, rB, 0, 0);
            read(rA, rB, 0, 1);
        };
        issueA(smem, 0, LD);
        issueB(smem + kHalf, 0, LD);
        start(smem + 2 * kHalf, smem, smem + kHalf);
        int u = 0;   // slot of the current stage's A half
        auto go = [&](int set) __attribute__((always_inline)) {
            barrier_vm<(R - 4) * LD>();   // the next stage has landed
            uint8_t* w = smem + u * kHalf;
            u = u + 2 == R ? 0 : u + 2;
            const uint8_t* r = smem + u * kHalf;
            turn(set, w, w + kHalf, r, r + kHalf);
        };
        int s = 0;
        for (; s + 2 < nst; s += 2) {
            go(0);
            go(1);
        }
        if (s + 1 < nst) {
            go(0);
            mma(1, 0);
            mma(1, 1);
        } else {
            mma(0, 0);
            mma(0, 1);
        }
    } else {
        // A stage is two k-steps, each one part, or two in 256-row tiles (the halves
        // of the wave's rows).  a: the rows' fragments of one part, b: the columns'
        // of one k-step, both twice: one set multiplies while the next is read.
        constexpr int AH = IB < 4 ? IB : 4, PK = IB / AH, kParts = 2 * PK;
        i32x4 a[2][AH], b[2][JB];
        auto read_a = [&](const uint8_t* half, int part, int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
            for (int i = i0; i < i1; ++i) a[part & 1][i] = fa.read(half, part % PK * AH + i, part / PK);
        };
        auto read_b = [&](const uint8_t* half, int ks) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < JB; ++j)   // gate/up: half of the blocks gate columns, half up columns
                b[ks][j] = fb.read(half + (GU && j >= JB / 2 ? BN / 2 * kStage : 0), GU ? j % (JB / 2) : j, ks);
        };
        auto mma = [&](int part, int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
            for (int i = i0; i < i1; ++i)
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    auto& c = acc[part % PK * AH + i][j];
                    c = Acc<E>::mma(b[part / PK][j], a[part & 1][i], c);
                }
            __builtin_amdgcn_sched_barrier(0);
        };
        // The products of `part` while the next part's fragments are read.  LDS
        // reads and direct loads go out a few at a time between products: together
        // they would fill the memory pipes' queues and hold up the products behind
        // them.
        auto step = [&](int part, const uint8_t* ha, const uint8_t* hb, auto&& load) __attribute__((always_inline)) {
            const int next = (part + 1) % kParts;
            mma(part, 0, AH / 4);
            if (next % PK == 0) read_b(hb, next / PK);
            read_a(ha, next, 0, AH / 2);
            __builtin_amdgcn_sched_barrier(0);
            mma(part, AH / 4, AH / 2);
            read_a(ha, next, AH / 2, AH);
            __builtin_amdgcn_sched_barrier(0);
            mma(part, AH / 2, AH - 1);
            load();
            __builtin_amdgcn_sched_barrier(0);
            mma(part, AH - 1, AH);
        };
        // One stage from its halves rA, rB, beginning with the previous stage's
        // last part; w0 and w1 are the halves that stage has left.  The restrict
        // qualifiers state that the loads into w0 and w1 do not touch rA and rB;
        // without them the compiler waits for every direct load before a
        // transposing read.
        auto turn = [&](uint8_t* __restrict__ w0, uint8_t* __restrict__ w1, const uint8_t* __restrict__ rA,
                        const uint8_t* __restrict__ rB) __attribute__((always_inline)) {
            // the halves' loads, in the order of the ring
            auto fill = [&](int q0, int q1) __attribute__((always_inline)) {
#pragma unroll
                for (int q = q0; q < q1; q += 2)
                    if ((q < LD) == (R % 2 == 1)) issueB(q < LD ? w0 : w1, q % LD, q % LD + 2);
                    else issueA(q < LD ? w0 : w1, q % LD, q % LD + 2);
            };
            constexpr int L = 2 * LD / kParts;
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                step((p + kParts - 1) % kParts, rA, rB, [&]() __attribute__((always_inline)) { fill(p * L, p * L + L); });
        };
        auto none = []() __attribute__((always_inline)) {};
        auto start = [&](uint8_t* __restrict__ w, const uint8_t* __restrict__ rA, const uint8_t* __restrict__ rB)
                         __attribute__((always_inline)) {
#pragma unroll
            for (int h = 2; h < R; ++h)
                if (h % 2) issueB(w + (h - 2) * kHalf, 0, LD);
                else issueA(w + (h - 2) * kHalf, 0, LD);
            barrier_vm<(R - 2) * LD>();   // the first two halves
            read_b(rB, 0);
            read_a(rA, 0, 0, AH);
#pragma unroll
            for (int p = 0; p + 1 < kParts; ++p) step(p, rA, rB, none);
        };

        issueA(smem, 0, LD);
        issueB(smem + kHalf, 0, LD);
        start(smem + 2 * kHalf, smem, smem + kHalf);
        int u = 0;   // slot of the previous stage's A half; the ring's order is A B A B A ...
        auto slot = [&](int i) __attribute__((always_inline)) { return smem + (u + i >= R ? u + i - R : u + i) * kHalf; };
        for (int s = 1; s < nst; ++s) {
            barrier_vm<(R - 4) * LD>();   // stage s has landed
            uint8_t* w0 = slot(0);
            uint8_t* w1 = slot(1);
            const uint8_t* rA = slot(2);
            const uint8_t* rB = slot(3);
            u = u + 2 >= R ? u + 2 - R : u + 2;
            turn(w0, w1, rA, rB);
        }
        mma(kParts - 1, 0, AH);
    }
    // the prefetched (zero) stages land before the ring becomes the epilogue's scratch
    barrier_vm<0>();

    finish<E, EPI, GU, IB, JB>(G, acc, smem, wave, lane, m0 + wm * IB * 16, n0 + wn * (GU ? JB * 8 : JB * 16), split);
}

// Workgroup `block` of the `blocks` that share out the tiles and splits of G.
template <int E, int LA, int LB, int EPI, bool GU, int BM, int BN, int R>
__device__ __forceinline__ void tile(const Args& G, int block, int blocks) {
    int tm, tn, split;
    tile_of(block, G.mt, G.nt, blocks, tm, tn, split);
    tile_at<E, LA, LB, EPI, GU, BM, BN, R>(G, tm, tn, split);
}

template <int E, int LA, int LB, int EPI, bool GU, int BM, int BN, int R>
__global__ __launch_bounds__(tile_threads(BM)) __attribute__((amdgpu_waves_per_eu(tile_waves(BM, R)))) void tile_kernel(Args G) {
    tile<E, LA, LB, EPI, GU, BM, BN, R>(G, blockIdx.x, gridDim.x);
}

// Raises a kernel's LDS limit, once on each device.
template <class K>
bool allow_lds(DeviceCache& ready, K* kernel, int bytes) {
    return per_device(ready, [&] {
        return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess ? 1 : 0;
    }) != 0;
}

// Tiles of G: sets mt and nt and returns the number of workgroups.
inline long count_tiles(Args& G, int edge, int cols) {
    G.mt = (G.M + edge - 1) / edge;
    G.nt = (G.N + cols - 1) / cols;
    return (long)G.mt * G.nt * G.splits;
}

// Launches one tiling; mt, nt and the grid follow from the sizes in G.
template <int E, int LA, int LB, int EPI, bool GU, int BM, int BN, int R>
hipError_t launch_tiles(Args G, hipStream_t s) {
    auto* k = tile_kernel<E, LA, LB, EPI, GU, BM, BN, R>;
    static DeviceCache ready;
    if (!allow_lds(ready, k, tile_lds(BM, R))) return hipErrorInvalidValue;
    const long total = count_tiles(G, BM, GU ? BN / 2 : BN);
    if (!grid_fits(total, tile_threads(BM))) return hipErrorInvalidValue;
    k<<<dim3((unsigned)total), dim3(tile_threads(BM)), tile_lds(BM, R), s>>>(G);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace moe
