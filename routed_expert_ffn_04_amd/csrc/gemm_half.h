// The tile at the end of an expert's rows where they fill at most half of it: 128 x 256
// outputs by the 512 threads of a 256 x 256 tile (bf16, rows of A with k contiguous).
//
// A 256-row tile with 100 rows takes as long as a full one, even when the waves without
// rows stand aside: the products are halved, but a stage then lasts as long as its loads
// are under way, and half of what LDS holds of A are copies of the last row.  Here the 16
// KiB that A takes a stage leave room for a ring of four halves of A and three of B, two
// stages of loads under way, and the waves share out k instead of rows: four take the
// first 32 k of a stage and four the second, each for 128 x 64 outputs, and the pairs add
// their sums at the end, so that every SIMD keeps two waves.  Forward pass of 8 experts
// of 7168 x 2048: 128 rows each 251 -> 189 us, 384 rows 326 -> 286.  With 32 experts, whose
// weights stream from HBM all the time, it gives 1 to 2 %.
#pragma once
#include "gemm_tile.h"

namespace moe {
namespace gemm {

template <int LB, int EPI, bool GU>
__device__ __forceinline__ void half_tile(const Args& G, int m0, int tn) {
    constexpr int BM = 128, BN = 256, KE = kStage / 2;
    constexpr int IB = 8, JB = 4, AH = 4;
    constexpr int LDA = 2, LDB = 4;
    constexpr int kA = BM * kStage, kB = BN * kStage, kRingA = 4, kRingB = 3;
    static_assert(kRingA * kA + kRingB * kB <= tile_lds(256, 5), "the LDS of a whole tile");
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    uint8_t* const ringB = smem + kRingA * kA;
    const int tid = threadIdx.x, lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wk = wave / 4, wn = wave % 4;
    const int n0 = tn * (GU ? BN / 2 : BN);
    const int nst = (G.K + KE - 1) / KE;

    // ---- loads, as in tile_at
    uint32_t offa[LDA], offb[LDB];
#pragma unroll
    for (int q = 0; q < LDA; ++q) {
        const int at = (wave * LDA + q) * 64 + lane, r = at / 8, c = (at % 8) ^ row_key(r);
        offa[q] = (uint32_t)(min(m0 + r, G.A.n - 1) - m0) * (uint32_t)G.A.ld + c * 16;
    }
    const bool up = GU && wave * LDB * 8 >= BN / 2;
#pragma unroll
    for (int q = 0; q < LDB; ++q) {
        const int at = (wave * LDB + q) * 64 + lane;
        if constexpr (LB == kRow) {
            const int r = at / 8, c = (at % 8) ^ row_key(r);
            offb[q] = (uint32_t)(min(n0 + r - (up ? BN / 2 : 0), G.B.n - 1) - n0) * (uint32_t)G.B.ld + c * 16;
        } else {
            constexpr int per = BN * 2 / 16;
            const int r = at / per, c = (at % per) ^ col_key<BN>(r);
            offb[q] = (uint32_t)r * (uint32_t)G.B.ld + (min(n0 + c * 8, G.B.n - 8) - n0) * 2;
        }
    }
    const uint8_t* pa = G.A.p + (size_t)m0 * G.A.ld;
    const uint8_t* pb = LB == kRow ? (up ? G.B.p2 : G.B.p) + (size_t)n0 * G.B.ld : G.B.p + (size_t)n0 * 2;
    const int kr = ((lane % 8) ^ (lane / 8)) * 8, kc = wave * LDB * 2 + lane / 32;
    constexpr bool TWO = LB == kCol;
    const int turn = TWO && G.turn ? G.turn : 0x7fffffff;
    const ptrdiff_t past_a = TWO && G.turn ? G.A.p2 - (G.A.p + (size_t)G.turn * 2) : 0;
    const ptrdiff_t past_b = TWO && G.turn ? G.B.p2 - (G.B.p + (size_t)G.turn * G.B.ld) : 0;
    const int end1 = TWO && G.turn ? min(G.len, G.K) : G.K;
    int ka = 0, kb = 0;
    auto issueA = [&](uint8_t* half) __attribute__((always_inline)) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know the resource's type
        const int left = (TWO && ka >= turn ? G.K : end1) - ka;
        auto rows = __builtin_amdgcn_make_buffer_rsrc((void*)(TWO && ka >= turn ? pa + past_a : pa), 0, (int)kFar, 0x00027000);
#pragma unroll
        for (int q = 0; q < LDA; ++q) {
            const uint32_t at = (kr ^ (q & 1) * 8) >= left ? kFar : offa[q];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (lds_void*)(half + (wave * LDA + q) * 1024), 16, at, 0, 0, 0);
        }
#endif
        ka += KE;
        pa += kStage;
    };
    auto issueB = [&](uint8_t* half, int q0, int q1) __attribute__((always_inline)) {
#ifdef __HIP_DEVICE_COMPILE__
        const int left = (TWO && kb >= turn ? G.K : end1) - kb;
        auto rows = __builtin_amdgcn_make_buffer_rsrc((void*)(TWO && kb >= turn ? pb + past_b : pb), 0, (int)kFar, 0x00027000);
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            const int k = LB == kRow ? kr ^ (q & 1) * 8 : kc + q * 2;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (lds_void*)(half + (wave * LDB + q) * 1024), 16,
                                                     k >= left ? kFar : offb[q], 0, 0, 0);
        }
#endif
        if (q1 == LDB) {
            kb += KE;
            pb += LB == kRow ? (size_t)kStage : (size_t)KE * G.B.ld;
        }
    };

    // ---- products: the wave's k-step of every stage, in two parts (halves of the rows)
    f32x4 acc[IB][JB];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j] = f32x4{};
    const Frag<kRow, BM> fa(0, lane);
    const Frag<LB, BN> fb(wn * (GU ? JB / 2 : JB), lane);
    const int oa = wk ? fa.off[1] : fa.off[0];
    const int ob = LB == kRow ? (wk ? fb.off[LB == kRow] : fb.off[0]) : wk * 32 * (BN * 2);
    i32x4 a[2][AH], b[2][JB];   // a: by part; b: by stage
    auto read_a = [&](const uint8_t* half, int part, int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
        for (int i = i0; i < i1; ++i) a[part][i] = *(const i32x4*)(half + oa + (part * AH + i) * 16 * kStage);
    };
    auto read_b = [&](const uint8_t* half, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const uint8_t* from = half + (GU && j >= JB / 2 ? BN / 2 * kStage : 0);
            const int block = GU ? j % (JB / 2) : j;
            if constexpr (LB == kRow) b[s][j] = *(const i32x4*)(from + ob + block * 16 * kStage);
            else b[s][j] = fb.read(from + ob, block, 0);
        }
    };
    auto mma = [&](int part, int s, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            auto& c = acc[part * AH + i][j];
            c = Acc<kBf16>::mma(b[s][j], a[part][i], c);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto first_part = [&](int s, const uint8_t* rA) __attribute__((always_inline)) {
        mma(0, s, 0);
        read_a(rA, 1, 0, 2);
        __builtin_amdgcn_sched_barrier(0);
        mma(0, s, 1);
        read_a(rA, 1, 2, 4);
        __builtin_amdgcn_sched_barrier(0);
        mma(0, s, 2);
        mma(0, s, 3);
    };
    // The stage in rA, rB with the fragments of set s, beginning with the second part of
    // the stage before; wB takes the stage after next, wA the one after that.  (The
    // restrict qualifiers: tile_at.)
    auto go_on = [&](int s, uint8_t* __restrict__ wA, uint8_t* __restrict__ wB, const uint8_t* __restrict__ rA,
                     const uint8_t* __restrict__ rB) __attribute__((always_inline)) {
        mma(1, s ^ 1, 0);
        read_b(rB, s);
        __builtin_amdgcn_sched_barrier(0);
        issueB(wB, 0, 2);
        mma(1, s ^ 1, 1);
        read_a(rA, 0, 0, 2);
        __builtin_amdgcn_sched_barrier(0);
        issueB(wB, 2, 4);
        mma(1, s ^ 1, 2);
        read_a(rA, 0, 2, 4);
        __builtin_amdgcn_sched_barrier(0);
        issueA(wA);
        __builtin_amdgcn_sched_barrier(0);
        mma(1, s ^ 1, 3);
        first_part(s, rA);
    };
    auto start = [&](uint8_t* __restrict__ wA, uint8_t* __restrict__ wB, const uint8_t* __restrict__ rA,
                     const uint8_t* __restrict__ rB) __attribute__((always_inline)) {
        issueB(wB, 0, LDB);
        issueA(wA);
        read_b(rB, 0);
        read_a(rA, 0, 0, AH);
        __builtin_amdgcn_sched_barrier(0);
        first_part(0, rA);
    };
    constexpr int kLater = 2 * LDA + LDB;   // loads under way behind those that a stage waits for
    issueA(smem);
    issueB(ringB, 0, LDB);
    issueA(smem + kA);
    issueB(ringB + kB, 0, LDB);
    issueA(smem + 2 * kA);
    barrier_vm<kLater>();
    start(smem + 3 * kA, ringB + 2 * kB, smem, ringB);
    int ua = 0, ub = 0;   // slots of the stage before
    auto go = [&](int s) __attribute__((always_inline)) {
        barrier_vm<kLater>();
        uint8_t* wA = smem + ua * kA;
        uint8_t* wB = ringB + ub * kB;
        ua = (ua + 1) % kRingA;
        ub = ub + 1 == kRingB ? 0 : ub + 1;
        go_on(s, wA, wB, smem + ua * kA, ringB + ub * kB);
    };
    int s = 1;
    for (; s + 1 < nst; s += 2) {
        go(1);
        go(0);
    }
    if (s < nst) {
        go(1);
#pragma unroll
        for (int i = 0; i < AH; ++i) mma(1, 1, i);
    } else {
#pragma unroll
        for (int i = 0; i < AH; ++i) mma(1, 0, i);
    }
    barrier_vm<0>();

    // ---- the two sums of every output: each wave keeps half of its rows and adds the other's
    f32x4* mine = (f32x4*)(smem + wave * (AH * JB * 1024)) + lane;
    const f32x4* other = (const f32x4*)(smem + (wave ^ 4) * (AH * JB * 1024)) + lane;
#pragma unroll
    for (int i = 0; i < AH; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) mine[(i * JB + j) * 64] = wk ? acc[i][j] : acc[AH + i][j];
    __syncthreads();
    f32x4 sum[AH][JB];
#pragma unroll
    for (int i = 0; i < AH; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) sum[i][j] = (wk ? acc[AH + i][j] : acc[i][j]) + other[(i * JB + j) * 64];
    __syncthreads();
    finish<kBf16, EPI, GU, AH, JB>(G, sum, smem, wave, lane, m0 + wk * AH * 16, n0 + wn * (GU ? JB * 8 : JB * 16), 0);
}

}  // namespace gemm
}  // namespace moe
