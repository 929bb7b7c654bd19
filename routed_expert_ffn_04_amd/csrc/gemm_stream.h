// Weight gradients of many experts, dW[m][n] = sum over the expert's rows k of
// A[k][m] B[k][n], as one stream of stages (bf16).
//
// An expert's reduction is as long as it has rows, often a few hundred: a tile that
// fills its ring, multiplies, drains and stores by itself spends half of its time on the
// first and the last of these (256 x 256 outputs, 512 rows: 22 us, 12 of them
// products; the outputs of all CUs at once take 6 us to HBM).  Here a workgroup takes
// its tiles one after the other and its ring never drains: the loads of the next tile's first
// stages go out while the last ones of this tile multiply.
//
// Tile.  256 x 256 outputs, 8 waves (2 x 4) of 128 x 64, stages of 32 rows (32 KiB), a
// ring of four, and 4 KiB a wave for what leaves: all of LDS.  Rows of k are met as
// they are stored, in pieces of 512 bytes, so short stages cost nothing in the loads.
// (256 x 128 outputs and two workgroups a CU: more of the rows are read again from
// HBM, 4.0 ms against 3.3 for 2048 rows an expert; 128 x 128: 1.4 to 1.6 times as long.)
//
// The accumulators leave between two parts of a stage: 16 rows at a time through LDS,
// so that a store writes whole lines.  (64-byte pieces of 16 rows straight from registers
// take the address unit 3.9 us a tile, lines 1.2.)  Memory operations of a wave
// retire in the order of their issue, and a stage's loads go out before the stores of the same
// turn, so the stores of a tile have three stages to reach L2 before anything waits.
//
// Each die takes an eighth of every expert's tiles (it would have the long experts for
// itself otherwise), and its workgroups tiles next to each other.
#pragma once
#include "gemm_tile.h"

namespace moe {
namespace gemm {

struct SumProduct {
    const uint8_t* A; const uint8_t* B;   // element (row 0, column 0)
    uint32_t lda, ldb;                    // bytes from row to row
    int M, N, mt, nt;                     // mt x nt tiles an expert
    int half;                             // row tiles from here on are those of a second matrix of M rows,
    uint32_t skip;                        // with A this many bytes further right (the gate and up gradients share B)
    uint8_t* out; uint8_t* out2;
    size_t step;                          // bytes from expert to expert
    int per;                              // most tiles of an expert that a die has
};
struct Stream {
    SumProduct P[2];
    const int32_t* offsets;
    int n, R;                             // experts, rows
    int first, total;                     // of the second product, and all: n * per
};

// Rows before expert e's, whatever the offsets hold.  The offsets do not change during a
// kernel, so for a uniform e they are read through the scalar cache (the compiler would
// take vector loads behind the stores, and wait for everything that is under way).
typedef const __attribute__((address_space(4))) int32_t* Constants;
__device__ __forceinline__ int rows_before(const int32_t* offsets, int e, int R) {
    return min(max(((Constants)(uintptr_t)offsets)[e], 0), R);
}

// Position j of a die's sequence: product, expert and tile; false where the die
// has a tile less.
struct SumTile {
    int i, e, second, tm, tn;             // second: of the second matrix
};
__device__ __forceinline__ bool sum_tile(const Stream& S, int die, int j, SumTile& t) {
    t.i = j >= S.first;
    if (t.i) j -= S.first;
    const SumProduct& P = S.P[t.i];
    t.e = j / P.per;
    j -= t.e * P.per;
    const int x = (die + t.e) % kXcds, tiles = P.mt * P.nt;   // the dies with a tile more take turns
    const int base = tiles / kXcds, extra = tiles % kXcds;
    if (j >= base + (x < extra ? 1 : 0)) return false;
    band_of(x * base + min(x, extra) + j, P.mt, P.nt, t.tm, t.tn);
    t.second = t.tm >= P.half;
    if (t.second) t.tm -= P.half;
    return true;
}

constexpr int kStreamM = 256, kStreamN = 256, kStreamK = 32, kStreamRing = 4;
constexpr int kStreamSlot = (kStreamM + kStreamN) * 2 * kStreamK, kStreamPiece = 4096;
constexpr int kStreamLds = kStreamRing * kStreamSlot + 8 * kStreamPiece;

__device__ __forceinline__ void stream(const Stream& S) {
    constexpr int IB = 8, JB = 4, AH = 4;                  // 16 x 16 blocks of a wave; of a part of its rows
    constexpr int LA = 2, LB = 2, L = LA + LB;             // loads of a lane and stage
    constexpr int R = kStreamRing;
    constexpr int kStores = IB * JB / 2;                   // of a wave and tile
    constexpr int KA = kStreamM * 2 * kStreamK;            // bytes of A in a slot
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wm = wave / 4, wn = wave % 4;
    const int die = blockIdx.x % kXcds, stride = gridDim.x / kXcds;

    auto next = [&](int j, SumTile& t) __attribute__((always_inline)) {
        while (j < S.total && !sum_tile(S, die, j, t)) j += stride;
        return j;
    };
    auto rows_of = [&](const SumTile& t, int& first) __attribute__((always_inline)) {
        first = rows_before(S.offsets, t.e, S.R);
        return max(rows_before(S.offsets, t.e + 1, S.R) - first, 0);
    };

    // ---- loads of a stage.  Slots of 16 bytes: rows kr + 2 q, chunk c.
    const int kr = wave * 4 + lane / 32;
    const uint8_t* pa;     // of the next stage
    const uint8_t* pb;
    uint32_t offa[LA], offb[LB], lda, ldb;
    int left, jl;          // rows from there on; its tile
    auto set = [&](const SumTile& t) __attribute__((always_inline)) {
        const SumProduct& P = S.P[t.i];
        int first;
        left = rows_of(t, first);
        lda = P.lda;
        ldb = P.ldb;
        const int m0 = t.tm * kStreamM, n0 = t.tn * kStreamN;
        pa = P.A + (size_t)first * lda + (size_t)m0 * 2 + (t.second ? P.skip : 0);
        pb = P.B + (size_t)first * ldb + (size_t)n0 * 2;
#pragma unroll
        for (int q = 0; q < LA; ++q) {
            const int r = kr + 2 * q, c = (lane % 32) ^ col_key<kStreamM>(r);
            offa[q] = (uint32_t)r * lda + min(c * 8, P.M - 8 - m0) * 2;
        }
#pragma unroll
        for (int q = 0; q < LB; ++q) {
            const int r = kr + 2 * q, c = (lane % 32) ^ col_key<kStreamN>(r);
            offb[q] = (uint32_t)r * ldb + min(c * 8, P.N - 8 - n0) * 2;
        }
    };
    // Loads [q0, q1) of the next stage.  A tile has an even number of stages; last: the second of a pair.
    auto issue = [&](uint8_t* slot, int q0, int q1, bool last) __attribute__((always_inline)) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know the resource's type
        auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)pa, 0, (int)kFar, 0x00027000);
        auto rb = __builtin_amdgcn_make_buffer_rsrc((void*)pb, 0, (int)kFar, 0x00027000);
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            if (q < LA) {
                const uint32_t at = kr + 2 * q >= left ? kFar : offa[q];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(slot + (wave * LA + q) * 1024), 16, at, 0, 0, 0);
            } else {
                const int p = q - LA;
                const uint32_t at = kr + 2 * p >= left ? kFar : offb[p];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(slot + KA + (wave * LB + p) * 1024), 16, at, 0, 0, 0);
            }
        }
#endif
        if (q1 == L) {
            pa += (size_t)kStreamK * lda;
            pb += (size_t)kStreamK * ldb;
            left -= kStreamK;
            if (last && left <= 0 && jl < S.total) {
                SumTile t;
                jl = next(jl + stride, t);
                if (jl < S.total) set(t);
            }
        }
    };

    SumTile cur;
    int jc = next(blockIdx.x / kXcds, cur);   // the tile that multiplies
    if (jc >= S.total) return;
    jl = jc;
    set(cur);
    auto pairs = [&](const SumTile& t) __attribute__((always_inline)) {   // of stages; without rows one, of zeros
        int first;
        return max((rows_of(t, first) + 2 * kStreamK - 1) / (2 * kStreamK), 1);
    };
    int todo = pairs(cur);

    f32x4 acc[IB][JB];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < IB; ++i)
#pragma unroll
            for (int j = 0; j < JB; ++j) acc[i][j] = f32x4{};
    };
    clear();
    // acc[i][j][v]: m = 16 i + l % 16, n = 16 j + 4 (l / 16) + v of the wave's part.  16
    // rows at a time pass through the wave's piece of LDS (two halves in turn; chunk c of 16 bytes of
    // row r at c ^ r % 8), so that a store writes whole lines: 8 rows of 128 bytes.
    // Whether all kStores stores went out.
    auto store = [&](const SumTile& t, uint8_t* piece) __attribute__((always_inline)) {
        const SumProduct& P = S.P[t.i];
        const int mw = t.tm * kStreamM + wm * 128, nw = t.tn * kStreamN + wn * 64;
        const bool whole = mw + 128 <= P.M && nw + 64 <= P.N;
        const uint32_t ld = (uint32_t)P.N * 2, at = (lane / 8) * ld + (lane % 8) * 16;
        uint8_t* base = (t.second ? P.out2 : P.out) + (size_t)t.e * P.step + (size_t)mw * ld + (size_t)nw * 2;
        const int r = lane % 16, g = lane / 16;
        uint8_t* in = piece + r * 128 + (g & 1) * 8;
        const uint8_t* out = piece + (lane / 8) * 128 + ((lane % 8) ^ (lane / 8)) * 16;
        auto pass = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const f32x4 v = acc[i][j];
                *(uint2*)(in + (i & 1) * 2048 + (((2 * j + (g >> 1)) ^ (r & 7)) << 4)) =
                    make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
            }
        };
        // non-temporal: gradients would push the rows that the die shares out of its L2
        auto put = [&](uint8_t* base, i32x4 v) __attribute__((always_inline)) { __builtin_nontemporal_store(v, (i32x4*)(base + at)); };
        auto row8 = [&](int i, int q) __attribute__((always_inline)) { return *(const i32x4*)(out + (i & 1) * 2048 + q * 1024); };
        if (whole) {
#pragma unroll
            for (int i = 0; i < IB; ++i) {
                wave_sync();
                pass(i);
                wave_sync();
#pragma unroll
                for (int q = 0; q < 2; ++q, base += 8 * (size_t)ld) put(base, row8(i, q));
            }
        } else {
#pragma unroll
            for (int i = 0; i < IB; ++i) {
                wave_sync();
                pass(i);
                wave_sync();
#pragma unroll
                for (int q = 0; q < 2; ++q, base += 8 * (size_t)ld) {
                    const i32x4 v = row8(i, q);
                    if (mw + 16 * i + 8 * q + lane / 8 < P.M && nw + (lane % 8) * 8 < P.N) put(base, v);
                }
            }
        }
        return whole;
    };

    // ---- products.  A stage is two parts, the halves of the wave's rows; the fragments of
    // the next part are read while one multiplies.
    const Frag<kCol, kStreamM> fa(wm * IB, lane);
    const Frag<kCol, kStreamN> fb(wn * JB, lane);
    i32x4 a[2][AH], b[2][JB];   // a: by part; b: by stage
    auto read_a = [&](const uint8_t* slot, int part, int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
        for (int i = i0; i < i1; ++i) a[part][i] = fa.read(slot, part * AH + i, 0);
    };
    auto read_b = [&](const uint8_t* slot, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < JB; ++j) b[s][j] = fb.read(slot + KA, j, 0);
    };
    auto mma = [&](int part, int s, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            auto& c = acc[part * AH + i][j];
            c = Acc<kBf16>::mma(b[s][j], a[part][i], c);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // The first part of a stage, while the second one's fragments are read.
    auto first_part = [&](int s, const uint8_t* r) __attribute__((always_inline)) {
        mma(0, s, 0);
        read_a(r, 1, 0, 2);
        __builtin_amdgcn_sched_barrier(0);
        mma(0, s, 1);
        read_a(r, 1, 2, 4);
        __builtin_amdgcn_sched_barrier(0);
        mma(0, s, 2);
        mma(0, s, 3);
    };
    int kept = 0;   // which of the last R - 1 turns stored a whole tile, by bits
    // Stage in slot r with the fragments of set s, beginning with the second part of
    // the stage before; the slot w takes the stage after next.  (The restrict
    // qualifiers: gemm_tile.h.)
    SumTile nxt;
    int jn = 0;
    auto turn = [&](int s, uint8_t* __restrict__ w, const uint8_t* __restrict__ r, uint8_t* __restrict__ piece, bool ended) __attribute__((always_inline)) {
        mma(1, s ^ 1, 0);
        read_b(r, s);
        __builtin_amdgcn_sched_barrier(0);
        issue(w, 0, 1, (s + R - 1) & 1);
        mma(1, s ^ 1, 1);
        read_a(r, 0, 0, 2);
        __builtin_amdgcn_sched_barrier(0);
        issue(w, 1, 2, (s + R - 1) & 1);
        mma(1, s ^ 1, 2);
        read_a(r, 0, 2, 4);
        __builtin_amdgcn_sched_barrier(0);
        issue(w, 2, 4, (s + R - 1) & 1);
        __builtin_amdgcn_sched_barrier(0);
        mma(1, s ^ 1, 3);
        kept = kept << 1 & ((1 << (R - 1)) - 1);
        if (ended) {
            kept |= store(cur, piece);
            clear();
            cur = nxt;
            jc = jn;
            todo = pairs(cur);
            __builtin_amdgcn_sched_barrier(0);
        }
        first_part(s, r);
    };
    auto start = [&](uint8_t* __restrict__ w, const uint8_t* __restrict__ r) __attribute__((always_inline)) {
        issue(w, 0, L, (R - 1) & 1);
        read_b(r, 0);
        read_a(r, 0, 0, AH);
        __builtin_amdgcn_sched_barrier(0);
        first_part(0, r);
    };
#pragma unroll
    for (int k = 0; k + 1 < R; ++k) issue(smem + k * kStreamSlot, 0, L, k & 1);
    barrier_vm<(R - 2) * L>();   // the first stage
    start(smem + (R - 1) * kStreamSlot, smem);
    int u = 0;   // slot of the stage before
    auto go = [&](int s, bool ended) __attribute__((always_inline)) {
        // The stage has landed: after its loads came those of R - 2 stages, and the stores
        // of a tile if one of the R - 1 turns since then stored it.
        if (kept) barrier_vm<(R - 2) * L + kStores>();
        else barrier_vm<(R - 2) * L>();
        uint8_t* w = smem + u * kStreamSlot;
        u = u + 1 == R ? 0 : u + 1;
        turn(s, w, smem + u * kStreamSlot, smem + R * kStreamSlot + wave * kStreamPiece, ended);
    };
    for (;;) {
        go(1, false);
        const bool ended = --todo == 0;
        if (ended) {
            jn = next(jc + stride, nxt);
            if (jn >= S.total) break;
        }
        go(0, ended);
    }
#pragma unroll
    for (int i = 0; i < AH; ++i) mma(1, 1, i);
    store(cur, smem + R * kStreamSlot + wave * kStreamPiece);
    barrier_vm<0>();   // no load is under way when the workgroup's LDS is given to another
}

}  // namespace gemm
}  // namespace moe
