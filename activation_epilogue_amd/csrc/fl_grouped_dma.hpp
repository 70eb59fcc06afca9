// fl_grouped_dma.hpp -- the experts' products: tiles fed by direct-to-LDS loads
// through a ring of K stages, MFMA blocks of 16x16 outputs.
//
// The three forms of fl_grouped.hpp differ in how an operand lies in memory:
//   forward   A rows K-contiguous (optionally read through an index), B[e] N-contiguous
//   backward  G rows K-contiguous, W[e] rows K-contiguous
//   gradient  A and G both with the summed dimension (the rows of the run) outermost
// so an operand's tile is either a set of rows of consecutive k (KC) or k-rows
// of consecutive columns (KR), and the tile code is the same for all.  A stage
// is 128 bytes of k: 64 k of 16-bit operands, 32 of fp32.
//
//   * Copies: one buffer load with the LDS bit moves 64 x 16 bytes into 1 KB of
//     LDS; the bank swizzle is applied on the global side.  Rows outside the
//     run, columns past the operand and k past the end get an offset that the
//     hardware's range check turns into zeros, so a partial tile costs no
//     traffic for what it lacks.  Pointers need element alignment only.
//   * MFMA operands: KC tiles are read with 16-byte reads, KR tiles with the
//     transposing 8-byte read (two for 8 consecutive k of one column; fp32:
//     four 4-byte reads of consecutive columns).  A 16-byte read holds 4 fp32
//     k, which four 16x16x4 MFMAs take one each: MFMA j sums k = 4*g + j over
//     the lane groups g, in both operands alike.
//   * A stage is two blocks of MFMAs.  The reads of the next block are
//     slotted between the MFMAs of the current one; the one barrier per stage
//     stands before the second block, which also issues the copies of the
//     stage NBUF ahead into the buffer that the barrier has freed.
//   * Epilogue: 16 rows at a time, a wave's accumulators pass through LDS so
//     that a lane then holds 16 bytes of one row: Y, X, pre and out move in
//     whole 128-byte lines per instruction.
//
// Measured (bf16, 8192x2 rows of 8 experts, K 4096, N 14336): forward with the
// pre-activation 1120 to 1180, backward 1170, weight gradient 1160 to 1175
// TFLOP/s (a dense library product of that size: 1370, 1570 with its right operand
// K-contiguous).  No one limit is reached: the matrix cores are busy 57 to 61% of
// the cycles, the waves wait 35 to 38% of theirs, and 6.7 GB a product (3.7 the
// gradient) come past the L2s, 4.1 TB/s.  32 tokens through 64 experts of
// 2048x1408, of which they meet 52: 5.5 TB/s of weights, bound by reading them;
// 4096 tokens through all: 730 TFLOP/s, bound by how runs of 384 rows fill tiles
// and rounds (4.1 rounds of work take 6).
#pragma once

#include "fl_dma16.hpp"
#include "fl_grouped.hpp"

namespace fl {


// A 16-bit load and its wait in one asm block: a load that the compiler tracks,
// on a branch of the K loop, would make it drain all copies in flight before
// later LDS reads.
__device__ __forceinline__ uint32_t load_u16_at(const void *p) {
    uint32_t v;
    asm volatile("global_load_ushort %0, %1, off\n\ts_waitcnt vmcnt(0)" : "=&v"(v) : "v"(p) : "memory");
    return v & 0xffffu;
}

// lds_copy16 with the streaming policy bit.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16_nt(i32x4_t rsrc, uint32_t voffset, uint32_t soffset, uint32_t lds_addr) {
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds" ::"v"(voffset), "s"(rsrc),
                 "s"(soffset), "s"(lds_addr)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// One operand's tile: R rows (KC) or R columns (KR), copied by WAVES waves.
template <int DT, int R, int WAVES, bool KC>
struct GroupedSide {
    static constexpr int ES = Io<DT>::size, EPC = 16 / ES;  // bytes of an element, elements of a chunk
    static constexpr int KS = 128 / ES;                     // k per stage
    static constexpr int ROW = R * ES;                      // KR: bytes of a k-row
    static constexpr int BYTES = R * 128;
    static constexpr int COPIES = R / (8 * WAVES);  // per wave and stage
    static constexpr int CB = ROW / 16;             // KR: chunks per k-row
    static constexpr int PARTS = KC ? 1 : ES;       // LDS reads per MFMA operand
    static_assert(COPIES >= 1 && COPIES * 8 * WAVES == R, "whole copies");
    static_assert(KC || CB == 16 || CB == 32, "KR swizzle");

    i32x4_t rsrc;
    uint32_t off[COPIES];  // byte offset of the lane's chunk at k = 0, kOob outside the operand
    int frag;              // LDS address of the wave's first operand read within the side (KC: at chunk 0)
    int fk;                // KC: chunk xor of the lane's row

    // 16-byte reads of 16 consecutive rows at one chunk per 16 lanes fall on
    // distinct banks (KC)
    __device__ __forceinline__ static int fa(int r) { return ((r >> 1) ^ ((r & 1) << 2)) & 7; }
    // KR: the 4 k-rows (and those 8 further) of a transposing read, or the
    // k-rows 4 apart of a 4-byte read, fall on distinct banks; always even
    __device__ __forceinline__ static int fb(int r) {
        if constexpr (ES == 4)
            return r & 12;
        else
            return ((0xAC60 >> (4 * (r & 3))) & 0xF) ^ ((r >> 2) & 2);
    }

    // Lane's place in copy i: its row (KC) or k-row (KR), and its chunk.
    __device__ __forceinline__ static void place(int wave, int lane, int i, int &row, int &chunk) {
        const int q = 64 * (wave * COPIES + i) + lane;
        if constexpr (KC) {
            row = q >> 3;
            chunk = (q & 7) ^ fa(row);
        } else {
            row = q / CB;
            chunk = (q % CB) ^ fb(row);
        }
    }

    // Copy i's k within the stage.
    __device__ __forceinline__ static int k(int wave, int lane, int i) {
        int row, chunk;
        place(wave, lane, i, row, chunk);
        return KC ? chunk * EPC : row;
    }

    // Operand reads for output rows (columns) w0 .. of the tile.
    __device__ __forceinline__ void set_frag(int w0, int lane) {
        const int g = lane >> 4, i = lane & 15;
        fk = 0;
        if constexpr (KC) {
            frag = (w0 + i) * 128;
            fk = g ^ fa(i);  // w0 is a multiple of 16; block kk flips bit 2
        } else if constexpr (ES == 2) {
            const int rk = g * 8 + (i >> 2), n = w0 + 4 * (i & 3);
            frag = rk * ROW + (((n >> 3) ^ fb(rk)) * 16) + ((n >> 2) & 1) * 8;
        } else {
            const int n = w0 + i;
            frag = g * 4 * ROW + (((n >> 2) ^ fb(g * 4)) * 16) + (n & 3) * 4;
        }
    }
    // Read P of the operand of 16-row block b at MFMA block kk.  (KR: the
    // wave's first column is a multiple of its columns, a power of two, so
    // that block b is one xor away.)
    template <int P>
    __device__ __forceinline__ void read(const FL_LDS char *s, int b, int kk, i32x2_t (&v)[2]) const {
        if constexpr (KC) {
            const u32x4_t t = *(const FL_LDS u32x4_t *)(s + frag + ((fk ^ (kk * 4)) * 16) + b * (16 * 128));
            v[0] = i32x2_t{(int)t[0], (int)t[1]};
            v[1] = i32x2_t{(int)t[2], (int)t[3]};
        } else if constexpr (ES == 2) {
            v[P] = __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((
                                                   FL_LDS s16x4_t *)(s + (frag ^ (b * 32)) + (kk * 32 + P * 4) * ROW)));
        } else {
            v[P >> 1][P & 1] = *(const FL_LDS int *)(s + (frag ^ (b * 64)) + (kk * 16 + P) * ROW);
        }
    }

    // Puts right what 16-byte copies get wrong in the last stage (kleft k of it
    // exist), on the chunks that this wave copied, after they landed:
    //  * the range check works on whole dwords, so an odd last 16-bit element
    //    of the operand reads as zero: it is loaded again by itself;
    //  * a KC chunk that crosses the end of k holds values of the next row.
    // left: elements from the stage's origin to the end of the operand; last:
    // its last element.
    __device__ __forceinline__ void fix_tail(FL_LDS char *s, int wave, int lane, int64_t left, int kleft,
                                             const void *last) const {
        if (ES == 4 && !KC) return;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int kc = k(wave, lane, i);
            if (off[i] == kOob || kc >= kleft) continue;
            const int64_t rest = left - (int64_t)(off[i] / ES);  // elements from the chunk's first to the end
            const int valid = kleft - kc;
            const bool odd = ES == 2 && rest < 8 && (rest & 1);
            if (!odd && (!KC || valid >= EPC)) continue;
            FL_LDS char *p = s + (wave * COPIES + i) * 1024 + lane * 16;
            u32x4_t v = *(FL_LDS u32x4_t *)p;
            if (odd) {
                const uint32_t x = load_u16_at(last);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (d == (int)(rest >> 1)) v[d] = x;  // (the element after it is past the end)
            }
            if constexpr (KC) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int n = valid * ES - 4 * d;  // bytes of dword d that exist
                    v[d] &= n >= 4 ? 0xffffffffu : n == 2 ? 0xffffu : 0u;
                }
            }
            *(FL_LDS u32x4_t *)p = v;
        }
    }
};

// One tile of BM x BN outputs on WM x WN waves.  NBUF stages of LDS.  NT: the
// weights stream past the L2.
template <int DT, int FORM, int BM_, int BN_, int WM, int WN, int NBUF_, bool NT>
struct GroupedTile {
    using io = Io<DT>;
    using raw = typename io::raw;
    static constexpr int BM = BM_, BN = BN_, NBUF = NBUF_;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int TM = BM / WM, TN = BN / WN, NRB = TM / 16, NI = TN / 16;
    using SideA = GroupedSide<DT, BM, WAVES, FORM != kFormGrad>;
    using SideB = GroupedSide<DT, BN, WAVES, FORM == kFormBwd>;
    static constexpr int ES = SideA::ES, EPC = SideA::EPC, KS = SideA::KS;
    static constexpr int MPB = ES == 4 ? 4 : 1;  // MFMAs per pair of operand reads
    static constexpr int BUF_BYTES = SideA::BYTES + SideB::BYTES;
    static constexpr int COPIES = SideA::COPIES + SideB::COPIES;
    static constexpr int SLOTS = NRB * NI * MPB;
    static constexpr int RA = SideA::PARTS, RB = SideB::PARTS, READS = NRB * RA + NI * RB;
    static constexpr int EPI_ROW = TN * 4 + 16;
    static constexpr int EPI_BYTES = WAVES * 16 * EPI_ROW;
    static constexpr int SMEM = NBUF * BUF_BYTES;
    static_assert(NBUF >= 2 && SMEM <= 163840 && EPI_BYTES <= BUF_BYTES, "LDS");
    static_assert((TN & (TN - 1)) == 0 && (TM & (TM - 1)) == 0, "power-of-two wave tiles");

    // A wave's place in the tile.  Waves w and w + 4 share a SIMD and differ in
    // their row and, shifted by half the columns, their column: where half of
    // the tile's rows or columns do not exist, each SIMD keeps one wave that
    // works, alone and so at twice the rate.
    __device__ __forceinline__ static int row_of(int wave) { return wave / WN; }
    __device__ __forceinline__ static int col_of(int wave) { return (wave + (wave >> 2) * (WN / 2)) % WN; }

    struct Ops {
        SideA A;
        SideB B;
        const char *pa, *pb;   // gradient: the stage's origin in A and G
        int64_t ra, rb;        // elements from the descriptor bases (gradient: the stage's origin) to the end
        int lda, ldb, depth;
    };
    struct Frags {
        i32x2_t a[NRB][2], b[NI][2];
    };

    struct Dst {  // LDS addresses of a wave's first copy of either operand
        uint32_t a, b;
    };
    // Copy I of stage kt (A's first).  CHECK: the stage may reach past the end
    // of k, where zeros are copied; all stages issue the same copies, so that
    // the waits are on constants.
    template <int I, bool CHECK>
    __device__ __forceinline__ static void copy_one(const Ops &o, int kt, Dst buf, int wave, int lane) {
        const int kleft = (int)((uint32_t)o.depth - (uint32_t)kt * KS);  // (kt * KS may pass 2^31 by itself)
        if constexpr (I < SideA::COPIES) {
            const uint32_t so = FORM == kFormGrad ? 0 : (uint32_t)kt * 128;
            const bool ok = !CHECK || SideA::k(wave, lane, I) < kleft;
            lds_copy16(o.A.rsrc, ok ? o.A.off[I] : kOob, so, buf.a + I * 1024);
        } else {
            constexpr int i = I - SideA::COPIES;
            const uint32_t so = FORM == kFormGrad  ? 0
                                : FORM == kFormBwd ? (uint32_t)kt * 128
                                                   : (uint32_t)kt * 128 * (uint32_t)o.ldb;
            const bool ok = !CHECK || SideB::k(wave, lane, i) < kleft;
            if constexpr (NT)
                lds_copy16_nt(o.B.rsrc, ok ? o.B.off[i] : kOob, so, buf.b + i * 1024);
            else
                lds_copy16(o.B.rsrc, ok ? o.B.off[i] : kOob, so, buf.b + i * 1024);
        }
    }
    template <int C0, int C1, bool CHECK>
    __device__ __forceinline__ static void copy_range(const Ops &o, int kt, Dst buf, int wave, int lane) {
        if constexpr (C0 < C1) {
            copy_one<C0, CHECK>(o, kt, buf, wave, lane);
            copy_range<C0 + 1, C1, CHECK>(o, kt, buf, wave, lane);
        }
    }
    __device__ __forceinline__ static Dst copy_base(uint32_t lds, int b, int wave) {
        const uint32_t s = lds + b * BUF_BYTES;
        return {(uint32_t)__builtin_amdgcn_readfirstlane(s + wave * SideA::COPIES * 1024),
                (uint32_t)__builtin_amdgcn_readfirstlane(s + SideA::BYTES + wave * SideB::COPIES * 1024)};
    }

    // The gradient's operands may span more than 2 GiB: their descriptors move
    // with the stages instead of a 32-bit offset.  pa, pb, ra, rb are those of
    // the stage copied last.
    __device__ __forceinline__ static void set_descriptors(Ops &o) {
        o.A.rsrc = sgpr_rsrc(o.pa, o.ra > 0 ? (size_t)o.ra * ES : 0);
        o.B.rsrc = sgpr_rsrc(o.pb, o.rb > 0 ? (size_t)o.rb * ES : 0);
    }
    __device__ __forceinline__ static void next_stage(Ops &o) {
        if constexpr (FORM == kFormGrad) {
            const int64_t da = (int64_t)KS * o.lda, db = (int64_t)KS * o.ldb;
            o.pa += da * ES;
            o.pb += db * ES;
            o.ra -= da;
            o.rb -= db;
            set_descriptors(o);
        }
    }

    template <int P>
    __device__ __forceinline__ static void read_piece(const Ops &o, const FL_LDS char *s, int kk, Frags &f) {
        // in the order the MFMAs take them: a0, b0 .. , a1 ..
        if constexpr (P < RA) {
            o.A.template read<P>(s, 0, kk, f.a[0]);
        } else if constexpr (P < RA + NI * RB) {
            constexpr int q = P - RA;
            o.B.template read<q % RB>(s + SideA::BYTES, q / RB, kk, f.b[q / RB]);
        } else {
            constexpr int q = P - NI * RB;
            o.A.template read<q % RA>(s, q / RA, kk, f.a[q / RA]);
        }
    }
    template <int P0, int P1>
    __device__ __forceinline__ static void read_range(const Ops &o, const FL_LDS char *s, int kk, Frags &f) {
        if constexpr (P0 < P1) {
            read_piece<P0>(o, s, kk, f);
            read_range<P0 + 1, P1>(o, s, kk, f);
        }
    }

    // MFMA I of a block, rows of blocks in snake order: consecutive MFMAs
    // share an operand (fewer operand bits toggle, a higher clock).
    template <int I>
    __device__ __forceinline__ static void mma(const Frags &f, f32x4_t (&acc)[NRB][NI]) {
        constexpr int q = I / MPB, mi = q / NI, ni = (mi & 1) ? NI - 1 - q % NI : q % NI;
        if constexpr (DT == FL_F32) {
            constexpr int j = I % MPB;
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __builtin_bit_cast(f32x2_t, f.b[ni][j >> 1])[j & 1], __builtin_bit_cast(f32x2_t, f.a[mi][j >> 1])[j & 1],
                acc[mi][ni], 0, 0, 0);
            return;
        }
        const auto av = __builtin_shufflevector(f.a[mi][0], f.a[mi][1], 0, 1, 2, 3);
        const auto bv = __builtin_shufflevector(f.b[ni][0], f.b[ni][1], 0, 1, 2, 3);
        if constexpr (DT == FL_F16)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, bv),
                                                                 __builtin_bit_cast(f16x8_t, av), acc[mi][ni], 0, 0, 0);
        else
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, bv),
                                                                  __builtin_bit_cast(bf16x8_t, av), acc[mi][ni], 0, 0, 0);
    }

    // One block: the MFMAs on `use`, the reads of block kk of `s` into `fill`
    // and the copies (0 none, 1 unchecked, 2 checked) of stage kt into `buf`
    // spread over them.
    template <int I, int COPY>
    __device__ __forceinline__ static void block(const Ops &o, const FL_LDS char *s, int kk, int kt, Dst buf,
                                                 int wave, int lane, const Frags &use, Frags &fill,
                                                 f32x4_t (&acc)[NRB][NI]) {
        if constexpr (I < SLOTS) {
            mma<I>(use, acc);
            if constexpr (COPY != 0)
                copy_range<(I * COPIES + SLOTS - 1) / SLOTS, ((I + 1) * COPIES + SLOTS - 1) / SLOTS, COPY == 2>(
                    o, kt, buf, wave, lane);
            read_range<I * READS / SLOTS, (I + 1) * READS / SLOTS>(o, s, kk, fill);
            __builtin_amdgcn_sched_barrier(0);
            block<I + 1, COPY>(o, s, kk, kt, buf, wave, lane, use, fill, acc);
        }
    }

    template <int N>
    __device__ __forceinline__ static void wait_vm() {
        __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
        asm volatile("" ::: "memory");
    }

    __device__ __forceinline__ static bool ragged(const GroupedArgs &a) {
        if (FORM == kFormBwd || ES == 4) return a.K % EPC;
        return (a.K | a.N) % EPC;
    }
    // fix_tail of both sides for stage kt; `ahead` stages after it are copied.
    __device__ __forceinline__ static void fix_tail(const GroupedArgs &a, const Ops &o, int kt, int ahead, int wave,
                                                    int lane, FL_LDS char *s) {
        const int64_t k0 = (int64_t)kt * KS;
        const int kleft = (int)(o.depth - k0);
        int64_t la = o.ra - k0, lb = o.rb - (FORM == kFormBwd ? k0 : k0 * o.ldb);
        if constexpr (FORM == kFormGrad) {
            la = o.ra + (int64_t)ahead * KS * o.lda;
            lb = o.rb + (int64_t)ahead * KS * o.ldb;
        }
        const int64_t nb = FORM == kFormGrad ? (int64_t)a.S * a.N : (int64_t)a.E * a.K * a.N;
        o.A.fix_tail(s, wave, lane, la, kleft, static_cast<const raw *>(a.A) + (a.A_rows * a.K - 1));
        o.B.fix_tail(s + SideA::BYTES, wave, lane, lb, kleft, static_cast<const raw *>(a.B) + (nb - 1));
    }

    // Stage kt in LDS buffer `buf`; its block 0 operands are in f[0].
    template <bool TAIL>
    __device__ __forceinline__ static void stage(const GroupedArgs &a, Ops &o, const FL_LDS char *lds, uint32_t addr,
                                                 int kt, int nk, int buf, int wave, int lane, Frags (&f)[2],
                                                 f32x4_t (&acc)[NRB][NI]) {
        block<0, 0>(o, lds + buf * BUF_BYTES, 1, 0, Dst{}, wave, lane, f[0], f[1], acc);
        const FL_LDS char *nxt = lds + (buf + 1 == NBUF ? 0 : buf + 1) * BUF_BYTES;
        turn<TAIL>(a, o, nxt, kt, nk, wave, lane);
        block<0, TAIL ? 2 : 1>(o, nxt, 0, kt + NBUF, copy_base(addr, buf, wave), wave, lane, f[1], f[0], acc);
    }

    // Between the blocks of stage kt: stage kt+1 has landed (in `nxt`), put
    // right if it is the last, and every wave is done with stage kt's buffer.
    template <bool TAIL>
    __device__ __forceinline__ static void turn(const GroupedArgs &a, Ops &o, const FL_LDS char *nxt, int kt, int nk,
                                                int wave, int lane) {
        if constexpr (TAIL) {
            if (ragged(a) && kt + 2 == nk) {
                wait_vm<(NBUF - 2) * COPIES>();  // the last stage has landed
                fix_tail(a, o, kt + 1, NBUF - 2, wave, lane, (FL_LDS char *)nxt);
            }
        }
        wait_vm<(NBUF - 2) * COPIES>();
        __syncthreads();
        next_stage(o);
    }

    // Copies of stages B0 .. B1-1 into the buffers of their numbers.
    template <int B0, int B1>
    __device__ __forceinline__ static void prefetch(Ops &o, int wave, int lane, uint32_t addr) {
#pragma unroll
        for (int b = B0; b < B1; ++b) {
            if (b > 0) next_stage(o);
            copy_range<0, COPIES, true>(o, b, copy_base(addr, b, wave), wave, lane);
        }
    }

    // The tile's product; stages 0 .. NBUF-1 are on their way.  An idle wave
    // (none of its outputs exist) only does its share of the copies.
    __device__ __forceinline__ static void product(const GroupedArgs &a, Ops &o, bool idle, int wave, int lane,
                                                   const FL_LDS char *lds, uint32_t addr, f32x4_t (&acc)[NRB][NI]) {
#pragma unroll
        for (int mi = 0; mi < NRB; ++mi)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        const int nk = o.depth > 0 ? (int)(((int64_t)o.depth + KS - 1) / KS) : 1;  // (no k: one stage of zeros)
        // whatever the epilogue before left in flight came after stage 0
        wait_vm<(NBUF - 1) * COPIES>();
        if (nk == 1 && ragged(a)) fix_tail(a, o, 0, NBUF - 1, wave, lane, (FL_LDS char *)lds);
        __syncthreads();
        int buf = 0, kt = 0;
        if (idle) {
#pragma unroll 1
            for (; kt < nk; ++kt) {
                asm volatile("" : "+v"(lane));
                const int next = buf + 1 == NBUF ? 0 : buf + 1;
                turn<true>(a, o, lds + next * BUF_BYTES, kt, nk, wave, lane);
                copy_range<0, COPIES, true>(o, kt + NBUF, copy_base(addr, buf, wave), wave, lane);
                buf = next;
            }
        } else {
            Frags f[2];
            read_range<0, READS>(o, lds, 0, f[0]);
#pragma unroll 1
            for (; kt < nk - (NBUF + 1); ++kt) {  // stages that copy a whole stage
                stage<false>(a, o, lds, addr, kt, nk, buf, wave, lane, f, acc);
                buf = buf + 1 == NBUF ? 0 : buf + 1;
            }
            int lt = lane;
#pragma unroll 1
            for (; kt < nk; ++kt) {
                asm volatile("" : "+v"(lt));  // what the checks derive from the lane is computed here, not kept
                stage<true>(a, o, lds, addr, kt, nk, buf, wave, lt, f, acc);
                buf = buf + 1 == NBUF ? 0 : buf + 1;
            }
        }
        // the look-ahead copies past the end land before the LDS is used again
        wait_vm<0>();
        __syncthreads();
    }

    // ---- epilogue: 16 bytes of a row in a lane
    static constexpr int VEC = EPC;  // columns
    struct Piece16 {
        u32x4_t w;
        __device__ __forceinline__ float get(int e) const {
            if constexpr (ES == 4)
                return __builtin_bit_cast(float, (uint32_t)w[e]);
            else
                return io::to_f32((raw)(w[e >> 1] >> (16 * (e & 1))));
        }
    };
    // Outputs are not read again here, nor are the epilogue's inputs: where
    // rows start on 128-byte lines (a.stream) they pass the L2 by (2 to 5%
    // faster; other rows would be written in partial lines, 10% slower).
    static constexpr int kStream = 2;  // cache policy operand: nt
    __device__ __forceinline__ static void store16(u32x4_t v, __amdgpu_buffer_rsrc_t r, uint32_t off, bool stream) {
        if (stream)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32_t, v), r, off, 0, kStream);
        else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32_t, v), r, off, 0, 0);
    }
    __device__ __forceinline__ static uint32_t at(uint32_t off, int bytes, bool ok) {
        return ok && off != kOob ? off + bytes : kOob;
    }
    __device__ __forceinline__ static Piece16 load(__amdgpu_buffer_rsrc_t r, uint32_t off, int valid, bool stream) {
        Piece16 v{};
        if (valid >= VEC) {
            if (stream)
                v.w = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kStream));
            else
                v.w = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
        } else {
#pragma unroll
            for (int e = 0; e < VEC - 1; ++e) {
                const uint32_t x = load_elem<ES>(r, at(off, e * ES, e < valid));
                v.w[e * ES / 4] |= x << (8 * (e * ES & 3));
            }
        }
        return v;
    }
    __device__ __forceinline__ static void store(const float (&v)[VEC], __amdgpu_buffer_rsrc_t r, uint32_t off, int valid,
                                                 bool stream) {
        u32x4_t w;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if constexpr (ES == 4)
                w[d] = __builtin_bit_cast(uint32_t, v[d]);
            else
                w[d] = io::pack2(v[2 * d], v[2 * d + 1]);
        }
        if (valid >= VEC) {
            store16(w, r, off, stream);
        } else {
#pragma unroll
            for (int e = 0; e < VEC - 1; ++e)
                store_elem<ES>((typename RawBits<ES>::T)(w[e * ES / 4] >> (8 * (e * ES & 3))), r, at(off, e * ES, e < valid));
        }
    }
    // the fp32 values themselves (16-bit types: two stores, halves of a line), which
    // keep to the L2 (fp32 gradients past it: 1135 and 1138 us, 37.1 and 37.6, 43.1 both)
    __device__ __forceinline__ static void store_f32(const float (&v)[VEC], __amdgpu_buffer_rsrc_t r, uint32_t off,
                                                     int valid) {
#pragma unroll
        for (int h = 0; h < VEC / 4; ++h) {
            const f32x4_t w = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            if (valid >= 4 * h + 4) {
                store16(__builtin_bit_cast(u32x4_t, w), r, at(off, h * 16, true), false);
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    store_elem<4>(__builtin_bit_cast(uint32_t, v[4 * h + e]), r,
                                  at(off, h * 16 + e * 4, 4 * h + e < valid));
            }
        }
    }

    struct Tile {
        int e, tn;     // expert, column tile
        int part;      // part of the sum
        int depth;     // summed elements
        int lo;        // first row of the run
        int m0, rows;  // first output row (within the operands: of all rows, or of the expert's dW), rows that exist
    };

    // PART: the fp32 sums go to the tile's part of a.part, and no further.
    template <int ACT, bool PART = false>
    __device__ __forceinline__ static void epilogue(const GroupedArgs &a, const Tile &t, int wave, int lane,
                                                    const f32x4_t (&acc)[NRB][NI], FL_LDS char *lds) {
        const int rows = t.rows, n0 = t.tn * BN;
        const bool stream = !PART && a.stream;
        const int64_t row0 = FORM == kFormGrad ? (int64_t)t.e * a.K + t.m0 : t.m0;
        const int wm = row_of(wave), wn = col_of(wave);
        constexpr int CPR = TN / VEC, RPP = 64 / CPR, PASSES = 16 / RPP;  // lanes per row, rows and passes per row block
        const int es = PART || (FORM == kFormGrad && a.dw_f32) ? 4 : ES;
        const int64_t org = row0 * a.N + n0;
        const size_t bytes = ((size_t)rows * a.N - n0) * es;
        const int64_t all_rows = FORM == kFormGrad ? (int64_t)a.E * a.K : a.S;
        void *to = PART ? static_cast<void *>(a.part + t.part * all_rows * a.N) : a.out;
        const __amdgpu_buffer_rsrc_t rO = make_rsrc(static_cast<char *>(to) + org * es, bytes);
        const __amdgpu_buffer_rsrc_t rO2 =
            make_rsrc(a.out2 ? static_cast<char *>(a.out2) + org * ES : nullptr, a.out2 ? bytes : 0);
        const __amdgpu_buffer_rsrc_t rY =
            make_rsrc(a.Y ? static_cast<const char *>(a.Y) + org * ES : nullptr, a.Y ? bytes : 0);
        const __amdgpu_buffer_rsrc_t rX =
            make_rsrc(a.X ? static_cast<const char *>(a.X) + org * ES : nullptr, a.X ? bytes : 0);
        const int col = wn * TN + (lane % CPR) * VEC, valid = a.N - n0 - col;
        FL_LDS char *w = lds + wave * 16 * EPI_ROW;
        auto offset = [&](int mi, int p) -> uint32_t {
            const int row = wm * TM + mi * 16 + p * RPP + lane / CPR;
            return row < rows && valid > 0 ? (uint32_t)(row * a.N + col) * es : kOob;
        };
        Piece16 bias{};
        if constexpr (FORM == kFormFwd && !PART) {
            if (a.bias) {
                const __amdgpu_buffer_rsrc_t rB = make_rsrc(
                    static_cast<const char *>(a.bias) + ((int64_t)t.e * a.N + n0) * ES, (size_t)(a.N - n0) * ES);
                bias = load(rB, valid > 0 ? (uint32_t)col * ES : kOob, valid, false);
            }
        }
        constexpr bool NEED_Y = ACT == FL_ACT_GLU, NEED_X = FORM == kFormBwd && ACT != FL_ACT_NONE;
        Piece16 yv[2][PASSES], xv[2][PASSES];  // of this row block and the next
        auto sides = [&](int mi) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                if constexpr (NEED_Y) yv[mi & 1][p] = load(rY, offset(mi, p), valid, stream);
                if constexpr (NEED_X) xv[mi & 1][p] = load(rX, offset(mi, p), valid, stream);
            }
        };
        sides(0);
#pragma unroll
        for (int mi = 0; mi < NRB; ++mi) {
            if (mi + 1 < NRB) sides(mi + 1);
            // lane: row lane % 16 of the block, columns ni*16 + (lane/16)*4 + 0..3
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
                *(FL_LDS f32x4_t *)(w + (lane & 15) * EPI_ROW + (ni * 16 + (lane >> 4) * 4) * 4) = acc[mi][ni];
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
            asm volatile("" ::: "memory");
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const FL_LDS char *s = w + (p * RPP + lane / CPR) * EPI_ROW + (lane % CPR) * (VEC * 4);
                f32x4_t q[VEC / 4];
#pragma unroll
                for (int h = 0; h < VEC / 4; ++h) q[h] = *(const FL_LDS f32x4_t *)(s + h * 16);
                const uint32_t off = offset(mi, p);
                float v[VEC], v2[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = q[i >> 2][i & 3];
                    const float y = NEED_Y ? yv[mi & 1][p].get(i) : 0.0f;
                    if constexpr (PART) {
                        v[i] = d;
                    } else if constexpr (FORM == kFormFwd) {
                        const float x = d + bias.get(i);
                        v2[i] = x;
                        v[i] = activate<ACT>(x, y);
                    } else if constexpr (FORM == kFormBwd) {
                        const float xs = NEED_X ? xv[mi & 1][p].get(i) : 0.0f;
                        v[i] = d * activate_grad<ACT>(xs, y);
                        v2[i] = d * xs;
                        asm("" : "+v"(v[i]), "+v"(v2[i]));  // fp32 before the cast, in every kernel alike
                    } else {
                        v[i] = d;
                    }
                }
                if (PART || (FORM == kFormGrad && a.dw_f32))
                    store_f32(v, rO, off, valid);
                else
                    store(v, rO, off, valid, stream);
                if (!PART && (FORM == kFormFwd ? a.out2 != nullptr : FORM == kFormBwd && ACT == FL_ACT_GLU))
                    store(v2, rO2, off, valid, stream);
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Tile number b of n.  Workgroups of one XCD (b modulo 8) take consecutive
    // tiles, so that its L2 serves their shared operands: of the list of all
    // experts' tiles or, with a.spread, of every expert's by itself.  An
    // expert's tiles are ordered in bands of a.group row tiles swept column by
    // column.
    __device__ __forceinline__ static bool find(const GroupedArgs &a, int b, int n, Tile &t) {
        t.part = 0;
        if (n <= 0) return false;  // (no expert has a row)
        if (a.parts > 1) {
            t.part = b / n;
            if (t.part >= a.parts) return false;
            b -= t.part * n;
        } else if (b >= n) {
            return false;
        }
        int m;
        if constexpr (FORM == kFormGrad) {
            // (an expert's tiles cost as much as it has rows, so always spread)
            const int tiles_m = (a.K + BM - 1) / BM, per = tiles_m * a.tiles_n;
            t.e = b / per;
            t.lo = run_bound(a, t.e);
            const int hi = run_bound(a, t.e + 1);
            t.depth = hi > t.lo ? hi - t.lo : 0;
            grouped_tile(xcd_logical(b - t.e * per, per), tiles_m, a.tiles_n, a.group, m, t.tn);
            t.m0 = m * BM;
            t.rows = a.K - t.m0 < BM ? a.K - t.m0 : BM;
        } else {
            const int pid = a.spread ? b : xcd_logical(b, n);
            const int q = pid / a.tiles_n;
            const RunTile r = find_run_tile(a, BM, q);
            if (r.e < 0) return false;
            const int cnt = row_tiles(r.hi - r.lo, BM);
            const int local = pid - (q - r.m) * a.tiles_n;
            if (r.m < 0 || r.m >= cnt || local < 0) return false;  // (offsets that are no plan's)
            grouped_tile(a.spread ? xcd_logical(local, cnt * a.tiles_n) : local, cnt, a.tiles_n, a.group, m, t.tn);
            if (m < 0 || m >= cnt || t.tn < 0 || t.tn >= a.tiles_n) return false;
            t.e = r.e;
            t.lo = r.lo;
            t.depth = a.K;
            t.m0 = r.lo + m * BM;
            t.rows = r.hi - t.m0 < BM ? r.hi - t.m0 : BM;
        }
        // scalars, so that descriptors and loop bounds are
        t.e = __builtin_amdgcn_readfirstlane(t.e);
        t.tn = __builtin_amdgcn_readfirstlane(t.tn);
        t.depth = __builtin_amdgcn_readfirstlane(t.depth);
        t.lo = __builtin_amdgcn_readfirstlane(t.lo);
        t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
        t.rows = __builtin_amdgcn_readfirstlane(t.rows);
        t.part = __builtin_amdgcn_readfirstlane(t.part);
        return true;
    }

    __device__ __forceinline__ static void setup(const GroupedArgs &a, const Tile &t, int wave, int lane, Ops &o) {
        const int n0 = t.tn * BN;
        int k0 = 0;  // the part's first k
        o.depth = t.depth;
        if (FORM != kFormBwd && a.parts > 1) {
            const int stages = (int)(((int64_t)t.depth + KS - 1) / KS);
            const int64_t len = (int64_t)((stages + a.parts - 1) / a.parts) * KS, k = t.part * len;
            k0 = k < t.depth ? (int)k : t.depth;
            o.depth = t.depth - k0 < len ? t.depth - k0 : (int)len;
        }
        o.lda = a.K;
        o.ldb = FORM == kFormBwd ? a.K : a.N;
        if constexpr (FORM == kFormGrad) {
            const int64_t r0 = (int64_t)t.lo + k0;
            o.pa = static_cast<const char *>(a.A) + (r0 * a.K + t.m0) * ES;
            o.pb = static_cast<const char *>(a.B) + (r0 * a.N + n0) * ES;
            o.ra = (a.S - r0) * a.K - t.m0;
            o.rb = (a.S - r0) * a.N - n0;
            set_descriptors(o);
        } else {
            const int64_t a0 = (FORM == kFormFwd && a.index ? 0 : (int64_t)t.m0 * a.K) + k0;
            o.ra = a.A_rows * a.K - a0;
            o.A.rsrc = sgpr_rsrc(static_cast<const char *>(a.A) + a0 * ES, o.ra > 0 ? (size_t)o.ra * ES : 0);
            const int64_t b0 = (int64_t)t.e * a.K * a.N + (FORM == kFormBwd ? (int64_t)n0 * a.K : (int64_t)k0 * a.N + n0);
            o.rb = (int64_t)a.E * a.K * a.N - b0;
            o.B.rsrc = sgpr_rsrc(static_cast<const char *>(a.B) + b0 * ES, (size_t)o.rb * ES);
        }
#pragma unroll
        for (int i = 0; i < SideA::COPIES; ++i) {
            int r, c;
            SideA::place(wave, lane, i, r, c);
            if constexpr (FORM == kFormGrad) {
                o.A.off[i] = c * EPC < t.rows ? (uint32_t)(r * o.lda + c * EPC) * ES : kOob;
            } else {
                int64_t row = r;
                bool ok = r < t.rows;
                if (FORM == kFormFwd && a.index) {
                    row = ok ? a.index[t.m0 + r] : 0;
                    ok = ok && row >= 0 && row < a.A_rows;
                }
                o.A.off[i] = ok ? ((uint32_t)row * (uint32_t)o.lda + c * EPC) * ES : kOob;
            }
        }
#pragma unroll
        for (int i = 0; i < SideB::COPIES; ++i) {
            int r, c;
            SideB::place(wave, lane, i, r, c);
            if constexpr (FORM == kFormBwd) {
                o.B.off[i] = n0 + r < a.N ? (uint32_t)(r * o.ldb + c * EPC) * ES : kOob;
            } else {
                o.B.off[i] = n0 + c * EPC < a.N ? (uint32_t)(r * o.ldb + c * EPC) * ES : kOob;
            }
        }
    }

    // Tiles blockIdx.x, + gridDim.x, ..  While a tile's epilogue runs in the
    // last LDS buffer, the first NBUF-1 stages of the next one are on their
    // way into the others.
    __device__ __forceinline__ static void run(const GroupedArgs &a, int act, char *smem) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        FL_LDS char *lds = (FL_LDS char *)smem;
        const uint32_t addr = (uint32_t)(uintptr_t)(FL_LDS void *)smem;
        const int64_t all = FORM == kFormGrad ? (int64_t)a.E * ((a.K + BM - 1) / BM) * a.tiles_n
                                              : (int64_t)count_run_tiles(a, BM) * a.tiles_n;
        const int n = __builtin_amdgcn_readfirstlane((int)(all < a.max_tiles ? all : a.max_tiles));
        int b = blockIdx.x;
        Tile t;
        if (!find(a, b, n, t)) return;
        Ops o;
        o.A.set_frag(row_of(wave) * TM, lane);
        o.B.set_frag(col_of(wave) * TN, lane);
        setup(a, t, wave, lane, o);
        prefetch<0, NBUF - 1>(o, wave, lane, addr);
        for (;;) {
            // addresses of a tile come from a copy of the lane made for it, so
            // that none is kept across its K loop
            int lo = lane;
            asm volatile("" : "+v"(lo));
            prefetch<NBUF - 1, NBUF>(o, wave, lo, addr);
            b += gridDim.x;
            Tile next;
            const bool more = find(a, b, n, next);
            f32x4_t acc[NRB][NI];
            const bool idle = row_of(wave) * TM >= t.rows || t.tn * BN + col_of(wave) * TN >= a.N;
            product(a, o, idle, wave, lo, lds, addr, acc);
            int le = lane;  // (and so for the next tile's and the epilogue's)
            asm volatile("" : "+v"(le));
            if (more) {
                setup(a, next, wave, le, o);
                prefetch<0, NBUF - 1>(o, wave, le, addr);
            }
            FL_LDS char *epi = lds + (NBUF - 1) * BUF_BYTES;
            if (idle)
                ;
            else if (FORM != kFormBwd && a.parts > 1)
                epilogue<FL_ACT_NONE, true>(a, t, wave, le, acc, epi);
            else if (FORM == kFormGrad || act == FL_ACT_NONE)
                epilogue<FL_ACT_NONE>(a, t, wave, le, acc, epi);
            else if (act == FL_ACT_RELU)
                epilogue<FL_ACT_RELU>(a, t, wave, le, acc, epi);
            else if (act == FL_ACT_GELU_TANH)
                epilogue<FL_ACT_GELU_TANH>(a, t, wave, le, acc, epi);
            else
                epilogue<FL_ACT_GLU>(a, t, wave, le, acc, epi);
            if (!more) break;
            t = next;
            __syncthreads();  // the last buffer is free for copies again
        }
    }
};

template <int DT, int FORM, int BM, int BN, int WM, int WN, int NBUF, int OCC, bool NT>
__global__ void __launch_bounds__(64 * WM * WN, OCC) grouped_dma_kernel(GroupedArgs a, int act) {
    using T = GroupedTile<DT, FORM, BM, BN, WM, WN, NBUF, NT>;
    __shared__ __attribute__((aligned(1024))) char smem[T::SMEM];
    T::run(a, act, smem);
}

}  // namespace fl
