// fl_mx4_tile.hpp -- gfx950 device code of the 4-bit linear layer for many rows:
// output tiles whose operands are staged through the LDS.
//
//   * A stage is 256 values of K: 128 bytes of codes of each of the tile's rows of
//     A and of B, copied straight into the LDS (16 bytes a lane), 8 chunks to a row
//     with chunk c of row r at c ^ fa(r), so that an operand read asks no bank
//     twice.  Two stages are held, or four (RING): while one is computed the copies of
//     the others land.
//     A copy costs by the lines it touches, 2 clocks each (a wave's copy of 64-byte
//     pieces takes twice the time of 128-byte ones).
//   * Scales are copied for four stages at a time, 32 bytes of each row (8 bytes of a
//     row for every stage would touch as many lines as the codes do).  What follows
//     a row's scales in memory is the next row's and may stand for NaN.  The last one to
//     four stages come first, so that the bytes behind the last block are cleared
//     before the loop (where a stage's scales are read, the wait for them to be cleared
//     takes 8% of the time; an outer loop around it as much).
//   * A wave owns 16 MI x 16 NI outputs.  Operands of the next half stage are read
//     while the matrix instructions of this one run, those of A into the registers
//     whose row of products is done; the one barrier of a stage comes when its second
//     half is in registers: behind it the stage's place is free for the copies of a
//     later one.
//   * The rows of B are placed so that the eight results that a lane has of an output
//     row in NI accumulators (two elements of four, one of eight) are neighbours,
//     and with them the four lanes of a row: 16-byte stores of 64 bytes in a row,
//     straight from the accumulators.
//
// Measured, bf16 from codes: 8192x8192x8192 246 us, 4.5 PFLOP/s; 8192x14336x4096 256
// us, with GELU 262.  The matrix cores alone, products of random codes out of registers,
// reach 6.4 at the 1.7 GHz that their power leaves.  A stage of 256x256 takes 1.7 us
// of which its 2048 clocks of products would take 1.25; its operand reads have the LDS
// busy for 1200 clocks (a sixth of them conflicts) and its copies for another 512, and a
// copy's lines take 1024 on their way.  Without the copies the first case took 209 us (of
// 255 then), without the reads as well 193.  A tile's own time, 8 us, is mostly its output, which
// all CUs write at once (33.5 MB, 6 us): workgroups that go from tile to tile and
// fetch the next one's first stages before that were slower (306 us against 287), as were
// touching lines ahead for the L2 (337 against 275), a ring of four halves of a stage,
// whose 64-byte rows are two lines' work for one (297 against 275), four waves of 128x128
// with half of the A reads (322 against 262: nothing runs while the one wave of a SIMD
// waits), and first workgroups that start staggered (no difference).
#pragma once

#include "fl_dma16.hpp"
#include "fl_mx4_linear.hpp"

namespace fl {

// lds_copy16 where `on` (uniform) is not 0, without a branch that the compiler sees: it
// would move the matrix instructions around it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16_if(uint32_t on, i32x4_t rsrc, uint32_t voffset, uint32_t lds_addr) {
    asm volatile("s_cmp_eq_u32 %3, 0\n\ts_cbranch_scc1 .Lskip%=\n\ts_mov_b32 m0, %2\n\t"
                 "buffer_load_dwordx4 %0, %1, 0 offen lds\n.Lskip%=:" ::"v"(voffset),
                 "s"(rsrc), "s"(lds_addr), "s"(__builtin_amdgcn_readfirstlane(on))
                 : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// v + step, not to be computed before a loop and kept.
__device__ __forceinline__ uint32_t add_now(uint32_t v, uint32_t step) {
    uint32_t r;
    asm volatile("v_add_u32 %0, %2, %1" : "=v"(r) : "v"(v), "s"(__builtin_amdgcn_readfirstlane(step)));
    return r;
}

// a < b ? x : y of uniform values, without a branch.
__device__ __forceinline__ int pick_less(int a, int b, int x, int y) {
    int r;
    asm("s_cmp_lt_i32 %1, %2\n\ts_cselect_b32 %0, %3, %4"
        : "=s"(r)
        : "s"(__builtin_amdgcn_readfirstlane(a)), "s"(__builtin_amdgcn_readfirstlane(b)),
          "s"(__builtin_amdgcn_readfirstlane(x)), "s"(__builtin_amdgcn_readfirstlane(y))
        : "scc");
    return r;
}

struct Mx4TileArgs {
    Mx4LinearArgs l;
    float *part;      // parts > 1: sums (parts, M, N)
    int parts;        // K is cut into this many runs of stages (K = 0: none)
    int part_stages;  // stages of a run
    int64_t n_from;   // the first tile's column, of tiles_m x tiles_n
    int tiles_m, tiles_n;
};

template <int DT, int MI, int NI, int WM, int WN, int RING>
struct Mx4Tile {
    static constexpr int WAVES = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
    static constexpr int A_BYTES = BM * 128, STAGE = (BM + BN) * 128, SCALES = (BM + BN) * 32;
    static constexpr int LDS = RING * STAGE + 2 * SCALES;           // RING stages, the scales of twice four
    static constexpr int NA = BM / 8 / WAVES, NB = BN / 8 / WAVES;  // copies of a wave and stage
    static constexpr int NS = (BM + BN) / 32 / WAVES;               // and of four stages' scales
    static constexpr int COPIES = NA + NB;
    // of a stage's copies those that go out in a second half, the rest in the half behind it
    static constexpr int FIRST = RING > 2 ? COPIES / 2 : COPIES;
    static_assert(NA * 8 * WAVES == BM && NB * 8 * WAVES == BN, "whole copies");
    static_assert((RING & (RING - 1)) == 0, "a stage's place is its number's low bits");

    // A 16-byte read is served 16 lanes at a time, lanes 0-3, 12-15 and 20-27 first
    // (measured): eight rows of a chunk c and the eight others of chunk c + 2.  Rows
    // of 128 bytes take half of the banks each; with bit 1 left alone the two sets'
    // chunks are the two halves of the row's eight, and no bank is asked twice.
    __device__ __forceinline__ static int fa(int r) { return (r >> 1 & 1) | (r & 4); }
    // Of the 32 bytes of scales of row r, the first 16 come second where this is 1: rows 8
    // apart are in the same banks.
    __device__ __forceinline__ static int fs(int r) { return r >> 3 & 1; }
    static constexpr int GROUP = 8 / NI;  // elements of an accumulator to eight columns
    static_assert(NI == 4 || NI == 8, "eight columns of a lane from whole accumulators");
    // the column of a wave's 16 NI that element r of accumulator ni has in the lanes of group q
    __device__ __forceinline__ static int wave_column(int q, int r, int ni) {
        return r / GROUP * 32 + q * 8 + r % GROUP * NI + ni;
    }
    // the tile's column at place p of its rows of B (row d of an operand becomes element d % 4 of lane group d / 4)
    __device__ __forceinline__ static int column(int p) {
        const int d = p & 15;
        return p / (16 * NI) * (16 * NI) + wave_column(d >> 2, d & 3, (p >> 4) % NI);
    }

    struct Operands {
        u32x4_t a[MI], b[2][NI];     // b: of this half and the next
        uint32_t sa[MI], sb[2][NI];  // two bytes, the halves'; sb: of this stage and the next
        int ahead;                   // the stage of K behind the ring
    };

    const Mx4LinearArgs &l;
    char *lds;
    i32x4_t ra, rb, rs;
    // Offsets of the lane's first copies of A, B and scales.  The others lie uniform steps
    // on; rows past the operand's last are past its descriptor's range.
    uint32_t va, vb, vs, step_s;
    int chunk;                             // of a row, that the lane copies
    uint32_t pitch;                        // of a row of codes
    uint32_t fa_at, fb_at, sa_at, sb_at;   // operand reads of the first half (the second's: one chunk on), scales
    int wave, lane;

    __device__ __forceinline__ Mx4Tile(const Mx4LinearArgs &args, char *mem, int64_t m0, int64_t n0) : l(args), lds(mem) {
        static_assert(NB % 2 == 0 && NB / 2 <= NI && 32 * WAVES * NS == BM + BN && NS <= 2 && BM % (32 * NS) == 0,
                      "the steps of copy and copy_scales");
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lane = threadIdx.x & 63;
        pitch = (uint32_t)l.blocks * 16;
        const int64_t m_left = l.M - m0 < BM ? l.M - m0 : BM, n_left = l.N - n0 < BN ? l.N - n0 : BN;
        ra = sgpr_rsrc(l.a_codes + m0 * pitch, (size_t)m_left * pitch);
        rb = sgpr_rsrc(l.b_codes + n0 * pitch, (size_t)n_left * pitch);
        chunk = (lane & 7) ^ fa(lane >> 3);
        va = (uint32_t)(wave * NA * 8 + (lane >> 3)) * pitch + chunk * 16;
        vb = (uint32_t)column(wave * NB * 8 + (lane >> 3)) * pitch + chunk * 16;
        const int p = wave * NS * 32 + (lane >> 1);  // A's rows, then B's places
        const bool of_a = wave * NS * 32 < BM;
        rs = of_a ? sgpr_rsrc(l.a_scales + m0 * l.blocks, (size_t)(l.M - m0) * l.blocks)
                  : sgpr_rsrc(l.b_scales + n0 * l.blocks, (size_t)(l.N - n0) * l.blocks);
        vs = (uint32_t)(of_a ? p : column(p - BM)) * (uint32_t)l.blocks + piece() * 16;
        step_s = (uint32_t)(of_a ? 32 : 2) * (uint32_t)l.blocks;
        const int d = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;
        fa_at = (wm * MI * 16 + d) * 128 + (2 * q ^ fa(d)) * 16;
        fb_at = A_BYTES + (wn * NI * 16 + d) * 128 + (2 * q ^ fa(d)) * 16;
        sa_at = RING * STAGE + (wm * MI * 16 + d) * 32 + fs(d) * 16 + 2 * q;
        sb_at = RING * STAGE + (BM + wn * NI * 16 + d) * 32 + fs(d) * 16 + 2 * q;
    }

    // Which 16 bytes of a row's scales the lane copies.
    __device__ __forceinline__ int piece() const { return (lane & 1) ^ fs(lane >> 1); }

    __device__ __forceinline__ uint32_t lds_at(uint32_t off) const {
        return (uint32_t)(uintptr_t)(FL_LDS char *)lds + off;
    }

    // Copy i of a wave of stage s of K, the j-th of its run: A's codes (8 rows on with
    // every copy), then B's (8 places on: lane group q + 2, 16 columns, or the next
    // accumulator, one column).  Past the last block zeros are copied, so no stage
    // needs a branch.
    __device__ __forceinline__ void copy(int s, int j, int i) const {
        const bool on = s * 8 + chunk < l.blocks;
        const uint32_t v = i < NA ? add_now(va, i * 8 * pitch) : add_now(vb, ((i - NA & 1) * 16 + (i - NA) / 2) * pitch);
        if (i < NA) {
            lds_copy16(ra, on ? v : kOob, (uint32_t)s * 128,
                       lds_at((j & RING - 1) * STAGE + (wave * NA + i) * 1024));
        } else {
            const int k = i - NA;
            lds_copy16(rb, on ? v : kOob, (uint32_t)s * 128,
                       lds_at((j & RING - 1) * STAGE + A_BYTES + (wave * NB + k) * 1024));
        }
    }
    // Copy i of a wave of the scales of stages s to s + 3, the t-th four of a run (32
    // rows or places, two accumulators, on).  The stage is in the lane's offset: 16 bytes
    // may pass the array's end, which only that is checked against.
    __device__ __forceinline__ void copy_scales(uint32_t on, int s, int t, int i) const {
        lds_copy16_if(on, rs, add_now(vs, i * step_s + s * 8),
                      lds_at(RING * STAGE + (t & 1) * SCALES + (wave * NS + i) * 1024));
    }
    __device__ __forceinline__ u32x4_t read16(uint32_t off) const { return *reinterpret_cast<const u32x4_t *>(lds + off); }
    __device__ __forceinline__ u32x4_t read_a(int j, int h, int mi) const {
        return read16((j & RING - 1) * STAGE + (fa_at ^ h * 16) + mi * 2048);
    }
    __device__ __forceinline__ u32x4_t read_b(int j, int h, int ni) const {
        return read16((j & RING - 1) * STAGE + (fb_at ^ h * 16) + ni * 2048);
    }
    // The scales of the last stage, of n < 8 blocks, once stages s to s + 3, the first four of
    // a run, have landed.  What follows them is the next row's and becomes zeros.  Four bytes
    // of a copy that pass the array's end did not come: a row's last one to three
    // where that is so (the last row's; one block: the last three's) are read here.
    __device__ __forceinline__ void last_scales(int s, int64_t m0, int64_t n0) const {
        const int n = l.blocks & 7, block = l.blocks - n;
        for (int p = threadIdx.x; p < BM + BN; p += 64 * WAVES) {
            const bool of_a = p < BM;
            const int64_t row = of_a ? m0 + p : n0 + column(p - BM), left = (of_a ? l.M : l.N) - row;
            const bool cut = left > 0 && left * l.blocks < (l.blocks & ~3) + 4;
            uint64_t *at = reinterpret_cast<uint64_t *>(lds + RING * STAGE + p * 32 + ((block - s * 8) ^ fs(p) * 16));
            uint64_t w = *at & ((1ull << (cut ? n & ~3 : n) * 8) - 1);
            for (int b = n & ~3; b < n && cut; ++b)
                w |= (uint64_t)(of_a ? l.a_scales : l.b_scales)[row * l.blocks + block + b] << b * 8;
            *at = w;
        }
    }
    __device__ __forceinline__ uint32_t read_scale(uint32_t at, int j, int i) const {
        return *reinterpret_cast<const uint16_t *>(lds + (j >> 2 & 1) * SCALES + (j & 1) * 8 + (at ^ (j & 2) * 8) + i * 512);
    }

    // What this wave has asked for, but for the last AHEAD copies, has landed and been read;
    // then everybody's.
    template <int AHEAD>
    __device__ __forceinline__ static void meet() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(AHEAD) : "memory");
    }

    // The stages of a run as they are computed: of more than four the last one to four as
    // begin to 3, then the others from `first` on as 4 to end; behind them none of K.
    struct Order {
        int first, last, end, none;
        __device__ __forceinline__ int stage(int j) const {
            return pick_less(j, end, j + pick_less(j, 4, last, first - 4), none);
        }
    };

    // A run of stages.
    __device__ __forceinline__ void run(f32x4_t (&acc)[MI][NI], int first, int stages, int64_t m0, int64_t n0) const {
        const int four = (stages - 1) / 4, begin = four ? 3 - (stages - 1) % 4 : 0;
        const Order r{first, first + four * 4 - begin, begin + stages, l.blocks};
#pragma unroll
        for (int i = 0; i < NS; ++i) copy_scales(1, r.last, 0, i);
#pragma unroll
        for (int i = 0; i < NS; ++i) copy_scales(1, first, 1, i);
#pragma unroll
        for (int j = 0; j < RING; ++j)
#pragma unroll
            for (int i = 0; i < (j < RING - 1 ? COPIES : FIRST); ++i) copy(r.stage(begin + j), begin + j, i);
        meet<(RING - 2) * COPIES + FIRST>();
        if ((l.blocks & 7) && (first + stages) * 8 >= l.blocks) {
            last_scales(r.last, m0, n0);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        Operands o;
        o.ahead = r.stage(begin + RING - 1);
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
            o.b[0][ni] = read_b(begin, 0, ni);
            o.sb[0][ni] = read_scale(sb_at, begin, ni);
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
            o.a[mi] = read_a(begin, 0, mi);
            o.sa[mi] = read_scale(sa_at, begin, mi);
        }
        // Words here, not 16 bits and zeros: the compiler would keep the 16 bits over the loop, and
        // put zeros to all of them, and wait for all of them, at its start.  lgkmcnt(0): what it
        // knows to be under way here it waits for in every stage.
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) asm volatile("" : "+v"(o.sa[mi]));
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) asm volatile("" : "+v"(o.sb[0][ni]));
        __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll 1
        for (int j = begin; j < r.end; ++j) {
            half<0, 0>(acc, o, j, r);
            half<1, 0>(acc, o, j, r);
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) o.sb[0][ni] = o.sb[1][ni];
        }
        meet<0>();  // the copies past the end
    }

    // The matrix instructions of half H of stage j, row by row of the wave's blocks, and
    // between them the operand reads of the half after it; in the second half also the
    // next stage's scales, the copies of stage j + RING and, in the first NS of four
    // stages, a copy of the scales of the next four.  The rows go forth and back:
    // neighbours share an operand.  Copies every second product measured the same as every
    // third, 2% faster than one after another.
    static constexpr int SLOTS = MI * NI, PACE = (SLOTS - NS) / FIRST < 3 ? (SLOTS - NS) / FIRST : 3;  // products to a copy
    template <int H, int I>
    __device__ __forceinline__ void half(f32x4_t (&acc)[MI][NI], Operands &o, int j, const Order &r) const {
        if constexpr (I < SLOTS) {
            constexpr int mi = I / NI, ni = mi & 1 ? NI - 1 - I % NI : I % NI;
            if constexpr (H == 1 && I == 0) {
                o.ahead = r.stage(j + RING);
                meet<(RING - 2) * COPIES>();
            }
            acc[mi][ni] = mfma_mx4(o.b[H][ni], o.a[mi], acc[mi][ni], o.sb[0][ni], o.sa[mi], H);
            if constexpr (H == 1 && I % PACE == 0 && I / PACE < FIRST) copy(o.ahead, j, I / PACE);
            if constexpr (H == 0 && I % PACE == 0 && FIRST + I / PACE < COPIES)
                copy(o.ahead, j + RING - 1, FIRST + I / PACE);
            if constexpr (H == 1 && I >= SLOTS - NS)
                copy_scales((j & 3) == 0 && j && j + 4 < r.end, r.first + j, (j >> 2) + 1, I - SLOTS + NS);
            // B's operands first, all of them are needed at once; A's where their row is done
            if constexpr (I < NI) {
                o.b[1 - H][I] = read_b(j + H, 1 - H, I);
                if constexpr (H == 1) o.sb[1][I] = read_scale(sb_at, j + 1, I);
            }
            if constexpr (I % NI == NI - 1) {
                o.a[mi] = read_a(j + H, 1 - H, mi);
                if constexpr (H == 1) o.sa[mi] = read_scale(sa_at, j + 1, mi);
            }
            __builtin_amdgcn_sched_barrier(0);
            half<H, I + 1>(acc, o, j, r);
        }
    }
};

// Eight neighbouring elements of an operand or output through a descriptor, 16 bytes at
// a time; kOob reads zeros and stores nothing.
template <int DT>
__device__ __forceinline__ void load_eight(__amdgpu_buffer_rsrc_t r, uint32_t off, float (&f)[8]) {
    constexpr int PIECES = Io<DT>::size / 2;
    u32x4_t w[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        w[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, i * 16, 0));
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const uint32_t u = DT == FL_F32 ? w[t / 4][t % 4] : w[0][t / 2];
        f[t] = DT == FL_F32    ? __builtin_bit_cast(float, u)
               : DT == FL_BF16 ? __builtin_bit_cast(float, t & 1 ? u & 0xffff0000u : u << 16)
                               : Io<FL_F16>::to_f32((uint16_t)(t & 1 ? u >> 16 : u));
    }
}
__device__ __forceinline__ void store_eight(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x4_t w = {f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32_t, w), r, off, i * 16, 0);
    }
}

typedef unsigned int v3u32_t __attribute__((ext_vector_type(3)));

// Rows of 16-bit outputs that start at odd multiples of 2 bytes, RUNS eights of each with
// a lane of every group: a lane stores from its second value on, with the first of the
// eight behind it, so that its 16 bytes start at a multiple of 4 (4096x3071x1536 bf16
// 27.9 -> 22.0 us; 4096x3070x1536 20.9).  What no neighbour takes goes by itself: the first
// value of a wave's row, and the last seven where the wave's row or the output's eights
// end (`after` says where another eight follows).
template <int DT, int RUNS>
__device__ __forceinline__ void store_odd(__amdgpu_buffer_rsrc_t r, const uint32_t (&off)[RUNS], const bool (&after)[RUNS],
                                          bool odd, int q, const uint32_t (&w)[RUNS][4]) {
    const int from = ((threadIdx.x & 63) + 16 & 63) * 4;
#pragma unroll
    for (int g = 0; g < RUNS; ++g) {
        const uint32_t mine = q ? w[g][0] : g + 1 < RUNS ? w[g + 1 < RUNS ? g + 1 : g][0] : 0u;
        const uint32_t next = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)mine);
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t up = e < 3 ? w[g][e < 3 ? e + 1 : e] : next;
            v[e] = odd ? w[g][e] >> 16 | up << 16 : w[g][e];
        }
        const bool whole = !odd || after[g], on = off[g] != kOob;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32_t, v), r, on && whole ? off[g] + 2 * odd : kOob, 0, 0);
        if (on && !whole) {
            __builtin_amdgcn_raw_buffer_store_b96(v3u32_t{v[0], v[1], v[2]}, r, off[g] + 2, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b16((unsigned short)v[3], r, off[g] + 14, 0, 0);
        }
        if (on && odd && g == 0 && q == 0) __builtin_amdgcn_raw_buffer_store_b16((unsigned short)w[g][0], r, off[g], 0, 0);
    }
}

// A wave's tile, straight from the accumulators, eight columns at a time: ACT, or -1
// for the sums of a part.  Rows and eights across the output's edge are left out.
// (m, n: the lane's first in the tile; m_left, n_left: of the output, from the tile's corner.)
template <class T, int DT, int ACT, int MI, int NI>
__device__ __forceinline__ void store_tile(const Mx4LinearArgs &l, float *part, const f32x4_t (&acc)[MI][NI], int64_t m0,
                                           int64_t n0, int m, int n, int64_t m_left, int64_t n_left) {
    constexpr int RUNS = 4 / T::GROUP, ES = ACT < 0 ? 4 : Io<DT>::size;
    const int q = (threadIdx.x & 63) >> 4;
    const int64_t corner = m0 * l.N + n0;
    const size_t rest = (size_t)(l.M * l.N - corner) * ES;
    const __amdgpu_buffer_rsrc_t ro =
        make_rsrc(ACT < 0 ? reinterpret_cast<char *>(part + corner) : static_cast<char *>(l.out) + corner * ES, rest);
    const __amdgpu_buffer_rsrc_t rr = make_rsrc(static_cast<const char *>(l.R) + corner * ES, l.R ? rest : 0);
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(static_cast<const char *>(l.Y) + corner * ES, l.Y ? rest : 0);
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(static_cast<const char *>(l.bias) + n0 * ES, l.bias ? (size_t)(l.N - n0) * ES : 0);
    float b[RUNS][8];
#pragma unroll
    for (int g = 0; g < RUNS; ++g)
        if constexpr (ACT >= 0) load_eight<DT>(rb, n + 32 * g + 8 <= n_left ? (uint32_t)(n + 32 * g) * ES : kOob, b[g]);
    // whether any row starts at an odd multiple of 2 bytes, and whether this lane's first does
    const bool any_odd = ES == 2 && ((uintptr_t)l.out >> 1 | l.N) & 1;
    const int odd = (int)((uintptr_t)l.out >> 1 & 1);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
        uint32_t w[RUNS][4], off[RUNS];
        bool after[RUNS];
#pragma unroll
        for (int g = 0; g < RUNS; ++g) {
            const bool on = m + mi * 16 < m_left && n + 32 * g + 8 <= n_left;
            const uint32_t at = on ? ((uint32_t)(m + mi * 16) * (uint32_t)l.N + (uint32_t)(n + 32 * g)) * ES : kOob;
            float x[8], y[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) x[t] = acc[mi][t % NI][g * T::GROUP + t / NI];
            if constexpr (ACT < 0) {
                store_eight(ro, at, x);
            } else {
#pragma unroll
                for (int t = 0; t < 8; ++t) x[t] += b[g][t];
                if (l.R) {
                    load_eight<DT>(rr, at, y);
#pragma unroll
                    for (int t = 0; t < 8; ++t) x[t] += y[t];
                }
                if constexpr (ACT == FL_ACT_GLU) load_eight<DT>(ry, at, y);
                activate_all<ACT>(x, y);
                if constexpr (ES == 2) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[g][e] = Io<DT>::pack2(x[2 * e], x[2 * e + 1]);
                    off[g] = at;
                    after[g] = (q < 3 || g + 1 < RUNS) && n + 32 * g + 16 <= n_left;
                    if (!any_odd)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(v4u32_t, u32x4_t{w[g][0], w[g][1], w[g][2], w[g][3]}), ro, at, 0, 0);
                } else {
                    store_eight(ro, at, x);
                }
            }
        }
        if constexpr (ES == 2 && ACT >= 0) {
            // (m0 + m) * N + n0 + n: n0 and n are even
            const bool o = (odd + (int)(m0 + m + mi * 16) * (int)(l.N & 1)) & 1;
            if (any_odd) store_odd<DT, RUNS>(ro, off, after, o, q, w);
        }
    }
}

// The columns behind the output's last whole eight, of which a lane of every row has
// them: through the LDS, four to a thread.
template <class T, int DT, int MI, int NI>
__device__ __forceinline__ void store_edge(const Mx4LinearArgs &l, float *part, const f32x4_t (&acc)[MI][NI], char *lds,
                                           int64_t m0, int64_t n0, int m, int n, int64_t m_left, int64_t n_left) {
    constexpr int RUNS = 4 / T::GROUP;
    f32x4_t *rows = reinterpret_cast<f32x4_t *>(lds);
#pragma unroll
    for (int g = 0; g < RUNS; ++g)
        if (n + 32 * g < n_left && n + 32 * g + 8 > n_left)
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x4_t v;
#pragma unroll
                    for (int t = 0; t < 4; ++t) v[t] = acc[mi][(4 * h + t) % NI][g * T::GROUP + (4 * h + t) / NI];
                    rows[(m + mi * 16) * 2 + h] = v;
                }
    __syncthreads();
    const int64_t n1 = n0 + n_left / 8 * 8;
    for (int i = threadIdx.x; i < T::BM * 2; i += 64 * T::WAVES) {
        const int64_t row = m0 + i / 2, col = n1 + i % 2 * 4;
        if (i / 2 >= m_left || col >= l.N) continue;
        float x[4] = {rows[i][0], rows[i][1], rows[i][2], rows[i][3]};
        if (part) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < l.N) part[row * l.N + col + e] = x[e];
        } else {
            finish_columns<DT>(l, row, col, x);
        }
    }
}

template <int DT, int MI, int NI, int WM, int WN, int PER_CU, int RING>
__global__ void __launch_bounds__(64 * WM * WN, PER_CU) mx4_tile_kernel(Mx4TileArgs a) {
    using T = Mx4Tile<DT, MI, NI, WM, WN, RING>;
    extern __shared__ __align__(1024) char lds[];  // T::LDS
    const int tiles = a.tiles_m * a.tiles_n;
    const int part = (int)(blockIdx.x / (unsigned)tiles), pid = (int)(blockIdx.x % (unsigned)tiles);
    int tm, tn;
    grouped_tile(xcd_logical(pid, tiles), a.tiles_m, a.tiles_n, 4, tm, tn);
    const int64_t m0 = (int64_t)tm * T::BM, n0 = a.n_from + (int64_t)tn * T::BN;
    const int all = (a.l.blocks + 7) / 8, first = part * a.part_stages;
    const int stages = all - first < a.part_stages ? all - first : a.part_stages;
    f32x4_t acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const T t(a.l, lds, m0, n0);
    t.run(acc, first, stages, m0, n0);
    // what follows is per lane and not to be computed before the loop and kept
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int m = t.wave / WN * (16 * MI) + (lane & 15), n = t.wave % WN * (16 * NI) + (lane >> 4) * 8;
    const int64_t m_left = a.l.M - m0, n_left = a.l.N - n0;
    float *sums = a.parts > 1 ? a.part + (int64_t)part * a.l.M * a.l.N : nullptr;
    if (sums)
        store_tile<T, DT, -1>(a.l, sums, acc, m0, n0, m, n, m_left, n_left);
    else if (a.l.act == FL_ACT_NONE)
        store_tile<T, DT, FL_ACT_NONE>(a.l, sums, acc, m0, n0, m, n, m_left, n_left);
    else if (a.l.act == FL_ACT_RELU)
        store_tile<T, DT, FL_ACT_RELU>(a.l, sums, acc, m0, n0, m, n, m_left, n_left);
    else if (a.l.act == FL_ACT_GELU_TANH)
        store_tile<T, DT, FL_ACT_GELU_TANH>(a.l, sums, acc, m0, n0, m, n, m_left, n_left);
    else
        store_tile<T, DT, FL_ACT_GLU>(a.l, sums, acc, m0, n0, m, n, m_left, n_left);
    if (n_left < T::BN && n_left % 8) store_edge<T, DT>(a.l, sums, acc, lds, m0, n0, m, n, m_left, n_left);
}

// The sums of the parts in their order, then the epilogue: four columns to a thread, the
// loads of eight parts under way at once (64 by 4096x14336 bf16 16.0 -> 15.2 us with its tiles).
// No parts: the layer of no K.  The blocks lie in two dimensions (one has less than 2^32 threads).
template <int DT>
__global__ void __launch_bounds__(256) mx4_join_kernel(Mx4TileArgs a) {
    const int64_t across = (a.l.N + 3) / 4;
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (i >= across * a.l.M) return;
    const int64_t m = i / across, n = (i - m * across) * 4;
    const int64_t left = a.l.N - n, step = a.l.M * a.l.N;
    const float *from = a.part + m * a.l.N + n;
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < a.parts; p += 8) {
        float f[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) load_floats<FL_F32>(from, (p + i) * step, p + i < a.parts ? left : 0, f[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] += f[i][t];
    }
    finish_columns<DT>(a.l, m, n, x);
}

// The kernels of one type (fl_mx4_inst.hip); Alone: on a CU each.
enum { kMx4Tile256, kMx4Tile128, kMx4Tile128Alone, kMx4Tiles };
struct Mx4TileShape {
    int bm, bn, waves;
};
constexpr Mx4TileShape kMx4TileShapes[kMx4Tiles] = {{256, 256, 8}, {128, 128, 4}, {128, 128, 8}};
struct Mx4StreamShape {
    int mt, nt, waves;  // 16 mt rows by 16 nt columns to a block of this many waves
};
template <int DT>
void launch_mx4_stream(const Mx4StreamShape &shape, const Mx4LinearArgs &a, hipStream_t st);
template <int DT>
void launch_mx4_tile(int variant, const Mx4TileArgs &a, hipStream_t st);
template <int DT>
void launch_mx4_join(const Mx4TileArgs &a, hipStream_t st);

}  // namespace fl
