// fl_mx4_linear.hpp -- gfx950 device code of the fused linear layer over
// microscaled 4-bit operands: out = act(A @ B + bias [+ R]).
//
// A has M rows and B N rows of K-contiguous codes, 16 bytes to a block of 32
// values, so a row is whole 16-byte chunks and both operands are read alike.
// v_mfma_scale_f32_16x16x128_f8f6f4 takes from lane l the 32 codes of row l % 16
// and block l / 16 of a depth of four blocks, and the block's scale as a byte of a
// register: a chunk as it lies in memory is an operand.  Which four blocks meet
// in an instruction does not matter as long as A and B agree: over 256 values
// lane l takes blocks 2 (l / 16) and 2 (l / 16) + 1, 32 neighbouring bytes, in two
// instructions, so that the lanes of a row read a whole line.  B goes in first:
// the result then has four neighbouring columns of one row in a lane.
// Products of codes are exact, they are summed in fp32 with the scales applied.
#pragma once

#include "fl_mx4.hpp"

namespace fl {

typedef int i32x8_mx_t __attribute__((ext_vector_type(8)));

struct Mx4LinearArgs {
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    const void *a_raw;           // A in the output's type instead of codes, quantised on its way in
    const void *bias, *Y, *R;    // each or null
    void *out;
    int64_t M, N;
    int K, blocks, act;
};

// n, m: operands of B and of A; the scales' byte `half`, 0 or 1, which has to be a constant.
__device__ __forceinline__ f32x4_t mfma_mx4(u32x4_t n, u32x4_t m, f32x4_t c, uint32_t n_scales, uint32_t m_scales,
                                            int half) {
    const i32x8_mx_t x{(int)n[0], (int)n[1], (int)n[2], (int)n[3], 0, 0, 0, 0};
    const i32x8_mx_t y{(int)m[0], (int)m[1], (int)m[2], (int)m[3], 0, 0, 0, 0};
    return half ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 1, (int)n_scales, 1, (int)m_scales)
                : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)n_scales, 0, (int)m_scales);
}

typedef uint32_t any2_u32_t __attribute__((aligned(2)));

// N neighbouring elements of an epilogue operand as floats, of which `left` exist.
template <int DT, int N>
__device__ __forceinline__ void load_floats(const void *p, int64_t at, int64_t left, float (&f)[N]) {
    using io = Io<DT>;
    using raw = typename io::raw;
    raw v[N];
    const raw *q = static_cast<const raw *>(p) + at;
    if (left >= N) {
#pragma unroll
        for (int i = 0; i < N * io::size / 4; ++i) {
            const uint32_t w = reinterpret_cast<const any2_u32_t *>(q)[i];
            __builtin_memcpy(reinterpret_cast<char *>(v) + 4 * i, &w, 4);
        }
    } else {
#pragma unroll
        for (int t = 0; t < N; ++t) v[t] = t < left ? q[t] : raw(0);
    }
#pragma unroll
    for (int t = 0; t < N; ++t) f[t] = io::to_f32(v[t]);
}

template <int ACT, int N>
__device__ __forceinline__ void activate_all(float (&x)[N], const float (&y)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) x[t] = activate<ACT>(x[t], y[t]);
}

// act(x + bias + R) of N neighbouring columns of a row, and the one store.
template <int DT, int N>
__device__ __forceinline__ void finish_columns(const Mx4LinearArgs &a, int64_t m, int64_t n, float (&x)[N]) {
    using io = Io<DT>;
    using raw = typename io::raw;
    const int64_t left = a.N - n, at = m * a.N + n;
    float f[N];
    if (a.bias) {
        load_floats<DT>(a.bias, n, left, f);
#pragma unroll
        for (int t = 0; t < N; ++t) x[t] += f[t];
    }
    if (a.R) {
        load_floats<DT>(a.R, at, left, f);
#pragma unroll
        for (int t = 0; t < N; ++t) x[t] += f[t];
    }
    if (a.act == FL_ACT_RELU) {
        activate_all<FL_ACT_RELU>(x, f);
    } else if (a.act == FL_ACT_GELU_TANH) {
        activate_all<FL_ACT_GELU_TANH>(x, f);
    } else if (a.act == FL_ACT_GLU) {
        load_floats<DT>(a.Y, at, left, f);
        activate_all<FL_ACT_GLU>(x, f);
    }
    raw v[N];
#pragma unroll
    for (int t = 0; t < N; ++t) v[t] = io::from_f32(x[t]);
    raw *q = static_cast<raw *>(a.out) + at;
    if (left >= N) {
#pragma unroll
        for (int i = 0; i < N * io::size / 4; ++i) {
            uint32_t w;
            __builtin_memcpy(&w, reinterpret_cast<char *>(v) + 4 * i, 4);
            reinterpret_cast<any2_u32_t *>(q)[i] = w;
        }
    } else {
#pragma unroll
        for (int t = 0; t < N; ++t)
            if (t < left) q[t] = v[t];
    }
}

// ------------------------------------------------------------------ few rows

// 16 MT rows by 16 NT columns to a block, whose WAVES waves share out K 256 values
// at a time: each streams its part of B's rows straight into registers, as they
// are operands; the waves' sums meet in the LDS in a fixed
// order.  No row of B is read twice as long as M <= 16 MT; A comes from the caches.
//
// A load costs by the lines it touches, so the scales, of which a step needs 8
// bytes of each row, are brought into the LDS in whole rows first, `panel` blocks of K
// at a time.  VALUES: A (MT = 1) is given as values; every block quantises them into
// the LDS, which takes less than another launch while they are few.
//
// Measured: one token by 14336x4096 fp16 with GELU 7.7 us, of which the launch takes 3
// (31.3 MB, 6.7 TB/s of the rest: L2s and matrix cores wait for memory).  More rows are
// bound by A, which every block reads again from the L2: 64 by 4096x14336 17 us.  Loads
// of the next step before this one's products: no gain (8.1 against 7.8 us; 64 rows from
// values 20.4 both), as the other waves' loads are under way already.
constexpr int kMx4ScalePad = 16;  // rows of scales 16 bytes past a multiple of 256: 16 rows in different banks

struct Mx4StreamArgs {
    Mx4LinearArgs l;
    int panel;       // blocks, a multiple of 256 (scales of 256 blocks: 256 bytes)
    int code_pitch;  // VALUES: bytes of a row of codes, 16 past whole pieces of 16 blocks: rows in different banks
};

template <int DT, int MT, int NT, int WAVES, bool VALUES>
__global__ void __launch_bounds__(64 * WAVES) mx4_stream_kernel(Mx4StreamArgs s) {
    static_assert(!VALUES || MT == 1, "few rows");
    extern __shared__ __align__(16) char lds[];
    const Mx4LinearArgs &a = s.l;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), d = lane & 15, q = lane >> 4;
    const uint32_t across = (uint32_t)((a.N + 16 * NT - 1) / (16 * NT));
    const int64_t n0 = (int64_t)(blockIdx.x % across) * (16 * NT), m0 = (int64_t)(blockIdx.x / across) * (16 * MT);
    const uint32_t pitch = (uint32_t)a.blocks * 16;
    const int n_left = (int)(a.N - n0 < 16 * NT ? a.N - n0 : 16 * NT), m_left = (int)(a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.b_codes + n0 * pitch, (size_t)n_left * pitch);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(VALUES ? nullptr : a.a_codes + m0 * pitch, VALUES ? 0 : (size_t)m_left * pitch);
    // in the LDS: rows of scales, B's then A's; the codes of A's values
    const int row_bytes = s.panel + kMx4ScalePad;
    char *b_scales = lds, *a_scales = lds + 16 * NT * row_bytes, *a_codes = a_scales + (VALUES ? m_left : 16 * MT) * row_bytes;
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    for (int p0 = 0; p0 < a.blocks; p0 += s.panel) {
        const int blocks = a.blocks - p0 < s.panel ? a.blocks - p0 : s.panel;  // of this panel
        u32x4_t b[NT][2], m[MT][2];
        const auto load = [&](int c0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int block = c0 + 2 * q + h;  // in the panel
                const bool on = block < blocks;
                const uint32_t at = (uint32_t)(p0 + block) * 16;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    b[j][h] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                              rb, on ? (uint32_t)(j * 16 + d) * pitch + at : kOob, 0, 0));
                if constexpr (!VALUES) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        m[i][h] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                                  ra, on ? (uint32_t)(i * 16 + d) * pitch + at : kOob, 0, 0));
                }
            }
        };
        load(wave * 8);
        // scales, 16 blocks to a thread; zeros behind a row's last and in rows that are none
        const int pieces = (blocks + 15) / 16, rows = VALUES ? 16 * NT : 16 * (NT + MT);
        for (int i = threadIdx.x; i < pieces * rows; i += 64 * WAVES) {
            const int row = i / pieces, k = (i - row * pieces) * 16;
            const bool of_b = row < 16 * NT;
            const int r = of_b ? row : row - 16 * NT;
            const uint8_t *src = (of_b ? a.b_scales + (n0 + r) * a.blocks : a.a_scales + (m0 + r) * a.blocks) + p0 + k;
            u32x4_t w{0, 0, 0, 0};
            if (r < (of_b ? n_left : m_left)) {
                if (k + 16 <= blocks) {
                    typedef uint32_t any1_u32x4_t __attribute__((ext_vector_type(4), aligned(1)));
                    w = *reinterpret_cast<const any1_u32x4_t *>(src);
                } else {
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (k + t < blocks) w[t / 4] |= (uint32_t)src[t] << (8 * (t % 4));
                }
            }
            *reinterpret_cast<u32x4_t *>(b_scales + row * row_bytes + k) = w;
        }
        if constexpr (VALUES) {
            // eight values to a thread, a block of 32 to four neighbours, up to whole pieces of 16 blocks
            // (the loads of four at once)
            constexpr int AHEAD = 4;
            const int per_row = pieces * 64, all = per_row * m_left;
            for (int i0 = 0; i0 < all; i0 += AHEAD * 64 * WAVES) {
                RowValues<DT, 8> v[AHEAD];
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    if (i0 + u * 64 * WAVES >= all) break;
                    const int i = i0 + u * 64 * WAVES + threadIdx.x, row = i / per_row, unit = i - row * per_row;
                    const int64_t k = (int64_t)p0 * 32 + unit * 8;
                    v[u].load(a.a_raw, (m0 + row) * a.K + k, row < m_left ? a.K - k : 0);
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    if (i0 + u * 64 * WAVES >= all) break;
                    const int i = i0 + u * 64 * WAVES + threadIdx.x, row = i / per_row, unit = i - row * per_row;
                    uint32_t top = magnitude_bits<DT>(v[u].w[0]);
#pragma unroll
                    for (int e = 1; e < RowValues<DT, 8>::WORDS; ++e)
                        top = larger_bits<DT>(top, magnitude_bits<DT>(v[u].w[e]));
                    top = larger_bits<DT>(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, true));
                    top = larger_bits<DT>(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, true));
                    const uint32_t sc = scale_byte<DT>(top);
                    if (row >= m_left) continue;
                    *reinterpret_cast<uint32_t *>(a_codes + row * s.code_pitch + unit * 4) =
                        sc == 255 ? 0 : codes8<DT>(v[u].w, scale_value(sc));
                    if ((unit & 3) == 0) a_scales[row * row_bytes + unit / 4] = (char)sc;
                }
            }
        }
        __syncthreads();
        for (int c0 = wave * 8; c0 < blocks;) {
            const int at = c0 + 2 * q;
            uint32_t sb[NT], sa[MT];
#pragma unroll
            for (int j = 0; j < NT; ++j) sb[j] = *reinterpret_cast<const uint16_t *>(b_scales + (j * 16 + d) * row_bytes + at);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                // a lane of no row takes the first's: its column of the results goes nowhere
                const int row = VALUES ? (d < m_left ? d : 0) : i * 16 + d;
                sa[i] = *reinterpret_cast<const uint16_t *>(a_scales + row * row_bytes + at);
                if constexpr (VALUES) {
                    m[i][0] = *reinterpret_cast<const u32x4_t *>(a_codes + row * s.code_pitch + at * 16);
                    m[i][1] = *reinterpret_cast<const u32x4_t *>(a_codes + row * s.code_pitch + at * 16 + 16);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = mfma_mx4(b[j][h], m[i][h], acc[i][j], sb[j], sa[i], h);
            c0 += WAVES * 8;
            if (c0 < blocks) load(c0);
        }
        __syncthreads();  // the scales are read; the next panel's, or the sums, take their place
    }
    // the sums of the waves, whose place the scales had
    f32x4_t *sums = reinterpret_cast<f32x4_t *>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[(wave * (MT * NT) + i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * NT * 64; t += 64 * WAVES) {
        const int l = t & 63, i = (t >> 6) / NT, j = (t >> 6) % NT;
        f32x4_t v = sums[t];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += sums[w * (MT * NT * 64) + t];
        const int64_t mm = m0 + i * 16 + (l & 15), n = n0 + j * 16 + (l >> 4) * 4;
        if (mm >= a.M || n >= a.N) continue;
        float x[4] = {v[0], v[1], v[2], v[3]};
        finish_columns<DT>(a, mm, n, x);
    }
}

}  // namespace fl
