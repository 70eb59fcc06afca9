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

__device__ __forceinline__ f32x4_t mfma_mx4(u32x4_t n, u32x4_t m, f32x4_t c, uint32_t n_scales, uint32_t m_scales,
                                            int step) {
    const i32x8_mx_t x{(int)n[0], (int)n[1], (int)n[2], (int)n[3], 0, 0, 0, 0};
    const i32x8_mx_t y{(int)m[0], (int)m[1], (int)m[2], (int)m[3], 0, 0, 0, 0};
    // 4: E2M1 operands; the selected byte of a scale register has to be a constant
    return step == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)n_scales, 0, (int)m_scales)
           : step == 1 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 1, (int)n_scales, 1, (int)m_scales)
           : step == 2 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 2, (int)n_scales, 2, (int)m_scales)
                       : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 3, (int)n_scales, 3, (int)m_scales);
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

// A lane's two chunks of 256 values of one row and their scales, from the rows
// that the descriptors start at; zeros where a row or a block is none.
struct Mx4Pair {
    u32x4_t c[2];
    uint32_t s;

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales, int row, int block,
                                         int blocks) {
        const bool two = block + 1 < blocks, one = block < blocks;
        const uint32_t at = (uint32_t)row * (uint32_t)blocks + (uint32_t)block;
        c[0] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(codes, one ? at * 16 : kOob, 0, 0));
        c[1] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(codes, two ? at * 16 + 16 : kOob, 0, 0));
        if (blocks & 1) {  // the last block of a row may be the first of a pair
            s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(scales, one ? at : kOob, 0, 0) & 0xffu;
            s |= ((uint32_t)__builtin_amdgcn_raw_buffer_load_b8(scales, two ? at + 1 : kOob, 0, 0) & 0xffu) << 8;
        } else {
            s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(scales, one ? at : kOob, 0, 0) & 0xffffu;
        }
    }
};

// The same from a row of values, quantised: a block of 32 is one lane's, so its
// largest magnitude takes no exchange.
template <int DT>
__device__ __forceinline__ void quantize_pair(Mx4Pair &p, const void *x, int64_t row, bool on, int block, int K) {
    using V = RowValues<DT, 32>;
    V v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t k = (int64_t)(block + h) * 32;
        v[h].load(x, row * K + k, on ? K - k : 0);
    }
    p.s = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t m = magnitude_bits<DT>(v[h].w[0]);
#pragma unroll
        for (int e = 1; e < V::WORDS; ++e) m = larger_bits<DT>(m, magnitude_bits<DT>(v[h].w[e]));
        const uint32_t s = scale_byte<DT>(m);
        p.s |= s << (8 * h);
#pragma unroll
        for (int g = 0; g < 4; ++g) p.c[h][g] = s == 255 ? 0 : codes8<DT>(v[h].w + g * (V::WORDS / 4), scale_value(s));
    }
}

// 16 MT rows by 16 NT columns to a block, whose WAVES waves share out K 256 values
// at a time: each streams its part of B's rows straight into registers, as they
// are operands, U steps in flight; the waves' sums meet in the LDS in a fixed
// order.  No row of B is read twice as long as M <= 16 MT; A comes from the caches.
template <int DT, int MT, int NT, int WAVES, int U, bool RAW>
__global__ void __launch_bounds__(64 * WAVES) mx4_stream_kernel(Mx4LinearArgs a) {
    __shared__ f32x4_t sums[WAVES][MT * NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = lane & 15, q = lane >> 4;
    const uint32_t across = (uint32_t)((a.N + 16 * NT - 1) / (16 * NT));
    const int64_t n0 = (int64_t)(blockIdx.x % across) * (16 * NT), m0 = (int64_t)(blockIdx.x / across) * (16 * MT);
    const size_t pitch = (size_t)a.blocks * 16;
    const int64_t n_left = a.N - n0 < 16 * NT ? a.N - n0 : 16 * NT, m_left = a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.b_codes + n0 * pitch, n_left * pitch);
    const __amdgpu_buffer_rsrc_t rbs = make_rsrc(a.b_scales + n0 * a.blocks, n_left * a.blocks);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(RAW ? nullptr : a.a_codes + m0 * pitch, RAW ? 0 : m_left * pitch);
    const __amdgpu_buffer_rsrc_t ras = make_rsrc(RAW ? nullptr : a.a_scales + m0 * a.blocks, RAW ? 0 : m_left * a.blocks);
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = wave * 8; b0 < a.blocks; b0 += WAVES * U * 8) {
        Mx4Pair b[U][NT], p[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) b[u][j].load(rb, rbs, j * 16 + d, b0 + u * WAVES * 8 + 2 * q, a.blocks);
        if constexpr (!RAW) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MT; ++i) p[u][i].load(ra, ras, i * 16 + d, b0 + u * WAVES * 8 + 2 * q, a.blocks);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (RAW) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    quantize_pair<DT>(p[u][i], a.a_raw, m0 + i * 16 + d, i * 16 + d < m_left,
                                      b0 + u * WAVES * 8 + 2 * q, a.K);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = mfma_mx4(b[u][j].c[h], p[u][i].c[h], acc[i][j], b[u][j].s, p[u][i].s, h);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * NT * 64; t += 64 * WAVES) {
        const int l = t & 63, i = (t >> 6) / NT, j = (t >> 6) % NT;
        f32x4_t s = sums[0][t >> 6][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += sums[w][t >> 6][l];
        const int64_t m = m0 + i * 16 + (l & 15), n = n0 + j * 16 + (l >> 4) * 4;
        if (m >= a.M || n >= a.N) continue;
        float x[4] = {s[0], s[1], s[2], s[3]};
        finish_columns<DT>(a, m, n, x);
    }
}

}  // namespace fl
