// fl_mx4.hpp -- gfx950 device code of microscaled 4-bit floating point: blocks
// of 32 values along K, each value a 4-bit E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives), each block one E8M0 byte s for its scale 2^(s - 127).
//
// Quantising a block: s = the exponent of its largest magnitude less 2 (E2M1's
// largest exponent), so the largest value lies in [4, 8) and what is above 6
// saturates; every element is divided by the scale, which is exact, and rounded
// to nearest, ties to the even code.  v_cvt_scalef32_pk_fp4_* does the division,
// the rounding and the saturation of two elements; it was checked against the
// definition for every fp16 and bf16 value and around every border in fp32.
// A block that holds an infinity or a NaN gets s = 255, which stands for NaN.
#pragma once

#include "fl_kernels.hpp"

namespace fl {

typedef uint32_t any2_u32x4_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t any4_u32x4_t __attribute__((ext_vector_type(4), aligned(4)));

// N elements of a row in their own type, 16 bytes to a word group: loads of any
// alignment that suits the elements, zeros from `left` elements on.
template <int DT, int N>
struct RowValues {
    using io = Io<DT>;
    using raw = typename io::raw;
    using wide = std::conditional_t<DT == FL_F32, any4_u32x4_t, any2_u32x4_t>;
    static constexpr int VEC = 16 / io::size, WORDS = N * io::size / 4;
    uint32_t w[WORDS];

    __device__ __forceinline__ void load(const void *p, int64_t at, int64_t left) {
        const raw *q = static_cast<const raw *>(p) + at;
        if (left >= N) {
#pragma unroll
            for (int i = 0; i < N / VEC; ++i) {
                const u32x4_t v = *reinterpret_cast<const wide *>(q + i * VEC);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * i + e] = v[e];
            }
        } else {
            raw v[N];
#pragma unroll
            for (int t = 0; t < N; ++t) v[t] = t < left ? q[t] : raw(0);
            __builtin_memcpy(w, v, sizeof(w));
        }
    }
};

// The larger of two words' magnitudes, as bits: half by half for 16-bit types.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t larger_bits(uint32_t a, uint32_t b) {
    if constexpr (DT == FL_F32) {
        return a > b ? a : b;
    } else {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                      __builtin_bit_cast(u16x2_t, b)));
    }
}
template <int DT>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t w) {
    return w & (DT == FL_F32 ? 0x7fffffffu : 0x7fff7fffu);
}

// The scale byte of a block whose largest magnitude has these bits (in its type;
// 16-bit types: the larger half).
template <int DT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
    if constexpr (DT != FL_F32) bits = (bits & 0xffffu) > (bits >> 16) ? bits & 0xffffu : bits >> 16;
    uint32_t e;
    if constexpr (DT == FL_F16)
        e = __builtin_bit_cast(uint32_t, Io<FL_F16>::to_f32((uint16_t)bits)) >> 23;
    else
        e = bits >> (DT == FL_F32 ? 23 : 7);
    return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}
__device__ __forceinline__ float scale_value(uint32_t s) {  // s < 255
    return __builtin_bit_cast(float, s ? s << 23 : 0x00400000u);
}

// Eight values (four words of 16-bit types, eight of fp32) as eight codes.
template <int DT>
__device__ __forceinline__ uint32_t codes8(const uint32_t *w, float scale) {
    uint32_t c = 0;
    if constexpr (DT == FL_F32) {
#define FL_PAIR(i) \
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __builtin_bit_cast(float, w[2 * i]), __builtin_bit_cast(float, w[2 * i + 1]), scale, i)
        FL_PAIR(0);
        FL_PAIR(1);
        FL_PAIR(2);
        FL_PAIR(3);
#undef FL_PAIR
    } else if constexpr (DT == FL_F16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, w[3]), scale, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[3]), scale, 3);
    }
    return c;
}

// Values and codes: x (rows,K), or (K,rows) where it is read transposed; codes
// (rows, 16 blocks), scales (rows, blocks).
struct Mx4Args {
    const void *x;
    void *y;
    uint8_t *codes, *scales;
    int64_t rows;
    int K, blocks;
};

constexpr int kMx4Units = 4;  // units of eight values to a thread

// The first unit of a block of 256 threads.  The blocks lie in two dimensions of the launch, as
// one has less than 2^32 threads; those behind the last unit find no row.
__device__ __forceinline__ int64_t mx4_first_unit() {
    return ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (256 * kMx4Units);
}

// Rows along K: eight values to a lane, a block to four neighbouring lanes.  Bound
// by memory (2 + 17/32 bytes a 16-bit value): 8192x4096 bf16 14.4 us, 5.9 TB/s.
template <int DT>
__global__ void __launch_bounds__(256) quantize_mx4_kernel(Mx4Args a) {
    const uint32_t per_row = (uint32_t)a.blocks * 4;
    const int64_t first = mx4_first_unit(), row0 = first / per_row;
    const uint32_t col0 = (uint32_t)(first - row0 * per_row);
    RowValues<DT, 8> v[kMx4Units];
    int64_t row[kMx4Units];
    uint32_t col[kMx4Units];
#pragma unroll
    for (int i = 0; i < kMx4Units; ++i) {
        const uint32_t u = col0 + i * 256 + threadIdx.x, over = u / per_row;
        row[i] = row0 + over;
        col[i] = u - over * per_row;
        v[i].load(a.x, row[i] * a.K + (int64_t)col[i] * 8, row[i] < a.rows ? a.K - (int64_t)col[i] * 8 : 0);
    }
#pragma unroll
    for (int i = 0; i < kMx4Units; ++i) {
        uint32_t m = magnitude_bits<DT>(v[i].w[0]);
#pragma unroll
        for (int e = 1; e < RowValues<DT, 8>::WORDS; ++e) m = larger_bits<DT>(m, magnitude_bits<DT>(v[i].w[e]));
        // lanes 1 and 2 apart
        m = larger_bits<DT>(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, true));
        m = larger_bits<DT>(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, true));
        const uint32_t s = scale_byte<DT>(m);
        if (row[i] >= a.rows) continue;
        const uint32_t c = s == 255 ? 0 : codes8<DT>(v[i].w, scale_value(s));
        *reinterpret_cast<uint32_t *>(a.codes + (row[i] * per_row + col[i]) * 4) = c;
        if ((threadIdx.x & 3) == 0) a.scales[row[i] * a.blocks + col[i] / 4] = (uint8_t)s;
    }
}

// Columns of a (K,rows) matrix along K: a lane takes one block of VEC
// neighbouring columns, 32 pieces of 16 bytes, and pairs values of the same column
// from neighbouring rows.  The eight lanes of a group take neighbouring blocks, so
// a wave reads whole lines of 128 bytes and writes each column's codes as whole
// lines too: nothing passes through the LDS.  8192x4096 bf16 15.9 us (5.3 TB/s), fp32
// 36 (4.2).  SPLIT 4: four neighbouring lanes share a block's rows, for matrices that
// would fill few waves (4097 rows of 1537 fp16 7.4 us, 2.2 TB/s; 15.0 with one lane).
template <int DT, int SPLIT>
__global__ void __launch_bounds__(256) quantize_mx4_transposed_kernel(Mx4Args a) {
    using P = RowValues<DT, 16 / Io<DT>::size>;
    constexpr int VEC = P::VEC, ROWS = 32 / SPLIT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = lane % SPLIT;
    const int64_t col0 = ((int64_t)blockIdx.x * 32 + wave * 8 + (lane >> 3)) * VEC;
    const int block = (int)blockIdx.y * (8 / SPLIT) + (lane & 7) / SPLIT;
    if (col0 >= a.rows || block >= a.blocks) return;
    P v[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int64_t at = (int64_t)block * 32 + part * ROWS + k;
        v[k].load(a.x, at * a.rows + col0, at < a.K ? a.rows - col0 : 0);
    }
    uint32_t m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        m[e] = magnitude_bits<DT>(v[0].w[e]);
#pragma unroll
        for (int k = 1; k < ROWS; ++k) m[e] = larger_bits<DT>(m[e], magnitude_bits<DT>(v[k].w[e]));
        if constexpr (SPLIT == 4) {  // lanes 1 and 2 apart
            m[e] = larger_bits<DT>(m[e], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m[e], 0xb1, 0xf, 0xf, true));
            m[e] = larger_bits<DT>(m[e], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m[e], 0x4e, 0xf, 0xf, true));
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const bool high = DT != FL_F32 && (j & 1);
        const int e = DT == FL_F32 ? j : j / 2;
        const uint32_t s = scale_byte<DT>(DT == FL_F32 ? m[e] : high ? m[e] >> 16 : m[e] & 0xffffu);
        if (col0 + j >= a.rows) break;
        uint32_t c[ROWS / 8] = {};
        if (s != 255) {
#pragma unroll
            for (int g = 0; g < ROWS / 8; ++g) {  // eight values along K at a time
                uint32_t w[8];
#pragma unroll
                for (int t = 0; t < (DT == FL_F32 ? 8 : 4); ++t) {
                    if constexpr (DT == FL_F32)
                        w[t] = v[8 * g + t].w[e];
                    else  // the same half of two neighbouring rows
                        w[t] = __builtin_amdgcn_perm(v[8 * g + 2 * t + 1].w[e], v[8 * g + 2 * t].w[e],
                                                     high ? 0x07060302u : 0x05040100u);
                }
                c[g] = codes8<DT>(w, scale_value(s));
            }
        }
        uint8_t *to = a.codes + ((col0 + j) * a.blocks + block) * 16;
        if constexpr (SPLIT == 4)
            *reinterpret_cast<uint32_t *>(to + part * 4) = c[0];
        else
            *reinterpret_cast<u32x4_t *>(to) = u32x4_t{c[0], c[1], c[2], c[3]};
        if (part == 0) a.scales[(col0 + j) * a.blocks + block] = (uint8_t)s;
    }
}

// The values again: eight to a lane.  The scale is multiplied with in fp32 (exact
// but at the ends of the range, where it overflows or is denormal as it should),
// then one rounding to the type.  8192x4096 bf16 15.1 us, 5.6 TB/s.
template <int DT>
__global__ void __launch_bounds__(256) dequantize_mx4_kernel(Mx4Args a) {
    using io = Io<DT>;
    using raw = typename io::raw;
    using wide = typename RowValues<DT, 8>::wide;
    const uint32_t per_row = (uint32_t)a.blocks * 4;
    const int64_t first = mx4_first_unit(), row0 = first / per_row;
    const uint32_t col0 = (uint32_t)(first - row0 * per_row);
    uint32_t c[kMx4Units], s[kMx4Units], col[kMx4Units];
    int64_t row[kMx4Units];
#pragma unroll
    for (int i = 0; i < kMx4Units; ++i) {
        const uint32_t u = col0 + i * 256 + threadIdx.x, over = u / per_row;
        row[i] = row0 + over;
        col[i] = u - over * per_row;
        const bool on = row[i] < a.rows;
        c[i] = on ? *reinterpret_cast<const uint32_t *>(a.codes + (row[i] * per_row + col[i]) * 4) : 0;
        s[i] = on ? a.scales[row[i] * a.blocks + col[i] / 4] : 0;
    }
#pragma unroll
    for (int i = 0; i < kMx4Units; ++i) {
        const int64_t left = row[i] < a.rows ? a.K - (int64_t)col[i] * 8 : 0;
        if (left <= 0) continue;
        f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], 1.0f, 3)};
        raw v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t)
            v[t] = io::from_f32(s[i] == 255 ? __builtin_nanf("") : ldexpf(p[t / 2][t & 1], (int)s[i] - 127));
        raw *q = static_cast<raw *>(a.y) + row[i] * a.K + (int64_t)col[i] * 8;
        if (left >= 8) {
#pragma unroll
            for (int h = 0; h < 8 / RowValues<DT, 8>::VEC; ++h) {
                u32x4_t w;
                __builtin_memcpy(&w, v + h * RowValues<DT, 8>::VEC, 16);
                *reinterpret_cast<wide *>(q + h * RowValues<DT, 8>::VEC) = w;
            }
        } else {
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t < left) q[t] = v[t];
        }
    }
}

}  // namespace fl
