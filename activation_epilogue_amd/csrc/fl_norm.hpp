// fl_norm.hpp -- gfx950 device code of layer norm, forward and backward.
//
//   mean = sum_h x / H,  rstd = 1 / sqrt(sum_h (x - mean)^2 / H + eps)
//   y  = (x - mean) * rstd * weight + bias
//   g  = dy * weight,  c1 = sum_h g / H,  c2 = sum_h g * xhat / H
//   dx = rstd * (g - c1 - xhat * c2) + R,   xhat = (x - mean) * rstd
//   dweight = sum_rows dy * xhat,  dbias = sum_rows dy
//
// Bound by memory: a row is read once, kept in registers in its own type, and
// the sums over it (the mean first, then the squares of what is left) are taken there
// in fp32; a mean far from zero is put right before (far_mean), so that it costs no digits.  A team of 16,
// 64, 256 or 1024 lanes holds a row, NV pieces of 16 bytes to a lane; teams go
// from row to row with the weight and bias in registers.  The backward kernel
// keeps a team's sums of dy * xhat and dy in registers too, over all of its
// rows; a block adds its teams' through the LDS and writes one row of partial
// sums, which column_join_kernel adds in a fixed order: no atomics.
//
// Measured, 16384x4096 bf16: forward 38.6 us (7.0 TB/s of the 268 MB, some of
// which the last-level cache serves), backward with a residual 102 us (5.3 TB/s of
// 537 MB; 89 us, 6.0 TB/s, without the weight's and bias's sums: their 16 MB of
// partial sums written and read and one more launch are the rest).  Outputs that
// pass the L2 by: forward 40.6 -> 42.6 us without.  The next row's loads ahead of
// this one's sums: no gain (8192x8192 114 us both) or worse (102 -> 128: the registers).
//
// Pieces are read and written 16 bytes wide whatever the rows' alignment (the
// hardware takes any that suits the elements); what is left behind the last
// whole piece goes an element to a lane.
#pragma once

#include "fl_kernels.hpp"

namespace fl {

struct NormArgs {
    const void *x, *weight, *bias;  // weight, bias: or null
    void *y;                        // forward: y; backward: dx
    float *mean, *rstd;             // forward: written, or null; backward: read
    const void *dy, *residual;      // backward (residual: or null)
    float *part;                    // backward: partial sums (blocks, 2, H)
    float *dweight, *dbias;         // backward: where there is one block, its sums go here (each or null)
    int64_t M;
    int H;
    float eps;
};

constexpr int kStream = 2;  // the nt bit of a buffer access: outputs pass the L2 by

// One 16-byte piece of a row, held as it lies in memory.
template <int DT>
struct RowPiece {
    using io = Io<DT>;
    using raw = typename io::raw;
    static constexpr int ES = io::size, VEC = 16 / ES;
    u32x4_t w;

    __device__ __forceinline__ float get(int t) const {
        // a value of its own: __builtin_bit_cast of a vector's element reads element 0
        const uint32_t u = w[DT == FL_F32 ? t : t / 2];
        if constexpr (DT == FL_F32)
            return __builtin_bit_cast(float, u);
        else if constexpr (DT == FL_BF16)
            return __builtin_bit_cast(float, t & 1 ? u & 0xffff0000u : u << 16);
        else
            return io::to_f32((raw)(t & 1 ? u >> 16 : u));
    }
    __device__ __forceinline__ void fill(float f) {
        float all[VEC];
#pragma unroll
        for (int t = 0; t < VEC; ++t) all[t] = f;
        set(all);
    }
    // Between two uses: the compiler would otherwise keep the piece's floats, twice
    // the registers of a 16-bit type, to save conversions that cost nothing here.
    __device__ __forceinline__ void keep_packed() {
        if constexpr (DT != FL_F32) asm volatile("" : "+v"(w));
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == FL_F32)
                w[k] = __builtin_bit_cast(uint32_t, f[k]);
            else
                w[k] = io::pack2(f[2 * k], f[2 * k + 1]);
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32_t, w), r, off, 0, kStream);
    }
    __device__ __forceinline__ static float load_one(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return io::to_f32(__builtin_bit_cast(raw, load_elem<ES>(r, off)));
    }
    __device__ __forceinline__ static void store_one(float f, __amdgpu_buffer_rsrc_t r, uint32_t off) {
        store_elem<ES>(__builtin_bit_cast(typename RawBits<ES>::T, io::from_f32(f)), r, off);
    }
};

// Where a lane's pieces of a row lie: the whole pieces of the row go round the
// team, and of the elements behind the last whole piece (fewer than there are
// lanes) lane x has the x-th.  Pieces and elements that a lane has not got are
// out of the descriptor's range: they read as zeros and are not stored, without
// a branch.
template <int DT, int TEAM, int NV>
struct RowPlace {
    static constexpr int VEC = RowPiece<DT>::VEC, ES = RowPiece<DT>::ES;
    uint32_t off[NV], one;
    bool tail;  // the same in every lane

    // row: of the block's rows
    __device__ __forceinline__ RowPlace(int H, int row, int x) {
        const int whole = H / VEC;
#pragma unroll
        for (int n = 0; n < NV; ++n)
            off[n] = n * TEAM + x < whole ? (uint32_t)(row * H + (n * TEAM + x) * VEC) * ES : kOob;
        tail = H % VEC != 0;
        one = x < H % VEC ? (uint32_t)(row * H + whole * VEC + x) * ES : kOob;
    }
};

// The sum over a wave's lanes (or a row of 16 of them), the same in each: moves
// between lanes on the vector unit.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float lane_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    // neighbours, pairs, mirrored halves and mirrored rows of 16
    v = lane_add<0xb1>(v);
    v = lane_add<0x4e>(v);
    v = lane_add<0x141>(v);
    v = lane_add<0x140>(v);
    if constexpr (LANES == 64) {  // lane 15 to the next row, lane 31 to the upper half: lane 63 has all
        v = lane_add<0x142, 0xa>(v);
        v = lane_add<0x143, 0xc>(v);
        v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    }
    return v;
}

// The sum over a team's lanes, in each of them.  Teams of several waves meet in
// `part`, which two calls in turn must not share (a wave may still be reading).
template <int TEAM>
__device__ __forceinline__ float row_sum(float v, float *part) {
    if constexpr (TEAM <= 64) {
        return lanes_sum<TEAM>(v);
    } else {
        constexpr int WAVES = TEAM / 64;
        const int wave = threadIdx.x / 64, first = wave / WAVES * WAVES;
        v = lanes_sum<64>(v);
        if ((threadIdx.x & 63) == 0) part[wave] = v;
        __syncthreads();
        float s = part[first];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += part[first + w];
        return s;
    }
}

// The mean in fp32 of many values is off by some last places of theirs, which a row
// keeps in every value: 4096 times 1000.1, of which nothing should be left, became 0.04 after
// 1/sqrt(1e-5).  Rows whose mean is above 16 of their deviation (of the others the
// error is below a few 2^-20 of it) take the mean again, of what the first leaves, and the
// squares with it: two sums more, in registers.  Taken in every row, at once with the squares,
// the new mean made 16384x256 fp32 6.3 us, 5.7 so.  Rows that do take it: 4097x1537 fp32 10.1 us,
// 8.5 those that do not, 8192x4096 40.4 and 39.5.
__device__ __forceinline__ bool far_mean(float mean, float variance) { return mean * mean > 256.0f * variance; }

constexpr int log2_of(int n) { return n > 1 ? 1 + log2_of((n + 1) / 2) : 0; }  // rounded up

template <int DT, int TEAM, int NV>
__global__ void __launch_bounds__(TEAM > 256 ? TEAM : 256) layer_norm_kernel(NormArgs a) {
    using P = RowPiece<DT>;
    constexpr int VEC = P::VEC, THREADS = TEAM > 256 ? TEAM : 256, TEAMS = THREADS / TEAM;
    // whether the sum of a row of equal values is exact, and with it their mean
    constexpr bool EVEN = (DT == FL_F32 ? 24 : DT == FL_F16 ? 11 : 8) + log2_of(TEAM * NV * VEC) <= 24;
    __shared__ float part[EVEN ? 2 : 4][THREADS / 64];
    const int x = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const float count = (float)a.H;  // divided by, not multiplied with its inverse: rows of equal values come out even
    const size_t row_bytes = (size_t)a.H * P::ES;
    P w[NV], b[NV];
    float w1 = 1.0f, b1 = 0.0f;
    {
        const RowPlace<DT, TEAM, NV> at(a.H, 0, x);
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.weight, a.weight ? row_bytes : 0);
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.bias, a.bias ? row_bytes : 0);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            w[n].load(rw, at.off[n]);
            b[n].load(rb, at.off[n]);
            if (!a.weight) w[n].fill(1.0f);
        }
        if (at.tail) {
            w1 = a.weight ? P::load_one(rw, at.one) : 1.0f;
            b1 = P::load_one(rb, at.one);
        }
    }
    const RowPlace<DT, TEAM, NV> at(a.H, team, x);
    for (int64_t r0 = (int64_t)blockIdx.x * TEAMS; r0 < a.M; r0 += (int64_t)gridDim.x * TEAMS) {
        const int64_t r = r0 + team, left = a.M - r0;
        const size_t bytes = (left < TEAMS ? left : TEAMS) * row_bytes;
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + r0 * row_bytes, bytes);
        const __amdgpu_buffer_rsrc_t ry = make_rsrc(static_cast<const char *>(a.y) + r0 * row_bytes, bytes);
        P p[NV];
        float s = 0.0f, p1 = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) p[n].load(rx, at.off[n]);
        if (at.tail) p1 = P::load_one(rx, at.one);
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int t = 0; t < VEC; ++t) s += p[n].get(t);
        float mean = row_sum<TEAM>(s + p1, part[0]) / count;
        const auto variance = [&](float *part) {
            float s = at.one != kOob ? (p1 - mean) * (p1 - mean) : 0.0f;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float q = 0.0f;
                p[n].keep_packed();
#pragma unroll
                for (int t = 0; t < VEC; ++t) {
                    const float d = p[n].get(t) - mean;
                    q = __builtin_fmaf(d, d, q);
                }
                s += at.off[n] != kOob ? q : 0.0f;
            }
            return row_sum<TEAM>(s, part) / count;
        };
        float var = variance(part[1]);
        if constexpr (!EVEN) {
            if (far_mean(mean, var)) {  // the same in a team
                s = at.one != kOob ? p1 - mean : 0.0f;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    float q = 0.0f;
                    p[n].keep_packed();
#pragma unroll
                    for (int t = 0; t < VEC; ++t) q += p[n].get(t) - mean;
                    s += at.off[n] != kOob ? q : 0.0f;
                }
                mean += row_sum<TEAM>(s, part[2]) / count;
                var = variance(part[3]);
            }
        }
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (x == 0 && r < a.M) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float v[VEC];
            p[n].keep_packed();
            w[n].keep_packed();
            b[n].keep_packed();
#pragma unroll
            for (int t = 0; t < VEC; ++t)
                v[t] = __builtin_fmaf((p[n].get(t) - mean) * rstd, w[n].get(t), b[n].get(t));
            p[n].set(v);
            p[n].store(ry, at.off[n]);
        }
        if (at.tail) P::store_one(__builtin_fmaf((p1 - mean) * rstd, w1, b1), ry, at.one);
    }
}

typedef uint32_t piece16_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t piece32_t __attribute__((ext_vector_type(4), aligned(4)));

// A piece of a row of any length: zeros past its end.
template <int DT>
struct LongPiece {
    using io = Io<DT>;
    using raw = typename io::raw;
    using wide = std::conditional_t<DT == FL_F32, piece32_t, piece16_t>;
    static constexpr int VEC = 16 / io::size;
    raw v[VEC];

    __device__ __forceinline__ void load(const void *p, int64_t row, int i, int H) {
        const raw *q = static_cast<const raw *>(p) + row * H + i;
        if (i <= H - VEC) {
            const wide w = *reinterpret_cast<const wide *>(q);
            __builtin_memcpy(v, &w, 16);
        } else {
#pragma unroll
            for (int t = 0; t < VEC; ++t) v[t] = t < H - i ? q[t] : raw(0);
        }
    }
    __device__ __forceinline__ void store(void *p, int64_t row, int i, int H) const {
        raw *q = static_cast<raw *>(p) + row * H + i;
        if (i <= H - VEC) {
            wide w;
            __builtin_memcpy(&w, v, 16);
            *reinterpret_cast<wide *>(q) = w;
        } else {
#pragma unroll
            for (int t = 0; t < VEC; ++t)
                if (t < H - i) q[t] = v[t];
        }
    }
    __device__ __forceinline__ float get(int t) const { return io::to_f32(v[t]); }
    __device__ __forceinline__ void set(int t, float f) { v[t] = io::from_f32(f); }
};

// Rows that no team's registers hold: a block per row, which reads it three times
// (from the L2 after the first), a row with a mean far from zero five times.
// 1024x40000 bf16 44 us, 4096x20000 80 (3.7 and 4.1 TB/s of what is read once and written).
template <int DT>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(NormArgs a) {
    using P = LongPiece<DT>;
    constexpr int VEC = P::VEC;
    __shared__ float part[4][16];
    for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
        float s = 0.0f;
        for (int64_t i = threadIdx.x * VEC; i < a.H; i += 1024 * VEC) {
            P p;
            p.load(a.x, r, (int)i, a.H);
#pragma unroll
            for (int t = 0; t < VEC; ++t) s += p.get(t);
        }
        float mean = row_sum<1024>(s, part[0]) / (float)a.H;
        const auto variance = [&](float *part) {
            float s = 0.0f;
            for (int64_t i = threadIdx.x * VEC; i < a.H; i += 1024 * VEC) {
                P p;
                p.load(a.x, r, (int)i, a.H);
#pragma unroll
                for (int t = 0; t < VEC; ++t) {
                    const float d = i + t < a.H ? p.get(t) - mean : 0.0f;
                    s = __builtin_fmaf(d, d, s);
                }
            }
            return row_sum<1024>(s, part) / (float)a.H;
        };
        float var = variance(part[1]);
        if (far_mean(mean, var)) {
            s = 0.0f;
            for (int64_t i = threadIdx.x * VEC; i < a.H; i += 1024 * VEC) {
                P p;
                p.load(a.x, r, (int)i, a.H);
#pragma unroll
                for (int t = 0; t < VEC; ++t) s += i + t < a.H ? p.get(t) - mean : 0.0f;
            }
            mean += row_sum<1024>(s, part[2]) / (float)a.H;
            var = variance(part[3]);
        }
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        for (int64_t i = threadIdx.x * VEC; i < a.H; i += 1024 * VEC) {
            P p, w, b;
            p.load(a.x, r, (int)i, a.H);
            if (a.weight) w.load(a.weight, 0, (int)i, a.H);
            if (a.bias) b.load(a.bias, 0, (int)i, a.H);
#pragma unroll
            for (int t = 0; t < VEC; ++t) {
                float v = (p.get(t) - mean) * rstd;
                if (a.weight) v *= w.get(t);
                if (a.bias) v += b.get(t);
                p.set(t, v);
            }
            p.store(a.y, r, (int)i, a.H);
        }
    }
}

// SUMS: also the weight's and the bias's gradient.  dx may be dy, x or the
// residual: a lane has read its pieces of them before it writes any.
template <int DT, int TEAM, int NV, bool SUMS>
__global__ void __launch_bounds__(TEAM > 512 ? TEAM : 512) layer_norm_bwd_kernel(NormArgs a) {
    using P = RowPiece<DT>;
    constexpr int VEC = P::VEC, THREADS = TEAM > 512 ? TEAM : 512, TEAMS = THREADS / TEAM;
    __shared__ float part[2][THREADS / 64];
    const int x = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const float count = (float)a.H;
    const size_t row_bytes = (size_t)a.H * P::ES;
    P w[NV];
    float sw[SUMS ? NV : 1][VEC], sb[SUMS ? NV : 1][VEC], w1 = 1.0f, sw1 = 0.0f, sb1 = 0.0f;
    {
        const RowPlace<DT, TEAM, NV> at(a.H, 0, x);
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.weight, a.weight ? row_bytes : 0);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            w[n].load(rw, at.off[n]);
            if (!a.weight) w[n].fill(1.0f);
            if constexpr (SUMS) {
#pragma unroll
                for (int t = 0; t < VEC; ++t) sw[n][t] = sb[n][t] = 0.0f;
            }
        }
        if (at.tail && a.weight) w1 = P::load_one(rw, at.one);
    }
    const RowPlace<DT, TEAM, NV> at(a.H, team, x);
    for (int64_t r0 = (int64_t)blockIdx.x * TEAMS; r0 < a.M; r0 += (int64_t)gridDim.x * TEAMS) {
        const int64_t left = a.M - r0, r = team < left ? r0 + team : r0;
        const size_t bytes = (left < TEAMS ? left : TEAMS) * row_bytes, from = r0 * row_bytes;
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(static_cast<const char *>(a.x) + from, bytes);
        const __amdgpu_buffer_rsrc_t rd = make_rsrc(static_cast<const char *>(a.dy) + from, bytes);
        const __amdgpu_buffer_rsrc_t rr = make_rsrc(static_cast<const char *>(a.residual) + from, a.residual ? bytes : 0);
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(static_cast<const char *>(a.y) + from, bytes);
        P p[NV], d[NV];
        float p1 = 0.0f, d1 = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            p[n].load(rx, at.off[n]);
            d[n].load(rd, at.off[n]);
        }
        if (at.tail) {
            p1 = P::load_one(rx, at.one);
            d1 = P::load_one(rd, at.one);
        }
        // a team without a row adds zeros: dy, mean and rstd are
        const float mean = team < left ? a.mean[r] : 0.0f, rstd = team < left ? a.rstd[r] : 0.0f;
        const float hat1 = (p1 - mean) * rstd;
        float c1 = d1 * w1, c2 = at.one != kOob ? c1 * hat1 : 0.0f;
        if constexpr (SUMS) {
            sw1 = __builtin_fmaf(d1, hat1, sw1);
            sb1 += d1;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float g[VEC], q = 0.0f;
            p[n].keep_packed();
            d[n].keep_packed();
            w[n].keep_packed();
#pragma unroll
            for (int t = 0; t < VEC; ++t) g[t] = d[n].get(t) * w[n].get(t);
#pragma unroll
            for (int t = 0; t < VEC; ++t) {
                const float hat = (p[n].get(t) - mean) * rstd;
                c1 += g[t];
                q = __builtin_fmaf(g[t], hat, q);
                if constexpr (SUMS) {
                    sw[n][t] = __builtin_fmaf(d[n].get(t), hat, sw[n][t]);
                    sb[n][t] += d[n].get(t);
                }
            }
            c2 += at.off[n] != kOob ? q : 0.0f;
            __builtin_amdgcn_sched_barrier(0);  // a piece's floats end with it: pieces in turn need fewer registers
        }
        c1 = row_sum<TEAM>(c1, part[0]) / count;
        c2 = row_sum<TEAM>(c2, part[1]) / count;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float v[VEC];
            p[n].keep_packed();
            d[n].keep_packed();
            w[n].keep_packed();
#pragma unroll
            for (int t = 0; t < VEC; ++t)
                v[t] = rstd * (d[n].get(t) * w[n].get(t) - c1 - (p[n].get(t) - mean) * rstd * c2);
            if (a.residual) {
                P res;
                res.load(rr, at.off[n]);
#pragma unroll
                for (int t = 0; t < VEC; ++t) v[t] += res.get(t);
            }
            p[n].set(v);
            p[n].store(ro, at.off[n]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (at.tail) {
            float v = rstd * (d1 * w1 - c1 - hat1 * c2);
            if (a.residual) v += P::load_one(rr, at.one);
            P::store_one(v, ro, at.one);
        }
    }
    if constexpr (SUMS) {
        // 16 bytes to a lane: element by element, lanes lie 32 bytes apart and each of their
        // stores meets a line of its own (1x16384 bf16 5.5 us, 17.3 so; 8192x8192 91, 97)
        typedef float four_t __attribute__((ext_vector_type(4), aligned(4)));
        float *to[2] = {a.dweight, a.dbias};
        if (gridDim.x > 1)
            for (int k = 0; k < 2; ++k) to[k] = a.part + ((int64_t)blockIdx.x * 2 + k) * a.H;
        const int whole = a.H / VEC * VEC;
        if constexpr (TEAMS == 1) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int h = 0; h < VEC / 4; ++h) {
                        const float(&v)[VEC] = k ? sb[n] : sw[n];
                        const int i = (n * TEAM + x) * VEC + h * 4;
                        if (i < whole && to[k])
                            *reinterpret_cast<four_t *>(to[k] + i) = four_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
                    }
            if (at.one != kOob && to[0]) to[0][whole + x] = sw1;
            if (at.one != kOob && to[1]) to[1][whole + x] = sb1;
        } else {
            constexpr int QUADS = VEC / 4;
            __shared__ __align__(16) f32x4_t sums[2][QUADS][TEAMS][TEAM];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                if (n) __syncthreads();
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int h = 0; h < QUADS; ++h) {
                        const float(&v)[VEC] = k ? sb[n] : sw[n];
                        sums[k][h][team][x] = f32x4_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
                    }
                __syncthreads();
                for (int c = threadIdx.x; c < 2 * QUADS * TEAM; c += THREADS) {
                    const int k = c / (QUADS * TEAM), h = c / TEAM % QUADS, l = c % TEAM;
                    const int i = (n * TEAM + l) * VEC + h * 4;
                    f32x4_t v = sums[k][h][0][l];
                    for (int m = 1; m < TEAMS; ++m) v += sums[k][h][m][l];
                    if (i < whole && to[k]) *reinterpret_cast<four_t *>(to[k] + i) = four_t{v[0], v[1], v[2], v[3]};
                }
            }
            if (at.tail) {
                float *one = reinterpret_cast<float *>(sums);  // (2, teams, VEC)
                __syncthreads();
                if (x < VEC) {
                    one[team * VEC + x] = sw1;
                    one[(TEAMS + team) * VEC + x] = sb1;
                }
                __syncthreads();
                if (threadIdx.x < 2 * VEC) {
                    const int k = threadIdx.x / VEC, e = threadIdx.x % VEC;
                    float v = one[k * TEAMS * VEC + e];
                    for (int m = 1; m < TEAMS; ++m) v += one[(k * TEAMS + m) * VEC + e];
                    if (e < a.H % VEC && to[k]) to[k][whole + e] = v;
                }
            }
        }
    }
}

// Rows that no team's registers hold: c1 and c2 of every row first, a block per
// row, then a block per piece of 256 lanes' columns and run of rows: everything is read
// twice.  1024x40000 bf16 94 us, 63 without the weight's and bias's sums, 4096x20000 164
// and 144 (3.4 TB/s of what is read once and written).
template <int DT>
__global__ void __launch_bounds__(1024) layer_norm_bwd_long_kernel(NormArgs a, float *c) {
    using P = LongPiece<DT>;
    constexpr int VEC = P::VEC;
    __shared__ float part[2][16];
    for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float c1 = 0.0f, c2 = 0.0f;
        for (int64_t i = threadIdx.x * VEC; i < a.H; i += 1024 * VEC) {
            P p, d, w;
            p.load(a.x, r, (int)i, a.H);
            d.load(a.dy, r, (int)i, a.H);
            if (a.weight) w.load(a.weight, 0, (int)i, a.H);
#pragma unroll
            for (int t = 0; t < VEC; ++t) {
                const float g = a.weight ? d.get(t) * w.get(t) : d.get(t);
                c1 += g;
                c2 = i + t < a.H ? __builtin_fmaf(g, (p.get(t) - mean) * rstd, c2) : c2;
            }
        }
        c1 = row_sum<1024>(c1, part[0]) / (float)a.H;
        c2 = row_sum<1024>(c2, part[1]) / (float)a.H;
        if (threadIdx.x == 0) {
            c[2 * r] = c1;
            c[2 * r + 1] = c2;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(256) layer_norm_bwd_columns_kernel(NormArgs a, const float *c) {
    using P = LongPiece<DT>;
    constexpr int VEC = P::VEC;
    const int64_t first = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (first >= a.H) return;
    const int i = (int)first;
    P w;
    if (a.weight) w.load(a.weight, 0, i, a.H);
    float sw[VEC], sb[VEC];
#pragma unroll
    for (int t = 0; t < VEC; ++t) sw[t] = sb[t] = 0.0f;
    for (int64_t r = blockIdx.y; r < a.M; r += gridDim.y) {
        const float mean = a.mean[r], rstd = a.rstd[r], c1 = c[2 * r], c2 = c[2 * r + 1];
        P p, d, res;
        p.load(a.x, r, i, a.H);
        d.load(a.dy, r, i, a.H);
        if (a.residual) res.load(a.residual, r, i, a.H);
#pragma unroll
        for (int t = 0; t < VEC; ++t) {
            const float dy = d.get(t), hat = (p.get(t) - mean) * rstd, g = a.weight ? dy * w.get(t) : dy;
            sw[t] = __builtin_fmaf(dy, hat, sw[t]);
            sb[t] += dy;
            float v = rstd * (g - c1 - hat * c2);
            if (a.residual) v += res.get(t);
            p.set(t, v);
        }
        p.store(a.y, r, i, a.H);
    }
    float *to[2] = {a.dweight, a.dbias};
    if (gridDim.y > 1)
        for (int k = 0; k < 2; ++k) to[k] = a.part ? a.part + ((int64_t)blockIdx.y * 2 + k) * a.H : nullptr;
#pragma unroll
    for (int t = 0; t < VEC; ++t) {
        if (i + t < a.H && to[0]) to[0][i + t] = sw[t];
        if (i + t < a.H && to[1]) to[1][i + t] = sb[t];
    }
}

// The sum of `rows` rows of partial sums (rows, 2, H): 32 columns to a block, 32
// runs of rows side by side, whose loads go out eight at a time.  blockIdx.y: 0
// the weight's, 1 the bias's.  The columns' blocks lie in the first and the last dimension of
// the launch (one has less than 2^32 threads: 2^27 columns).
__global__ void __launch_bounds__(1024) column_join_kernel(NormArgs a, int rows) {
    __shared__ float sums[32][32];
    float *out = blockIdx.y ? a.dbias : a.dweight;
    if (!out) return;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t i = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * 32 + x;
    float s = 0.0f;
    if (i < a.H) {
#pragma unroll 8
        for (int r = y; r < rows; r += 32) s += a.part[((int64_t)r * 2 + blockIdx.y) * a.H + i];
    }
    sums[y][x] = s;
    __syncthreads();
    if (y || i >= a.H) return;
#pragma unroll
    for (int k = 1; k < 32; ++k) s += sums[k][x];
    out[i] = s;
}

// The gradients of no rows.
__global__ void __launch_bounds__(256) zero_columns_kernel(NormArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.H) return;
    if (a.dweight) a.dweight[i] = 0.0f;
    if (a.dbias) a.dbias[i] = 0.0f;
}

}  // namespace fl
