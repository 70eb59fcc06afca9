// fl_grouped.hpp -- gfx950 device code of the experts' products: the fused
// linear layer, its backward epilogue and its weight gradients over runs of
// rows, one run per expert.
//
// Three forms of product over the rows r of expert e:
//   kFormFwd    X[r,:] = A[r,:] @ B[e]        B[e] (K,N), N contiguous
//   kFormBwd    D[r,:] = G[r,:] @ W[e]^T      W[e] (N,K), K contiguous
//   kFormGrad   dW[e]  = sum_r A[r,:]^T G[r,:]
// The host knows how many rows there are, not where an expert's run starts or
// ends: every workgroup finds its tile from the device array of offsets.
#pragma once

#include "fl_kernels.hpp"

namespace fl {

enum Form { kFormFwd = 0, kFormBwd = 1, kFormGrad = 2 };

struct GroupedArgs {
    const void *A;           // forward: (A_rows,K); backward: G (S,K); gradient: A (S,K)
    const int32_t *index;    // forward: row of A for every row, or null
    const int32_t *offsets;  // (E+1,)
    const void *B;           // forward: (E,K,N); backward: W (E,N,K); gradient: G (S,N)
    const void *bias;        // forward: (E,N) or null
    const void *Y;           // the gate's operand (S,N)
    const void *X;           // backward: the saved pre-activation (S,N), null without an activation
    void *out;               // out, dX (S,N), or dW (E,K,N)
    void *out2;              // forward: pre or null; backward: dY of the gate (S,N)
    float *dbias;            // gradient: (E,N) or null
    int64_t A_rows;
    int S, N, K, E;
    int dw_f32;              // gradient: dW in fp32 (else in the dtype)
    int tiles_n;
};

// Expert e's rows, limited to [0, S] whatever the array holds.
__device__ __forceinline__ int run_bound(const GroupedArgs &a, int e) {
    const int v = a.offsets[e];
    return v < 0 ? 0 : v > a.S ? a.S : v;
}

struct RunTile {
    int e;       // expert, -1 past the last tile
    int lo, hi;  // its rows
    int m;       // tile within the run
    int total;   // row tiles of all experts
};

// Row tile `tile` of the experts' runs cut into tiles of bm rows (each run
// from its own start): every wave scans the runs 64 at a time.
__device__ __forceinline__ RunTile find_run_tile(const GroupedArgs &a, int bm, int tile) {
    const int lane = threadIdx.x & 63;
    RunTile t{-1, 0, 0, 0, 0};
    int base = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        const int lo = e < a.E ? run_bound(a, e) : 0, hi = e < a.E ? run_bound(a, e + 1) : 0;
        const int n = hi > lo ? (hi - lo + bm - 1) / bm : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(incl, o);
            if (lane >= o) incl += v;
        }
        const uint64_t past = __ballot(base + incl > tile);
        if (t.e < 0 && past) {
            const int l = __builtin_ctzll(past);
            t.e = e0 + l;
            t.lo = __builtin_amdgcn_readlane(lo, l);
            t.hi = __builtin_amdgcn_readlane(hi, l);
            t.m = tile - base - __builtin_amdgcn_readlane(incl - n, l);
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    t.total = base;
    return t;
}

// ------------------------------------------------------- staged by elements

// The kernel for every dtype, size and alignment: 64x64 tiles, 4 waves of one
// 32x32 block each, K stages of 32 values loaded by elements into LDS.
template <int DT, int FORM, int ACT>
struct GroupedPlain {
    using io = Io<DT>;
    using raw = typename io::raw;
    static constexpr int BM = 64, BN = 64, BK = 32;
    static constexpr int ROW = BK + 16 / io::size;  // padded LDS row
    static constexpr int THREADS = 256;

    __device__ static void run(const GroupedArgs &a, raw *As, raw *Bs) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        const int wm = wave >> 1, wn = wave & 1;
        const raw *A = static_cast<const raw *>(a.A);
        const raw *B = static_cast<const raw *>(a.B);
        int e, lo, hi, m0;  // m0: first row (of the product) of the tile; its rows end at mend
        const int n0 = (int)(blockIdx.x % a.tiles_n) * BN;
        int mend, depth;
        if constexpr (FORM == kFormGrad) {
            const int per = a.K ? (a.K + BM - 1) / BM : 1;  // (no columns of A: dbias alone)
            const int q = blockIdx.x / a.tiles_n;
            e = q / per;
            lo = run_bound(a, e);
            hi = run_bound(a, e + 1);
            m0 = (q % per) * BM;
            mend = a.K;
            depth = hi > lo ? hi - lo : 0;
        } else {
            const RunTile t = find_run_tile(a, BM, blockIdx.x / a.tiles_n);
            if (t.e < 0) return;
            e = t.e;
            lo = t.lo;
            hi = t.hi;
            m0 = lo + t.m * BM;
            mend = hi;
            depth = a.K;
        }
        f32x16_t acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
        float dsum = 0.0f;
        for (int k0 = 0; k0 < depth; k0 += BK) {
#pragma unroll
            for (int i = 0; i < BM * BK / THREADS; ++i) {
                const int q = tid + i * THREADS;
                // consecutive threads along the operand's contiguous dimension
                const int r = FORM == kFormGrad ? q % BM : q / BK, k = FORM == kFormGrad ? q / BM : q % BK;
                raw v = raw(0);
                if (k0 + k < depth && m0 + r < mend) {
                    if constexpr (FORM == kFormGrad) {
                        v = A[(int64_t)(lo + k0 + k) * a.K + m0 + r];
                    } else {
                        const int64_t row = FORM == kFormFwd && a.index ? a.index[m0 + r] : m0 + r;
                        if (row >= 0 && row < a.A_rows) v = A[row * a.K + k0 + k];
                    }
                }
                As[r * ROW + k] = v;
            }
#pragma unroll
            for (int i = 0; i < BN * BK / THREADS; ++i) {
                const int q = tid + i * THREADS;
                const int n = FORM == kFormBwd ? q / BK : q % BN, k = FORM == kFormBwd ? q % BK : q / BN;
                raw v = raw(0);
                if (k0 + k < depth && n0 + n < a.N) {
                    if constexpr (FORM == kFormFwd)
                        v = B[((int64_t)e * a.K + k0 + k) * a.N + n0 + n];
                    else if constexpr (FORM == kFormBwd)
                        v = B[((int64_t)e * a.N + n0 + n) * a.K + k0 + k];
                    else
                        v = B[(int64_t)(lo + k0 + k) * a.N + n0 + n];
                }
                Bs[n * ROW + k] = v;
            }
            __syncthreads();
            const int lr = lane & 31, lg = lane >> 5;
            if constexpr (DT == FL_F32) {
#pragma unroll
                for (int k = 0; k < BK; k += 2)
                    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(Bs[(wn * 32 + lr) * ROW + k + lg],
                                                               As[(wm * 32 + lr) * ROW + k + lg], acc, 0, 0, 0);
            } else {
#pragma unroll
                for (int k = 0; k < BK; k += 16) {
                    const u32x4_t bv = *reinterpret_cast<const u32x4_t *>(&Bs[(wn * 32 + lr) * ROW + k + lg * 8]);
                    const u32x4_t av = *reinterpret_cast<const u32x4_t *>(&As[(wm * 32 + lr) * ROW + k + lg * 8]);
                    if constexpr (DT == FL_F16)
                        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, bv),
                                                                     __builtin_bit_cast(f16x8_t, av), acc, 0, 0, 0);
                    else
                        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, bv),
                                                                      __builtin_bit_cast(bf16x8_t, av), acc, 0, 0, 0);
                }
            }
            if (FORM == kFormGrad && a.dbias && m0 == 0 && tid < BN) {
#pragma unroll
                for (int k = 0; k < BK; ++k) dsum += io::to_f32(Bs[tid * ROW + k]);
            }
            __syncthreads();
        }
        if (FORM == kFormGrad && a.dbias && m0 == 0 && tid < BN && n0 + tid < a.N)
            a.dbias[(int64_t)e * a.N + n0 + tid] = dsum;
        // lane l: row l%32, columns q*8 + (l/32)*4 + 0..3 of its wave's block
        const int row = m0 + wm * 32 + (lane & 31);
        if (row >= mend) return;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = n0 + wn * 32 + q * 8 + (lane >> 5) * 4 + i;
                if (col >= a.N) continue;
                const float s = acc[q * 4 + i];
                if constexpr (FORM == kFormGrad) {
                    const int64_t o = ((int64_t)e * a.K + row) * a.N + col;
                    if (a.dw_f32)
                        static_cast<float *>(a.out)[o] = s;
                    else
                        static_cast<raw *>(a.out)[o] = io::from_f32(s);
                } else {
                    const int64_t o = (int64_t)row * a.N + col;
                    const float y = ACT == FL_ACT_GLU ? io::to_f32(static_cast<const raw *>(a.Y)[o]) : 0.0f;
                    if constexpr (FORM == kFormFwd) {
                        const float b =
                            a.bias ? io::to_f32(static_cast<const raw *>(a.bias)[(int64_t)e * a.N + col]) : 0.0f;
                        const float x = s + b;
                        if (a.out2) static_cast<raw *>(a.out2)[o] = io::from_f32(x);
                        static_cast<raw *>(a.out)[o] = io::from_f32(activate<ACT>(x, y));
                    } else {
                        const float xs = a.X ? io::to_f32(static_cast<const raw *>(a.X)[o]) : 0.0f;
                        const float dx = s * activate_grad<ACT>(xs, y);
                        static_cast<raw *>(a.out)[o] = io::from_f32(dx);
                        if constexpr (ACT == FL_ACT_GLU) static_cast<raw *>(a.out2)[o] = io::from_f32(s * xs);
                    }
                }
            }
        }
    }
};

template <int DT, int FORM, int ACT>
__global__ void __launch_bounds__(256) grouped_plain_kernel(GroupedArgs a) {
    using T = GroupedPlain<DT, FORM, ACT>;
    __shared__ __attribute__((aligned(16))) typename T::raw As[T::BM * T::ROW], Bs[T::BN * T::ROW];
    T::run(a, As, Bs);
}

typedef void (*grouped_launcher)(const GroupedArgs &, int64_t grid, hipStream_t);

// Launchers of the kernel for (DT, form, act); each dtype's are compiled in
// their own unit.
template <int DT>
grouped_launcher pick_grouped_plain(int form, int act);

}  // namespace fl
