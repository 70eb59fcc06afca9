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
    int group;               // row tiles per band of the tile order
    int spread;              // nonzero: each XCD takes its share of every expert's tiles
    int max_tiles;           // limit on the tiles found from the offsets
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

// Row tiles of all experts: the runs cut into tiles of bm rows (each run from
// its own start).
__device__ __forceinline__ int count_run_tiles(const GroupedArgs &a, int bm) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e = lane; e < a.E; e += 64) {
        const int lo = run_bound(a, e), hi = run_bound(a, e + 1);
        n += hi > lo ? (hi - lo + bm - 1) / bm : 0;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
    return __builtin_amdgcn_readfirstlane(n);
}

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

// ------------------------------------------------------------- fp32 products

// 64x64 tiles, 4 waves of one 32x32 block each (v_mfma_f32_32x32x2_f32), K
// stages of 32 values loaded by elements into LDS.
template <int FORM, int ACT>
struct GroupedF32 {
    static constexpr int BM = 64, BN = 64, BK = 32;
    static constexpr int ROW = BK + 4;  // padded LDS row
    static constexpr int THREADS = 256;

    __device__ static void run(const GroupedArgs &a, float *As, float *Bs) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        const int wm = wave >> 1, wn = wave & 1;
        const float *A = static_cast<const float *>(a.A);
        const float *B = static_cast<const float *>(a.B);
        int e, lo, hi, m0;  // m0: first row (of the product) of the tile; its rows end at mend
        const int n0 = (int)(blockIdx.x % a.tiles_n) * BN;
        int mend, depth;
        if constexpr (FORM == kFormGrad) {
            const int per = (a.K + BM - 1) / BM;
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
        for (int k0 = 0; k0 < depth; k0 += BK) {
#pragma unroll
            for (int i = 0; i < BM * BK / THREADS; ++i) {
                const int q = tid + i * THREADS;
                // consecutive threads along the operand's contiguous dimension
                const int r = FORM == kFormGrad ? q % BM : q / BK, k = FORM == kFormGrad ? q / BM : q % BK;
                float v = 0.0f;
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
                float v = 0.0f;
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
#pragma unroll
            for (int k = 0; k < BK; k += 2)
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(Bs[(wn * 32 + lr) * ROW + k + lg],
                                                           As[(wm * 32 + lr) * ROW + k + lg], acc, 0, 0, 0);
            __syncthreads();
        }
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
                    static_cast<float *>(a.out)[((int64_t)e * a.K + row) * a.N + col] = s;
                } else {
                    const int64_t o = (int64_t)row * a.N + col;
                    const float y = ACT == FL_ACT_GLU ? static_cast<const float *>(a.Y)[o] : 0.0f;
                    if constexpr (FORM == kFormFwd) {
                        const float x = s + (a.bias ? static_cast<const float *>(a.bias)[(int64_t)e * a.N + col] : 0.0f);
                        if (a.out2) static_cast<float *>(a.out2)[o] = x;
                        static_cast<float *>(a.out)[o] = activate<ACT>(x, y);
                    } else {
                        const float xs = a.X ? static_cast<const float *>(a.X)[o] : 0.0f;
                        static_cast<float *>(a.out)[o] = s * activate_grad<ACT>(xs, y);
                        if constexpr (ACT == FL_ACT_GLU) static_cast<float *>(a.out2)[o] = s * xs;
                    }
                }
            }
        }
    }
};

template <int FORM, int ACT>
__global__ void __launch_bounds__(256) grouped_f32_kernel(GroupedArgs a) {
    using T = GroupedF32<FORM, ACT>;
    __shared__ __attribute__((aligned(16))) float As[T::BM * T::ROW], Bs[T::BN * T::ROW];
    T::run(a, As, Bs);
}

// ----------------------------------------------------- the bias gradient

// dbias[e] = the sum of expert e's rows of G: a block sums 128 columns of one
// expert in 16 groups of rows (group g: rows g, g+16, ..), then adds the groups
// in order.  A pass over G of its own: 1/K of the operations of dW.
constexpr int kColumns = 128, kRowGroups = 16;
typedef uint32_t u32x4_unaligned __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
__global__ void __launch_bounds__(256) grouped_column_sum_kernel(GroupedArgs a) {
    using io = Io<DT>;
    using raw = typename io::raw;
    // a thread's 8 columns, in 16-byte loads (which may be unaligned); at the
    // end of a row it loads the row's last 8 and keeps its own
    constexpr int PER = 8;
    __shared__ float part[kRowGroups][kColumns];
    const int blocks_n = (a.N + kColumns - 1) / kColumns;
    const int e = blockIdx.x / blocks_n, c0 = (blockIdx.x % blocks_n) * kColumns;
    const int g = threadIdx.x / (kColumns / PER), c = c0 + (threadIdx.x % (kColumns / PER)) * PER;
    const int lo = run_bound(a, e), hi = run_bound(a, e + 1);
    const raw *G = static_cast<const raw *>(a.B);
    float sum[PER];
#pragma unroll
    for (int t = 0; t < PER; ++t) sum[t] = 0.0f;
    const int at = c + PER <= a.N ? c : a.N - PER;
    if (at >= 0) {
        constexpr int W = PER * io::size / 16;
#pragma unroll 4
        for (int64_t r = lo + g; r < hi; r += kRowGroups) {
            const u32x4_unaligned *p = reinterpret_cast<const u32x4_unaligned *>(G + r * a.N + at);
            raw v[PER];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const u32x4_t q = p[w];
                __builtin_memcpy(&v[w * PER / W], &q, 16);
            }
#pragma unroll
            for (int t = 0; t < PER; ++t) sum[t] += io::to_f32(v[t]);
        }
    } else {  // fewer than 8 columns in all
        for (int64_t r = lo + g; r < hi; r += kRowGroups)
            for (int t = 0; t < PER; ++t)
                if (at + t >= 0) sum[t] += io::to_f32(G[r * a.N + at + t]);
    }
#pragma unroll
    for (int t = 0; t < PER; ++t)
        if (at + t >= c) part[g][at + t - c0] = sum[t];
    __syncthreads();
    if (threadIdx.x < kColumns && c0 + (int)threadIdx.x < a.N) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kRowGroups; ++i) s += part[i][threadIdx.x];
        a.dbias[(int64_t)e * a.N + c0 + threadIdx.x] = s;
    }
}

typedef void (*grouped_launcher)(const GroupedArgs &, int64_t grid, hipStream_t);

// The tiles of grouped_dma_kernel (fl_grouped_dma.hpp), for 16-bit operands.
// time: of one workgroup per slot (256 CUs x per_cu), relative to 256x256 tiles
// at large sizes (8192x2 rows of 8 experts, K 4096, N 14336: 1030, 950, 810, 605
// and 370 TFLOP/s).
struct GroupedTileShape {
    int bm, bn, per_cu;
    float time;
};
enum GroupedVariant { kTile256x256 = 0, kTile256x128, kTile128x128, kTile64x128, kTile32x128, kGroupedVariants };
constexpr GroupedTileShape kGroupedTiles[kGroupedVariants] = {
    {256, 256, 1, 1.0f}, {256, 128, 1, 0.54f}, {128, 128, 2, 0.64f}, {64, 128, 2, 0.425f}, {32, 128, 2, 0.35f}};
typedef void (*grouped_dma_launcher)(const GroupedArgs &, int act, int64_t grid, hipStream_t);
// Compiled one dtype and form to a unit; the gradient has the first and the third tile only.
template <int DT, int FORM>
grouped_dma_launcher pick_grouped_dma_form(int variant);

// Launcher of the fp32 kernel for (form, act).
grouped_launcher pick_grouped_f32(int form, int act);
template <int DT>
void launch_column_sum(const GroupedArgs &a, hipStream_t s);

}  // namespace fl
