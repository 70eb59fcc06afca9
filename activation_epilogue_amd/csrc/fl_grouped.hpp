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

// The tiles of grouped_dma_kernel (fl_grouped_dma.hpp).  time: of a round (one
// workgroup in every slot, 256 CUs x per_cu), in units of the widest tile's at
// large sizes (8192x2 rows of 8 experts, K 4096, N 14336: 1030, 950, 810, 605
// and 370 TFLOP/s).  fp32 has one tile: 64x64 reaches 130 TFLOP/s at 4096x2
// rows, K 2048, N 4096 (128x128: 114 to 134, and half as much where there are
// few tiles).
struct GroupedTileShape {
    int bm, bn, per_cu;
    float time;
    bool grad;  // compiled for the gradient too
};
enum GroupedVariant { kTile256x256 = 0, kTile256x128, kTile128x128, kTile64x128, kTile32x128, kTileF32, kGroupedVariants };
constexpr GroupedTileShape kGroupedTiles[kGroupedVariants] = {
    {256, 256, 1, 1.0f, true}, {256, 128, 1, 0.54f, false}, {128, 128, 2, 0.64f, true},
    {64, 128, 2, 0.425f, false}, {32, 128, 2, 0.35f, false}, {64, 64, 3, 1.0f, true}};
typedef void (*grouped_launcher)(const GroupedArgs &, int act, int64_t grid, hipStream_t);
// One dtype and form to a compiled unit.
template <int DT, int FORM>
grouped_launcher pick_grouped(int variant);
template <int DT>
void launch_column_sum(const GroupedArgs &a, hipStream_t s);

}  // namespace fl
