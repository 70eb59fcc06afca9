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
    int stream;              // nonzero: rows of the outputs in the dtype (and of Y, X) start on 128-byte lines
    int parts;               // K is summed in 4, 8 or 16 parts by different workgroups (1: whole)
    float *part;             // parts > 1: fp32 sums, (parts, S, N) or, gradient, (parts, E*K, N)
    int max_tiles;           // limit on the tiles found from the offsets
};

// Expert e's rows, limited to [0, S] whatever the array holds.
__device__ __forceinline__ int run_bound(const GroupedArgs &a, int e) {
    const int v = a.offsets[e];
    return v < 0 ? 0 : v > a.S ? a.S : v;
}

// Row tiles of a run of `rows` rows (which may be next to 2^31, so nothing is
// added to them).
__device__ __forceinline__ int row_tiles(int rows, int bm) { return rows > 0 ? (rows - 1) / bm + 1 : 0; }

struct RunTile {
    int e;       // expert, -1 past the last tile
    int lo, hi;  // its rows
    int m;       // tile within the run
};

// Row tiles of all experts: the runs cut into tiles of bm rows (each run from
// its own start).
__device__ __forceinline__ int count_run_tiles(const GroupedArgs &a, int bm) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e = lane; e < a.E; e += 64) {
        const int lo = run_bound(a, e), hi = run_bound(a, e + 1);
        n += row_tiles(hi - lo, bm);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
    return __builtin_amdgcn_readfirstlane(n);
}

// Row tile `tile` of the experts' runs cut into tiles of bm rows (each run
// from its own start): every wave scans the runs 64 at a time.
__device__ __forceinline__ RunTile find_run_tile(const GroupedArgs &a, int bm, int tile) {
    const int lane = threadIdx.x & 63;
    RunTile t{-1, 0, 0, 0};
    int base = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        const int lo = e < a.E ? run_bound(a, e) : 0, hi = e < a.E ? run_bound(a, e + 1) : 0;
        const int n = row_tiles(hi - lo, bm);
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
    return t;
}

// ----------------------------------------------------- the bias gradient

// dbias[e] = the sum of expert e's rows of G: a block sums 128 columns of one
// expert in 64 groups of rows (group g: rows g, g+64, ..), then adds the groups
// in order.  A pass over G of its own: 1/K of the operations of dW.  Many rows
// in flight per block, because few columns make few blocks.
constexpr int kColumns = 128, kRowGroups = 64;
typedef uint32_t u32x4_unaligned __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
__global__ void __launch_bounds__(1024) grouped_column_sum_kernel(GroupedArgs a) {
    using io = Io<DT>;
    using raw = typename io::raw;
    // a thread's 8 columns, in 16-byte loads (which may be unaligned); at the
    // end of a row it loads the row's last 8 and keeps its own
    constexpr int PER = 8;
    __shared__ float part[kRowGroups][kColumns];
    const int e = blockIdx.y, c0 = blockIdx.x * kColumns;
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
        for (int64_t r = (int64_t)lo + g; r < hi; r += kRowGroups) {
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
        for (int64_t r = (int64_t)lo + g; r < hi; r += kRowGroups)
            for (int t = 0; t < PER; ++t)
                if (at + t >= 0) sum[t] += io::to_f32(G[r * a.N + at + t]);
    }
#pragma unroll
    for (int t = 0; t < PER; ++t)
        if (at + t >= c) part[g][at + t - c0] = sum[t];
    __syncthreads();
    constexpr int SEGS = 1024 / kColumns;
    const int col = threadIdx.x % kColumns, seg = threadIdx.x / kColumns;
    float s = 0.0f;
    if (c0 + col < a.N) {
#pragma unroll
        for (int i = 0; i < kRowGroups / SEGS; ++i) s += part[seg * (kRowGroups / SEGS) + i][col];
        part[seg * (kRowGroups / SEGS)][col] = s;
    }
    __syncthreads();
    if (seg == 0 && c0 + col < a.N) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < SEGS; ++i) s += part[i * (kRowGroups / SEGS)][col];
        a.dbias[(int64_t)e * a.N + c0 + col] = s;
    }
}

// ------------------------------------------------------ joining parts of K

// Adds the parts' sums in order and ends as the tiles' epilogue does.  Forward:
// a block takes 1024 columns of one row; gradient: of one row of dW.  Four parts
// are loaded at a time (one after the other, 16 parts took 16 round trips to
// memory: 25 against 16 us for 2 rows of 1024).
template <int DT, int FORM>
__global__ void __launch_bounds__(256) grouped_join_kernel(GroupedArgs a, int act) {
    using io = Io<DT>;
    using raw = typename io::raw;
    const int64_t r = blockIdx.x, rows = gridDim.x;
    int e = -1;
    if constexpr (FORM == kFormFwd) {  // the row's expert, the first whose run has it
        for (int e0 = 0; e0 < a.E && e < 0; e0 += 64) {
            const int x = e0 + (threadIdx.x & 63);
            const uint64_t has = __ballot(x < a.E && r >= run_bound(a, x) && r < run_bound(a, x + 1));
            if (has) e = e0 + __builtin_ctzll(has);
        }
        if (e < 0) return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = blockIdx.y * 1024 + i * 256 + threadIdx.x;
        if (c >= a.N) break;
        const int64_t o = r * a.N + c;
        float d = 0.0f;
        for (int p = 0; p < a.parts; p += 4) {  // (4, 8 or 16 parts)
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = a.part[(p + i) * rows * a.N + o];
            d += v[0];
            d += v[1];
            d += v[2];
            d += v[3];
        }
        if constexpr (FORM == kFormGrad) {
            if (a.dw_f32)
                static_cast<float *>(a.out)[o] = d;
            else
                static_cast<raw *>(a.out)[o] = io::from_f32(d);
        } else {
            const float x =
                d + (a.bias ? io::to_f32(static_cast<const raw *>(a.bias)[(int64_t)e * a.N + c]) : 0.0f);
            const float y = act == FL_ACT_GLU ? io::to_f32(static_cast<const raw *>(a.Y)[o]) : 0.0f;
            const float v = act == FL_ACT_RELU        ? activate<FL_ACT_RELU>(x, y)
                            : act == FL_ACT_GELU_TANH ? activate<FL_ACT_GELU_TANH>(x, y)
                            : act == FL_ACT_GLU       ? activate<FL_ACT_GLU>(x, y)
                                                      : activate<FL_ACT_NONE>(x, y);
            if (a.out2) static_cast<raw *>(a.out2)[o] = io::from_f32(x);
            static_cast<raw *>(a.out)[o] = io::from_f32(v);
        }
    }
}

// The tiles of grouped_dma_kernel (fl_grouped_dma.hpp) and the figures of the model
// that chooses among them (plan_grouped), fitted to measured choices.  At 45 sizes
// from 2 rows to a training step, forward and backward, the chosen tile is within
// 2% of the best one 67 times of 90, within 15% 88 times, and at worst 32% behind
// (300 rows of one 4096x4096 expert).  time: of a round (one workgroup in every
// slot, 256 CUs x per_cu), in units of the widest tile's.  For scale, 16384 rows of
// 8 experts, K 4096, N 14336, forward: 1554, 1922, 1942, 2322 and 7310 us; fp32, 8192
// rows of 8 experts, K 2048, N 4096: 1052 us (131 TFLOP/s) and 1109, but 200 rows of
// 6 experts, K 768, N 1000: 18.9 and 13.4.  128x128 fp32 tiles: 114 to 134 TFLOP/s,
// and half as much where there are few.
struct GroupedTileShape {
    int bm, bn, per_cu;
    float time;
    float stage;   // us of one stage where a CU has one workgroup
    float rate;    // TB/s of weights (few rows of 8 experts of 4096x14336: 0.94 GB, more than the last-level cache)
    bool grad;     // compiled for the gradient too
};
enum GroupedVariant {
    kTile256x256 = 0, kTile256x128, kTile128x128, kTile64x256, kTile32x128, kTileF32, kTileF32x32, kGroupedVariants
};
constexpr GroupedTileShape kGroupedTiles[kGroupedVariants] = {
    {256, 256, 1, 1.0f, 1.9f, 4.4f, true}, {256, 128, 1, 0.565f, 0.95f, 5.0f, false},
    {128, 128, 2, 0.64f, 0.5f, 4.9f, true}, {64, 256, 1, 0.49f, 0.5f, 6.2f, false},
    {32, 128, 2, 0.35f, 0.23f, 6.0f, false}, {64, 64, 3, 1.0f, 0.58f, 0.0f, true},
    {32, 64, 4, 0.8f, 0.3f, 0.0f, false}};
typedef void (*grouped_launcher)(const GroupedArgs &, int act, int64_t grid, hipStream_t);
// One dtype and form to a compiled unit.  nt: the weights pass the L2 by (tiles of
// at most 64 rows only).
template <int DT, int FORM>
grouped_launcher pick_grouped(int variant, bool nt);
template <int DT>
void launch_column_sum(const GroupedArgs &a, hipStream_t s);
template <int DT, int FORM>
void launch_join(const GroupedArgs &a, int act, hipStream_t s);

}  // namespace fl
