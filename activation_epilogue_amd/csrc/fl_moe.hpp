// fl_moe.hpp -- gfx950 device code of the router, the plan and the movement
// of rows between token order and expert order.
#pragma once

#include "fl_kernels.hpp"

namespace fl {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 64;

template <int DT>
__device__ __forceinline__ float load_f32(const void *p, int64_t i) {
    return Io<DT>::to_f32(static_cast<const typename Io<DT>::raw *>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_f32(void *p, int64_t i, float v) {
    static_cast<typename Io<DT>::raw *>(p)[i] = Io<DT>::from_f32(v);
}

// Sums and maxima over the 64 lanes, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o));
    return v;
}

// ------------------------------------------------------------------ router

struct RouteArgs {
    const void *logits;
    const float *bias;  // or null
    int32_t *experts;
    float *weights;
    const float *dweights;  // backward
    void *dlogits;          // backward
    int T, E, k;
    int groups, top_groups, group_top;
    int sigmoid, raw;
    float scale;
};

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + expf(-x)); }
// log of the sigmoid, without overflow at either end
__device__ __forceinline__ float log_sigmoid(float x) {
    return __builtin_fminf(x, 0.0f) - log1pf(expf(-__builtin_fabsf(x)));
}
// x - m where m is the largest logit: 0 at the largest even if it is infinite
template <class F>
__device__ __forceinline__ F below(F x, F m) {
    return x == m ? F(0) : x - m;
}

// The largest key of the wave, ties to the lowest expert; e < 0 where no
// lane has one left.
__device__ __forceinline__ void wave_best(double &key, int &e) {
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const double k2 = __shfl_xor(key, o);
        const int e2 = __shfl_xor(e, o);
        const bool take = e2 >= 0 && (e < 0 || k2 > key || (k2 == key && e2 < e));
        key = take ? k2 : key;
        e = take ? e2 : e;
    }
}

// One wave per token; expert e = lane + 64*i sits in register i of its lane.
// Keys and scores that decide a choice are 64-bit; the weights are 32-bit.
template <int DT, int EPL>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
    __shared__ double gkeys[4][EPL > 1 ? EPL * 64 : 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double *gk = gkeys[wave];
    for (int64_t t0 = (int64_t)blockIdx.x * 4; t0 < a.T; t0 += (int64_t)gridDim.x * 4) {
        const int64_t t = t0 + wave;
        const bool on = t < a.T;
        float x[EPL];
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            x[i] = on && e < a.E ? load_f32<DT>(a.logits, t * a.E + e) : kNegInf;
            if (!(x[i] > kNegInf)) x[i] = kNegInf;  // NaN counts as masked
            m = __builtin_fmaxf(m, x[i]);
        }
        m = wave_max(m);
        const bool sums = a.groups > 1 && a.group_top == 2;
        double key[EPL], score[EPL];
        if (a.bias || sums) {
            double z = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const double xd = x[i];
                score[i] = a.sigmoid ? 1.0 / (1.0 + exp(-xd)) : x[i] > kNegInf ? exp(below(xd, (double)m)) : 0.0;
                z += score[i];
            }
            if (!a.sigmoid) {
                z = wave_sum(z);
#pragma unroll
                for (int i = 0; i < EPL; ++i) score[i] /= z;
            }
        }
        bool live[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            key[i] = a.bias ? score[i] + (double)(e < a.E ? a.bias[e] : 0.0f) : (double)x[i];
            live[i] = x[i] > kNegInf && key[i] > (double)kNegInf;  // (a NaN key fails)
        }
        if (a.groups > 1) {
            // lane g scores run g from the keys of its experts
            const int per = a.E / a.groups;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (lane + 64 * i < a.E)
                    gk[lane + 64 * i] = live[i] ? (sums && !a.bias ? score[i] : key[i]) : (double)kNegInf;
            __syncthreads();
            double gs = 0.0;
            int g = -1;
            if (lane < a.groups) {
                double b1 = kNegInf, b2 = kNegInf;
                for (int j = 0; j < per; ++j) {
                    const double v = gk[lane * per + j];
                    if (v > b1) {
                        b2 = b1;
                        b1 = v;
                    } else if (v > b2) {
                        b2 = v;
                    }
                }
                gs = a.group_top == 2 && b2 > (double)kNegInf ? b1 + b2 : b1;
                g = b1 > (double)kNegInf ? lane : -1;
            }
            uint64_t kept = 0;
            for (int j = 0; j < a.top_groups; ++j) {
                double bk = gs;
                int bg = (kept >> lane) & 1 ? -1 : g;
                wave_best(bk, bg);
                if (bg < 0) break;
                kept |= 1ull << bg;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                live[i] = live[i] && ((kept >> ((lane + 64 * i) / per)) & 1);
            __syncthreads();
        }
        // choice j ends up in lane j
        int sel = -1;
        for (int j = 0; j < a.k; ++j) {
            double bk = 0.0;
            int be = -1;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (live[i] && (be < 0 || key[i] > bk)) {
                    bk = key[i];
                    be = lane + 64 * i;
                }
            wave_best(bk, be);
            if (be < 0) break;
            if (lane == j) sel = be;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (be == lane + 64 * i) live[i] = false;
        }
        float xs = kNegInf;  // the chosen expert's logit
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float v = __shfl(x[i], sel & 63);
            if (sel >= 0 && (sel >> 6) == i) xs = v;
        }
        float w;
        if (!a.raw) {
            // s_i / sum s = softmax of the chosen experts' log scores: no
            // quotient of two underflowed numbers
            const float l = sel < 0 ? kNegInf : a.sigmoid ? log_sigmoid(xs) : xs;
            const float lm = wave_max(l);
            const float p = sel < 0 ? 0.0f : expf(below(l, lm));
            w = p / wave_sum(p);
        } else if (a.sigmoid) {
            w = sigmoid_f32(xs);
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) z += x[i] > kNegInf ? expf(below(x[i], m)) : 0.0f;
            z = wave_sum(z);
            w = expf(below(xs, m)) / z;
        }
        if (on && lane < a.k) {
            a.experts[t * a.k + lane] = sel;
            a.weights[t * a.k + lane] = sel < 0 ? 0.0f : w * a.scale;
        }
    }
}

// The logits' gradient, one wave per token.  Renormalised weights are a
// softmax over the chosen experts alone, w = scale * p: dl_i = p_i (dw_i -
// sum dw p) scale (times 1 - s_i for the sigmoid), and 0 for the others; raw
// softmax weights take the whole row: dl_j = s_j (ds_j - sum_i s_i ds_i).
template <int DT, int EPL>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
        float x[EPL], d[EPL];
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            x[i] = e < a.E ? load_f32<DT>(a.logits, t * a.E + e) : kNegInf;
            if (!(x[i] > kNegInf)) x[i] = kNegInf;
            m = __builtin_fmaxf(m, x[i]);
            d[i] = 0.0f;
        }
        int sel = lane < a.k ? a.experts[t * a.k + lane] : -1;
        float dw = lane < a.k ? a.dweights[t * a.k + lane] * a.scale : 0.0f;
        float xs = kNegInf;
        const int at = sel >= 0 && sel < a.E ? sel : 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float v = __shfl(x[i], at & 63);
            if ((at >> 6) == i) xs = v;
        }
        if (sel < 0 || sel >= a.E || !(xs > kNegInf)) {
            sel = -1;
            dw = 0.0f;
        }
        float ds;  // this lane's choice: the gradient of its score, or of its log score
        if (!a.raw) {
            const float l = sel < 0 ? kNegInf : a.sigmoid ? log_sigmoid(xs) : xs;
            const float lm = wave_max(l);
            const float p = sel < 0 ? 0.0f : expf(below(l, lm));
            const float z = wave_sum(p);
            const float w = sel < 0 ? 0.0f : p / z;
            ds = w * (dw - wave_sum(dw * w));
            if (a.sigmoid) ds *= sigmoid_f32(-xs);
        } else if (a.sigmoid) {
            ds = dw * sigmoid_f32(xs) * sigmoid_f32(-xs);
        } else {
            ds = dw;
        }
        if (sel < 0) ds = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int e = __shfl(sel, j);
            const float v = __shfl(ds, j);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e == lane + 64 * i) d[i] += v;
        }
        if (a.raw && !a.sigmoid) {
            m = wave_max(m);
            float z = 0.0f, s[EPL], c = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = x[i] > kNegInf ? expf(below(x[i], m)) : 0.0f;
                z += s[i];
            }
            z = wave_sum(z);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = s[i] > 0.0f ? s[i] / z : 0.0f;
                c += s[i] * d[i];
            }
            c = wave_sum(c);
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] = s[i] * (d[i] - c);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E) store_f32<DT>(a.dlogits, t * a.E + e, d[i]);
        }
    }
}

// -------------------------------------------------------------------- plan

// A stable counting sort of the slots by expert.  Block b owns the kPlanChunk
// slots from b*kPlanChunk, wave w of it a run of kPlanRun of them.
constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanChunk = 4096;
constexpr int kPlanRun = kPlanChunk / kPlanWaves;

struct PlanArgs {
    const int32_t *experts;
    int32_t *offsets, *token_of_row, *row_of_slot;
    int32_t *counts;  // (blocks, E), null for one block
    int64_t S;
    int k, E;
};

__device__ __forceinline__ int slot_expert(const PlanArgs &a, int64_t s) {
    const int e = s < a.S ? a.experts[s] : -1;
    return e >= 0 && e < a.E ? e : -1;
}

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(PlanArgs a) {
    __shared__ int cnt[kMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * kPlanChunk;
    for (int i = threadIdx.x; i < kPlanChunk; i += kPlanThreads) {
        const int e = slot_expert(a, s0 + i);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = cnt[e];
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
    __shared__ int run[kPlanWaves][kMaxExperts];  // counts of a wave's run, then its next row of every expert
    __shared__ int first[kMaxExperts + 1];        // first row of every expert
    __shared__ int before[kMaxExperts];           // this block's first row within the expert
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t s0 = (int64_t)blockIdx.x * kPlanChunk + wave * kPlanRun;
    for (int e = lane; e < a.E; e += 64) run[wave][e] = 0;
    __syncthreads();
    for (int i = lane; i < kPlanRun; i += 64) {
        const int e = slot_expert(a, s0 + i);
        if (e >= 0) atomicAdd(&run[wave][e], 1);
    }
    __syncthreads();
    // every expert's rows in earlier blocks, and in all of them
    for (int e = tid; e < a.E; e += kPlanThreads) {
        int all = 0, prev = 0;
        if (a.counts) {
            for (int b = 0; b < (int)gridDim.x; ++b) {
                const int c = a.counts[(int64_t)b * a.E + e];
                if (b < (int)blockIdx.x) prev += c;
                all += c;
            }
        } else {
            for (int w = 0; w < kPlanWaves; ++w) all += run[w][e];
        }
        before[e] = prev;
        first[e] = all;
    }
    __syncthreads();
    if (wave == 0) {
        int base = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const int e = e0 + lane;
            const int c = e < a.E ? first[e] : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o);
                if (lane >= o) incl += v;
            }
            if (e < a.E) first[e] = base + incl - c;
            base += __shfl(incl, 63);
        }
        if (lane == 0) first[a.E] = base;
    }
    __syncthreads();
    const int total = first[a.E];
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.E; e += kPlanThreads) a.offsets[e] = first[e];
    for (int e = tid; e < a.E; e += kPlanThreads) {
        int at = first[e] + before[e];
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = run[w][e];
            run[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    volatile int *next = run[wave];
    for (int i = 0; i < kPlanRun; i += 64) {
        const int64_t s = s0 + i + lane;
        if (s0 + i >= a.S) break;
        const int e = slot_expert(a, s);
        // the lanes of this step with the same expert
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; (1 << b) < a.E; ++b) {
            const uint64_t m = __ballot((e >> b) & 1);
            same &= ((e >> b) & 1) ? m : ~m;
        }
        int row = -1;
        const uint64_t lower = same & ((1ull << lane) - 1);
        if (e >= 0) row = next[e] + __popcll(lower);
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && lower == 0) next[e] = row + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (s < a.S) a.row_of_slot[s] = row;
        if (row >= 0) a.token_of_row[row] = (int32_t)(s / a.k);
    }
    // rows past the last expert's
    for (int i = tid; i < kPlanChunk; i += kPlanThreads) {
        const int64_t r = (int64_t)blockIdx.x * kPlanChunk + i;
        if (r >= total && r < a.S) a.token_of_row[r] = -1;
    }
}

// ---------------------------------------------------------------- movement

// VEC elements of a row at a time: 16 bytes where rows start on 16-byte
// boundaries, else one element.
template <int DT, bool VECTOR>
struct Piece {
    using io = Io<DT>;
    using raw = typename io::raw;
    static constexpr int VEC = VECTOR ? 16 / io::size : 1;
    raw v[VEC];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const raw *q = static_cast<const raw *>(p) + i;
        if constexpr (VECTOR) {
            const u32x4_t w = *reinterpret_cast<const u32x4_t *>(q);
            __builtin_memcpy(v, &w, 16);
        } else {
            v[0] = *q;
        }
    }
    __device__ __forceinline__ void store(void *p, int64_t i) const {
        raw *q = static_cast<raw *>(p) + i;
        if constexpr (VECTOR) {
            u32x4_t w;
            __builtin_memcpy(&w, v, 16);
            *reinterpret_cast<u32x4_t *>(q) = w;
        } else {
            *q = v[0];
        }
    }
    __device__ __forceinline__ float get(int t) const { return io::to_f32(v[t]); }
    __device__ __forceinline__ void set(int t, float f) { v[t] = io::from_f32(f); }
};

struct MoveArgs {
    const void *src, *src2;
    const int32_t *map;
    const float *weights;
    void *dst;
    float *dweights;
    int64_t T, S, H;
    int k;
};

template <int DT, bool VECTOR>
__global__ void __launch_bounds__(256) gather_kernel(MoveArgs a) {
    using P = Piece<DT, VECTOR>;
    const int64_t pieces = a.H / P::VEC;
    for (int64_t r = blockIdx.x; r < a.S; r += gridDim.x) {
        const int64_t t = a.map[r];
        const bool on = t >= 0 && t < a.T;
        for (int64_t c = threadIdx.x; c < pieces; c += 256) {
            P p{};
            if (on) p.load(a.src, t * a.H + c * P::VEC);
            p.store(a.dst, r * a.H + c * P::VEC);
        }
    }
}

// src: rows; src2: the residual or null.
template <int DT, bool VECTOR>
__global__ void __launch_bounds__(256) combine_kernel(MoveArgs a) {
    using P = Piece<DT, VECTOR>;
    const int64_t pieces = a.H / P::VEC;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int64_t c = threadIdx.x + (int64_t)blockIdx.y * 256; c < pieces; c += (int64_t)gridDim.y * 256) {
            float acc[P::VEC];
#pragma unroll
            for (int e = 0; e < P::VEC; ++e) acc[e] = 0.0f;
            for (int j = 0; j < a.k; ++j) {
                const int64_t r = a.map[t * a.k + j];
                if (r < 0 || r >= a.S) continue;
                const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
                P p;
                p.load(a.src, r * a.H + c * P::VEC);
#pragma unroll
                for (int e = 0; e < P::VEC; ++e) acc[e] = __builtin_fmaf(w, p.get(e), acc[e]);
            }
            P o;
            if (a.src2) {
                o.load(a.src2, t * a.H + c * P::VEC);
#pragma unroll
                for (int e = 0; e < P::VEC; ++e) acc[e] += o.get(e);
            }
#pragma unroll
            for (int e = 0; e < P::VEC; ++e) o.set(e, acc[e]);
            o.store(a.dst, t * a.H + c * P::VEC);
        }
    }
}

// src: dout; src2: rows (read for dweights); dst: drows or null.  drows may be
// rows: a row's piece is read before it is written, by the same thread.
template <int DT, bool VECTOR>
__global__ void __launch_bounds__(256) combine_bwd_kernel(MoveArgs a) {
    using P = Piece<DT, VECTOR>;
    __shared__ float part[4];
    const int64_t pieces = a.H / P::VEC;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t s = blockIdx.x; s < a.T * a.k; s += gridDim.x) {
        const int64_t t = s / a.k, r = a.map[s];
        const bool on = r >= 0 && r < a.S;
        const float w = a.weights ? a.weights[s] : 1.0f;
        float dot = 0.0f;
        if (on) {
            for (int64_t c = threadIdx.x; c < pieces; c += 256) {
                P d, y;
                d.load(a.src, t * a.H + c * P::VEC);
                if (a.dweights) {
                    y.load(a.src2, r * a.H + c * P::VEC);
#pragma unroll
                    for (int e = 0; e < P::VEC; ++e) dot = __builtin_fmaf(d.get(e), y.get(e), dot);
                }
                if (a.dst) {
#pragma unroll
                    for (int e = 0; e < P::VEC; ++e) d.set(e, w * d.get(e));
                    d.store(a.dst, r * a.H + c * P::VEC);
                }
            }
        }
        if (a.dweights) {
            dot = wave_sum(dot);
            __syncthreads();
            if (lane == 0) part[wave] = dot;
            __syncthreads();
            if (threadIdx.x == 0) a.dweights[s] = part[0] + part[1] + part[2] + part[3];
        }
    }
}

}  // namespace fl
