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

// Sums and extremes over a team of 16 or 64 lanes, the same in every lane of
// it: moves between neighbouring lanes on the vector unit (an LDS permute costs
// ten times the latency, and a router is a chain of such steps).
template <int CTRL, int ROWS = 0xf, class V>
__device__ __forceinline__ V lane_move(V old, V v) {
    typedef int words __attribute__((ext_vector_type(sizeof(V) / 4)));
    words o, w, r;
    __builtin_memcpy(&o, &old, sizeof(V));
    __builtin_memcpy(&w, &v, sizeof(V));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(V) / 4); ++i)
        r[i] = __builtin_amdgcn_update_dpp(o[i], w[i], CTRL, ROWS, 0xf, false);
    V out;
    __builtin_memcpy(&out, &r, sizeof(V));
    return out;
}
template <class V>
__device__ __forceinline__ V read_lane(V v, int lane) {
    typedef int words __attribute__((ext_vector_type(sizeof(V) / 4)));
    words w;
    __builtin_memcpy(&w, &v, sizeof(V));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(V) / 4); ++i) w[i] = __builtin_amdgcn_readlane(w[i], lane);
    V out;
    __builtin_memcpy(&out, &w, sizeof(V));
    return out;
}
struct Add {
    template <class V> __device__ static V zero(V) { return V(0); }
    __device__ static float of(float a, float b) { return a + b; }
    __device__ static double of(double a, double b) { return a + b; }
};
struct Larger {  // `zero`: what a lane without a source takes, itself
    template <class V> __device__ static V zero(V v) { return v; }
    __device__ static float of(float a, float b) { return __builtin_fmaxf(a, b); }
    __device__ static double of(double a, double b) { return __builtin_fmax(a, b); }
};
struct Lower {
    template <class V> __device__ static V zero(V v) { return v; }
    __device__ static int of(int a, int b) { return a < b ? a : b; }
};
template <class OP, int TEAM, class V>
__device__ __forceinline__ V team_reduce(V v) {
    static_assert(TEAM == 16 || TEAM == 64, "a row of lanes or a wave");
    if constexpr (TEAM == 16) {
        // lanes 1 and 2 apart, then mirrored halves and rows: every lane adds
        // the same pairs (a rotation would not, and its lanes' sums differ)
        v = OP::of(v, lane_move<0xb1>(v, v));
        v = OP::of(v, lane_move<0x4e>(v, v));
        v = OP::of(v, lane_move<0x141>(v, v));
        return OP::of(v, lane_move<0x140>(v, v));
    } else {  // shifts of the row by 1, 2, 4, 8: its lane 15 holds the row's; then broadcasts of lanes 15 and 31
        v = OP::of(v, lane_move<0x111>(OP::zero(v), v));
        v = OP::of(v, lane_move<0x112>(OP::zero(v), v));
        v = OP::of(v, lane_move<0x114>(OP::zero(v), v));
        v = OP::of(v, lane_move<0x118>(OP::zero(v), v));
        v = OP::of(v, lane_move<0x142, 0xa>(OP::zero(v), v));
        v = OP::of(v, lane_move<0x143, 0xc>(OP::zero(v), v));
        return read_lane(v, 63);
    }
}
template <int TEAM, class V>
__device__ __forceinline__ V team_sum(V v) { return team_reduce<Add, TEAM>(v); }
template <int TEAM, class V>
__device__ __forceinline__ V team_max(V v) { return team_reduce<Larger, TEAM>(v); }
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }

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

// The token's logits, masked ones -inf (NaN counts as masked), and the largest.
// All loads go out together, from clamped addresses: none waits behind a branch.
template <int DT, int EPL, int TEAM>
__device__ __forceinline__ float load_logits(const RouteArgs &a, int64_t t, int lane, float (&x)[EPL]) {
    const int64_t row = (t < a.T ? t : a.T - 1) * a.E;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + TEAM * i;
        x[i] = load_f32<DT>(a.logits, row + (e < a.E ? e : 0));
    }
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const bool is = t < a.T && lane + TEAM * i < a.E && x[i] > kNegInf;
        x[i] = is ? x[i] : kNegInf;
        m = __builtin_fmaxf(m, x[i]);
    }
    return team_max<TEAM>(m);
}

// The k largest keys (-inf: not to be chosen), ties to the lowest expert:
// choice j ends up in lane j of the team, -1 where no key is left.
template <int EPL, int TEAM, class F>
__device__ __forceinline__ int choose(F (&key)[EPL], int k, int lane) {
    constexpr int NONE = 0x7fffffff;
    int sel = -1;
    for (int j = 0; j < k; ++j) {
        F b = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) b = larger(b, key[i]);
        b = team_max<TEAM>(b);
        int e = NONE;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) e = key[i] == b ? lane + TEAM * i : e;
        e = team_reduce<Lower, TEAM>(e);
        if (lane == j && b > F(kNegInf)) sel = e;
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = e == lane + TEAM * i ? F(kNegInf) : key[i];
    }
    return sel;
}

// A token's choice.  With neither a bias nor sums over a run the logits are
// the keys, as they are (F fp32); else scores and keys are computed in 64 bits,
// since a choice between two experts hangs on differences that fp32 scores do
// not resolve.  (fp32 keys, and 64-bit ones where a margin left the choice
// open, took as long or longer: some wave of a launch always needs both.)
template <int EPL, int TEAM, class F>
__device__ __forceinline__ int pick(const RouteArgs &a, const float (&x)[EPL],
                                    const float (&bias)[EPL], float m, int per, int lane, F *gk) {
    constexpr bool WIDE = sizeof(F) == 8;
    const bool sums = WIDE && a.groups > 1 && a.group_top == 2;
    F key[EPL], score[EPL];
    if constexpr (WIDE) {
        F z = F(0);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const F v = x[i];
            score[i] = x[i] > kNegInf ? (a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(below(v, F(m)))) : 0.0;
            z += score[i];
        }
        if (!a.sigmoid) {
            z = team_sum<TEAM>(z);
#pragma unroll
            for (int i = 0; i < EPL; ++i) score[i] /= z;
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        F v = F(x[i]);
        if (WIDE && a.bias) v = score[i] + F(bias[i]);
        key[i] = x[i] > kNegInf && v > F(kNegInf) ? v : F(kNegInf);  // (a NaN key is no key)
    }
    if (a.groups > 1) {
        // TEAM / 2^ceil(log2 groups) lanes find the largest two keys of a run together
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            gk[lane + TEAM * i] = sums && !a.bias && key[i] > F(kNegInf) ? score[i] : key[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        int share = TEAM;
        while (TEAM / share < a.groups) share >>= 1;
        const int g = lane / share;
        F b1 = F(kNegInf), b2 = F(kNegInf);
        if (g < a.groups)
            for (int j = lane % share; j < per; j += share) {
                const F v = gk[g * per + j];
                b2 = larger(b2, v < b1 ? v : b1);
                b1 = larger(b1, v);
            }
        for (int o = 1; o < share; o <<= 1) {
            const F o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
            b2 = larger(larger(b2, o2), b1 < o1 ? b1 : o1);
            b1 = larger(b1, o1);
        }
        F gs = a.group_top == 2 && b2 > F(kNegInf) ? b1 + b2 : b1;
        uint64_t kept = 0;
        for (int j = 0; j < a.top_groups; ++j) {
            const F b = team_max<TEAM>(gs);
            const int best = team_reduce<Lower, TEAM>(gs == b ? g : 63);
            if (b > F(kNegInf)) kept |= 1ull << best;
            if (g == best) gs = F(kNegInf);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + TEAM * i;
            if (e < a.E && !((kept >> (e / per)) & 1)) key[i] = F(kNegInf);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    return choose<EPL, TEAM>(key, a.k, lane);
}

// A team of lanes per token (16: four tokens to a wave, the same steps for all
// of them); expert e = lane + TEAM*i sits in register i of its lane.  Bound by
// the issue of the k rounds of `choose`, for few tokens by their latency.
// Teams of 16 against whole waves: 16384 tokens of 64 experts, k 6: 5.7 and
// 13.5 us; 256 experts in 8 runs, sigmoid, bias: 16384 tokens 34 and 42 us, 4096
// tokens 14 both, 32 tokens 12.5 and 7.7.
template <int DT, int EPL, int TEAM>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
    constexpr int TOKENS = 256 / TEAM;
    __shared__ double gkeys[TOKENS][EPL * TEAM];
    const int lane = threadIdx.x % TEAM, slot = threadIdx.x / TEAM;
    const int per = a.E / a.groups;
    float bias[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + TEAM * i;
        bias[i] = a.bias ? a.bias[e < a.E ? e : 0] : 0.0f;
    }
    // (waves run together to the last token: no lane leaves its wave)
    for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.T; t0 += (int64_t)gridDim.x * TOKENS) {
        const int64_t t = t0 + slot;
        const bool on = t < a.T;
        float x[EPL];
        const float m = load_logits<DT, EPL, TEAM>(a, t, lane, x);
        const int sel =
            a.bias || (a.groups > 1 && a.group_top == 2)
                ? pick<EPL, TEAM>(a, x, bias, m, per, lane, gkeys[slot])
                : pick<EPL, TEAM>(a, x, bias, m, per, lane, reinterpret_cast<float *>(gkeys[slot]));
        const float xs = sel >= 0 ? load_f32<DT>(a.logits, t * a.E + sel) : kNegInf;
        float w;
        if (!a.raw) {
            // s_i / sum s = softmax of the chosen experts' log scores: no
            // quotient of two underflowed numbers
            const float l = sel < 0 ? kNegInf : a.sigmoid ? log_sigmoid(xs) : xs;
            const float lm = team_max<TEAM>(l);
            const float p = sel < 0 ? 0.0f : expf(below(l, lm));
            w = p / team_sum<TEAM>(p);
        } else if (a.sigmoid) {
            w = sigmoid_f32(xs);
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) z += x[i] > kNegInf ? expf(below(x[i], m)) : 0.0f;
            z = team_sum<TEAM>(z);
            w = expf(below(xs, m)) / z;
        }
        if (on && lane < a.k) {
            a.experts[t * a.k + lane] = sel;
            a.weights[t * a.k + lane] = sel < 0 ? 0.0f : w * a.scale;
        }
    }
}

// The logits' gradient, a team of lanes per token.  Renormalised weights are a
// softmax over the chosen experts alone, w = scale * p: dl_i = p_i (dw_i -
// sum dw p) scale (times 1 - s_i for the sigmoid), and 0 for the others; raw
// softmax weights take the whole row: dl_j = s_j (ds_j - sum_i s_i ds_i).
// 16384 tokens of 64 experts: 3.9 us, 2.1 MB written, most of it the launch.
template <int DT, int EPL, int TEAM>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteArgs a) {
    constexpr int TOKENS = 256 / TEAM;
    const int lane = threadIdx.x % TEAM, slot = threadIdx.x / TEAM;
    for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < a.T; t0 += (int64_t)gridDim.x * TOKENS) {
        const int64_t t = t0 + slot;
        const bool on = t < a.T;
        const bool whole = a.raw && !a.sigmoid;
        int sel = on && lane < a.k ? a.experts[t * a.k + lane] : -1;
        float dw = on && lane < a.k ? a.dweights[t * a.k + lane] * a.scale : 0.0f;
        float xs = sel >= 0 && sel < a.E ? load_f32<DT>(a.logits, t * a.E + sel) : kNegInf;
        if (!(xs > kNegInf)) {
            sel = -1;
            dw = 0.0f;
        }
        float ds;  // this lane's choice: the gradient of its score, or of its log score
        if (!a.raw) {
            const float l = sel < 0 ? kNegInf : a.sigmoid ? log_sigmoid(xs) : xs;
            const float lm = team_max<TEAM>(l);
            const float p = sel < 0 ? 0.0f : expf(below(l, lm));
            const float z = team_sum<TEAM>(p);
            const float w = sel < 0 ? 0.0f : p / z;
            ds = w * (dw - team_sum<TEAM>(dw * w));
            if (a.sigmoid) ds *= sigmoid_f32(-xs);
        } else if (a.sigmoid) {
            ds = dw * sigmoid_f32(xs) * sigmoid_f32(-xs);
        } else {
            ds = dw;
        }
        if (sel < 0) ds = 0.0f;
        float d[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int e = __shfl(sel, j, TEAM);
            const float v = __shfl(ds, j, TEAM);
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] += e == lane + TEAM * i ? v : 0.0f;
        }
        if (whole) {
            float z = 0.0f, s[EPL], c = 0.0f;
            const float m = load_logits<DT, EPL, TEAM>(a, t, lane, s);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = s[i] > kNegInf ? expf(below(s[i], m)) : 0.0f;
                z += s[i];
            }
            z = team_sum<TEAM>(z);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = s[i] > 0.0f ? s[i] / z : 0.0f;
                c += s[i] * d[i];
            }
            c = team_sum<TEAM>(c);
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] = s[i] * (d[i] - c);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + TEAM * i;
            if (on && e < a.E) store_f32<DT>(a.dlogits, t * a.E + e, d[i]);
        }
    }
}

// -------------------------------------------------------------------- plan

// A stable counting sort of the slots by expert.  A block owns CHUNK slots, a
// wave of it a run of kPlanRun of them, kept in registers between counting and
// placing.  Up to kPlanSmall slots one block of 4 waves does it all (the fewest
// steps from launch to end); above, blocks of 16 waves, and where there are
// several, a launch before them counts every block's slots.  Bound by the
// latency of its phases: 192 slots 4.0 us, 524288 slots of 256 experts 3 + 10 us
// (6.3 MB).
// Up to kPlanDirect blocks each adds the counts of all of them by itself, which
// saves a launch but grows with their square; above, a launch between sums them
// (256 experts, all launches: 256 blocks 18.5 us each adding and 19.2 summed, 512
// blocks 36 and 30, 2048 blocks 277 and 91; 1024 experts: 2048 blocks 893 and
// 141; 2^28 slots of 256 experts 3.3 ms).
constexpr int kPlanRun = 256;
constexpr int kPlanSmall = 4 * kPlanRun, kPlanChunk = 16 * kPlanRun;
constexpr int kPlanDirect = 256;

struct PlanArgs {
    const int32_t *experts;
    int32_t *offsets, *token_of_row, *row_of_slot;
    int32_t *counts;  // (blocks, E), null for one block
    int64_t S;
    int k, E;
    int summed;       // counts hold the rows before each block instead, and a line of totals
};

__device__ __forceinline__ int slot_expert(const PlanArgs &a, int64_t s) {
    const int e = s < a.S ? a.experts[s] : -1;
    return e >= 0 && e < a.E ? e : -1;
}

__global__ void __launch_bounds__(1024) plan_count_kernel(PlanArgs a) {
    __shared__ int cnt[kMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += 1024) cnt[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * kPlanChunk;
#pragma unroll
    for (int i = 0; i < kPlanChunk / 1024; ++i) {
        const int e = slot_expert(a, s0 + threadIdx.x + i * 1024);
        if (e >= 0) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 1024) a.counts[(int64_t)blockIdx.x * a.E + e] = cnt[e];
}

// Turns counts, (blocks, E), into every expert's rows before each block, with
// a line of totals behind them: a block takes `cols` experts (a power of two, at
// most 64), cut into 1024 / cols runs of lines.
__global__ void __launch_bounds__(1024) plan_sum_kernel(PlanArgs a, int blocks, int cols) {
    __shared__ int sums[1024];
    const int x = threadIdx.x % cols, part = threadIdx.x / cols, parts = 1024 / cols;
    const int e = blockIdx.x * cols + x;
    const int per = (blocks + parts - 1) / parts;
    const int b0 = part * per < blocks ? part * per : blocks, b1 = b0 + per < blocks ? b0 + per : blocks;
    int sum = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += a.counts[(int64_t)b * a.E + e];
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (e >= a.E) return;
    int at = 0;
    for (int p = 0; p < part; ++p) at += sums[p * cols + x];
    constexpr int AHEAD = 8;  // lines loaded before they are written over
    for (int b = b0; b < b1; b += AHEAD) {
        int c[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) c[i] = b + i < b1 ? a.counts[(int64_t)(b + i) * a.E + e] : 0;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (b + i < b1) a.counts[(int64_t)(b + i) * a.E + e] = at;
            at += c[i];
        }
    }
    if (part == parts - 1) a.counts[(int64_t)blocks * a.E + e] = at;
}

// EC: an upper limit of E, a power of two.
template <int WAVES, int EC>
__global__ void __launch_bounds__(64 * WAVES) plan_kernel(PlanArgs a) {
    constexpr int THREADS = 64 * WAVES, CHUNK = WAVES * kPlanRun, STEPS = kPlanRun / 64;
    constexpr int PARTS = THREADS > EC ? THREADS / EC : 1;
    __shared__ int run[WAVES][EC];           // counts of a wave's run, then its next row of every expert
    __shared__ int first[EC + 1];            // first row of every expert
    __shared__ int before[EC];               // this block's first row within the expert
    __shared__ int sums[PARTS][EC], prevs[PARTS][EC];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t s0 = (int64_t)blockIdx.x * CHUNK + wave * kPlanRun;
    int ex[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) ex[i] = slot_expert(a, s0 + i * 64 + lane);
    for (int e = lane; e < a.E; e += 64) run[wave][e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (ex[i] >= 0) atomicAdd(&run[wave][ex[i]], 1);
    __syncthreads();
    // every expert's rows in earlier blocks, and in all of them
    if (a.counts && !a.summed) {
        const int part = tid / EC;
        for (int e = tid % EC; e < a.E; e += PARTS == 1 ? THREADS : EC) {
            int all = 0, prev = 0;
#pragma unroll 8
            for (int b = part; b < (int)gridDim.x; b += PARTS) {
                const int c = a.counts[(int64_t)b * a.E + e];
                prev += b < (int)blockIdx.x ? c : 0;
                all += c;
            }
            sums[part][e] = all;
            prevs[part][e] = prev;
        }
        __syncthreads();
    }
    for (int e = tid; e < a.E; e += THREADS) {
        int all = 0, prev = 0;
        if (a.summed) {
            all = a.counts[(int64_t)gridDim.x * a.E + e];
            prev = a.counts[(int64_t)blockIdx.x * a.E + e];
        } else if (a.counts) {
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                all += sums[p][e];
                prev += prevs[p][e];
            }
        } else {
#pragma unroll
            for (int w = 0; w < WAVES; ++w) all += run[w][e];
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
        for (int e = tid; e <= a.E; e += THREADS) a.offsets[e] = first[e];
    for (int e = tid; e < a.E; e += THREADS) {
        int at = first[e] + before[e];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int c = run[w][e];
            run[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    volatile int *next = run[wave];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t s = s0 + i * 64 + lane;
        const int e = ex[i];
        // the lanes of this step with the same expert
        uint64_t same = __ballot(e >= 0);
        if (same) {
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
            if (row >= 0) {
                a.row_of_slot[s] = row;
                a.token_of_row[row] = (int32_t)(s / a.k);
            }
        }
        if (e < 0 && s < a.S) a.row_of_slot[s] = -1;
    }
    // rows past the last expert's
    for (int i = tid; i < CHUNK; i += THREADS) {
        const int64_t r = (int64_t)blockIdx.x * CHUNK + i;
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
    __device__ __forceinline__ void load_nt(const void *p, int64_t i) {
        const raw *q = static_cast<const raw *>(p) + i;
        if constexpr (VECTOR) {
            const u32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(q));
            __builtin_memcpy(v, &w, 16);
        } else {
            v[0] = *q;
        }
    }
    __device__ __forceinline__ void store_nt(void *p, int64_t i) const {
        raw *q = static_cast<raw *>(p) + i;
        if constexpr (VECTOR) {
            u32x4_t w;
            __builtin_memcpy(&w, v, 16);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t *>(q));
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

// COLS lanes to a row, 256 / COLS rows to a block: rows shorter than 256 pieces
// leave no lanes idle.  Rows move once, so they pass the L2 by (nt: 3 to 8%
// faster).  Bound by memory, at 8192x2 rows of 4096 bf16: gather 38 us (5.2
// TB/s), combine 38 (5.2), its gradient 60 (5.6).
template <int DT, bool VECTOR, int COLS>
__global__ void __launch_bounds__(256) gather_kernel(MoveArgs a) {
    using P = Piece<DT, VECTOR>;
    constexpr int ROWS = 256 / COLS;
    const int64_t pieces = a.H / P::VEC;
    const int x = threadIdx.x % COLS, y = threadIdx.x / COLS;
    for (int64_t r = (int64_t)blockIdx.x * ROWS + y; r < a.S; r += (int64_t)gridDim.x * ROWS) {
        const int64_t t = a.map[r];
        const bool on = t >= 0 && t < a.T;
        for (int64_t c = x + (int64_t)blockIdx.y * COLS; c < pieces; c += (int64_t)gridDim.y * COLS) {
            P p{};
            if (on) p.load(a.src, t * a.H + c * P::VEC);
            p.store_nt(a.dst, r * a.H + c * P::VEC);
        }
    }
}

// src: rows; src2: the residual or null.
template <int DT, bool VECTOR, int COLS>
__global__ void __launch_bounds__(256) combine_kernel(MoveArgs a) {
    using P = Piece<DT, VECTOR>;
    constexpr int ROWS = 256 / COLS;
    const int64_t pieces = a.H / P::VEC;
    const int x = threadIdx.x % COLS, y = threadIdx.x / COLS;
    for (int64_t t = (int64_t)blockIdx.x * ROWS + y; t < a.T; t += (int64_t)gridDim.x * ROWS) {
        for (int64_t c = x + (int64_t)blockIdx.y * COLS; c < pieces; c += (int64_t)gridDim.y * COLS) {
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
            o.store_nt(a.dst, t * a.H + c * P::VEC);
        }
    }
}

// src: dout; src2: rows (read for dweights); dst: drows or null.  drows may be
// rows: a row's piece is read before it is written, by the same thread.  COLS
// 64: a wave per slot, which adds its dot product without a barrier.
template <int DT, bool VECTOR, int COLS>
__global__ void __launch_bounds__(256) combine_bwd_kernel(MoveArgs a) {
    using P = Piece<DT, VECTOR>;
    constexpr int SLOTS = 256 / COLS;
    static_assert(COLS == 64 || COLS == 256, "a wave or a block per slot");
    __shared__ float part[4];
    const int64_t pieces = a.H / P::VEC, slots = a.T * a.k;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, x = threadIdx.x % COLS;
    for (int64_t s0 = (int64_t)blockIdx.x * SLOTS; s0 < slots; s0 += (int64_t)gridDim.x * SLOTS) {
        const int64_t s = s0 + threadIdx.x / COLS;
        const int64_t r = s < slots ? a.map[s] : -1, t = s / a.k;
        const bool on = r >= 0 && r < a.S;
        const float w = on && a.weights ? a.weights[s] : 1.0f;
        float dot = 0.0f;
        if (on) {
#pragma unroll 4
            for (int64_t c = x; c < pieces; c += COLS) {
                P d, y;
                d.load(a.src, t * a.H + c * P::VEC);
                if (a.dweights) {
                    y.load_nt(a.src2, r * a.H + c * P::VEC);
#pragma unroll
                    for (int e = 0; e < P::VEC; ++e) dot = __builtin_fmaf(d.get(e), y.get(e), dot);
                }
                if (a.dst) {
#pragma unroll
                    for (int e = 0; e < P::VEC; ++e) d.set(e, w * d.get(e));
                    d.store_nt(a.dst, r * a.H + c * P::VEC);
                }
            }
        }
        if (a.dweights) {
            dot = team_sum<64>(dot);
            if constexpr (COLS == 64) {
                if (lane == 0 && s < slots) a.dweights[s] = dot;
            } else {
                __syncthreads();
                if (lane == 0) part[wave] = dot;
                __syncthreads();
                if (threadIdx.x == 0) a.dweights[s] = part[0] + part[1] + part[2] + part[3];
            }
        }
    }
}

}  // namespace fl
