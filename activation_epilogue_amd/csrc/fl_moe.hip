// fl_moe.hip -- host side of the C ABI declared in include/fused_moe.h:
// argument validation, the choice of kernels and their launches on the
// caller's stream.  Device code is in fl_moe.hpp and fl_grouped.hpp.
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "fl_grouped.hpp"
#include "fl_moe.hpp"
#include "fused_moe.h"

namespace {

thread_local char g_err[512];

fl_status fail(fl_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return s;
}

void clear_error() { g_err[0] = '\0'; }

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr size_t kTwoGiB = 0x80000000ull;
constexpr int kCus = 256;  // workgroups of a persistent kernel that fill the chip, one per CU

size_t elem_size(int dtype) { return dtype == FL_F32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p % n) == 0; }

bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes) {
    if (!a || !b || abytes == 0 || bbytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

// An operand of a call: name, bytes it spans, alignment; `out` is written.
struct Operand {
    const char *name;
    const void *p;
    size_t bytes, align;
    bool out, optional;
    const void *same;  // an input this output may equal exactly
};

template <int N>
fl_status check_operands(const Operand (&ops)[N]) {
    for (const Operand &o : ops) {
        if (!o.p && o.bytes && !o.optional) return fail(FL_ERR_INVALID_ARG, "%s is NULL", o.name);
        if (o.p && !aligned(o.p, o.align))
            return fail(FL_ERR_INVALID_ARG, "%s (%p) is not aligned to %zu bytes", o.name, o.p, o.align);
    }
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            const Operand &o = ops[i], &q = ops[j];
            if (i == j || !o.out || (q.out && j < i)) continue;
            if (!q.out && o.same && o.p == q.p && o.same == q.p) continue;
            if (overlaps(o.p, o.bytes, q.p, q.bytes))
                return fail(FL_ERR_INVALID_ARG, "%s overlaps %s", o.name, q.name);
        }
    return FL_OK;
}

template <int N>
fl_status check_sizes(const int64_t (&v)[N]) {
    for (int64_t x : v)
        if (x < 0) return fail(FL_ERR_INVALID_ARG, "negative size %lld", (long long)x);
    for (int64_t x : v)
        if (x > kMaxDim) return fail(FL_ERR_UNSUPPORTED, "sizes above 2^31-1 are not supported");
    return FL_OK;
}

fl_status check_dtype(int d) {
    return d == FL_F32 || d == FL_F16 || d == FL_BF16 ? FL_OK : fail(FL_ERR_INVALID_ARG, "unknown dtype %d", d);
}

fl_status check_slots(int64_t T, int64_t k) {
    if (k && T > kMaxDim / k) return fail(FL_ERR_UNSUPPORTED, "more than 2^31-1 slots (T*k)");
    return FL_OK;
}

fl_status check_launch(const char *what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(FL_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
    return FL_OK;
}

// ------------------------------------------------------------------ router

fl_status route_options(const fl_route_options *opt, int64_t E, fl::RouteArgs &a) {
    const fl_route_options o = opt ? *opt : fl_route_options{};
    if (o.score != FL_SCORE_SOFTMAX && o.score != FL_SCORE_SIGMOID)
        return fail(FL_ERR_INVALID_ARG, "unknown score %d", o.score);
    if (o.raw != 0 && o.raw != 1) return fail(FL_ERR_INVALID_ARG, "raw must be 0 or 1");
    if (!isfinite(o.scale)) return fail(FL_ERR_INVALID_ARG, "scale must be finite");
    const int groups = o.groups ? o.groups : 1, top = o.top_groups ? o.top_groups : 1;
    const int gtop = o.group_top ? o.group_top : 1;
    if (groups < 1 || groups > 64 || E % groups)
        return fail(FL_ERR_INVALID_ARG, "groups (%d) must divide the %lld experts and be at most 64", groups,
                    (long long)E);
    if (top < 1 || top > groups) return fail(FL_ERR_INVALID_ARG, "top_groups (%d) must be 1 to groups (%d)", top, groups);
    if (gtop != 1 && gtop != 2) return fail(FL_ERR_INVALID_ARG, "group_top must be 1 or 2");
    a.sigmoid = o.score == FL_SCORE_SIGMOID;
    a.raw = o.raw;
    a.scale = o.scale != 0.0f ? o.scale : 1.0f;
    a.groups = groups;
    a.top_groups = top;
    a.group_top = gtop;
    return FL_OK;
}

fl_status check_route(int64_t T, int64_t E, int64_t k, int dtype) {
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    if ((s = check_sizes({T, E, k})) != FL_OK) return s;
    if (E < 1 || E > fl::kMaxExperts)
        return fail(FL_ERR_UNSUPPORTED, "E (%lld) must be 1 to %d", (long long)E, fl::kMaxExperts);
    if (k < 1 || k > E) return fail(FL_ERR_INVALID_ARG, "k (%lld) must be 1 to E (%lld)", (long long)k, (long long)E);
    if (k > fl::kMaxChoices) return fail(FL_ERR_UNSUPPORTED, "k (%lld) above %d", (long long)k, fl::kMaxChoices);
    return check_slots(T, k);
}

// Teams of 16 lanes wherever a team holds the experts (8 to a lane, 16 where
// there are tokens enough to hide the longer steps), the choices and the runs;
// else whole waves.
template <int DT, bool BWD, int EPL, int TEAM>
void launch_route_team(const fl::RouteArgs &a, hipStream_t st) {
    constexpr int TOKENS = 256 / TEAM;
    const int64_t blocks = ((int64_t)a.T + TOKENS - 1) / TOKENS;
    const dim3 grid((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20));
    if (BWD)
        hipLaunchKernelGGL((fl::route_bwd_kernel<DT, EPL, TEAM>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((fl::route_kernel<DT, EPL, TEAM>), grid, dim3(256), 0, st, a);
}

template <int DT, bool BWD, int TEAM>
void launch_route_dt(const fl::RouteArgs &a, hipStream_t st) {
    if (a.E <= TEAM)
        launch_route_team<DT, BWD, 1, TEAM>(a, st);
    else if (a.E <= 2 * TEAM)
        launch_route_team<DT, BWD, 2, TEAM>(a, st);
    else if (a.E <= 4 * TEAM)
        launch_route_team<DT, BWD, 4, TEAM>(a, st);
    else if (a.E <= 8 * TEAM)
        launch_route_team<DT, BWD, 8, TEAM>(a, st);
    else
        launch_route_team<DT, BWD, 16, TEAM>(a, st);
}

template <int DT, bool BWD>
void launch_route_dt(const fl::RouteArgs &a, hipStream_t st) {
    if (a.E <= (a.T < 4096 ? 128 : 256) && a.k <= 16 && a.groups <= 16)
        launch_route_dt<DT, BWD, 16>(a, st);
    else
        launch_route_dt<DT, BWD, 64>(a, st);
}

template <bool BWD>
void launch_route(int dtype, const fl::RouteArgs &a, hipStream_t st) {
    if (dtype == FL_F32)
        launch_route_dt<FL_F32, BWD>(a, st);
    else if (dtype == FL_F16)
        launch_route_dt<FL_F16, BWD>(a, st);
    else
        launch_route_dt<FL_BF16, BWD>(a, st);
}

// ---------------------------------------------------------------- movement

#define FL_MOVE_COLS(kernel, dtype, vec, cols, grid, st, a)                                            \
    do {                                                                                               \
        if ((dtype) == FL_F32) {                                                                       \
            if (vec) hipLaunchKernelGGL((fl::kernel<FL_F32, true, cols>), grid, dim3(256), 0, st, a);  \
            else hipLaunchKernelGGL((fl::kernel<FL_F32, false, cols>), grid, dim3(256), 0, st, a);     \
        } else if ((dtype) == FL_F16) {                                                                \
            if (vec) hipLaunchKernelGGL((fl::kernel<FL_F16, true, cols>), grid, dim3(256), 0, st, a);  \
            else hipLaunchKernelGGL((fl::kernel<FL_F16, false, cols>), grid, dim3(256), 0, st, a);     \
        } else {                                                                                       \
            if (vec) hipLaunchKernelGGL((fl::kernel<FL_BF16, true, cols>), grid, dim3(256), 0, st, a); \
            else hipLaunchKernelGGL((fl::kernel<FL_BF16, false, cols>), grid, dim3(256), 0, st, a);    \
        }                                                                                              \
    } while (0)
#define FL_MOVE(kernel, dtype, vec, pieces, rows, st, a)                                          \
    do {                                                                                          \
        if ((pieces) <= 64)                                                                       \
            FL_MOVE_COLS(kernel, dtype, vec, 64, move_grid(rows, pieces, 64), st, a);             \
        else if ((pieces) <= 128)                                                                 \
            FL_MOVE_COLS(kernel, dtype, vec, 128, move_grid(rows, pieces, 128), st, a);           \
        else                                                                                      \
            FL_MOVE_COLS(kernel, dtype, vec, 256, move_grid(rows, pieces, 256), st, a);           \
    } while (0)

bool rows_aligned(int dtype, int64_t H, const void *p, const void *q, const void *r) {
    return (H * elem_size(dtype)) % 16 == 0 && aligned(p, 16) && aligned(q, 16) && aligned(r, 16);
}

unsigned grid_of(int64_t n) { return (unsigned)(n < 1 ? 1 : n < 1 << 22 ? n : 1 << 22); }

// Blocks of 256 / cols rows; few rows are cut along their pieces as well.
dim3 move_grid(int64_t rows, int64_t pieces, int cols) {
    const int64_t y = rows < 65536 ? (pieces + cols - 1) / cols : 1;
    return dim3(grid_of((rows * cols + 255) / 256), (unsigned)(y < 64 ? y : 64));
}

// ------------------------------------------------------- experts' products

fl_status check_grouped(int64_t S, int64_t N, int64_t K, int64_t E, int act, int dtype) {
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    if (act < FL_ACT_NONE || act > FL_ACT_GLU) return fail(FL_ERR_INVALID_ARG, "unknown activation %d", act);
    if ((s = check_sizes({S, N, K, E})) != FL_OK) return s;
    if (E < 1 || E > fl::kMaxExperts)
        return fail(FL_ERR_UNSUPPORTED, "E (%lld) must be 1 to %d", (long long)E, fl::kMaxExperts);
    const size_t es = elem_size(dtype);
    if ((size_t)K * es * 256 >= kTwoGiB || (size_t)N * es * 256 >= kTwoGiB)
        return fail(FL_ERR_UNSUPPORTED, "K or N too large (256 rows must span < 2 GiB)");
    if ((size_t)K * N * es >= kTwoGiB)
        return fail(FL_ERR_UNSUPPORTED, "B too large (an expert's K x N elements must span < 2 GiB)");
    return FL_OK;
}

// Most row tiles that S rows in at most E runs can be cut into.
int64_t most_row_tiles(int64_t S, int64_t E, int64_t bm) {
    const int64_t runs = E < S ? E : S;
    return (S + runs * (bm - 1)) / bm;
}

template <int DT>
fl::grouped_launcher pick_grouped_dt(int form, int variant, bool nt) {
    return form == fl::kFormFwd   ? fl::pick_grouped<DT, fl::kFormFwd>(variant, nt)
           : form == fl::kFormBwd ? fl::pick_grouped<DT, fl::kFormBwd>(variant, nt)
                                  : fl::pick_grouped<DT, fl::kFormGrad>(variant, nt);
}

fl::grouped_launcher pick_grouped(int dtype, int form, int variant, bool nt) {
    return dtype == FL_F32   ? pick_grouped_dt<FL_F32>(form, variant, nt)
           : dtype == FL_F16 ? pick_grouped_dt<FL_F16>(form, variant, nt)
                             : pick_grouped_dt<FL_BF16>(form, variant, nt);
}

template <int FORM>
void join_form(int dtype, const fl::GroupedArgs &a, int act, hipStream_t st) {
    if (dtype == FL_F32)
        fl::launch_join<FL_F32, FORM>(a, act, st);
    else if (dtype == FL_F16)
        fl::launch_join<FL_F16, FORM>(a, act, st);
    else
        fl::launch_join<FL_BF16, FORM>(a, act, st);
}

void join(int dtype, int form, const fl::GroupedArgs &a, int act, hipStream_t st) {
    if (form == fl::kFormGrad)
        join_form<fl::kFormGrad>(dtype, a, act, st);
    else
        join_form<fl::kFormFwd>(dtype, a, act, st);
}

// The tile: the one of least estimated time, in rounds of a full chip.  Runs end
// inside a tile, so S rows in R runs make about S/bm + R/2 row tiles (at least
// R); rounds beyond the first end ragged, half a round on average; the time is
// at least that of the weights.  Wide low tiles stream weights best where they
// fill the chip and runs have one of them (8 experts of 4096x14336, 256 rows: 160
// us, 207 with 32x128; but 64 experts of 2048x1408, 384 rows: 67 us, 59 with
// 32x128).
//
// Where the chosen tiles leave most of the chip idle and the sum is long, it is
// cut into 4, 8 or 16 parts for more workgroups, whose fp32 sums another launch
// joins (4 us and a little per part), if that takes clearly less time than the
// stages of one workgroup, as far as the memory (6 TB/s) can follow.  Measured
// without and with: bf16, one token through 2 of 8 experts, K 4096, N 1024: 19.4
// -> 14.1 us; fp32: 75.8 -> 20.8 us; weight gradient of 16384 rows, 2 experts,
// 256x256: 67.7 -> 15.9 us.
struct GroupedPlan {
    int variant, parts;
};

GroupedPlan plan_grouped(int dtype, int form, int64_t S, int64_t N, int64_t K, int64_t E) {
    GroupedPlan best{-1, 1};
    double least = 0.0, tiles = 0.0;
    for (int v = 0; v < fl::kGroupedVariants; ++v) {
        const fl::GroupedTileShape &t = fl::kGroupedTiles[v];
        if ((v >= fl::kTileF32) != (dtype == FL_F32) || (form == fl::kFormGrad && !t.grad)) continue;
        double m;
        if (form == fl::kFormGrad) {
            m = (double)E * ((K + t.bm - 1) / t.bm);
        } else {
            const double runs = (double)(E < S ? E : S);
            m = (double)S / t.bm + 0.5 * runs;
            m = m > runs ? m : runs;
        }
        const double n = (N + t.bn - 1) / t.bn, x = m * n / (kCus * t.per_cu);
        double time = t.time * (x <= 1.0 ? 1.0 : x + 0.5);
        if (dtype != FL_F32 && form != fl::kFormGrad) {
            if (v == fl::kTile64x256) {
                if (x < 1.0) continue;
                if (S <= 48 * E) time *= 0.7;
            }
            if (x <= 0.5 && t.per_cu == 2) time *= 0.75;  // workgroups with a CU to themselves
            // tiles that are mostly empty skip their empty half
            if (t.bm >= 128) time *= S <= E * t.bm / 4 ? 0.7 : S <= E * t.bm / 2 ? 0.85 : 1.0;
            // the weights: at most once for a low tile, once for a run of high ones
            const double reads = (t.bm <= 64 ? m : (double)(E < S ? E : S)) * n;
            const double memory = reads * t.bn * 128 / (t.rate * 1e6) / 1.9;  // of a round's 1.9 us a stage
            time = time > memory ? time : memory;
        }
        m *= n;
        if (best.variant < 0 || time < least) {
            least = time;
            tiles = m;
            best.variant = v;
        }
    }
    const int64_t ks = dtype == FL_F32 ? 32 : 64, depth = form == fl::kFormGrad ? S / E : K;
    const fl::GroupedTileShape &t = fl::kGroupedTiles[best.variant];
    const double stages = (double)((depth + ks - 1) / ks);
    const double memory = tiles * stages * (t.bm + t.bn) * 128 / 6e6;
    double limit = 0.85 * (4.0 + (stages * t.stage > memory ? stages * t.stage : memory));  // a clear gain, or none
    for (int p = 4; form != fl::kFormBwd && p <= 16 && p * 4 <= stages && p * tiles <= kCus * t.per_cu; p *= 2) {
        const double each = stages / p * t.stage;
        const double time = 8.0 + 0.1 * p + (each > memory ? each : memory);
        if (time < limit) {
            limit = time;
            best.parts = p;
        }
    }
    return best;
}

size_t grouped_workspace(int form, int64_t S, int64_t N, int64_t K, int64_t E, int dtype) {
    if (S == 0 || N == 0 || K == 0) return 0;
    const GroupedPlan p = plan_grouped(dtype, form, S, N, K, E);
    return p.parts > 1 ? (size_t)p.parts * (form == fl::kFormGrad ? E * K : S) * N * 4 : 0;
}

fl_status launch_grouped(fl::GroupedArgs &a, int form, int act, int dtype, void *workspace, void *stream,
                         const char *what) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    const GroupedPlan p = plan_grouped(dtype, form, a.S, a.N, a.K, a.E);
    const fl::GroupedTileShape &t = fl::kGroupedTiles[p.variant];
    a.tiles_n = (int)((a.N + t.bn - 1) / t.bn);
    // bands of 8 row tiles: prompts through 64 experts 210 us, 218 with 4 or
    // 16; weight gradient (operands of equal height) 1614 us with 4, 1627 with 8
    a.group = form == fl::kFormGrad ? 4 : 8;
    // Spread over the XCDs, an expert's tiles load its weights into every L2
    // but the work is even whatever the runs' lengths: 1780 against 1820 us
    // where an expert has 470 tiles, 233 against 210 us where it has 22 (the
    // border lies somewhere between).
    a.spread = (int64_t)a.S / a.E / t.bm * a.tiles_n >= 128;
    a.stream = (size_t)a.N * elem_size(dtype) % 128 == 0 && aligned(a.out, 128) && aligned(a.out2, 128);
    a.parts = workspace ? p.parts : 1;
    a.part = static_cast<float *>(workspace);
    const int64_t tiles_m = form == fl::kFormGrad ? a.E * (((int64_t)a.K + t.bm - 1) / t.bm) : most_row_tiles(a.S, a.E, t.bm);
    const int64_t tiles = tiles_m * a.tiles_n, grid = tiles * a.parts, slots = kCus * t.per_cu;
    if (grid > kMaxDim - slots)  // (a workgroup's next tile is its last plus the grid)
        return fail(FL_ERR_UNSUPPORTED, "too many output tiles");
    a.max_tiles = (int)tiles;
    if (form == fl::kFormGrad && a.dbias) {
        if (dtype == FL_F32)
            fl::launch_column_sum<FL_F32>(a, st);
        else if (dtype == FL_F16)
            fl::launch_column_sum<FL_F16>(a, st);
        else
            fl::launch_column_sum<FL_BF16>(a, st);
        const fl_status s = check_launch(what);
        if (s != FL_OK) return s;
    }
    if (grid == 0) return FL_OK;
    // Weights that are read once, by runs of one low tile each, stream past the
    // L2: 64 experts of 2048x1408, 192 rows 58 and 66 us; fp32, 8 experts of
    // 4096x4096, 16 rows 91 and 99.  Runs of several tiles read them again, from
    // the L2: 2 experts of 4096x1024, 1000 rows 31 us past it, 22 through it; one
    // of 4096x4096, 300 rows 54 and 34.
    const bool nt = t.bm <= 64 && a.S <= (int64_t)t.bm * (a.E < a.S ? a.E : a.S);
    pick_grouped(dtype, form, p.variant, nt)(a, act, grid < slots ? grid : slots, st);
    if (a.parts > 1) {
        const fl_status s = check_launch(what);
        if (s != FL_OK) return s;
        join(dtype, form, a, act, st);
    }
    return check_launch(what);
}

}  // namespace

extern "C" {

fl_status fl_moe_route(const void *logits, const float *bias, int32_t *experts, float *weights, int64_t T, int64_t E,
                       int64_t k, fl_dtype dtype, const fl_route_options *opt, void *stream) {
    clear_error();
    fl_status s = check_route(T, E, k, dtype);
    if (s != FL_OK) return s;
    fl::RouteArgs a{};
    if ((s = route_options(opt, E, a)) != FL_OK) return s;
    const size_t es = elem_size(dtype), slots = (size_t)T * k;
    const Operand ops[] = {{"logits", logits, (size_t)T * E * es, es, false, false, nullptr},
                           {"bias", bias, (size_t)E * 4, 4, false, true, nullptr},
                           {"experts", experts, slots * 4, 4, true, false, nullptr},
                           {"weights", weights, slots * 4, 4, true, false, nullptr}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (T == 0) return FL_OK;
    a.logits = logits;
    a.bias = bias;
    a.experts = experts;
    a.weights = weights;
    a.T = (int)T;
    a.E = (int)E;
    a.k = (int)k;
    launch_route<false>(dtype, a, static_cast<hipStream_t>(stream));
    return check_launch("moe_route");
}

fl_status fl_moe_route_bwd(const void *logits, const int32_t *experts, const float *dweights, void *dlogits, int64_t T,
                           int64_t E, int64_t k, fl_dtype dtype, const fl_route_options *opt, void *stream) {
    clear_error();
    fl_status s = check_route(T, E, k, dtype);
    if (s != FL_OK) return s;
    fl::RouteArgs a{};
    if ((s = route_options(opt, E, a)) != FL_OK) return s;
    const size_t es = elem_size(dtype), slots = (size_t)T * k;
    const Operand ops[] = {{"logits", logits, (size_t)T * E * es, es, false, false, nullptr},
                           {"experts", experts, slots * 4, 4, false, false, nullptr},
                           {"dweights", dweights, slots * 4, 4, false, false, nullptr},
                           {"dlogits", dlogits, (size_t)T * E * es, es, true, false, logits}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (T == 0) return FL_OK;
    a.logits = logits;
    a.experts = const_cast<int32_t *>(experts);
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.T = (int)T;
    a.E = (int)E;
    a.k = (int)k;
    launch_route<true>(dtype, a, static_cast<hipStream_t>(stream));
    return check_launch("moe_route_bwd");
}

fl_status fl_moe_plan_workspace_bytes(int64_t T, int64_t k, int64_t E, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(FL_ERR_INVALID_ARG, "bytes is NULL");
    fl_status s = check_sizes({T, k, E});
    if (s != FL_OK) return s;
    if (E < 1 || E > fl::kMaxExperts)
        return fail(FL_ERR_UNSUPPORTED, "E (%lld) must be 1 to %d", (long long)E, fl::kMaxExperts);
    if ((s = check_slots(T, k)) != FL_OK) return s;
    const int64_t blocks = (T * k + fl::kPlanChunk - 1) / fl::kPlanChunk;
    *bytes = blocks > 1 ? (size_t)(blocks + (blocks > fl::kPlanDirect)) * E * 4 : 0;
    return FL_OK;
}

fl_status fl_moe_plan(const int32_t *experts, int32_t *offsets, int32_t *token_of_row, int32_t *row_of_slot, int64_t T,
                      int64_t k, int64_t E, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    fl_status s = fl_moe_plan_workspace_bytes(T, k, E, &need);
    if (s != FL_OK) return s;
    const size_t slots = (size_t)T * k;
    if (need && (!workspace || workspace_bytes < need))
        return fail(FL_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const Operand ops[] = {{"experts", experts, slots * 4, 4, false, false, nullptr},
                           {"offsets", offsets, (size_t)(E + 1) * 4, 4, true, false, nullptr},
                           {"token_of_row", token_of_row, slots * 4, 4, true, false, nullptr},
                           {"row_of_slot", row_of_slot, slots * 4, 4, true, false, nullptr},
                           {"workspace", need ? workspace : nullptr, need, 4, true, true, nullptr}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    fl::PlanArgs a{};
    a.experts = experts;
    a.offsets = offsets;
    a.token_of_row = token_of_row;
    a.row_of_slot = row_of_slot;
    a.counts = need ? static_cast<int32_t *>(workspace) : nullptr;
    a.S = (int64_t)slots;
    a.k = k ? (int)k : 1;
    a.E = (int)E;
    const int64_t blocks = (a.S + fl::kPlanChunk - 1) / fl::kPlanChunk;
    const dim3 grid((unsigned)(blocks ? blocks : 1));
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (need) hipLaunchKernelGGL(fl::plan_count_kernel, grid, dim3(1024), 0, st, a);
    a.summed = blocks > fl::kPlanDirect;
    if (a.summed) {
        int cols = 64;
        while (cols > 8 && cols / 2 >= E) cols /= 2;
        hipLaunchKernelGGL(fl::plan_sum_kernel, dim3((unsigned)((E + cols - 1) / cols)), dim3(1024), 0, st, a,
                           (int)blocks, cols);
    }
    if (a.S <= fl::kPlanSmall) {
        if (E <= 256)
            hipLaunchKernelGGL((fl::plan_kernel<4, 256>), grid, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((fl::plan_kernel<4, 1024>), grid, dim3(256), 0, st, a);
    } else if (E <= 256) {
        hipLaunchKernelGGL((fl::plan_kernel<16, 256>), grid, dim3(1024), 0, st, a);
    } else {
        hipLaunchKernelGGL((fl::plan_kernel<16, 1024>), grid, dim3(1024), 0, st, a);
    }
    return check_launch("moe_plan");
}

fl_status fl_moe_gather(const void *X, const int32_t *index, void *rows, int64_t T, int64_t S, int64_t H,
                        fl_dtype dtype, void *stream) {
    clear_error();
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    if ((s = check_sizes({T, S, H})) != FL_OK) return s;
    const size_t es = elem_size(dtype);
    const Operand ops[] = {{"X", X, (size_t)T * H * es, es, false, false, nullptr},
                           {"index", index, (size_t)S * 4, 4, false, false, nullptr},
                           {"rows", rows, (size_t)S * H * es, es, true, false, nullptr}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (S == 0 || H == 0) return FL_OK;
    fl::MoveArgs a{};
    a.src = X;
    a.map = index;
    a.dst = rows;
    a.T = T;
    a.S = S;
    a.H = H;
    const bool vec = rows_aligned(dtype, H, X, rows, nullptr);
    FL_MOVE(gather_kernel, dtype, vec, vec ? (int64_t)(H * es / 16) : H, S, static_cast<hipStream_t>(stream), a);
    return check_launch("moe_gather");
}

fl_status fl_moe_combine(const void *rows, const int32_t *row_of_slot, const float *weights, const void *R, void *out,
                         int64_t T, int64_t k, int64_t S, int64_t H, fl_dtype dtype, void *stream) {
    clear_error();
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    if ((s = check_sizes({T, k, S, H})) != FL_OK) return s;
    if ((s = check_slots(T, k)) != FL_OK) return s;
    const size_t es = elem_size(dtype), slots = (size_t)T * k;
    const Operand ops[] = {{"rows", rows, (size_t)S * H * es, es, false, false, nullptr},
                           {"row_of_slot", row_of_slot, slots * 4, 4, false, false, nullptr},
                           {"weights", weights, slots * 4, 4, false, true, nullptr},
                           {"R", R, (size_t)T * H * es, es, false, true, nullptr},
                           {"out", out, (size_t)T * H * es, es, true, false, R}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (T == 0 || H == 0) return FL_OK;
    fl::MoveArgs a{};
    a.src = rows;
    a.src2 = R;
    a.map = row_of_slot;
    a.weights = weights;
    a.dst = out;
    a.T = T;
    a.S = S;
    a.H = H;
    a.k = (int)k;
    const bool vec = rows_aligned(dtype, H, rows, R, out);
    FL_MOVE(combine_kernel, dtype, vec, vec ? (int64_t)(H * es / 16) : H, T, static_cast<hipStream_t>(stream), a);
    return check_launch("moe_combine");
}

fl_status fl_moe_combine_bwd(const void *dout, const void *rows, const int32_t *row_of_slot, const float *weights,
                             void *drows, float *dweights, int64_t T, int64_t k, int64_t S, int64_t H, fl_dtype dtype,
                             void *stream) {
    clear_error();
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    if ((s = check_sizes({T, k, S, H})) != FL_OK) return s;
    if ((s = check_slots(T, k)) != FL_OK) return s;
    const size_t es = elem_size(dtype), slots = (size_t)T * k;
    // (an empty output has no address)
    if (!drows && !dweights && slots && S && H)
        return fail(FL_ERR_INVALID_ARG, "drows and dweights are both NULL");
    const Operand ops[] = {{"dout", dout, (size_t)T * H * es, es, false, false, nullptr},
                           {"rows", rows, dweights ? (size_t)S * H * es : 0, es, false, !dweights, nullptr},
                           {"row_of_slot", row_of_slot, slots * 4, 4, false, false, nullptr},
                           {"weights", weights, slots * 4, 4, false, true, nullptr},
                           {"drows", drows, (size_t)S * H * es, es, true, true, rows},
                           {"dweights", dweights, slots * 4, 4, true, true, nullptr}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (slots == 0 || (!drows && !dweights)) return FL_OK;
    fl::MoveArgs a{};
    a.src = dout;
    a.src2 = rows;
    a.map = row_of_slot;
    a.weights = weights;
    a.dst = drows;
    a.dweights = dweights;
    a.T = T;
    a.S = S;
    a.H = H;
    a.k = (int)k;
    const bool vec = rows_aligned(dtype, H, dout, dweights ? rows : nullptr, drows);
    // a wave per slot where they fill the chip (16384 slots of 1024 bf16: 32 us,
    // a block per slot 48), a block where there are few
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (slots >= 4096)
        FL_MOVE_COLS(combine_bwd_kernel, dtype, vec, 64, dim3(grid_of((int64_t)(slots + 3) / 4)), st, a);
    else
        FL_MOVE_COLS(combine_bwd_kernel, dtype, vec, 256, dim3(grid_of((int64_t)slots)), st, a);
    return check_launch("moe_combine_bwd");
}

fl_status fl_grouped_workspace_bytes(int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(FL_ERR_INVALID_ARG, "bytes is NULL");
    const fl_status s = check_grouped(S, N, K, E, FL_ACT_NONE, dtype);
    if (s != FL_OK) return s;
    *bytes = grouped_workspace(fl::kFormFwd, S, N, K, E, dtype);
    return FL_OK;
}

fl_status fl_grouped_grad_workspace_bytes(int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(FL_ERR_INVALID_ARG, "bytes is NULL");
    const fl_status s = check_grouped(S, N, K, E, FL_ACT_NONE, dtype);
    if (s != FL_OK) return s;
    *bytes = grouped_workspace(fl::kFormGrad, S, N, K, E, dtype);
    return FL_OK;
}

fl_status fl_grouped_linear(const void *A, const int32_t *index, const int32_t *offsets, const void *B,
                            const void *bias, const void *Y, void *out, void *pre, int64_t A_rows, int64_t S,
                            int64_t N, int64_t K, int64_t E, fl_act act, fl_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
    clear_error();
    fl_status s = check_grouped(S, N, K, E, act, dtype);
    if (s != FL_OK) return s;
    if ((s = check_sizes({A_rows})) != FL_OK) return s;
    const size_t need = grouped_workspace(fl::kFormFwd, S, N, K, E, dtype);
    const size_t es = elem_size(dtype), o_bytes = (size_t)S * N * es;
    if (!index && A_rows < S)
        return fail(FL_ERR_INVALID_ARG, "A has %lld rows, %lld needed without an index", (long long)A_rows,
                    (long long)S);
    if (index && (size_t)A_rows * K * es >= kTwoGiB)
        return fail(FL_ERR_UNSUPPORTED, "A too large for an index (it must span < 2 GiB; fl_moe_gather has no limit)");
    if (act == FL_ACT_GLU && !Y && o_bytes) return fail(FL_ERR_INVALID_ARG, "the gate needs Y");
    if (act != FL_ACT_GLU && Y) return fail(FL_ERR_INVALID_ARG, "Y is only used by the gate (FL_ACT_GLU)");
    if (need && (!workspace || workspace_bytes < need))
        return fail(FL_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const Operand ops[] = {{"A", A, (size_t)A_rows * K * es, es, false, S == 0 || N == 0, nullptr},
                           {"index", index, (size_t)S * 4, 4, false, true, nullptr},
                           {"offsets", offsets, (size_t)(E + 1) * 4, 4, false, false, nullptr},
                           {"B", B, (size_t)E * K * N * es, es, false, S == 0, nullptr},
                           {"bias", bias, (size_t)E * N * es, es, false, true, nullptr},
                           {"Y", Y, o_bytes, es, false, true, nullptr},
                           {"out", out, o_bytes, es, true, false, Y},
                           {"pre", pre, o_bytes, es, true, true, nullptr},
                           {"workspace", need ? workspace : nullptr, need, 16, true, true, nullptr}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (S == 0 || N == 0) return FL_OK;
    fl::GroupedArgs a{};
    a.A = A;
    a.index = index;
    a.offsets = offsets;
    a.B = B;
    a.bias = bias;
    a.Y = Y;
    a.out = out;
    a.out2 = pre;
    a.A_rows = A_rows;
    a.S = (int)S;
    a.N = (int)N;
    a.K = (int)K;
    a.E = (int)E;
    return launch_grouped(a, fl::kFormFwd, act, dtype, need ? workspace : nullptr, stream, "grouped_linear");
}

fl_status fl_grouped_linear_bwd(const void *G, const int32_t *offsets, const void *W, const void *X, const void *Y,
                                void *dX, void *dY, int64_t S, int64_t N, int64_t K, int64_t E, fl_act act,
                                fl_dtype dtype, void *stream) {
    clear_error();
    fl_status s = check_grouped(S, N, K, E, act, dtype);
    if (s != FL_OK) return s;
    const size_t es = elem_size(dtype), o_bytes = (size_t)S * N * es;
    if (act != FL_ACT_NONE && !X && o_bytes) return fail(FL_ERR_INVALID_ARG, "X is NULL");
    if (act == FL_ACT_GLU && !Y && o_bytes) return fail(FL_ERR_INVALID_ARG, "the gate needs Y");
    if (act != FL_ACT_GLU && (Y || dY))
        return fail(FL_ERR_INVALID_ARG, "Y and dY are only used by the gate (FL_ACT_GLU)");
    const Operand ops[] = {{"G", G, (size_t)S * K * es, es, false, N == 0, nullptr},
                           {"offsets", offsets, (size_t)(E + 1) * 4, 4, false, false, nullptr},
                           {"W", W, (size_t)E * N * K * es, es, false, S == 0, nullptr},
                           {"X", X, o_bytes, es, false, true, nullptr},
                           {"Y", Y, o_bytes, es, false, true, nullptr},
                           {"dX", dX, o_bytes, es, true, false, X},
                           {"dY", dY, act == FL_ACT_GLU ? o_bytes : 0, es, true, act != FL_ACT_GLU, Y}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (S == 0 || N == 0) return FL_OK;
    fl::GroupedArgs a{};
    a.A = G;
    a.offsets = offsets;
    a.B = W;
    a.X = act == FL_ACT_NONE ? nullptr : X;
    a.Y = Y;
    a.out = dX;
    a.out2 = dY;
    a.A_rows = S;
    a.S = (int)S;
    a.N = (int)N;
    a.K = (int)K;
    a.E = (int)E;
    return launch_grouped(a, fl::kFormBwd, act, dtype, nullptr, stream, "grouped_linear_bwd");
}

fl_status fl_grouped_weight_grad(const void *A, const void *G, const int32_t *offsets, void *dW, float *dbias,
                                 int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, fl_dtype dw_dtype,
                                 void *stream) {
    return fl_grouped_weight_grad_ws(A, G, offsets, dW, dbias, S, N, K, E, dtype, dw_dtype, nullptr, 0, stream);
}

fl_status fl_grouped_weight_grad_ws(const void *A, const void *G, const int32_t *offsets, void *dW, float *dbias,
                                    int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, fl_dtype dw_dtype,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    fl_status s = check_grouped(S, N, K, E, FL_ACT_NONE, dtype);
    if (s != FL_OK) return s;
    if (dw_dtype != dtype && dw_dtype != FL_F32)
        return fail(FL_ERR_INVALID_ARG, "dW is in the operands' dtype or fp32 (got %d)", (int)dw_dtype);
    if ((size_t)N * elem_size(dw_dtype) * 256 >= kTwoGiB)
        return fail(FL_ERR_UNSUPPORTED, "N too large (256 rows of dW must span < 2 GiB)");
    const size_t need = grouped_workspace(fl::kFormGrad, S, N, K, E, dtype);
    if (workspace && workspace_bytes < need)
        return fail(FL_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    const size_t es = elem_size(dtype), des = elem_size(dw_dtype);
    const Operand ops[] = {{"A", A, (size_t)S * K * es, es, false, N == 0, nullptr},
                           {"G", G, (size_t)S * N * es, es, false, false, nullptr},
                           {"offsets", offsets, (size_t)(E + 1) * 4, 4, false, false, nullptr},
                           {"dW", dW, (size_t)E * K * N * des, des, true, false, nullptr},
                           {"dbias", dbias, (size_t)E * N * 4, 4, true, true, nullptr},
                           {"workspace", workspace, workspace ? need : 0, 16, true, true, nullptr}};
    if ((s = check_operands(ops)) != FL_OK) return s;
    if (N == 0 || (K == 0 && !dbias)) return FL_OK;
    fl::GroupedArgs a{};
    a.A = A;
    a.offsets = offsets;
    a.B = G;
    a.out = dW;
    a.dbias = dbias;
    a.dw_f32 = dw_dtype == FL_F32;
    a.A_rows = S;
    a.S = (int)S;
    a.N = (int)N;
    a.K = (int)K;
    a.E = (int)E;
    return launch_grouped(a, fl::kFormGrad, FL_ACT_NONE, dtype, need ? workspace : nullptr, stream, "grouped_weight_grad");
}

const char *fl_moe_last_error(void) { return g_err; }

}  // extern "C"
