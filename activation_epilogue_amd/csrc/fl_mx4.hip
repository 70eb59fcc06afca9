// fl_mx4.hip -- host side of the C ABI declared in include/fused_mx4.h:
// argument validation, the choice of kernels and their launches on the
// caller's stream.  Device code is in fl_mx4.hpp (quantising), fl_mx4_linear.hpp
// and fl_mx4_tile.hpp (the linear layer; its kernels are built by fl_mx4_inst.hip).
#include "fl_check.hpp"
#include "fl_mx4_tile.hpp"
#include "fused_mx4.h"

namespace {

int64_t blocks_of(int64_t K) { return (K + 31) / 32; }

// Whether four lanes share a block's 32 rows: where that many lanes do not fill the chip a
// lane's share is what is waited for (bf16 7 rows of 373: 5.6 us, 15.7 with one lane to a
// block; 2247 of 2091: 9.8, 22.0; 4096 of 2048: 5.5, 7.7; 4096 of 4096: 9.4, 9.0; 14336 of
// 4096: 27.5, 26.1).  A launch has 65535 blocks in its second dimension.
bool split_columns(const fl::Mx4Args &a) { return a.rows * a.blocks <= 3 << 17 && a.blocks <= 2 * 65535; }

// Blocks of 1024 units of eight values, in two dimensions (mx4_first_unit).
dim3 grid_of_units(const fl::Mx4Args &a) {
    const int64_t per_block = 256 * fl::kMx4Units, all = (a.rows * a.blocks * 4 + per_block - 1) / per_block;
    const int64_t across = all < 1 << 20 ? all : 1 << 20;
    return dim3((unsigned)across, (unsigned)((all + across - 1) / across));
}

template <int DT>
void launch_quantize(const fl::Mx4Args &a, bool transposed, hipStream_t st) {
    if (transposed) {
        const int64_t per_block = 32 * (DT == FL_F32 ? 4 : 8);
        const unsigned across = (unsigned)((a.rows + per_block - 1) / per_block);
        if (split_columns(a))
            hipLaunchKernelGGL((fl::quantize_mx4_transposed_kernel<DT, 4>), dim3(across, (unsigned)((a.blocks + 1) / 2)),
                               dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((fl::quantize_mx4_transposed_kernel<DT, 1>), dim3(across, (unsigned)((a.blocks + 7) / 8)),
                               dim3(256), 0, st, a);
    } else {
        hipLaunchKernelGGL((fl::quantize_mx4_kernel<DT>), grid_of_units(a), dim3(256), 0, st, a);
    }
}

void quantize(const fl::Mx4Args &a, bool transposed, int dtype, hipStream_t st) {
    if (dtype == FL_F32)
        launch_quantize<FL_F32>(a, transposed, st);
    else if (dtype == FL_F16)
        launch_quantize<FL_F16>(a, transposed, st);
    else
        launch_quantize<FL_BF16>(a, transposed, st);
}

// rows x K values, their codes and scales.
fl_status check_matrix(int64_t rows, int64_t K, int dtype) {
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    if ((s = check_sizes({rows, K})) != FL_OK) return s;
    // units of 1024 to a launch's block, blocks of 8 K blocks in its second dimension
    if (rows && blocks_of(K) > ((int64_t)1 << 38) / rows)
        return fail(FL_ERR_UNSUPPORTED, "more than 2^38 blocks");
    if (blocks_of(K) > 8 * 65535) return fail(FL_ERR_UNSUPPORTED, "K (%lld) above 2^24 - 256", (long long)K);
    return FL_OK;
}

constexpr int64_t kLinearK = 1 << 22;

// How a linear layer runs: the streaming kernel for few rows, else tiles of a
// size, K in parts where there are few of them; the epilogue alone for no K.
struct LinearPlan {
    bool stream, quantize;  // quantize: A's values first, into the workspace
    fl::Mx4StreamShape shape;
    int variant, parts, part_stages;  // parts 0: the epilogue alone
    int64_t first_columns;  // of 256x256 tiles, the rest of 128x128 by another launch; 0: all of one size
    size_t codes, scales, sums;  // bytes of the workspace, in this order
};

size_t align16(size_t n) { return (n + 15) / 16 * 16; }
double ceil_div(double a, double b) { return (double)(int64_t)((a + b - 1) / b); }

// Of the ways below the one of the least estimated time, in us (the constants fitted to
// every shape's and tile's times at 270 random sizes, M 1 to 8192, N and K 64 to 24576;
// at 100 others what is chosen takes the fastest's time in the mean, 1.14 times it at most):
//   streaming   3, and a round of the chip 0.3 for each 16x16 of outputs and 0.25 for each
//               16 rows of A or B and 1024 values of K.  One token by 14336x4096: 7.7 us,
//               tiles 33; 64 by 4096x14336: 17.1, tiles 14.9; 128 by 14336x4096: 26, tiles
//               13.7.  64 by 64 outputs to a block, seldom the least: 33 by 13961x3612 10.6,
//               13.2 without (tiles), 39 by 13972x4985 15.6 and 16.1.
//   256x256     3.4, and a round 7.5 + 1.62 a stage of 256 values of K.
//   128x128     3.4, and two to a CU: a round 4.3 + 1.24 a stage, a part of one a third
//               more than its share and not under 0.54.  4608x4096x4096 55 us, 63 with
//               256x256; 8192x14336x4096 312 and 256.  Up to 256 of them, which have a
//               CU to themselves, of eight waves with four stages under way: 2 + 0.52 a
//               stage (128 by 14336x4096 13.7 us, 14.9 as the others are).
//   both        256x256 for whole rounds of the chip, 2 for a second launch of 128x128 for
//               the columns behind them: 4096x4352x14336 152 us, 186 and 164 with one of
//               them.
//   parts of K  a join of 4, and the sums written and read at 5 TB/s: 128 by 4096x14336
//               43 us in one part, 20 in 8.
double tiles_time(int variant, double tiles, double stages) {
    if (variant == fl::kMx4Tile256) return ceil_div(tiles, 256) * (7.5 + 1.62 * stages);
    if (variant == fl::kMx4Tile128Alone) return 2 + 0.52 * stages;
    const double rounds = (double)(int64_t)(tiles / 512), rest = tiles / 512 - rounds;
    return (rounds == 0 ? 1 : rest == 0 ? rounds : rounds + (rest < 0.21 ? 0.54 : rest + 0.33)) * (4.3 + 1.24 * stages);
}

// The 128x128 tile of so many.
int small_tile(double tiles) { return tiles <= 256 ? fl::kMx4Tile128Alone : fl::kMx4Tile128; }

LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, bool values) {
    LinearPlan p{};
    const int64_t blocks = blocks_of(K), stages = (blocks + 7) / 8;
    p.parts = 1;
    p.part_stages = (int)stages;
    p.stream = true;
    p.shape = {1, 1, 8};
    if (!M || !N) return p;
    if (!K) {
        p.stream = false;
        p.parts = 0;
        return p;
    }
    double least = 1e30;
    for (int mt = 1; mt <= 4 && M <= 512; mt *= 2)
        for (int nt = 1; nt <= 4; nt *= 2) {
            if (mt * nt == 4 && mt != nt) continue;  // 2 by 2 has their products with fewer rows
            if ((mt > 1 && M <= 8 * mt) || (M <= 2 && nt > 1)) continue;  // measured slower
            const double rounds = ceil_div(ceil_div(N, 16 * nt) * ceil_div(M, 16 * mt), 256);
            const double rows = M < 16 * mt ? M / 16.0 : mt;  // of A, in units of 16
            const double time = 3 + rounds * (0.3 * mt * nt + 0.25 * (rows + nt) * K / 1024);
            if (time < least) {
                least = time;
                p.shape = {mt, nt, 8};
            }
        }
    // a block to a CU: 1 by 4096x4096 4.2 us, 4.4 with eight waves; 69x235x15993 9.1, 9.5; but
    // two or three of them, 211x608x239, 6.6 and 4.4
    if (p.shape.mt == 1 && p.shape.nt == 1 && ceil_div(M, 16) * ceil_div(N, 16) <= 256) p.shape.waves = 16;
    for (int size : {fl::kMx4Tile256, fl::kMx4Tile128}) {
        const fl::Mx4TileShape &t = fl::kMx4TileShapes[size];
        const double tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn);
        for (int parts = 1; parts <= 16; ++parts) {
            const int64_t run = (stages + parts - 1) / parts;
            if (parts > 1 && (run < 2 || tiles * parts > 512 || (stages + run - 1) / run != parts)) continue;
            const double x = tiles * parts;
            const int v = size == fl::kMx4Tile256 ? size : small_tile(x);
            const double time = 3.4 + (parts > 1 ? 4 + parts * (double)M * N * 8 / 5e6 : 0) + tiles_time(v, x, run);
            if (time < least) {
                least = time;
                p.stream = false;
                p.variant = v;
                p.parts = parts;
                p.part_stages = (int)run;
            }
        }
    }
    const int64_t down = (M + 255) / 256, across = (N + 255) / 256, rounds = down * across / 256;
    const int64_t whole = rounds * 256 / down;  // columns of tiles that fill them
    if (whole > 0 && whole < across) {
        const double rest = ceil_div(M, 128) * ceil_div(N - whole * 256, 128);  // of the small ones
        const double time = 3.4 + tiles_time(fl::kMx4Tile256, whole * down, stages) + 2 +
                            tiles_time(small_tile(rest), rest, stages);
        if (time < least) {
            p.stream = false;
            p.variant = fl::kMx4Tile256;
            p.parts = 1;
            p.part_stages = (int)stages;
            p.first_columns = whole * 256;
        }
    }
    // Few values every block quantises for itself, which is less than another launch's 2.9 us
    // while 0.06 us for 1024 values past three times that, more where a CU has several blocks, are (16 by
    // 1024x1024 bf16 4.4 us, 6.6 with the launch; 8 by 4096x4096 6.0, 7.0; 12: 7.3, 7.3; 4 by
    // 14336x4096 9.4, 10.8; 8: 11.5, 11.1).
    const double on_a_cu = N > 4096 ? N / 4096.0 : 1;
    p.quantize = values && !(p.stream && p.shape.mt == 1 && M <= 16 &&
                             ((double)M * K / 1024 - 3) * (0.65 + 0.35 * on_a_cu) <= 42);
    if (p.quantize) {
        p.codes = (size_t)(M * blocks * 16);
        p.scales = align16((size_t)(M * blocks));
    }
    if (p.parts > 1) p.sums = (size_t)p.parts * M * N * 4;
    return p;
}

// The variant of the second launch, for the columns behind the first's.
int second_tile(const LinearPlan &p, int64_t M, int64_t N) {
    const fl::Mx4TileShape &t = fl::kMx4TileShapes[fl::kMx4Tile128];
    return small_tile(ceil_div(M, t.bm) * ceil_div(N - p.first_columns, t.bn));
}

size_t linear_bytes(const LinearPlan &p) { return p.codes + p.scales + p.sums; }

template <int DT>
void launch_linear(const LinearPlan &p, fl::Mx4LinearArgs l, uint8_t *ws, hipStream_t st) {
    if (p.quantize) {
        fl::Mx4Args q{};
        q.x = l.a_raw;
        q.codes = ws;
        q.scales = ws + p.codes;
        q.rows = l.M;
        q.K = l.K;
        q.blocks = l.blocks;
        launch_quantize<DT>(q, false, st);
        l.a_raw = nullptr;
        l.a_codes = q.codes;
        l.a_scales = q.scales;
    }
    if (p.stream) {
        fl::launch_mx4_stream<DT>(p.shape, l, st);
        return;
    }
    fl::Mx4TileArgs a{};
    a.l = l;
    a.part = reinterpret_cast<float *>(ws + p.codes + p.scales);
    a.parts = p.parts;
    a.part_stages = p.part_stages;
    if (p.parts == 0) return fl::launch_mx4_join<DT>(a, st);
    const auto launch = [&](int variant, int64_t from, int64_t to) {
        const fl::Mx4TileShape &t = fl::kMx4TileShapes[variant];
        a.n_from = from;
        a.tiles_m = (int)((l.M + t.bm - 1) / t.bm);
        a.tiles_n = (int)((to - from + t.bn - 1) / t.bn);
        fl::launch_mx4_tile<DT>(variant, a, st);
    };
    if (p.first_columns) {
        launch(p.variant, 0, p.first_columns);
        launch(second_tile(p, l.M, l.N), p.first_columns, l.N);
    } else {
        launch(p.variant, 0, l.N);
    }
}

fl_status check_linear(int64_t M, int64_t N, int64_t K, int dtype) {
    fl_status s = check_matrix(M, K, dtype);
    if (s != FL_OK || (s = check_matrix(N, K, dtype)) != FL_OK) return s;
    // 32-bit offsets: into 256 rows of codes (512 MiB at that K) and of the output; values are read by 64-bit ones
    if (K >= kLinearK || (size_t)N * elem_size(dtype) * 256 >= kTwoGiB)
        return fail(FL_ERR_UNSUPPORTED, "K or N too large (K must be below 2^22, 256 rows of out span < 2 GiB)");
    if (((N + 15) / 16) * ((M + 15) / 16) > kMaxDim)
        return fail(FL_ERR_UNSUPPORTED, "more than 2^31-1 tiles of 16x16 outputs");
    return FL_OK;
}

}  // namespace

extern "C" {

const char *fl_mx4_last_error(void) { return g_err; }

fl_status fl_quantize_mx4(const void *X, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, int32_t transposed,
                          fl_dtype dtype, void *stream) {
    clear_error();
    fl_status s = check_matrix(rows, K, dtype);
    if (s != FL_OK) return s;
    if (transposed != 0 && transposed != 1) return fail(FL_ERR_INVALID_ARG, "transposed must be 0 or 1");
    const size_t es = elem_size(dtype), blocks = (size_t)blocks_of(K);
    if ((s = check_operands({{"X", X, (size_t)rows * K * es, es, false, false, nullptr},
                             {"codes", codes, rows * blocks * 16, 16, true, false, nullptr},
                             {"scales", scales, rows * blocks, 1, true, false, nullptr}})) != FL_OK)
        return s;
    if (rows == 0 || K == 0) return FL_OK;
    fl::Mx4Args a{};
    a.x = X;
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.K = (int)K;
    a.blocks = (int)blocks;
    quantize(a, transposed, dtype, static_cast<hipStream_t>(stream));
    return check_launch("fl_quantize_mx4");
}

fl_status fl_dequantize_mx4(const uint8_t *codes, const uint8_t *scales, void *X, int64_t rows, int64_t K,
                            fl_dtype dtype, void *stream) {
    clear_error();
    fl_status s = check_matrix(rows, K, dtype);
    if (s != FL_OK) return s;
    const size_t es = elem_size(dtype), blocks = (size_t)blocks_of(K);
    if ((s = check_operands({{"codes", codes, rows * blocks * 16, 16, false, false, nullptr},
                             {"scales", scales, rows * blocks, 1, false, false, nullptr},
                             {"X", X, (size_t)rows * K * es, es, true, false, nullptr}})) != FL_OK)
        return s;
    if (rows == 0 || K == 0) return FL_OK;
    fl::Mx4Args a{};
    a.y = X;
    a.codes = const_cast<uint8_t *>(codes);
    a.scales = const_cast<uint8_t *>(scales);
    a.rows = rows;
    a.K = (int)K;
    a.blocks = (int)blocks;
    const dim3 grid = grid_of_units(a);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == FL_F32)
        hipLaunchKernelGGL((fl::dequantize_mx4_kernel<FL_F32>), grid, dim3(256), 0, st, a);
    else if (dtype == FL_F16)
        hipLaunchKernelGGL((fl::dequantize_mx4_kernel<FL_F16>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((fl::dequantize_mx4_kernel<FL_BF16>), grid, dim3(256), 0, st, a);
    return check_launch("fl_dequantize_mx4");
}

fl_status fl_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t values, fl_dtype dtype, size_t *bytes) {
    clear_error();
    fl_status s = check_linear(M, N, K, dtype);
    if (s != FL_OK) return s;
    if (values != 0 && values != 1) return fail(FL_ERR_INVALID_ARG, "values must be 0 or 1");
    if (!bytes) return fail(FL_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = linear_bytes(plan_linear(M, N, K, values));
    return FL_OK;
}

fl_status fl_mx4_linear_plan(int64_t M, int64_t N, int64_t K, int32_t values, fl_dtype dtype, fl_mx4_plan *plan) {
    clear_error();
    fl_status s = check_linear(M, N, K, dtype);
    if (s != FL_OK) return s;
    if (values != 0 && values != 1) return fail(FL_ERR_INVALID_ARG, "values must be 0 or 1");
    if (!plan) return fail(FL_ERR_INVALID_ARG, "plan is NULL");
    *plan = fl_mx4_plan{};
    plan->parts = 1;
    if (!M || !N || !K) return FL_OK;
    const LinearPlan p = plan_linear(M, N, K, values);
    plan->quantize = p.quantize ? 1 : values ? 2 : 0;
    plan->kernel = p.stream ? 1 : 2;
    if (p.stream) {
        plan->rows = 16 * p.shape.mt;
        plan->columns = 16 * p.shape.nt;
        plan->waves = p.shape.waves;
        return FL_OK;
    }
    const fl::Mx4TileShape &t = fl::kMx4TileShapes[p.variant];
    plan->rows = t.bm;
    plan->columns = t.bn;
    plan->waves = t.waves;
    plan->parts = p.parts;
    if ((plan->first_columns = p.first_columns)) {
        const fl::Mx4TileShape &u = fl::kMx4TileShapes[second_tile(p, M, N)];
        plan->second_rows = u.bm;
        plan->second_columns = u.bn;
        plan->second_waves = u.waves;
    }
    return FL_OK;
}

fl_status fl_fused_linear_mx4(const void *A, const uint8_t *A_scales, const uint8_t *B, const uint8_t *B_scales,
                              const void *bias, const void *Y, const void *R, void *out, int64_t M, int64_t N,
                              int64_t K, fl_act act, fl_dtype dtype, void *workspace, size_t workspace_bytes,
                              void *stream) {
    clear_error();
    fl_status s = check_linear(M, N, K, dtype);
    if (s != FL_OK) return s;
    if (act < FL_ACT_NONE || act > FL_ACT_GLU) return fail(FL_ERR_INVALID_ARG, "unknown activation %d", act);
    if (act == FL_ACT_GLU && !Y && M && N) return fail(FL_ERR_INVALID_ARG, "the gate needs Y");
    if (act != FL_ACT_GLU && Y) return fail(FL_ERR_INVALID_ARG, "Y is only used by the gate (FL_ACT_GLU)");
    const bool values = !A_scales;
    const LinearPlan plan = plan_linear(M, N, K, values);
    const size_t need = linear_bytes(plan);
    if (need && (!workspace || workspace_bytes < need))
        return fail(FL_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const size_t es = elem_size(dtype), blocks = (size_t)blocks_of(K), outs = (size_t)M * N * es;
    const bool live = M && N;  // nothing is read otherwise
    const void *same = out == Y ? Y : R;
    if ((s = check_operands({{"A", A, !live ? 0 : values ? (size_t)M * K * es : M * blocks * 16, values ? es : 16, false, false, nullptr},
                             {"A_scales", A_scales, live && !values ? M * blocks : 0, 1, false, false, nullptr},
                             {"B", B, live ? N * blocks * 16 : 0, 16, false, false, nullptr},
                             {"B_scales", B_scales, live ? N * blocks : 0, 1, false, false, nullptr},
                             {"bias", bias, live ? (size_t)N * es : 0, es, false, true, nullptr},
                             {"Y", Y, outs, es, false, true, nullptr},
                             {"R", R, outs, es, false, true, nullptr},
                             {"out", out, outs, es, true, false, same},
                             {"workspace", workspace, need, 16, true, true, nullptr}})) != FL_OK)
        return s;
    if (!live) return FL_OK;
    fl::Mx4LinearArgs a{};
    a.a_codes = values ? nullptr : static_cast<const uint8_t *>(A);
    a.a_scales = A_scales;
    a.a_raw = values && K ? A : nullptr;
    a.b_codes = B;
    a.b_scales = B_scales;
    a.bias = bias;
    a.Y = Y;
    a.R = R;
    a.out = out;
    a.M = M;
    a.N = N;
    a.K = (int)K;
    a.blocks = (int)blocks;
    a.act = act;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (dtype == FL_F32)
        launch_linear<FL_F32>(plan, a, ws, st);
    else if (dtype == FL_F16)
        launch_linear<FL_F16>(plan, a, ws, st);
    else
        launch_linear<FL_BF16>(plan, a, ws, st);
    return check_launch("fl_fused_linear_mx4");
}

}  // extern "C"
