// fl_norm.hip -- host side of the C ABI declared in include/fused_norm.h:
// argument validation, the choice of kernels and their launches on the
// caller's stream.  Device code is in fl_norm.hpp.
#include <math.h>

#include "fl_check.hpp"
#include "fl_norm.hpp"
#include "fused_norm.h"

namespace {

constexpr int kBwdBlocks = 512;  // of 512 threads, two of which a CU holds
constexpr int64_t kGridMax = 1 << 20;

fl_status check_norm(int64_t M, int64_t H, int dtype) {
    fl_status s = check_dtype(dtype);
    if (s != FL_OK) return s;
    return check_sizes({M, H});
}

int64_t pieces_of(int64_t H, int dtype) { return dtype == FL_F32 ? (H + 3) / 4 : (H + 7) / 8; }

template <int DT, int TEAM, int NV>
void launch_fwd(const fl::NormArgs &a, hipStream_t st) {
    constexpr int threads = TEAM > 256 ? TEAM : 256, teams = threads / TEAM;
    const int64_t blocks = (a.M + teams - 1) / teams;
    hipLaunchKernelGGL((fl::layer_norm_kernel<DT, TEAM, NV>), dim3((unsigned)(blocks < kGridMax ? blocks : kGridMax)),
                       dim3(threads), 0, st, a);
}

// The smallest team whose lanes hold the row in 16 to 64 bytes each, 128 where it
// takes many: rows of 1024 bf16 take 11.6 us with 64 lanes and 21.4 with 256
// (16384 rows), of 2048 21.9 and 22.9, of 4096 40.6 and 38.6; 256 columns 11.6 with 16
// lanes, 19.5 with 64 (65536 rows).  Few rows do not fill the chip, and a lane's share
// is what they wait for: 1725 bf16 take 3.0 us with 256 lanes and 3.6 with 64 (8 to 256
// rows), 4.3 and 4.2 (1024).  1024 lanes for longer ones do not help: 8 rows of 8192 bf16 3.6
// us both ways, 512 4.7 and 5.2; of 16384 4.5 with 256, 4.3 with 1024, 6.1 and 6.5.
template <int DT>
void launch_fwd_dt(const fl::NormArgs &a, hipStream_t st) {
    const int64_t p = pieces_of(a.H, DT);
    if (p <= 16)
        launch_fwd<DT, 16, 1>(a, st);
    else if (p <= 32)
        launch_fwd<DT, 16, 2>(a, st);
    else if (p <= 64)
        launch_fwd<DT, 64, 1>(a, st);
    else if (p <= 128)
        launch_fwd<DT, 64, 2>(a, st);
    else if (p <= 256 && a.M <= 512)
        launch_fwd<DT, 256, 1>(a, st);
    else if (p <= 256)
        launch_fwd<DT, 64, 4>(a, st);
    else if (p <= 512)
        launch_fwd<DT, 256, 2>(a, st);
    else if (p <= 1024)
        launch_fwd<DT, 256, 4>(a, st);
    else if (p <= 2048)
        launch_fwd<DT, 256, 8>(a, st);
    else if (p <= 4096)
        launch_fwd<DT, 1024, 4>(a, st);
    else
        hipLaunchKernelGGL((fl::layer_norm_long_kernel<DT>), dim3((unsigned)(a.M < kGridMax ? a.M : kGridMax)),
                           dim3(1024), 0, st, a);
}

// The team of the backward kernel, and its blocks where they keep sums: each
// leaves a row of partial sums (8 H bytes), so no more of them than are resident
// at once (16384x4096 bf16: 512 or, of 1024 lanes, 256), half as many where a team has
// fewer than four rows (1024x4096 bf16 13 us, 18 with 512 blocks; 4096x1000 9.6, 11.1),
// and a block for a team's row each where they are fewer still (512x4096 11.4 us).  Teams of
// 1024 lanes, of which a CU holds one: 256x8192 13.4 us, 15.4 with all 256 blocks, 256x16384
// 19.2 and 23.3, 512 24.0 and 24.3; from there on all would be better, 768 27.3 and 25.9,
// 1023 31.3 and 28.5.  The
// rows of two blocks are left to one, and those of three, which needs no join: 4x4096
// bf16 7.3 us, 8.2 with it, 6x4096 8.7 and 8.2, and 3.4 of the host's time.
// The sums of a lane take two registers an element, so teams are larger than the
// forward's: 2048 columns 55 us with 256 lanes, 66 with 64; 512 columns 29 us with 64
// lanes, 75 with 256.  Up to 2048 rows of 216 bf16 take 64 lanes with half of the sums each
// (128 rows 5.5 us, 7.0 with 16 lanes; 2048: 6.5, 7.7; 8192: 9.2, 8.4).
struct BwdShape {
    int team, nv, blocks;  // team 0: the long kernels
};

BwdShape bwd_shape(int64_t M, int64_t H, int dtype) {
    const int64_t p = pieces_of(H, dtype);
    BwdShape b{};
    if (p <= 16 || (p <= 32 && M > 2048))
        b = {16, p <= 16 ? 1 : 2, 0};
    else if (p <= 128)
        b = {64, p <= 64 ? 1 : 2, 0};
    else if (p <= 512)
        b = {256, p <= 256 ? 1 : 2, 0};
    else if (p <= 2048)
        b = {1024, p <= 1024 ? 1 : 2, 0};
    else if (p <= 4096 && dtype == FL_F32)
        b = {1024, 4, 0};
    const int64_t rows = b.team && b.team < 512 ? 512 / b.team : 1;  // of a block at once
    const int64_t blocks = (M + rows - 1) / rows, most = b.team == 1024 ? kBwdBlocks / 2 : kBwdBlocks;
    b.blocks = blocks <= 3 ? 1 : (int)(blocks < most / 2 ? blocks : blocks < most * 4 ? most / 2 : most);
    return b;
}

// sums: whether the weight's or the bias's gradient is asked for.
size_t bwd_bytes(int64_t M, int64_t H, int dtype, bool sums) {
    if (M == 0 || H == 0) return 0;
    const BwdShape b = bwd_shape(M, H, dtype);
    const size_t part = sums && b.blocks > 1 ? (size_t)b.blocks * 2 * H * 4 : 0;
    return b.team ? part : part + (size_t)M * 8;
}

template <int DT, int TEAM, int NV>
void launch_bwd(const fl::NormArgs &a, int blocks, bool sums, hipStream_t st) {
    constexpr int threads = TEAM > 512 ? TEAM : 512;
    if (sums) {
        hipLaunchKernelGGL((fl::layer_norm_bwd_kernel<DT, TEAM, NV, true>), dim3(blocks), dim3(threads), 0, st, a);
    } else {
        const int64_t all = (a.M + threads / TEAM - 1) / (threads / TEAM);
        hipLaunchKernelGGL((fl::layer_norm_bwd_kernel<DT, TEAM, NV, false>),
                           dim3((unsigned)(all < kGridMax ? all : kGridMax)), dim3(threads), 0, st, a);
    }
}

template <int DT>
void launch_bwd_dt(const fl::NormArgs &a, const BwdShape &b, bool sums, float *c, hipStream_t st) {
    if (b.team == 0) {
        const int64_t rows = a.M < kGridMax ? a.M : kGridMax;
        hipLaunchKernelGGL((fl::layer_norm_bwd_long_kernel<DT>), dim3((unsigned)rows), dim3(1024), 0, st, a, c);
        const int64_t cols = (pieces_of(a.H, DT) + 255) / 256;
        hipLaunchKernelGGL((fl::layer_norm_bwd_columns_kernel<DT>), dim3((unsigned)cols, (unsigned)b.blocks), dim3(256),
                           0, st, a, c);
    }
#define FL_BWD(t, n) else if (b.team == t && b.nv == n) launch_bwd<DT, t, n>(a, b.blocks, sums, st)
    FL_BWD(16, 1);
    FL_BWD(16, 2);
    FL_BWD(64, 1);
    FL_BWD(64, 2);
    FL_BWD(256, 1);
    FL_BWD(256, 2);
    FL_BWD(1024, 1);
    FL_BWD(1024, 2);
    else if constexpr (DT == FL_F32) launch_bwd<DT, 1024, 4>(a, b.blocks, sums, st);
#undef FL_BWD
}

}  // namespace

extern "C" {

const char *fl_norm_last_error(void) { return g_err; }

fl_status fl_layer_norm(const void *X, const void *weight, const void *bias, void *Y, float *mean, float *rstd,
                        int64_t M, int64_t H, float eps, fl_dtype dtype, void *stream) {
    clear_error();
    fl_status s = check_norm(M, H, dtype);
    if (s != FL_OK) return s;
    if (!(eps >= 0.0f) || isinf(eps)) return fail(FL_ERR_INVALID_ARG, "eps (%g) must be finite and not negative", eps);
    const size_t es = elem_size(dtype), rows = (size_t)M * H * es, stats = H ? (size_t)M * 4 : 0;
    if ((s = check_operands({{"X", X, rows, es, false, false, nullptr},
                             {"weight", weight, (size_t)H * es, es, false, true, nullptr},
                             {"bias", bias, (size_t)H * es, es, false, true, nullptr},
                             {"Y", Y, rows, es, true, false, X},
                             {"mean", mean, stats, 4, true, true, nullptr},
                             {"rstd", rstd, stats, 4, true, true, nullptr}})) != FL_OK)
        return s;
    if (M == 0 || H == 0) return FL_OK;
    fl::NormArgs a{};
    a.x = X;
    a.weight = weight;
    a.bias = bias;
    a.y = Y;
    a.mean = mean;
    a.rstd = rstd;
    a.M = M;
    a.H = (int)H;
    a.eps = eps;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == FL_F32)
        launch_fwd_dt<FL_F32>(a, st);
    else if (dtype == FL_F16)
        launch_fwd_dt<FL_F16>(a, st);
    else
        launch_fwd_dt<FL_BF16>(a, st);
    return check_launch("fl_layer_norm");
}

fl_status fl_layer_norm_bwd_workspace_bytes(int64_t M, int64_t H, fl_dtype dtype, size_t *bytes) {
    clear_error();
    fl_status s = check_norm(M, H, dtype);
    if (s != FL_OK) return s;
    if (!bytes) return fail(FL_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = bwd_bytes(M, H, dtype, true);
    return FL_OK;
}

fl_status fl_layer_norm_bwd(const void *dY, const void *X, const void *weight, const float *mean, const float *rstd,
                            const void *R, void *dX, float *dweight, float *dbias, int64_t M, int64_t H,
                            fl_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    fl_status s = check_norm(M, H, dtype);
    if (s != FL_OK) return s;
    const bool sums = dweight || dbias;
    const size_t need = bwd_bytes(M, H, dtype, sums);
    if (need && (!workspace || workspace_bytes < need))
        return fail(FL_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const size_t es = elem_size(dtype), rows = (size_t)M * H * es, stats = H ? (size_t)M * 4 : 0;
    // dX may be any of the three operands of its shape
    const void *same = dX == dY ? dY : dX == X ? X : R;
    if ((s = check_operands({{"dY", dY, rows, es, false, false, nullptr},
                             {"X", X, rows, es, false, false, nullptr},
                             {"weight", weight, (size_t)H * es, es, false, true, nullptr},
                             {"mean", mean, stats, 4, false, false, nullptr},
                             {"rstd", rstd, stats, 4, false, false, nullptr},
                             {"R", R, rows, es, false, true, nullptr},
                             {"dX", dX, rows, es, true, false, same},
                             {"dweight", dweight, (size_t)H * 4, 4, true, true, nullptr},
                             {"dbias", dbias, (size_t)H * 4, 4, true, true, nullptr},
                             {"workspace", workspace, need, 16, true, true, nullptr}})) != FL_OK)
        return s;
    if (H == 0) return FL_OK;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    fl::NormArgs a{};
    a.H = (int)H;
    a.dweight = dweight;
    a.dbias = dbias;
    if (M == 0) {
        if (!dweight && !dbias) return FL_OK;
        hipLaunchKernelGGL(fl::zero_columns_kernel, dim3((unsigned)((H + 255) / 256)), dim3(256), 0, st, a);
        return check_launch("fl_layer_norm_bwd");
    }
    a.x = X;
    a.weight = weight;
    a.y = dX;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dy = dY;
    a.residual = R;
    a.M = M;
    const BwdShape b = bwd_shape(M, H, dtype);
    const bool join = sums && b.blocks > 1;
    a.part = join ? static_cast<float *>(workspace) : nullptr;
    float *c = b.team ? nullptr : static_cast<float *>(workspace) + (join ? (size_t)b.blocks * 2 * H : 0);
    if (dtype == FL_F32)
        launch_bwd_dt<FL_F32>(a, b, sums, c, st);
    else if (dtype == FL_F16)
        launch_bwd_dt<FL_F16>(a, b, sums, c, st);
    else
        launch_bwd_dt<FL_BF16>(a, b, sums, c, st);
    if (join) {
        const int64_t cols = (H + 31) / 32, across = cols < kGridMax ? cols : kGridMax;
        hipLaunchKernelGGL(fl::column_join_kernel, dim3((unsigned)across, 2, (unsigned)((cols + across - 1) / across)),
                           dim3(1024), 0, st, a, b.blocks);
    }
    return check_launch("fl_layer_norm_bwd");
}

}  // extern "C"
