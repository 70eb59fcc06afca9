// fl_mx4_inst.hip -- the 4-bit linear layer's kernels for one type (FL_INST_DTYPE)
// of bias, Y, R, output and values of A.
#include "fl_mx4_tile.hpp"

namespace fl {

namespace {

template <int DT, int MT, int NT, int WAVES, int U>
void launch_stream(const Mx4LinearArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)(((a.N + 16 * NT - 1) / (16 * NT)) * ((a.M + 16 * MT - 1) / (16 * MT))));
    if (a.a_raw)
        hipLaunchKernelGGL((mx4_stream_kernel<DT, MT, NT, WAVES, U, true>), grid, dim3(64 * WAVES), 0, st, a);
    else
        hipLaunchKernelGGL((mx4_stream_kernel<DT, MT, NT, WAVES, U, false>), grid, dim3(64 * WAVES), 0, st, a);
}

template <int DT, int MI, int NI, int WM, int WN, int PER_CU>
void launch_tile(const Mx4TileArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((mx4_tile_kernel<DT, MI, NI, WM, WN, PER_CU>),
                       dim3((unsigned)(a.tiles_m * a.tiles_n) * (unsigned)a.parts), dim3(64 * WM * WN), 0, st, a);
}

}  // namespace

template <>
void launch_mx4_stream<FL_INST_DTYPE>(int variant, const Mx4LinearArgs &a, hipStream_t st) {
    constexpr int DT = FL_INST_DTYPE;
    (void)variant;
    launch_stream<DT, 1, 1, 4, 2>(a, st);
}

template <>
void launch_mx4_tile<FL_INST_DTYPE>(int variant, const Mx4TileArgs &a, hipStream_t st) {
    constexpr int DT = FL_INST_DTYPE;
    if (variant == kMx4Tile256)
        launch_tile<DT, 8, 4, 2, 4, 1>(a, st);
    else
        launch_tile<DT, 4, 4, 2, 2, 2>(a, st);
    if (a.parts > 1) {
        const int64_t quads = (a.l.N + 3) / 4 * a.l.M;
        hipLaunchKernelGGL((mx4_join_kernel<DT>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, a);
    }
}

}  // namespace fl
