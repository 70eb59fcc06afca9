// fl_mx4_inst.hip -- the 4-bit linear layer's kernels for one type (FL_INST_DTYPE)
// of bias, Y, R, output and values of A.
#include "fl_mx4_tile.hpp"

namespace fl {

namespace {

template <int DT, int MT, int NT, int WAVES, bool VALUES>
void launch_stream_of(const Mx4LinearArgs &l, hipStream_t st) {
    // the largest panel whose scales (and codes of A's values) take 48 KB
    const int64_t rows = VALUES ? l.M : 16 * MT, all = (l.blocks + 15) / 16 * 16;
    int64_t panel = 256;
    auto code_pitch = [&](int64_t n) { return VALUES ? (n < all ? n : all) * 16 + 16 : 0; };
    auto bytes = [&](int64_t n) {
        return 16 * NT * (n + kMx4ScalePad) + rows * (n + kMx4ScalePad) + rows * code_pitch(n);
    };
    while (panel < l.blocks && bytes(panel + 256) <= 49152) panel += 256;
    const int64_t sums = (int64_t)WAVES * MT * NT * 1024, lds = bytes(panel) > sums ? bytes(panel) : sums;
    const dim3 grid((unsigned)(((l.N + 16 * NT - 1) / (16 * NT)) * ((l.M + 16 * MT - 1) / (16 * MT))));
    hipLaunchKernelGGL((mx4_stream_kernel<DT, MT, NT, WAVES, VALUES>), grid, dim3(64 * WAVES), (size_t)lds, st,
                       Mx4StreamArgs{l, (int)panel, (int)code_pitch(panel)});
}

template <int DT, int MI, int NI, int WM, int WN, int PER_CU, int RING>
void launch_tile(const Mx4TileArgs &a, hipStream_t st) {
    constexpr size_t lds = Mx4Tile<DT, MI, NI, WM, WN, RING>::LDS;
    hipLaunchKernelGGL((mx4_tile_kernel<DT, MI, NI, WM, WN, PER_CU, RING>),
                       dim3((unsigned)(a.tiles_m * a.tiles_n) * (unsigned)a.parts), dim3(64 * WM * WN),
                       lds, st, a);
}

}  // namespace

template <>
void launch_mx4_stream<FL_INST_DTYPE>(const Mx4StreamShape &shape, const Mx4LinearArgs &a, hipStream_t st) {
    constexpr int DT = FL_INST_DTYPE;
    if (a.a_raw) {
        if (shape.waves == 16) return launch_stream_of<DT, 1, 1, 16, true>(a, st);
        return shape.nt == 1 ? launch_stream_of<DT, 1, 1, 8, true>(a, st) : launch_stream_of<DT, 1, 2, 8, true>(a, st);
    }
    if (shape.waves == 16) return launch_stream_of<DT, 1, 1, 16, false>(a, st);
#define FL_STREAM(m, n) \
    if (shape.mt == m && shape.nt == n) return launch_stream_of<DT, m, n, 8, false>(a, st)
    FL_STREAM(1, 1);
    FL_STREAM(1, 2);
    FL_STREAM(2, 1);
    FL_STREAM(2, 2);
    FL_STREAM(2, 4);
    FL_STREAM(4, 2);
    FL_STREAM(4, 4);
#undef FL_STREAM
}

template <>
void launch_mx4_join<FL_INST_DTYPE>(const Mx4TileArgs &a, hipStream_t st) {
    const int64_t blocks = ((a.l.N + 3) / 4 * a.l.M + 255) / 256, across = blocks < 1 << 20 ? blocks : 1 << 20;
    hipLaunchKernelGGL((mx4_join_kernel<FL_INST_DTYPE>), dim3((unsigned)across, (unsigned)((blocks + across - 1) / across)),
                       dim3(256), 0, st, a);
}

template <>
void launch_mx4_tile<FL_INST_DTYPE>(int variant, const Mx4TileArgs &a, hipStream_t st) {
    constexpr int DT = FL_INST_DTYPE;
    if (variant == kMx4Tile256)
        launch_tile<DT, 8, 4, 2, 4, 1, 2>(a, st);
    else if (variant == kMx4Tile128)
        launch_tile<DT, 4, 4, 2, 2, 2, 2>(a, st);
    else
        launch_tile<DT, 2, 4, 4, 2, 1, 4>(a, st);
    if (a.parts > 1) launch_mx4_join<DT>(a, st);
}

}  // namespace fl
