// fl_grouped_inst.hip -- instantiates the experts' products for one dtype and
// one form (and the join of parts, and with the gradient the column sum).  Built once per dtype and
// form with -DFL_INST_DTYPE=<fl_dtype value> -DFL_INST_FORM=<form>.
#include "fl_grouped_dma.hpp"

#if !defined(FL_INST_DTYPE) || !defined(FL_INST_FORM)
#error "define FL_INST_DTYPE and FL_INST_FORM"
#endif

namespace fl {

template <int BM, int BN, int WM, int WN, int NBUF, int OCC, bool NT>
static void launch(const GroupedArgs &a, int act, int64_t grid, hipStream_t s) {
    hipLaunchKernelGGL((grouped_dma_kernel<FL_INST_DTYPE, FL_INST_FORM, BM, BN, WM, WN, NBUF, OCC, NT>),
                       dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, a, act);
}

template <int BM, int BN, int WM, int WN, int NBUF, int OCC>
static grouped_launcher low(bool nt) {
    return nt ? launch<BM, BN, WM, WN, NBUF, OCC, true> : launch<BM, BN, WM, WN, NBUF, OCC, false>;
}

template <>
grouped_launcher pick_grouped<FL_INST_DTYPE, FL_INST_FORM>(int variant, bool nt) {
#if FL_INST_FORM == 2  // (every operand is read by several tiles)
#if FL_INST_DTYPE == 0
    return launch<64, 64, 2, 2, 3, 3, false>;
#else
    if (variant == kTile256x256) return launch<256, 256, 2, 4, 2, 1, false>;
    return launch<128, 128, 2, 2, 2, 2, false>;
#endif
#elif FL_INST_DTYPE == 0
    if (variant == kTileF32x32) return low<32, 64, 2, 2, 3, 4>(nt);
    return low<64, 64, 2, 2, 3, 3>(nt);
#else
    if (variant == kTile256x256) return launch<256, 256, 2, 4, 2, 1, false>;
    if (variant == kTile256x128) return launch<256, 128, 4, 2, 3, 1, false>;
    if (variant == kTile64x256) return low<64, 256, 2, 4, 4, 1>(nt);
    if (variant == kTile32x128) return low<32, 128, 1, 4, 4, 2>(nt);
    return launch<128, 128, 2, 2, 2, 2, false>;
#endif
}

#if FL_INST_FORM == 2
template <>
void launch_column_sum<FL_INST_DTYPE>(const GroupedArgs &a, hipStream_t s) {
    // (a dimension of a launch has less than 2^32 threads: not both in one)
    const dim3 grid((unsigned)((a.N + kColumns - 1) / kColumns), (unsigned)a.E);
    hipLaunchKernelGGL((grouped_column_sum_kernel<FL_INST_DTYPE>), grid, dim3(1024), 0, s, a);
}
#endif

#if FL_INST_FORM != 1
template <>
void launch_join<FL_INST_DTYPE, FL_INST_FORM>(const GroupedArgs &a, int act, hipStream_t s) {
    const unsigned rows = FL_INST_FORM == 2 ? (unsigned)((int64_t)a.E * a.K) : (unsigned)a.S;
    hipLaunchKernelGGL((grouped_join_kernel<FL_INST_DTYPE, FL_INST_FORM>), dim3(rows, (a.N + 1023) / 1024), dim3(256), 0,
                       s, a, act);
}
#endif

}  // namespace fl
