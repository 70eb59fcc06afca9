// fl_grouped_dma_inst.hip -- instantiates the experts' products on direct-to-LDS
// tiles for one 16-bit dtype and one form.  Built once per dtype and form with
// -DFL_INST_DTYPE=<fl_dtype value> -DFL_INST_FORM=<form>.
#include "fl_grouped_dma.hpp"

#if !defined(FL_INST_DTYPE) || !defined(FL_INST_FORM)
#error "define FL_INST_DTYPE and FL_INST_FORM"
#endif

namespace fl {

template <int DT, int FORM, int BM, int BN, int WM, int WN, int NBUF, int OCC>
static void launch_dma(const GroupedArgs &a, int act, int64_t grid, hipStream_t s) {
    hipLaunchKernelGGL((grouped_dma_kernel<DT, FORM, BM, BN, WM, WN, NBUF, OCC>), dim3((unsigned)grid),
                       dim3(64 * WM * WN), 0, s, a, act);
}

template <>
grouped_dma_launcher pick_grouped_dma_form<FL_INST_DTYPE, FL_INST_FORM>(int variant) {
    constexpr int DT = FL_INST_DTYPE, FORM = FL_INST_FORM;
    if (variant == kTile256x256) return launch_dma<DT, FORM, 256, 256, 2, 4, 2, 1>;
    if (variant == kTile128x128) return launch_dma<DT, FORM, 128, 128, 2, 2, 2, 2>;
    if constexpr (FORM != kFormGrad) {
        if (variant == kTile256x128) return launch_dma<DT, FORM, 256, 128, 4, 2, 3, 1>;
        if (variant == kTile64x128) return launch_dma<DT, FORM, 64, 128, 1, 4, 3, 2>;
        if (variant == kTile32x128) return launch_dma<DT, FORM, 32, 128, 1, 4, 4, 2>;
    }
    return nullptr;
}

}  // namespace fl
