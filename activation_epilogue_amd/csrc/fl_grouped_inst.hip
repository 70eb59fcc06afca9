// fl_grouped_inst.hip -- instantiates the column sum for one dtype, and for
// fp32 the experts' products (16-bit operands: fl_grouped_dma_inst.hip).
// Built once per dtype with -DFL_INST_DTYPE=<fl_dtype value>.
#include "fl_grouped.hpp"

#ifndef FL_INST_DTYPE
#error "define FL_INST_DTYPE"
#endif

namespace fl {

#if FL_INST_DTYPE == 0
template <int FORM, int ACT>
static void launch_f32(const GroupedArgs &a, int64_t grid, hipStream_t s) {
    hipLaunchKernelGGL((grouped_f32_kernel<FORM, ACT>), dim3((unsigned)grid), dim3(256), 0, s, a);
}

template <int FORM>
static grouped_launcher pick_act(int act) {
    switch (act) {
    case FL_ACT_NONE: return launch_f32<FORM, FL_ACT_NONE>;
    case FL_ACT_RELU: return launch_f32<FORM, FL_ACT_RELU>;
    case FL_ACT_GELU_TANH: return launch_f32<FORM, FL_ACT_GELU_TANH>;
    default: return launch_f32<FORM, FL_ACT_GLU>;
    }
}

grouped_launcher pick_grouped_f32(int form, int act) {
    if (form == kFormFwd) return pick_act<kFormFwd>(act);
    if (form == kFormBwd) return pick_act<kFormBwd>(act);
    return launch_f32<kFormGrad, FL_ACT_NONE>;
}
#endif

template <>
void launch_column_sum<FL_INST_DTYPE>(const GroupedArgs &a, hipStream_t s) {
    const unsigned blocks = (unsigned)a.E * (unsigned)((a.N + kColumns - 1) / kColumns);
    hipLaunchKernelGGL((grouped_column_sum_kernel<FL_INST_DTYPE>), dim3(blocks), dim3(256), 0, s, a);
}

}  // namespace fl
