// fl_grouped_inst.hip -- instantiates the experts' products for one dtype.
// Built once per dtype with -DFL_INST_DTYPE=<fl_dtype value>.
#include "fl_grouped.hpp"

#ifndef FL_INST_DTYPE
#error "define FL_INST_DTYPE"
#endif

namespace fl {
namespace {

template <int DT, int FORM, int ACT>
void launch_plain(const GroupedArgs &a, int64_t grid, hipStream_t s) {
    hipLaunchKernelGGL((grouped_plain_kernel<DT, FORM, ACT>), dim3((unsigned)grid), dim3(256), 0, s, a);
}

template <int DT, int FORM>
grouped_launcher pick_plain_act(int act) {
    switch (act) {
    case FL_ACT_NONE: return launch_plain<DT, FORM, FL_ACT_NONE>;
    case FL_ACT_RELU: return launch_plain<DT, FORM, FL_ACT_RELU>;
    case FL_ACT_GELU_TANH: return launch_plain<DT, FORM, FL_ACT_GELU_TANH>;
    default: return launch_plain<DT, FORM, FL_ACT_GLU>;
    }
}

}  // namespace

template <>
grouped_launcher pick_grouped_plain<FL_INST_DTYPE>(int form, int act) {
    constexpr int DT = FL_INST_DTYPE;
    if (form == kFormFwd) return pick_plain_act<DT, kFormFwd>(act);
    if (form == kFormBwd) return pick_plain_act<DT, kFormBwd>(act);
    return launch_plain<DT, kFormGrad, FL_ACT_NONE>;
}

}  // namespace fl
