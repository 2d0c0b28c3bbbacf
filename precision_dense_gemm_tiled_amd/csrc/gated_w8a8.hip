// The gated block in 8-bit integers: H = act((A Bg^T) sa sg) ((A Bu^T) sa su), both products of a
// tile in one workgroup (half of its columns are Bg's, half Bu's), so that a lane
// holds the two sums of an output and nothing but H is written.
#include "linear_device.h"

namespace mpg {

hipError_t launch_gated_w8a8(int type, const Lin &p, const LinPlan &plan, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return lin_run<PtI8, _Float16, LIN_GATED>(p, plan, stream);
    case MPGEMM_TYPE_BF16: return lin_run<PtI8, __bf16, LIN_GATED>(p, plan, stream);
    default: return lin_run<PtI8, float, LIN_GATED>(p, plan, stream);
    }
}

hipError_t launch_gated_w8a8_x(int type, const Lin &p, const LinX &x, const LinPlan &plan, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return lin_run_x<_Float16, LIN_GATED>(p, x, plan, stream);
    case MPGEMM_TYPE_BF16: return lin_run_x<__bf16, LIN_GATED>(p, x, plan, stream);
    default: return lin_run_x<float, LIN_GATED>(p, x, plan, stream);
    }
}

}  // namespace mpg
