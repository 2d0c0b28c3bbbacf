// The gated block in 16 bits: H = act(X Wg^T) (X Wu^T), fp32 sums, the activation and the
// product in fp32, one rounding. A tile's columns are half Wg's, half Wu's (phase_tile.h), so that a
// lane holds the two sums of an output: X goes through LDS once for both, and nothing but H
// (and G and U, each rounded once, where the backward pass is to have them) is written. 4096 x 10240 x 4096 in bf16 with G
// and U: 464 to 510 us by the card (1.3 to 1.5 PFLOP/s; the library's plain product of that size 433 to 453); one token 30.7 (168 MB, 5.5 TB/s).
#include "linear_device.h"

namespace mpg {

hipError_t launch_gated(int type, const Lin &p, const LinPlan &plan, hipStream_t stream) {
    return type == MPGEMM_TYPE_F16 ? lin_run<PtF16, _Float16, LIN_GATED>(p, plan, stream)
                                   : lin_run<PtBF16, __bf16, LIN_GATED>(p, plan, stream);
}

}  // namespace mpg
