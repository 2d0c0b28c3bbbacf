// Backward pass of the gated block H = act(G) U, G = X Wg^T, U = X Wu^T:
//   dG = dH U act'(G)    dU = dH act(G)          (one pass over dH, G and U)
//   dX = dG Wg + dU Wu = [dG, dU] [Wg; Wu]       (one product over 2 N)
//   [dWg; dWu] = [dG, dU]^T X                    (one product over M)
// dG and dU are held side by side in the operands' 16-bit type, as the matrix instruction takes them:
// one rounding each (half a step relative to the value), next to which the
// rounding of the results is as large. The weights and X enter across the axis that is summed and are
// transposed on their way out of LDS (ds_read_tr), so that no transposed copy of them is made.
#include "linear_device.h"

namespace mpg {

// 8 columns of a row per thread. Bound by memory: 10 bytes per element of dH.
template <typename T, int ACT>
__global__ __launch_bounds__(256) void gated_grads_kernel(GatedGrads p) {
    const int per_row = p.part / 8, parts = (per_row + 255) / 256;
    const int m = blockIdx.x / parts, n0 = ((blockIdx.x - m * parts) * 256 + (int)threadIdx.x) * 8;
    if (n0 >= p.part)
        return;
    typedef T eight __attribute__((ext_vector_type(8)));
    const T *dh = static_cast<const T *>(p.dh) + (int64_t)m * p.lddh, *g = static_cast<const T *>(p.g) + (int64_t)m * p.ldg,
            *u = static_cast<const T *>(p.u) + (int64_t)m * p.ldu;
    const bool vec = n0 + 8 <= p.N && lin_vec<T>(p.dh, p.lddh) && lin_vec<T>(p.g, p.ldg) && lin_vec<T>(p.u, p.ldu);
    eight vh = {}, vg = {}, vu = {};
    if (vec) {
        vh = *reinterpret_cast<const eight *>(dh + n0);
        vg = *reinterpret_cast<const eight *>(g + n0);
        vu = *reinterpret_cast<const eight *>(u + n0);
    } else {
#pragma unroll
        for (int d = 0; d < 8; ++d)
            if (n0 + d < p.N) {
                vh[d] = dh[n0 + d];
                vg[d] = g[n0 + d];
                vu[d] = u[n0 + d];
            }
    }
    eight a, b;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const float h = (float)vh[d], x = (float)vg[d];
        a[d] = (T)(h * (float)vu[d] * lin_slope<ACT>(x));
        b[d] = (T)(h * lin_act<ACT>(x));
    }
    T *o = static_cast<T *>(p.d) + (int64_t)m * 2 * p.part + n0;
    *reinterpret_cast<eight *>(o) = a;
    *reinterpret_cast<eight *>(o + p.part) = b;
}

template <typename T>
static void grads_type(const GatedGrads &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.M * (unsigned)((p.part / 8 + 255) / 256)), nt(256);
    if (p.act == MPGEMM_ACT_SILU)
        hipLaunchKernelGGL((gated_grads_kernel<T, MPGEMM_ACT_SILU>), grid, nt, 0, stream, p);
    else if (p.act == MPGEMM_ACT_GELU)
        hipLaunchKernelGGL((gated_grads_kernel<T, MPGEMM_ACT_GELU>), grid, nt, 0, stream, p);
    else
        hipLaunchKernelGGL((gated_grads_kernel<T, MPGEMM_ACT_GELU_TANH>), grid, nt, 0, stream, p);
}

hipError_t launch_gated_grads(int type, const GatedGrads &p, hipStream_t stream) {
    if (type == MPGEMM_TYPE_F16)
        grads_type<_Float16>(p, stream);
    else
        grads_type<__bf16>(p, stream);
    return hipGetLastError();
}

hipError_t launch_gated_dx(int type, const Lin &p, const LinPlan &plan, hipStream_t stream) {
    if (type == MPGEMM_TYPE_F16)
        lin_tile<PtF16, _Float16, LIN_DX>(p, plan, stream);
    else
        lin_tile<PtBF16, __bf16, LIN_DX>(p, plan, stream);
    return hipGetLastError();
}

hipError_t launch_gated_dw(int type, const Lin &p, const LinPlan &plan, hipStream_t stream) {
    if (type == MPGEMM_TYPE_F16)
        lin_tile<PtF16, _Float16, LIN_DW>(p, plan, stream);
    else
        lin_tile<PtBF16, __bf16, LIN_DW>(p, plan, stream);
    return hipGetLastError();
}

}  // namespace mpg
