// Backward pass of the gated block H = act(G) U, G = X Wg^T, U = X Wu^T:
//   dG = dH U act'(G)    dU = dH act(G)          (one pass over dH, G and U)
//   dX = dG Wg + dU Wu = [dG, dU] [Wg; Wu]       (one product over 2 N)
//   [dWg; dWu] = [dG, dU]^T X                    (one product over M)
// dG and dU are held side by side in the operands' 16-bit type, as the matrix instruction takes them:
// one rounding each (half a step relative to the value, in fp16 within that type's range), next to which the
// rounding of the results is as large. The weights and X enter across the axis that is summed and are
// transposed on their way out of LDS (ds_read_tr), so that no transposed copy of them is made.
#include "linear_device.h"

namespace mpg {

// 8 columns of a row per thread, 2^lx threads side by side in a row (a power of two: no division by a
// row's pieces), the rest of the workgroup's 256 over rows. Bound by memory: 10 bytes per element of dH, 4096 x 10240 in 63 us
// (6.7 TB/s, some of it from the last level of cache). Rows that are not at multiples of 16 bytes are read by the element (4096 x
// 10241: the whole backward pass with K = 4096 takes 1215 us, with padded rows 1085).
template <typename T, int ACT>
__global__ __launch_bounds__(256) void gated_grads_kernel(GatedGrads p, int lx) {
    const int parts = (p.part / 8 + (1 << lx) - 1) >> lx, rb = blockIdx.x / parts;
    const int m = rb * (256 >> lx) + (threadIdx.x >> lx);
    const int n0 = (((blockIdx.x - rb * parts) << lx) + (threadIdx.x & ((1 << lx) - 1))) * 8;
    if (n0 >= p.part || m >= p.M)
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
    int lx = 3;   // (part is a multiple of 64)
    while (lx < 8 && p.part / 8 % (2 << lx) == 0)
        ++lx;
    const int rows = 256 >> lx;
    const dim3 grid((unsigned)((p.M + rows - 1) / rows) * (unsigned)((p.part / 8) >> lx)), nt(256);
    if (p.act == MPGEMM_ACT_SILU)
        hipLaunchKernelGGL((gated_grads_kernel<T, MPGEMM_ACT_SILU>), grid, nt, 0, stream, p, lx);
    else if (p.act == MPGEMM_ACT_GELU)
        hipLaunchKernelGGL((gated_grads_kernel<T, MPGEMM_ACT_GELU>), grid, nt, 0, stream, p, lx);
    else
        hipLaunchKernelGGL((gated_grads_kernel<T, MPGEMM_ACT_GELU_TANH>), grid, nt, 0, stream, p, lx);
}

hipError_t launch_gated_grads(int type, const GatedGrads &p, hipStream_t stream) {
    if (type == MPGEMM_TYPE_F16)
        grads_type<_Float16>(p, stream);
    else
        grads_type<__bf16>(p, stream);
    return hipGetLastError();
}

// Both products in one grid, first the tiles of dX, whose sums are longer: dW's run beside them and
// a launch less is waited for (777 x 1000 x 520, f16: 22.0 us, in two launches 28.6). Bound by the
// matrix units' power like the forward pass: 4096 x 10240 x 4096 in bf16 940 to 1000 us for 1374 GFLOP (the library's two
// products, one with its right operand and one with both across k, 519 and 613), behind 63 us of gated_grads_kernel.
template <class E, typename OUT, int BM, int BN, int WGM, int WGN, int NS>
__global__ __launch_bounds__(64 * WGM * WGN) void gated_pair_kernel(Lin dx, Lin dw, int first) {
    typedef LinTile<E, OUT, LIN_DX, BM, BN, WGM, WGN, NS> X;
    typedef LinTile<E, OUT, LIN_DW, BM, BN, WGM, WGN, NS> W;
    static_assert(X::PT::LDS_BYTES == W::PT::LDS_BYTES, "one buffer");
    __shared__ __attribute__((aligned(16))) uint8_t smem[X::PT::LDS_BYTES];
    if ((int)blockIdx.x < first)
        X::run(dx, blockIdx.x, first, smem);
    else
        W::run(dw, blockIdx.x - first, gridDim.x - first, smem);
}

template <class E, typename OUT, int BM, int BN, int WGM, int WGN, int NS>
static void pair_one(const Lin &dx, const Lin &dw, hipStream_t stream) {
    typedef LinTile<E, OUT, LIN_DX, BM, BN, WGM, WGN, NS> X;
    typedef LinTile<E, OUT, LIN_DW, BM, BN, WGM, WGN, NS> W;
    const int first = X::tiles_m(dx) * X::tiles_n(dx);
    hipLaunchKernelGGL((gated_pair_kernel<E, OUT, BM, BN, WGM, WGN, NS>), dim3((unsigned)first + (unsigned)W::tiles_m(dw) * (unsigned)W::tiles_n(dw)),
                       dim3(64 * WGM * WGN), 0, stream, dx, dw, first);
}

template <class E, typename OUT>
static hipError_t pair_type(const Lin &dx, const Lin &dw, const LinPlan &plan, hipStream_t stream) {
    switch (plan.cfg) {
    case 0: pair_one<E, OUT, 256, 256, 2, 4, 2>(dx, dw, stream); break;
    case 1: pair_one<E, OUT, 128, 128, 2, 2, 2>(dx, dw, stream); break;
    default: pair_one<E, OUT, 64, 64, 2, 2, 4>(dx, dw, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_gated_pair(int type, const Lin &dx, const Lin &dw, const LinPlan &plan, hipStream_t stream) {
    return type == MPGEMM_TYPE_F16 ? pair_type<PtF16, _Float16>(dx, dw, plan, stream) : pair_type<PtBF16, __bf16>(dx, dw, plan, stream);
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
