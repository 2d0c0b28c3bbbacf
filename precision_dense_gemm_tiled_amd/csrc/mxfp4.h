// Internal interface of the MXFP4 kernels (quantisation, product). Arguments
// reaching these launchers have already been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mpgemm.h"

namespace mpg {

// Quantisation of X (M x K, MPGEMM_TYPE_*, row stride ldx elements) along rows
// (q, s), columns (qt, st) or both; strides of codes and scales in bytes.
struct MxQuantize {
    const void *x;
    int64_t ldx;
    uint8_t *q, *s, *qt, *st;
    int64_t ldq, lds, ldqt, ldst;
    int M, K;
};
hipError_t launch_mx_quantize(int type, const MxQuantize &p, hipStream_t stream);

struct MxDequantize {
    const uint8_t *q, *s;
    void *y;
    int64_t ldq, lds, ldy;
    int M, K;
};
hipError_t launch_mx_dequantize(int type, const MxDequantize &p, hipStream_t stream);

// C = A B^T + bias with both operands in MXFP4: nb blocks of 32 per row.
struct MxGemm {
    const uint8_t *a, *sa, *b, *sb;
    int64_t lda, ldsa, ldb, ldsb;   // bytes
    const void *bias;               // N values of the result's type, or null
    void *c;
    int64_t ldc;                    // elements
    int M, N, nb;
};

// The same with A quantised in the kernel from X (K elements per row).
struct MxSkinnyX {
    const void *x;
    int64_t ldx;
    int K;
    int rlog;   // set by the launcher: log2 of the rows held per block, at least M
};

// What a product runs, decided from the sizes alone.
enum MxKind { MX_SKINNY = 0, MX_TILE = 1, MX_EMPTY = 2 };
struct MxPlan {
    int kind;
    int cfg;       // skinny: blocks of 16 rows; tile: index of the tile table
    int ks;        // K slices (tile kernel): fp32 partial results in the workspace when > 1
    int slice;     // stages of 8 blocks per slice
    int64_t partial_bytes;
    int cus;       // CUs of the device
};
MxPlan plan_mx(int64_t M, int64_t N, int64_t nb, int cu_count);
// Whether the product quantises the activations itself.
bool mx_fuses(const MxPlan &plan, int64_t M, int64_t nb);
hipError_t launch_mx_gemm(int type, const MxGemm &p, const MxPlan &plan, float *partial, hipStream_t stream);
// Two products in one launch, where mx_pairs allows it: p in `type`, q in fp32.
bool mx_pairs(const MxPlan &p, const MxPlan &q);
hipError_t launch_mx_pair(int type, const MxGemm &p, const MxGemm &q, int cus, hipStream_t stream);
hipError_t launch_mx_gemm_x(int type, const MxGemm &p, const MxSkinnyX &x, const MxPlan &plan, hipStream_t stream);

// Newton-Schulz orthogonalisation (see the public header).
struct NewtonSchulz {
    const void *g;
    void *y;
    int64_t ldg, strideg, ldy, stridey;
    int batch, M, N;
    int steps;
    float a, b, c, eps;
    int cus;   // CUs of the device
};
// Whether the kernels' number format holds the iteration with these coefficients.
bool newton_schulz_supported(int steps, float a, float b, float c);
int64_t newton_schulz_bytes(int64_t batch, int64_t M, int64_t N);
hipError_t launch_newton_schulz(int type, const NewtonSchulz &p, void *workspace, hipStream_t stream);

}  // namespace mpg
