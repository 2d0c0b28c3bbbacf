// Internal interface of the 8-bit integer linear layer and of the gated
// feed-forward block. Arguments reaching these launchers have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mpgemm.h"

namespace mpg {

// X (M x K, MPGEMM_TYPE_*, row stride ldx elements) into codes and scales. pad: the
// codes' rows are filled with zeros up to the next multiple of 16.
struct I8Quantize {
    const void *x;
    int64_t ldx;
    int8_t *q;
    int64_t ldq;
    float *s;
    int M, K;
    bool pad;
};
hipError_t launch_i8_quantize(int type, const I8Quantize &p, hipStream_t stream);

struct I8Dequantize {
    const int8_t *q;
    int64_t ldq;
    const float *s;
    void *y;
    int64_t ldy;
    int M, K;
};
hipError_t launch_i8_dequantize(int type, const I8Dequantize &p, hipStream_t stream);

// What a product of the layers computes from A (M x K, along k) and B. The tile kernels take rows at
// multiples of 16 bytes, and along k zeros from K to the next multiple (of integers in A alone):
//   SCALED  int8: C = (A B^T) sa sb + bias
//   GATED   C = act(A B0^T) (A B1^T), of int8 operands each product scaled; G and U where wanted
//   DX      C = A [B0; B1], A M x 2 Kp, B0 and B1 K x N (across k), K of each
//   DW      rows [0, N1) of A^T B to C, with two parts rows [Kp, Kp + N1) to C2; A K x parts Kp, B K x N, both across k
enum LinMode { LIN_SCALED = 0, LIN_GATED = 1, LIN_DX = 2, LIN_DW = 3 };

struct Lin {
    const uint8_t *a, *b[2];
    int64_t lda, ldb[2];     // bytes
    const float *sa, *sb[2];
    const void *bias;        // of the result's type, or null
    void *c, *c2;            // (DW)
    void *g, *u;             // (GATED, or null)
    int64_t ldc, ldc2, ldg, ldu;   // elements
    int M, N, K;             // of the result; of the sum (DX: of one of its two parts)
    int part, parts;         // (DX, DW) the columns of A that belong to one part, padding included; (DW) its parts, 1 or 2
    int act;
};

enum LinKind { LINK_EMPTY = 0, LINK_SKINNY = 1, LINK_TILE = 2 };
struct LinPlan {
    int kind;
    int cfg;    // skinny: fragments of 16 rows; tile: index of the tile table
    int cus;
};
LinPlan plan_lin(int mode, int64_t M, int64_t N, int64_t K, int elem_bytes, int cu_count);
LinPlan plan_lin_pair(int64_t M, int64_t part, int parts, int64_t K, int cu_count);
hipError_t launch_w8a8(int type, const Lin &p, const LinPlan &plan, hipStream_t stream);
hipError_t launch_gated_w8a8(int type, const Lin &p, const LinPlan &plan, hipStream_t stream);
hipError_t launch_gated(int type, const Lin &p, const LinPlan &plan, hipStream_t stream);
hipError_t launch_gated_dx(int type, const Lin &p, const LinPlan &plan, hipStream_t stream);
hipError_t launch_gated_dw(int type, const Lin &p, const LinPlan &plan, hipStream_t stream);
// Both in one launch.
hipError_t launch_gated_pair(int type, const Lin &dx, const Lin &dw, const LinPlan &plan, hipStream_t stream);

// Few activations, quantised by every workgroup of the product itself.
bool lin_fuses(const LinPlan &plan, int64_t M, int64_t K);
struct LinX {
    const void *x;
    int64_t ldx;
};
hipError_t launch_w8a8_x(int type, const Lin &p, const LinX &x, const LinPlan &plan, hipStream_t stream);
hipError_t launch_gated_w8a8_x(int type, const Lin &p, const LinX &x, const LinPlan &plan, hipStream_t stream);

// D = [dG, dU] (M x 2 part, 16 bits, zeros from N to part) from dH, G and U.
struct GatedGrads {
    const void *dh, *g, *u;
    int64_t lddh, ldg, ldu;
    void *d;
    int M, N, part, act;
};
hipError_t launch_gated_grads(int type, const GatedGrads &p, hipStream_t stream);

// Copies of up to three matrices with rows at multiples of 16 bytes, zeros in the padding.
struct LinCopy {
    const uint8_t *from[3];
    uint8_t *to[3];
    int64_t ldf[3], ldt[3];   // bytes
    int rows[3], row_bytes[3];
};
hipError_t launch_lin_copy(const LinCopy &p, hipStream_t stream);
// C (M x N) = copies of `row` (N values of `type`), or zeros: the result of an empty sum.
hipError_t launch_lin_fill(int type, void *c, int64_t ldc, int M, int N, const void *row, hipStream_t stream);

}  // namespace mpg
