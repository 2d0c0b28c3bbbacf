// C-ABI of the MXFP4 calls and of the Newton-Schulz update: argument checks
// (before any HIP call), scratch layout and dispatch. The public contract is
// in include/mpgemm.h.
#include "mpgemm.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "handle.h"
#include "mxfp4.h"

using mpg::DeviceGuard;

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 23;   // bytes; 256 rows of it stay below 2^31
constexpr int64_t kMaxDim = MPGEMM_MAX_K_MXFP4;

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
int64_t blocks_of(int64_t k) { return (k + 31) / 32; }
int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
bool type_ok(int type) { return type >= MPGEMM_TYPE_F16 && type <= MPGEMM_TYPE_F32; }
int size_of(int type) { return type == MPGEMM_TYPE_F32 ? 4 : 2; }

// A plain matrix of `cols` columns (element-aligned rows).
mpgemm_status_t check_plain(const void *p, int64_t ld, int64_t cols, int type) {
    if (!p || ld < cols)
        return MPGEMM_ERR_INVALID_ARG;
    if (misaligned(p, size_of(type)) || ld > INT64_MAX / 8 / (kMaxDim + 1))
        return MPGEMM_ERR_UNSUPPORTED;
    return MPGEMM_OK;
}

// Codes and scales of rows of k elements.
mpgemm_status_t check_held(const uint8_t *q, int64_t ldq, const uint8_t *s, int64_t lds, int64_t k) {
    if (!q || !s || ldq < 16 * blocks_of(k) || lds < blocks_of(k))
        return MPGEMM_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(s, 16) || ldq % 16 != 0 || lds % 16 != 0 || ldq >= kMaxStride ||
        lds >= kMaxStride)
        return MPGEMM_ERR_UNSUPPORTED;
    return MPGEMM_OK;
}

mpgemm_status_t check_workspace(const void *ws, int64_t bytes, int64_t need) {
    if (need < 0)
        return MPGEMM_ERR_UNSUPPORTED;
    if (need > 0 && (!ws || bytes < need))
        return MPGEMM_ERR_INVALID_ARG;
    return need > 0 && misaligned(ws, 16) ? MPGEMM_ERR_UNSUPPORTED : MPGEMM_OK;
}

// Scratch of one held matrix (rows x k): codes, then scales.
struct Held {
    int64_t ldq, lds, q_bytes, bytes;
    Held(int64_t rows, int64_t k)
        : ldq(16 * blocks_of(k)), lds(round_up(blocks_of(k), 16)), q_bytes(rows * ldq), bytes(q_bytes + rows * lds) {}
};

// Sizes that a product takes: the tile grid is one 32-bit dimension.
bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    return M <= kMaxDim && N <= kMaxDim && K <= kMaxDim && ((M + 63) / 64) * ((N + 63) / 64) <= INT_MAX;
}

mpgemm_status_t status_of(hipError_t e) { return e == hipSuccess ? MPGEMM_OK : MPGEMM_ERR_HIP; }

mpg::MxGemm product(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *SA,
                    int64_t ldsa, const uint8_t *B, int64_t ldb, const uint8_t *SB, int64_t ldsb,
                    const void *bias, void *C, int64_t ldc) {
    mpg::MxGemm p;
    p.a = A;
    p.sa = SA;
    p.b = B;
    p.sb = SB;
    p.lda = lda;
    p.ldsa = ldsa;
    p.ldb = ldb;
    p.ldsb = ldsb;
    p.bias = bias;
    p.c = C;
    p.ldc = ldc;
    p.M = (int)M;
    p.N = (int)N;
    p.nb = (int)blocks_of(K);
    return p;
}

}  // namespace

extern "C" {

mpgemm_status_t mpgemm_quantize_mxfp4(mpgemm_handle_t h, int64_t M, int64_t K, int type, const void *X,
                                      int64_t ldx, uint8_t *Q, int64_t ldq, uint8_t *S, int64_t lds,
                                      uint8_t *QT, int64_t ldqt, uint8_t *ST, int64_t ldst, void *stream) {
    if (M < 0 || K < 0 || !type_ok(type))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return MPGEMM_OK;
    const bool rows = Q || S, cols = QT || ST;
    if (!rows && !cols)
        return MPGEMM_ERR_INVALID_ARG;
    if (M > kMaxDim || K > kMaxDim)
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = check_plain(X, ldx, K, type);
    if (st == MPGEMM_OK && rows)
        st = check_held(Q, ldq, S, lds, K);
    if (st == MPGEMM_OK && cols)
        st = check_held(QT, ldqt, ST, ldst, M);
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const mpg::MxQuantize p{X, ldx, Q, S, QT, ST, ldq, lds, ldqt, ldst, (int)M, (int)K};
    return status_of(mpg::launch_mx_quantize(type, p, static_cast<hipStream_t>(stream)));
}

mpgemm_status_t mpgemm_dequantize_mxfp4(mpgemm_handle_t h, int64_t M, int64_t K, const uint8_t *Q,
                                        int64_t ldq, const uint8_t *S, int64_t lds, int type, void *Y,
                                        int64_t ldy, void *stream) {
    if (M < 0 || K < 0 || !type_ok(type))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return MPGEMM_OK;
    if (M > kMaxDim || K > kMaxDim)
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = check_held(Q, ldq, S, lds, K);
    if (st == MPGEMM_OK)
        st = check_plain(Y, ldy, K, type);
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const mpg::MxDequantize p{Q, S, Y, ldq, lds, ldy, (int)M, (int)K};
    return status_of(mpg::launch_mx_dequantize(type, p, static_cast<hipStream_t>(stream)));
}

int64_t mpgemm_run_mxfp4_workspace(int64_t M, int64_t N, int64_t K, int cu_count) {
    if (M < 0 || N < 0 || K < 0 || cu_count < 1 || !sizes_ok(M, N, K))
        return -1;
    if (M == 0 || N == 0)
        return 0;
    return mpg::plan_mx(M, N, blocks_of(K), cu_count).partial_bytes;
}

mpgemm_status_t mpgemm_run_mxfp4(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, const uint8_t *A,
                                 int64_t lda, const uint8_t *SA, int64_t ldsa, const uint8_t *B,
                                 int64_t ldb, const uint8_t *SB, int64_t ldsb, const void *bias, int type,
                                 void *C, int64_t ldc, void *workspace, int64_t workspace_bytes,
                                 void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type_ok(type))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    if (!sizes_ok(M, N, K))
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = check_plain(C, ldc, N, type);
    if (st == MPGEMM_OK && K > 0)
        st = check_held(A, lda, SA, ldsa, K);
    if (st == MPGEMM_OK && K > 0)
        st = check_held(B, ldb, SB, ldsb, K);
    if (st != MPGEMM_OK)
        return st;
    if (misaligned(bias, size_of(type)))
        return MPGEMM_ERR_UNSUPPORTED;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    const mpg::MxPlan plan = mpg::plan_mx(M, N, blocks_of(K), h->cu_count);
    st = check_workspace(workspace, workspace_bytes, plan.partial_bytes);
    if (st != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    return status_of(mpg::launch_mx_gemm(type, product(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, bias, C, ldc),
                                         plan, static_cast<float *>(workspace), static_cast<hipStream_t>(stream)));
}

int64_t mpgemm_run_mxfp4_dyn_workspace(int64_t M, int64_t N, int64_t K, int cu_count) {
    const int64_t partial = mpgemm_run_mxfp4_workspace(M, N, K, cu_count);
    if (partial < 0 || M == 0 || N == 0 || K == 0)
        return partial;
    if (mpg::mx_fuses(mpg::plan_mx(M, N, blocks_of(K), cu_count), M, blocks_of(K)))
        return 0;
    return round_up(Held(M, K).bytes, 256) + partial;
}

mpgemm_status_t mpgemm_run_mxfp4_dyn(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int type,
                                     const void *X, int64_t ldx, const uint8_t *W, int64_t ldw,
                                     const uint8_t *SW, int64_t ldsw, const void *bias, void *Y,
                                     int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type_ok(type))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    if (!sizes_ok(M, N, K))
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = check_plain(Y, ldy, N, type);
    if (st == MPGEMM_OK && K > 0)
        st = check_plain(X, ldx, K, type);
    if (st == MPGEMM_OK && K > 0)
        st = check_held(W, ldw, SW, ldsw, K);
    if (st != MPGEMM_OK)
        return st;
    if (misaligned(bias, size_of(type)))
        return MPGEMM_ERR_UNSUPPORTED;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    const mpg::MxPlan plan = mpg::plan_mx(M, N, blocks_of(K), h->cu_count);
    const bool fused = mpg::mx_fuses(plan, M, blocks_of(K));
    const Held a(M, K);
    const int64_t a_bytes = fused || K == 0 ? 0 : round_up(a.bytes, 256);
    st = check_workspace(workspace, workspace_bytes, a_bytes + plan.partial_bytes);
    if (st != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *q = static_cast<uint8_t *>(workspace);
    const mpg::MxGemm p = product(M, N, K, q, a.ldq, q + a.q_bytes, a.lds, W, ldw, SW, ldsw, bias, Y, ldy);
    if (fused) {
        const mpg::MxSkinnyX x{X, ldx, (int)K, 0};
        return status_of(mpg::launch_mx_gemm_x(type, p, x, plan, s));
    }
    if (K > 0) {
        const mpg::MxQuantize z{X, ldx, q, q + a.q_bytes, nullptr, nullptr, a.ldq, a.lds, 0, 0, (int)M, (int)K};
        const hipError_t e = mpg::launch_mx_quantize(type, z, s);
        if (e != hipSuccess)
            return MPGEMM_ERR_HIP;
    }
    return status_of(mpg::launch_mx_gemm(type, p, plan, reinterpret_cast<float *>(q + a_bytes), s));
}

int64_t mpgemm_run_mxfp4_backward_workspace(int64_t M, int64_t N, int64_t K, int cu_count) {
    const int64_t px = mpgemm_run_mxfp4_workspace(M, K, N, cu_count);
    const int64_t pw = mpgemm_run_mxfp4_workspace(N, K, M, cu_count);
    if (px < 0 || pw < 0)
        return -1;
    if (M == 0 || N == 0 || K == 0)
        return 0;
    return round_up(Held(M, N).bytes, 256) + round_up(Held(N, M).bytes, 256) + (px > pw ? px : pw);
}

mpgemm_status_t mpgemm_run_mxfp4_backward(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int type,
                                          const void *dY, int64_t lddy, const uint8_t *WT, int64_t ldwt,
                                          const uint8_t *SWT, int64_t ldswt, const uint8_t *XT,
                                          int64_t ldxt, const uint8_t *SXT, int64_t ldsxt, void *dX,
                                          int64_t lddx, float *dW, int64_t lddw, void *workspace,
                                          int64_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type_ok(type) || (!dX && !dW))
        return MPGEMM_ERR_INVALID_ARG;
    if (K == 0 || (M == 0 && N == 0))
        return MPGEMM_OK;
    if (!sizes_ok(M, K, N) || !sizes_ok(N, K, M))
        return MPGEMM_ERR_UNSUPPORTED;
    const bool some = M > 0 && N > 0;   // else a gradient of zeros
    const bool want_x = dX && M > 0, want_w = dW && N > 0;
    mpgemm_status_t st = MPGEMM_OK;
    if (some)
        st = check_plain(dY, lddy, N, type);
    if (st == MPGEMM_OK && want_x)
        st = check_plain(dX, lddx, K, type);
    if (st == MPGEMM_OK && want_w)
        st = check_plain(dW, lddw, K, MPGEMM_TYPE_F32);
    if (st == MPGEMM_OK && want_x && some)
        st = check_held(WT, ldwt, SWT, ldswt, N);
    if (st == MPGEMM_OK && want_w && some)
        st = check_held(XT, ldxt, SXT, ldsxt, M);
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, mpgemm_run_mxfp4_backward_workspace(M, N, K, h->cu_count));
    if (st != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Held r(M, N), c(N, M);
    uint8_t *rq = static_cast<uint8_t *>(workspace), *cq = rq + round_up(r.bytes, 256);
    float *partial = reinterpret_cast<float *>(cq + round_up(c.bytes, 256));
    if (some) {
        const mpg::MxQuantize z{dY, lddy, want_x ? rq : nullptr, rq + r.q_bytes, want_w ? cq : nullptr, cq + c.q_bytes,
                                r.ldq, r.lds, c.ldq, c.lds, (int)M, (int)N};
        if (mpg::launch_mx_quantize(type, z, s) != hipSuccess)
            return MPGEMM_ERR_HIP;
    }
    const mpg::MxPlan plan_x = mpg::plan_mx(M, K, blocks_of(N), h->cu_count);
    const mpg::MxPlan plan_w = mpg::plan_mx(N, K, blocks_of(M), h->cu_count);
    const mpg::MxGemm px =
        product(M, K, N, rq, r.ldq, rq + r.q_bytes, r.lds, WT, ldwt, SWT, ldswt, nullptr, dX, lddx);
    const mpg::MxGemm pw =
        product(N, K, M, cq, c.ldq, cq + c.q_bytes, c.lds, XT, ldxt, SXT, ldsxt, nullptr, dW, lddw);
    if (want_x && want_w && mpg::mx_pairs(plan_x, plan_w))
        return status_of(mpg::launch_mx_pair(type, px, pw, h->cu_count, s));
    if (want_x && mpg::launch_mx_gemm(type, px, plan_x, partial, s) != hipSuccess)
        return MPGEMM_ERR_HIP;
    if (want_w && mpg::launch_mx_gemm(MPGEMM_TYPE_F32, pw, plan_w, partial, s) != hipSuccess)
        return MPGEMM_ERR_HIP;
    return MPGEMM_OK;
}

int64_t mpgemm_run_newton_schulz_workspace(int64_t batch, int64_t M, int64_t N) {
    if (batch < 0 || M < 0 || N < 0 || batch > 65535 || M > 65536 || N > 65536)
        return -1;
    return mpg::newton_schulz_bytes(batch, M, N);
}

mpgemm_status_t mpgemm_run_newton_schulz(mpgemm_handle_t h, int64_t batch, int64_t M, int64_t N, int type,
                                         const void *G, int64_t ldg, int64_t strideg, int steps,
                                         const float *coeffs, float eps, void *Y, int64_t ldy,
                                         int64_t stridey, void *workspace, int64_t workspace_bytes,
                                         void *stream) {
    if (batch < 0 || M < 0 || N < 0 || steps < 0 || !type_ok(type) || !(eps >= 0.f) || (steps > 0 && !coeffs))
        return MPGEMM_ERR_INVALID_ARG;
    if (batch == 0 || M == 0 || N == 0)
        return MPGEMM_OK;
    if (type == MPGEMM_TYPE_F32 || steps > 100 || mpgemm_run_newton_schulz_workspace(batch, M, N) < 0)
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = check_plain(G, ldg, N, type);
    if (st == MPGEMM_OK)
        st = check_plain(Y, ldy, N, type);
    if (st != MPGEMM_OK)
        return st;
    if (batch > 1 && (strideg < 0 || stridey < (M - 1) * ldy + N))
        return MPGEMM_ERR_INVALID_ARG;
    if (strideg > INT64_MAX / 8 / 65536 || stridey > INT64_MAX / 8 / 65536)
        return MPGEMM_ERR_UNSUPPORTED;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    const float zero[3] = {0.f, 0.f, 0.f};
    const float *k = coeffs ? coeffs : zero;
    if (!mpg::newton_schulz_supported(steps, k[0], k[1], k[2]))
        return MPGEMM_ERR_UNSUPPORTED;
    st = check_workspace(workspace, workspace_bytes, mpgemm_run_newton_schulz_workspace(batch, M, N));
    if (st != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const mpg::NewtonSchulz p{G, Y, ldg, strideg, ldy, stridey, (int)batch, (int)M, (int)N, steps, k[0], k[1], k[2], eps, h->cu_count};
    return status_of(mpg::launch_newton_schulz(type, p, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
