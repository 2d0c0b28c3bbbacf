// C-ABI of the 8-bit integer linear layer and of the gated feed-forward block:
// argument checks (before any HIP call), scratch layout and dispatch. The public
// contract is in include/mpgemm.h.
#include "mpgemm.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <initializer_list>

#include "handle.h"
#include "linear.h"

using mpg::DeviceGuard;

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 23;   // bytes; 128 rows of it stay below 2^30
constexpr int64_t kMaxDim = MPGEMM_MAX_DIM_LINEAR;
constexpr int64_t kMaxAlong = MPGEMM_MAX_ALONG_LINEAR;

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
bool type_ok(int type) { return type >= MPGEMM_TYPE_F16 && type <= MPGEMM_TYPE_F32; }
bool type16(int type) { return type == MPGEMM_TYPE_F16 || type == MPGEMM_TYPE_BF16; }
bool act_ok(int act) { return act >= MPGEMM_ACT_SILU && act <= MPGEMM_ACT_GELU_TANH; }
int size_of(int type) { return type == MPGEMM_TYPE_F32 ? 4 : 2; }

// A matrix with element-aligned rows of `cols` elements of `size` bytes.
mpgemm_status_t check_rows(const void *p, int64_t ld, int64_t cols, int size) {
    if (!p || ld < cols)
        return MPGEMM_ERR_INVALID_ARG;
    if (misaligned(p, size) || ld > INT64_MAX / 8 / (kMaxDim + 1))
        return MPGEMM_ERR_UNSUPPORTED;
    return MPGEMM_OK;
}

mpgemm_status_t check_scales(const float *s) {
    return !s ? MPGEMM_ERR_INVALID_ARG : misaligned(s, 4) ? MPGEMM_ERR_UNSUPPORTED : MPGEMM_OK;
}

mpgemm_status_t check_bias(const void *b, int type) {
    return misaligned(b, size_of(type)) ? MPGEMM_ERR_UNSUPPORTED : MPGEMM_OK;
}

mpgemm_status_t check_workspace(const void *ws, int64_t bytes, int64_t need) {
    if (need > 0 && (!ws || bytes < need))
        return MPGEMM_ERR_INVALID_ARG;
    return need > 0 && misaligned(ws, 16) ? MPGEMM_ERR_UNSUPPORTED : MPGEMM_OK;
}

// The first of several checks that failed.
mpgemm_status_t first(std::initializer_list<mpgemm_status_t> all) {
    for (mpgemm_status_t s : all)
        if (s != MPGEMM_OK)
            return s;
    return MPGEMM_OK;
}

mpgemm_status_t status_of(hipError_t e) { return e == hipSuccess ? MPGEMM_OK : MPGEMM_ERR_HIP; }

// Sizes that a product takes (grids are one 32-bit dimension).
bool sizes_ok(int64_t M, int64_t N, int64_t K, int64_t along) {
    return M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= along &&
           ((M + 63) / 64) * ((N + 31) / 32) <= INT_MAX;
}

// An operand of a tile kernel: its rows as they are, or a copy in the workspace where they do
// not start at multiples of 16 bytes, lie too far apart (a single row has no stride: its length is none), or
// (padded) end inside 16 bytes that have to hold zeros behind them.
struct Operand {
    const uint8_t *p;
    int64_t ld, rows, bytes;   // ld and bytes of a row, in bytes
    bool padded;
    Operand(const void *at, int64_t stride, int64_t r, int64_t row_bytes, bool pad)
        : p(static_cast<const uint8_t *>(at)), ld(r <= 1 ? round_up(row_bytes, 16) : stride), rows(r), bytes(row_bytes), padded(pad) {}
    bool needs_copy() const {
        return misaligned(p, 16) || ld % 16 != 0 || (rows > 1 && ld >= kMaxStride) || (padded && bytes % 16 != 0);
    }
    int64_t copy_bytes() const { return round_up(rows * round_up(bytes, 16), 256); }
};

// Copies those of up to three operands that need it (one launch), from `ws` on.
struct Copies {
    mpg::LinCopy c = {};
    int n = 0;
    uint8_t *ws;
    explicit Copies(void *w) : ws(static_cast<uint8_t *>(w)) {}
    void add(Operand &o) {
        if (o.needs_copy())
            put(o);
    }
    void put(Operand &o) {
        c.from[n] = o.p;
        c.to[n] = ws;
        c.ldf[n] = o.ld;
        c.ldt[n] = round_up(o.bytes, 16);
        c.rows[n] = (int)o.rows;
        c.row_bytes[n] = (int)o.bytes;
        ws += o.copy_bytes();
        o.p = c.to[n];
        o.ld = c.ldt[n];
        ++n;
    }
    hipError_t launch(hipStream_t stream) const { return n ? mpg::launch_lin_copy(c, stream) : hipSuccess; }
};

int64_t copies_of(std::initializer_list<const Operand *> all) {
    int64_t n = 0;
    for (const Operand *o : all)
        n += o->needs_copy() ? o->copy_bytes() : 0;
    return n;
}

int64_t copy_of(int64_t rows, int64_t row_bytes) { return round_up(rows * round_up(row_bytes, 16), 256); }

// Scratch of activations quantised by a launch before the product: codes, then scales.
struct Codes {
    int64_t ld, s_at, bytes;
    Codes(int64_t M, int64_t K) : ld(round_up(K, 128)), s_at(round_up(M * ld, 256)), bytes(s_at + round_up(4 * M, 256)) {}
};

mpg::Lin product(int64_t M, int64_t N, int64_t K, void *C, int64_t ldc) {
    mpg::Lin p = {};
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.c = C;
    p.ldc = ldc;
    return p;
}

// Columns of D = [dG, dU] that belong to dG: whole stages of the product over them.
int64_t part_of(int64_t N) { return round_up(N, 64); }

// ---- one implementation for the plain and the gated product on integers

struct I8Args {
    int64_t M, N, K;
    int type, act;
    bool gated;
    const void *X;            // quantised in the call ...
    int64_t ldx;
    const int8_t *A;          // ... or held
    int64_t lda;
    const float *SA;
    const int8_t *B[2];
    int64_t ldb[2];
    const float *SB[2];
    const void *bias;
    void *C;
    int64_t ldc;
};

mpgemm_status_t check_i8(const I8Args &a) {
    const int parts = a.gated ? 2 : 1;
    if (a.M < 0 || a.N < 0 || a.K < 0 || !type_ok(a.type) || (a.gated && !act_ok(a.act)))
        return MPGEMM_ERR_INVALID_ARG;
    if (a.M == 0 || a.N == 0)
        return MPGEMM_OK;
    if (!sizes_ok(a.M, a.N, a.K, MPGEMM_MAX_K_INT))
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = first({check_rows(a.C, a.ldc, a.N, size_of(a.type)), check_bias(a.bias, a.type)});
    if (a.K > 0) {
        if (a.X)
            st = first({st, check_rows(a.X, a.ldx, a.K, size_of(a.type))});
        else
            st = first({st, check_rows(a.A, a.lda, a.K, 1), check_scales(a.SA)});
        for (int w = 0; w < parts; ++w)
            st = first({st, check_rows(a.B[w], a.ldb[w], a.K, 1), check_scales(a.SB[w])});
    }
    return st;
}

mpgemm_status_t run_i8(mpgemm_handle_t h, const I8Args &a, bool dyn, void *workspace, int64_t workspace_bytes, void *stream) {
    mpgemm_status_t st = check_i8(a);
    if (st != MPGEMM_OK || a.M == 0 || a.N == 0)
        return st;
    if (dyn && a.K > 0 && !a.X)
        return MPGEMM_ERR_INVALID_ARG;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    const int mode = a.gated ? mpg::LIN_GATED : mpg::LIN_SCALED;
    const mpg::LinPlan plan = mpg::plan_lin(mode, a.M, a.N, a.K, 1, h->cu_count);
    const bool fused = dyn && mpg::lin_fuses(plan, a.M, a.K), tile = plan.kind == mpg::LINK_TILE;
    const Codes codes(a.M, a.K);
    Operand oa(a.A, a.lda, a.M, a.K, true), ob(a.B[0], a.ldb[0], a.N, a.K, false), oc(a.B[1], a.ldb[1], a.N, a.K, false);
    const int64_t own = dyn && !fused && plan.kind != mpg::LINK_EMPTY ? codes.bytes : 0;
    int64_t need = own;
    if (tile)
        need += (dyn ? 0 : copies_of({&oa})) + copies_of({&ob}) + (a.gated ? copies_of({&oc}) : 0);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (plan.kind == mpg::LINK_EMPTY)
        return status_of(mpg::launch_lin_fill(a.type, a.C, a.ldc, (int)a.M, (int)a.N, a.bias, s));
    mpg::Lin p = product(a.M, a.N, a.K, a.C, a.ldc);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (own) {
        float *scales = reinterpret_cast<float *>(ws + codes.s_at);
        const mpg::I8Quantize q{a.X, a.ldx, reinterpret_cast<int8_t *>(ws), codes.ld, scales, (int)a.M, (int)a.K, true};
        const hipError_t e = mpg::launch_i8_quantize(a.type, q, s);
        if (e != hipSuccess)
            return MPGEMM_ERR_HIP;
        oa = Operand(ws, codes.ld, a.M, a.K, false);   // (padded as it is)
        p.sa = scales;
    } else if (!dyn) {
        p.sa = a.SA;
    }
    if (tile) {
        Copies c(ws + own);
        c.add(oa);
        c.add(ob);
        if (a.gated)
            c.add(oc);
        const hipError_t e = c.launch(s);
        if (e != hipSuccess)
            return MPGEMM_ERR_HIP;
    }
    p.a = oa.p;
    p.lda = oa.ld;
    p.b[0] = ob.p;
    p.b[1] = oc.p;
    p.ldb[0] = ob.ld;
    p.ldb[1] = oc.ld;
    p.sb[0] = a.SB[0];
    p.sb[1] = a.SB[1];
    p.bias = a.bias;
    p.act = a.act;
    if (fused) {
        const mpg::LinX x{a.X, a.ldx};
        return status_of(a.gated ? mpg::launch_gated_w8a8_x(a.type, p, x, plan, s) : mpg::launch_w8a8_x(a.type, p, x, plan, s));
    }
    return status_of(a.gated ? mpg::launch_gated_w8a8(a.type, p, plan, s) : mpg::launch_w8a8(a.type, p, plan, s));
}

int64_t workspace_i8(int64_t M, int64_t N, int64_t K, bool gated, bool dyn, int aligned, int cu_count) {
    if (cu_count <= 0 || !sizes_ok(M, N, K, MPGEMM_MAX_K_INT))
        return -1;
    if (M == 0 || N == 0 || K == 0)
        return 0;
    const mpg::LinPlan plan = mpg::plan_lin(gated ? mpg::LIN_GATED : mpg::LIN_SCALED, M, N, K, 1, cu_count);
    int64_t n = dyn && !mpg::lin_fuses(plan, M, K) ? Codes(M, K).bytes : 0;
    if (plan.kind == mpg::LINK_TILE && !dyn && (!aligned || K % 16 != 0))
        n += copy_of(M, K);
    if (plan.kind == mpg::LINK_TILE && !aligned)
        n += (gated ? 2 : 1) * copy_of(N, K);
    return n;
}

}  // namespace

extern "C" {

mpgemm_status_t mpgemm_quantize_i8(mpgemm_handle_t h, int64_t M, int64_t K, int type, const void *X, int64_t ldx,
                                   int8_t *Q, int64_t ldq, float *S, void *stream) {
    if (M < 0 || K < 0 || !type_ok(type))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return MPGEMM_OK;
    if (M > kMaxDim || K > kMaxDim)
        return MPGEMM_ERR_UNSUPPORTED;
    const mpgemm_status_t st = first({check_rows(X, ldx, K, size_of(type)), check_rows(Q, ldq, K, 1), check_scales(S)});
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const mpg::I8Quantize p{X, ldx, Q, ldq, S, (int)M, (int)K, false};
    return status_of(mpg::launch_i8_quantize(type, p, static_cast<hipStream_t>(stream)));
}

mpgemm_status_t mpgemm_dequantize_i8(mpgemm_handle_t h, int64_t M, int64_t K, const int8_t *Q, int64_t ldq,
                                     const float *S, int type, void *Y, int64_t ldy, void *stream) {
    if (M < 0 || K < 0 || !type_ok(type))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0)
        return MPGEMM_OK;
    if (M > kMaxDim || K > kMaxDim)
        return MPGEMM_ERR_UNSUPPORTED;
    const mpgemm_status_t st = first({check_rows(Q, ldq, K, 1), check_scales(S), check_rows(Y, ldy, K, size_of(type))});
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const mpg::I8Dequantize p{Q, ldq, S, Y, ldy, (int)M, (int)K};
    return status_of(mpg::launch_i8_dequantize(type, p, static_cast<hipStream_t>(stream)));
}

mpgemm_status_t mpgemm_run_w8a8(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda,
                                const float *SA, const int8_t *B, int64_t ldb, const float *SB, const void *bias,
                                int type, void *C, int64_t ldc, void *workspace, int64_t workspace_bytes, void *stream) {
    const I8Args a{M, N, K, type, 0, false, nullptr, 0, A, lda, SA, {B, nullptr}, {ldb, 0}, {SB, nullptr}, bias, C, ldc};
    return run_i8(h, a, false, workspace, workspace_bytes, stream);
}

int64_t mpgemm_run_w8a8_workspace(int64_t M, int64_t N, int64_t K, int aligned, int cu_count) {
    return workspace_i8(M, N, K, false, false, aligned, cu_count);
}

mpgemm_status_t mpgemm_run_w8a8_dyn(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int type, const void *X,
                                    int64_t ldx, const int8_t *W, int64_t ldw, const float *SW, const void *bias,
                                    void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream) {
    if (M > 0 && N > 0 && K > 0 && !X)
        return MPGEMM_ERR_INVALID_ARG;
    const I8Args a{M, N, K, type, 0, false, X, ldx, nullptr, 0, nullptr, {W, nullptr}, {ldw, 0}, {SW, nullptr}, bias, Y, ldy};
    return run_i8(h, a, true, workspace, workspace_bytes, stream);
}

int64_t mpgemm_run_w8a8_dyn_workspace(int64_t M, int64_t N, int64_t K, int aligned, int cu_count) {
    return workspace_i8(M, N, K, false, true, aligned, cu_count);
}

mpgemm_status_t mpgemm_run_gated_w8a8(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int act, const int8_t *A,
                                      int64_t lda, const float *SA, const int8_t *Wg, int64_t ldwg, const float *SG,
                                      const int8_t *Wu, int64_t ldwu, const float *SU, int type, void *H, int64_t ldh,
                                      void *workspace, int64_t workspace_bytes, void *stream) {
    const I8Args a{M, N, K, type, act, true, nullptr, 0, A, lda, SA, {Wg, Wu}, {ldwg, ldwu}, {SG, SU}, nullptr, H, ldh};
    return run_i8(h, a, false, workspace, workspace_bytes, stream);
}

int64_t mpgemm_run_gated_w8a8_workspace(int64_t M, int64_t N, int64_t K, int aligned, int cu_count) {
    return workspace_i8(M, N, K, true, false, aligned, cu_count);
}

mpgemm_status_t mpgemm_run_gated_w8a8_dyn(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int type, int act,
                                          const void *X, int64_t ldx, const int8_t *Wg, int64_t ldwg, const float *SG,
                                          const int8_t *Wu, int64_t ldwu, const float *SU, void *H, int64_t ldh,
                                          void *workspace, int64_t workspace_bytes, void *stream) {
    if (M > 0 && N > 0 && K > 0 && !X)
        return MPGEMM_ERR_INVALID_ARG;
    const I8Args a{M, N, K, type, act, true, X, ldx, nullptr, 0, nullptr, {Wg, Wu}, {ldwg, ldwu}, {SG, SU}, nullptr, H, ldh};
    return run_i8(h, a, true, workspace, workspace_bytes, stream);
}

int64_t mpgemm_run_gated_w8a8_dyn_workspace(int64_t M, int64_t N, int64_t K, int aligned, int cu_count) {
    return workspace_i8(M, N, K, true, true, aligned, cu_count);
}

mpgemm_status_t mpgemm_run_gated(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int type, int act, const void *X,
                                 int64_t ldx, const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu, void *H,
                                 int64_t ldh, void *G, int64_t ldg, void *U, int64_t ldu, void *workspace,
                                 int64_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type16(type) || !act_ok(act) || (G == nullptr) != (U == nullptr))
        return MPGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0)
        return MPGEMM_OK;
    if (!sizes_ok(M, N, K, kMaxAlong))
        return MPGEMM_ERR_UNSUPPORTED;
    mpgemm_status_t st = check_rows(H, ldh, N, 2);
    if (G)
        st = first({st, check_rows(G, ldg, N, 2), check_rows(U, ldu, N, 2)});
    if (K > 0)
        st = first({st, check_rows(X, ldx, K, 2), check_rows(Wg, ldwg, K, 2), check_rows(Wu, ldwu, K, 2)});
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    const mpg::LinPlan plan = mpg::plan_lin(mpg::LIN_GATED, M, N, K, 2, h->cu_count);
    Operand ox(X, 2 * ldx, M, 2 * K, true), og(Wg, 2 * ldwg, N, 2 * K, true), ou(Wu, 2 * ldwu, N, 2 * K, true);
    const bool tile = plan.kind == mpg::LINK_TILE;
    if ((st = check_workspace(workspace, workspace_bytes, tile ? copies_of({&ox, &og, &ou}) : 0)) != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (plan.kind == mpg::LINK_EMPTY) {
        hipError_t e = mpg::launch_lin_fill(type, H, ldh, (int)M, (int)N, nullptr, s);
        if (G && e == hipSuccess)
            e = mpg::launch_lin_fill(type, G, ldg, (int)M, (int)N, nullptr, s);
        if (G && e == hipSuccess)
            e = mpg::launch_lin_fill(type, U, ldu, (int)M, (int)N, nullptr, s);
        return status_of(e);
    }
    mpg::Lin p = product(M, N, K, H, ldh);
    if (tile) {
        Copies c(workspace);
        c.add(ox);
        c.add(og);
        c.add(ou);
        if (c.launch(s) != hipSuccess)
            return MPGEMM_ERR_HIP;
    }
    p.a = ox.p;
    p.lda = ox.ld;
    p.b[0] = og.p;
    p.b[1] = ou.p;
    p.ldb[0] = og.ld;
    p.ldb[1] = ou.ld;
    p.act = act;
    p.g = G;
    p.u = U;
    p.ldg = ldg;
    p.ldu = ldu;
    return status_of(mpg::launch_gated(type, p, plan, s));
}

int64_t mpgemm_run_gated_workspace(int64_t M, int64_t N, int64_t K, int aligned, int cu_count) {
    if (cu_count <= 0 || !sizes_ok(M, N, K, kMaxAlong))
        return -1;
    if (M == 0 || N == 0 || K == 0 || (aligned && K % 8 == 0) || mpg::plan_lin(mpg::LIN_GATED, M, N, K, 2, cu_count).kind != mpg::LINK_TILE)
        return 0;
    return copy_of(M, 2 * K) + 2 * copy_of(N, 2 * K);
}

mpgemm_status_t mpgemm_run_gated_backward(mpgemm_handle_t h, int64_t M, int64_t N, int64_t K, int type, int act,
                                          const void *dH, int64_t lddh, const void *X, int64_t ldx, const void *Wg,
                                          int64_t ldwg, const void *Wu, int64_t ldwu, const void *G, int64_t ldg,
                                          const void *U, int64_t ldu, void *dX, int64_t lddx, void *dWg, int64_t lddwg,
                                          void *dWu, int64_t lddwu, void *workspace, int64_t workspace_bytes, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type16(type) || !act_ok(act))
        return MPGEMM_ERR_INVALID_ARG;
    const bool need_dx = dX && M > 0 && K > 0, need_dw = (dWg || dWu) && N > 0 && K > 0;
    if (!need_dx && !need_dw)
        return MPGEMM_OK;
    if (!sizes_ok(M, K, N, kMaxAlong / 2) || !sizes_ok(2 * part_of(N), K, 0, 0))
        return MPGEMM_ERR_UNSUPPORTED;
    const bool sums = M > 0 && N > 0;   // (else the gradients are sums of nothing)
    mpgemm_status_t st = MPGEMM_OK;
    if (sums)
        st = first({check_rows(dH, lddh, N, 2), check_rows(G, ldg, N, 2), check_rows(U, ldu, N, 2)});
    if (need_dx)
        st = first({st, check_rows(dX, lddx, K, 2)});
    if (need_dx && sums)
        st = first({st, check_rows(Wg, ldwg, K, 2), check_rows(Wu, ldwu, K, 2)});
    if (need_dw && sums)
        st = first({st, check_rows(X, ldx, K, 2)});
    if (need_dw && dWg)
        st = first({st, check_rows(dWg, lddwg, K, 2)});
    if (need_dw && dWu)
        st = first({st, check_rows(dWu, lddwu, K, 2)});
    if (st != MPGEMM_OK)
        return st;
    if (!h)
        return MPGEMM_ERR_INVALID_ARG;
    const int64_t part = part_of(N), d_bytes = round_up(M * 2 * part * 2, 256);
    Operand ox(X, 2 * ldx, M, 2 * K, false), og(Wg, 2 * ldwg, N, 2 * K, false), ou(Wu, 2 * ldwu, N, 2 * K, false);
    // (both weights go through the same offsets: they have to have one row stride)
    const bool strides = og.ld == ou.ld, copy_w = need_dx && (og.needs_copy() || ou.needs_copy() || !strides);
    int64_t need = sums ? d_bytes : 0;
    if (sums)
        need += (need_dw && ox.needs_copy() ? ox.copy_bytes() : 0) + (copy_w ? og.copy_bytes() + ou.copy_bytes() : 0);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != MPGEMM_OK)
        return st;
    DeviceGuard dg(h->device);
    if (!dg.ok)
        return MPGEMM_ERR_HIP;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (!sums) {
        hipError_t e = hipSuccess;
        if (need_dx)
            e = mpg::launch_lin_fill(type, dX, lddx, (int)M, (int)K, nullptr, s);
        if (need_dw && dWg && e == hipSuccess)
            e = mpg::launch_lin_fill(type, dWg, lddwg, (int)N, (int)K, nullptr, s);
        if (need_dw && dWu && e == hipSuccess)
            e = mpg::launch_lin_fill(type, dWu, lddwu, (int)N, (int)K, nullptr, s);
        return status_of(e);
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Copies c(ws + d_bytes);
    if (need_dw)
        c.add(ox);
    if (copy_w) {
        c.put(og);
        c.put(ou);
    }
    if (c.launch(s) != hipSuccess)
        return MPGEMM_ERR_HIP;
    const mpg::GatedGrads gp{dH, G, U, lddh, ldg, ldu, ws, (int)M, (int)N, (int)part, act};
    if (mpg::launch_gated_grads(type, gp, s) != hipSuccess)
        return MPGEMM_ERR_HIP;
    // (dWu alone: from its part of [dG, dU])
    const int parts = dWg && dWu ? 2 : 1;
    mpg::Lin x = product(M, K, N, dX, lddx), w = dWg ? product(N, K, M, dWg, lddwg) : product(N, K, M, dWu, lddwu);
    x.a = ws;
    w.a = dWg ? ws : ws + 2 * part;
    w.parts = parts;
    x.lda = w.lda = 2 * part * 2;
    x.part = w.part = (int)part;
    x.b[0] = og.p;
    x.b[1] = ou.p;
    x.ldb[0] = x.ldb[1] = og.ld;
    w.c2 = parts == 2 ? dWu : nullptr;
    w.ldc2 = lddwu;
    w.b[0] = ox.p;
    w.ldb[0] = ox.ld;
    if (need_dx && need_dw)
        return status_of(mpg::launch_gated_pair(type, x, w, mpg::plan_lin_pair(M, part, parts, K, h->cu_count), s));
    return status_of(need_dx ? mpg::launch_gated_dx(type, x, mpg::plan_lin(mpg::LIN_DX, M, K, 2 * part, 2, h->cu_count), s)
                             : mpg::launch_gated_dw(type, w, mpg::plan_lin(mpg::LIN_DW, parts * part, K, M, 2, h->cu_count), s));
}

int64_t mpgemm_run_gated_backward_workspace(int64_t M, int64_t N, int64_t K, int aligned, int cu_count) {
    if (cu_count <= 0 || !sizes_ok(M, K, N, kMaxAlong / 2) || !sizes_ok(2 * part_of(N), K, 0, 0))
        return -1;
    if (M == 0 || N == 0 || K == 0)
        return 0;
    return round_up(M * 2 * part_of(N) * 2, 256) + (aligned ? 0 : copy_of(M, 2 * K) + 2 * copy_of(N, 2 * K));
}

}  // extern "C"
