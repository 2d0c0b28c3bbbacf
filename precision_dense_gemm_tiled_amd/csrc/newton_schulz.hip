// Newton-Schulz orthogonalisation of a batch of matrices:
//   X = G / (|G|_F + eps), then `steps` times X <- Q X with Q = a I + b A + c A A, A = X X^T
// on the smaller side (X is m x n with m <= n, G or its transpose).
//
// Every Q is a polynomial of A, so all of them commute and the iteration needs
// X at its ends only:
//   A = X X^T;   per step: Q = a I + b A + c A A,  T = Q A,  A <- Q T,  W <- Q W;   X <- W X.
// Per step that is four symmetric m x m products (the tiles on and below the
// diagonal, the others mirrored), 4 m^3 flop, against m^2 n + m^3 + 2 m^2 n for
// forming A and Q X anew: the same for a square matrix, less than a third at n = 4 m.
// What it costs is accuracy: an error of A in the direction of a small singular value
// grows by about a^2 per step, as that eigenvalue of A does, and A has to be formed
// anew from X once it is no longer small; see group_length.
//
// Every product is of fp32 quality at the fp16 matrix rate: a factor is held as
// the sum of two fp16 values of a scaled matrix, h = fp16(2^e x), l = fp16(2^e x - h):
// 22 significant bits, and a product is h h + h l + l h with fp32 sums; l l is below
// the rounding of the sum. The exponents e put each matrix's spectral norm, which
// bounds its entries, at about 2^13 of fp16's 2^16. They come from bounds that
// follow from |singular values of X| <= 1 and the polynomial, and are found per
// matrix on the GPU (ns_factors), so any |G| against eps works; polynomials for
// which the bounds say nothing are refused (newton_schulz_supported). G itself (fp16
// or bf16) needs one part: scaled by a power of two it is an fp16 matrix exactly, but
// for entries below 2^-26 |G|. So the first A is one product and the first W X two.
// Single fp16 values without the l part are not enough: off by 1.5e-3 of the norm on
// gradients of rank 64 plus noise, 3e-3 on rank 8 with noise of 1e-2 below it (bf16's
// own rounding: 1.7e-3, fp16's: 2.1e-4; with the l part: nothing next to either).
//
// Bound by the matrix units' power for large matrices (2048 x 8192, W X: 1.2 PFLOP/s of
// fp16 products between the others at 1.9 GHz, 1.6 alone; the library's bf16 product reaches
// 1.47), by waits for symmetric products on a workgroup per CU (253 tiles of 96 x 96 at 2048:
// 36 us, 24.5 without loads and LDS reads), by launches and the way to L2 for small ones
// (12 x 512 x 512: 11 to 15 us a product, about 6 of them with no K loop).
// Therefore a matrix with a side up to 128 takes all steps of a group in one launch
// (ns_small_kernel), and A = X X^T of a long and narrow X is split along n.
#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "mxfp4.h"
#include "lds_dma.h"

namespace mpg {

typedef int ns_i32x4 __attribute__((ext_vector_type(4)));
typedef float ns_f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 ns_f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t ns_u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t ns_u32x4 __attribute__((ext_vector_type(4)));

// A matrix of one part (rows of `ld` fp16 values) or two (rows of `ld` / 64 lines of
// 128 bytes, each 32 h and their 32 l: the 128 bytes that a stage of the products
// takes from a row are one cache line).
struct NsMat {
    uint16_t *p;
    int64_t ld, stride;   // in 16-bit values; stride between matrices of the batch
};

__device__ __forceinline__ uint16_t ns_half(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
__device__ __forceinline__ float ns_f32(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }

// x as h | l << 16
__device__ __forceinline__ uint32_t ns_split(float x) {
    const uint16_t h = ns_half(x);
    return h | ((uint32_t)ns_half(x - ns_f32(h)) << 16);
}

// ------------------------------------------------------------ ends

// 8 elements of a row from column c0 on, zeros past the row's end.
template <typename T, bool VEC>
__device__ __forceinline__ void ns_load8(const T *row, int c0, int cols, T (&v)[8]) {
    if (VEC && c0 + 8 <= cols) {
        const ns_u32x4 w = *reinterpret_cast<const ns_u32x4 *>(row + c0);
        __builtin_memcpy(v, &w, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c0 + i < cols ? row[c0 + i] : (T)0.f;
    }
}

// Sums of squares of G: workgroup b of the gridDim.x of a matrix takes the 64 x 64 tiles
// b, b + gridDim.x, ... In 64 bits: bf16 squares leave the range of fp32 at both ends,
// and the pass is bound by memory.
constexpr int NS_SUMS = 1024;

// Sum over the workgroup's 256 threads, in every thread, in a fixed order.
__device__ __forceinline__ double ns_block_sum(double s, double *red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = s;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void ns_square_kernel(NewtonSchulz p, int batch0, int across, int tiles, double *sums) {
    __shared__ double red[4];
    const int tid = threadIdx.x;
    const T *G = (const T *)p.g + (int64_t)(batch0 + blockIdx.y) * p.strideg;
    double s = 0.;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int r0 = t / across * 64 + tid / 8, c0 = t % across * 64 + (tid & 7) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r0 + 32 * i < p.M) {
                T v[8];
                ns_load8<T, VEC>(G + (int64_t)(r0 + 32 * i) * p.ldg, c0, p.N, v);
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    s += (double)(float)v[d] * (double)(float)v[d];
            }
    }
    s = ns_block_sum(s, red);
    if (tid == 0)
        sums[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// Factors of the products' epilogues, for each step.
enum { NS_Q_ACC, NS_Q_ADD, NS_Q_ONE, NS_T, NS_A, NS_W, NS_GRAM, NS_APPLY, NS_FACTORS };

struct NsGroups {
    int len, longer;   // groups of len + 1 steps, `longer` of them, then of len
    __host__ __device__ bool starts(int k) const {
        const int head = longer * (len + 1);
        return k < head ? k % (len + 1) == 0 : (k - head) % len == 0;
    }
};

// Exponent that takes a matrix of spectral norm `bound` to about 2^13. (Norms below
// 2^-100, the squares of tiny singular values, count as that: it keeps the factors,
// 2^(difference of exponents), in fp32's range, and nothing of such an A reaches Q.)
__device__ __forceinline__ int ns_exponent(float bound) {
    return bound < FLT_MAX ? 13 - (ilogbf(fmaxf(bound, 0x1p-100f)) + 1) : 0;
}

// |G| of a matrix and what follows from it, in every thread.
struct NsNorm {
    double norm, inv;   // inv: 1 / (|G| + eps)
    bool finite;        // false for NaN, and for 0 / 0
    int ex;             // G is scaled by 2^ex
    __device__ __forceinline__ NsNorm(const double *sums, int count, float eps, double *red) {
        double s = 0.;
        for (int i = threadIdx.x; i < count; i += 256)
            s += sums[i];
        norm = sqrt(ns_block_sum(s, red));
        inv = 1. / (norm + (double)eps);
        finite = norm < DBL_MAX && inv < DBL_MAX;
        ex = finite && norm > 0. ? min(12 - ilogb(norm), 126) : 0;
    }
};

// The factors of every step's products of a matrix, by one wavefront.
__device__ __forceinline__ void ns_factors(const NewtonSchulz &p, NsGroups gr, const NsNorm &g, int lane, float *factors) {
    // The singular values x of X lie in [0, r]. Lane t looks at four x of [0, r]: the
    // largest |Q|, |T| = |x^2 Q| and next r = |x Q|. The factors are products of
    // powers of two with exponents in the range of a double.
    auto two = [](int e) { return ldexp(1., e); };
    float r = g.finite ? (float)fmin(g.norm * g.inv, 1.) : 1.f, wb = 1.f;
    double to_x = g.inv * two(-g.ex);   // stored X -> X
    int ew = 0;
    for (int k = 0; k < p.steps; ++k) {
        float v[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = r * ((float)(4 * lane + i) * (1.f / 255.f)), x2 = x * x;
            const float q = fabsf(p.a + x2 * (p.b + x2 * p.c));
            v[0] = fmaxf(v[0], q);
            v[1] = fmaxf(v[1], q * x2);
            v[2] = fmaxf(v[2], q * x);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
#pragma unroll
            for (int d = 0; d < 3; ++d)
                v[d] = fmaxf(v[d], __shfl_xor(v[d], o));
        // exponents of this step's matrices
        const int ea = ns_exponent(r * r), eq = ns_exponent(v[0]), et = ns_exponent(v[1]), ea2 = ns_exponent(v[2] * v[2]);
        const bool first = gr.starts(k), last = k + 1 == p.steps || gr.starts(k + 1);
        wb = first ? v[0] : wb * v[0];
        const int ew2 = first ? eq : ns_exponent(wb);
        const int ex = k + 1 < p.steps ? ns_exponent(v[2]) : 0;
        if (lane < NS_FACTORS) {
            const double base = lane == NS_Q_ACC ? (double)p.c : lane == NS_Q_ADD ? (double)p.b : lane == NS_Q_ONE ? (double)p.a
                                : lane == NS_GRAM ? to_x * to_x : lane == NS_APPLY ? to_x : 1.;
            const int e = lane == NS_Q_ACC ? eq - 2 * ea : lane == NS_Q_ADD ? eq - ea : lane == NS_Q_ONE ? eq
                          : lane == NS_T ? et - eq - ea : lane == NS_A ? ea2 - eq - et : lane == NS_W ? ew2 - eq - ew
                          : lane == NS_GRAM ? ea : ex - ew2;
            // (finite, so that zeros stay zeros)
            factors[k * NS_FACTORS + lane] =
                (float)fmin(fmax(base * two(e), -(double)FLT_MAX), (double)FLT_MAX);
        }
        ew = ew2;
        if (last)
            to_x = two(-ex);
        r = v[2];
    }
}

// G (M x N), scaled by a power of two, as X (m x n, padded) and X^T, and the factors (one
// workgroup per matrix). FLIP: G is taller than wide, X = G^T. Every workgroup sums the
// sums of squares: a launch less. A |G| that is not finite makes X, and with it the whole
// result, NaN.
template <typename T, bool FLIP, bool VEC>
__global__ __launch_bounds__(256) void ns_load_kernel(NewtonSchulz p, NsGroups gr, int batch0, const double *sums, int count,
                                                      float *factors, NsMat X, NsMat XT) {
    __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];
    __shared__ double red[4];
    const int tid = threadIdx.x;
    const T *G = (const T *)p.g + (int64_t)(batch0 + blockIdx.z) * p.strideg;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    const NsNorm norm(sums + (int64_t)blockIdx.z * count, count, p.eps, red);
    const float up = norm.finite ? (float)ldexp(1., norm.ex) : __builtin_nanf("");
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid < 64)
        ns_factors(p, gr, norm, tid, factors + (int64_t)blockIdx.z * p.steps * NS_FACTORS);
    const NsMat own = FLIP ? XT : X, other = FLIP ? X : XT;   // own: rows as G's
    const int g = tid & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int rl = tid / 8 + 32 * i;
        uint16_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (r0 + rl < p.M) {
            T v[8];
            ns_load8<T, VEC>(G + (int64_t)(r0 + rl) * p.ldg, c0 + 8 * g, p.N, v);
#pragma unroll
            for (int d = 0; d < 8; ++d)
                h[d] = ns_half((float)v[d] * up);
        }
        ns_u32x4 w;
        __builtin_memcpy(&w, h, 16);
        *reinterpret_cast<ns_u32x4 *>(own.p + (int64_t)blockIdx.z * own.stride + (int64_t)(r0 + rl) * own.ld + c0 + 8 * g) = w;
        *reinterpret_cast<ns_u32x4 *>(&tile[rl][8 * g]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int cl = (tid & 31) + 32 * i, rg = tid / 32;   // 8 rows of a column
        uint16_t h[8];
#pragma unroll
        for (int d = 0; d < 8; ++d)
            h[d] = tile[8 * rg + d][cl];
        ns_u32x4 w;
        __builtin_memcpy(&w, h, 16);
        *reinterpret_cast<ns_u32x4 *>(other.p + (int64_t)blockIdx.z * other.stride + (int64_t)(c0 + cl) * other.ld + r0 + 8 * rg) = w;
    }
}

// Y = G / (|G| + eps) (no steps)
template <typename T>
__global__ __launch_bounds__(256) void ns_scale_kernel(NewtonSchulz p, int batch0, const double *sums, int count) {
    __shared__ double red[4];
    const int z = batch0 + blockIdx.z;
    const T *G = (const T *)p.g + (int64_t)z * p.strideg;
    T *Y = (T *)p.y + (int64_t)z * p.stridey;
    const int64_t total = (int64_t)p.M * p.N;
    const NsNorm norm(sums + (int64_t)blockIdx.z * count, count, p.eps, red);
    const double s = norm.finite ? norm.inv : (double)__builtin_nanf("");
    for (int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x; f < total; f += (int64_t)gridDim.x * 256) {
        const int64_t r = f / p.N, c = f - r * p.N;
        Y[r * p.ldy + c] = (T)(float)((double)(float)G[r * p.ldg + c] * s);
    }
}

// ------------------------------------------------------------ products

// out = f[0] a b^T (+ f[add] add + f[one] I)
struct NsJob {
    NsMat a, b;       // operands, K contiguous
    NsMat add, out, outt;
    int factor;       // index of the epilogue's factor among the step's
};

struct NsGemm {
    NsJob job[2];
    int jobs, nz;
    int M, N, K;      // padded to 64
    int tiles_m, tiles;
    const float *factors;   // of this step, NS_FACTORS each, `fstride` floats between matrices
    int64_t fstride;
    // NS_PART: `jobs` slices of K, of `slice` each but the last; slice i of a matrix goes to
    // part + i M M, `pstride` floats between matrices
    float *part;
    int64_t pstride;
    int slice;
};

// Results: NS_SYM a symmetric matrix (tiles on and below the diagonal, mirrored),
// NS_POLY the same with the multiples of `add` and of the identity, NS_X a matrix
// and its transpose, NS_OUT the caller's Y, NS_PART the plain fp32 sums of a slice of K of
// a symmetric matrix, on and below the diagonal.
enum { NS_SYM, NS_POLY, NS_X, NS_OUT, NS_PART };

// Tile t of rows x cols: bands of NS_BAND rows, column by column, so that the tiles that
// an XCD works on at a time share few rows and columns of the operands (32 of them: 8 + 4).
constexpr int NS_BAND = 8;

__device__ __forceinline__ void ns_tile(int t, int rows, int cols, int &tm, int &tn) {
    const int r0 = t / (NS_BAND * cols) * NS_BAND, u = t - r0 * cols, h = min(NS_BAND, rows - r0);
    tn = u / h;
    tm = r0 + u - tn * h;
}

// The same for the tiles on and below the diagonal.
__device__ __forceinline__ void ns_lower_tile(int t, int rows, int &tm, int &tn) {
    int r = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);   // t's row if they went row by row
    while ((r + 1) * (r + 2) / 2 <= t)
        ++r;
    while (r * (r + 1) / 2 > t)
        --r;
    const int r0 = r / NS_BAND * NS_BAND, h = min(NS_BAND, rows - r0);
    int u = t - r0 * (r0 + 1) / 2;
    if (u < r0 * h) {
        tn = u / h;
        tm = r0 + u - tn * h;
        return;
    }
    u -= r0 * h;
    int c = 0;
    while (u >= h - c)
        u -= h - c++;
    tn = r0 + c;
    tm = tn + u;
}

// PA, PB: parts of the operands. C tile of 2 WT x 2 WT per workgroup, four
// wavefronts of WT x WT, stages of KS of K in an LDS ring of NS slots. 16-byte chunk c
// of LDS row r sits at c ^ swz(r). A 16-byte read is served in four groups of 16 lanes,
// 0-3, 12-15 and 20-27 the first, 4-11, 16-19 and 28-31 the second: half of the rows with
// one chunk and the other half with its neighbour. swz(r) is even and takes every even
// value once in each half, so a group has all banks once. (With r % 8 ^ r / 8 % 2 half of the
// LDS cycles were conflicts; 2048 x 8192: 1072 -> 1030 us.)
template <int PA, int PB, int WT, int KS, int NS>
struct NsTile {
    static constexpr int BT = 2 * WT, TB = WT / 16, STEPS = KS / 32;
    static constexpr int RBA = 2 * PA * KS, RBB = 2 * PB * KS;        // bytes of a row and stage
    static constexpr int CA = RBA / 16, CB = RBB / 16;                // chunks
    static constexpr int RSA = 256 / CA, RSB = 256 / CB;              // rows of a round of loads
    // (a last round past the tile's rows loads rows that nobody reads)
    static constexpr int RA = (BT + RSA - 1) / RSA, RB = (BT + RSB - 1) / RSB, NL = RA + RB;
    static constexpr int A_BYTES = RA * RSA * RBA, STAGE = A_BYTES + RB * RSB * RBB;
    static constexpr int PITCH = WT + 1, EPI = 4 * WT * PITCH * 4;
    static constexpr int LDS = NS * STAGE > EPI ? NS * STAGE : EPI;
    static_assert(LDS <= 160 * 1024 && NS >= 2 && (NS - 1) * NL < 64, "ring");

    template <int CHUNKS>
    static __device__ __forceinline__ int swz(int row) {
        return CHUNKS == 16 ? (row & 7) * 2 : CHUNKS == 8 ? row & 6 : (row >> 2) & 2;
    }
};

// 8 columns of a two-part row from column c0 (a multiple of 8) on.
__device__ __forceinline__ int64_t ns_column(int c0) { return (int64_t)(c0 / 32) * 64 + c0 % 32; }

// 8 words h | l << 16 into the row.
__device__ __forceinline__ void ns_store8(uint16_t *row, int c0, const uint32_t (&u)[8]) {
    ns_u32x4 h, l;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        h[d] = __builtin_amdgcn_perm(u[2 * d + 1], u[2 * d], 0x05040100u);
        l[d] = __builtin_amdgcn_perm(u[2 * d + 1], u[2 * d], 0x07060302u);
    }
    ns_u32x4 *to = reinterpret_cast<ns_u32x4 *>(row + ns_column(c0));
    to[0] = h;
    to[4] = l;
}

template <typename T, int MODE, int PA, int PB, int WT, int KS, int NS>
__global__ __launch_bounds__(256, 2) void ns_gemm_kernel(NsGemm p, NewtonSchulz q, int batch0) {
    typedef NsTile<PA, PB, WT, KS, NS> S;
    constexpr bool SYM = MODE == NS_SYM || MODE == NS_POLY || MODE == NS_PART;
    __shared__ __attribute__((aligned(16))) uint8_t smem[S::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // consecutive workgroups go to the 8 XCDs in turn, each with its own L2: give
    // every XCD a contiguous range of (matrix, product, tile)
    int bid = blockIdx.x;
    {
        const int n = gridDim.x, xcd = bid % 8, base = n / 8, rem = n % 8;
        bid = xcd * base + (xcd < rem ? xcd : rem) + bid / 8;
    }
    const int t = bid % p.tiles, jz = bid / p.tiles;
    const int jn = jz % p.jobs;
    const int64_t z = jz / p.jobs;
    const NsJob &job = p.job[MODE == NS_PART ? 0 : jn];
    const int k0 = MODE == NS_PART ? jn * p.slice : 0;
    int tm, tn;
    if (SYM)
        ns_lower_tile(t, p.tiles_m, tm, tn);
    else
        ns_tile(t, p.tiles_m, p.tiles / p.tiles_m, tm, tn);
    const int row0 = tm * S::BT, col0 = tn * S::BT;

    // (rows past the padding repeat the last: not stored)
    const uint8_t *srca[S::RA], *srcb[S::RB];
    {
        const int ra = tid / S::CA, ca = (tid % S::CA) ^ S::template swz<S::CA>(ra);
        const int rb = tid / S::CB, cb = (tid % S::CB) ^ S::template swz<S::CB>(rb);
        const uint16_t *pa = job.a.p + z * job.a.stride, *pb = job.b.p + z * job.b.stride;
#pragma unroll
        for (int i = 0; i < S::RA; ++i)
            srca[i] = reinterpret_cast<const uint8_t *>(pa + (int64_t)min(row0 + ra + i * S::RSA, p.M - 1) * job.a.ld + k0 * PA) + ca * 16;
#pragma unroll
        for (int i = 0; i < S::RB; ++i)
            srcb[i] = reinterpret_cast<const uint8_t *>(pb + (int64_t)min(col0 + rb + i * S::RSB, p.N - 1) * job.b.ld + k0 * PB) + cb * 16;
    }
    const int KT = (MODE == NS_PART ? min(p.K - k0, p.slice) : p.K) / KS;
    // (every call issues NL loads: stages past the last re-read it)
    auto dma = [&](int e) {
        const int kt = min(e, KT - 1);
        uint8_t *st = smem + (e % NS) * S::STAGE;
#pragma unroll
        for (int i = 0; i < S::RA; ++i)
            dma16(srca[i] + (int64_t)kt * S::RBA, st + (wave * (64 / S::CA) + i * S::RSA) * S::RBA);
#pragma unroll
        for (int i = 0; i < S::RB; ++i)
            dma16(srcb[i] + (int64_t)kt * S::RBB, st + S::A_BYTES + (wave * (64 / S::CB) + i * S::RSB) * S::RBB);
    };

    const int wm0 = (wave >> 1) * WT, wn0 = (wave & 1) * WT;
    constexpr int TB = S::TB;
    ns_f32x4 acc[TB][TB];
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            acc[i][j] = ns_f32x4{};
    // A stage's fragments: lane l has row l % 16 of a block and the 8 of K of quarter
    // l / 16 of a step.
    struct Frags {
        ns_i32x4 a[PA][TB], b[PB][TB];
    };
    auto read = [&](int e, int s, Frags &f) {
        const uint8_t *st = smem + (e % NS) * S::STAGE;
        const int q = lane >> 4, r = lane & 15;
        {
#pragma unroll
            for (int k = 0; k < TB; ++k) {
                const int ra = wm0 + k * 16 + r;
#pragma unroll
                for (int l = 0; l < PA; ++l)
                    f.a[l][k] = *reinterpret_cast<const ns_i32x4 *>(
                        st + ra * S::RBA + ((((s * PA + l) * 4 + q) ^ S::template swz<S::CA>(ra)) * 16));
            }
#pragma unroll
            for (int k = 0; k < TB; ++k) {
                const int rb = wn0 + k * 16 + r;
#pragma unroll
                for (int l = 0; l < PB; ++l)
                    f.b[l][k] = *reinterpret_cast<const ns_i32x4 *>(
                        st + S::A_BYTES + rb * S::RBB + ((((s * PB + l) * 4 + q) ^ S::template swz<S::CB>(rb)) * 16));
            }
        }
    };
    // products lo ... hi - 1 of a stage: in each step l h, h l, h h of each block
    constexpr int BLOCKS = TB * TB, TERMS = PA + PB - 1, NMF = BLOCKS * TERMS;
    auto mfmas = [&](const Frags &f, int lo, int hi) {
#pragma unroll
        for (int n = lo; n < hi; ++n) {
            const int term = n / BLOCKS, i = n % BLOCKS / TB, j = n % TB;
            const bool last = term == TERMS - 1;
            const int x = !last && PA == 2 && term == 0 ? 1 : 0, y = !last && x == 0 ? 1 : 0;
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(ns_f16x8, f.a[x][i]),
                                                               __builtin_bit_cast(ns_f16x8, f.b[y][j]), acc[i][j], 0, 0, 0);
        }
    };

    Frags f0, f1;
#pragma unroll
    for (int e = 0; e < NS; ++e)
        dma(e);
    wait_vm_lds<(NS - 1) * S::NL>();
    lds_barrier();
    read(0, 0, f0);
    // Under the products of a step the next step's fragments are read. The barrier says
    // that stage e + 1 has landed and that everybody has read stage e: the loads of stage
    // e + NS go into e's slot. (No branch in it: the compiler moves products past one.)
    auto step1 = [&](int e, const Frags &f, Frags &next) {   // stages of one step
        __builtin_amdgcn_sched_barrier(0);
        mfmas(f, 0, NMF / 2);
        __builtin_amdgcn_sched_barrier(0);
        wait_vm_lds<(NS - 2) * S::NL>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read(e + 1, 0, next);
        dma(e + NS);
        mfmas(f, NMF / 2, NMF);
        __builtin_amdgcn_sched_barrier(0);
    };
    int e = 0;
    if constexpr (S::STEPS == 1) {
        for (; e + 1 < KT; e += 2) {
            step1(e, f0, f1);
            step1(e + 1, f1, f0);
        }
        if (e < KT)
            step1(e, f0, f1);
    } else {
        for (; e < KT; ++e) {
            __builtin_amdgcn_sched_barrier(0);
            read(e, 1, f1);
            mfmas(f0, 0, NMF);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm_lds<(NS - 2) * S::NL>();
            lds_barrier();
            __builtin_amdgcn_sched_barrier(0);
            read(e + 1, 0, f0);
            dma(e + NS);
            mfmas(f1, 0, NMF);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Epilogue through LDS, a WT x WT block per wavefront: rows first (8 columns per
    // lane, stored along rows), then columns (stored into the transpose). Of a symmetric
    // matrix only what is on or below the diagonal is used, and the rest is its mirror
    // image: the results do not depend on the size of the tiles, and so not on the
    // batch. 16 x 16 blocks are below the diagonal (stored both ways), above it (not
    // stored) or on it (the elements above taken from below, stored along rows).
    constexpr int LPR = WT / 8, ITEMS = WT * LPR, PASSES = (ITEMS + 63) / 64;
    const int rb = row0 + wm0, cb = col0 + wn0;
    const bool inside = rb < p.M && cb < p.N && !(SYM && cb >= rb + WT);
    const float *fac = p.factors + z * p.fstride;
    const float kp = MODE == NS_PART ? 1.f : fac[job.factor];
    const float kadd = MODE == NS_POLY ? fac[NS_Q_ADD] : 0.f, kone = MODE == NS_POLY ? fac[NS_Q_ONE] : 0.f;
    auto item = [&](int i, int &r, int &c) {   // row and first column (or the other way round) of a lane's 8 elements
        const int g = i * 64 + lane;
        r = g / LPR;
        c = g % LPR * 8;
        return ITEMS % 64 == 0 || g < ITEMS;
    };
    // (all of `add` on its way before the accumulators go through LDS)
    constexpr int ADDS = MODE == NS_POLY ? PASSES : 1;
    ns_u32x4 ah[ADDS], al[ADDS];
    if constexpr (MODE == NS_POLY) {
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            int r, c;
            item(i, r, c);
            const ns_u32x4 *from = reinterpret_cast<const ns_u32x4 *>(
                job.add.p + z * job.add.stride + (int64_t)min(rb + r, p.M - 1) * job.add.ld + ns_column(min(cb + c, p.N - 8)));
            ah[i] = from[0];
            al[i] = from[4];
        }
    }
    // (the ring's last loads have landed and every wavefront is past its last read)
    wait_vm_lds<0>();
    __syncthreads();
    if (!inside)
        return;
    uint32_t *w = reinterpret_cast<uint32_t *>(smem) + wave * WT * S::PITCH;
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[(i * 16 + 4 * (lane >> 4) + r) * S::PITCH + j * 16 + (lane & 15)] = __float_as_uint(acc[i][j][r]);
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        int rl, c;
        if (!item(i, rl, c))
            continue;
        uint32_t *from = w + rl * S::PITCH + c;
        const int row = rb + rl, col = cb + c;
        if (row >= p.M || col >= p.N)
            continue;
        const int over = SYM ? (col & ~15) - (row & ~15) : -1;   // > 0 above the diagonal's blocks, 0 on it
        float v[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const bool mirror = SYM && over == 0 && col + d > row;
            v[d] = __uint_as_float(mirror ? w[(col + d - rb) * S::PITCH + row - cb] : from[d]) * kp;
        }
        if constexpr (MODE == NS_POLY) {
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const uint32_t hh = (ah[i][d / 2] >> (16 * (d & 1))) & 0xFFFF, ll = (al[i][d / 2] >> (16 * (d & 1))) & 0xFFFF;
                v[d] = __builtin_fmaf(kadd, ns_f32(hh) + ns_f32(ll), v[d]) + (row == col + d ? kone : 0.f);
            }
        }
        if constexpr (MODE == NS_OUT) {
            // Y's rows are the product's: X's, or with M > N the rows of X^T
            if (row < q.M) {
                T *Y = (T *)q.y + (batch0 + z) * q.stridey + (int64_t)row * q.ldy + col;
                T o[8];
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    o[d] = (T)v[d];
                if (col + 8 <= q.N && (reinterpret_cast<uintptr_t>(Y) & 15) == 0) {
                    ns_u32x4 u;
                    __builtin_memcpy(&u, o, 16);
                    *reinterpret_cast<ns_u32x4 *>(Y) = u;
                } else {
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        if (col + d < q.N)
                            Y[d] = o[d];
                }
            }
        } else if constexpr (MODE == NS_PART) {
            if (over <= 0) {
                ns_f32x4 *to = reinterpret_cast<ns_f32x4 *>(p.part + z * p.pstride + ((int64_t)jn * p.M + row) * p.M + col);
                to[0] = ns_f32x4{v[0], v[1], v[2], v[3]};
                to[1] = ns_f32x4{v[4], v[5], v[6], v[7]};
            }
        } else {
            uint32_t u[8];
#pragma unroll
            for (int d = 0; d < 8; ++d)
                u[d] = ns_split(v[d]);
            if (over < 0) {
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    from[d] = u[d];
            }
            if (over <= 0)
                ns_store8(job.out.p + z * job.out.stride + (int64_t)row * job.out.ld, col, u);
        }
    }
    if (MODE == NS_OUT || MODE == NS_PART || (SYM && cb >= rb + WT - 16))   // (nothing of the block is below the diagonal)
        return;
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        int cl, r;
        if (!item(i, cl, r))
            continue;
        const int row = cb + cl, col = rb + r;   // of the transpose
        if (row >= p.N || col >= p.M || (SYM && (row & ~15) >= (col & ~15)))
            continue;
        uint32_t u[8];
#pragma unroll
        for (int d = 0; d < 8; ++d)
            u[d] = w[(r + d) * S::PITCH + cl];
        ns_store8(job.outt.p + z * job.outt.stride + (int64_t)row * job.outt.ld, col, u);
    }
}

// A = the sum of the slices, in their order, of one 64 x 64 tile on or below the
// diagonal.
__global__ __launch_bounds__(256) void ns_join_kernel(NsGemm p) {
    __shared__ float tile[64][65];
    const int tid = threadIdx.x, t = blockIdx.x;
    const int64_t z = blockIdx.y;
    int tm, tn;
    ns_lower_tile(t, p.tiles_m, tm, tn);
    const int row0 = tm * 64, col0 = tn * 64;
    const float k = p.factors[z * p.fstride + NS_GRAM];
    const float *part = p.part + z * p.pstride;
    const int64_t size = (int64_t)p.M * p.M;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 16 + tid / 16, c = tid % 16 * 4;
        ns_f32x4 v = {};
        if ((col0 + c & ~15) <= (row0 + r & ~15))   // (the others are not there)
            for (int s = 0; s < p.jobs; ++s)
                v += *reinterpret_cast<const ns_f32x4 *>(part + s * size + (int64_t)(row0 + r) * p.M + col0 + c);
#pragma unroll
        for (int d = 0; d < 4; ++d)
            tile[r][c + d] = v[d] * k;
    }
    __syncthreads();
    const NsMat &out = p.job[0].out;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = i * 32 + tid / 8, c = tid % 8 * 8;
        uint32_t u[8], w[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            u[d] = ns_split(row0 == col0 && c + d > r ? tile[c + d][r] : tile[r][c + d]);
            w[d] = ns_split(tile[c + d][r]);
        }
        ns_store8(out.p + z * out.stride + (int64_t)(row0 + r) * out.ld, col0 + c, u);
        if (row0 != col0)
            ns_store8(out.p + z * out.stride + (int64_t)(col0 + r) * out.ld, row0 + c, w);
    }
}

// ------------------------------------------------------------ small matrices

// All steps of a group for matrices of MP x MP, one per workgroup: A comes from the slices
// of X X^T, A (in turn T) and Q stay in LDS, W in memory, where the apply takes it from.
// One 64 x 64: 74 -> 45 us, 64 x 4096: 166 -> 65 us, 16 of them 187 -> 83.
//
// In LDS a row is 4 MP bytes, 32 h and their 32 l in turn, its 16-byte chunks permuted
// within 256 bytes by the row as in NsTile. A lane's four sums are consecutive down a
// column; all matrices are symmetric, so they are stored along the row of that number.
// The next A is Q A Q with one Q on either side: nothing here makes the matrices
// symmetric, and Q Q A would lift A's roundings between large and small singular values by
// a^2 a step (128 x 128 of rank 1, four steps in bf16: off by 7e-2 of the norm), this by a.
struct NsSmall {
    const float *part;
    int64_t pstride;
    int slices, steps;
    NsMat w[2];             // the result in w[(steps - 1) % 2]
    const float *factors;   // of the group's first step
    int64_t fstride;
};

template <int MP>
__global__ __launch_bounds__(512) void ns_small_kernel(NsSmall p) {
    constexpr int ROW = MP * 4, SIZE = MP * ROW, WM = MP / 4, WN = MP / 2, TM = WM / 16, TN = WN / 16;
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * SIZE];
    constexpr int A = 0, Q = SIZE;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t z = blockIdx.x;
    const float *fac = p.factors + z * p.fstride;
    // byte of element k (of part l) of a row
    auto at = [](int row, int k, int l) {
        return row * ROW + (k / 64) * 256 + ((((k / 32 & 1) * 8 + l * 4 + k % 32 / 8) ^ (row & 7) * 2) * 16) + k % 8 * 2;
    };
    {
        const float *part = p.part + z * p.pstride, k = fac[NS_GRAM];
        for (int f = tid; f < MP * MP / 4; f += 512) {
            const int r = f / (MP / 4), c = f % (MP / 4) * 4;
            if ((c & ~15) > (r & ~15))   // (not there)
                continue;
            ns_f32x4 v = {};
            for (int s = 0; s < p.slices; ++s)
                v += *reinterpret_cast<const ns_f32x4 *>(part + ((int64_t)s * MP + r) * MP + c);
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (c + d <= r) {
                    const uint32_t u = ns_split(v[d] * k);
                    *reinterpret_cast<uint16_t *>(smem + A + at(r, c + d, 0)) = (uint16_t)u;
                    *reinterpret_cast<uint16_t *>(smem + A + at(r, c + d, 1)) = (uint16_t)(u >> 16);
                    *reinterpret_cast<uint16_t *>(smem + A + at(c + d, r, 0)) = (uint16_t)u;
                    *reinterpret_cast<uint16_t *>(smem + A + at(c + d, r, 1)) = (uint16_t)(u >> 16);
                }
        }
    }
    __syncthreads();

    const int m0 = (wave >> 1) * WM, n0 = (wave & 1) * WN, q = lane >> 4, r16 = lane & 15;
    typedef ns_f32x4 Acc[TM][TN];
    auto in_lds = [&](int x) {
        return [=](int row, int k, int l) { return *reinterpret_cast<const ns_i32x4 *>(smem + x + at(row, 32 * k + 8 * q, l)); };
    };
    auto in_memory = [&](const NsMat &x) {
        const uint16_t *from = x.p + z * x.stride;
        const int64_t ld = x.ld;
        return [=](int row, int k, int l) { return *reinterpret_cast<const ns_i32x4 *>(from + row * ld + 64 * k + 32 * l + 8 * q); };
    };
    // acc = x y^T
    auto product = [&](auto x, auto y, Acc &acc) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = ns_f32x4{};
#pragma unroll
        for (int k = 0; k < MP / 32; ++k) {
            ns_i32x4 a[2][TM], b[2][TN];
#pragma unroll
            for (int l = 0; l < 2; ++l) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    a[l][i] = x(m0 + 16 * i + r16, k, l);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    b[l][j] = y(n0 + 16 * j + r16, k, l);
            }
#pragma unroll
            for (int term = 0; term < 3; ++term)   // l h, h l, h h
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(ns_f16x8, a[term == 0][i]),
                                                                           __builtin_bit_cast(ns_f16x8, b[term == 1][j]),
                                                                           acc[i][j], 0, 0, 0);
        }
    };
    // four split values into row `row` from column c0 (a multiple of 4) on
    auto pack = [](const float (&v)[4], ns_u32x2 &h, ns_u32x2 &l) {
        uint32_t u[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
            u[d] = ns_split(v[d]);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            h[d] = __builtin_amdgcn_perm(u[2 * d + 1], u[2 * d], 0x05040100u);
            l[d] = __builtin_amdgcn_perm(u[2 * d + 1], u[2 * d], 0x07060302u);
        }
    };
    auto to_lds = [&](int x) {
        return [=](int row, int c0, ns_u32x2 h, ns_u32x2 l) {
            *reinterpret_cast<ns_u32x2 *>(smem + x + at(row, c0, 0)) = h;
            *reinterpret_cast<ns_u32x2 *>(smem + x + at(row, c0, 1)) = l;
        };
    };
    auto to_memory = [&](const NsMat &x) {
        uint16_t *to = x.p + z * x.stride;
        const int64_t ld = x.ld;
        return [=](int row, int c0, ns_u32x2 h, ns_u32x2 l) {
            *reinterpret_cast<ns_u32x2 *>(to + row * ld + ns_column(c0)) = h;
            *reinterpret_cast<ns_u32x2 *>(to + row * ld + ns_column(c0) + 32) = l;
        };
    };
    auto store = [&](const Acc &acc, float k, auto to) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = n0 + 16 * j + r16, c0 = m0 + 16 * i + 4 * q;
                const float v[4] = {acc[i][j][0] * k, acc[i][j][1] * k, acc[i][j][2] * k, acc[i][j][3] * k};
                ns_u32x2 h, l;
                pack(v, h, l);
                to(row, c0, h, l);
            }
    };

    Acc acc;
    for (int s = 0; s < p.steps; ++s, fac += NS_FACTORS) {
        // Q = a I + b A + c A A; the first is W too
        product(in_lds(A), in_lds(A), acc);
        const float kadd = fac[NS_Q_ADD], kone = fac[NS_Q_ONE], kacc = fac[NS_Q_ACC];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = n0 + 16 * j + r16, c0 = m0 + 16 * i + 4 * q;
                const ns_u32x2 h = *reinterpret_cast<const ns_u32x2 *>(smem + A + at(row, c0, 0));
                const ns_u32x2 l = *reinterpret_cast<const ns_u32x2 *>(smem + A + at(row, c0, 1));
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float x = ns_f32(h[d / 2] >> (16 * (d & 1)) & 0xFFFF) + ns_f32(l[d / 2] >> (16 * (d & 1)) & 0xFFFF);
                    acc[i][j][d] = __builtin_fmaf(kadd, x, acc[i][j][d] * kacc) + (row == c0 + d ? kone : 0.f);
                }
            }
        store(acc, 1.f, to_lds(Q));
        if (s == 0)
            store(acc, 1.f, to_memory(p.w[0]));
        __syncthreads();
        if (s > 0) {   // W <- Q W
            product(in_lds(Q), in_memory(p.w[(s - 1) & 1]), acc);
            store(acc, fac[NS_W], to_memory(p.w[s & 1]));
        }
        if (s + 1 < p.steps) {
            product(in_lds(A), in_lds(Q), acc);   // T = Q A (stored as the transpose of A Q) in A's place
            __syncthreads();
            store(acc, fac[NS_T], to_lds(A));
            __syncthreads();
            product(in_lds(Q), in_lds(A), acc);   // A <- Q T^T = Q A Q
            __syncthreads();
            store(acc, fac[NS_A], to_lds(A));
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------ host

namespace {

struct NsPlan {
    int64_t mp, np;          // padded sizes
    int64_t per;             // bytes per matrix
    int64_t chunk;           // matrices in one go
    int64_t sums;            // partial sums of squares
};

constexpr int kMaxSteps = 100;

// Matrices are processed in chunks whose scratch stays below 4 GiB (one matrix
// at least), which keeps the workspace of a long batch bounded.
NsPlan ns_plan(int64_t batch, int64_t M, int64_t N) {
    NsPlan pl;
    const int64_t m = M < N ? M : N, n = M < N ? N : M;
    pl.mp = (m + 63) / 64 * 64;
    pl.np = (n + 63) / 64 * 64;
    pl.sums = (pl.mp / 64) * (pl.np / 64);
    if (pl.sums > NS_SUMS)
        pl.sums = NS_SUMS;
    pl.per = 3 * pl.mp * pl.np * 4 + 5 * pl.mp * pl.mp * 4 + pl.sums * 8 + kMaxSteps * NS_FACTORS * 4;
    const int64_t most = (int64_t)4 << 30;
    pl.chunk = most / pl.per;
    if (pl.chunk < 1)
        pl.chunk = 1;
    if (pl.chunk > batch)
        pl.chunk = batch;
    return pl;
}

// Steps between two A = X X^T. A's own rounding grows within a group, in the directions
// of small singular values, and reaches Q through b A. Taken to be off by 2^-23 a^(2 (L - 1)) of
// the norm after L steps (a Q Q A that nothing makes symmetric: 2.1e-3 for L = 5, a = 3.4445),
// below 1/8 of a half step of the output type: four steps for bf16, three for fp16 with
// these coefficients, and five steps are three and two. It is less where A stays
// symmetric: 3e-5 for L = 4 on rank 4, next to 1e-5 of the iteration in fp32. That is the group's
// share; what the rounding of X itself leaves grows by a per step however the steps are
// grouped (see the public header).
int group_length(int type, float a) {
    const double limit = type == MPGEMM_TYPE_F16 ? 0x1p-14 : 0x1p-11;
    const double grow = (double)a * a > 1. ? (double)a * a : 1.;
    double err = 0x1p-23;
    int len = 1;
    while (len < 8 && err * grow <= limit) {
        err *= grow;
        ++len;
    }
    return len;
}

}  // namespace

// The exponents follow a bound r of X's largest singular value, r <- max |x Q(x)| over
// [0, r] from 1 on, while the value itself may start as small as 1 / sqrt(m) >= 2^-8.
// fp16's h + l have 2^-37 of r; the polynomial must keep whatever starts in [2^-8, 1]
// above 2^-14 r, which leaves them 22 bits. (a, b, c) that orthogonalise do. Powers
// (a = 0) and polynomials that grow with every step do not: r and the matrix part by
// the third or fifth power of what they were apart, at every step.
bool newton_schulz_supported(int steps, float a, float b, float c) {
    constexpr int POINTS = 33, GRID = 64;
    float x[POINTS], r = 1.f;
    for (int i = 0; i < POINTS; ++i)
        x[i] = exp2f(-8.f + 0.25f * (float)i);
    auto next = [&](float v) { return v * (a + v * v * (b + v * v * c)); };
    for (int k = 0; k < steps; ++k) {
        float top = 0.f;
        for (int i = 1; i <= GRID; ++i)
            top = fmaxf(top, fabsf(next(r * (float)i / GRID)));
        for (int i = 0; i < POINTS; ++i) {
            x[i] = next(x[i]);
            if (!(fabsf(x[i]) >= 0x1p-14f * top) || !(top < FLT_MAX))
                return false;
        }
        r = top;
    }
    return true;
}

int64_t newton_schulz_bytes(int64_t batch, int64_t M, int64_t N) {
    if (batch == 0 || M == 0 || N == 0)
        return 0;
    const NsPlan pl = ns_plan(batch, M, N);
    return (pl.chunk * pl.per + 255) / 256 * 256;
}

// Tile sizes: us for a stage and for the ends of a workgroup that has a CU for itself
// (symmetric 2048 x 2048 on 528, 253 and 136 workgroups: 36.8, 31.0 and 47.1 us; 12 of 512 x 512 on
// 432, 252 and 120: 11.2, 14.6 and 20.5; 2048 x 8192 on 4096, 1892 and 1024: 181, 149 and 130). 32 has the
// most workgroups, 64 the fewest loads per flop.
struct NsSize {
    int wt;
    double stage, ends;
};
static const NsSize kNsSizes[] = {{32, 0.21, 0.3}, {48, 0.40, 3.0}, {64, 0.63, 4.4}};

template <typename T, int MODE, int PA, int PB>
static void ns_product(NsGemm g, const NewtonSchulz &p, int z0, int cus, hipStream_t stream) {
    constexpr bool sym = MODE == NS_SYM || MODE == NS_POLY;
    constexpr int KS = PA + PB == 2 ? 64 : 32;
    auto count = [&](int bt) {
        const int64_t tm = (g.M + bt - 1) / bt, tn = (g.N + bt - 1) / bt;
        return sym ? tm * (tm + 1) / 2 : tm * tn;
    };
    int wt = 32;
    double best = 0;
    for (const NsSize &z : kNsSizes) {
        // workgroups per CU, a begun one for half (they run side by side)
        const double r = (double)(count(2 * z.wt) * g.jobs * g.nz) / cus, rounds = r <= 1 ? 1 : (r + ceil(r)) / 2;
        const double cost = rounds * (g.K / KS * z.stage + z.ends);
        if (z.wt == 32 || cost < best) {
            best = cost;
            wt = z.wt;
        }
    }
    g.tiles_m = (g.M + 2 * wt - 1) / (2 * wt);
    g.tiles = (int)count(2 * wt);
    const dim3 grid((unsigned)((int64_t)g.tiles * g.jobs * g.nz));
    // Workgroups that have a CU for themselves wait at their barriers for nobody's benefit
    // and for loads from beyond L2: deeper rings, and for tiles of 64 stages of two steps, half
    // the barriers (1024 x 1024: 300 -> 212 us). Where several share a CU small rings let more of
    // them in (symmetric 2048 on 528 tiles of 64: 36.8 -> 49.4; 2048 x 8192 on 1024 of 128: 130 ->
    // 167). In between, tiles of 64 in stages of two steps, without the depth: on 300
    // 28.0 -> 22.6, on 432 11.2 -> 11.9.
    const bool alone = grid.x <= (unsigned)cus;
    if (wt == 32 && alone)
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 32, 64, 4>), grid, dim3(256), 0, stream, g, p, z0);
    else if (wt == 32 && 2 * (int64_t)grid.x <= 3 * (int64_t)cus)
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 32, 64, 2>), grid, dim3(256), 0, stream, g, p, z0);
    else if (wt == 32)
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 32, KS, 2>), grid, dim3(256), 0, stream, g, p, z0);
    else if (wt == 48 && alone)
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 48, KS, 3>), grid, dim3(256), 0, stream, g, p, z0);
    else if (wt == 48)
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 48, KS, 2>), grid, dim3(256), 0, stream, g, p, z0);
    else if (alone)
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 64, KS, 4>), grid, dim3(256), 0, stream, g, p, z0);
    else
        hipLaunchKernelGGL((ns_gemm_kernel<T, MODE, PA, PB, 64, KS, 2>), grid, dim3(256), 0, stream, g, p, z0);
}

template <typename T, bool VEC>
static hipError_t ns_type(int type, const NewtonSchulz &p, void *workspace, hipStream_t stream) {
    const NsPlan pl = ns_plan(p.batch, p.M, p.N);
    const bool flip = p.M > p.N;
    const int mp = (int)pl.mp, np = (int)pl.np;
    const int64_t xs = pl.mp * pl.np, as = pl.mp * pl.mp;
    uint16_t *w = (uint16_t *)workspace;
    auto mat = [&](int64_t ld, int64_t size) {   // two parts
        NsMat r = {w, 2 * ld, 2 * size};
        w += 2 * pl.chunk * size;
        return r;
    };
    auto one = [](NsMat m) {   // one part in the same place
        m.ld /= 2;
        m.stride /= 2;
        return m;
    };
    const NsMat X = mat(np, xs);
    NsMat XT = mat(mp, xs), XT2 = mat(mp, xs);
    const NsMat A = mat(mp, as), Tm = mat(mp, as);
    NsMat Q = mat(mp, as), W = mat(mp, as), W2 = mat(mp, as);
    double *sums = (double *)w;
    float *factors = (float *)(sums + pl.chunk * pl.sums);
    const int across = (p.N + 63) / 64, tiles = across * ((p.M + 63) / 64), count = (int)pl.sums;

    // Per step and m^3 flop: L steps in a group cost (3 n / m + 4 L - 3) / L products. For a
    // square matrix that is 4 whatever L is, and single steps need fewer launches
    // (12 x 512 x 512: a fifth less time).
    const bool small = mp <= 128;
    const int most = small || pl.np * 4 >= pl.mp * 5 ? group_length(type, p.a) : 1, groups = (p.steps + most - 1) / most;
    NsGroups gr = {1, 0};
    if (groups > 0) {
        gr.len = p.steps / groups;
        gr.longer = p.steps % groups;
    }

    // A of few tiles and a long n: slices of n, of 256 at least, as many as give the tiles
    // of one matrix a workgroup per CU. 256 x 4096 227 -> 182 us, 700 x 3000 315 -> 271, four of
    // 500 x 4000 327 -> 292; with n = 2 m the join costs more than it gives (16 of 512 x 1024:
    // 342 -> 361). ns_small_kernel adds them up in one workgroup, so few of 128 x 128. Not a
    // matter of the batch: the sums are the same in any.
    const int t64 = mp / 64, tiles64 = t64 * (t64 + 1) / 2;
    int split = np / (mp == 128 ? 512 : 256);
    for (const int most_slices : {mp == 128 ? 8 : 16, np / mp, 256 / tiles64})
        split = split < most_slices ? split : most_slices;
    if (split < 1 || (!small && np / mp < 4))
        split = 1;
    const int slice = (np / 64 + split - 1) / split * 64;
    split = (np + slice - 1) / slice;

    for (int64_t b0 = 0; b0 < p.batch; b0 += pl.chunk) {
        const int nz = (int)(p.batch - b0 < pl.chunk ? p.batch - b0 : pl.chunk);
        const int z0 = (int)b0;
        hipLaunchKernelGGL((ns_square_kernel<T, VEC>), dim3(count, nz), dim3(256), 0, stream, p, z0, across, tiles, sums);
        if (p.steps == 0) {
            const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
            hipLaunchKernelGGL((ns_scale_kernel<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096), 1, nz), dim3(256), 0, stream, p, z0, sums, count);
        } else if (flip) {
            hipLaunchKernelGGL((ns_load_kernel<T, true, VEC>), dim3(mp / 64, np / 64, nz), dim3(256), 0, stream, p, gr, z0, sums, count, factors, one(X), one(XT));
        } else {
            hipLaunchKernelGGL((ns_load_kernel<T, false, VEC>), dim3(np / 64, mp / 64, nz), dim3(256), 0, stream, p, gr, z0, sums, count, factors, one(X), one(XT));
        }
        for (int s = 0; s < p.steps; ++s) {
            const bool first = gr.starts(s), last = s + 1 == p.steps, ends = last || gr.starts(s + 1);
            NsGemm g = {};
            g.jobs = 1;
            g.nz = nz;
            g.M = g.N = mp;
            g.factors = factors + (int64_t)s * NS_FACTORS;
            g.fstride = (int64_t)p.steps * NS_FACTORS;
            if (first) {   // A = X X^T
                g.K = np;
                g.job[0] = {X, X, A, A, A, NS_GRAM};
                if (s == 0)
                    g.job[0].a = g.job[0].b = one(X);
                if (split > 1 || small) {
                    g.part = reinterpret_cast<float *>(XT2.p);   // (free between two applies)
                    g.pstride = xs;
                    g.slice = slice;
                    g.jobs = split;
                    g.tiles = tiles64;
                    g.tiles_m = t64;
                    const dim3 grid((unsigned)((int64_t)tiles64 * split * nz));
                    if (s == 0)
                        hipLaunchKernelGGL((ns_gemm_kernel<T, NS_PART, 1, 1, 32, 64, 4>), grid, dim3(256), 0, stream, g, p, z0);
                    else
                        hipLaunchKernelGGL((ns_gemm_kernel<T, NS_PART, 2, 2, 32, 64, 4>), grid, dim3(256), 0, stream, g, p, z0);
                    if (!small)
                        hipLaunchKernelGGL(ns_join_kernel, dim3(tiles64, nz), dim3(256), 0, stream, g);
                } else if (s == 0) {
                    ns_product<T, NS_SYM, 1, 1>(g, p, z0, p.cus, stream);
                } else {
                    ns_product<T, NS_SYM, 2, 2>(g, p, z0, p.cus, stream);
                }
                if (small) {   // the whole group
                    int len = 1;
                    while (s + len < p.steps && !gr.starts(s + len))
                        ++len;
                    const NsSmall q = {g.part, g.pstride, split, len, {W, W2}, g.factors, g.fstride};
                    if (mp == 64)
                        hipLaunchKernelGGL((ns_small_kernel<64>), dim3(nz), dim3(512), 0, stream, q);
                    else
                        hipLaunchKernelGGL((ns_small_kernel<128>), dim3(nz), dim3(512), 0, stream, q);
                    if (len % 2 == 0) {
                        const NsMat t = W;
                        W = W2;
                        W2 = t;
                    }
                }
                g.jobs = 1;
            }
            if (!small) {
                g.K = mp;
                g.job[0] = {A, A, A, Q, Q, NS_Q_ACC};
                ns_product<T, NS_POLY, 2, 2>(g, p, z0, p.cus, stream);
                // T = Q A and W <- Q W, side by side (the first W is Q itself, the last T is not needed)
                g.jobs = 0;
                if (!ends)
                    g.job[g.jobs++] = {Q, A, A, Tm, Tm, NS_T};
                if (!first)
                    g.job[g.jobs++] = {Q, W, W, W2, W2, NS_W};
                if (g.jobs)
                    ns_product<T, NS_SYM, 2, 2>(g, p, z0, p.cus, stream);
                if (!ends) {   // A <- Q T
                    g.jobs = 1;
                    g.job[0] = {Q, Tm, A, A, A, NS_A};
                    ns_product<T, NS_SYM, 2, 2>(g, p, z0, p.cus, stream);
                }
                if (first) {
                    const NsMat t = Q;
                    Q = W;
                    W = t;
                } else {
                    const NsMat t = W;
                    W = W2;
                    W2 = t;
                }
            }
            if (!ends)
                continue;
            // X <- W X; X^T is the operand whose rows run along the contracted axis
            g.jobs = 1;
            g.K = mp;
            const bool exact = s + 1 <= gr.len + (gr.longer > 0);   // G's own X: one part
            const NsMat xt = exact ? one(XT) : XT;
            if (last && !flip) {
                g.M = mp;
                g.N = np;
                g.job[0] = {W, xt, W, X, X, NS_APPLY};
                if (exact)
                    ns_product<T, NS_OUT, 2, 1>(g, p, z0, p.cus, stream);
                else
                    ns_product<T, NS_OUT, 2, 2>(g, p, z0, p.cus, stream);
            } else if (last) {
                g.M = np;
                g.N = mp;
                g.job[0] = {xt, W, W, X, X, NS_APPLY};
                if (exact)
                    ns_product<T, NS_OUT, 1, 2>(g, p, z0, p.cus, stream);
                else
                    ns_product<T, NS_OUT, 2, 2>(g, p, z0, p.cus, stream);
            } else {
                g.M = mp;
                g.N = np;
                g.job[0] = {W, xt, W, X, XT2, NS_APPLY};
                if (exact)
                    ns_product<T, NS_X, 2, 1>(g, p, z0, p.cus, stream);
                else
                    ns_product<T, NS_X, 2, 2>(g, p, z0, p.cus, stream);
                const NsMat t = XT;
                XT = XT2;
                XT2 = t;
            }
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_newton_schulz(int type, const NewtonSchulz &p, void *workspace, hipStream_t stream) {
    // (both types have 2 bytes)
    const bool vec = (reinterpret_cast<uintptr_t>(p.g) & 15) == 0 && p.ldg % 8 == 0 && p.strideg % 8 == 0;
    if (type == MPGEMM_TYPE_F16)
        return vec ? ns_type<_Float16, true>(type, p, workspace, stream) : ns_type<_Float16, false>(type, p, workspace, stream);
    return vec ? ns_type<__bf16, true>(type, p, workspace, stream) : ns_type<__bf16, false>(type, p, workspace, stream);
}

}  // namespace mpg
