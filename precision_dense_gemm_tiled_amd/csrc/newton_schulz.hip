// Newton-Schulz orthogonalisation of a batch of matrices:
//   X = G / (|G|_F + eps), then `steps` times
//   A = X X^T,  P = b A + c A A,  X <- a X + P X
// on the smaller side (X is m x n with m <= n, G or its transpose).
//
// Every product is of fp32 quality at the bf16 matrix rate: each factor is held
// as the sum of two bf16 values, h + l (h = bf16(x), l = bf16(x - h): 16
// significant bits with the full range of fp32), and a product is
// h h + h l + l h with fp32 sums; l l is below the rounding of the sum. One
// bf16 (or fp16) value per factor is not enough: the polynomial multiplies the
// small singular values by about a at every step (485 times in all with the
// usual coefficients), and their rounding errors with them. Measured against
// 64 bits on gradients of rank 64 plus noise, 1024 x 256: 2.3e-2 with one bf16
// value, 3e-3 with one fp16 value, 2e-4 (the output's own rounding, fp16) with
// two.
//
// Layout: X is needed with n contiguous (A = X X^T contracts over n) and with m
// contiguous (P X contracts over m), so both are stored; A and P are symmetric
// and only the tiles on and below the diagonal are computed, the others
// mirrored. Rows and columns are padded with zeros to multiples of 64, which
// the products keep zero.
#include <cfloat>

#include "mxfp4.h"
#include "lds_dma.h"

namespace mpg {

typedef int ns_i32x4 __attribute__((ext_vector_type(4)));
typedef float ns_f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 ns_bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t ns_u32x2 __attribute__((ext_vector_type(2)));

// A matrix of h and l parts, rows of `ld` elements.
struct NsMat {
    uint16_t *h, *l;
    int64_t ld, stride;   // elements; stride between matrices of the batch
};

__device__ __forceinline__ uint16_t ns_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ float ns_f32(uint32_t h) { return __uint_as_float(h << 16); }

// x as h | l << 16
__device__ __forceinline__ uint32_t ns_split(float x) {
    const uint16_t h = ns_bf16(x);
    return h | ((uint32_t)ns_bf16(x - ns_f32(h)) << 16);
}

// Sum over the workgroup's 256 threads, in every thread, in a fixed order.
__device__ __forceinline__ float ns_block_sum(float v, float *red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// G (M x N) -> X (m x n, padded) and X^T, unscaled, and the sum of squares of
// each 64 x 64 tile. FLIP: G is taller than wide, X = G^T.
template <typename T, bool FLIP>
__global__ __launch_bounds__(256) void ns_load_kernel(NewtonSchulz p, int batch0, NsMat X, NsMat XT, float *sums) {
    __shared__ uint32_t tile[64][65];
    __shared__ float red[4];
    const int tid = threadIdx.x;
    const T *G = (const T *)p.g + (int64_t)(batch0 + blockIdx.z) * p.strideg;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    const NsMat own = FLIP ? XT : X, other = FLIP ? X : XT;   // own: rows as G's
    const int64_t ob = (int64_t)blockIdx.z * own.stride, tb = (int64_t)blockIdx.z * other.stride;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int rl = i * 4 + tid / 64, cl = tid & 63;
        const int row = r0 + rl, col = c0 + cl;
        const float x = row < p.M && col < p.N ? (float)G[(int64_t)row * p.ldg + col] : 0.f;
        sq += x * x;
        const uint32_t w = ns_split(x);
        own.h[ob + (int64_t)row * own.ld + col] = (uint16_t)w;
        own.l[ob + (int64_t)row * own.ld + col] = (uint16_t)(w >> 16);
        tile[rl][cl] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int cl = i * 4 + tid / 64, rl = tid & 63;
        const uint32_t w = tile[rl][cl];
        other.h[tb + (int64_t)(c0 + cl) * other.ld + r0 + rl] = (uint16_t)w;
        other.l[tb + (int64_t)(c0 + cl) * other.ld + r0 + rl] = (uint16_t)(w >> 16);
    }
    const float s = ns_block_sum(sq, red);
    if (tid == 0)
        sums[((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = s;
}

// inv[z] = 1 / (sqrt(sum of the tiles' sums) + eps)
__global__ __launch_bounds__(256) void ns_norm_kernel(const float *sums, int tiles, float eps, float *inv) {
    __shared__ float red[4];
    float s = 0.f;
    for (int i = threadIdx.x; i < tiles; i += 256)
        s += sums[(int64_t)blockIdx.x * tiles + i];
    s = ns_block_sum(s, red);
    if (threadIdx.x == 0) {
        const float d = sqrtf(s) + eps;
        inv[blockIdx.x] = d > 0.f ? fminf(1.f / d, FLT_MAX) : 1.f / d;   // (finite, so that zeros stay zeros)
    }
}

// Y = inv G (no steps)
template <typename T>
__global__ __launch_bounds__(256) void ns_scale_kernel(NewtonSchulz p, int batch0, const float *inv) {
    const int z = batch0 + blockIdx.z;
    const T *G = (const T *)p.g + (int64_t)z * p.strideg;
    T *Y = (T *)p.y + (int64_t)z * p.stridey;
    const int64_t total = (int64_t)p.M * p.N;
    for (int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x; f < total; f += (int64_t)gridDim.x * 256) {
        const int64_t r = f / p.N, c = f - r * p.N;
        Y[r * p.ldy + c] = (T)((float)G[r * p.ldg + c] * inv[blockIdx.z]);
    }
}

enum { NS_GRAM = 0, NS_POLY = 1, NS_STEP = 2, NS_LAST = 3 };

struct NsGemm {
    NsMat a, b;        // operands, K contiguous
    int M, N, K;       // padded to 64
    NsMat add;         // POLY: A; STEP, LAST: X (the old iterate)
    NsMat out, outt;   // result and its transpose (STEP: X and X^T)
    float ka, kc;      // result = ka * add + kc * (a b^T)
    const float *inv;  // the first step's factors: GRAM scales by inv^2, STEP and LAST by inv; or null
};

// C tile of 128 x 128 per workgroup, four wavefronts of 64 x 64, stages of 32 of
// K (64 bytes per row and part) in a two-slot LDS ring. 16-byte chunk c of LDS
// row r at c ^ swz(r).
template <typename T, int MODE>
__global__ __launch_bounds__(256) void ns_gemm_kernel(NsGemm p, NewtonSchulz q, int batch0, int tiles_m,
                                                      int tiles_n) {
    constexpr int BT = 128, BKB = 64, CPR = 4, RS = 64, PART = BT * BKB, STAGE = 4 * PART;
    constexpr int PITCH = 65;
    constexpr int LDS = 2 * STAGE > 4 * 64 * PITCH * 4 ? 2 * STAGE : 4 * 64 * PITCH * 4;
    __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr bool SYM = MODE == NS_GRAM || MODE == NS_POLY;
    int tm, tn;
    if (SYM) {   // lower triangle: tile t is (tm, tn), tn <= tm
        tm = (int)((sqrtf(8.f * blockIdx.x + 1.f) - 1.f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= (int)blockIdx.x)
            ++tm;
        while (tm * (tm + 1) / 2 > (int)blockIdx.x)
            --tm;
        tn = blockIdx.x - tm * (tm + 1) / 2;
    } else {
        tm = blockIdx.x % tiles_m;
        tn = blockIdx.x / tiles_m;
    }
    const int row0 = tm * BT, col0 = tn * BT;
    const int64_t z = blockIdx.z;
    auto swz = [](int row) { return ((row >> 1) & 3) ^ ((row >> 3) & 1); };

    const int r0 = tid / CPR, cg = (tid % CPR) ^ swz(r0);
    const uint8_t *base[4] = {(const uint8_t *)(p.a.h + z * p.a.stride), (const uint8_t *)(p.a.l + z * p.a.stride),
                              (const uint8_t *)(p.b.h + z * p.b.stride), (const uint8_t *)(p.b.l + z * p.b.stride)};
    int64_t off[4];   // rows row0 + r0 (+ 64), col0 + r0 (+ 64)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool isa = i < 2;
        int r = (isa ? row0 : col0) + r0 + (i & 1) * RS;
        r = min(r, (isa ? p.M : p.N) - 1);   // (rows past the padding repeat: not stored)
        off[i] = (int64_t)r * (isa ? p.a.ld : p.b.ld) * 2 + cg * 16;
    }
    const int KT = p.K / 32;
    auto dma = [&](int e) {
        const int kt = min(e, KT - 1);
#pragma unroll
        for (int part = 0; part < 4; ++part)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                dma16(base[part] + off[(part >> 1) * 2 + i] + (int64_t)kt * BKB,
                      smem + (e & 1) * STAGE + part * PART + (wave * 16 + i * RS) * BKB);
    };

    const int wm0 = (wave >> 1) * 64, wn0 = (wave & 1) * 64;
    ns_f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            acc[i][j] = ns_f32x16{};
    dma(0);
    for (int e = 0; e < KT; ++e) {
        // this wavefront's loads of stage e have landed; the barrier makes them
        // everybody's, and says that stage e - 1 has been read
        wait_vm_lds<0>();
        lds_barrier();
        dma(e + 1);
        const uint8_t *S = smem + (e & 1) * STAGE;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = 2 * s + (lane >> 5);
            ns_i32x4 f[4][2];
#pragma unroll
            for (int part = 0; part < 4; ++part)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = (part < 2 ? wm0 : wn0) + i * 32 + (lane & 31);
                    f[part][i] = *reinterpret_cast<const ns_i32x4 *>(S + part * PART + r * BKB + ((c ^ swz(r)) * 16));
                }
            auto mf = [&](int x, int y) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            __builtin_bit_cast(ns_bf16x8, f[x][i]), __builtin_bit_cast(ns_bf16x8, f[y][j]),
                            acc[i][j], 0, 0, 0);
            };
            mf(1, 2);
            mf(0, 3);
            mf(0, 2);
        }
    }
    wait_vm_lds<0>();
    __syncthreads();

    // Epilogue through LDS, a 64 x 64 block per wavefront: rows first (old
    // values added, stored along rows), then columns (stored into the transpose).
    uint32_t *w = reinterpret_cast<uint32_t *>(smem) + wave * 64 * PITCH;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                w[(i * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4) * PITCH + j * 32 + (lane & 31)] =
                    __float_as_uint(acc[i][j][r]);
    wave_lds_fence();
    const int rb = row0 + wm0, cb = col0 + wn0;
    if (rb >= p.M || cb >= p.N)   // (whole 64 x 64 blocks: the padding's granularity)
        return;
    float kx = p.ka, kp = p.kc;
    if (p.inv) {
        const float s = p.inv[z];
        if (MODE == NS_GRAM) {
            kp = s;   // applied twice below: s * s may leave the range of fp32
        } else {
            kx *= s;
            kp *= s;
        }
    }
    const int lr = lane >> 4, lc = lane & 15;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int rl = i * 4 + lr;
        uint32_t *src = w + rl * PITCH + lc * 4;
        float v[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
            v[d] = __uint_as_float(src[d]) * kp;
        if (MODE == NS_GRAM && p.inv) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                v[d] *= kp;
        }
        const int row = rb + rl, col = cb + lc * 4;
        if constexpr (MODE != NS_GRAM) {
            const int64_t o = z * p.add.stride + (int64_t)row * p.add.ld + col;
            const ns_u32x2 h = *reinterpret_cast<const ns_u32x2 *>(p.add.h + o);
            const ns_u32x2 l = *reinterpret_cast<const ns_u32x2 *>(p.add.l + o);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t hh = (h[d / 2] >> (16 * (d & 1))) & 0xFFFF, ll = (l[d / 2] >> (16 * (d & 1))) & 0xFFFF;
                v[d] = __builtin_fmaf(kx, ns_f32(hh) + ns_f32(ll), v[d]);
            }
        }
        if constexpr (MODE == NS_LAST) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                src[d] = __float_as_uint(v[d]);
            if (q.M <= q.N && row < q.M) {
                T *Y = (T *)q.y + (batch0 + z) * q.stridey + (int64_t)row * q.ldy;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (col + d < q.N)
                        Y[col + d] = (T)v[d];
            }
        } else {
            uint32_t t[4];
#pragma unroll
            for (int d = 0; d < 4; ++d)
                src[d] = t[d] = ns_split(v[d]);
            const int64_t o = z * p.out.stride + (int64_t)row * p.out.ld + col;
            *reinterpret_cast<ns_u32x2 *>(p.out.h + o) =
                ns_u32x2{(t[0] & 0xFFFF) | (t[1] << 16), (t[2] & 0xFFFF) | (t[3] << 16)};
            *reinterpret_cast<ns_u32x2 *>(p.out.l + o) =
                ns_u32x2{(t[0] >> 16) | (t[1] & 0xFFFF0000u), (t[2] >> 16) | (t[3] & 0xFFFF0000u)};
        }
    }
    if (SYM && tm == tn)
        return;   // the wavefronts of a diagonal tile store all of it along rows
    if (MODE == NS_LAST && q.M <= q.N)
        return;
    wave_lds_fence();
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int cl = i * 4 + lr;
        uint32_t t[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
            t[d] = w[(lc * 4 + d) * PITCH + cl];
        const int row = cb + cl, col = rb + lc * 4;   // of the transpose
        if constexpr (MODE == NS_LAST) {
            if (row < q.M) {
                T *Y = (T *)q.y + (batch0 + z) * q.stridey + (int64_t)row * q.ldy;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (col + d < q.N)
                        Y[col + d] = (T)__uint_as_float(t[d]);
            }
        } else {
            const int64_t o = z * p.outt.stride + (int64_t)row * p.outt.ld + col;
            *reinterpret_cast<ns_u32x2 *>(p.outt.h + o) =
                ns_u32x2{(t[0] & 0xFFFF) | (t[1] << 16), (t[2] & 0xFFFF) | (t[3] << 16)};
            *reinterpret_cast<ns_u32x2 *>(p.outt.l + o) =
                ns_u32x2{(t[0] >> 16) | (t[1] & 0xFFFF0000u), (t[2] >> 16) | (t[3] & 0xFFFF0000u)};
        }
    }
}

namespace {

struct NsPlan {
    int64_t mp, np;          // padded sizes
    int64_t per;             // bytes per matrix
    int64_t chunk;           // matrices in one go
    int64_t tiles;
};

// Matrices are processed in chunks whose scratch stays below 4 GiB (one matrix
// at least), which keeps the workspace of a long batch bounded.
NsPlan ns_plan(int64_t batch, int64_t M, int64_t N) {
    NsPlan pl;
    const int64_t m = M < N ? M : N, n = M < N ? N : M;
    pl.mp = (m + 63) / 64 * 64;
    pl.np = (n + 63) / 64 * 64;
    pl.tiles = (pl.mp / 64) * (pl.np / 64);
    pl.per = 3 * pl.mp * pl.np * 4 + 2 * pl.mp * pl.mp * 4 + (pl.tiles + 1) * 4;
    const int64_t most = (int64_t)4 << 30;
    pl.chunk = most / pl.per;
    if (pl.chunk < 1)
        pl.chunk = 1;
    if (pl.chunk > batch)
        pl.chunk = batch;
    return pl;
}

}  // namespace

int64_t newton_schulz_bytes(int64_t batch, int64_t M, int64_t N) {
    if (batch == 0 || M == 0 || N == 0)
        return 0;
    const NsPlan pl = ns_plan(batch, M, N);
    return (pl.chunk * pl.per + 255) / 256 * 256;
}

template <typename T>
static hipError_t ns_type(const NewtonSchulz &p, void *workspace, hipStream_t stream) {
    const NsPlan pl = ns_plan(p.batch, p.M, p.N);
    const bool flip = p.M > p.N;
    const int mp = (int)pl.mp, np = (int)pl.np;
    const int64_t xs = pl.mp * pl.np, as = pl.mp * pl.mp;
    uint16_t *w = (uint16_t *)workspace;
    auto mat = [&](int64_t ld, int64_t size) {
        NsMat r = {w, w + pl.chunk * size, ld, size};
        w += 2 * pl.chunk * size;
        return r;
    };
    const NsMat X = mat(np, xs);
    NsMat XT[2];
    XT[0] = mat(mp, xs);
    XT[1] = mat(mp, xs);
    const NsMat A = mat(mp, as), P = mat(mp, as);
    float *sums = (float *)w, *inv = sums + pl.chunk * pl.tiles;
    const int tm = (mp + 127) / 128, tn = (np + 127) / 128;

    for (int64_t b0 = 0; b0 < p.batch; b0 += pl.chunk) {
        const unsigned nz = (unsigned)(p.batch - b0 < pl.chunk ? p.batch - b0 : pl.chunk);
        const int z0 = (int)b0;
        if (flip)
            hipLaunchKernelGGL((ns_load_kernel<T, true>), dim3(mp / 64, np / 64, nz), dim3(256), 0, stream, p, z0, X, XT[0], sums);
        else
            hipLaunchKernelGGL((ns_load_kernel<T, false>), dim3(np / 64, mp / 64, nz), dim3(256), 0, stream, p, z0, X, XT[0], sums);
        hipLaunchKernelGGL(ns_norm_kernel, dim3(nz), dim3(256), 0, stream, sums, (int)pl.tiles, p.eps, inv);
        if (p.steps == 0) {
            const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
            hipLaunchKernelGGL((ns_scale_kernel<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096), 1, nz), dim3(256), 0, stream, p, z0, inv);
        }
        for (int s = 0; s < p.steps; ++s) {
            const float *sc = s == 0 ? inv : nullptr;
            const NsMat &xt = XT[s & 1], &xt2 = XT[(s + 1) & 1];
            NsGemm g = {X, X, mp, mp, np, X, A, A, 0.f, 1.f, sc};
            hipLaunchKernelGGL((ns_gemm_kernel<T, NS_GRAM>), dim3(tm * (tm + 1) / 2, 1, nz), dim3(256), 0, stream, g, p, z0, tm, tm);
            g = {A, A, mp, mp, mp, A, P, P, p.b, p.c, nullptr};
            hipLaunchKernelGGL((ns_gemm_kernel<T, NS_POLY>), dim3(tm * (tm + 1) / 2, 1, nz), dim3(256), 0, stream, g, p, z0, tm, tm);
            g = {P, xt, mp, np, mp, X, X, xt2, p.a, 1.f, sc};
            if (s + 1 < p.steps)
                hipLaunchKernelGGL((ns_gemm_kernel<T, NS_STEP>), dim3(tm * tn, 1, nz), dim3(256), 0, stream, g, p, z0, tm, tn);
            else
                hipLaunchKernelGGL((ns_gemm_kernel<T, NS_LAST>), dim3(tm * tn, 1, nz), dim3(256), 0, stream, g, p, z0, tm, tn);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_newton_schulz(int type, const NewtonSchulz &p, void *workspace, hipStream_t stream) {
    return type == MPGEMM_TYPE_F16 ? ns_type<_Float16>(p, workspace, stream) : ns_type<__bf16>(p, workspace, stream);
}

}  // namespace mpg
