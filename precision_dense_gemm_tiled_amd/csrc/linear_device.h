// Kernels shared by the 8-bit integer linear layer and the gated block: the tile
// kernel with its epilogues and the kernel of few rows.
#pragma once

#include "linear.h"
#include "phase_tile.h"

namespace mpg {

// ------------------------------------------------------------------ activations
//
// In fp32, by the hardware's exp2 and reciprocal (1 ulp each). The sigmoid forms are exact in
// their limits: exp2 overflows to infinity, whose reciprocal is 0.
__device__ __forceinline__ float lin_sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}

// exp(-v^2 / 2), and with it (1 + erf(v / sqrt 2)) / 2, the normal distribution at v, to a few 2^-23 of its value: 1 + erf
// cancels far below zero (at -5.5 in fp32 the sum is 0, half of it should be 1.9e-8). The distribution at -a over exp(-a^2 / 2) is
// t P(t), t = 1 / (1 + 0.21 a), with a polynomial of degree 8 fitted in 64 bits to the least relative error over a from 0 to
// 13.5 (1.3e-8; past that the exponential is 0). (Gated 2048 x 10240 x 4096 on integers with gelu 166 us; by erfc 188, by 1 + erf
// 176; with silu 156.)
__device__ __forceinline__ float lin_bell(float v) { return __builtin_amdgcn_exp2f(-0.72134752f * v * v); }
__device__ __forceinline__ float lin_normal(float v, float bell) {
    const float t = __builtin_amdgcn_rcpf(1.f + 0.21f * fabsf(v));
    float p = -0.0720338523f;
    p = fmaf(p, t, 0.285452783f);
    p = fmaf(p, t, -0.334188461f);
    p = fmaf(p, t, 0.354032308f);
    p = fmaf(p, t, -0.0972447917f);
    p = fmaf(p, t, 0.126354769f);
    p = fmaf(p, t, 0.0687901378f);
    p = fmaf(p, t, 0.0851293951f);
    p = fmaf(p, t, 0.0837077051f);
    const float tail = bell * (t * p);
    return v < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float lin_act(float v) {
    if constexpr (ACT == MPGEMM_ACT_SILU)
        return v * lin_sigmoid(v);
    else if constexpr (ACT == MPGEMM_ACT_GELU)
        return v * lin_normal(v, lin_bell(v));
    else   // 0.5 (1 + tanh z) = sigmoid(2 z)
        return v * lin_sigmoid(1.59576912f * (v + 0.044715f * v * v * v));
}

// The derivative. (w: where the factor that it multiplies has reached its limit, v's size no longer matters.)
template <int ACT>
__device__ __forceinline__ float lin_slope(float v) {
    const float w = fminf(fmaxf(v, -256.f), 256.f);
    if constexpr (ACT == MPGEMM_ACT_SILU) {
        const float s = lin_sigmoid(v);
        return s + s * (1.f - s) * w;
    } else if constexpr (ACT == MPGEMM_ACT_GELU) {
        const float bell = lin_bell(v);
        return lin_normal(v, bell) + 0.39894228f * w * bell;
    } else {
        const float s = lin_sigmoid(1.59576912f * (v + 0.044715f * v * v * v));
        return s + s * (1.f - s) * w * 1.59576912f * (1.f + 0.134145f * w * w);
    }
}

// ------------------------------------------------------------------ tiles

// Consecutive workgroups go to the 8 XCDs in turn, each with its own L2: give
// every XCD a contiguous range of tiles, walked in groups of 4 tile rows (4096 x 10240 x 4096 gated, bf16: 495 us,
// in groups of 8 499, of 16 513).
__device__ __forceinline__ void lin_tile_of(int bid, int nblk, int tiles_m, int tiles_n, int &tm, int &tn) {
    int logical = bid;
    if (nblk >= 8) {
        const int xcd = bid % 8, base = nblk / 8, rem = nblk % 8;
        logical = xcd * base + (xcd < rem ? xcd : rem) + bid / 8;
    }
    constexpr int GROUP = 4;
    const int group = logical / (GROUP * tiles_n);
    const int first = group * GROUP;
    const int rows = tiles_m - first < GROUP ? tiles_m - first : GROUP;
    const int in = logical - group * GROUP * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
}

template <typename OUT>
__device__ __forceinline__ uint32_t lin_pack(float a, float b) {
    typedef OUT two __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, two{(OUT)a, (OUT)b});
}

// Stores FN fragments of one row per lane: value d of fragment j is column cb + 16 j + 4 (lane / 16) + d.
// Of 16-bit results two fragments are exchanged between neighbouring quarters of the
// wavefront (v_permlane16_swap), after which a lane holds 8 columns in a row and
// 16 rows x 64 bytes go out in one instruction of 16 bytes per lane.
template <typename OUT, int FN>
__device__ __forceinline__ void lin_store(OUT *row, bool in, bool vec, int cb, int N, int lane, const float (&v)[FN][4]) {
    const int q = lane >> 4;
    if constexpr (sizeof(OUT) == 4) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = cb + 16 * j + 4 * q;
            if (in && vec && n + 4 <= N)
                *reinterpret_cast<pt_f32x4 *>(row + n) = pt_f32x4{v[j][0], v[j][1], v[j][2], v[j][3]};
            else if (in)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (n + d < N)
                        row[n + d] = v[j][d];
        }
    } else if constexpr (FN % 2 == 0) {
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
            const auto lo = __builtin_amdgcn_permlane16_swap(lin_pack<OUT>(v[j][0], v[j][1]), lin_pack<OUT>(v[j + 1][0], v[j + 1][1]), false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(lin_pack<OUT>(v[j][2], v[j][3]), lin_pack<OUT>(v[j + 1][2], v[j + 1][3]), false, false);
            const pt_u32x4 w = {lo[0], hi[0], lo[1], hi[1]};
            const int n = cb + 16 * (j + (q & 1)) + 8 * (q >> 1);
            if (in && vec && n + 8 <= N)
                *reinterpret_cast<pt_u32x4 *>(row + n) = w;
            else if (in)
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    if (n + d < N)
                        reinterpret_cast<uint16_t *>(row)[n + d] = (uint16_t)(w[d / 2] >> (16 * (d % 2)));
        }
    } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t lo = lin_pack<OUT>(v[j][0], v[j][1]), hi = lin_pack<OUT>(v[j][2], v[j][3]);
            const int n = cb + 16 * j + 4 * q;
            if (in && vec && n + 4 <= N) {
                *reinterpret_cast<uint2 *>(row + n) = uint2{lo, hi};
            } else if (in) {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (n + d < N)
                        reinterpret_cast<uint16_t *>(row)[n + d] = (uint16_t)((d < 2 ? lo : hi) >> (16 * (d % 2)));
            }
        }
    }
}

template <typename OUT>
__device__ __forceinline__ bool lin_vec(const void *c, int64_t ldc) {
    return (reinterpret_cast<uintptr_t>(c) & 15) == 0 && (ldc * (int64_t)sizeof(OUT)) % 16 == 0;
}

// A row's address; nullptr + offset is never formed.
template <typename OUT>
__device__ __forceinline__ OUT *lin_row(void *c, int64_t ldc, int m) {
    return c ? static_cast<OUT *>(c) + (int64_t)m * ldc : nullptr;
}

template <class E, typename OUT, int MODE, int ACT, class PT>
__device__ __forceinline__ void lin_epilogue(const Lin &p, int row0, int col0, int lane, int wave,
                                             const typename E::Acc (&acc)[2][2][PT::FM][PT::FN]) {
    constexpr bool SCALED = sizeof(typename E::T) == 1;
    constexpr int FM = PT::FM, FN = PT::FN, BPARTS = MODE == LIN_GATED ? 1 : 2;
    const int wm = (wave / PT::WGN_) * PT::WM, wn = (wave % PT::WGN_) * PT::WN, q = lane >> 4;
    const bool vec = lin_vec<OUT>(p.c, p.ldc) && (MODE != LIN_DW || lin_vec<OUT>(p.c2, p.ldc2));
    const bool vecg = lin_vec<OUT>(p.g, p.ldg) && lin_vec<OUT>(p.u, p.ldu);
#pragma unroll
    for (int hb = 0; hb < BPARTS; ++hb) {
        const int cb = col0 + hb * PT::HN + wn;
        float s0[FN][4], s1[FN][4], bias[FN][4];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int n = min(cb + 16 * j + 4 * q + d, p.N - 1);
                s0[j][d] = SCALED ? p.sb[0][n] : 1.f;
                s1[j][d] = SCALED && MODE == LIN_GATED ? p.sb[1][n] : 1.f;
                bias[j][d] = MODE == LIN_SCALED && p.bias ? (float)static_cast<const OUT *>(p.bias)[n] : 0.f;
            }
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                int m = row0 + ha * PT::HM + wm + 16 * i + (lane & 15);
                void *c = p.c;
                int64_t ldc = p.ldc;
                if (MODE == LIN_DW && m >= p.part) {
                    c = p.c2;
                    ldc = p.ldc2;
                    m -= p.part;
                }
                const bool in = m < p.M;
                const float sa = SCALED ? p.sa[min(m, p.M - 1)] : 1.f;
                float v[FN][4], g[FN][4], u[FN][4];
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        if constexpr (MODE == LIN_GATED) {
                            g[j][d] = (float)acc[ha][0][i][j][d];
                            u[j][d] = (float)acc[ha][1][i][j][d];
                            if (SCALED) {
                                g[j][d] = g[j][d] * sa * s0[j][d];
                                u[j][d] = u[j][d] * sa * s1[j][d];
                            }
                            v[j][d] = lin_act<ACT>(g[j][d]) * u[j][d];
                        } else if constexpr (MODE == LIN_SCALED) {
                            v[j][d] = (float)acc[ha][hb][i][j][d] * sa * s0[j][d] + bias[j][d];
                        } else {
                            v[j][d] = acc[ha][hb][i][j][d];
                        }
                    }
                lin_store<OUT, FN>(lin_row<OUT>(c, ldc, m), in && c, vec, cb, p.N, lane, v);
                if (MODE == LIN_GATED && !SCALED && p.g) {
                    lin_store<OUT, FN>(lin_row<OUT>(p.g, p.ldg, m), in, vecg, cb, p.N, lane, g);
                    lin_store<OUT, FN>(lin_row<OUT>(p.u, p.ldu, m), in, vecg, cb, p.N, lane, u);
                }
                __builtin_amdgcn_sched_barrier(0);   // (one row's registers at a time)
            }
    }
}

// Tile `bid` of a grid of `nblk`. GATED: a tile's columns are BN / 2 of either weight.
template <class E, typename OUT, int MODE, int BM, int BN, int WGM, int WGN, int NS>
struct LinTile {
    static constexpr bool AC = MODE == LIN_DW, BC = MODE == LIN_DX || MODE == LIN_DW;
    typedef PhaseTile<E, BM, BN, WGM, WGN, NS, AC, BC, MODE == LIN_DX> PT;
    static constexpr int EB = sizeof(typename E::T), CN = MODE == LIN_GATED ? BN / 2 : BN;

    static __host__ __device__ int rows(const Lin &p) { return MODE == LIN_DW ? p.parts * p.part : p.M; }
    static __host__ __device__ int tiles_m(const Lin &p) { return (rows(p) + BM - 1) / BM; }
    static __host__ __device__ int tiles_n(const Lin &p) { return (p.N + CN - 1) / CN; }

    static __device__ __forceinline__ void run(const Lin &p, int bid, int nblk, uint8_t *smem) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        int tm, tn;
        lin_tile_of(bid, nblk, tiles_m(p), tiles_n(p), tm, tn);
        const int row0 = tm * BM, col0 = tn * CN;
        PtSource A, B;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ra = row0 + h * PT::HM, rb = MODE == LIN_GATED ? col0 : col0 + h * PT::HN;
            A.p[h] = p.a + (AC ? (int64_t)ra * EB : (int64_t)ra * p.lda);
            A.rows[h] = rows(p) - ra;
            A.ld[h] = p.lda;
            const int w = MODE == LIN_GATED ? h : 0;
            B.p[h] = p.b[w] + (BC ? (int64_t)rb * EB : (int64_t)rb * p.ldb[w]);
            B.next[h] = MODE == LIN_DX ? p.b[1] + (int64_t)rb * EB : nullptr;
            B.rows[h] = p.N - rb;
            B.ld[h] = p.ldb[w];
        }
        const int chunks = BC ? p.K : (p.K * EB + 15) / 16;
        A.chunks = MODE == LIN_DX ? 2 * p.part / 8 : chunks;
        B.chunks = chunks;
        B.split = p.part / 64;
        const int stages = MODE == LIN_DX ? 2 * p.part / 64 : BC ? (p.K + 63) / 64 : (chunks + 7) / 8;
        typename E::Acc acc[2][2][PT::FM][PT::FN];
        PT::mainloop(A, B, stages, smem, tid, lane, wave, acc);
        if constexpr (MODE == LIN_GATED) {
            if (p.act == MPGEMM_ACT_SILU)
                lin_epilogue<E, OUT, MODE, MPGEMM_ACT_SILU, PT>(p, row0, col0, lane, wave, acc);
            else if (p.act == MPGEMM_ACT_GELU)
                lin_epilogue<E, OUT, MODE, MPGEMM_ACT_GELU, PT>(p, row0, col0, lane, wave, acc);
            else
                lin_epilogue<E, OUT, MODE, MPGEMM_ACT_GELU_TANH, PT>(p, row0, col0, lane, wave, acc);
        } else {
            lin_epilogue<E, OUT, MODE, 0, PT>(p, row0, col0, lane, wave, acc);
        }
    }
};

template <class E, typename OUT, int MODE, int BM, int BN, int WGM, int WGN, int NS>
__global__ __launch_bounds__(64 * WGM * WGN) void lin_tile_kernel(Lin p) {
    typedef LinTile<E, OUT, MODE, BM, BN, WGM, WGN, NS> LT;
    __shared__ __attribute__((aligned(16))) uint8_t smem[LT::PT::LDS_BYTES];
    LT::run(p, blockIdx.x, gridDim.x, smem);
}

template <class E, typename OUT, int MODE, int BM, int BN, int WGM, int WGN, int NS>
static void lin_tile_one(const Lin &p, hipStream_t stream) {
    typedef LinTile<E, OUT, MODE, BM, BN, WGM, WGN, NS> LT;
    hipLaunchKernelGGL((lin_tile_kernel<E, OUT, MODE, BM, BN, WGM, WGN, NS>), dim3((unsigned)LT::tiles_m(p) * (unsigned)LT::tiles_n(p)),
                       dim3(64 * WGM * WGN), 0, stream, p);
}

template <class E, typename OUT, int MODE>
static void lin_tile(const Lin &p, const LinPlan &plan, hipStream_t stream) {
    switch (plan.cfg) {
    case 0: lin_tile_one<E, OUT, MODE, 256, 256, 2, 4, 2>(p, stream); break;
    case 1: lin_tile_one<E, OUT, MODE, 128, 128, 2, 2, 2>(p, stream); break;
    case 2: lin_tile_one<E, OUT, MODE, 64, 64, 2, 2, 4>(p, stream); break;
    default:
        if constexpr (MODE == LIN_SCALED || MODE == LIN_GATED)
            lin_tile_one<E, OUT, MODE, 64, 128, 2, 2, 4>(p, stream);
        break;
    }
}

// ------------------------------------------------------------------ few rows

// 16 bytes at any alignment (one load: gfx950 reads unaligned addresses).
__device__ __forceinline__ pt_u32x4 lin_load16(const uint8_t *s) {
    typedef pt_u32x4 any __attribute__((aligned(1)));
    return *reinterpret_cast<const any *>(s);
}

// The same with zeros in the place of what is at or past `left` bytes, which is not read.
template <typename T>
__device__ __forceinline__ pt_u32x4 lin_load16_part(const uint8_t *s, int left) {
    if (left >= 16)
        return lin_load16(s);
    pt_u32x4 v = {0, 0, 0, 0};
    constexpr int PER = 4 / (int)sizeof(T);
    for (int w = 0; w < 4; ++w) {
        uint32_t x = 0;
        for (int i = 0; i < PER; ++i) {
            const int at = (w * PER + i) * (int)sizeof(T);
            uint32_t e = 0;
            if (at < left)
                e = sizeof(T) == 1 ? (uint32_t)s[at] : (uint32_t)s[at] | (uint32_t)s[at + 1] << 8;
            x |= e << (8 * (int)sizeof(T) * i);
        }
        v[w] = x;
    }
    return v;
}

// Largest magnitude as an fp32 bit pattern (NaN over infinity over finite), joined over a wavefront: within
// rows of 16 lanes by DPP, then over the rows by lane swaps.
__device__ __forceinline__ uint32_t lin_wave_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // lanes 1 0 3 2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // lanes 2 3 0 1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // half rows mirrored
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));   // rows mirrored
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(b[0], b[1]);
}

// Scale and how a row is divided by it: values and scale go through 2^up, exact, where the scale
// would be near the subnormals. A row with a NaN or an infinity gets a NaN scale and zeros.
struct I8Row {
    float scale, s, inv, up;
};
__device__ __forceinline__ I8Row i8_row(uint32_t amax) {
    I8Row r;
    const float top = __uint_as_float(amax);
    r.scale = top / 127.f;
    r.up = top < 0x1p-60f ? 0x1p90f : 1.f;
    r.s = r.scale * r.up;
    r.inv = r.s > 0.f ? 1.f / r.s : 0.f;
    if (amax >= 0x7F800000u) {
        r.scale = __uint_as_float(0x7FC00000u);
        r.s = r.inv = 0.f;
        r.up = 0.f;
    }
    return r;
}

// The nearest integer to x / s, ties to even: the product with the reciprocal may be off by one next to a
// half, and the remainder, which is exact, says so.
__device__ __forceinline__ int i8_code(float x, const I8Row &r) {
    x *= r.up;
    float n = rintf(x * r.inv);
    const float d = fmaf(-n, r.s, x), over = 2.f * fabsf(d) - r.s;
    const bool odd = ((int)n & 1) != 0;
    if (r.inv != 0.f && (over > 0.f || (over == 0.f && odd)))
        n += copysignf(1.f, d);
    n = fminf(fmaxf(n, -127.f), 127.f);
    return r.inv != 0.f ? (int)n : 0;
}

// 8 elements of a row from k0 on as fp32, zeros past K. vec: 16-byte aligned rows and K a multiple of 8.
template <typename T>
__device__ __forceinline__ void i8_load8(const T *x, int k0, int K, bool vec, float (&v)[8]) {
    typedef T eight __attribute__((ext_vector_type(8)));
    if (vec && k0 < K) {
        const eight e = *reinterpret_cast<const eight *>(x + k0);
#pragma unroll
        for (int d = 0; d < 8; ++d)
            v[d] = (float)e[d];
    } else {
#pragma unroll
        for (int d = 0; d < 8; ++d)
            v[d] = k0 + d < K ? (float)x[k0 + d] : 0.f;
    }
}

__device__ __forceinline__ uint32_t i8_amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 8; ++d)
        m = max(m, __float_as_uint(v[d]) & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ uint2 i8_codes8(const float (&v)[8], const I8Row &r) {
    uint2 w;
    w.x = w.y = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        w.x |= ((uint32_t)i8_code(v[d], r) & 0xFFu) << (8 * d);
        w.y |= ((uint32_t)i8_code(v[4 + d], r) & 0xFFu) << (8 * d);
    }
    return w;
}

constexpr int LIN_SKINNY_WAVES = 8;
// GATED: up to here 8 columns of either weight per workgroup, in one fragment, else 16 in two (16 bits, through 10240 x 4096: 4 rows
// 31.8 us, in two 36.0; 8 rows 35.8 and 36.4, on integers 21.5 and 19.6).
constexpr int LIN_HALF_ROWS = 4;
constexpr int LIN_X_MAX = 32;   // rows of 512 activations, a wavefront's load, that the fused kernel takes

// One output from its sums (of either weight).
template <class E, typename OUT, int MODE, typename Num, int NB>
__device__ __forceinline__ void lin_output(const Lin &p, int m, int n, float sa, const Num (&t)[NB]) {
    constexpr bool SCALED = sizeof(typename E::T) == 1;
    float v = (float)t[0];
    if (SCALED)
        v = v * sa * p.sb[0][n];
    if constexpr (MODE == LIN_GATED) {
        float u = (float)t[1];
        if (SCALED)
            u = u * sa * p.sb[1][n];
        if (!SCALED && p.g) {
            static_cast<OUT *>(p.g)[(int64_t)m * p.ldg + n] = (OUT)v;
            static_cast<OUT *>(p.u)[(int64_t)m * p.ldu + n] = (OUT)u;
        }
        v = (p.act == MPGEMM_ACT_SILU ? lin_act<MPGEMM_ACT_SILU>(v)
             : p.act == MPGEMM_ACT_GELU ? lin_act<MPGEMM_ACT_GELU>(v) : lin_act<MPGEMM_ACT_GELU_TANH>(v)) * u;
    } else if (p.bias) {
        v += (float)static_cast<const OUT *>(p.bias)[n];
    }
    static_cast<OUT *>(p.c)[(int64_t)m * p.ldc + n] = (OUT)v;
}

// Up to 32 rows: 16 MF rows x 16 NF columns (of each weight) per workgroup, operands straight from memory
// into the matrix unit's registers, which read each weight once; K in groups of 128 bytes dealt out to the
// 8 wavefronts in turn. At step s of a group, lane quarter q takes bytes 64 s + 16 q of its row, so that a
// load instruction reads 64 contiguous bytes of each of 16 rows. AHEAD groups are on their way from the
// start on (three; of 32 rows two: integers 32 x 20480 x 4096 26.2 us, with three 29.4, with one 30.8). The wavefronts'
// sums are joined in LDS in the order of the wavefronts.
// Bound by what a CU can have on its way to it, about 28 bytes a ns: one token in 16 bits through 168 MB of weights 30.7 us; 16 rows
// of integers through 8192 x 8192 16.3, for each CU 262 KB of weights and 131 KB of activations. (A load for every
// group, so that the compiler's waits leave the later groups on their way, costs more in loads past the end: 21.4.)
// X: the activations are quantised by every workgroup (MF = 1, few of them). LOOP: two workgroups per
// CU go on to further columns with those (gated 1 x 10240 x 4096 17.7 us, 21.7 with a workgroup for each 8
// columns; where nothing is quantised the loop has no gain: 16 bits 31.9 and 30.8).
template <class E, typename OUT, int MODE, int MF, int NF, bool HALF, bool X, bool LOOP>
__global__ __launch_bounds__(64 * LIN_SKINNY_WAVES) void lin_skinny_kernel(Lin p, LinX px) {
    constexpr int NW = LIN_SKINNY_WAVES, NT = 64 * NW, GB = 128, AHEAD = MF == 1 ? 3 : 2, NB = MODE == LIN_GATED && !HALF ? 2 : 1, EB = sizeof(typename E::T);
    constexpr bool SCALED = EB == 1;
    typedef typename E::Acc Acc;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    typedef decltype(Acc{}[0] + Acc{}[0]) Num;
    Num (*red)[MF * NB * NF][4][64] = reinterpret_cast<Num (*)[MF * NB * NF][4][64]>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, r = lane & 15;
    constexpr int COLS = HALF ? 8 : 16 * NF;
    int n0 = blockIdx.x * COLS;
    const int bytes = p.K * EB, full = bytes / GB, groups = (bytes + GB - 1) / GB;

    const uint8_t *b[NB][NF], *a[MF];
    auto columns = [&]() {
#pragma unroll
        for (int w = 0; w < NB; ++w)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                b[w][j] = HALF ? (r < 8 ? p.b[0] : p.b[1]) + (int64_t)min(n0 + (r & 7), p.N - 1) * (r < 8 ? p.ldb[0] : p.ldb[1])
                               : p.b[w] + (int64_t)min(n0 + 16 * j + r, p.N - 1) * p.ldb[w];
    };
    columns();
#pragma unroll
    for (int i = 0; i < MF; ++i)
        a[i] = X ? nullptr : p.a + (int64_t)min(16 * i + r, p.M - 1) * p.lda;
    auto load = [&](const uint8_t *row, int g, pt_u32x4 (&v)[2]) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            v[s] = lin_load16(row + (int64_t)g * GB + 64 * s + 16 * q);
    };
    auto load_rest = [&](const uint8_t *row, int g, pt_u32x4 (&v)[2]) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = g * GB + 64 * s + 16 * q;
            v[s] = lin_load16_part<typename E::T>(row + at, bytes - at);
        }
    };

    // A group's operands (the activations that the kernel has quantised stay in LDS).
    struct Group {
        pt_u32x4 b[NB][NF][2], a[X ? 1 : MF][2];
    } gr[AHEAD];
    auto load_group = [&](int g, Group &v) {
#pragma unroll
        for (int w = 0; w < NB; ++w)
#pragma unroll
            for (int j = 0; j < NF; ++j)
                load(b[w][j], g, v.b[w][j]);
        if constexpr (!X) {
#pragma unroll
            for (int i = 0; i < MF; ++i)
                load(a[i], g, v.a[i]);
        }
    };
    auto first_groups = [&]() {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            if (wave + d * NW < full)
                load_group(wave + d * NW, gr[d]);
    };
    // the activations' codes: rows of `codes_ld` bytes (a multiple of 512, and 16 so that rows start at different banks)
    uint8_t *codes = smem + sizeof(Num) * NW * MF * NB * NF * 256;
    const int per_row = (p.K + 511) / 512 * 64, codes_ld = per_row * 8 + 16;
    float *scales = reinterpret_cast<float *>(codes + (size_t)p.M * codes_ld);
    if constexpr (X) {
        typedef OUT T;
        uint32_t *top = reinterpret_cast<uint32_t *>(scales + 16);
        const bool vec = p.K % 8 == 0 && (reinterpret_cast<uintptr_t>(px.x) & 15) == 0 && (px.ldx * (int64_t)sizeof(T)) % 16 == 0;
        float v[LIN_X_MAX / NW][8];
#pragma unroll
        for (int i = 0; i < LIN_X_MAX / NW; ++i) {
            const int f = i * NT + tid, row = f / per_row;
            if (row < p.M)   // (the same row for a whole wavefront)
                i8_load8<T>(static_cast<const T *>(px.x) + (int64_t)row * px.ldx, (f - row * per_row) * 8, p.K, vec, v[i]);
        }
        first_groups();   // (behind the activations: loads return in order)
        if (tid < 16)
            top[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LIN_X_MAX / NW; ++i) {
            const int row = (i * NT + tid) / per_row;
            if (row < p.M) {
                const uint32_t m = lin_wave_max(i8_amax8(v[i]));
                if (lane == 0)
                    atomicMax(&top[row], m);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LIN_X_MAX / NW; ++i) {
            const int f = i * NT + tid, row = f / per_row, k0 = (f - row * per_row) * 8;
            if (row < p.M) {
                const I8Row s = i8_row(top[row]);
                *reinterpret_cast<uint2 *>(codes + (size_t)row * codes_ld + k0) = i8_codes8(v[i], s);
                if (k0 == 0)
                    scales[row] = s.scale;
            }
        }
        __syncthreads();
    } else {
        first_groups();
    }

    Acc acc[NB][MF][NF];
    auto products = [&](const Group &v) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int w = 0; w < NB; ++w)
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int j = 0; j < NF; ++j)
                        acc[w][i][j] = E::mfma(v.a[i][s], v.b[w][j][s], acc[w][i][j]);
    };
    auto coded = [&](int g, Group &v) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            v.a[0][s] = *reinterpret_cast<const pt_u32x4 *>(codes + (size_t)min(r, p.M - 1) * codes_ld + g * GB + 64 * s + 16 * q);
    };
    auto group = [&](int g, Group &v) {
        if constexpr (X)
            coded(g, v);
        products(v);
        if (g + AHEAD * NW < full)
            load_group(g + AHEAD * NW, v);
    };
    for (;;) {
#pragma unroll
        for (int w = 0; w < NB; ++w)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[w][i][j] = Acc{};
        for (int g = wave; g < full; g += AHEAD * NW)
#pragma unroll
            for (int d = 0; d < AHEAD; ++d)
                if (g + d * NW < full)
                    group(g + d * NW, gr[d]);
        if (groups > full && full % NW == wave) {
            if constexpr (X) {
                coded(full, gr[0]);
            } else {
#pragma unroll
                for (int i = 0; i < MF; ++i)
                    load_rest(a[i], full, gr[0].a[i]);
            }
#pragma unroll
            for (int w = 0; w < NB; ++w)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    load_rest(b[w][j], full, gr[0].b[w][j]);
            products(gr[0]);
        }
        // register d of lane l: row 4 (l / 16) + d, column l % 16 of the block
#pragma unroll
        for (int w = 0; w < NB; ++w)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        red[wave][(w * MF + i) * NF + j][d][lane] = acc[w][i][j][d];
        __syncthreads();
        for (int f = tid; f < MF * 16 * COLS; f += NT) {
            // consecutive threads take consecutive columns
            constexpr int PARTS = MODE == LIN_GATED ? 2 : 1;
            const int col = f % COLS, row = f / COLS, i = row / 16, d = row % 4;
            Num t[PARTS] = {};
#pragma unroll
            for (int w = 0; w < PARTS; ++w) {
                const int c = HALF ? col + 8 * w : col, block = ((HALF ? 0 : w) * MF + i) * NF + c / 16;
#pragma unroll
                for (int x = 0; x < NW; ++x)
                    t[w] += red[x][block][d][(row % 16) / 4 * 16 + c % 16];
            }
            const int n = n0 + col;
            if (row < p.M && n < p.N)
                lin_output<E, OUT, MODE>(p, row, n, !SCALED ? 1.f : X ? scales[row] : p.sa[row], t);
        }
        if constexpr (!LOOP)
            break;
        n0 += gridDim.x * COLS;
        if (n0 >= p.N)
            break;
        columns();
        first_groups();
        wait_lds_only();
        lds_barrier();   // (the sums have been read)
    }
}

template <class E, typename OUT, int MODE, int MF, int NF, bool HALF, bool X>
static void lin_skinny_one(const Lin &p, const LinX &x, const LinPlan &plan, hipStream_t stream) {
    constexpr int NB = MODE == LIN_GATED && !HALF ? 2 : 1, COLS = HALF ? 8 : 16 * NF, NT = 64 * LIN_SKINNY_WAVES;
    const unsigned lds = MF * NB * NF * LIN_SKINNY_WAVES * 1024u + (X ? (unsigned)p.M * ((p.K + 511) / 512 * 512 + 16) + 128 : 0);
    const int blocks = (p.N + COLS - 1) / COLS, at_once = 2 * plan.cus;
    if (X && blocks > at_once)
        hipLaunchKernelGGL((lin_skinny_kernel<E, OUT, MODE, MF, NF, HALF, X, X>), dim3(at_once), dim3(NT), lds, stream, p, x);
    else
        hipLaunchKernelGGL((lin_skinny_kernel<E, OUT, MODE, MF, NF, HALF, X, false>), dim3(blocks), dim3(NT), lds, stream, p, x);
}

template <class E, typename OUT, int MODE, int NF>
static void lin_skinny(const Lin &p, const LinPlan &plan, hipStream_t stream) {
    if (plan.cfg == 1)
        lin_skinny_one<E, OUT, MODE, 1, NF, false, false>(p, LinX{}, plan, stream);
    else
        lin_skinny_one<E, OUT, MODE, 2, NF, false, false>(p, LinX{}, plan, stream);
}

template <class E, typename OUT, int MODE>
static hipError_t lin_run(const Lin &p, const LinPlan &plan, hipStream_t stream) {
    if (plan.kind == LINK_SKINNY) {
        // 32 columns per workgroup, 16 of two weights or 32 of one, once 16 would go round the CUs more than
        // once: the activations are then read half as often (16 rows through 6144 x 4096 8.3 us, with 16 columns
        // 10.1; through 4096 x 4096 8.2 and 6.8).
        if (MODE == LIN_SCALED && p.N > 16 * plan.cus)
            lin_skinny<E, OUT, MODE, MODE == LIN_SCALED ? 2 : 1>(p, plan, stream);
        else if (MODE == LIN_GATED && p.M <= LIN_HALF_ROWS)
            lin_skinny_one<E, OUT, MODE, 1, 1, MODE == LIN_GATED, false>(p, LinX{}, plan, stream);
        else
            lin_skinny<E, OUT, MODE, 1>(p, plan, stream);
    } else {
        lin_tile<E, OUT, MODE>(p, plan, stream);
    }
    return hipGetLastError();
}

// On integers, the activations quantised in the kernel.
template <typename OUT, int MODE>
static hipError_t lin_run_x(const Lin &p, const LinX &x, const LinPlan &plan, hipStream_t stream) {
    if (MODE == LIN_GATED && p.M <= LIN_HALF_ROWS)
        lin_skinny_one<PtI8, OUT, MODE, 1, 1, MODE == LIN_GATED, true>(p, x, plan, stream);
    else
        lin_skinny_one<PtI8, OUT, MODE, 1, 1, false, true>(p, x, plan, stream);
    return hipGetLastError();
}

}  // namespace mpg
