// MXFP4 product C = A B^T + bias on gfx950's scaled matrix instructions.
//
// C[m][n] = sum over blocks of 2^(sa - 127 + sb - 127) * (sum of 32 products
// of e2m1 values). v_mfma_scale_f32_16x16x128_f8f6f4 takes one block of 32 codes
// (16 bytes) and its scale byte per lane for each operand, so the 16-byte
// chunks of the stored rows are the fragments and the stored e8m0 bytes the
// scales: nothing is unpacked. Lane l supplies row l % 16 and block l / 16 of a
// step; which blocks of K make up a step is free, as long as both operands
// agree. The scale bytes of the blocks that a lane takes over several steps are
// one word, and the step selects the byte.
//
// Two kernels:
//   tile    operands through LDS (compute and L2 bandwidth bound)
//   skinny  up to 64 rows (mx_is_skinny): operands straight from memory into the matrix unit's
//           registers, K over the wavefronts of a workgroup (bound by reading
//           B once); few activations are quantised in it
#include "mxfp4.h"
#include "mxfp4_device.h"
#include "lds_dma.h"

namespace mpg {

typedef int mx_i32x4 __attribute__((ext_vector_type(4)));
typedef int mx_i32x8 __attribute__((ext_vector_type(8)));
typedef float mx_f32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of zeros: the source of blocks past a row's end.
__device__ const u32x4 kMxZeros = {0, 0, 0, 0};

__device__ __forceinline__ mx_i32x8 mx_widen(mx_i32x4 v) { return mx_i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// One step with byte S of the scale words. The operand format 4 is e2m1.
template <int S>
__device__ __forceinline__ mx_f32x4 mx_mfma16(mx_i32x4 x, mx_i32x4 y, mx_f32x4 c, int sx, int sy) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_widen(x), mx_widen(y), c, 4, 4, S, sx, S, sy);
}

// Consecutive workgroups go to the 8 XCDs in turn, each with its own L2: give
// every XCD a contiguous range of tiles, walked in groups of 8 tile rows.
__device__ __forceinline__ void mx_tile_of(int bid, int nblk, int tiles_m, int tiles_n, int &tm, int &tn) {
    int logical = bid;
    if (nblk >= 8) {
        const int xcd = bid % 8, base = nblk / 8, rem = nblk % 8;
        logical = xcd * base + (xcd < rem ? xcd : rem) + bid / 8;
    }
    constexpr int GROUP = 8;
    const int group = logical / (GROUP * tiles_n);
    const int first = group * GROUP;
    const int rows = tiles_m - first < GROUP ? tiles_m - first : GROUP;
    const int in = logical - group * GROUP * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
}

template <typename T>
__device__ __forceinline__ float mx_bias(const void *bias, int n) {
    return bias ? (float)((const T *)bias)[n] : 0.f;
}

// ------------------------------------------------------------------ tile

// BM x BN output tile, WGM x WGN wavefronts, stages of 8 blocks of K (128
// bytes per row) in an NS-deep LDS ring filled with direct-to-LDS loads.
// 16-byte chunk c of LDS row r sits at c ^ swz(r), which keeps the fragment
// reads (one chunk column over 16 rows) free of bank conflicts. At step s (of two)
// of a stage, lane quarter q reads chunk 2 q + s.
//
// Scales: 16 bytes per row, two stages' worth, in a two-slot ring of their
// own; each lane reads the two bytes of its row, stage and quarter once per stage.
//
// The 16 x 16 x 128 shape: with random codes a stream of independent matrix
// instructions alone runs at 7.2 PFLOP/s in it and at 6.5 in 32 x 32 x 64 (9.4 and 9.2 on
// zeros: the clock follows the power, and this shape moves half the sums per product).
//
// The main loop runs over pairs of stages and has no branch: with one (for the
// scales of every other stage, or for the last stage's partial rows) the compiler
// moved all of a stage's matrix instructions past it, behind the wait for the next
// stage.
template <int BM, int BN, int WGM, int WGN, int NS>
struct MxTile {
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    static constexpr int WTM = BM / WGM, WTN = BN / WGN, TM = WTM / 16, TN = WTN / 16, HM = TM / 2, HN = TN / 2;
    static constexpr int BKB = 128, CPR = 8, RS = NT / CPR;
    static constexpr int A_PER_T = BM / RS, B_PER_T = BN / RS, NL = A_PER_T + B_PER_T;
    static constexpr int SROUNDS = (BM + BN + NT - 1) / NT;
    static constexpr int STAGE = (BM + BN) * BKB, SCALES = SROUNDS * NT * 16;   // (whole rounds)
    static constexpr int LDS_BYTES = NS * STAGE + 2 * SCALES;
    static_assert(RS % 16 == 0 && BM % RS == 0 && BN % RS == 0 && (BM + BN) % 64 == 0 && BM % 64 == 0, "staging");
    static_assert(TM % 2 == 0 && TN % 2 == 0, "quadrants");
    static_assert(NS >= 2 && LDS_BYTES <= 160 * 1024 && (NS - 2) * NL < 64, "ring");

    static __device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

    // The fragments of half of the wavefront's rows (or columns) at a step.
    template <int N>
    static __device__ __forceinline__ void read_half(const uint8_t *rows, int first, int chunk, int lane, mx_i32x4 (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = first + i * 16 + (lane & 15);
            f[i] = *reinterpret_cast<const mx_i32x4 *>(rows + r * BKB + ((chunk ^ swz(r)) * 16));
        }
    }

    // A quadrant of a step. Operands swapped, so each accumulator block is the
    // transpose of its C block: register d of lane l holds row l % 16, column 4 (l / 16) + d.
    template <int S>
    static __device__ __forceinline__ void quadrant(const mx_i32x4 (&a)[HM], const mx_i32x4 (&b)[HN], const int (&sa)[TM],
                                                    const int (&sb)[TN], int i0, int j0, mx_f32x4 (&acc)[TM][TN]) {
#pragma unroll
        for (int i = 0; i < HM; ++i)
#pragma unroll
            for (int j = 0; j < HN; ++j)
                acc[i0 + i][j0 + j] = mx_mfma16<S>(b[j], a[i], acc[i0 + i][j0 + j], sb[j0 + j], sa[i0 + i]);
    }

    // Stages [e0, e1) of 8 blocks, e0 even; only the last stage of a row may be
    // partial. The sums start from the bias.
    template <typename OUT>
    static __device__ __forceinline__ void mainloop(const MxGemm &p, uint8_t *smem, int row0, int col0, int e0,
                                                    int e1, int tid, int lane, int wave,
                                                    mx_f32x4 (&acc)[TM][TN]) {
        const int wm0 = (wave / WGN) * WTM, wn0 = (wave % WGN) * WTN, quarter = lane >> 4;
        const int nb = p.nb, last = (nb + 7) / 8 - 1;
        const int r0 = tid / CPR, cg = (tid % CPR) ^ swz(r0);
        const uint8_t *Ab = p.a + (int64_t)row0 * p.lda, *Bb = p.b + (int64_t)col0 * p.ldb;
        const uint8_t *SAb = p.sa + (int64_t)row0 * p.ldsa, *SBb = p.sb + (int64_t)col0 * p.ldsb;
        const int a_rows = p.M - row0, b_rows = p.N - col0;
        // (rows past the matrix repeat its last row: their outputs are not stored)
        uint32_t off[NL];
        const uint8_t *ssrc[SROUNDS];
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const bool isa = i < A_PER_T;
            const int rows = isa ? a_rows : b_rows;
            int r = r0 + (isa ? i : i - A_PER_T) * RS;
            r = r < rows ? r : rows - 1;
            off[i] = (uint32_t)r * (uint32_t)(isa ? p.lda : p.ldb) + cg * 16;
        }
#pragma unroll
        for (int i = 0; i < SROUNDS; ++i) {
            const int t = min(i * NT + tid, BM + BN - 1);
            const bool isa = t < BM;
            const int rows = isa ? a_rows : b_rows;
            int r = isa ? t : t - BM;
            r = r < rows ? r : rows - 1;
            ssrc[i] = (isa ? SAb : SBb) + (uint32_t)r * (uint32_t)(isa ? p.ldsa : p.ldsb);
        }
        const int wrow = wave * (64 / CPR);
        uint8_t *sc = smem + NS * STAGE;

        // every call issues NL loads: stages past the last re-read it
        auto dma_stage = [&](int e) {
            const int kt = e < last ? e : last;
            const bool in = kt * 8 + cg < nb;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const bool isa = i < A_PER_T;
                const uint8_t *src = (isa ? Ab : Bb) + (int64_t)kt * BKB + off[i];
                src = in ? src : reinterpret_cast<const uint8_t *>(&kMxZeros);
                dma16(src, smem + (e % NS) * STAGE + (isa ? 0 : BM * BKB) +
                               (wrow + (isa ? i : i - A_PER_T) * RS) * BKB);
            }
        };
        // scale bytes of stages 2 q and 2 q + 1 (a chunk that starts inside the row)
        auto dma_scales = [&](int q) {
            const int qc = 2 * q <= last ? q : last / 2;
#pragma unroll
            for (int i = 0; i < SROUNDS; ++i)
                dma16(ssrc[i] + 16 * qc, sc + (q & 1) * SCALES + (i * NT + wave * 64) * 16);
        };
        auto read_scales = [&](int e, int (&sa)[TM], int (&sb)[TN]) {
            const uint8_t *s = sc + ((e >> 1) & 1) * SCALES + 8 * (e & 1) + 2 * quarter;
            // (the bytes of blocks past the row's end are cleared: a stray 255 would be NaN)
            const int left = nb - 8 * min(e, last) - 2 * quarter;
            const int keep = left >= 2 ? 0xFFFF : left == 1 ? 0xFF : 0;
#pragma unroll
            for (int i = 0; i < TM; ++i)
                sa[i] = *reinterpret_cast<const uint16_t *>(s + (wm0 + i * 16 + (lane & 15)) * 16) & keep;
#pragma unroll
            for (int j = 0; j < TN; ++j)
                sb[j] = *reinterpret_cast<const uint16_t *>(s + (BM + wn0 + j * 16 + (lane & 15)) * 16) & keep;
        };

#pragma unroll
        for (int j = 0; j < TN; ++j) {
            mx_f32x4 b = {};
            if (p.bias) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int n = col0 + wn0 + 16 * j + 4 * quarter + d;
                    b[d] = (float)((const OUT *)p.bias)[n < p.N ? n : p.N - 1];
                }
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
                acc[i][j] = b;
        }

        mx_i32x4 a0[2][HM], a1[HM], b0[2][HN], b1[HN];
        int sa0[TM], sb0[TN], sa1[TM], sb1[TN];
        // Loads retire in order and the scales of a pair are issued ahead of its
        // stages, so the wait that proves a stage has landed proves its scales too.
        dma_scales(e0 >> 1);
#pragma unroll
        for (int e = 0; e < NS - 1; ++e)
            dma_stage(e0 + e);
        wait_vm_lds<(NS - 2) * NL>();
        lds_barrier();
        read_half(smem + (e0 % NS) * STAGE, wm0, 2 * quarter, lane, a0[0]);
        read_half(smem + (e0 % NS) * STAGE + BM * BKB, wn0, 2 * quarter, lane, b0[0]);
        read_scales(e0, sa0, sb0);

        // Stage e: the loads of stage e + NS - 1 go into the slot that stage
        // e - 1 has left (before an even stage the next pair's scales, into the slot
        // of the pair before this one). A step goes round its quadrants, each of which
        // needs one new half of the fragments, read during the quadrant before; half way
        // through the second step the barrier publishes stage e + 1, whose first halves
        // and scales are read under the other two quadrants.
        auto stage = [&](int e, bool even, const int (&sa)[TM], const int (&sb)[TN], int (&na)[TM], int (&nb2)[TN]) {
            const uint8_t *A = smem + (e % NS) * STAGE, *B = A + BM * BKB;
            const uint8_t *An = smem + ((e + 1) % NS) * STAGE, *Bn = An + BM * BKB;
            const int c0 = 2 * quarter, c1 = c0 + 1;
            __builtin_amdgcn_sched_barrier(0);
            if (even)
                dma_scales((e >> 1) + 1);
            dma_stage(e + NS - 1);
            read_half(B, wn0 + HN * 16, c0, lane, b1);
            quadrant<0>(a0[0], b0[0], sa, sb, 0, 0, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(A, wm0 + HM * 16, c0, lane, a1);
            quadrant<0>(a0[0], b1, sa, sb, 0, HN, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(A, wm0, c1, lane, a0[1]);
            quadrant<0>(a1, b1, sa, sb, HM, HN, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(B, wn0, c1, lane, b0[1]);
            quadrant<0>(a1, b0[0], sa, sb, HM, 0, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(B, wn0 + HN * 16, c1, lane, b1);
            quadrant<1>(a0[1], b0[1], sa, sb, 0, 0, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(A, wm0 + HM * 16, c1, lane, a1);
            quadrant<1>(a0[1], b1, sa, sb, 0, HN, acc);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm_lds<(NS - 2) * NL>();
            lds_barrier();
            __builtin_amdgcn_sched_barrier(0);
            read_half(An, wm0, c0, lane, a0[0]);
            read_scales(e + 1, na, nb2);
            quadrant<1>(a1, b1, sa, sb, HM, HN, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(Bn, wn0, c0, lane, b0[0]);
            quadrant<1>(a1, b0[1], sa, sb, HM, 0, acc);
            __builtin_amdgcn_sched_barrier(0);
        };
        int e = e0;
        for (; e + 1 < e1; e += 2) {
            stage(e, true, sa0, sb0, sa1, sb1);
            stage(e + 1, false, sa1, sb1, sa0, sb0);
        }
        if (e < e1)
            stage(e, true, sa0, sb0, sa1, sb1);
        wait_vm_lds<0>();
    }

    // C through LDS: each wavefront writes 32 rows of its outputs (four
    // consecutive columns per lane) into its own region and reads whole row
    // segments back for 16-byte stores. Chunk c of row r sits at
    // c ^ (r % chunks per row).
    template <typename OUT>
    static __device__ __forceinline__ void epilogue(const MxGemm &p, uint8_t *smem, int row0, int col0, int lane,
                                                    int wave, const mx_f32x4 (&acc)[TM][TN]) {
        constexpr int RB = WTN * (int)sizeof(OUT), CPW = RB / 16;
        constexpr int EPC = 16 / (int)sizeof(OUT);   // outputs per chunk
        static_assert(NW * 32 * RB <= LDS_BYTES && (CPW & (CPW - 1)) == 0 && CPW >= 4, "epilogue staging");
        const int wm0 = (wave / WGN) * WTM, wn0 = (wave % WGN) * WTN;
        uint8_t *region = smem + wave * 32 * RB;
        OUT *C = reinterpret_cast<OUT *>(p.c);
        const bool vec = (reinterpret_cast<uintptr_t>(C) & 15) == 0 && (p.ldc * sizeof(OUT)) % 16 == 0;
        __syncthreads();   // every wavefront is past its last fragment read
        typedef OUT out4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < TM; i += 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int rl = 16 * h + (lane & 15), cl = 16 * j + 4 * (lane >> 4);
                    out4 v;
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        v[d] = (OUT)acc[i + h][j][d];
                    *reinterpret_cast<out4 *>(region + rl * RB + (((cl / EPC) ^ (rl & (CPW - 1))) * 16) +
                                              (cl % EPC) * (int)sizeof(OUT)) = v;
                }
            wave_lds_fence();
#pragma unroll
            for (int q = 0; q < 32 * CPW / 64; ++q) {
                const int f = q * 64 + lane;
                const int r = f / CPW, c = f % CPW;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(region + r * RB + ((c ^ (r & (CPW - 1))) * 16));
                const int row = row0 + wm0 + i * 16 + r, col = col0 + wn0 + c * EPC;
                if (row < p.M) {
                    OUT *dst = C + (int64_t)row * p.ldc + col;
                    if (vec && col + EPC <= p.N) {
                        // non-temporal: C is not read back here
                        __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(dst));
                    } else {
#pragma unroll
                        for (int d = 0; d < EPC; ++d)
                            if (col + d < p.N) {
                                if constexpr (sizeof(OUT) == 4)
                                    reinterpret_cast<uint32_t *>(dst)[d] = v[d];
                                else
                                    reinterpret_cast<uint16_t *>(dst)[d] = (uint16_t)(v[d / 2] >> (16 * (d % 2)));
                            }
                    }
                }
            }
            wave_lds_fence();
        }
    }
};

template <typename OUT, typename MT>
__device__ __forceinline__ void mx_tile(const MxGemm &p, uint8_t *smem, int row0, int col0, int e0, int e1) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    mx_f32x4 acc[MT::TM][MT::TN];
    MT::template mainloop<OUT>(p, smem, row0, col0, e0, e1, tid, lane, wave, acc);
    MT::template epilogue<OUT>(p, smem, row0, col0, lane, wave, acc);
}

// OUT: the result's type; with K split over gridDim.y, slice y writes its fp32
// sums to rows y M ... of p.c (no bias) and mx_join_kernel adds them.
template <typename OUT, int BM, int BN, int WGM, int WGN, int NS>
__global__ __launch_bounds__(64 * WGM * WGN) void mx_tile_kernel(MxGemm p, int tiles_m, int tiles_n, int slice) {
    typedef MxTile<BM, BN, WGM, WGN, NS> MT;
    __shared__ __attribute__((aligned(16))) uint8_t smem[MT::LDS_BYTES];
    int tm, tn;
    mx_tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn);
    const int e0 = blockIdx.y * slice, e1 = min(e0 + slice, (p.nb + 7) / 8);
    if (gridDim.y > 1)
        p.c = (float *)p.c + (int64_t)blockIdx.y * p.M * p.ldc;
    mx_tile<OUT, MT>(p, smem, tm * BM, tn * BN, e0, e1);
}

// Two products in one grid, p's tiles and then q's, whose result is fp32: the second
// one's first tiles run beside the first one's last, and a small backward pass saves a launch (777 x 1000 x 520 17.0 -> 12.3 us;
// 4096^3 within noise).
template <typename OUT, int BM, int BN, int WGM, int WGN, int NS>
__global__ __launch_bounds__(64 * WGM * WGN) void mx_pair_kernel(MxGemm p, MxGemm q, int ptiles) {
    typedef MxTile<BM, BN, WGM, WGN, NS> MT;
    __shared__ __attribute__((aligned(16))) uint8_t smem[MT::LDS_BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // one main loop for both, none of which has a bias
    const bool second = (int)blockIdx.x >= ptiles;
    MxGemm g = second ? q : p;
    g.bias = nullptr;
    int tm, tn;
    mx_tile_of(second ? blockIdx.x - ptiles : blockIdx.x, second ? gridDim.x - ptiles : ptiles, (g.M + BM - 1) / BM,
               (g.N + BN - 1) / BN, tm, tn);
    mx_f32x4 acc[MT::TM][MT::TN];
    MT::template mainloop<float>(g, smem, tm * BM, tn * BN, 0, (g.nb + 7) / 8, tid, lane, wave, acc);
    if (second)
        MT::template epilogue<float>(g, smem, tm * BM, tn * BN, lane, wave, acc);
    else
        MT::template epilogue<OUT>(g, smem, tm * BM, tn * BN, lane, wave, acc);
}

// C = sum of ks slices of M x N fp32 partial results (row stride ldp) + bias,
// in the order of the slices. ks = 0: the bias alone (K = 0).
template <typename OUT>
__global__ __launch_bounds__(256) void mx_join_kernel(const float *part, int64_t ldp, int ks, MxGemm p) {
    const int64_t total = (int64_t)p.M * p.N;
    for (int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x; f < total; f += (int64_t)gridDim.x * 256) {
        const int m = (int)(f / p.N), n = (int)(f - (int64_t)m * p.N);
        float s = 0.f;
        for (int k = 0; k < ks; ++k)
            s += part[((int64_t)k * p.M + m) * ldp + n];
        ((OUT *)p.c)[(int64_t)m * p.ldc + n] = (OUT)(s + mx_bias<OUT>(p.bias, n));
    }
}

// ------------------------------------------------------------------ skinny

// 16 MF rows x 16 NF columns per workgroup, K in groups of 16 blocks dealt out
// to the 8 wavefronts in turn. At step s of a group, lane quarter q takes block
// 4 s + q, so that a load instruction reads 64 contiguous bytes of each of 16 rows; the
// scale bytes of its four blocks are picked from the row's 16. B of the next group is on
// its way during a group. The wavefronts' sums are joined in LDS in the order of the
// wavefronts. FUSED (MF = 1): a lane quantises the 32 activations of its block in
// registers; rows past M are zero.

constexpr int MX_FUSE_PIECES = 4;

// Bytes 4 s + quarter of a row's 16 scale bytes as byte s of a word, those of blocks
// >= left (blocks of the row from the group's first one on) cleared: their codes
// are read as zeros, and a stray 255 would make them NaN.
__device__ __forceinline__ int mx_pick_scales(u32x4 w, int quarter, int left) {
    const uint32_t sel = (uint32_t)quarter + ((uint32_t)(quarter + 4) << 8);
    const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], sel), hi = __builtin_amdgcn_perm(w[3], w[2], sel);
    const uint32_t v = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    const int n = (left - quarter + 3) >> 2;   // of this quarter's four blocks inside the row
    return n >= 4 ? (int)v : n <= 0 ? 0 : (int)(v & ((1u << (8 * n)) - 1u));
}

template <typename T, int MF, int NF, int PIECES, bool VEC>
__global__ __launch_bounds__(512) void mx_skinny_kernel(MxGemm p, MxSkinnyX px) {
    constexpr int NW = 8;
    constexpr bool FUSED = PIECES > 0;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float (*red)[MF * NF][4][64] = reinterpret_cast<float (*)[MF * NF][4][64]>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int n0 = blockIdx.x * 16 * NF;
    const int nb = p.nb, groups = (nb + 15) / 16;
    uint8_t *codes = smem + sizeof(float) * NW * MF * NF * 256;   // FUSED: 16 bytes per block and row
    uint8_t *scales = codes + ((size_t)(groups * 16) << (px.rlog + 4));   // a word per group, quarter and row
    const int rmask = (1 << px.rlog) - 1;

    // The four blocks and the scales of one group of a row.
    struct Rows {
        mx_i32x4 v[4];
        u32x4 s;
    };
    const uint8_t *bq[NF], *bs[NF], *aq[MF], *as[MF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const int n = min(n0 + 16 * j + r, p.N - 1);
        bq[j] = p.b + (int64_t)n * p.ldb;
        bs[j] = p.sb + (int64_t)n * p.ldsb;
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const int m = min(16 * i + r, p.M - 1);
        aq[i] = FUSED ? nullptr : p.a + (int64_t)m * p.lda;
        as[i] = FUSED ? nullptr : p.sa + (int64_t)m * p.ldsa;
    }
    // (No branches: a wait for all loads would stand behind each. Blocks past the row's
    // end are its last one again, under a scale of 0; A's codes are cleared too.)
    auto load = [&](const uint8_t *row, const uint8_t *scales, int g, Rows &x) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            x.v[s] = *reinterpret_cast<const mx_i32x4 *>(row + (int64_t)min(16 * g + 4 * s + q, nb - 1) * 16);
        x.s = *reinterpret_cast<const u32x4 *>(scales + 16 * g);
    };

    mx_f32x4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
            acc[i][j] = mx_f32x4{};

    Rows b[NF], bn[NF];
    auto first_group = [&]() {
        if (wave < groups) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
                load(bq[j], bs[j], wave, b[j]);
        }
    };
    if constexpr (!FUSED) {
        first_group();
    } else {
        // pieces of 8 elements, of whole groups; VEC: K is a multiple of 8
        const int per_row = groups * 64;
        uint32_t u[PIECES][MxPack<T>::WORDS8];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int f = i * 512 + tid, row = f / per_row, k0 = (f - row * per_row) * 8;
            const T *x = (const T *)px.x + (int64_t)min(row, p.M - 1) * px.ldx;
            if constexpr (VEC) {
                mx_load8<T, true>(x, min(k0, px.K - 8), px.K, u[i]);
#pragma unroll
                for (int d = 0; d < MxPack<T>::WORDS8; ++d)
                    u[i][d] = k0 < px.K ? u[i][d] : 0;
            } else {
                mx_load8<T, false>(x, k0, px.K, u[i]);
            }
        }
        first_group();   // (behind the activations: loads return in order)
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int f = i * 512 + tid, row = f / per_row, piece = f - row * per_row, blk = piece >> 2;
            uint32_t am = mx_amax8<T>(u[i]);
            am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0xB1, 0xF, 0xF, false));
            am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x4E, 0xF, 0xF, false));
            const uint32_t sc = mx_scale_of(am), w = mx_pack8<T>(u[i], sc);
            if (row < p.M) {
                *reinterpret_cast<uint32_t *>(codes + ((((size_t)blk << px.rlog) + ((row ^ blk) & rmask)) * 16 + (piece & 3) * 4)) = w;
                // block 16 g + 4 s + quarter: byte s of its word
                if ((piece & 3) == 0)
                    scales[(((size_t)((blk >> 4) * 4 + (blk & 3)) << px.rlog) + row) * 4 + ((blk >> 2) & 3)] = (uint8_t)sc;
            }
        }
        __syncthreads();
    }
    for (int g = wave; g < groups; g += NW) {
        const int left = nb - 16 * g;
        Rows a[MF];
        int sa[MF];
        if constexpr (!FUSED) {
#pragma unroll
            for (int i = 0; i < MF; ++i)
                load(aq[i], as[i], g, a[i]);
        }
        if (g + NW < groups) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
                load(bq[j], bs[j], g + NW, bn[j]);
        }
        if constexpr (FUSED) {
            // (rows past M repeat others: their outputs are not stored)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int blk = 16 * g + 4 * s + q;
                a[0].v[s] = *reinterpret_cast<const mx_i32x4 *>(codes + (((size_t)blk << px.rlog) + ((r ^ blk) & rmask)) * 16);
            }
            sa[0] = *reinterpret_cast<const int *>(scales + (((size_t)(4 * g + q) << px.rlog) + (r & rmask)) * 4);
        } else {
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                sa[i] = mx_pick_scales(a[i].s, q, left);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    a[i].v[s] = 4 * s + q < left ? a[i].v[s] : mx_i32x4{0, 0, 0, 0};
            }
        }
        int sb[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j)
            sb[j] = mx_pick_scales(b[j].s, q, left);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                acc[i][j] = mx_mfma16<0>(a[i].v[0], b[j].v[0], acc[i][j], sa[i], sb[j]);
                acc[i][j] = mx_mfma16<1>(a[i].v[1], b[j].v[1], acc[i][j], sa[i], sb[j]);
                acc[i][j] = mx_mfma16<2>(a[i].v[2], b[j].v[2], acc[i][j], sa[i], sb[j]);
                acc[i][j] = mx_mfma16<3>(a[i].v[3], b[j].v[3], acc[i][j], sa[i], sb[j]);
            }
#pragma unroll
        for (int j = 0; j < NF; ++j)
            b[j] = bn[j];
    }
    // register d of lane l: row 4 (l / 16) + d, column l % 16 of the block
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                red[wave][i * NF + j][d][lane] = acc[i][j][d];
    __syncthreads();
    for (int f = tid; f < MF * NF * 256; f += 512) {
        // consecutive threads take consecutive columns
        const int col = f % (16 * NF), row = f / (16 * NF);
        const int i = row / 16, j = col / 16, d = row % 4, l = (row % 16) / 4 * 16 + col % 16;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            s += red[w][i * NF + j][d][l];
        const int n = n0 + col;
        if (row < p.M && n < p.N)
            ((T *)p.c)[(int64_t)row * p.ldc + n] = (T)(s + mx_bias<T>(p.bias, n));
    }
}

// ------------------------------------------------------------------ host

// Tile configurations, and what a round of them over all CUs costs against the
// others (4096^3, bf16: 38 us in 256 x 256 tiles, 47 in 128 x 128; 2048 x 4096 x 4096: 31 and 24; 333 x 5000 x
// 2100: 11.4 in 128 x 128, 8.7 in 64 x 64; 1000 x 520 x 777: 8.8 and 5.4).
struct MxCfg { int BM, BN; double cost; };
static const MxCfg kMxCfg[] = {{256, 256, 4.0}, {128, 128, 1.25}, {64, 64, 0.5}};

static int64_t mx_tiles(int c, int64_t M, int64_t N) {
    return ((M + kMxCfg[c].BM - 1) / kMxCfg[c].BM) * ((N + kMxCfg[c].BN - 1) / kMxCfg[c].BN);
}

// The cheapest configuration for a grid of tiles(c) workgroups.
template <typename F>
static int mx_cheapest(int cu_count, F tiles) {
    int cfg = 0;
    double best = 0;
    for (int c = 0; c < 3; ++c) {
        const double cost = kMxCfg[c].cost * (double)((tiles(c) + cu_count - 1) / cu_count);
        if (c == 0 || cost < best) {
            best = cost;
            cfg = c;
        }
    }
    return cfg;
}

// Few rows: the skinny kernel, whose workgroups each read all the activations, while their
// 32 columns go round the CUs once (M of 17 to 64) or a few times; then tiles of 64. Skinny and
// tile, us, weights cold, at K = 4096: 64 x 8192 11.2 and 12.9, 64 x 10240 19.3 and 11.7, 32 x 8192 8.5 and 11.9,
// 32 x 10240 14.0 and 11.4, 64 x 28672 36.9 and 19.4, 16 x 16384 12.5 and 12.0, 16 x 28672 20.9 and 15.9, 8 x 28672 18.7
// and 16.7, 1 x 28672 17.2 and 16.5, where the tiles need a launch for the activations as well.
// The same ends at K = 1024: 64 x 8192 5.4 and 5.6, 64 x 10240 8.7 and 5.6, 32 x 10240 6.7 and 5.6; at 16384: 32 x 8192
// 24.3 and 24.5, 32 x 10240 42.6 and 35.1, 16 x 28672 65.6 and 56.0.
// A long K splits over workgroups in tiles, over the eight wavefronts of one here, and more
// rows make its steps longer: tiles where M K passes 400000. 64 x 4096: K = 6144 1.11 times
// the skinny kernel's time in tiles, 8192 0.89, 16384 0.65; 48 x 1024: 6144 1.15, 8192 0.93, 16384 0.72; 32 x 4096: 12288 1.10,
// 16384 0.97; 32 x 2048: 8192 0.92, 16384 0.68; 24 x 1024 and 17 x 4096 at 16384 1.06 and 1.19.
static bool mx_is_skinny(int64_t M, int64_t N, int64_t nb, int cu_count) {
    if (M > 16 && M * nb > 400000 / 32)
        return false;
    return M <= 4 || (M <= 16 && N < 96 * cu_count) || (M <= 32 && N < 40 * cu_count) || (M <= 64 && N <= 32 * cu_count);
}

MxPlan plan_mx(int64_t M, int64_t N, int64_t nb, int cu_count) {
    MxPlan pl = {MX_TILE, 0, 1, 0, 0, cu_count};
    if (nb == 0) {
        pl.kind = MX_EMPTY;
        return pl;
    }
    if (mx_is_skinny(M, N, nb, cu_count)) {
        pl.kind = MX_SKINNY;
        pl.cfg = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
        return pl;
    }
    pl.cfg = mx_cheapest(cu_count, [&](int c) { return mx_tiles(c, M, N); });
    const int64_t stages = (nb + 7) / 8, t = mx_tiles(pl.cfg, M, N);
    pl.slice = (int)stages;
    // too few tiles for the chip and a long K: split it
    if (t * 2 <= cu_count && stages >= 8) {
        int64_t ks = cu_count / t;
        if (ks > stages / 4)
            ks = stages / 4;
        if (ks > 16)
            ks = 16;
        if (ks > 1) {
            pl.slice = (int)((stages + ks - 1) / ks + 1) / 2 * 2;   // (a slice starts at an even stage)
            pl.ks = (int)((stages + pl.slice - 1) / pl.slice);
            if (pl.ks > 1)
                pl.partial_bytes = pl.ks * M * ((N + 3) / 4 * 4) * 4;
        }
    }
    return pl;
}

static int mx_rlog(int64_t M) { return M <= 1 ? 0 : M <= 2 ? 1 : M <= 4 ? 2 : M <= 8 ? 3 : 4; }

// LDS bytes of quantised activations: codes and scale words of whole groups.
static unsigned mx_fused_bytes(int64_t nb, int rlog) { return (unsigned)(((nb + 15) / 16 * (4096 + 256)) >> (4 - rlog)); }

// Few activations: every workgroup quantises all of them. Fused and with a launch of
// the quantisation kernel before (us, other weights each call): 1 x 4096 x 4096 5.0 and 7.3,
// 4 x 4096 x 4096 6.0 and 7.8, 1 x 8192 x 8192 11.6 and 12.3; 16 x 4096 x 4096 10.6 and 8.1, 16 x 8192 x 8192
// 25 and 14.
bool mx_fuses(const MxPlan &plan, int64_t M, int64_t nb) {
    return plan.kind == MX_SKINNY && M <= 16 && M * ((nb + 15) / 16) <= MX_FUSE_PIECES * 512 / 64;
}

template <typename OUT, int BM, int BN, int WGM, int WGN, int NS>
static void tile_one(const MxGemm &p, const MxPlan &plan, hipStream_t stream) {
    const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
    hipLaunchKernelGGL((mx_tile_kernel<OUT, BM, BN, WGM, WGN, NS>), dim3((unsigned)(tm * tn), plan.ks),
                       dim3(64 * WGM * WGN), 0, stream, p, tm, tn, plan.slice);
}

template <typename OUT>
static void tile_cfg(const MxGemm &p, const MxPlan &plan, hipStream_t stream) {
    switch (plan.cfg) {
    case 0: tile_one<OUT, 256, 256, 4, 2, 2>(p, plan, stream); break;
    case 1: tile_one<OUT, 128, 128, 2, 2, 2>(p, plan, stream); break;
    default: tile_one<OUT, 64, 64, 2, 2, 3>(p, plan, stream); break;
    }
}

template <typename OUT>
static void join(const float *part, int64_t ldp, int ks, const MxGemm &p, hipStream_t stream) {
    const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
    hipLaunchKernelGGL((mx_join_kernel<OUT>), dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, stream,
                       part, ldp, ks, p);
}

// 32 columns per workgroup once 16 would go round the CUs more than once: the activations are
// then read, and in the fused form quantised, half as often. 16 and 32 columns, us, weights cold, at K =
// 4096: 64 rows x 4096 9.2 and 10.4, x 4160 15.6 and 10.4, x 8191 17.0 and 11.3; 32 x 4160 9.8 and 7.8; 16 x 4160 7.4
// and 6.5, at K = 1024 3.7 and 3.8. Up to four rows there is little to read, and in the fused form
// the other way round (4 x 4160 x 1024 3.6 and 3.9): from the width on that gives every CU 32.
template <typename T, int MF, int PIECES, bool VEC>
static void skinny_one(const MxGemm &p, const MxSkinnyX &px, int cus, hipStream_t stream) {
    const unsigned fused = PIECES > 0 ? mx_fused_bytes(p.nb, px.rlog) : 0;
    if (p.M <= 4 ? p.N >= 32 * cus : p.N > 16 * cus)
        hipLaunchKernelGGL((mx_skinny_kernel<T, MF, 2, PIECES, VEC>), dim3((p.N + 31) / 32), dim3(512), MF * 16384 + fused, stream, p, px);
    else
        hipLaunchKernelGGL((mx_skinny_kernel<T, MF, 1, PIECES, VEC>), dim3((p.N + 15) / 16), dim3(512), MF * 8192 + fused, stream, p, px);
}

template <typename T>
static hipError_t gemm_type(const MxGemm &p, const MxPlan &plan, float *partial, hipStream_t stream) {
    const int cus = plan.cus;
    if (plan.kind == MX_EMPTY) {
        join<T>(nullptr, 0, 0, p, stream);
    } else if (plan.kind == MX_SKINNY) {
        const MxSkinnyX px = {};
        if (plan.cfg == 1)
            skinny_one<T, 1, 0, true>(p, px, cus, stream);
        else if (plan.cfg == 2)
            skinny_one<T, 2, 0, true>(p, px, cus, stream);
        else
            skinny_one<T, 4, 0, true>(p, px, cus, stream);
    } else if (plan.ks > 1) {
        MxGemm s = p;
        s.c = partial;
        s.ldc = (p.N + 3) / 4 * 4;
        s.bias = nullptr;
        tile_cfg<float>(s, plan, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        join<T>(partial, s.ldc, plan.ks, p, stream);
    } else {
        tile_cfg<T>(p, plan, stream);
    }
    return hipGetLastError();
}

hipError_t launch_mx_gemm(int type, const MxGemm &p, const MxPlan &plan, float *partial, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return gemm_type<_Float16>(p, plan, partial, stream);
    case MPGEMM_TYPE_BF16: return gemm_type<__bf16>(p, plan, partial, stream);
    default: return gemm_type<float>(p, plan, partial, stream);
    }
}

bool mx_pairs(const MxPlan &a, const MxPlan &b) {
    return a.kind == MX_TILE && b.kind == MX_TILE && a.ks == 1 && b.ks == 1;
}

template <typename T>
static hipError_t pair_type(const MxGemm &p, const MxGemm &q, int cus, hipStream_t stream) {
    auto tiles = [&](int c) { return mx_tiles(c, p.M, p.N) + mx_tiles(c, q.M, q.N); };
    const int c = mx_cheapest(cus, tiles), first = (int)mx_tiles(c, p.M, p.N);
    const dim3 grid((unsigned)tiles(c));
    if (c == 0)
        hipLaunchKernelGGL((mx_pair_kernel<T, 256, 256, 4, 2, 2>), grid, dim3(512), 0, stream, p, q, first);
    else if (c == 1)
        hipLaunchKernelGGL((mx_pair_kernel<T, 128, 128, 2, 2, 2>), grid, dim3(256), 0, stream, p, q, first);
    else
        hipLaunchKernelGGL((mx_pair_kernel<T, 64, 64, 2, 2, 3>), grid, dim3(256), 0, stream, p, q, first);
    return hipGetLastError();
}

hipError_t launch_mx_pair(int type, const MxGemm &p, const MxGemm &q, int cus, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return pair_type<_Float16>(p, q, cus, stream);
    case MPGEMM_TYPE_BF16: return pair_type<__bf16>(p, q, cus, stream);
    default: return pair_type<float>(p, q, cus, stream);
    }
}

template <typename T>
static hipError_t gemm_x_type(const MxGemm &p, const MxSkinnyX &px, int cus, hipStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(px.x) & 15) == 0 && (px.ldx * sizeof(T)) % 16 == 0 && px.K % 8 == 0;
    if (!vec)
        skinny_one<T, 1, MX_FUSE_PIECES, false>(p, px, cus, stream);
    else if (p.M * ((p.nb + 15) / 16) * 64 <= 512)
        skinny_one<T, 1, 1, true>(p, px, cus, stream);
    else
        skinny_one<T, 1, MX_FUSE_PIECES, true>(p, px, cus, stream);
    return hipGetLastError();
}

hipError_t launch_mx_gemm_x(int type, const MxGemm &p, const MxSkinnyX &px, const MxPlan &plan, hipStream_t stream) {
    if (!mx_fuses(plan, p.M, p.nb))
        return hipErrorInvalidValue;
    MxSkinnyX x = px;
    x.rlog = mx_rlog(p.M);
    switch (type) {
    case MPGEMM_TYPE_F16: return gemm_x_type<_Float16>(p, x, plan.cus, stream);
    case MPGEMM_TYPE_BF16: return gemm_x_type<__bf16>(p, x, plan.cus, stream);
    default: return gemm_x_type<float>(p, x, plan.cus, stream);
    }
}

}  // namespace mpg
