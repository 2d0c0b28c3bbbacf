// Main loop of the 16-bit and 8-bit integer tile kernels of the linear layers
// (w8a8.hip, gated.hip): a BM x BN tile of sum_k a(m, k) b(n, k) on gfx950's
// 16x16 matrix instructions.
//
// A stage is 128 bytes of k for every row (64 elements of 16 bits, 128 of 8). It
// is loaded and used in halves: A's tile rows [0, BM / 2) and [BM / 2, BM), B's
// the same, and a wavefront owns the same part of either half, so that a stage is
// four phases, one for each pair of halves:
//   phase 0  A0 B0     1  A0 B1     2  A1 B1     3  A1 B0
// Each phase needs one new half, whose fragments are read from LDS during the
// phase before, and frees the LDS of one half, which a direct-to-LDS load of a
// later stage fills from the next phase on. Two stages of LDS then hold six
// halves on their way while two are in use: the wait at the end of a phase leaves
// those six outstanding and never drains the loads.
//
// Operands are stored along k (a row is one m or n, as the weights and activations
// of a forward pass) or across it (a row is one k, as in the products of a
// backward pass: COL); those go through LDS as they are and the reads transpose
// them (ds_read_tr).
#pragma once

#include <type_traits>

#include "lds_dma.h"

namespace mpg {

typedef uint32_t pt_u32x4 __attribute__((ext_vector_type(4)));
typedef float pt_f32x4 __attribute__((ext_vector_type(4)));
typedef int pt_i32x4 __attribute__((ext_vector_type(4)));
typedef short pt_i16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 pt_f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 pt_bf16x8 __attribute__((ext_vector_type(8)));

// Range of the buffer that a half's loads go through: offsets from here on load zeros.
constexpr uint32_t kPtRange = 0x7FFFFFF0u;

// Element types: the matrix instruction takes 16 bytes per lane of either operand.
struct PtF16 {
    typedef _Float16 T;
    typedef pt_f32x4 Acc;
    static __device__ __forceinline__ Acc mfma(pt_u32x4 a, pt_u32x4 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(pt_f16x8, a), __builtin_bit_cast(pt_f16x8, b), c, 0, 0, 0);
    }
};
struct PtBF16 {
    typedef __bf16 T;
    typedef pt_f32x4 Acc;
    static __device__ __forceinline__ Acc mfma(pt_u32x4 a, pt_u32x4 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(pt_bf16x8, a), __builtin_bit_cast(pt_bf16x8, b), c, 0, 0, 0);
    }
};
struct PtI8 {
    typedef int8_t T;
    typedef pt_i32x4 Acc;
    static __device__ __forceinline__ Acc mfma(pt_u32x4 a, pt_u32x4 b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(pt_i32x4, a), __builtin_bit_cast(pt_i32x4, b), c, 0, 0, 0);
    }
};

// An operand of a tile: p[h] is the first row (COL: column) of half h, whose rows past rows[h]
// repeat the last (their outputs are not stored; a half without rows is not touched).
// Along k: ld[h] bytes between rows, `chunks` 16-byte chunks of k. Across k: ld[0] bytes
// between k's, `chunks` k's (columns are read in whole chunks of 16 bytes). JOIN: from stage
// `split` on, the k's go on at next[h], `chunks` of them again.
struct PtSource {
    const uint8_t *p[2], *next[2];
    int64_t ld[2];
    int rows[2];
    int chunks, split;
};

template <class E, int BM, int BN, int WGM, int WGN, bool ACOL, bool BCOL, bool JOIN = false>
struct PhaseTile {
    static constexpr int NW = WGM * WGN, NT = 64 * NW, WGN_ = WGN;
    static constexpr int HM = BM / 2, HN = BN / 2;             // rows of a half
    static constexpr int WM = HM / WGM, WN = HN / WGN;         // of those, a wavefront's
    static constexpr int FM = WM / 16, FN = WN / 16;           // fragments
    static constexpr int LA = HM * 8 / NT, LB = HN * 8 / NT;   // loads of a half per thread
    static constexpr int L = LA > LB ? LA : LB;
    static constexpr int SA = HM * 128, SB = HN * 128;         // bytes of a half
    static constexpr int LDS_BYTES = 4 * (SA + SB);
    static_assert(LA == LB && HM * 8 % NT == 0 && HN * 8 % NT == 0, "every half takes the same number of loads");
    static_assert(WM % 16 == 0 && WN % 16 == 0 && 6 * L < 64 && LDS_BYTES <= 160 * 1024, "tile");
    static_assert(sizeof(typename E::T) == 2 || (!ACOL && !BCOL), "bytes are not transposed");

    typedef typename E::Acc Acc;
    static constexpr int EB = sizeof(typename E::T);

    // Along k, 16-byte chunk c of row r sits at c ^ swz(r): the reads of a chunk over 16 rows are
    // free of bank conflicts. Across k, a row holds the half's columns in 32-byte slots
    // of 16; slot p of row k sits at p ^ turn(k), which spreads the 8 rows that 32 lanes read over all banks.
    static __device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
    template <int H>
    static __device__ __forceinline__ int turn(int k) {
        constexpr int slots = H / 16;   // 8, 4 or 2 (powers of two)
        static_assert(slots == 2 || slots == 4 || slots == 8, "slots");
        return ((k & 3) | ((k >> 1) & 4)) / (8 / slots);
    }

    // The source offsets of a thread's loads of half h (bytes from p[h]; a half without rows is not touched).
    template <bool COL, int H>
    static __device__ __forceinline__ void offsets(const PtSource &s, int h, int tid, uint32_t (&off)[L]) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int f = j * NT + tid;
            if constexpr (COL) {
                constexpr int cpr = H / 8;
                const int k = f / cpr, c = f % cpr;
                const int col = min((((c >> 1) ^ turn<H>(k)) * 2 + (c & 1)) * 8, (s.rows[h] - 1) / 8 * 8);
                off[j] = (uint32_t)k * (uint32_t)s.ld[0] + (uint32_t)col * 2;
            } else {
                const int r = f / 8, c = (f % 8) ^ swz(r);
                off[j] = (uint32_t)min(r, s.rows[h] - 1) * (uint32_t)s.ld[h] + c * 16;
            }
            if (s.rows[h] <= 0)
                off[j] = kPtRange;
        }
    }

    // Loads of half h of stage e into `lds`. Buffer loads: one 32-bit offset per load in registers
    // (the 64-bit addresses of the global form do not fit beside the sums), and what is past the
    // operand's end gets an offset out of the buffer's range, which loads zeros.
    template <bool COL, int H>
    static __device__ __forceinline__ void load(const PtSource &s, int h, int e, const uint32_t (&off)[L], uint8_t *lds,
                                                int tid, int wave) {
        const uint8_t *from = s.p[h];
        if (COL && JOIN) {
            from = e < s.split ? from : s.next[h];
            e = e < s.split ? e : e - s.split;
        }
        const uint8_t *base = from + (COL ? (int64_t)e * 64 * s.ld[0] : (int64_t)e * 128);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, kPtRange, 0x00020000);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int f = j * NT + tid;
            const int at = COL ? f / (H / 8) : (f % 8) ^ swz(f / 8);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(lds + (j * NT + wave * 64) * 16), 16,
                                                     at < s.chunks - (COL ? 64 : 8) * e ? off[j] : kPtRange, 0, 0, 0);
        }
    }

    // N fragments (of 16 rows from `first` on) of both steps of a stage's half. Step s of lane
    // quarter q takes k chunk 4 s + q.
    template <bool COL, int H, int N>
    static __device__ __forceinline__ void read(const uint8_t *lds, int first, int lane, pt_u32x4 (&f)[N][2]) {
        const int q = lane >> 4, i = lane & 15;
        if constexpr (COL) {
            constexpr int RB = H * 2;
            const int g = turn<H>(8 * q + (i >> 2));
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint8_t *a = lds + (8 * q + (i >> 2)) * RB + ((first / 16 + n) ^ g) * 32 + (i & 3) * 8;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    typedef __attribute__((address_space(3))) pt_i16x4 lds4;
                    const pt_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(a + 32 * s * RB));
                    const pt_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(a + (32 * s + 4) * RB));
                    f[n][s] = __builtin_bit_cast(pt_u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
            }
        } else {
            const uint8_t *a = lds + (first + i) * 128;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    f[n][s] = *reinterpret_cast<const pt_u32x4 *>(a + n * 2048 + (((4 * s + q) ^ swz(i)) * 16));
        }
    }

    // Operands swapped, so each accumulator block is the transpose of its block of the
    // result: register d of lane l holds row l % 16, column 4 (l / 16) + d.
    static __device__ __forceinline__ void quadrant(const pt_u32x4 (&a)[FM][2], const pt_u32x4 (&b)[FN][2], Acc (&acc)[FM][FN]) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = E::mfma(b[j][s], a[i][s], acc[i][j]);
    }

    // The order of a phase's instructions: the next half's reads (R of them) one behind each of the
    // first matrix instructions, then the loads. Left alone, the compiler gathers them in front
    // or behind. (8192^3 in bf16: 787 us left alone, 759 in this order, 789 with all reads first.)
    template <int R>
    static __device__ __forceinline__ void weave() {
        constexpr int MM = FM * FN * 2;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, MM, 0);
    }

    // The sums of stages [0, stages): acc[ha][hb][i][j], half and fragment of either operand.
    static __device__ __forceinline__ void mainloop(const PtSource &A, const PtSource &B, int stages, uint8_t *smem,
                                                    int tid, int lane, int wave, Acc (&acc)[2][2][FM][FN]) {
        const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN;
        uint32_t oa[2][L], ob[2][L];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            offsets<ACOL, HM>(A, h, tid, oa[h]);
            offsets<BCOL, HN>(B, h, tid, ob[h]);
        }
        uint8_t *la = smem, *lb = smem + 4 * SA;   // half h of the stage in slot e % 2: [2 h + e % 2]
        auto load_a = [&](int h, int e) { load<ACOL, HM>(A, h, e, oa[h], la + (2 * h + (e & 1)) * SA, tid, wave); };
        auto load_b = [&](int h, int e) { load<BCOL, HN>(B, h, e, ob[h], lb + (2 * h + (e & 1)) * SB, tid, wave); };
        pt_u32x4 a0[FM][2], a1[FM][2], bx[FN][2], by[FN][2];
        auto read_a = [&](int h, int slot, pt_u32x4 (&f)[FM][2]) { read<ACOL, HM>(la + (2 * h + slot) * SA, wm, lane, f); };
        auto read_b = [&](int h, int slot, pt_u32x4 (&f)[FN][2]) { read<BCOL, HN>(lb + (2 * h + slot) * SB, wn, lane, f); };
        constexpr int RA = FM * (ACOL ? 4 : 2), RB = FN * (BCOL ? 4 : 2);
        auto end_phase = [&]() {
            __builtin_amdgcn_sched_barrier(0);
            wait_vm_lds<6 * L>();
            lds_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            load_a(0, e);
            load_b(0, e);
            load_b(1, e);
            load_a(1, e);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[h >> 1][h & 1][i][j] = Acc{};
        end_phase();
        read_a(0, 0, a0);
        read_b(0, 0, bx);
        end_phase();
        load_a(0, 2);
        end_phase();
        // Stage e in slot S, with B0's fragments in b and B1's to come into c
        auto stage = [&](int e, int slot, pt_u32x4 (&b)[FN][2], pt_u32x4 (&c)[FN][2]) {
            read_b(1, slot, c);
            load_b(0, e + 2);
            quadrant(a0, b, acc[0][0]);
            weave<RB>();
            end_phase();
            read_a(1, slot, a1);
            load_b(1, e + 2);
            quadrant(a0, c, acc[0][1]);
            weave<RA>();
            end_phase();
            read_a(0, slot ^ 1, a0);
            load_a(1, e + 2);
            quadrant(a1, c, acc[1][1]);
            weave<RA>();
            end_phase();
            read_b(0, slot ^ 1, c);
            load_a(0, e + 3);
            quadrant(a1, b, acc[1][0]);
            weave<RB>();
            end_phase();
        };
        // (past the last stage zeros are loaded, and an odd number of stages takes one of zeros too)
        for (int e = 0; e < stages; e += 2) {
            stage(e, 0, bx, by);
            stage(e + 1, 1, by, bx);
        }
        wait_vm_lds<0>();
        __syncthreads();
    }

    // One more step for the elements of a last chunk that K (in bytes, along k) ends in: straight from
    // memory, in the lanes of the first quarter, the others zero.
    static __device__ __forceinline__ void tail(const PtSource &A, const PtSource &B, int bytes, int lane, int wave,
                                                Acc (&acc)[2][2][FM][FN]) {
        const int wm = (wave / WGN) * WM, wn = (wave % WGN) * WN, from = bytes / 16 * 16, n = (bytes - from) / EB;
        auto part = [&](const PtSource &s, int h, int row) {
            typedef typename std::conditional<EB == 1, uint8_t, uint16_t>::type Bits;
            Bits e[16 / EB] = {};
            if (s.rows[h] > 0 && lane < 16) {
                const Bits *src = reinterpret_cast<const Bits *>(s.p[h] + (int64_t)min(row, s.rows[h] - 1) * s.ld[h] + from);
#pragma unroll
                for (int k = 0; k < 16 / EB; ++k)
                    if (k < n)
                        e[k] = src[k];
            }
            pt_u32x4 v;
            __builtin_memcpy(&v, e, 16);
            return v;
        };
        pt_u32x4 a[2][FM], b[2][FN];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
                a[h][i] = part(A, h, wm + 16 * i + (lane & 15));
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[h][j] = part(B, h, wn + 16 * j + (lane & 15));
        }
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[ha][hb][i][j] = E::mfma(b[hb][j], a[ha][i], acc[ha][hb][i][j]);
    }
};

}  // namespace mpg
