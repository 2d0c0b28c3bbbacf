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
// later stage fills two phases on. Two stages of LDS (NS; small tiles have more) then hold
// four to six halves on their way; the wait before a barrier leaves four of them outstanding and
// never drains the loads. There is a barrier behind every second phase (behind every one: 8192^3 in bf16
// 741 us for 734, 4096 x 20480 x 4096 497 for 490).
//
// Bound by the matrix units' power: tiles of 256 x 256 in bf16 take 730 us for 8192^3 (1.51 PFLOP/s, the gated block of
// 8192 x 4096 x 8192; the library's plain product 680 on that card), in integers 376 to 396 us (2.8 to 2.9 POP/s;
// the library's 463). The clock falls to 1.7 to 1.85 GHz under it (2.4 at rest), and the units are busy in
// 73 to 76 % of its cycles; no cycle of LDS is lost to bank conflicts.
//
// Operands are stored along k (a row is one m or n, as the weights and activations
// of a forward pass) or across it (a row is one k, as in the products of a
// backward pass: COL); those go through LDS as they are and the reads transpose
// them (ds_read_tr).
#pragma once

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
// Along k: ld[h] bytes between rows, `chunks` 16-byte chunks of k (behind k's end the last has to hold
// zeros, of integers in one of the operands). Across k: ld[0] bytes
// between k's, `chunks` k's (columns are read in whole chunks of 16 bytes). JOIN: from stage
// `split` on, the k's go on at next[h], `chunks` of them again.
struct PtSource {
    const uint8_t *p[2], *next[2];
    int64_t ld[2];
    int rows[2];
    int chunks, split;
};

template <class E, int BM, int BN, int WGM, int WGN, int NS, bool ACOL, bool BCOL, bool JOIN = false>
struct PhaseTile {
    static constexpr int NW = WGM * WGN, NT = 64 * NW, WGN_ = WGN;
    static constexpr int HM = BM / 2, HN = BN / 2;             // rows of a half
    static constexpr int WM = HM / WGM, WN = HN / WGN;         // of those, a wavefront's
    static constexpr int FM = WM / 16, FN = WN / 16;           // fragments
    static constexpr int LA = HM * 8 / NT, LB = HN * 8 / NT;   // loads of a half per thread
    static constexpr int LS = 2 * (LA + LB);                   // of a stage
    static constexpr int SA = HM * 128, SB = HN * 128;         // bytes of a half
    static constexpr int LDS_BYTES = 2 * NS * (SA + SB);
    static constexpr bool PHASED = FM * FN >= 4;               // (below)
    static_assert(HM * 8 % NT == 0 && HN * 8 % NT == 0 && (LA == LB || !PHASED), "loads");
    static_assert(WM % 16 == 0 && WN % 16 == 0 && (NS - 1) * LS < 64 && NS % 2 == 0 && NS >= (PHASED ? 2 : 4) && LDS_BYTES <= 160 * 1024, "tile");
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
        return ((k & 3) | ((k >> 2) & 4)) / (8 / slots);
    }

    // The source offsets of a thread's loads of half h (bytes from p[h]; a half without rows is not touched).
    template <bool COL, int H, int L>
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

    // Loads of half h of stage e into `lds`, stage after stage (at_k, across k: where the next
    // stage begins). Buffer loads: one 32-bit offset per load in registers (the 64-bit addresses
    // of the global form do not fit beside the sums), and what is past the operand's end gets an
    // offset out of the buffer's range, which loads zeros. Kernels with
    // transposing reads write the load as an instruction of its own: the compiler takes those
    // reads as possible uses of any load to LDS before them and would wait for all loads in
    // front of each (4096 x 4096 x 20480 with B across k: 579 us, 461 without those waits;
    // 20480 x 4096 x 4096 with both: 548 and 495). The load has no result in registers; its
    // LDS address is an operand bound to m0, so the compiler knows of that register's use.
    template <bool COL, int H, int L>
    static __device__ __forceinline__ void load(const PtSource &s, int h, int e, const uint8_t *(&at_k)[2], const uint32_t (&off)[L],
                                                uint8_t *lds, int tid, int wave) {
        const uint8_t *base = s.p[h];
        if constexpr (COL) {
            base = at_k[h];
            at_k[h] = JOIN && e + 1 == s.split ? s.next[h] : base + 64 * s.ld[0];
            if (JOIN)
                e = e < s.split ? e : e - s.split;
        }
        const uint32_t ahead = COL ? 0 : e * 128;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int f = j * NT + tid;
            const int at = COL ? f / (H / 8) : (f % 8) ^ swz(f / 8);
            const uint32_t o = at < s.chunks - (COL ? 64 : 8) * e ? off[j] : kPtRange;
            typedef __attribute__((address_space(3))) uint8_t lds_byte;
            lds_byte *to = (lds_byte *)(lds + (j * NT + wave * 64) * 16);
            if constexpr (ACOL || BCOL) {
                const uint64_t at64 = reinterpret_cast<uint64_t>(base);
                const pt_u32x4 r = {(uint32_t)at64, (uint32_t)(at64 >> 32) & 0xFFFFu, kPtRange, 0x00020000u};
                asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                             : : "{m0}"((uint32_t)(uintptr_t)to), "v"(o), "s"(r), "s"(ahead));
            } else {
                const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, kPtRange, 0x00020000);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, o, ahead, 0, 0);
            }
        }
    }

    // N fragments (of 16 rows from `first` on) of both steps of a stage's half. Step s of lane
    // quarter q takes k chunk 2 q + s (with 4 s + q the row reads had conflicts in half of their cycles).
    template <bool COL, int H, int N>
    static __device__ __forceinline__ void read(const uint8_t *lds, int first, int lane, pt_u32x4 (&f)[N][2]) {
        const int q = lane >> 4, i = lane & 15;
        if constexpr (COL) {
            constexpr int RB = H * 2;
            const int g = turn<H>(16 * q + (i >> 2));
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint8_t *a = lds + (16 * q + (i >> 2)) * RB + ((first / 16 + n) ^ g) * 32 + (i & 3) * 8;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    typedef __attribute__((address_space(3))) pt_i16x4 lds4;
                    const pt_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(a + 8 * s * RB));
                    const pt_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(a + (8 * s + 4) * RB));
                    f[n][s] = __builtin_bit_cast(pt_u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
            }
        } else {
            const uint8_t *a = lds + (first + i) * 128;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    f[n][s] = *reinterpret_cast<const pt_u32x4 *>(a + n * 2048 + (((2 * q + s) ^ swz(i)) * 16));
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
    // first matrix instructions (the shorter transposing reads two), then the loads. Left alone, the
    // compiler gathers them in front or behind. (8192^3 in bf16: 787 us left alone, 759 in this order,
    // 789 with all reads first.) The loads that are instructions of their own go where they fit.
    template <int R, bool COL>
    static __device__ __forceinline__ void weave() {
        constexpr int MM = FM * FN * 2, AT = COL ? 2 : 1, L = LA;
#pragma unroll
        for (int i = 0; i < R / AT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, AT, 0);
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
        uint32_t oa[2][LA], ob[2][LB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            offsets<ACOL, HM>(A, h, tid, oa[h]);
            offsets<BCOL, HN>(B, h, tid, ob[h]);
        }
        uint8_t *la = smem, *lb = smem + 2 * NS * SA;   // half h of stage e: [NS h + e % NS]
        const uint8_t *ka[2] = {A.p[0], A.p[1]}, *kb[2] = {B.p[0], B.p[1]};
        auto load_a = [&](int h, int e, int slot) { load<ACOL, HM>(A, h, e, ka, oa[h], la + (NS * h + slot) * SA, tid, wave); };
        auto load_b = [&](int h, int e, int slot) { load<BCOL, HN>(B, h, e, kb, ob[h], lb + (NS * h + slot) * SB, tid, wave); };
        auto read_a = [&](int h, int slot, pt_u32x4 (&f)[FM][2]) { read<ACOL, HM>(la + (NS * h + slot) * SA, wm, lane, f); };
        auto read_b = [&](int h, int slot, pt_u32x4 (&f)[FN][2]) { read<BCOL, HN>(lb + (NS * h + slot) * SB, wn, lane, f); };
#pragma unroll
        for (int e = 0; e < NS; ++e) {
            load_a(0, e, e);
            load_b(0, e, e);
            load_b(1, e, e);
            load_a(1, e, e);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[h >> 1][h & 1][i][j] = Acc{};
        if constexpr (PHASED) {
            pt_u32x4 a0[FM][2], a1[FM][2], bx[FN][2], by[FN][2];
            constexpr int RA = FM * (ACOL ? 4 : 2), RB = FN * (BCOL ? 4 : 2);
            // Behind phases 0 and 2 the wavefront's own reads have to be done, behind 1 and 3 everybody's, and
            // the loads of the two halves that the next two phases read: all but the last 4 (NS - 1) halves.
            auto mid_phase = [&]() {
                __builtin_amdgcn_sched_barrier(0);
                wait_lds_only();
                __builtin_amdgcn_sched_barrier(0);
            };
            auto end_phase = [&]() {
                __builtin_amdgcn_sched_barrier(0);
                wait_vm_lds<(NS - 1) * LS>();
                lds_barrier();
                __builtin_amdgcn_sched_barrier(0);
            };
            end_phase();
            read_a(0, 0, a0);
            read_b(0, 0, bx);
            end_phase();
            // Stage e in its slot, with B0's fragments in b and B1's to come into c. A half's LDS is loaded into
            // after the barrier behind the phase that read it.
            auto stage = [&](int e, int slot, pt_u32x4 (&b)[FN][2], pt_u32x4 (&c)[FN][2]) {
                read_b(1, slot, c);
                load_a(0, e + NS, slot);
                quadrant(a0, b, acc[0][0]);
                weave<RB, BCOL>();
                mid_phase();
                read_a(1, slot, a1);
                load_b(0, e + NS, slot);
                quadrant(a0, c, acc[0][1]);
                weave<RA, ACOL>();
                end_phase();
                read_a(0, (slot + 1) % NS, a0);
                load_b(1, e + NS, slot);
                quadrant(a1, c, acc[1][1]);
                weave<RA, ACOL>();
                mid_phase();
                read_b(0, (slot + 1) % NS, c);
                load_a(1, e + NS, slot);
                quadrant(a1, b, acc[1][0]);
                weave<RB, BCOL>();
                end_phase();
            };
            for (int e = 0; e < stages; e += NS)   // (past the last stage zeros are loaded)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    if (i > 0 && e + i >= stages)
                        break;
                    if (i % 2 == 0)
                        stage(e + i, i, bx, by);
                    else
                        stage(e + i, i, by, bx);
                }
        } else {
            // Small tiles: a stage at a time, its fragments read during the stage before. (A phase of two matrix
            // instructions does not cover the reads' way: 64 x 64 tiles took 0.67 us a stage in phases.)
            struct Frags {
                pt_u32x4 a[2][FM][2], b[2][FN][2];
            } f0, f1;
            auto read_stage = [&](int slot, Frags &f) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    read_a(h, slot, f.a[h]);
                    read_b(h, slot, f.b[h]);
                }
            };
            auto next = [&]() {
                __builtin_amdgcn_sched_barrier(0);
                wait_vm_lds<(NS - 2) * LS>();   // all but the last NS - 2 stages have landed
                lds_barrier();
                __builtin_amdgcn_sched_barrier(0);
            };
            auto stage = [&](int e, int slot, const Frags &f, Frags &n) {
                next();
                load_a(0, e + NS, slot);
                load_b(0, e + NS, slot);
                load_b(1, e + NS, slot);
                load_a(1, e + NS, slot);
                read_stage((slot + 1) % NS, n);
#pragma unroll
                for (int ha = 0; ha < 2; ++ha)
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
                        quadrant(f.a[ha], f.b[hb], acc[ha][hb]);
            };
            wait_vm_lds<(NS - 1) * LS>();
            lds_barrier();
            read_stage(0, f0);
            for (int e = 0; e < stages; e += NS)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    if (i > 0 && e + i >= stages)
                        break;
                    if (i % 2 == 0)
                        stage(e + i, i, f0, f1);
                    else
                        stage(e + i, i, f1, f0);
                }
        }
        wait_vm_lds<0>();
        __syncthreads();
    }
};

}  // namespace mpg
