// MXFP4 quantisation and dequantisation.
//
// A block is 32 elements along the contracted axis: one scale byte b, the
// biased exponent of a power of two, and 32 e2m1 codes. With E the exponent
// field of amax seen as an fp32 number (so floor(log2 amax) = E - 127 when it
// is normal there),
//   b = max(E - 2, 0)        code = e2m1(x / 2^(b - 127))
// which puts amax into [4, 8): the top binade of e2m1 (values over 6 saturate
// to 6). E = 255 (NaN or infinity in the block) gives b = 255, the e8m0 NaN. An
// fp32-subnormal amax has E = 0 and b = 0: the smallest scale, 2^-127. amax is
// taken on the bit patterns without their sign, as integers, which orders
// magnitudes and keeps NaN on top. The division and rounding (nearest, ties to
// even, saturating) are v_cvt_scalef32_pk_fp4_*, which was compared with the
// definition for every fp16 and bf16 value and every scale.
//
// Bound by memory: 2 or 4 bytes read, 17/32 of a byte written per orientation.
#include "mxfp4.h"
#include "mxfp4_device.h"

namespace mpg {

// Threads of a workgroup over (rows, pieces of 8 elements): 2^tlog of the 256 side by
// side along a row. A thread takes 4 rows, all loaded before the first is worked on, where
// that leaves 8 workgroups per CU, else one. (One piece per thread found by a 64-bit
// division: 12.3 us for the values of 4096 x 4096 in bf16, this 8.0.)
struct MxSpread {
    int tlog;
    bool four;
    dim3 grid;
    MxSpread(int64_t M, int64_t pieces) {
        for (tlog = 2; tlog < 8 && (1 << tlog) < pieces; ++tlog)
            ;
        const int64_t across = (pieces + (1 << tlog) - 1) >> tlog, per = 256 >> tlog;
        four = (M + per * 4 - 1) / (per * 4) * across >= 2048;
        const int64_t rows = four ? per * 4 : per;
        grid = dim3((unsigned)((M + rows - 1) / rows), (unsigned)across);
    }
};

// Rows only: a lane owns 8 consecutive elements (one 16-byte load where the
// rows are 16-byte aligned and the type has 2 bytes), a block is 4 lanes, whose
// maximum is taken with two DPP moves; each lane stores its 8 codes as one
// word, the block's first lane the scale.
template <typename T, bool VEC, int ROWS>
__global__ __launch_bounds__(256) void mx_quantize_rows_kernel(MxQuantize p, int tlog, int pieces) {
    const int piece = (int)(blockIdx.y << tlog) + (threadIdx.x & ((1 << tlog) - 1)), k0 = piece * 8;
    const int step = 256 >> tlog, row0 = (int)blockIdx.x * step * ROWS + (threadIdx.x >> tlog);
    if (piece >= pieces)   // (whole blocks: pieces is a multiple of 4)
        return;
    uint32_t u[ROWS][MxPack<T>::WORDS8];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        if (row0 + i * step < p.M)
            mx_load8<T, VEC>((const T *)p.x + (int64_t)(row0 + i * step) * p.ldx, k0, p.K, u[i]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = row0 + i * step;
        if (row >= p.M)
            return;
        uint32_t am = mx_amax8<T>(u[i]);
        // the four lanes of a block are in one DPP quad and take part together
        am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0xB1, 0xF, 0xF, false));
        am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x4E, 0xF, 0xF, false));
        const uint32_t b = mx_scale_of(am);
        *reinterpret_cast<uint32_t *>(p.q + (int64_t)row * p.ldq + piece * 4) = mx_pack8<T>(u[i], b);
        if ((threadIdx.x & 3) == 0)
            p.s[(int64_t)row * p.lds + piece / 4] = (uint8_t)b;
    }
}

// Columns, or both orientations: one 128 x 128 tile per workgroup. The tile is
// read once, coalesced; the row codes come from the registers of that read as
// in the kernel above, and the elements go to LDS, from which each thread then
// takes 32 rows of a word (two columns of a 2-byte type, one of fp32). In LDS
// the words of a row are permuted in groups of 16 by the row's block (word c of
// block g at c ^ 16 (g % 4)): the 64 lanes of a wavefront read 16 words in each
// of 4 blocks of rows, and the permutation puts them into 64 different banks.
// The block index is the fastest one over the lanes, so four lanes store 64
// contiguous bytes of column codes and, joined, the 4 scale bytes.
template <typename T, bool VEC, bool ROWS>
__global__ __launch_bounds__(256) void mx_quantize_both_kernel(MxQuantize p, int tiles_k) {
    constexpr int TR = 128, TC = 128;
    constexpr int WPR = TC * (int)sizeof(T) / 4;   // words per row
    __shared__ __attribute__((aligned(16))) uint32_t tile[TR * WPR];
    const int tid = threadIdx.x;
    const int row0 = (int)(blockIdx.x / tiles_k) * TR, col0 = (int)(blockIdx.x % tiles_k) * TC;
    constexpr int W8 = MxPack<T>::WORDS8;   // words of 8 elements

    // 16 lanes per row, 16 rows per pass
    const int lc = tid % 16, lr = tid / 16;
    const int k0 = col0 + lc * 8;
    uint32_t u[TR / 16][W8];
#pragma unroll
    for (int i = 0; i < TR / 16; ++i) {
        const int row = row0 + i * 16 + lr;
        if (row < p.M) {
            mx_load8<T, VEC>((const T *)p.x + (int64_t)row * p.ldx, k0, p.K, u[i]);
        } else {
#pragma unroll
            for (int d = 0; d < W8; ++d)
                u[i][d] = 0;
        }
    }
#pragma unroll
    for (int i = 0; i < TR / 16; ++i) {
        const int rl = i * 16 + lr, row = row0 + rl;
        const int x = 16 * ((rl / 32) & 3);
#pragma unroll
        for (int d = 0; d < W8; d += 4)
            *reinterpret_cast<u32x4 *>(tile + rl * WPR + ((lc * W8 + d) ^ x)) =
                u32x4{u[i][d], u[i][d + 1], u[i][d + 2], u[i][d + 3]};
        if constexpr (ROWS) {
            uint32_t am = mx_amax8<T>(u[i]);
            am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0xB1, 0xF, 0xF, false));
            am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x4E, 0xF, 0xF, false));
            const uint32_t b = mx_scale_of(am);
            const uint32_t w = mx_pack8<T>(u[i], b);
            // (a block that starts inside K is stored whole, zeros past K)
            if (row < p.M && (k0 & ~31) < p.K) {
                *reinterpret_cast<uint32_t *>(p.q + (int64_t)row * p.ldq + k0 / 2) = w;
                if ((lc & 3) == 0)
                    p.s[(int64_t)row * p.lds + k0 / 32] = (uint8_t)b;
            }
        }
    }
    __syncthreads();

    constexpr int CPT = 4 / (int)sizeof(T);   // columns per thread and task
    const int g = tid & 3;                    // block of 32 rows
    const int nbm = (p.M + 31) / 32, gb = row0 / 32 + g;
#pragma unroll
    for (int task = 0; task < WPR / 64; ++task) {
        const int c = task * 64 + tid / 4;    // word of the row
        const uint32_t *src = tile + g * 32 * WPR + (c ^ (16 * g));
        uint32_t v[32];
#pragma unroll
        for (int r = 0; r < 32; ++r)
            v[r] = src[r * WPR];
        uint32_t b[CPT], w[CPT][4];
        mx_columns<T>(v, b, w);
#pragma unroll
        for (int e = 0; e < CPT; ++e) {
            const int col = col0 + c * CPT + e;
            // the four blocks' scale bytes, in every lane of the quad
            uint32_t sb = b[e] << (8 * g);
            sb |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sb, 0xB1, 0xF, 0xF, false);
            sb |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sb, 0x4E, 0xF, 0xF, false);
            if (col < p.K && gb < nbm) {
                *reinterpret_cast<u32x4 *>(p.qt + (int64_t)col * p.ldqt + (int64_t)gb * 16) =
                    u32x4{w[e][0], w[e][1], w[e][2], w[e][3]};
                uint8_t *s = p.st + (int64_t)col * p.ldst + gb;
                if (gb - g + 4 <= nbm) {
                    if (g == 0)
                        *reinterpret_cast<uint32_t *>(s) = sb;
                } else {
                    *s = (uint8_t)b[e];
                }
            }
        }
    }
}

// A lane turns 8 codes (one word) into 8 values; threads as for the rows above.
template <typename T, bool VEC, int ROWS>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(MxDequantize p, int tlog, int pieces) {
    const int piece = (int)(blockIdx.y << tlog) + (threadIdx.x & ((1 << tlog) - 1)), k0 = piece * 8;
    const int step = 256 >> tlog, row0 = (int)blockIdx.x * step * ROWS + (threadIdx.x >> tlog);
    if (piece >= pieces)
        return;
    uint32_t w[ROWS], b[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = row0 + i * step;
        w[i] = row < p.M ? *reinterpret_cast<const uint32_t *>(p.q + (int64_t)row * p.ldq + piece * 4) : 0;
        b[i] = row < p.M ? p.s[(int64_t)row * p.lds + piece / 4] : 0;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = row0 + i * step;
        if (row >= p.M)
            return;
        T *y = (T *)p.y + (int64_t)row * p.ldy;
        uint32_t v[MxPack<T>::WORDS8];
        mx_unpack8<T>(w[i], b[i], v);
        if (VEC && k0 + 8 <= p.K) {
#pragma unroll
            for (int d = 0; d < MxPack<T>::WORDS8; d += 4)
                *reinterpret_cast<u32x4 *>((uint32_t *)(y + k0) + d) = u32x4{v[d], v[d + 1], v[d + 2], v[d + 3]};
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d)
                if (k0 + d < p.K) {
                    if constexpr (sizeof(T) == 4)
                        reinterpret_cast<uint32_t *>(y)[k0 + d] = v[d];
                    else
                        reinterpret_cast<uint16_t *>(y)[k0 + d] = (uint16_t)(v[d / 2] >> (16 * (d & 1)));
                }
        }
    }
}

template <typename T>
static hipError_t quantize_type(const MxQuantize &p, hipStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (p.ldx * sizeof(T)) % 16 == 0;
    if (!p.qt) {
        const int pieces = (p.K + 31) / 32 * 4;
        const MxSpread at(p.M, pieces);
        if (vec && at.four)
            hipLaunchKernelGGL((mx_quantize_rows_kernel<T, true, 4>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
        else if (vec)
            hipLaunchKernelGGL((mx_quantize_rows_kernel<T, true, 1>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
        else if (at.four)
            hipLaunchKernelGGL((mx_quantize_rows_kernel<T, false, 4>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
        else
            hipLaunchKernelGGL((mx_quantize_rows_kernel<T, false, 1>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
        return hipGetLastError();
    }
    const int tiles_k = (p.K + 127) / 128;
    const int64_t tiles = (int64_t)((p.M + 127) / 128) * tiles_k;
    if (tiles > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles);
    if (p.q) {
        if (vec)
            hipLaunchKernelGGL((mx_quantize_both_kernel<T, true, true>), grid, dim3(256), 0, stream, p, tiles_k);
        else
            hipLaunchKernelGGL((mx_quantize_both_kernel<T, false, true>), grid, dim3(256), 0, stream, p, tiles_k);
    } else {
        if (vec)
            hipLaunchKernelGGL((mx_quantize_both_kernel<T, true, false>), grid, dim3(256), 0, stream, p, tiles_k);
        else
            hipLaunchKernelGGL((mx_quantize_both_kernel<T, false, false>), grid, dim3(256), 0, stream, p, tiles_k);
    }
    return hipGetLastError();
}

hipError_t launch_mx_quantize(int type, const MxQuantize &p, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return quantize_type<_Float16>(p, stream);
    case MPGEMM_TYPE_BF16: return quantize_type<__bf16>(p, stream);
    default: return quantize_type<float>(p, stream);
    }
}

template <typename T>
static hipError_t dequantize_type(const MxDequantize &p, hipStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(p.y) & 15) == 0 && (p.ldy * sizeof(T)) % 16 == 0;
    const int pieces = (p.K + 7) / 8;
    const MxSpread at(p.M, pieces);
    if (vec && at.four)
        hipLaunchKernelGGL((mx_dequantize_kernel<T, true, 4>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
    else if (vec)
        hipLaunchKernelGGL((mx_dequantize_kernel<T, true, 1>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
    else if (at.four)
        hipLaunchKernelGGL((mx_dequantize_kernel<T, false, 4>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
    else
        hipLaunchKernelGGL((mx_dequantize_kernel<T, false, 1>), at.grid, dim3(256), 0, stream, p, at.tlog, pieces);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(int type, const MxDequantize &p, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return dequantize_type<_Float16>(p, stream);
    case MPGEMM_TYPE_BF16: return dequantize_type<__bf16>(p, stream);
    default: return dequantize_type<float>(p, stream);
    }
}

}  // namespace mpg
