// The linear layer in 8-bit integers: Y = (A B^T) sa sb + bias with a scale for
// each token and each output channel; its quantiser and planning.
//
// The integer sums are exact; scales and bias are applied in fp32 and the
// result is rounded once. Tiles: 16x16x64 integer matrix instructions on the
// main loop of phase_tile.h; few rows: one pass over the weight (linear_device.h).
#include "linear_device.h"

namespace mpg {

// ------------------------------------------------------------------ quantisation

// One row per workgroup of 64 W threads (W = 1: four rows of one wavefront each): every thread keeps
// P pieces of 8 elements, 64 W P 8 in all, and the row is read once. P = 0: longer rows, read
// twice. Bound by memory, the reads of a row on their way together: 10240 x 4096 bf16 in 30 us (4.2 TB/s), and by
// one read, join and write behind one another where there are few rows (16 x 8192 4.1, 64 x 4096 3.2).
template <typename T, int W, int P>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void i8_quantize_kernel(I8Quantize p) {
    constexpr int NT = 64 * W;
    const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x, lane = threadIdx.x & 63;
    const int row = W == 1 ? blockIdx.x * 4 + threadIdx.x / 64 : blockIdx.x;
    if (W == 1 && row >= p.M)
        return;
    const T *x = static_cast<const T *>(p.x) + (int64_t)row * p.ldx;
    int8_t *qr = p.q + (int64_t)row * p.ldq;
    const bool vec = p.K % 8 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (p.ldx * (int64_t)sizeof(T)) % 16 == 0;
    const bool qvec = (reinterpret_cast<uintptr_t>(p.q) & 7) == 0 && p.ldq % 8 == 0;
    const int end = p.pad ? (p.K + 15) / 16 * 16 : p.K;
    float v[P > 0 ? P : 1][8];
    uint32_t m = 0;
    if constexpr (P > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            i8_load8<T>(x, (i * NT + t) * 8, p.K, vec, v[i]);
#pragma unroll
        for (int i = 0; i < P; ++i)
            m = max(m, i8_amax8(v[i]));
    } else {
        for (int k0 = t * 8; k0 < p.K; k0 += NT * 8) {
            i8_load8<T>(x, k0, p.K, vec, v[0]);
            m = max(m, i8_amax8(v[0]));
        }
    }
    m = lin_wave_max(m);
    if constexpr (W > 1) {
        __shared__ uint32_t top[W];
        if (lane == 0)
            top[threadIdx.x / 64] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w)
            m = max(m, top[w]);
    }
    const I8Row r = i8_row(m);
    if (t == 0)
        p.s[row] = r.scale;
    auto put = [&](int k0, const float (&e)[8]) {
        if (k0 >= end)
            return;
        const uint2 c = i8_codes8(e, r);
        if (qvec && k0 + 8 <= end) {
            *reinterpret_cast<uint2 *>(qr + k0) = c;
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d)
                if (k0 + d < end)
                    qr[k0 + d] = (int8_t)((d < 4 ? c.x : c.y) >> (8 * (d % 4)));
        }
    };
    if constexpr (P > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            put((i * NT + t) * 8, v[i]);
    } else {
        for (int k0 = t * 8; k0 < end; k0 += NT * 8) {
            i8_load8<T>(x, k0, p.K, vec, v[0]);
            put(k0, v[0]);
        }
    }
}

template <typename T>
static void quantize_type(const I8Quantize &p, hipStream_t stream) {
    const int K = p.K;
    const dim3 rows((unsigned)p.M), fours((unsigned)((p.M + 3) / 4)), nt(256);
    if (K <= 512)
        hipLaunchKernelGGL((i8_quantize_kernel<T, 1, 1>), fours, nt, 0, stream, p);
    else if (K <= 2048)
        hipLaunchKernelGGL((i8_quantize_kernel<T, 4, 1>), rows, nt, 0, stream, p);
    else if (K <= 4096)
        hipLaunchKernelGGL((i8_quantize_kernel<T, 8, 1>), rows, dim3(512), 0, stream, p);
    else if (K <= 8192)
        hipLaunchKernelGGL((i8_quantize_kernel<T, 16, 1>), rows, dim3(1024), 0, stream, p);
    else
        hipLaunchKernelGGL((i8_quantize_kernel<T, 16, 0>), rows, dim3(1024), 0, stream, p);
}

// A launch has fewer than 2^32 threads: more rows than this take several.
constexpr int LIN_ROWS_AT_ONCE = 1 << 21;

hipError_t launch_i8_quantize(int type, const I8Quantize &all, hipStream_t stream) {
    for (int64_t row = 0; row < all.M; row += LIN_ROWS_AT_ONCE) {
        I8Quantize p = all;
        p.x = static_cast<const uint8_t *>(all.x) + row * all.ldx * (type == MPGEMM_TYPE_F32 ? 4 : 2);
        p.q = all.q + row * all.ldq;
        p.s = all.s + row;
        p.M = (int)(all.M - row < LIN_ROWS_AT_ONCE ? all.M - row : LIN_ROWS_AT_ONCE);
        switch (type) {
        case MPGEMM_TYPE_F16: quantize_type<_Float16>(p, stream); break;
        case MPGEMM_TYPE_BF16: quantize_type<__bf16>(p, stream); break;
        default: quantize_type<float>(p, stream); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// 8 elements per thread, 2^LX threads per row piece and the rest of the workgroup's 256 over rows. Bound by
// memory: 10240 x 4096 to bf16 in 20 us (6.2 TB/s, the codes from the last level of cache).
template <typename T, int LX>
__global__ __launch_bounds__(256) void i8_dequantize_kernel(I8Dequantize p, int per_row) {
    const int parts = (per_row + (1 << LX) - 1) >> LX;
    const int rb = blockIdx.x / parts, part = blockIdx.x - rb * parts;
    const int row = rb * (256 >> LX) + (threadIdx.x >> LX), k0 = ((part << LX) + (threadIdx.x & ((1 << LX) - 1))) * 8;
    if (row >= p.M || k0 >= p.K)
        return;
    const int8_t *q = p.q + (int64_t)row * p.ldq + k0;
    T *y = static_cast<T *>(p.y) + (int64_t)row * p.ldy + k0;
    const float s = p.s[row];
    const bool vec = k0 + 8 <= p.K && (reinterpret_cast<uintptr_t>(p.q) & 7) == 0 && p.ldq % 8 == 0 && lin_vec<T>(p.y, p.ldy);
    if (vec) {
        const uint2 w = *reinterpret_cast<const uint2 *>(q);
        typedef T eight __attribute__((ext_vector_type(8)));
        eight e;
#pragma unroll
        for (int d = 0; d < 8; ++d)
            e[d] = (T)((float)(int8_t)((d < 4 ? w.x : w.y) >> (8 * (d % 4))) * s);
        *reinterpret_cast<eight *>(y) = e;
    } else {
#pragma unroll
        for (int d = 0; d < 8; ++d)
            if (k0 + d < p.K)
                y[d] = (T)((float)q[d] * s);
    }
}

template <typename T, int LX>
static void dequantize_one(const I8Dequantize &p, hipStream_t stream) {
    const int per_row = (p.K + 7) / 8, rows = 256 >> LX;
    const int64_t blocks = (int64_t)((p.M + rows - 1) / rows) * ((per_row + (1 << LX) - 1) >> LX);
    hipLaunchKernelGGL((i8_dequantize_kernel<T, LX>), dim3((unsigned)blocks), dim3(256), 0, stream, p, per_row);
}

template <typename T>
static void dequantize_type(const I8Dequantize &p, hipStream_t stream) {
    if (p.K <= 256)
        dequantize_one<T, 5>(p, stream);
    else
        dequantize_one<T, 8>(p, stream);
}

hipError_t launch_i8_dequantize(int type, const I8Dequantize &all, hipStream_t stream) {
    const int64_t parts = (all.K + 2047) / 2048, step = (LIN_ROWS_AT_ONCE + parts - 1) / parts;
    for (int64_t row = 0; row < all.M; row += step) {
        I8Dequantize p = all;
        p.q = all.q + row * all.ldq;
        p.s = all.s + row;
        p.y = static_cast<uint8_t *>(all.y) + row * all.ldy * (type == MPGEMM_TYPE_F32 ? 4 : 2);
        p.M = (int)(all.M - row < step ? all.M - row : step);
        switch (type) {
        case MPGEMM_TYPE_F16: dequantize_type<_Float16>(p, stream); break;
        case MPGEMM_TYPE_BF16: dequantize_type<__bf16>(p, stream); break;
        default: dequantize_type<float>(p, stream); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// ------------------------------------------------------------------ copies and fills

// Matrix blockIdx.y's rows, 16 bytes per thread, into rows at multiples of 16 bytes with zeros behind.
__global__ __launch_bounds__(256) void lin_copy_kernel(LinCopy p) {
    const int w = blockIdx.y, bytes = p.row_bytes[w], chunks = (bytes + 15) / 16;
    const int64_t total = (int64_t)p.rows[w] * chunks;
    for (int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x; f < total; f += (int64_t)gridDim.x * 256) {
        const int row = (int)(f / chunks), c = (int)(f - (int64_t)row * chunks);
        const uint8_t *s = p.from[w] + (int64_t)row * p.ldf[w] + 16 * c;
        *reinterpret_cast<pt_u32x4 *>(p.to[w] + (int64_t)row * p.ldt[w] + 16 * c) = lin_load16_part<uint8_t>(s, bytes - 16 * c);
    }
}

hipError_t launch_lin_copy(const LinCopy &p, hipStream_t stream) {
    int64_t most = 1;
    int n = 0;
    for (int w = 0; w < 3; ++w)
        if (p.to[w]) {
            const int64_t b = ((int64_t)p.rows[w] * ((p.row_bytes[w] + 15) / 16) + 255) / 256;
            most = b > most ? b : most;
            n = w + 1;
        }
    hipLaunchKernelGGL(lin_copy_kernel, dim3((unsigned)(most < 4096 ? most : 4096), n), dim3(256), 0, stream, p);
    return hipGetLastError();
}

// C (M x N, row stride ldc), each row a copy of `row`, or zeros: results of empty sums.
template <typename T>
__global__ __launch_bounds__(256) void lin_fill_kernel(T *c, int64_t ldc, int M, int N, const T *row) {
    const int64_t total = (int64_t)M * N;
    for (int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x; f < total; f += (int64_t)gridDim.x * 256) {
        const int m = (int)(f / N), n = (int)(f - (int64_t)m * N);
        c[(int64_t)m * ldc + n] = row ? row[n] : T(0);
    }
}

hipError_t launch_lin_fill(int type, void *c, int64_t ldc, int M, int N, const void *row, hipStream_t stream) {
    const int64_t blocks = ((int64_t)M * N + 255) / 256;
    const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
    if (type == MPGEMM_TYPE_F32)
        hipLaunchKernelGGL((lin_fill_kernel<uint32_t>), grid, dim3(256), 0, stream, static_cast<uint32_t *>(c), ldc, M, N,
                           static_cast<const uint32_t *>(row));
    else
        hipLaunchKernelGGL((lin_fill_kernel<uint16_t>), grid, dim3(256), 0, stream, static_cast<uint16_t *>(c), ldc, M, N,
                           static_cast<const uint16_t *>(row));
    return hipGetLastError();
}

// ------------------------------------------------------------------ plan

// Tiles, what one takes of a CU's time, in us, apart from its stages and for a stage (128 bytes of k), and how many
// are on a CU at once (LDS). Measured, with 2.5 us of a launch: 5 rounds of 64 stages in tiles of 256 491 us (gated 4096 x 10240 x
// 4096), 2 of 16 47.7; 4.3 of 16 in tiles of 128 38.3 (gated 1920 x 4736 x 1024), one of 32 18.6; 17 of 6 in tiles of 64 35.9 (gated
// 1088 x 8192 x 384), one of 32 10.9. The last, of the forward products only, is between the two small ones: integers 200 x
// 8192 x 8192 in one round 27.4 us, in two of 64 x 64 32.5, in one of 128 x 128 39.8; 333 x 5000 x 2112 11.8, 12.7 and 14.0.
// Up to 128 x 128 a stage takes its bytes at about 70 a ns on their way into the CU, whatever the number of stages ahead.
struct LinCfg { int BM, BN; double tile, stage; int at_once; };
static const LinCfg kLinCfg[] = {{256, 256, 6.0, 1.25, 1}, {128, 128, 1.4, 0.46, 2}, {64, 64, 1.0, 0.2, 2}, {64, 128, 2.6, 0.34, 1}};

static int64_t lin_tiles(int mode, int c, int64_t M, int64_t N) {
    const int64_t cn = mode == LIN_GATED ? kLinCfg[c].BN / 2 : kLinCfg[c].BN;
    return ((M + kLinCfg[c].BM - 1) / kLinCfg[c].BM) * ((N + cn - 1) / cn);
}

static double lin_tile_us(int c, int64_t stages) { return kLinCfg[c].tile + kLinCfg[c].stage * (double)stages; }

template <typename F>
static int lin_cheapest(int cfgs, F us) {
    int cfg = 0;
    for (int c = 1; c < cfgs; ++c)
        if (us(c) < us(cfg))
            cfg = c;
    return cfg;
}

// Up to 32 rows the skinny kernel, whose workgroups each read all the activations; then tiles.
// Skinny and tiles of 64, us: integers 32 x 4096 x 4096 8.7 and 10.2, 64 x 4096 x 4096 12.2 and 10.5, 64 x 8192 x 8192 27.8
// and 22.7, 16 x 8192 x 8192 16.8 and 19.4; gated 16 x 4096 x 4096 14.6 and 18.5, 64 x 4096 x 4096 25.9 and 21.0.
LinPlan plan_lin(int mode, int64_t M, int64_t N, int64_t K, int elem_bytes, int cu_count) {
    LinPlan pl = {LINK_TILE, 0, cu_count};
    if (K == 0) {
        pl.kind = LINK_EMPTY;
        return pl;
    }
    if (M <= 32 && (mode == LIN_SCALED || mode == LIN_GATED)) {
        pl.kind = LINK_SKINNY;
        pl.cfg = M <= 16 ? 1 : 2;
        return pl;
    }
    const int64_t stages = (K * elem_bytes + 127) / 128;
    pl.cfg = lin_cheapest(mode == LIN_SCALED || mode == LIN_GATED ? 4 : 3, [&](int c) {
        // rounds over the CUs, of two tiles at once in halves
        const int64_t n = kLinCfg[c].at_once, rounds = (n * lin_tiles(mode, c, M, N) + cu_count - 1) / cu_count;
        return lin_tile_us(c, stages) * (rounds > n ? (double)rounds / (double)n : 1.0);
    });
    return pl;
}

// Both products of the backward pass in one grid, M x K over 2 part and (one weight's gradient or both) parts part x K over M:
// the work spread over the CUs, or the longest tile.
LinPlan plan_lin_pair(int64_t M, int64_t part, int parts, int64_t K, int cu_count) {
    return {LINK_TILE, lin_cheapest(3, [&](int c) {
                const double x = lin_tile_us(c, 2 * part / 64), w = lin_tile_us(c, (M + 63) / 64);
                const double all = (x * (double)lin_tiles(LIN_DX, c, M, K) + w * (double)lin_tiles(LIN_DW, c, parts * part, K)) / cu_count;
                return all > x ? (all > w ? all : w) : (x > w ? x : w);
            }), cu_count};
}

// Few activations: every workgroup of the product quantises all of them. In wavefront loads of 512 of a row, up to 16, of one
// or two rows up to 32. In the product and by a launch before it, us: 1 x 4096 x 4096 6.1 and 8.2, 1 x 8192 x 16384 29.7 and
// 37.3, 2 x 8192 x 8192 15.5 and 18.9, 2 x 4096 x 8192 11.9 and 11.0 (the rule has no N: it takes the slower side there), 4 x 4096 x
// 2048 5.8 and 7.0, 8 x 4096 x 1024 5.2 and 5.5; 4 x 8192 x 4096 12.8 and 11.2, 8 x 8192 x 2048 10.9 and 8.6, 16 x 4096 x 1024 7.3 and 5.8.
bool lin_fuses(const LinPlan &plan, int64_t M, int64_t K) {
    return plan.kind == LINK_SKINNY && M <= 16 && M * ((K + 511) / 512) <= (M <= 2 ? LIN_X_MAX : LIN_X_MAX / 2);
}

// ------------------------------------------------------------------ product

hipError_t launch_w8a8(int type, const Lin &p, const LinPlan &plan, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return lin_run<PtI8, _Float16, LIN_SCALED>(p, plan, stream);
    case MPGEMM_TYPE_BF16: return lin_run<PtI8, __bf16, LIN_SCALED>(p, plan, stream);
    default: return lin_run<PtI8, float, LIN_SCALED>(p, plan, stream);
    }
}

hipError_t launch_w8a8_x(int type, const Lin &p, const LinX &x, const LinPlan &plan, hipStream_t stream) {
    switch (type) {
    case MPGEMM_TYPE_F16: return lin_run_x<_Float16, LIN_SCALED>(p, x, plan, stream);
    case MPGEMM_TYPE_BF16: return lin_run_x<__bf16, LIN_SCALED>(p, x, plan, stream);
    default: return lin_run_x<float, LIN_SCALED>(p, x, plan, stream);
    }
}

}  // namespace mpg
