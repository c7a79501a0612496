// mlp_ops_norm.hip -- the root-mean-square norm with the residual's addition, and the rounding to the 8-bit format.
// Both are bound by bytes: each input is read once and each output written once.  A lane holds chunks of 8 elements,
// so 16 neighbouring lanes hold a block of 128, whose largest value they find among themselves.  Measured: the norm of
// 65,536 x 1,024 BF16 with a residual into 8 bits 90 us (472 MB, 5.2 TB/s, what a large copy reaches), without a residual 49
// (201 MB: 72 % of the vector cycles, most of them the rounding's); 65,536 x 1,024 by rows 37 us; 32 matrices of
// 2,048 x 2,048 by blocks 87 us (403 MB, 4.6 TB/s).  Small rows are bound by latencies: each chunk's load is waited for before
// the next one's, a last chunk's elements one by one (5,003 x 1,001 of FP16 6.6 us, x 1,007 8.0).
#include <hip/hip_runtime.h>

#include "mlp_ops_device.h"
#include "mlp_ops_fp8_kernels.h"
#include "mlp_ops_quant.h"

namespace mlpk {

namespace {

// 8 elements as they lie in memory, at any alignment of an element.
template <class T>
struct Chunk {
    u4 v;
};
template <>
struct Chunk<float> {
    Float8 v;
};

template <class T>
__device__ __forceinline__ Chunk<T> load_chunk(const T *row, int col, int width)
{
    Chunk<T> c;
    if constexpr (sizeof(T) == 2) {
        c.v = load16_tail(row, col, width);
    } else {
        if (col + 8 <= width) {
            c.v = *(const Float8 *)(row + col);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                c.v.v[j] = col + j < width ? row[col + j] : 0.0f;
        }
    }
    return c;
}

template <class T>
__device__ __forceinline__ f8 unpack(const Chunk<T> &c)
{
    if constexpr (sizeof(T) == 2)
        return __builtin_convertvector(__builtin_bit_cast(typename Vec8<T>::type, c.v), f8);
    else
        return f8{c.v.v[0], c.v.v[1], c.v.v[2], c.v.v[3], c.v.v[4], c.v.v[5], c.v.v[6], c.v.v[7]};
}

// 8 values rounded to T (nearest even), those inside the row.
template <class T>
__device__ __forceinline__ void store_chunk(T *row, int col, int width, f8 v)
{
    struct __attribute__((packed, aligned(sizeof(T)))) Out8 {
        T v[8];
    };
    if (col + 8 <= width) {
        if constexpr (sizeof(T) == 2) {
            ((Unaligned16 *)(row + col))->v = __builtin_bit_cast(u4, __builtin_convertvector(v, typename Vec8<T>::type));
        } else {
            Out8 o;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o.v[j] = v[j];
            *(Out8 *)(row + col) = o;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (col + j < width)
                row[col + j] = (T)v[j];
    }
}

// 8 values of a block as E4M3 (`block` is the largest of its 16 lanes' values), and its scale by the `first` of them.
__device__ __forceinline__ void store_eight(uint8_t *row, float *scales, int col, int width, f8 v, float block, bool first)
{
    struct __attribute__((packed, aligned(1))) Bytes8 {
        unsigned v[2];
    };
    const float s = scale_of(block), inv = inverse(s);
    if (col >= width)
        return;
    const Bytes8 o = {{to_e4m3x4(v[0], v[1], v[2], v[3], inv), to_e4m3x4(v[4], v[5], v[6], v[7], inv)}};
    if (first)
        scales[col / kFp8Block] = s;
    if (col + 8 <= width) {
        *(Bytes8 *)(row + col) = o;
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (col + j < width)
                row[col + j] = (uint8_t)(o.v[j / 4] >> (8 * (j % 4)));
    }
}

// Sum over LANES neighbouring lanes (16, 32 or 64), or over a workgroup of LANES threads.
template <int LANES>
__device__ __forceinline__ double sum_lanes(double v, double *lds)
{
    constexpr int IN_WAVE = LANES < 64 ? LANES : 64;
#pragma unroll
    for (int d = IN_WAVE / 2; d; d /= 2)
        v += __shfl_xor(v, d);
    if constexpr (LANES > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();  // the sums of the row before have been read
        if ((threadIdx.x & 63) == 0)
            lds[wave] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int i = 1; i < LANES / 64; ++i)
            v += lds[i];
    }
    return v;
}

// LANES lanes take a row, each CH chunks (chunk i * LANES + lane), or with LOOP as many rounds of CH as it needs, the
// second pass reading the row again.  Up to 64 lanes: several rows in a workgroup of 256.
template <class T, int LANES, int CH, bool LOOP>
__global__ __launch_bounds__(LANES <= 256 ? 256 : LANES) void rms_norm(NormArgs p)
{
    constexpr int ROWS = LANES <= 64 ? 256 / LANES : 1;
    __shared__ double lds[LANES > 64 ? LANES / 64 : 1];
    const int lane = LANES <= 64 ? threadIdx.x % LANES : threadIdx.x;
    const bool first = lane % 16 == 0;
    const T *const weight = (const T *)p.weight;
    const int rounds = LOOP ? (p.width + LANES * CH * 8 - 1) / (LANES * CH * 8) : 1;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + (LANES <= 64 ? threadIdx.x / LANES : 0); row < p.rows; row += (int64_t)gridDim.x * ROWS) {
        const T *const x = (const T *)p.x + row * p.ldx;
        const T *const r = p.residual ? (const T *)p.residual + row * p.ldr : nullptr;
        T *const total = p.total ? (T *)p.total + row * p.ldt : nullptr;
        f8 t[CH];
        double sum = 0.0;
        for (int k = 0; k < rounds; ++k) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int col = ((k * CH + i) * LANES + lane) * 8;
                t[i] = (f8)0.0f;
                if (col < p.width) {
                    t[i] = unpack(load_chunk(x, col, p.width));
                    if (r) {
                        t[i] += unpack(load_chunk(r, col, p.width));
                        if constexpr (sizeof(T) == 2)  // the stream's own precision
                            t[i] = __builtin_convertvector(__builtin_convertvector(t[i], typename Vec8<T>::type), f8);
                        if (total)
                            store_chunk(total, col, p.width, t[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum = fma((double)t[i][j], (double)t[i][j], sum);
        }
        sum = sum_lanes<LANES>(sum, lds);
        const float scale = (float)(1.0 / sqrt(sum / p.width + (double)p.eps));
        for (int k = 0; k < rounds; ++k) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int col = ((k * CH + i) * LANES + lane) * 8;
                if (LOOP) {
                    t[i] = (f8)0.0f;
                    if (col < p.width) {
                        if (total) {  // x or the residual may be total itself
                            t[i] = unpack(load_chunk(total, col, p.width));
                        } else {
                            t[i] = unpack(load_chunk(x, col, p.width));
                            if (r) {
                                t[i] += unpack(load_chunk(r, col, p.width));
                                if constexpr (sizeof(T) == 2)
                                    t[i] = __builtin_convertvector(__builtin_convertvector(t[i], typename Vec8<T>::type), f8);
                            }
                        }
                    }
                }
                f8 y = t[i] * scale;
                if (weight && col < p.width)
                    y *= unpack(load_chunk(weight, col, p.width));
                if (p.y && col < p.width) {
                    if (p.y_fp32)
                        store_chunk((float *)p.y + row * p.ldy, col, p.width, y);
                    else
                        store_chunk((T *)p.y + row * p.ldy, col, p.width, y);
                }
                if (p.values)
                    store_eight(p.values + row * p.ldv, p.scales + row * p.lds, col, p.width, y, max16(largest<8>(y)), first);
            }
        }
    }
}

// A scale for each row and 128 columns: 16 lanes take one, a thread U chunks, all requested before the first is used.
template <class T, class INDEX>
__global__ __launch_bounds__(256) void quantize_rows(QuantizeArgs p)
{
    constexpr int U = 4;
    const INDEX blocks = (p.width + kFp8Block - 1) / kFp8Block, rows = (INDEX)(p.used ? min((int64_t)max(*p.used, 0), p.rows) : p.rows);
    const INDEX all = rows * blocks, step = (INDEX)gridDim.x * 16;
    const T *const x = (const T *)p.x + blockIdx.y * p.x_stride;
    uint8_t *const values = p.values + blockIdx.y * p.v_stride;
    float *const scales = p.scales + blockIdx.y * p.s_stride;
    const int lane = threadIdx.x % 16;
    for (INDEX first = (INDEX)blockIdx.x * 16 + threadIdx.x / 16; first < all; first += U * step) {
        Chunk<T> c[U];
        INDEX row[U];
        int col[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const INDEX i = first + u * step < all ? first + u * step : all - 1;
            row[u] = i / blocks;
            col[u] = (int)(i - row[u] * blocks) * kFp8Block + lane * 8;
            if (col[u] < p.width)
                c[u] = load_chunk(x + (int64_t)row[u] * p.ldx, col[u], p.width);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (first + u * step >= all)  // the same for the 16 lanes
                break;
            const f8 v = col[u] < p.width ? unpack(c[u]) : (f8)0.0f;
            store_eight(values + (int64_t)row[u] * p.ldv, scales + (int64_t)row[u] * p.lds, col[u], p.width, v, max16(largest<8>(v)), lane == 0);
        }
    }
}

// A scale for each 128 rows and 128 columns: a workgroup takes one, a thread 8 chunks of rows 16 apart.
template <class T>
__global__ __launch_bounds__(256) void quantize_blocks(QuantizeArgs p)
{
    constexpr int U = kFp8Block / 16;
    __shared__ float part[2][16];
    const unsigned across = (p.width + kFp8Block - 1) / kFp8Block;
    const int64_t down = (p.rows + kFp8Block - 1) / kFp8Block, all = down * across;
    const T *const x = (const T *)p.x + blockIdx.y * p.x_stride;
    uint8_t *const values = p.values + blockIdx.y * p.v_stride;
    float *const scales = p.scales + blockIdx.y * p.s_stride;
    const int lane = threadIdx.x % 16, r = threadIdx.x / 16;
    int turn = 0;
    for (int64_t b = blockIdx.x; b < all; b += gridDim.x, turn ^= 1) {
        const int64_t down_at = b / across, row0 = down_at * kFp8Block;
        const int col = (int)(b - down_at * across) * kFp8Block + lane * 8;
        Chunk<T> c[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row0 + 16 * u + r < p.rows && col < p.width)
                c[u] = load_chunk(x + (row0 + 16 * u + r) * p.ldx, col, p.width);
        float m = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row0 + 16 * u + r < p.rows && col < p.width)
                m = fmaxf(m, largest<8>(unpack(c[u])));
        m = max16(m);
        if (lane == 0)
            part[turn][r] = m;
        __syncthreads();  // the other half of `part` is written next, so one barrier a block is enough
        m = max16(part[turn][lane]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row0 + 16 * u + r < p.rows)
                store_eight(values + (row0 + 16 * u + r) * p.ldv, scales + down_at * p.lds, col, p.width,
                            col < p.width ? unpack(c[u]) : (f8)0.0f, m, lane == 0 && r == 0 && u == 0);
    }
}

// ---- which kernel ---------------------------------------------------------------------------------

// Lanes and chunks for a row: one chunk a lane where that fills the lanes, and registers few enough that a CU holds several
// workgroups, of which some wait for memory while others compute.  us, BF16 into 8 bits (and with a residual into both):
//   65,536 x 1,024   64x2 49 (112)      256x1 82 (117): below 1,024 rows, where only latency counts, 256x1
//   32,768 x 2,048   256x1 52 (107)     64x4 55 (120), 256x2 67 (109)
//   32,768 x 4,096   256x2 99 (221)     512x1 107 (217), 256x4 180 (249)
//   8,192 x 8,192    512x2 57 (110)     256x4 76 (125), 1024x1 76 (110)
//   4,096 x 16,384   512x2 twice 59 (127)   1024x2 78 (124), 512x4 97 (144): the second reading comes from the caches
//   4,096 x 32,768   512x2 twice 118 (260)  1024x2 twice 144 (254), 1024x4 211 (288, registers spilled)
//   1,024 x 65,536   1024x4 twice 66 to 69 (145)  512x4 twice 68 (173)
struct NormForm {
    int lanes, chunks;
    bool loop;
};
constexpr NormForm kNormForms[] = {{16, 1, false}, {64, 1, false}, {64, 2, false}, {256, 1, false},
                                   {256, 2, false}, {512, 2, false}, {512, 2, true}, {1024, 4, true}};

int choose_norm(const NormArgs &p)
{
    if (p.width <= 128)
        return 0;
    if (p.rows >= 1024 && p.width <= 1024)
        return p.width <= 512 ? 1 : 2;
    return p.width <= 2048 ? 3 : p.width <= 4096 ? 4 : p.width <= 8192 ? 5 : p.width <= 32768 ? 6 : 7;
}

template <class T>
hipError_t launch_norm_typed(const NormArgs &p, hipStream_t stream)
{
    const int form = choose_norm(p);
    const NormForm f = kNormForms[form];
    const int rows = f.lanes <= 64 ? 256 / f.lanes : 1, threads = f.lanes <= 256 ? 256 : f.lanes;
    const int64_t blocks = (p.rows + rows - 1) / rows, most = 256 * 64;
    const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(threads);
    switch (form) {
    case 0: hipLaunchKernelGGL((rms_norm<T, 16, 1, false>), grid, block, 0, stream, p); break;
    case 1: hipLaunchKernelGGL((rms_norm<T, 64, 1, false>), grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL((rms_norm<T, 64, 2, false>), grid, block, 0, stream, p); break;
    case 3: hipLaunchKernelGGL((rms_norm<T, 256, 1, false>), grid, block, 0, stream, p); break;
    case 4: hipLaunchKernelGGL((rms_norm<T, 256, 2, false>), grid, block, 0, stream, p); break;
    case 5: hipLaunchKernelGGL((rms_norm<T, 512, 2, false>), grid, block, 0, stream, p); break;
    case 6: hipLaunchKernelGGL((rms_norm<T, 512, 2, true>), grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL((rms_norm<T, 1024, 4, true>), grid, block, 0, stream, p); break;
    }
    return hipGetLastError();
}

template <class T>
hipError_t launch_quantize_typed(const QuantizeArgs &q, int block_rows, hipStream_t stream)
{
    const int64_t across = (q.width + kFp8Block - 1) / kFp8Block;
    if (block_rows == 1) {
        const int64_t all = q.rows * across, blocks = (all + 63) / 64, most = 256 * 32;  // 16 blocks of 128, four times
        const dim3 grid((unsigned)(blocks < most ? blocks : most), (unsigned)q.count);
        if (all < (int64_t)1 << 30)  // and so are the last steps past it
            hipLaunchKernelGGL((quantize_rows<T, unsigned>), grid, dim3(256), 0, stream, q);
        else
            hipLaunchKernelGGL((quantize_rows<T, int64_t>), grid, dim3(256), 0, stream, q);
    } else {
        const int64_t all = (q.rows + kFp8Block - 1) / kFp8Block * across, most = 256 * 32;
        hipLaunchKernelGGL((quantize_blocks<T>), dim3((unsigned)(all < most ? all : most), (unsigned)q.count), dim3(256), 0, stream, q);
    }
    return hipGetLastError();
}

}  // namespace

const char *norm_kernel(const NormArgs &p, int)
{
    static const char *const names[] = {"16x1", "64x1", "64x2", "256x1", "256x2", "512x2", "512x2 twice", "1024x4 twice"};
    return names[choose_norm(p)];
}

hipError_t launch_norm(const NormArgs &p, int dtype, hipStream_t stream)
{
    return dtype == kFp16 ? launch_norm_typed<_Float16>(p, stream)
           : dtype == kBf16 ? launch_norm_typed<__bf16>(p, stream)
                            : launch_norm_typed<float>(p, stream);
}

hipError_t launch_quantize(const QuantizeArgs &q, int dtype, int block_rows, hipStream_t stream)
{
    return dtype == kFp16 ? launch_quantize_typed<_Float16>(q, block_rows, stream)
           : dtype == kBf16 ? launch_quantize_typed<__bf16>(q, block_rows, stream)
                            : launch_quantize_typed<float>(q, block_rows, stream);
}

}  // namespace mlpk
