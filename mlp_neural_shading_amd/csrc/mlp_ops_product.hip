// mlp_ops_product.hip -- one affine layer with its epilogue, dense or over the rows routed to experts:
//   y[r][o] = round(act(sum_i x[r][i] w[o][i] + b[o]) + residual[r][o])
// and gated, act(z[o]) * z[out + o] of a w with twice the rows.  x and w are row-major, so both
// operands run along K and are staged alike.
#include <hip/hip_runtime.h>

#include "mlp_ops_kernels.h"

namespace mlpk {

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f8 __attribute__((ext_vector_type(8)));
typedef float f16x __attribute__((ext_vector_type(16)));
typedef unsigned int u4 __attribute__((ext_vector_type(4)));

constexpr float kSlope = 0.01000213623046875f;  // half(0.01)

template <class T>
struct Vec8;
template <>
struct Vec8<_Float16> {
    typedef h8 type;
};
template <>
struct Vec8<__bf16> {
    typedef b8 type;
};

__device__ __forceinline__ f16x mfma32(h8 a, h8 b, f16x c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f16x mfma32(b8 a, b8 b, f16x c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }

// The epilogue's activation, FP32 to FP32.  NaN stays NaN.
__device__ __forceinline__ float activate(float v, int act)
{
    switch (act) {
    case 1:
        return v < 0.0f ? v * kSlope : v;
    case 2:
        return v < 0.0f ? 0.0f : v;
    case 3:
        return 0.5f * v * (1.0f + erff(v * 0.70710678118654752440f));
    case 4:
        return v / (1.0f + __expf(-v));
    default:
        return v;
    }
}

// 16 bytes from an address aligned to an element only (the hardware takes any alignment).
struct __attribute__((packed, aligned(2))) Unaligned16 {
    u4 v;
};
template <bool A16, class T>
__device__ __forceinline__ u4 load16(const T *p)
{
    if constexpr (A16)
        return *(const u4 *)p;
    else
        return ((const Unaligned16 *)p)->v;
}

// The 8 columns from `col` of a row of `width`, zero past its end; reads no byte past it.
template <bool A16, class T>
__device__ __forceinline__ u4 load16_tail(const T *row, int col, int width)
{
    if (col + 8 <= width)
        return load16<A16>(row + col);
    typename Vec8<T>::type v = (typename Vec8<T>::type)(T)0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (col + j < width)
            v[j] = row[col + j];
    return __builtin_bit_cast(u4, v);
}

// Which tile of rows a workgroup of a grouped product takes.  Expert e's rows are the slots
// [offsets[e], offsets[e + 1]); its tiles of BN rows follow those of expert e - 1.  The counts are on the
// device only, so the grid covers the most tiles there can be (rows / BN + experts) and a workgroup finds
// its own by a scan over the experts, 64 at a time, one per lane.  Offsets are clamped to [0, rows].
struct RowTile {
    int expert;
    int row0, row1;  // slots of this tile: [row0, row1)
};

__device__ __forceinline__ int tiles_of(const int32_t *offsets, int experts, int rows, int bn, int e, int &begin, int &end)
{
    begin = end = 0;
    if (e >= experts)
        return 0;
    begin = min(max(offsets[e], 0), rows);
    end = min(max(offsets[e + 1], 0), rows);
    return end > begin ? (end - begin - 1) / bn + 1 : 0;
}

__device__ __forceinline__ int total_tiles(const int32_t *offsets, int experts, int rows, int bn)
{
    int sum = 0, b, e;
    for (int base = 0; base < experts; base += 64)
        sum += tiles_of(offsets, experts, rows, bn, base + (threadIdx.x & 63), b, e);
#pragma unroll
    for (int d = 32; d; d >>= 1)
        sum += __shfl_xor(sum, d);
    return __builtin_amdgcn_readfirstlane(sum);
}

__device__ __forceinline__ bool find_tile(const int32_t *offsets, int experts, int rows, int bn, int tile, RowTile &out)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base < experts; base += 64) {
        int begin, end;
        const int count = tiles_of(offsets, experts, rows, bn, base + lane, begin, end);
        int upto = count;  // inclusive scan
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d);
            upto += lane >= d ? v : 0;
        }
        const int mine = tile - before - (upto - count);  // this tile within the lane's expert
        const unsigned long long hit = __ballot(mine >= 0 && mine < count);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int r0 = begin + mine * bn;  // valid in lane src
            out.expert = base + src;
            out.row0 = __builtin_amdgcn_readfirstlane(__shfl(r0, src));
            out.row1 = min(out.row0 + bn, __builtin_amdgcn_readfirstlane(__shfl(end, src)));
            return true;
        }
        before += __builtin_amdgcn_readfirstlane(__shfl(upto, 63));
    }
    return false;
}

// Tile t of n for workgroup b: XCD x = b % 8 takes the x-th contiguous run, so workgroups that share rows
// or weights share that XCD's L2.  -1: none.
__device__ __forceinline__ int64_t xcd_tile(unsigned b, int64_t n)
{
    const int64_t per = (n + 7) / 8, t = (int64_t)(b % 8) * per + b / 8;
    return b / 8 < per && t < n ? t : -1;
}

constexpr int BK = 64;  // K per stage: 128 bytes of every row

// WM x WN waves, each MT x NT MFMA tiles of 32 weight rows x 32 rows.  LDS holds two stages of both
// operands, 128 bytes a row; chunk c (16 bytes) of row r sits at r * 128 + 16 (c ^ ((r / 2) % 8)), so the
// 16 rows that one 256-byte LDS cycle of a fragment read serves fall in 16 different slots.
// A gated layer's tile takes 32 gate rows, the 32 rows they gate, and so on: tile rows
// 64 i .. 64 i + 31 are gates and 64 i + 32 .. 64 i + 63 their partners, so a lane holds both.
template <class T, class OUT, bool GROUPED, bool GATED, bool A16, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(64 * WM *WN) void product_tile(ProductArgs p)
{
    typedef typename Vec8<T>::type V8;
    constexpr int TH = 64 * WM * WN, BM = 32 * WM * MT, BN = 32 * WN * NT;
    constexpr int BO = GATED ? BM / 2 : BM;       // outputs per tile
    constexpr int OW = GATED ? MT * 16 : MT * 32;  // outputs per wave
    constexpr int CA = BM * 8 / TH, CB = BN * 8 / TH;  // 16-byte chunks per thread and stage
    constexpr int A_ST = BM * 128, STAGE = (BM + BN) * 128;
    static_assert(CA * TH == BM * 8 && CB * TH == BN * 8 && (TH / 8) % 16 == 0, "whole chunks per thread, one swizzle per thread");
    static_assert(!GATED || MT % 2 == 0, "gate and partner tiles in one wave");
    static_assert(WM * WN * 32 * OW * 4 <= 2 * STAGE, "the epilogue's FP32 rows fit the stages");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];

    const int n_out = (p.out + BO - 1) / BO;
    int64_t row0, row1;
    int ot;
    const T *w = (const T *)p.w;
    const T *bias = (const T *)p.bias;
    if constexpr (GROUPED) {
        const int64_t t = xcd_tile(blockIdx.x, (int64_t)total_tiles(p.offsets, p.experts, (int)p.rows, BN) * n_out);
        RowTile rt;
        if (t < 0 || !find_tile(p.offsets, p.experts, (int)p.rows, BN, (int)(t / n_out), rt))
            return;  // whole workgroup, before any barrier
        ot = (int)(t % n_out);
        row0 = rt.row0;
        row1 = rt.row1;
        w += rt.expert * p.w_stride;
        if (bias)
            bias += (int64_t)rt.expert * p.out * (GATED ? 2 : 1);
    } else {
        const int64_t t = xcd_tile(blockIdx.x, (p.rows + BN - 1) / BN * n_out);
        if (t < 0)
            return;
        ot = (int)(t % n_out);
        row0 = t / n_out * BN;
        row1 = row0 + BN < p.rows ? row0 + BN : p.rows;
    }
    const int o0 = ot * BO;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave % WM, wn = wave / WM;
    const int g = lane >> 5, n = lane & 31;

    // The rows this thread stages: chunk c = tid % 8 of tile rows tid / 8 + i * TH / 8.  Rows past the end
    // repeat the last one; what they give is never stored.
    const int c = tid & 7;
    const T *wp[CA], *xp[CB];
#pragma unroll
    for (int i = 0; i < CA; ++i) {
        const int r = (tid >> 3) + i * (TH / 8);
        int o = GATED ? o0 + (r >> 6) * 32 + (r & 31) : o0 + r;
        o = o < p.out ? o : p.out - 1;
        if (GATED && (r & 32))
            o += p.out;
        wp[i] = w + (int64_t)o * p.ldw + 8 * c;
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
        int64_t r = row0 + (tid >> 3) + i * (TH / 8);
        r = r < row1 ? r : row1 - 1;
        if (GROUPED && p.slots) {
            const int a = min(max(p.slots[r], 0), (int)p.rows - 1);
            r = a / p.k;
        }
        xp[i] = (const T *)p.x + r * p.ldx + 8 * c;
    }
    const int st = (tid >> 3) * 128 + 16 * (c ^ ((tid >> 4) & 7));

    // Bias: lane (g, n) of MFMA tile (mt, nt) holds tile rows 32 mt + 8 q + 4 g + i (i = 0 .. 3) of row n.
    f16x acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        f16x b = (f16x)0.0f;
        if (bias) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int r = (wm * MT + mt) * 32 + 8 * (j >> 2) + 4 * g + (j & 3);
                const int o = GATED ? o0 + (r >> 6) * 32 + (r & 31) : o0 + r;
                if (o < p.out)
                    b[j] = (float)bias[o + (GATED && (r & 32) ? p.out : 0)];
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = b;
    }

    u4 ra[CA], rb[CB];
    const int full = p.in / BK;  // stages without a tail
    const int steps = (p.in + BK - 1) / BK;
    auto load = [&](int s) {
#pragma unroll
        for (int i = 0; i < CA; ++i)
            ra[i] = load16<A16>(wp[i] + s * BK);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            rb[i] = load16<A16>(xp[i] + s * BK);
    };
    auto load_tail = [&]() {
#pragma unroll
        for (int i = 0; i < CA; ++i)
            ra[i] = load16_tail<A16>(wp[i] - 8 * c, full * BK + 8 * c, p.in);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            rb[i] = load16_tail<A16>(xp[i] - 8 * c, full * BK + 8 * c, p.in);
    };
    auto store = [&](int s) {
        uint8_t *d = lds + (s & 1) * STAGE + st;
#pragma unroll
        for (int i = 0; i < CA; ++i)
            *(u4 *)(d + i * (TH / 8) * 128) = ra[i];
#pragma unroll
        for (int i = 0; i < CB; ++i)
            *(u4 *)(d + A_ST + i * (TH / 8) * 128) = rb[i];
    };
    const int a_rd = (wm * MT * 32 + n) * 128, b_rd = A_ST + (wn * NT * 32 + n) * 128, swz = (n >> 1) & 7;
    auto multiply = [&](int s) {
        const uint8_t *d = lds + (s & 1) * STAGE;
#pragma unroll
        for (int kb = 0; kb < BK / 16; ++kb) {
            const int ch = 16 * ((2 * kb + g) ^ swz);
            V8 a[MT], b[NT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                a[mt] = *(const V8 *)(d + a_rd + mt * 32 * 128 + ch);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                b[nt] = *(const V8 *)(d + b_rd + nt * 32 * 128 + ch);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    acc[mt][nt] = mfma32(a[mt], b[nt], acc[mt][nt]);
        }
    };
    if (full)
        load(0);
    else
        load_tail();
    store(0);
    __syncthreads();
    int s = 0;
    for (; s + 1 < full; ++s) {
        load(s + 1);
        multiply(s);
        store(s + 1);
        __syncthreads();
    }
    if (s + 1 < steps) {  // a partial last stage
        load_tail();
        multiply(s);
        store(s + 1);
        __syncthreads();
        ++s;
    }
    multiply(s);
    __syncthreads();

    // Epilogue, 32 rows of the wave at a time through its own LDS region (no barrier: one wave writes and
    // reads it): lane (g, n) writes its outputs of row n in FP32, 4 at a time (chunk k of row n at
    // n * OW * 4 + 16 (k ^ (n % NCH))), then the lanes read whole rows back, 8 outputs each, add the residual, round and
    // store 16 (FP32: 32) bytes.
    constexpr int NCH = OW / 4, LPR = OW / 8, RPI = 64 / LPR;  // chunks per row; lanes per row; rows per instruction
    uint8_t *ob = lds + wave * (32 * OW * 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; mt += GATED ? 2 : 1)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = activate(acc[mt][nt][4 * q + i], p.act);
                    if constexpr (GATED)
                        v[i] *= acc[mt + 1][nt][4 * q + i];
                }
                const int k = (GATED ? mt / 2 : mt) * 8 + 2 * q + g;
                *(f4 *)(ob + n * (OW * 4) + 16 * (k ^ (n & (NCH - 1)))) = v;
            }
        const int o = o0 + wm * OW + 8 * (lane % LPR);
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {
            const int rl = i * RPI + lane / LPR;
            const int64_t row = row0 + (wn * NT + nt) * 32 + rl;
            const int k = 2 * (lane % LPR);
            const f4 lo = *(const f4 *)(ob + rl * (OW * 4) + 16 * (k ^ (rl & (NCH - 1))));
            const f4 hi = *(const f4 *)(ob + rl * (OW * 4) + 16 * ((k + 1) ^ (rl & (NCH - 1))));
            if (row >= row1 || o >= p.out)
                continue;
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = lo[j];
                v[4 + j] = hi[j];
            }
            OUT *y = (OUT *)p.y + row * p.ldy + o;
            const OUT *res = p.residual ? (const OUT *)p.residual + row * p.ldr + o : nullptr;
            struct __attribute__((packed, aligned(2))) Out8 {
                OUT v[8];
            };
            if (o + 8 <= p.out) {
                if (res) {
                    const Out8 r = *(const Out8 *)res;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] += (float)r.v[j];
                }
                Out8 out;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    out.v[j] = (OUT)v[j];  // nearest even
                *(Out8 *)y = out;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (o + j < p.out)
                        y[j] = (OUT)(v[j] + (res ? (float)res[j] : 0.0f));
            }
        }
    }
}

// One token's row of a combined product: k FP32 rows by the router's weights, in the order of j.
template <class OUT>
__global__ __launch_bounds__(256) void combine_rows(CombineArgs c)
{
    const int chunks = (c.out + 3) / 4;
    const int64_t n = c.tokens * c.k;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < c.tokens * chunks; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / chunks;
        const int o = (int)(i - t * chunks) * 4;
        f4 v = (f4)0.0f;
        for (int j = 0; j < c.k; ++j) {
            const int place = c.places[t * c.k + j];
            if (place < 0 || place >= n)
                continue;  // dropped
            const f4 part = *(const f4 *)(c.part + (int64_t)place * c.ldp + o);
            const float weight = c.weight ? c.weight[t * c.k + j] : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = fmaf(weight, part[e], v[e]);
        }
        OUT *y = (OUT *)c.y + t * c.ldy + o;
        const OUT *res = c.residual ? (const OUT *)c.residual + t * c.ldr + o : nullptr;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (o + e < c.out)
                y[e] = (OUT)(v[e] + (res ? (float)res[e] : 0.0f));
    }
}

constexpr int kTileRows = 64, kTileOut = 64;  // of the one tile below (a gated tile: half the outputs)

int64_t tiles_most(const ProductArgs &p, bool gated, bool grouped)
{
    const int64_t bo = gated ? kTileOut / 2 : kTileOut, n_out = (p.out + bo - 1) / bo;
    const int64_t row_tiles = grouped ? p.rows / kTileRows + (p.rows < p.experts ? p.rows : p.experts) : (p.rows + kTileRows - 1) / kTileRows;
    return (row_tiles * n_out + 7) / 8 * 8;
}

template <class T, class OUT, bool GROUPED, bool GATED>
hipError_t launch(const ProductArgs &p, hipStream_t stream)
{
    const bool a16 = p.ldx % 8 == 0 && p.ldw % 8 == 0 && p.w_stride % 8 == 0 && (((uintptr_t)p.x | (uintptr_t)p.w) & 15) == 0;
    const dim3 grid((unsigned)tiles_most(p, GATED, GROUPED));
    constexpr int WM = GATED ? 1 : 2, WN = GATED ? 2 : 2, MT = GATED ? 2 : 1;
    if (a16)
        hipLaunchKernelGGL((product_tile<T, OUT, GROUPED, GATED, true, WM, WN, MT, 1>), grid, dim3(64 * WM * WN), 0, stream, p);
    else
        hipLaunchKernelGGL((product_tile<T, OUT, GROUPED, GATED, false, WM, WN, MT, 1>), grid, dim3(64 * WM * WN), 0, stream, p);
    return hipGetLastError();
}

template <class T, class OUT>
hipError_t launch(const ProductArgs &p, bool gated, bool grouped, hipStream_t stream)
{
    if (grouped)
        return gated ? launch<T, OUT, true, true>(p, stream) : launch<T, OUT, true, false>(p, stream);
    return gated ? launch<T, OUT, false, true>(p, stream) : launch<T, OUT, false, false>(p, stream);
}

}  // namespace

bool product_fits(const ProductArgs &p, bool gated, bool grouped)
{
    return tiles_most(p, gated, grouped) * 256 <= UINT32_MAX;  // a grid counts its threads in 32 bits
}

hipError_t launch_product(const ProductArgs &p, int dtype, int out_dtype, bool gated, bool grouped, hipStream_t stream)
{
    if (dtype == kFp16)
        return out_dtype == kFp32 ? launch<_Float16, float>(p, gated, grouped, stream)
                                  : launch<_Float16, _Float16>(p, gated, grouped, stream);
    return out_dtype == kFp32 ? launch<__bf16, float>(p, gated, grouped, stream) : launch<__bf16, __bf16>(p, gated, grouped, stream);
}

hipError_t launch_combine(const CombineArgs &c, int out_dtype, hipStream_t stream)
{
    const int64_t work = c.tokens * ((c.out + 3) / 4), most = 256 * 32;
    const dim3 grid((unsigned)((work + 255) / 256 < most ? (work + 255) / 256 : most));
    if (out_dtype == kFp16)
        hipLaunchKernelGGL(combine_rows<_Float16>, grid, dim3(256), 0, stream, c);
    else if (out_dtype == kBf16)
        hipLaunchKernelGGL(combine_rows<__bf16>, grid, dim3(256), 0, stream, c);
    else
        hipLaunchKernelGGL(combine_rows<float>, grid, dim3(256), 0, stream, c);
    return hipGetLastError();
}

}  // namespace mlpk
