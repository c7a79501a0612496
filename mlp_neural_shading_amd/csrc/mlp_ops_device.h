// mlp_ops_device.h -- device code that the products of mlp_ops.h and mlp_ops_fp8.h share: the activations, which tile a
// workgroup takes, the bias as an operand, and the epilogue.
#pragma once

#include <hip/hip_runtime.h>

#include "mlp_ops_kernels.h"
#include "mlp_ops_tiles.h"

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

__device__ __forceinline__ f4 mfma16(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mfma16(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// v (1 + erf(v / sqrt 2)) / 2 = max(v, 0) - |v| h, h = erfc(|v| / sqrt 2) / 2.  log2 h is smooth, so h = 2^P(|v|) with
// a polynomial of degree 10, fitted to log2 h on [0, 5.6] by weighted least squares, the weights moved until the error is
// level: 4e-8 of P, or where |P| < 1 of 1.  With P's roundings in FP32 and the exponential's, h is off by at most
// (2.1 max(1, |P|) + 2) 2^-24 of itself: FP32's accuracy, and better than 1 + erf, which cancels, for negative v.  P falls
// ever faster beyond 5.6.  (Degree 8, 2^-16 of h: 191 us for 65,536 x 1,024 -> 1,024 with a residual, 193 with this.)
// One exponential and 13 full-rate operations; the activation of a 256 x 256 tile is not hidden by its matrix products.
__device__ __forceinline__ float gelu(float v)
{
    const float a = fabsf(v);
    float q = -2.30524932e-08f;
    q = fmaf(q, a, 7.04902789e-07f);
    q = fmaf(q, a, -9.25929726e-06f);
    q = fmaf(q, a, 6.62075327e-05f);
    q = fmaf(q, a, -0.000243540169f);
    q = fmaf(q, a, -7.60762559e-05f);
    q = fmaf(q, a, 0.00704031996f);
    q = fmaf(q, a, -0.052503895f);
    q = fmaf(q, a, -0.45920074f);
    q = fmaf(q, a, -1.15110648f);
    q = fmaf(q, a, -0.99999994f);
    const float h = __builtin_amdgcn_exp2f(q);
    return fmaf(-fminf(a, 100.0f), h, fmaxf(v, 0.0f));  // infinity times 0 would be NaN; a NaN is in h
}

// v / (1 + exp(-v)), as v (2^-32 / (2^-32 + 2^-32 exp(-v))): the reciprocal's argument stays below 2^126 down to v = -109, so
// that its result, normal or 0, is 0 only where the quotient is below FP32 too.
__device__ __forceinline__ float silu(float v)
{
    const float e = __builtin_amdgcn_exp2f(fmaf(v, -1.44269504088896340736f, -32.0f));
    return v * (__builtin_amdgcn_rcpf(0x1p-32f + e) * 0x1p-32f);
}

// The same for FP32 outputs, to a few roundings: exp(-|v|) from exp2 of the product with log2(e) and of what that rounds
// away, scaled where it is subnormal; the quotient with a step of Newton's.  (65,536 x 1,024 -> 1,024 into FP32: 205 us;
// 218 as expf and a division, 190 with the other form.)
__device__ __forceinline__ float silu_full(float v)
{
#pragma clang fp contract(off)  // p + 64 is of the rounded p
    const float a = fminf(fabsf(v), 200.0f);  // a NaN is in the last product
    const float p = a * -1.44269504088896340736f;
    const float rest = fmaf(a, -1.92596299e-08f, fmaf(a, -1.44269504088896340736f, -p));  // log2(e) in two parts
    const bool small = p < -120.0f;
    float e = __builtin_amdgcn_exp2f(small ? p + 64.0f : p);
    e = fmaf(e, rest * 0.693147180559945f, e) * (small ? 0x1p-64f : 1.0f);
    const float d = 1.0f + e, r = __builtin_amdgcn_rcpf(d), n = v < 0.0f ? e : 1.0f, q = n * r;
    return v * fmaf(fmaf(-d, q, n), r, q);
}

// Calls f with the epilogue's activation (MLP_EPI_*, kSiluFull), FP32 to FP32; NaN stays NaN.  The choice is made once
// for a tile of sums, by comparisons: a table of jumps cost 5 us of 159 in 65,536 x 1,024 -> 1,024 with SiLU.  (Once for
// all of a wave's tiles, the compiler merges 128 sums from six branches and spills them.)
template <class F>
__device__ __forceinline__ void with_activation(int act, F f)
{
    if (act == 0)
        f([](float v) { return v; });
    else if (act == 1)
        f([](float v) { return v < 0.0f ? v * kSlope : v; });
    else if (act == 2)
        f([](float v) { return v < 0.0f ? 0.0f : v; });
    else if (act == 3)
        f([](float v) { return gelu(v); });
    else if (act == 4)
        f([](float v) { return silu(v); });
    else
        f([](float v) { return silu_full(v); });
}

template <int V>
struct Number {
    static constexpr int value = V;
};

// 16 bytes from an address aligned to an element only: one load, which the hardware takes at any alignment, at
// full rate where it happens to be aligned.
struct __attribute__((packed, aligned(2))) Unaligned16 {
    u4 v;
};
template <class T>
__device__ __forceinline__ u4 load16(const T *p)
{
    return ((const Unaligned16 *)p)->v;
}

// The 8 columns from `col` of a row of `width`, zero past its end; reads no byte past it.
template <class T>
__device__ __forceinline__ u4 load16_tail(const T *row, int col, int width)
{
    if (col + 8 <= width)
        return load16(row + col);
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
    return tiles_in(begin, end, bn);
}

// Inclusive sum over the wave: within rows of 16 lanes, then row 0 into row 1 and 2 into 3, then the first half into
// the second.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31 into rows 2 and 3
    return v;
}

__device__ __forceinline__ int total_tiles(const int32_t *offsets, int experts, int rows, int bn)
{
    int sum = 0, b, e;
    for (int base = 0; base < experts; base += 64)
        sum += tiles_of(offsets, experts, rows, bn, base + (threadIdx.x & 63), b, e);
    return __builtin_amdgcn_readlane(wave_scan(sum), 63);
}

__device__ __forceinline__ bool find_tile(const int32_t *offsets, int experts, int rows, int bn, int tile, RowTile &out)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base < experts; base += 64) {
        int begin, end;
        const int count = tiles_of(offsets, experts, rows, bn, base + lane, begin, end);
        const int upto = wave_scan(count);
        const int mine = tile - before - (upto - count);  // this tile within the lane's expert
        const unsigned long long hit = __ballot(mine >= 0 && mine < count);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            out.expert = base + src;
            out.row0 = __builtin_amdgcn_readlane(tile_begin(begin, bn, mine), src);
            out.row1 = tile_end(out.row0, __builtin_amdgcn_readlane(end, src), bn);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
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

// One workgroup's tile: which rows of y, which outputs, whose weights.
template <class T>
struct Tile {
    int64_t row0, row1;  // rows (slots) [row0, row1)
    int o0;              // first output
    int expert;          // 0 in a dense product
    const T *w, *bias;
};

constexpr int kBlockRows = 4;

// This workgroup's tile of BO outputs x BN rows; false if it has none.
template <class T, bool GROUPED, bool GATED, int BO, int BN>
__device__ __forceinline__ bool take_tile(const ProductArgs &p, Tile<T> &tile)
{
    const int n_out = (p.out + BO - 1) / BO;
    tile.expert = 0;
    tile.w = (const T *)p.w;
    tile.bias = (const T *)p.bias;
    const int row_tiles = GROUPED ? total_tiles(p.offsets, p.experts, (int)p.rows, BN) : (int)((p.rows + BN - 1) / BN);
    const int64_t t = xcd_tile(blockIdx.x, (int64_t)row_tiles * n_out);
    if (t < 0)
        return false;
    // Blocks of kBlockRows row tiles, the rows of a block fastest: the 32 workgroups that an XCD runs at once
    // then read 4 row panels and 8 weight panels instead of 2 and 16 (1 and 32).
    const int block = (int)(t / ((int64_t)kBlockRows * n_out)), in_block = (int)(t - (int64_t)block * kBlockRows * n_out);
    const int rows_here = min(kBlockRows, row_tiles - block * kBlockRows);
    const int rt = block * kBlockRows + in_block % rows_here;
    tile.o0 = in_block / rows_here * BO;
    if constexpr (GROUPED) {
        RowTile r;
        if (!find_tile(p.offsets, p.experts, (int)p.rows, BN, rt, r))
            return false;
        tile.row0 = r.row0;
        tile.row1 = r.row1;
        tile.expert = r.expert;
        tile.w += r.expert * p.w_stride;
        if (tile.bias)
            tile.bias += (int64_t)r.expert * p.out * (GATED ? 2 : 1);
    } else {
        tile.row0 = (int64_t)rt * BN;
        tile.row1 = tile.row0 + BN < p.rows ? tile.row0 + BN : p.rows;
    }
    return true;
}

// The weight row behind row r of a tile.  A gated layer's tile takes 32 gate rows, the 32 rows they gate, and
// so on (tile rows 64 i .. 64 i + 31 and 64 i + 32 .. 64 i + 63), so one wave holds both.  Rows past the last
// repeat it; what they give is never stored.
template <bool GATED>
__device__ __forceinline__ int weight_row(int o0, int r, int out)
{
    int o = GATED ? o0 + (r >> 6) * 32 + (r & 31) : o0 + r;
    o = o < out ? o : out - 1;
    return GATED && (r & 32) ? o + out : o;
}

// The row of x behind row r of a tile's rows [row0, row1), the last one where r is past it.
template <bool GROUPED>
__device__ __forceinline__ int64_t input_row(const ProductArgs &p, int64_t r, int64_t row1)
{
    r = r < row1 ? r : row1 - 1;
    if (GROUPED && p.slots) {
        const int a = min(max(p.slots[r], 0), (int)p.rows - 1);
        r = a / p.k;
    }
    return r;
}

// The bias as the C operand: lane (g, n) of an MFMA tile holds its rows 8 q + 4 g + i (i = 0 .. 3) of column n.
template <class T, bool GATED>
__device__ __forceinline__ f16x bias_tile(const T *bias, int o0, int r0, int g, int out)
{
    struct __attribute__((packed, aligned(2))) Half4 {
        T v[4];
    };
    f16x b = (f16x)0.0f;
    if (bias)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = r0 + 8 * q + 4 * g;
            if ((GATED ? o0 + (r >> 6) * 32 + (r & 31) : o0 + r) + 3 < out) {
                const Half4 v = *(const Half4 *)(bias + weight_row<GATED>(o0, r, out));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[4 * q + i] = (float)v.v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[4 * q + i] = (float)bias[weight_row<GATED>(o0, r + i, out)];
            }
        }
    return b;
}

struct __attribute__((packed, aligned(2))) Float8 {
    float v[8];
};

// The epilogue of one wave: MT x NT MFMA tiles whose first weight row is tile row r0 and first row `row` (the same
// in all lanes).  One 32 x 32 tile of outputs at a time: the activation and the gate on the sums as they lie, then
// through 4 KB of LDS of the wave's own (no barrier: one wave writes and reads it) into rows, from which a lane takes
// 8 outputs and stores them at once.  Without a residual the outputs are rounded before LDS (chunk k of 8 bytes of row
// n at n * 64 + 8 (k ^ 2 ((n / 4) % 4))); with one, or in FP32, after it and after the addition (chunk k of 16 bytes at
// n * 128 + 16 (k ^ ((n / 2) % 8))).  The residual is requested kAhead tiles ahead: its latency would otherwise stand
// once per tile.  Addresses are a base per tile plus 32 bits per lane (262,144 rows 64 -> 64: 20.4 -> 18.7 us with both).
// SIXTEEN: a tile is four of 16 x 16, of which lane (g, n) holds outputs 4 g .. 4 g + 3 of row n: element 4 e + i is that
// of outputs 16 (e / 2) .. and rows 16 (e % 2) ..  OUT: what is written, where the kernel is for one kind (the branches of
// the others cost 10 us of 96 in 65,536 x 1,024 -> 1,024 with 8-bit operands).
enum { kAnyRows = -1, kHalfRows, kWholeRows };  // 16 bits or FP32 by p.y_fp32, 16 bits, FP32
template <class T, bool GATED, bool SIXTEEN = false, int OUT = kAnyRows, class ARGS, int MT, int NT>
__device__ __forceinline__ void epilogue(const ARGS &p, f16x (&acc)[MT][NT], uint8_t *ob, int o0, int r0, int64_t row, int64_t row1)
{
    typedef typename Vec8<T>::type V8;
    typedef T V4 __attribute__((ext_vector_type(4)));
    struct __attribute__((packed, aligned(2))) Half8 {
        V8 v;
    };
    const int lane = threadIdx.x & 63, g = lane >> 5, n = lane & 31;
    constexpr int MO = GATED ? MT / 2 : MT, TILES = MO * NT, AHEAD = SIXTEEN ? 2 : 4, kAhead = TILES < AHEAD ? TILES : AHEAD;
    const bool y_fp32 = OUT == kAnyRows ? p.y_fp32 : OUT == kWholeRows;
    const int first = o0 + (GATED ? r0 / 2 : r0);            // output
    const int rows = (int)(row1 - row < 32 * NT ? row1 - row : 32 * NT);  // may be 0 or less
    const int outs = p.out - first;
    const int oc = 8 * (lane & 3), rl = lane >> 2;  // this lane's outputs and (of 16 at a time) row
    const bool half_res = p.residual && !y_fp32;
    T *const y16 = (T *)p.y + row * p.ldy + first;
    float *const y32 = (float *)p.y + row * p.ldy + first;
    const T *const r16 = (const T *)p.residual + row * p.ldr + first;
    const float *const r32 = (const float *)p.residual + row * p.ldr + first;
    const int ldy = (int)p.ldy, ldr = (int)p.ldr;  // below 2^25
    // this lane's offset in rows 16 i + rl of a tile; tile t begins at row 32 (t / MO), output 32 (t % MO)
    const unsigned y_at[2] = {(unsigned)(rl * ldy + oc), (unsigned)((16 + rl) * ldy + oc)};
    const unsigned r_at[2] = {(unsigned)(rl * ldr + oc), (unsigned)((16 + rl) * ldr + oc)};
    Half8 res[TILES][2];
    auto fetch = [&](int t) {
        const T *const base = r16 + (int64_t)(32 * (t / MO)) * ldr + 32 * (t % MO);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (32 * (t / MO) + 16 * i + rl < rows && 32 * (t % MO) + oc + 8 <= outs)
                res[t][i] = *(const Half8 *)(base + r_at[i]);
    };
    if (half_res)
#pragma unroll
        for (int t = 0; t < kAhead; ++t)
            fetch(t);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
        const int mt = (t % MO) * (GATED ? 2 : 1), nt = t / MO;
        if constexpr (SIXTEEN)  // also where this tile is left out
            if (half_res && t + kAhead < TILES)
                fetch(t + kAhead);
        if (32 * nt >= rows || 32 * (t % MO) >= outs)
            continue;
        f16x z = acc[mt][nt];
        with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                z[j] = act(z[j]);
        });
        if constexpr (GATED)
            z *= acc[mt + 1][nt];
        const int left = outs - 32 * (t % MO) - oc;  // outputs from this lane's first on
        const int64_t y_tile = (int64_t)(32 * nt) * ldy + 32 * (t % MO), r_tile = (int64_t)(32 * nt) * ldr + 32 * (t % MO);
        if (!p.residual && !y_fp32) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f4 v = {z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
                const int r = SIXTEEN ? 16 * (q % 2) + (lane & 15) : n, k = SIXTEEN ? 4 * (q / 2) + (lane >> 4) : 2 * q + g;
                *(V4 *)(ob + r * 64 + 8 * (k ^ (2 * ((r >> 2) & 3)))) = __builtin_convertvector(v, V4);  // nearest even
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rt = 16 * i + rl;
                const u4 v = *(const u4 *)(ob + rt * 64 + 8 * ((oc / 4) ^ (2 * ((rt >> 2) & 3))));
                if (32 * nt + rt >= rows || left <= 0)
                    continue;
                T *const y = y16 + y_tile + y_at[i];
                if (left >= 8) {
                    ((Unaligned16 *)y)->v = v;
                } else {  // the last outputs of a width that is no multiple of 8
#pragma unroll
                    for (int j = 0; j < 7; ++j)
                        if (j < left)
                            y[j] = __builtin_bit_cast(V8, v)[j];
                }
            }
            continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = SIXTEEN ? 16 * (q % 2) + (lane & 15) : n, k = SIXTEEN ? 4 * (q / 2) + (lane >> 4) : 2 * q + g;
            *(f4 *)(ob + r * 128 + 16 * (k ^ ((r >> 1) & 7))) = f4{z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
        }
        if constexpr (!SIXTEEN)  // kAhead is a multiple of MO: a tile that is left out has its successor left out too
            if (half_res && t + kAhead < TILES)
                fetch(t + kAhead);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rt = 16 * i + rl;
            if (32 * nt + rt >= rows || left <= 0)
                continue;
            const uint8_t *lr = ob + rt * 128;
            const int sw = (rt >> 1) & 7;
            if (left >= 8) {
                const f4 lo = *(const f4 *)(lr + 16 * ((oc / 4) ^ sw)), hi = *(const f4 *)(lr + 16 * ((oc / 4 + 1) ^ sw));
                f8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                if (y_fp32) {
                    if (p.residual) {
                        const Float8 r = *(const Float8 *)(r32 + r_tile + r_at[i]);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[j] += r.v[j];
                    }
                    Float8 y;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y.v[j] = v[j];
                    *(Float8 *)(y32 + y_tile + y_at[i]) = y;
                } else {
                    Half8 y;
                    y.v = __builtin_convertvector(v + __builtin_convertvector(res[t][i].v, f8), V8);  // nearest even
                    *(Half8 *)(y16 + y_tile + y_at[i]) = y;
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < left; ++j) {
                    float v = *(const float *)(lr + 16 * ((oc / 4 + j / 4) ^ sw) + 4 * (j % 4));
                    if (p.residual)
                        v += y_fp32 ? r32[r_tile + r_at[i] + j] : (float)r16[r_tile + r_at[i] + j];
                    if (y_fp32)
                        y32[y_tile + y_at[i] + j] = v;
                    else
                        y16[y_tile + y_at[i] + j] = (T)v;
                }
            }
        }
    }
}

}  // namespace

}  // namespace mlpk
