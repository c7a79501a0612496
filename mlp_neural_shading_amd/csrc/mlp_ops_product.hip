// mlp_ops_product.hip -- one affine layer with its epilogue, dense or over the rows routed to experts:
//   y[r][o] = round(act(sum_i x[r][i] w[o][i] + b[o]) + residual[r][o])
// and gated, act(z[o]) * z[out + o] of a w with twice the rows.  x and w are row-major, so both
// operands run along K and are staged alike.
#include <hip/hip_runtime.h>

#include "mlp_ops_device.h"

namespace mlpk {

namespace {

// WM x WN waves, each MT x NT MFMA tiles of 32 weight rows x 32 rows, K advancing 64 per stage through two
// stages of LDS: each thread loads its chunks of stage s + 1 into registers while stage s is multiplied (requesting
// s + 2 as well gained nothing: 5,003 x 1,001 -> 777 38 against 34 us).
// Bound by its loads' latency: 5,003 x 1,001 -> 777 FP16 33 us, where rows lie at odd elements; by the rows' bytes in
// 262,144 rows 64 -> 64 by expert, 24 us, 67 MB.
// 128 bytes a row; chunk c (16 bytes) of row r sits at slot c ^ ((r / 2) % 8): the 16 rows that one 256-byte
// LDS cycle of a fragment read serves fall in 16 different slots.
template <class T, bool GROUPED, bool GATED, int WM, int WN, int MT, int NT, int WPE>
__global__ __launch_bounds__(64 * WM *WN) __attribute__((amdgpu_waves_per_eu(WPE, WPE))) void product_tile(ProductArgs p)
{
    typedef typename Vec8<T>::type V8;
    constexpr int BK = 64, TH = 64 * WM * WN, BM = 32 * WM * MT, BN = 32 * WN * NT;
    constexpr int RPP = TH / 8;  // rows the workgroup stages at a time, one chunk per thread
    constexpr int CA = BM / RPP, CB = BN / RPP;
    constexpr int A_ST = BM * 128, STAGE = (BM + BN) * 128;
    static_assert(CA * RPP == BM && CB * RPP == BN && RPP % 16 == 0, "whole chunks per thread, one swizzle per thread");
    static_assert(!GATED || MT % 2 == 0, "gate and partner tiles in one wave");
    static_assert(WM * WN * 4096 <= 2 * STAGE, "the epilogue's rows fit the stages");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];

    Tile<T> tile;
    if (!take_tile<T, GROUPED, GATED, (GATED ? BM / 2 : BM), BN>(p, tile))
        return;  // whole workgroup, before any barrier
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int g = lane >> 5, n = lane & 31;
    const int c = tid % 8, r_in = tid / 8;
    const T *wp[CA], *xp[CB];
#pragma unroll
    for (int i = 0; i < CA; ++i)
        wp[i] = tile.w + (int64_t)weight_row<GATED>(tile.o0, r_in + i * RPP, p.out) * p.ldw + 8 * c;
#pragma unroll
    for (int i = 0; i < CB; ++i)
        xp[i] = (const T *)p.x + input_row<GROUPED>(p, tile.row0 + r_in + i * RPP, tile.row1) * p.ldx + 8 * c;
    const int st = r_in * 128 + 16 * (c ^ ((r_in >> 1) & 7));

    f16x acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const f16x b = bias_tile<T, GATED>(tile.bias, tile.o0, (wm * MT + mt) * 32, g, p.out);
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
            ra[i] = load16(wp[i] + s * BK);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            rb[i] = load16(xp[i] + s * BK);
    };
    auto load_tail = [&]() {
#pragma unroll
        for (int i = 0; i < CA; ++i)
            ra[i] = load16_tail(wp[i] - 8 * c, full * BK + 8 * c, p.in);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            rb[i] = load16_tail(xp[i] - 8 * c, full * BK + 8 * c, p.in);
    };
    auto store = [&](int s) {
        uint8_t *d = lds + (s & 1) * STAGE + st;
#pragma unroll
        for (int i = 0; i < CA; ++i)
            *(u4 *)(d + i * RPP * 128) = ra[i];
#pragma unroll
        for (int i = 0; i < CB; ++i)
            *(u4 *)(d + A_ST + i * RPP * 128) = rb[i];
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
    epilogue<T, GATED>(p, acc, lds + wave * 4096, tile.o0, wm * MT * 32, tile.row0 + wn * NT * 32, tile.row1);
}

// The same for rows that are 4-byte aligned: the stages go from memory into LDS directly, NS of them in flight.
// A stage is 64 columns, 128 bytes of every row: whole cache lines (at 32 columns each line came from L2 twice).
// A stage's last quarter is multiplied after the barrier that frees it, while the next stage's first fragments are
// read, so the matrix unit does not wait for LDS there.  A width that is no whole number of stages ends with one of the
// row's last 64 columns, requested like the others and multiplied without what it has of the stage before (20,000 x
// 1,008 -> 768 with 256 x 256, 128 x 128 and 128 x 64 tiles 34, 44 and 56 us; 38, 51 and 65 with the rest loaded when
// the whole stages are done).
// Bound by the matrix unit and the power it may draw: 8,192 x 4,096 -> 4,096 BF16 222 us, 1,240 TFLOP/s of the 1,519 that
// the largest library product reaches; the unit is busy 65 % of the cycles at 1.82 GHz, LDS 26 %, L2 serves 80 %.
// A wave's 128 x 64 sums take 6 operands from LDS for 8 products; two stages of 64 columns were faster than
// four or five of 32 (222 against 237 and 240).
template <class T, bool GROUPED, bool GATED, int WM, int WN, int MT, int NT, int NS, int WPE>
__global__ __launch_bounds__(64 * WM *WN) __attribute__((amdgpu_waves_per_eu(WPE, WPE))) void product_big(ProductArgs p)
{
    typedef typename Vec8<T>::type V8;
    constexpr int BK = 64, TH = 64 * WM * WN, BM = 32 * WM * MT, BN = 32 * WN * NT;
    constexpr int RPP = TH / 8;
    constexpr int CA = BM / RPP, CB = BN / RPP;  // 16-byte loads per thread and stage
    constexpr int A_ST = BM * 128, STAGE = (BM + BN) * 128;
    static_assert(CA * RPP == BM && CB * RPP == BN && RPP % 16 == 0, "whole chunks per thread, one swizzle per thread");
    static_assert(!GATED || MT % 2 == 0, "gate and partner tiles in one wave");
    static_assert(WM * WN * 4096 <= STAGE, "the epilogue's rows fit a stage");
    static_assert(NS == 2 || NS == 3, "");
    // A variable each: the compiler then knows that a load into one does not touch another.
    __shared__ __attribute__((aligned(16))) uint8_t l0[STAGE], l1[STAGE], l2[NS == 3 ? STAGE : 16];

    Tile<T> tile;
    if (!take_tile<T, GROUPED, GATED, (GATED ? BM / 2 : BM), BN>(p, tile))
        return;  // whole workgroup, before any barrier
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int g = lane >> 5, n = lane & 31;
    const int r_in = tid / 8;
    const int c = (tid & 7) ^ ((r_in >> 1) & 7);  // the chunk that this thread's slot holds
    const T *src[CA + CB];
#pragma unroll
    for (int i = 0; i < CA; ++i)
        src[i] = tile.w + (int64_t)weight_row<GATED>(tile.o0, r_in + i * RPP, p.out) * p.ldw + 8 * c;
#pragma unroll
    for (int i = 0; i < CB; ++i)
        src[CA + i] = (const T *)p.x + input_row<GROUPED>(p, tile.row0 + r_in + i * RPP, tile.row1) * p.ldx + 8 * c;

    const int full = p.in / BK, rest = p.in - full * BK;
    // After the whole stages come the row's last 64 columns, some of them a second time; past them they are requested
    // again, unused, and so is the last whole stage where `rest` is 0, or odd (4-byte aligned loads cannot reach it).
    const int last_step = rest % 2 ? 0 : rest;
    int issued = 0;  // stages requested
    auto request = [&](uint8_t *dst) {
        const int step = issued + 1 < full ? BK : issued + 1 == full ? last_step : 0;
#pragma unroll
        for (int i = 0; i < CA + CB; ++i) {
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src[i],
                                             (__attribute__((address_space(3))) void *)(dst + wave * 1024 + i * (TH * 16)), 16, 0, 0);
            src[i] += step;
        }
        ++issued;
    };
    V8 fa[2][MT], fb[2][NT];
    const int a_rd = (wm * MT * 32 + n) * 128, b_rd = A_ST + (wn * NT * 32 + n) * 128, swz = (n >> 1) & 7;
    auto read = [&](const uint8_t *d, int kb) {
        const int ch = 16 * ((2 * kb + g) ^ swz);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            fa[kb & 1][mt] = *(const V8 *)(d + a_rd + mt * 32 * 128 + ch);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            fb[kb & 1][nt] = *(const V8 *)(d + b_rd + nt * 32 * 128 + ch);
    };
    f16x acc[MT][NT];
    auto multiply = [&](int kb) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                acc[mt][nt] = mfma32(fa[kb & 1][mt], fb[kb & 1][nt], acc[mt][nt]);
    };
    auto mix = [&]() {  // one MFMA, then one LDS read
#pragma unroll
        for (int i = 0; i < (MT * NT < MT + NT ? MT * NT : MT + NT); ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if constexpr (MT * NT > MT + NT)
            __builtin_amdgcn_sched_group_barrier(0x008, MT * NT - MT - NT, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int AHEAD = (NS - 2) * (CA + CB);  // loads still in flight when the next stage has to be there
    // One stage, whose first fragments have been read: cur is its buffer, nxt the next stage's.
    auto quarters = [&](const uint8_t *__restrict cur) {
#pragma unroll
        for (int kb = 0; kb < 3; ++kb) {
            read(cur, kb + 1);
            multiply(kb);
            mix();
        }
    };
    auto last = [&](const uint8_t *__restrict nxt, uint8_t *__restrict freed) {
        request(freed);
        read(nxt, 0);
        multiply(3);
        mix();
    };
    auto turn = [&](auto ahead) {
        constexpr int V = decltype(ahead)::value;
        __builtin_amdgcn_s_waitcnt(0x0070 | (V & 15) | (V >> 4) << 14);  // vmcnt(V) lgkmcnt(0)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
#define MLP_STAGE(CUR, NXT)                                                                                    \
    quarters(CUR);                                                                                             \
    turn(Number<AHEAD>{});                                                                                     \
    last(NXT, CUR);                                                                                            \
    if (++s == full)                                                                                           \
        break;
    if (full) {
        request(l0);
        request(l1);
        if constexpr (NS == 3)
            request(l2);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const f16x b = bias_tile<T, GATED>(tile.bias, tile.o0, (wm * MT + mt) * 32, g, p.out);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = b;
    }
    if (full) {
        turn(Number<(NS - 1) * (CA + CB)>{});
        read(l0, 0);
        for (int s = 0;;) {
            MLP_STAGE(l0, l1)
            if constexpr (NS == 3) {
                MLP_STAGE(l1, l2)
                MLP_STAGE(l2, l0)
            } else {
                MLP_STAGE(l1, l0)
            }
        }
    }
#undef MLP_STAGE
    __builtin_amdgcn_s_waitcnt(0x0070);  // the requests past the end
    __syncthreads();
    if (rest) {
        const uint8_t *d = NS == 2 ? (full % 2 ? l1 : l0) : full % 3 == 0 ? l0 : full % 3 == 1 ? l1 : l2;
        int skip = BK - rest;  // columns of the last 64 that the whole stages have had
        if (!full || !last_step) {  // the rest and zeros, through registers
#pragma unroll
            for (int i = 0; i < CA + CB; ++i) {
                const T *row = src[i] - 8 * c - (full ? (full - 1) * BK : 0);
                *(u4 *)(l0 + tid * 16 + i * (TH * 16)) = load16_tail(row, full * BK + 8 * c, p.in);
            }
            __syncthreads();
            d = l0;
            skip = 0;
        }
#pragma unroll 1
        for (int kb = skip / 16; kb < 4; ++kb) {
            const int ch = 16 * ((2 * kb + g) ^ swz), first = skip - 8 * (2 * kb + g);
            auto keep = [&](const uint8_t *at) {
                u4 v = *(const u4 *)at;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = 2 * i >= first ? v[i] : 0u;
                return __builtin_bit_cast(V8, v);
            };
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                fa[0][mt] = keep(d + a_rd + mt * 32 * 128 + ch);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                fb[0][nt] = keep(d + b_rd + nt * 32 * 128 + ch);
            multiply(0);
        }
        __syncthreads();
    }
    epilogue<T, GATED>(p, acc, l0 + wave * 4096, tile.o0, wm * MT * 32, tile.row0 + wn * NT * 32, tile.row1);
}

// Narrow layers over many rows, up to 64 weight rows and 64 columns: bound by the bytes of x and y.  A wave
// keeps the whole weight matrix and the bias in registers, as MFMA operands, and takes kRounds tiles of 32 rows, each
// straight from memory as the other operand (lane (g, n) loads the 16 bytes of row n at columns 16 kb + 8 g), two tiles
// ahead.  No barrier anywhere; LDS only turns the outputs into rows (1,048,576 rows 32 -> 32 FP16: 47 us).
template <class T, bool GROUPED, bool GATED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void product_narrow(ProductArgs p)
{
    typedef typename Vec8<T>::type V8;
    constexpr int MT = 2, KB = 4, BO = GATED ? 16 * MT : 32 * MT, kRounds = 4, kAhead = 2, BN = 4 * 32 * kRounds;
    __shared__ __attribute__((aligned(16))) uint8_t lds[4 * 4096];
    Tile<T> tile;
    if (!take_tile<T, GROUPED, GATED, BO, BN>(p, tile))
        return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 5, n = lane & 31;
    const int64_t first = tile.row0 + wave * (32 * kRounds);
    if (first >= tile.row1)
        return;

    int64_t rows[kRounds];  // of x: known before the first is needed, the routed ones are looked up
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
        rows[i] = input_row<GROUPED>(p, first + 32 * i + n, tile.row1);
    V8 a[MT][KB];
    f16x bias[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const T *w = tile.w + (int64_t)weight_row<GATED>(tile.o0, 32 * mt + n, p.out) * p.ldw;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
            a[mt][kb] = __builtin_bit_cast(V8, load16_tail(w, 16 * kb + 8 * g, p.in));
        bias[mt] = bias_tile<T, GATED>(tile.bias, tile.o0, 32 * mt, g, p.out);
    }
    const bool whole = p.in == 16 * KB;
    u4 b[kRounds][KB];
    auto load = [&](int i) {
        const T *x = (const T *)p.x + rows[i] * p.ldx;
        if (whole) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                b[i][kb] = load16(x + 16 * kb + 8 * g);
        } else {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                b[i][kb] = load16_tail(x, 16 * kb + 8 * g, p.in);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        load(i);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int64_t row = first + 32 * i;
        if (row >= tile.row1)
            break;
        if (i + kAhead < kRounds)
            load(i + kAhead);
        f16x acc[MT][1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            acc[mt][0] = bias[mt];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                acc[mt][0] = mfma32(a[mt][kb], __builtin_bit_cast(V8, b[i][kb]), acc[mt][0]);
        }
        epilogue<T, GATED>(p, acc, lds + wave * 4096, tile.o0, 0, row, tile.row1);
    }
}

// Few rows: a workgroup of NW waves (blockDim / 64, at most 16) takes 16 * MA weight rows and up to 16 rows of
// x, and its waves share K: each multiplies a run of columns straight from memory (16 x 16 x 32 MFMA, weights = A,
// x = B; lane (g, n) loads the 16 bytes of row n at columns 8 g), kDepth steps requested at once, and the waves'
// sums meet in LDS.  Every wave's loads are independent, with no LDS or barrier between them; the weights' bytes are
// the floor (7 x 2,048 -> 2 x 4,096 gated: 33.6 MB, 8.8-11 us; 1 x 1,024 -> 1,024: 4.2, two latencies).  Taking 32 or
// 64 rows at once instead of several workgroups that read the same weights from L2 was slower (32 x 4,096 -> 4,096: 20
// against 14 us; 64 x 4,096 -> 1,024: 27 against 10).
template <class T, bool GROUPED, bool GATED, int MA>
__global__ __launch_bounds__(1024) void product_few(ProductArgs p)
{
    typedef typename Vec8<T>::type V8;
    static_assert(!GATED || MA == 2, "16 gates and the 16 they gate");
    constexpr int BO = GATED ? 16 : 16 * MA, BN = 16, kDepth = 4;
    constexpr int SUMS = 16 * MA * BN;  // per wave
    extern __shared__ float sums[];      // [NW][MA][16 rows of x][16 weight rows]

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nw = blockDim.x >> 6, g = lane >> 4, n = lane & 15;
    const int n_out = (p.out + BO - 1) / BO;
    const int o0 = (int)(blockIdx.x % n_out) * BO;
    int64_t row0 = (int64_t)(blockIdx.x / n_out) * BN, row1 = row0 + BN < p.rows ? row0 + BN : p.rows;
    const T *w = (const T *)p.w, *bias = (const T *)p.bias;
    if constexpr (GROUPED) {
        RowTile rt;
        if (!find_tile(p.offsets, p.experts, (int)p.rows, BN, (int)(blockIdx.x / n_out), rt))
            return;  // whole workgroup
        row0 = rt.row0;
        row1 = rt.row1;
        w += rt.expert * p.w_stride;
        if (bias)
            bias += (int64_t)rt.expert * p.out * (GATED ? 2 : 1);
    }
    const T *wp[MA];
#pragma unroll
    for (int i = 0; i < MA; ++i) {
        int o = o0 + (GATED ? 0 : 16 * i) + n;
        o = (o < p.out ? o : p.out - 1) + (GATED && i ? p.out : 0);
        wp[i] = w + (int64_t)o * p.ldw;
    }
    const T *xp = (const T *)p.x + input_row<GROUPED>(p, row0 + n, row1) * p.ldx;

    f4 acc[MA];
#pragma unroll
    for (int j = 0; j < MA; ++j)
        acc[j] = (f4)0.0f;
    const int share = ((p.in + nw - 1) / nw + 31) / 32 * 32;
    const int begin = wave * share, end = min(begin + share, p.in);
    int k = begin;
    u4 a[kDepth][MA], b[kDepth];
    auto multiply = [&](int d) {
#pragma unroll
        for (int j = 0; j < MA; ++j)
            acc[j] = mfma16(__builtin_bit_cast(V8, a[d][j]), __builtin_bit_cast(V8, b[d]), acc[j]);
    };
    for (; k + 32 * kDepth <= end; k += 32 * kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
#pragma unroll
            for (int j = 0; j < MA; ++j)
                a[d][j] = load16(wp[j] + k + 32 * d + 8 * g);
            b[d] = load16(xp + k + 32 * d + 8 * g);
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            multiply(d);
    }
    for (; k < end; k += 32) {  // the rest, and a last step of fewer than 32 columns
#pragma unroll
        for (int j = 0; j < MA; ++j)
            a[0][j] = load16_tail(wp[j], k + 8 * g, p.in);
        b[0] = load16_tail(xp, k + 8 * g, p.in);
        multiply(0);
    }
    // Lane (g, n) of an MFMA tile holds weight rows 4 g .. 4 g + 3 of row n.
#pragma unroll
    for (int j = 0; j < MA; ++j)
        *(f4 *)(sums + wave * SUMS + (j * 16 + n) * 16 + 4 * g) = acc[j];
    __syncthreads();
    for (int i = tid; i < BO * BN; i += blockDim.x) {
        // 16 outputs of a row together
        const int ol = i % 16, oj = GATED ? 0 : i / 16 % MA, rl = i / BO;
        const int at = (oj * 16 + rl) * 16 + ol;
        const int o = o0 + 16 * oj + ol;
        const int64_t row = row0 + rl;
        if (o >= p.out || row >= row1)
            continue;
        float z = bias ? (float)bias[o] : 0.0f, u = GATED && bias ? (float)bias[o + p.out] : 0.0f;
        for (int v = 0; v < nw; ++v) {
            z += sums[v * SUMS + at];
            if constexpr (GATED)
                u += sums[v * SUMS + at + 256];
        }
        with_activation(p.act, [&](auto act) { z = act(z); });
        if constexpr (GATED)
            z *= u;
        if (p.residual)
            z += p.y_fp32 ? ((const float *)p.residual)[row * p.ldr + o] : (float)((const T *)p.residual)[row * p.ldr + o];
        if (p.y_fp32)
            ((float *)p.y)[row * p.ldy + o] = z;
        else
            ((T *)p.y)[row * p.ldy + o] = (T)z;
    }
}

// One token's row of a combined product: k FP32 rows by the router's weights, in the order of j, 4 outputs per thread.
// Bound by the rows' bytes (8,192 tokens x 4 x 2,048: 335 MB, 66 us, the rate of a large copy): four rows are requested at once, and
// the division by the row's chunks is in 32 bits where the call is small enough.
template <class T, class INDEX>
__global__ __launch_bounds__(256) void combine_rows(CombineArgs c)
{
    struct __attribute__((packed, aligned(sizeof(T)))) Out4 {
        T v[4];
    };
    const INDEX chunks = (c.out + 3) / 4, all = (INDEX)c.tokens * chunks;
    const int64_t n = c.tokens * c.k;
    for (INDEX i = (INDEX)blockIdx.x * 256 + threadIdx.x; i < all; i += (INDEX)gridDim.x * 256) {
        const INDEX t = i / chunks;
        const int o = (int)(i - t * chunks) * 4;
        const int32_t *places = c.places + (int64_t)t * c.k;
        const float *weights = c.weight + (int64_t)t * c.k;
        f4 v = (f4)0.0f;
        for (int j0 = 0; j0 < c.k; j0 += 4) {
            f4 part[4];
            float weight[4];
            bool on[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int place = j0 + j < c.k ? places[j0 + j] : -1;
                on[j] = place >= 0 && place < n;  // else dropped
                weight[j] = on[j] && c.weight ? weights[j0 + j] : 1.0f;
                part[j] = (f4)0.0f;
                if (on[j])
                    part[j] = *(const f4 *)(c.part + (int64_t)place * c.ldp + o);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (on[j])
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = fmaf(weight[j], part[j][e], v[e]);
        }
        T *y = (T *)c.y + (int64_t)t * c.ldy + o;
        const T *res = c.residual ? (const T *)c.residual + (int64_t)t * c.ldr + o : nullptr;
        if (o + 4 <= c.out) {
            if (res) {
                const Out4 r = *(const Out4 *)res;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] += (float)r.v[e];
            }
            Out4 out;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out.v[e] = (T)v[e];
            *(Out4 *)y = out;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (o + e < c.out)
                    y[e] = (T)(v[e] + (res ? (float)res[e] : 0.0f));
        }
    }
}

// ---- which kernel ---------------------------------------------------------------------------------

// kBig 256 weight rows x 256 rows, kMid 128 x 128, kSmall 128 x 64 (all three straight into LDS), kTile 64 x 128 through
// registers, kFew 16 x 16, kFewWide 32 x 16, kNarrow 64 x 512 (K up to 64).
enum Form { kBig, kMid, kSmall, kTile, kFew, kFewWide, kNarrow };
struct Shape {
    int bm, bn, threads;
};
constexpr Shape kShapes[] = {{256, 256, 512}, {128, 128, 256}, {128, 64, 256}, {64, 128, 256}, {16, 16, 1024}, {32, 16, 1024},
                             {64, 512, 256}};

// Row tiles of bn rows there can be at most.
int64_t row_tiles(const ProductArgs &p, bool grouped, int bn)
{
    return grouped ? p.rows / bn + (p.rows < p.experts ? p.rows : p.experts) : (p.rows + bn - 1) / bn;
}

int64_t tiles_most(const ProductArgs &p, bool gated, bool grouped, Form f)
{
    const Shape s = kShapes[f];
    const int64_t bo = gated ? (f == kFew || f == kFewWide ? 16 : s.bm / 2) : s.bm;
    const int64_t tiles = (p.out + bo - 1) / bo * row_tiles(p, grouped, s.bn);
    return f == kFew || f == kFewWide ? tiles : (tiles + 7) / 8 * 8;  // the XCDs' runs are equally long
}

// Rounds of tiles over the chip, `at_once` of them per round; where a CU runs two, a last round that is at most half
// full takes 0.6 of one.
float rounds(int64_t tiles, int at_once, bool two_per_cu)
{
    const float whole = (float)(tiles / at_once), rest = (float)(tiles % at_once) / at_once;
    return whole + (rest == 0.0f ? 0.0f : two_per_cu && rest <= 0.5f ? 0.6f : 1.0f);
}

// The kernel, for 256 CUs (MI355X); times in us and BF16, narrow layers in FP16, of every kernel forced on the size:
//   - fewer than 1,024 tiles of 16 x 16: kFew, whose waves share K, from 512 on 32 weight rows at a time.  Before that
//     border: 64 x 4,096 -> 1,024 10 (kFewWide 14, kSmall 21), 32 x 4,096 -> 4,096 kFewWide 14 (17; 21), 100 x 256 ->
//     2,000 6.6 (6.4; 6.4).  Behind it kSmall, though it fills few CUs: 300 x 1,024 -> 1,024 8 (kFewWide 11), 64 x
//     1,024 -> 4,096 8.1 (8.3), 64 x 4,096 -> 4,096 21 (24), 17 x 4,096 -> 2 x 4,096 21 (23), 256 x 4,096 -> 4,096 22 (86);
//   - at most 64 weight rows: kTile (262,144 rows 64 -> 64 18, kMid 26; 100,000 x 512 -> 64 29, kMid 35), or kNarrow from
//     1,024 of its tiles on (1,048,576 rows 32 -> 32 47, kTile 76; 64 -> 64 by expert 80, kTile 108).  Below: 500,000 rows
//     64 -> 64 kTile 29, kNarrow 35; by expert, 262,144 rows, 25 and 29; but 262,144 rows 32 -> 32 22 and 14;
//   - rows that are not 4-byte aligned (an odd width): kTile, which takes them;
//   - else the one of kBig, kMid and kSmall that takes the least time by its rounds, each of so much per 1,024 columns
//     and so much for its start and epilogue, as fitted to 65,536 x 1,024 -> 1,024 (139, 191 and 226 us),
//     8,192 x 4,096 -> 4,096 (222, 281 and 363) and 1,048,576 x 64 -> 128 (207, 133 and 192).  It gives kSmall for
//     512 x 1,024 -> 4,096 (9; kMid 13) and 512 x 4,096 -> 4,096 (24; 39), kMid for 1,024 x 4,096 -> 4,096 (43; kSmall 45,
//     kBig 75) and 2,048^3 (25; 25, 42).  One round of few tiles takes as long as one of all CUs: 64 to 512 x 4,096 ->
//     4,096 all 21 to 24.
//     The experts' last tiles count as half full, and kBig and kMid are for 192 and 96 rows per expert and more.  32 experts,
//     2,048 -> 2 x 1,024, by rows per expert: 64 kSmall 70 (kMid 94), 128 kMid 96 (kSmall 90), 192 kMid 107 (113; kBig
//     122), 256 kMid 126 (kBig 128), 512 kMid 206 (kBig 185), 1,024 kBig 309 (kMid 356).
Form choose_form(const ProductArgs &p, bool gated, bool grouped)
{
    const bool even = p.ldx % 2 == 0 && p.ldw % 2 == 0 && p.w_stride % 2 == 0 && (((uintptr_t)p.x | (uintptr_t)p.w) & 3) == 0;
    const int64_t wide = (int64_t)p.out * (gated ? 2 : 1);
    const int64_t few = row_tiles(p, grouped, 16) * ((wide + 15) / 16);
    if (few < 1024)
        return gated || few >= 512 ? kFewWide : kFew;
    if (wide <= 64 && p.in <= 64 && row_tiles(p, false, 512) >= 1024)
        return kNarrow;
    if (!even || wide <= 64)
        return kTile;
    const int64_t used = !grouped ? 0 : p.rows < p.experts ? p.rows : p.experts;
    auto tiles = [&](Form f) {
        const int64_t bm = kShapes[f].bm, bn = kShapes[f].bn;
        return (grouped ? p.rows / bn + (used + 1) / 2 : (p.rows + bn - 1) / bn) * ((wide + bm - 1) / bm);
    };
    const float k = (float)p.in / 1024.0f;
    const float big = rounds(tiles(kBig), 256, false) * (26.5f * k + 9.5f);
    const float mid = rounds(tiles(kMid), 512, true) * (15.5f * k + 8.5f);
    const float small = rounds(tiles(kSmall), 512, true) * (10.4f * k + 5.5f);
    const int64_t each = used ? p.rows / used : INT64_MAX;  // rows per expert
    if (each >= 192 && big <= mid && big <= small)
        return kBig;
    return each >= 96 && mid <= small ? kMid : kSmall;
}

template <class T, bool GROUPED, bool GATED>
hipError_t launch(const ProductArgs &p, hipStream_t stream)
{
    const Form form = choose_form(p, GATED, GROUPED);
    const dim3 grid((unsigned)tiles_most(p, GATED, GROUPED, form)), block(kShapes[form].threads);
    switch (form) {
    case kBig:
        hipLaunchKernelGGL((product_big<T, GROUPED, GATED, 2, 4, 4, 2, 2, 2>), grid, block, 0, stream, p);
        break;
    case kMid:
        hipLaunchKernelGGL((product_big<T, GROUPED, GATED, 2, 2, 2, 2, 2, 2>), grid, block, 0, stream, p);
        break;
    case kSmall:
        hipLaunchKernelGGL((product_big<T, GROUPED, GATED, 2, 2, 2, 1, 3, 2>), grid, block, 0, stream, p);
        break;
    case kTile:
        hipLaunchKernelGGL((product_tile<T, GROUPED, GATED, 1, 4, 2, 1, 3>), grid, block, 0, stream, p);
        break;
    case kNarrow:
        hipLaunchKernelGGL((product_narrow<T, GROUPED, GATED>), grid, block, 0, stream, p);
        break;
    default:
        // 64 columns or more for each of up to 16 waves
        const int waves = p.in >= 1024 ? 16 : p.in >= 512 ? 8 : p.in >= 256 ? 4 : p.in >= 128 ? 2 : 1;
        const size_t lds = (size_t)waves * kShapes[form].bm * 16 * 4;
        if (GATED || form == kFewWide)
            hipLaunchKernelGGL((product_few<T, GROUPED, GATED, 2>), grid, dim3(64 * waves), lds, stream, p);
        else
            hipLaunchKernelGGL((product_few<T, GROUPED, GATED, GATED ? 2 : 1>), grid, dim3(64 * waves), lds, stream, p);
    }
    return hipGetLastError();
}

template <class T>
hipError_t launch(const ProductArgs &p, bool gated, bool grouped, hipStream_t stream)
{
    if (grouped)
        return gated ? launch<T, true, true>(p, stream) : launch<T, true, false>(p, stream);
    return gated ? launch<T, false, true>(p, stream) : launch<T, false, false>(p, stream);
}

}  // namespace

bool product_fits(const ProductArgs &p, bool gated, bool grouped)
{
    const Form form = choose_form(p, gated, grouped);
    return tiles_most(p, gated, grouped, form) * kShapes[form].threads <= UINT32_MAX;  // a grid counts its threads in 32 bits
}

const char *product_kernel(const ProductArgs &p, bool gated, bool grouped)
{
    static const char *const names[] = {"big", "mid", "small", "tile", "few", "few wide", "narrow"};
    return names[choose_form(p, gated, grouped)];
}

hipError_t launch_product(const ProductArgs &p, int dtype, bool gated, bool grouped, hipStream_t stream)
{
    return dtype == kFp16 ? launch<_Float16>(p, gated, grouped, stream) : launch<__bf16>(p, gated, grouped, stream);
}

template <class T>
hipError_t launch_combine_typed(const CombineArgs &c, hipStream_t stream)
{
    const int64_t work = c.tokens * ((c.out + 3) / 4), most = 256 * 32, blocks = (work + 255) / 256;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    if (work < (int64_t)1 << 31)  // and so is the last step past it
        hipLaunchKernelGGL((combine_rows<T, unsigned>), grid, dim3(256), 0, stream, c);
    else
        hipLaunchKernelGGL((combine_rows<T, int64_t>), grid, dim3(256), 0, stream, c);
    return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs &c, int out_dtype, hipStream_t stream)
{
    return out_dtype == kFp16 ? launch_combine_typed<_Float16>(c, stream)
           : out_dtype == kBf16 ? launch_combine_typed<__bf16>(c, stream)
                                : launch_combine_typed<float>(c, stream);
}

}  // namespace mlpk
