// mlp_ops_route.hip -- the router's choice of experts, and the order of rows by expert.
#include <hip/hip_runtime.h>

#include "mlp_ops_kernels.h"

namespace mlpk {

namespace {

// ---- the router --------------------------------------------------------------------------------

constexpr double kNone = -__builtin_huge_val();  // the choice of an expert that cannot be chosen

// Without a bias, and without a sum of two scores, the logits give the order: a score rises with its logit, also where
// two scores are equal in 64 bits.  (But beside a logit of +infinity the softmax's other scores are all 0.)
__device__ __forceinline__ bool logits_order(const RouteArgs &r) { return !r.bias && (r.topk_groups == r.groups || r.group_top == 1); }

__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = fmax(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// The largest value and the lowest index that has it, over the wave.
__device__ __forceinline__ void wave_argmax(double &v, int &i)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const double ov = __shfl_xor(v, d);
        const int oi = __shfl_xor(i, d);
        if (ov > v || (ov == v && oi < i)) {
            v = ov;
            i = oi;
        }
    }
}

// One wave per token; lane l holds the experts l, l + 64, ...  Scores and choices in 64 bits: two experts'
// choices may lie closer together than FP32 tells apart.
template <class T, int VPL>
__global__ __launch_bounds__(64) void route_tokens(RouteArgs r)
{
    extern __shared__ double choice_lds[];  // [experts] choices, then [groups] group values
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < r.tokens; t += gridDim.x) {
        const T *x = (const T *)r.logits + t * r.ld;
        double score[VPL], choice[VPL];
        bool open[VPL];
        double m = kNone;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * 64 + lane;
            score[v] = e < r.experts ? (double)(float)x[e] : kNone;
            open[v] = score[v] > kNone;  // neither NaN nor -infinity
            choice[v] = score[v];
            m = open[v] ? fmax(m, score[v]) : m;
        }
        bool by_logit = logits_order(r);
        if (r.sigmoid) {
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                score[v] = open[v] ? 1.0 / (1.0 + exp(-score[v])) : 0.0;
        } else {
            m = wave_max(m);
            by_logit = by_logit && m < __builtin_huge_val();
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                score[v] = !open[v] ? 0.0 : score[v] == m ? 1.0 : exp(score[v] - m);  // of infinities too
                sum += score[v];
            }
            sum = wave_sum(sum);
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                score[v] = open[v] ? score[v] / sum : 0.0;
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * 64 + lane;
            if (!by_logit)
                choice[v] = open[v] ? score[v] + (r.bias ? (double)r.bias[e] : 0.0) : kNone;
            if (!(choice[v] > kNone))
                choice[v] = kNone;
        }
        if (r.topk_groups < r.groups) {
            const int per = r.experts / r.groups;
            double *value = choice_lds + r.experts;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (v * 64 + lane < r.experts)
                    choice_lds[v * 64 + lane] = choice[v];
            __syncthreads();
            for (int g = lane; g < r.groups; g += 64) {
                double first = kNone, second = kNone;
                for (int i = 0; i < per; ++i) {
                    const double cv = choice_lds[g * per + i];
                    if (cv > first) {
                        second = first;
                        first = cv;
                    } else if (cv > second) {
                        second = cv;
                    }
                }
                value[g] = r.group_top == 2 && second > kNone ? first + second : first;
            }
            __syncthreads();
            // chosen groups are marked by NaN
            for (int i = 0; i < r.topk_groups; ++i) {
                double best = kNone;
                int at = r.groups;
                for (int g = lane; g < r.groups; g += 64)
                    if (value[g] > best) {
                        best = value[g];
                        at = g;
                    }
                wave_argmax(best, at);
                if (!(best > kNone))
                    break;
                __syncthreads();
                if (lane == 0)
                    value[at] = __builtin_nan("");
                __syncthreads();
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int e = v * 64 + lane;
                if (e < r.experts) {
                    const double gv = value[e / per];
                    if (gv == gv)
                        choice[v] = kNone;
                }
            }
            __syncthreads();
        }
        double my_score = 0.0, sum = 0.0;
        int my_index = -1;
        for (int j = 0; j < r.k; ++j) {
            double best = kNone;
            int at = r.experts;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (choice[v] > best) {
                    best = choice[v];
                    at = v * 64 + lane;
                }
            wave_argmax(best, at);
            if (!(best > kNone))
                break;
            double s = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (at == v * 64 + lane) {
                    choice[v] = kNone;
                    s = score[v];
                }
            s = __shfl(s, at & 63);
            sum += s;
            if (lane == j) {
                my_index = at;
                my_score = s;
            }
        }
        if (lane < r.k) {
            double w = my_score;
            if (r.renormalise)
                w = sum > 0.0 ? w / sum : 0.0;
            r.index[t * r.k + lane] = my_index;
            r.weight[t * r.k + lane] = (float)(w * (double)r.scale);
        }
    }
}

// ---- the same, L lanes per token ------------------------------------------------------------------
//
// For up to L * VPL experts: a token has L = 16 or 64 lanes, so 64 / L tokens share a wave, and a group of experts a run
// of r.lanes of them, a power of two (without groups, all L); lane i of a group holds its experts VPL i .. VPL i + VPL - 1.
// The choice runs on FP32 keys first (the logits where they give the order, else score + bias), brought to whole numbers
// of 31 bits: the key's place between the token's smallest and largest above the expert's index counted down, so that
// every key differs and equal ones go to the lower index.  The next best key below b is then the largest key - b mod
// 2^32: one subtraction and half a maximum per expert and pick, against a comparison, a search and a removal.  Where
// neighbours among the k + 1 best lie within the error that a key may have, and are not the same logit and bias, the
// order is not certain: some more are picked, one per lane, and these are ranked by their logits or choices in 64 bits.  (Where
// the k-th and the next are the same, all that lies near them is looked at.)  Where even that may leave one out, or two
// groups' values are too near, the token chooses once more on 64-bit keys of all experts (done each time, that cost 11 us
// of 42).  The chosen scores themselves, and the softmax's sum, are computed in 64 bits.  65,536 tokens x 256 experts,
// sigmoid, 8 groups, k = 8: 35 to 40 us, bound by the instructions of the picks, groups and scores; the logits' bytes alone take 7.

constexpr float kLow = -__builtin_huge_valf();

// Of numbers, no NaN among them: the median of three is one instruction, fmaxf two (it quiets its operands first).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -kLow); }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, kLow); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

// Reductions over a token's lanes, the result in all of them: rotations within a row of 16 lanes, then swaps of
// rows and of halves.
template <int L, class F>
__device__ __forceinline__ unsigned lanes_reduce(unsigned v, F f)
{
    v = f(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));  // row_ror 8, 4, 2, 1
    v = f(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
    v = f(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
    v = f(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
    if constexpr (L == 64) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = f(r[0], r[1]);
        const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = f(h[0], h[1]);
    }
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v)
{
    return __builtin_bit_cast(float, lanes_reduce<L>(__builtin_bit_cast(unsigned, v), [](unsigned a, unsigned b) {
                                  return __builtin_bit_cast(unsigned, larger(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
                              }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    return __builtin_bit_cast(float, lanes_reduce<L>(__builtin_bit_cast(unsigned, v), [](unsigned a, unsigned b) {
                                  return __builtin_bit_cast(unsigned, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                              }));
}
template <int L>
__device__ __forceinline__ unsigned lanes_max(unsigned v)
{
    return lanes_reduce<L>(v, [](unsigned a, unsigned b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ double lanes_sum(double v)
{
#pragma unroll
    for (int d = L / 2; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896340736f); }

template <class T, int N>
struct __attribute__((packed, aligned(2))) Packed {
    T v[N];
};

// The experts of a token's lane `me`: [e0, end), none where end <= e0.
__device__ __forceinline__ void experts_of(const RouteArgs &r, int me, int vpl, int &e0, int &end)
{
    const int g = me / r.lanes, per = r.experts / r.groups;
    const bool grouped = r.topk_groups < r.groups;
    e0 = grouped ? g * per + (me - g * r.lanes) * vpl : me * vpl;
    end = grouped ? (g < r.groups ? (g + 1) * per : 0) : r.experts;
}
// The expert number v of lane i.
__device__ __forceinline__ int expert_of(const RouteArgs &r, int i, int vpl, int v)
{
    const int g = i / r.lanes;
    return r.topk_groups < r.groups ? g * (r.experts / r.groups) + (i - g * r.lanes) * vpl + v : i * vpl + v;
}

// This lane's logits, of the experts [e0, end); -infinity for NaN and past the last one.
template <class T, int VPL>
__device__ __forceinline__ void load_logits(const T *logit, int e0, int end, float (&x)[VPL])
{
    if (e0 + VPL <= end) {
        const Packed<T, VPL> p = *(const Packed<T, VPL> *)(logit + e0);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            x[v] = (float)p.v[v];
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float z = (float)logit[e0 + v < end ? e0 + v : 0];
            x[v] = e0 + v < end ? z : kLow;
        }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        x[v] = fmaxf(x[v], kLow);  // the maximum of a NaN and a number is the number
}

// The middle one of first >= second and v.
__device__ __forceinline__ float middle(float first, float second, float v) { return __builtin_amdgcn_fmed3f(first, second, v); }
__device__ __forceinline__ double middle(double first, double second, double v) { return fmax(second, fmin(first, v)); }

// exp to 2^-30 of its value: 2^n times the Taylor polynomial of degree 8 on |r| <= ln(2) / 2 (its next
// term is below 2^-32).
__device__ __forceinline__ double exp_near(double v)
{
    const double n = rint(v * 1.4426950408889634);
    const double r = fma(n, -0.6931471805599453, v);
    double q = 1.0 / 40320;
    q = fma(q, r, 1.0 / 5040);
    q = fma(q, r, 1.0 / 720);
    q = fma(q, r, 1.0 / 120);
    q = fma(q, r, 1.0 / 24);
    q = fma(q, r, 1.0 / 6);
    q = fma(q, r, 0.5);
    q = fma(q, r, 1.0);
    q = fma(q, r, 1.0);
    return ldexp(q, (int)n);
}
// exp to 2^-28.5 of its value, for -700 <= v <= 0, for the softmax's sum: the polynomial of degree 6 through exp at the
// Chebyshev points of |r| <= ln(2) / 2.  2^52 * 1.5 + n holds the whole number n in its low bits, which go to the
// exponent directly.  (65,536 x 256 FP32, k = 8, without renormalisation: 33 us, 37 with exp_near, 28 with an FP32 sum.)
__device__ __forceinline__ double exp_term(double v)
{
    constexpr double kWhole = 6755399441055744.0;
    const double t = fma(v, 1.4426950408889634, kWhole), n = t - kWhole;
    const double r = fma(n, -0.6931471805599453, v);
    double q = 0.0013941108452345638;
    q = fma(q, r, 0.008375126406656224);
    q = fma(q, r, 0.04166635289651486);
    q = fma(q, r, 0.16666415514550614);
    q = fma(q, r, 0.5000000047117842);
    q = fma(q, r, 1.0000000377162372);
    q = fma(q, r, 1.0);
    const unsigned long long bits = __builtin_bit_cast(unsigned long long, q);
    const unsigned high = (unsigned)(bits >> 32) + ((unsigned)__builtin_bit_cast(unsigned long long, t) << 20);
    return __builtin_bit_cast(double, (unsigned long long)high << 32 | (unsigned)bits);
}
// exp to a few parts of 2^-52, for v <= 0: degree 13.  The argument is reduced by Cody and Waite's method: ln 2 cut to its
// first 32 bits, so that n times it is exact, and the rest.
__device__ __forceinline__ double exp_exact(double v)
{
    const double n = rint(fmax(v, -800.0) * 1.4426950408889634);
    const double r = fma(n, -1.9082149292705877e-10, fma(n, -0.6931471803691238, fmax(v, -800.0)));
    double q = 1.0 / 6227020800;
    q = fma(q, r, 1.0 / 479001600);
    q = fma(q, r, 1.0 / 39916800);
    q = fma(q, r, 1.0 / 3628800);
    q = fma(q, r, 1.0 / 362880);
    q = fma(q, r, 1.0 / 40320);
    q = fma(q, r, 1.0 / 5040);
    q = fma(q, r, 1.0 / 720);
    q = fma(q, r, 1.0 / 120);
    q = fma(q, r, 1.0 / 24);
    q = fma(q, r, 1.0 / 6);
    q = fma(q, r, 0.5);
    q = fma(q, r, 1.0);
    q = fma(q, r, 1.0);
    return ldexp(q, (int)n);
}
// 1 / v for a normal v: the hardware's estimate and a step of Newton's.
__device__ __forceinline__ double one_over(double v)
{
    const double e = __builtin_amdgcn_rcp(v);
    return fma(e, fma(-v, e, 1.0), e);
}

// Masks the keys of the groups that are not among the topk_groups best.  In FP32 (`near`: how far two keys may lie
// from their true distance, apart from the roundings of sums; 0 for exact keys) clears `sure` where two groups are too near each other.
template <class K, int L, int VPL>
__device__ __forceinline__ void mask_groups(const RouteArgs &r, K (&key)[VPL], K near, bool &sure)
{
    const int lane = threadIdx.x & 63, me = lane & (L - 1), row = lane - me;
    const K none = -__builtin_huge_valf();
    const int lanes = r.lanes;  // of a group
    K first = none, second = none;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        second = middle(first, second, key[v]);
        first = larger(first, key[v]);
    }
    for (int d = 1; d < lanes; d <<= 1) {
        const K of = __shfl_xor(first, d), os = __shfl_xor(second, d);
        const K low = of < first ? of : first, high = os > second ? os : second;
        first = of > first ? of : first;
        second = low > high ? low : high;
    }
    K value = first;
    if (r.group_top == 2 && second > none) {
        value = first + second;
        if constexpr (sizeof(K) == 4)  // below FP32 it is still not none; two of them come out as too near
            value = larger(value, -3.402823466e38f);
    }
    int better = 0;  // groups before this one
    if constexpr (L == 16 && sizeof(K) == 4) {
        // By rotations: every group's first lane offers its value to the 15 others, and a lane that is not the first
        // meets that of its own group too.
        const float offer = me % lanes ? kLow : (float)value;
#define MLP_RANK(n)                                                                                            \
    {                                                                                                          \
        const float o = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, offer), 0x120 + n, 0xf, 0xf, true)); \
        better += me >= n ? o >= value : o > value; /* from lane me - n, or me - n + 16 */                     \
    }
        MLP_RANK(1) MLP_RANK(2) MLP_RANK(3) MLP_RANK(4) MLP_RANK(5) MLP_RANK(6) MLP_RANK(7) MLP_RANK(8)
        MLP_RANK(9) MLP_RANK(10) MLP_RANK(11) MLP_RANK(12) MLP_RANK(13) MLP_RANK(14) MLP_RANK(15)
#undef MLP_RANK
        better -= me % lanes ? 1 : 0;
    } else {
        for (int d = lanes; d < L; d += lanes) {
            const int at = (me + d) & (L - 1);  // a lane of the group d / lanes further
            const K other = __shfl(value, row + at);
            better += at < me ? other >= value : other > value;
        }
    }
    const bool out = better >= r.topk_groups || !(value > none);
    if (near > 0) {  // FP32: the worst group taken and the best one left
        // Half a step of each key for the addition of its bias, half a one of the sum, and of these bounds themselves;
        // the parts may be far larger than the value.
        const float parts = fabsf((float)first) + (r.group_top == 2 && second > none ? fabsf((float)second) : 0.0f);
        const float off = fminf(parts, 3.402823466e38f) * (1.0f / (1 << 22));
        const float taken = -lanes_max<L>(out ? kLow : off - (float)value), left = lanes_max<L>(out && first > kLow ? (float)value + off : kLow);
        if (left > kLow && !(taken - left > 2 * near))
            sure = false;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        key[v] = out ? none : key[v];
}

// The choice on exact logits or 64-bit keys: in lane j < k the j-th best expert, -1 where none is left.
template <class T, int L, int VPL>
__device__ __forceinline__ int choose_exactly(const RouteArgs &r, const T *logit)
{
    const int lane = threadIdx.x & 63, me = lane & (L - 1);
    int e0, end;
    experts_of(r, me, VPL, e0, end);
    float x[VPL];
    load_logits<T, VPL>(logit, e0, end, x);
    double key[VPL], scale = 1.0;
    float top = kLow;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        top = fmaxf(top, x[v]);
    top = lanes_max<L>(top);
    const bool by_logit = logits_order(r) && (r.sigmoid || top < __builtin_huge_valf());  // the same in a token's lanes
    if (r.sigmoid) {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            key[v] = 1.0 / (1.0 + exp(-(double)x[v]));
    } else {
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const double e = exp((double)x[v] - (double)top);
            key[v] = !(x[v] > kLow) ? 0.0 : x[v] == top ? 1.0 : e;  // of infinities too
            sum += key[v];
        }
        scale = 1.0 / lanes_sum<L>(sum);
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        key[v] = by_logit ? (double)x[v] : key[v] * scale + (r.bias ? (double)r.bias[e0 + v < end ? e0 + v : 0] : 0.0);
        key[v] = x[v] > kLow && key[v] > kNone ? key[v] : kNone;
    }
    bool unused;
    if (r.topk_groups < r.groups)
        mask_groups<double, L, VPL>(r, key, 0.0, unused);
    int index = -1;
    for (int j = 0; j < r.k; ++j) {
        double best = kNone;
        int at = r.experts;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (key[v] > best) {
                best = key[v];
                at = e0 + v;
            }
#pragma unroll
        for (int d = L / 2; d; d >>= 1) {
            const double ov = __shfl_xor(best, d);
            const int oi = __shfl_xor(at, d);
            if (ov > best || (ov == best && oi < at)) {
                best = ov;
                at = oi;
            }
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            key[v] = e0 + v == at ? kNone : key[v];
        if (me == j && best > kNone)
            index = at;
    }
    return index;
}

template <class T, int L, int VPL>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void route_lanes(RouteArgs r)
{
    const int lane = threadIdx.x & 63, me = lane & (L - 1), row = lane - me;
    int e0, last;
    experts_of(r, me, VPL, e0, last);
    constexpr unsigned kIndex = L * VPL - 1;             // the bits of the lane and number
    // Places for the keys, as many as FP32 counts and 31 bits hold; 0 for masked ones.
    constexpr unsigned kPlaces = L * VPL <= 256 ? 1u << 23 : 1u << 22;
    static_assert((uint64_t)kPlaces * (L * VPL) <= 1u << 31, "31 bits");
    const bool by_logit = logits_order(r);
    float bias[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        bias[v] = 0.0f;
    if (r.bias && e0 + VPL <= last) {
        struct __attribute__((packed, aligned(4))) Floats {
            float v[VPL];
        };
        const Floats f = *(const Floats *)(r.bias + e0);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            bias[v] = f.v[v];
    } else if (r.bias) {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            bias[v] = r.bias[e0 + v < last ? e0 + v : 0];
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        bias[v] = fmaxf(bias[v], kLow);  // a NaN masks
    // One round of tokens per wave: in a loop over rounds, the compiler moves the constants of the 64-bit exp before
    // it, and the common path spills.
    const int64_t t = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 / L) + lane / L;
    const bool live = t < r.tokens;
    const T *logit = (const T *)r.logits + (live ? t : r.tokens - 1) * r.ld;
    float key[VPL];
    load_logits<T, VPL>(logit, e0, last, key);
    float top = kLow;       // softmax: largest logit
    double total = 1.0;     // what the scores are divided by without renormalisation
    bool infinite = false;  // softmax: a logit of +infinity; the others' scores are then exactly 0
    float near = 0.0f;
    if (r.sigmoid) {
        if (!by_logit) {
            // A score is off by less than 2^-22: its argument's roundings through a slope of |x| s (1 - s) < 0.23,
            // a step of exp through a quarter, half a one of the sum and one of the reciprocal; two keys by 2^-21.
            near = 1.0f / (1 << 21);
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const float s = __builtin_amdgcn_rcpf(1.0f + exp_of(-key[v])) + bias[v];
                key[v] = key[v] > kLow ? s : kLow;
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            top = larger(top, key[v]);
        top = lanes_max<L>(top);
        infinite = top == __builtin_huge_valf();
        if (!r.renormalise && !infinite) {
            total = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v)  // exactly 1 for the largest, 2^-1009 for a masked one
                total += exp_term(fmax((double)key[v] - (double)top, -700.0));
            total = lanes_sum<L>(total);
        }
        if (!by_logit || infinite) {
            float e[VPL], sum = 0.0f;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const float ev = exp_of(key[v] - top);
                e[v] = key[v] == top ? 1.0f : ev;
                sum += key[v] > kLow ? e[v] : 0.0f;
            }
            sum = lanes_sum<L>(sum);
            if (infinite)
                total = sum;  // how many they are
            if (!by_logit) {
                // off by less than 2^-18 of the largest score: exp, and 16 + 6 additions in the sum
                const float scale = __builtin_amdgcn_rcpf(sum);
                near = scale * (1.0f / (1 << 17));
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    const float s = e[v] * scale + bias[v];
                    key[v] = key[v] > kLow ? s : kLow;
                }
            } else if (infinite) {
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    key[v] = key[v] > kLow ? e[v] : kLow;
            }
        }
    }
    bool sure = true;
    if (r.topk_groups < r.groups)
        mask_groups<float, L, VPL>(r, key, near, sure);

    float high = kLow, low = -kLow;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        high = larger(high, key[v]);
        low = smaller(low, key[v] > kLow ? key[v] : -kLow);
    }
    high = lanes_max<L>(high);
    low = fmaxf(-lanes_max<L>(-low), high - 64.0f);  // what lies further off shares the last place
    // Keys that all lie within 2^23 / 2^100 of each other fill fewer places: no step is infinite, and they count as near.
    const float step = high > low ? fminf((float)(kPlaces - 4) / (high - low), 0x1p100f) : 0.0f;  // infinite keys: 0 or not sure
    if (!(high - low < -kLow) && high > kLow)
        sure = false;
    unsigned place[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        // all of it without a branch, which the compiler would otherwise make of each
        const unsigned q = (unsigned)(__builtin_amdgcn_fmed3f(key[v] - low, 0.0f, 1e30f) * step + 1.0f);
        const unsigned keep = key[v] > kLow ? ~0u : 0u;
        place[v] = (q * (L * VPL) + (kIndex - (unsigned)(me * VPL + v))) & keep;
    }
    unsigned best = 0x80000000u, picked = 0u;
    auto pick = [&](int from, int to) {  // lane j gets the j-th best place
        for (int j = from; j < to; ++j) {
            unsigned below = place[0] - best;
#pragma unroll
            for (int v = 1; v < VPL; ++v)
                below = max(below, place[v] - best);
            best += lanes_max<L>(below);
            picked = me == j ? best : picked;
        }
    };
    auto valid = [&]() {  // 0, a masked key's place, is the last of a token; behind it they begin again
        const unsigned long long ends = __ballot(picked == 0u) >> row;
        return ends & ((2ull << me) - 1) ? 0u : picked;
    };
    auto expert_at = [&](unsigned place) {
        const int at = (int)(kIndex - (place & kIndex));
        return place ? expert_of(r, at / VPL, VPL, at % VPL) : -1;
    };
    pick(0, r.k + 1);
    const unsigned mine = valid(), next = __shfl(mine, row + ((me + 1) & (L - 1)));
    int index = expert_at(mine);
    // places are off by 1 each, and by what the keys are off
    const float doubt = 3.0f + step * (near + fmaxf(fabsf(high), fabsf(low)) * (1.0f / (1 << 22)));
    auto apart = [&](unsigned a, unsigned b) { return (float)(a / (L * VPL) - b / (L * VPL)); };
    bool ordered = true, equal = false;
    if (mine && next && me < r.k && !(apart(mine, next) > doubt)) {
        const int after = expert_at(next);
        ordered = logit[index] == logit[after] && (!r.bias || r.bias[index] == r.bias[after]);
        equal = ordered && me == r.k - 1;
    }
    if (__any(equal)) {  // the k-th and the next are: what is near them has to be so too
        const int edge = __shfl(equal ? index : -1, row + r.k - 1);
        const unsigned kth = __shfl(mine, row + r.k - 1);
        if (edge >= 0) {
            // below the k-th place by at most `doubt`, and two more for what apart() cuts off
            const unsigned reach = ((unsigned)fminf(doubt, (float)kPlaces) + 2u) * (L * VPL);
            const float x_edge = fmaxf((float)logit[edge], kLow);
            bool other = false;
            if (by_logit && !infinite) {  // the keys are the logits
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    other |= (kth - 1u - place[v] < reach) & (key[v] != x_edge);
            } else {
                const float b_edge = r.bias ? r.bias[edge] : 0.0f;
                float x[VPL];
                load_logits<T, VPL>(logit, e0, last, x);
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    if (place[v] && kth - 1u - place[v] < reach)
                        other = other || x[v] != x_edge || (r.bias && r.bias[e0 + v] != b_edge);
            }
            ordered = ordered && !other;
        }
    }
    // Each token takes what its own row needs, whatever its neighbours in the wave need.
    const unsigned long long of_token = L < 64 ? ((1ull << (L & 63)) - 1) << row : ~0ull;
    const bool near_ones = sure && (__ballot(!ordered) & of_token);
    if (__any(near_ones)) {
        const int count = r.k + 8 < L - 1 ? r.k + 8 : L - 1;  // candidates
        pick(r.k + 1, count);
        const unsigned place_of = valid();
        const int candidate = me < count ? expert_at(place_of) : -1;
        const unsigned kth = __shfl(place_of, row + r.k - 1), end = __shfl(place_of, row + count - 1);
        if (near_ones && end && !(apart(kth, end) > 2.0f * doubt))
            sure = false;  // one that was not picked may be as good
        double exact = kNone;
        if (candidate >= 0) {
            const double z = (double)(float)logit[candidate], b = r.bias ? (double)r.bias[candidate] : 0.0;
            if (by_logit && !infinite) {
                exact = z;
            } else if (r.sigmoid) {
                const double e = exp_exact(-fabs(z));
                exact = (z < 0.0 ? e : 1.0) / (1.0 + e) + b;
            } else {
                exact = z == (double)top ? 1.0 : exp_exact(z - (double)top);
            }
        }
        if (!r.sigmoid && !by_logit) {
            float x[VPL];
            load_logits<T, VPL>(logit, e0, last, x);
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const double e = exp_exact((double)x[v] - (double)top);
                sum += !(x[v] > kLow) ? 0.0 : x[v] == top ? 1.0 : e;
            }
            sum = lanes_sum<L>(sum);
            if (candidate >= 0)
                exact = exact / sum + (r.bias ? (double)r.bias[candidate] : 0.0);
        }
        int rank = 0;
        for (int j = 0; j < count; ++j) {
            const double other = __shfl(exact, row + j);
            const int of = __shfl(candidate, row + j);
            rank += other > exact || (other == exact && of < candidate);
        }
        // to the lane of its rank; those that are none all rank behind the candidates
        const int to = candidate >= 0 ? rank : L - 1;
        const int moved = __builtin_amdgcn_ds_permute((row + to) * 4, candidate);
        // a lane that nobody sends to reads 0
        const int held = __popcll(__ballot(candidate >= 0) & of_token);
        if (near_ones)
            index = me < held ? moved : -1;
    }
    if (me >= r.k)
        index = -1;
    if (__any(!sure)) {
        const int chosen = choose_exactly<T, L, VPL>(r, logit);
        index = sure ? index : chosen;
    }

    // The chosen scores, in lane j the j-th.
    double score = 0.0;
    if (index >= 0) {
        const double z = (double)(float)logit[index];
        if (r.sigmoid) {
            const double e = exp_near(fmax(-fabs(z), -800.0));  // 0 from there on
            score = (z < 0.0 ? e : 1.0) * one_over(1.0 + e);
        } else {
            score = (float)z == top ? 1.0 : exp_near(fmax(z - (double)top, -800.0));
        }
    }
    const double part = r.renormalise ? lanes_sum<L>(score) : total;
    if (live && me < r.k) {
        r.index[t * r.k + me] = index;
        const double w = part > 1e-300 ? score * one_over(part) : part > 0.0 ? score / part : 0.0;
        r.weight[t * r.k + me] = index >= 0 ? (float)(w * (double)r.scale) : 0.0f;
    }
}

// Lanes per group where `lanes` lanes of vpl experts each serve this router (room for k + 1 picks, and for every
// group's lanes), else 0.
int lanes_per_group(const RouteArgs &r, int lanes, int vpl)
{
    if (r.k >= lanes)
        return 0;
    if (r.topk_groups == r.groups)
        return r.experts <= lanes * vpl ? lanes : 0;
    int each = 1;
    while (each * vpl < r.experts / r.groups)
        each *= 2;
    return r.groups * each <= lanes ? each : 0;
}

template <class T, int L, int VPL>
hipError_t launch_lanes(const RouteArgs &r, int each, hipStream_t stream)
{
    constexpr int64_t kMost = (int64_t)1 << 25;  // tokens per launch: a grid counts its threads in 32 bits
    hipError_t err = hipSuccess;
    for (int64_t t = 0; t < r.tokens && err == hipSuccess; t += kMost) {
        RouteArgs part = r;
        part.lanes = each;
        part.tokens = r.tokens - t < kMost ? r.tokens - t : kMost;
        part.logits = (const T *)r.logits + t * r.ld;
        part.index += t * r.k;
        part.weight += t * r.k;
        const int64_t blocks = (part.tokens + 4 * (64 / L) - 1) / (4 * (64 / L));
        hipLaunchKernelGGL((route_lanes<T, L, VPL>), dim3((unsigned)blocks), dim3(256), 0, stream, part);
        err = hipGetLastError();
    }
    return err;
}

// The layout that serves this router, and its lanes per group in `each`.
enum RouteForm { kLanes16x4, kLanes16x8, kLanes16x16, kLanes64x8, kWave };
RouteForm choose_route(const RouteArgs &r, int &each)
{
    if ((each = lanes_per_group(r, 16, 4)))
        return kLanes16x4;
    if ((each = lanes_per_group(r, 16, 8)))
        return kLanes16x8;
    if ((each = lanes_per_group(r, 16, 16)))
        return kLanes16x16;
    if ((each = lanes_per_group(r, 64, 8)))
        return kLanes64x8;
    return kWave;
}

template <class T>
hipError_t launch_route_typed(const RouteArgs &r, hipStream_t stream)
{
    int each;
    switch (choose_route(r, each)) {
    case kLanes16x4:
        return launch_lanes<T, 16, 4>(r, each, stream);
    case kLanes16x8:
        return launch_lanes<T, 16, 8>(r, each, stream);
    case kLanes16x16:
        return launch_lanes<T, 16, 16>(r, each, stream);
    case kLanes64x8:
        return launch_lanes<T, 64, 8>(r, each, stream);
    case kWave:
        break;
    }
    const dim3 grid((unsigned)(r.tokens < 256 * 64 ? r.tokens : 256 * 64));
    const size_t lds = (size_t)(r.experts + r.groups) * sizeof(double);
    const int vpl = (r.experts + 63) / 64;
    if (vpl <= 1)
        hipLaunchKernelGGL((route_tokens<T, 1>), grid, dim3(64), lds, stream, r);
    else if (vpl <= 2)
        hipLaunchKernelGGL((route_tokens<T, 2>), grid, dim3(64), lds, stream, r);
    else if (vpl <= 4)
        hipLaunchKernelGGL((route_tokens<T, 4>), grid, dim3(64), lds, stream, r);
    else if (vpl <= 8)
        hipLaunchKernelGGL((route_tokens<T, 8>), grid, dim3(64), lds, stream, r);
    else
        hipLaunchKernelGGL((route_tokens<T, 16>), grid, dim3(64), lds, stream, r);
    return hipGetLastError();
}

// ---- the order of rows by expert: a stable counting sort ---------------------------------------
//
// The assignments are cut into nb chunks, one per workgroup (at most kMaxChunks, of kChunk assignments or
// more).  dispatch_count counts each chunk's experts; dispatch_place gives every assignment its slot: the slots of the
// experts before it, of its expert in the chunks before, in the waves before (each wave has a contiguous share of the
// chunk) and in its wave before it, the last by matching the lanes of equal expert bit by bit.  The counts of the
// chunks before are summed by dispatch_place itself where there are few (kOwnSum), else by dispatch_scan in between.
// Every sum is of whole numbers and every position follows from the order alone, so the result is the same each time.
// Up to kChunk assignments take dispatch_place alone, in one workgroup.  The indices are read twice and a slot and a
// place written for each; a chain of loads, scans and barriers bounds it below some millions of assignments
// (1,048,576 over 16 experts: 12.5 us, the bytes alone 2.4).
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int64_t kChunk = 4096, kMaxChunks = 1024;
constexpr int64_t kOwnSum = 8192;  // counts (65,536 x 8 assignments, 256 experts, 32,768 counts: 20 us summed, 16 scanned)
constexpr int kHeld = kChunk / kThreads;  // indices per lane of a chunk of kChunk

int64_t chunk_of(int64_t n)
{
    const int64_t c = (n + kMaxChunks - 1) / kMaxChunks;
    return c <= kChunk ? kChunk : (c + kThreads - 1) / kThreads * kThreads;
}

// Exclusive scan over the workgroup; `total` gets the sum.  `sums`: kWaves + 1 ints of LDS.
__device__ __forceinline__ int block_scan(int v, int *sums, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        upto += lane >= d ? o : 0;
    }
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int s = sums[w];
        before += w < wave ? s : 0;
        total += s;
    }
    __syncthreads();
    return before + upto - v;
}

__global__ __launch_bounds__(kThreads) void dispatch_count(DispatchArgs d, int64_t chunk)
{
    extern __shared__ int counts[];  // [experts]
    for (int e = threadIdx.x; e < d.experts; e += kThreads)
        counts[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * chunk, end = begin + chunk < d.n ? begin + chunk : d.n;
    for (int64_t i0 = begin + threadIdx.x; i0 < end; i0 += kHeld * kThreads) {
        int e[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            e[j] = i0 + j * kThreads < end ? d.index[i0 + j * kThreads] : -1;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if ((unsigned)e[j] < (unsigned)d.experts)
                atomicAdd(&counts[e[j]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < d.experts; e += kThreads)
        d.workspace[(int64_t)blockIdx.x * d.experts + e] = counts[e];
}

// Turns each expert's counts into the number in the chunks before; the totals go behind them.
__global__ __launch_bounds__(kThreads) void dispatch_scan(DispatchArgs d, int nb)
{
    __shared__ int sums[kWaves];
    int *mine = d.workspace + (int64_t)threadIdx.x * d.experts + blockIdx.x;
    const int v = (int)threadIdx.x < nb ? *mine : 0;
    int total;
    const int before = block_scan(v, sums, total);
    if ((int)threadIdx.x < nb)
        *mine = before;
    if (threadIdx.x == 0)
        d.workspace[(int64_t)d.experts * nb + blockIdx.x] = total;
}

enum { kOne, kSums, kScanned };  // the only workgroup; sums the counts itself; after dispatch_scan

template <int HOW>
__global__ __launch_bounds__(kThreads) void dispatch_place(DispatchArgs d, int64_t chunk, int nb)
{
    extern __shared__ int next[];  // [kWaves][experts]: counts, then the next slot; kSums: [2][experts] sums behind
    __shared__ int sums[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = d.experts;
    int *all = next + kWaves * E, *before = all + E;
    const int64_t share = chunk / kWaves;
    const int64_t block0 = blockIdx.x * chunk, block1 = block0 + chunk < d.n ? block0 + chunk : d.n;
    const int64_t begin = block0 + wave * share, end = begin + share < block1 ? begin + share : block1;
    int held[kHeld];  // this lane's indices, all of them in a chunk of kChunk
    auto fetch = [&](int64_t i0) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            held[j] = i0 + 64 * j + lane < end ? d.index[i0 + 64 * j + lane] : -1;
    };
    fetch(begin);
    for (int i = tid; i < (kWaves + (HOW == kSums ? 2 : 0)) * E; i += kThreads)
        next[i] = 0;
    __syncthreads();
    int *mine = next + wave * E;
    for (int64_t i0 = begin; i0 < end; i0 += 64 * kHeld) {
        if (i0 != begin)
            fetch(i0);
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if ((unsigned)held[j] < (unsigned)E)
                atomicAdd(&mine[held[j]], 1);
    }
    if constexpr (HOW == kSums)
        for (int i = tid; i < nb * E; i += kThreads) {
            const int v = d.workspace[i], e = i % E;
            atomicAdd(&all[e], v);
            if (i / E < (int)blockIdx.x)
                atomicAdd(&before[e], v);
        }
    __syncthreads();
    int count = 0;
    if (tid < E) {
        if constexpr (HOW == kOne)
            for (int w = 0; w < kWaves; ++w)
                count += next[w * E + tid];
        else
            count = HOW == kSums ? all[tid] : d.workspace[(int64_t)E * nb + tid];
    }
    int total;
    const int base = block_scan(count, sums, total);
    if (tid < E) {
        int at = base + (HOW == kOne ? 0 : HOW == kSums ? before[tid] : d.workspace[(int64_t)blockIdx.x * E + tid]);
        for (int w = 0; w < kWaves; ++w) {
            const int in_wave = next[w * E + tid];
            next[w * E + tid] = at;
            at += in_wave;
        }
        if (blockIdx.x == 0) {
            d.offsets[tid] = base;
            if (tid == 0)
                d.offsets[E] = total;
        }
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < E)
        ++bits;
    for (int64_t i0 = begin; i0 < end; i0 += 64 * kHeld) {
        if (share > 64 * kHeld)
            fetch(i0);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int64_t i = i0 + 64 * j + lane;
            const int e = held[j];
            const bool live = (unsigned)e < (unsigned)E;
            unsigned long long peers = __ballot(live);
            for (int b = 0; b < bits; ++b) {
                const unsigned long long set = __ballot((e >> b) & 1);
                peers &= (e >> b) & 1 ? set : ~set;
            }
            const int rank = __popcll(peers & ((1ull << lane) - 1));
            int slot = -1;
            if (live)
                slot = mine[e] + rank;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every lane has read before one adds
            __builtin_amdgcn_wave_barrier();
            if (live && rank == 0)
                mine[e] += __popcll(peers);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (i < end) {
                d.places[i] = slot;
                if (live)
                    d.slots[slot] = (int)i;
            }
        }
    }
    for (int64_t i = block0 + tid; i < block1; i += kThreads)  // slots not in use
        if (i >= total)
            d.slots[i] = -1;
}

}  // namespace

const char *route_kernel(const RouteArgs &r)
{
    static const char *const names[] = {"lanes 16x4", "lanes 16x8", "lanes 16x16", "lanes 64x8", "wave"};
    int each;
    return names[choose_route(r, each)];
}

hipError_t launch_route(const RouteArgs &r, int dtype, hipStream_t stream)
{
    return dtype == kFp16 ? launch_route_typed<_Float16>(r, stream)
           : dtype == kBf16 ? launch_route_typed<__bf16>(r, stream)
                            : launch_route_typed<float>(r, stream);
}

int64_t dispatch_workspace_entries(int64_t n, int experts)
{
    const int64_t chunk = chunk_of(n), nb = (n + chunk - 1) / chunk;
    return nb <= 1 ? 0 : experts * (nb + 1);
}

hipError_t launch_dispatch(const DispatchArgs &d, hipStream_t stream)
{
    const int64_t chunk = chunk_of(d.n);
    const int nb = (int)((d.n + chunk - 1) / chunk);
    const size_t lds = (size_t)d.experts * sizeof(int);
    if (nb <= 1) {
        hipLaunchKernelGGL(dispatch_place<kOne>, dim3(1), dim3(kThreads), kWaves * lds, stream, d, chunk, 1);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(dispatch_count, dim3(nb), dim3(kThreads), lds, stream, d, chunk);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && nb * (int64_t)d.experts <= kOwnSum) {
        hipLaunchKernelGGL(dispatch_place<kSums>, dim3(nb), dim3(kThreads), (kWaves + 2) * lds, stream, d, chunk, nb);
        return hipGetLastError();
    }
    if (err == hipSuccess) {
        hipLaunchKernelGGL(dispatch_scan, dim3(d.experts), dim3(kThreads), 0, stream, d, nb);
        err = hipGetLastError();
    }
    if (err == hipSuccess) {
        hipLaunchKernelGGL(dispatch_place<kScanned>, dim3(nb), dim3(kThreads), kWaves * lds, stream, d, chunk, nb);
        err = hipGetLastError();
    }
    return err;
}

}  // namespace mlpk
