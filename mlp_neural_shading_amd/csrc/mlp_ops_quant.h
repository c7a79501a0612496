// mlp_ops_quant.h -- device code for the 8-bit format of include/mlp_ops_fp8.h.
#pragma once

#include <hip/hip_runtime.h>

namespace mlpk {

namespace {

// The largest finite magnitude of v, 0 if there is none.  The test of each element costs as much as the rest and is made
// only where their sum is not finite: wherever one of them is not, and hardly ever else.
template <int N, class V>
__device__ __forceinline__ float largest(const V &v)
{
    float m = 0.0f, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        m = fmaxf(m, fabsf(v[j]));
        sum += v[j];
    }
    if (!(fabsf(sum) < __builtin_inff())) {
        m = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            m = fmaxf(m, fabsf(v[j]) < __builtin_inff() ? fabsf(v[j]) : 0.0f);
    }
    return m;
}

// The scale of a block whose largest finite magnitude is amax: the quotient by 448 to nearest, its estimate corrected by
// what is left of amax, which is exact.  2^-126 keeps its reciprocal finite.
__device__ __forceinline__ float scale_of(float amax)
{
    constexpr float k = 1.0f / 448.0f;
    const float q = amax * k;
    return fmaxf(fmaf(fmaf(-448.0f, q, amax), k, q), 0x1p-126f);
}

// 1 / scale to nearest, for a scale in [2^-126, 2^120].
__device__ __forceinline__ float inverse(float scale)
{
    const float r = __builtin_amdgcn_rcpf(scale);
    return fmaf(fmaf(-scale, r, 1.0f), r, r);
}

// Four values times inv, in E4M3, nearest even.  |v| * (1 / scale) is at most 448 (1 + 2^-22), which rounds to 448;
// infinities become NaN.
__device__ __forceinline__ unsigned to_e4m3x4(float a, float b, float c, float d, float inv)
{
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, lo, true);
}

// The largest of 16 neighbouring lanes (a row of the wave), in all of them.
__device__ __forceinline__ float max16(float v)
{
    auto turn = [](float w, auto n) {
        constexpr int ROR = 0x120 + decltype(n)::value;
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, w), ROR, 0xf, 0xf, true));
    };
    v = fmaxf(v, turn(v, Number<8>{}));
    v = fmaxf(v, turn(v, Number<4>{}));
    v = fmaxf(v, turn(v, Number<2>{}));
    return fmaxf(v, turn(v, Number<1>{}));
}

}  // namespace

}  // namespace mlpk
