// mlp_ops_quant.h -- device code for the 8-bit format of include/mlp_ops_fp8.h.
#pragma once

#include <hip/hip_runtime.h>

namespace mlpk {

namespace {

// |v| where it enters a block's largest value: 0 for NaN and infinities.
__device__ __forceinline__ float finite_abs(float v)
{
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}

// The scale of a block whose largest finite magnitude is amax.  2^-126 keeps its reciprocal finite.
__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax / 448.0f, 0x1p-126f); }

// v / scale for the rounding: |v| * (1 / scale) is at most 448 (1 + 2^-22), which rounds to 448; infinities become NaN.
__device__ __forceinline__ float scaled(float v, float inv) { return fabsf(v) < __builtin_inff() ? v * inv : __builtin_nanf(""); }

// Four values times inv, in E4M3, nearest even.
__device__ __forceinline__ unsigned to_e4m3x4(float a, float b, float c, float d, float inv)
{
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(a, inv), scaled(b, inv), 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(c, inv), scaled(d, inv), lo, true);
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
