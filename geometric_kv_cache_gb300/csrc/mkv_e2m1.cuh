// 4-bit codes (internal): E2M1 values with an E4M3 scale per 16 dims, as the
// pages of mkv.h hold them, to fp16 and from fp32.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mkv {
namespace dev {

// The four bytes of w, two E2M1 codes each, to fp16 pairs (exact; the lower
// code in the lower half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight fp32 to E2M1 codes, to nearest (ties to the even code), saturated at 6;
// f[0] in the lowest four bits.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&f)[8])
{
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}

// Eight codes with zeros without a sign.
__device__ __forceinline__ uint32_t plain_zeros(uint32_t w)
{
    const uint32_t some = (w | w >> 1 | w >> 2) & 0x11111111u;  // one per code that is not zero
    return w & (some * 15u);
}

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// max|f| over eight values, NaN if one is.
__device__ __forceinline__ float largest8(const float (&f)[8])
{
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
    return m;
}

// E4M3 codes of two fp32 (to nearest, saturated at 448; NaN stays NaN), a in the lower byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float a, float b)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t code)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

// What a group's values are multiplied by to become codes: (1 / scale) / s, 0 where s is 0.
__device__ __forceinline__ float code_factor(uint32_t s, float inv)
{
    const float v = e4m3_to_f32(s);
    return v == 0.f ? 0.f : __fdiv_rn(inv, v);
}

// Eight values of a group as codes.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float r)
{
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(x[i], r);
    return plain_zeros(f32x8_to_e2m1(t));
}

}  // namespace dev
}  // namespace mkv
