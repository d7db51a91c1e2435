// What the two rotary appends share (internal): tokens of packed rows, bf16 and
// E4M3 rows from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mkv_device.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

// Two fp32 to a bf16 pair (round to nearest even), the first in the lower half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack8(const float f[8])
{
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Eight values times `inv` (the reciprocal of the scale) as E4M3 codes: rounded
// to 8 bits from fp32, not through bf16, and saturated at +-448.
__device__ __forceinline__ uint2 quant8(const float f[8], float inv)
{
    uint16_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
}

// The row that token t belongs to, for a whole warp: the number of b with
// q_start[b + 1] <= t, found 32 ways at a time; -1 when t is in no row.
__device__ __forceinline__ int row_of_token(const int32_t *q_start, int batch, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = batch;
    while (n > 32) {
        const int step = (n + 31) / 32, x = (lane + 1) * step;  // q_start[lo + x]: where part `lane` ends
        const int below = __popc(__ballot_sync(kFull, x <= n && q_start[lo + x] <= t));
        lo += below * step;
        n = min(step, n - below * step);
    }
    lo += __popc(__ballot_sync(kFull, lane < n && q_start[lo + lane + 1] <= t));
    return lo < batch && q_start[lo] <= t && t < q_start[lo + 1] ? lo : -1;
}

}  // namespace
}  // namespace mkv
