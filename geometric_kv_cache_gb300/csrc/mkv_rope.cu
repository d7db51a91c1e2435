// sm_103a rotary positions of a step's new queries and keys, with the keys
// and values written into their pages (mkv_rope_append).
//
// Pair i of a row turns by a = positions[t] * inv_freq[i]:
//     (x, y) -> factor * (x cos a - y sin a, x sin a + y cos a).
// The angle matters modulo a full turn, and far positions make it large (a
// million radians at pair 0), so it is kept as a 64-bit fraction of a turn:
// F_i = inv_freq[i] / (2 pi) * 2^64 modulo 2^64, once per thread in 64-bit
// floating point, then positions[t] * F_i modulo 2^64 as an integer product
// -- exact, where a product in fp32 would be off by 0.06 radians at a million
// -- read as a signed fraction in [-1/2, 1/2) turn.
//
// Every element is read and written once (bytes: q twice, k, v and their
// stored form), so HBM is the floor; sines and cosines are shared by all heads
// of a token through shared memory.
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
constexpr int kRopeMaxTokens = 4;   // tokens per CTA
constexpr int kMaxPairs = 128;      // rot_dim / 2 at head dim 256

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

// Eight values as E4M3 codes of value / scale: one rounding from fp32 (not
// through bf16), saturated at +-448.
__device__ __forceinline__ uint2 quant8(const float f[8], float scale)
{
    uint16_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] / scale, f[2 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
}

// The row of q_start that token t belongs to, or -1: the last b with
// q_start[b] <= t, if t < q_start[b + 1].
__device__ __forceinline__ int row_of_token(const int32_t *q_start, int batch, int t)
{
    int lo = 0, hi = batch;  // q_start[lo] <= t < q_start[hi], if it is inside at all
    if (t < q_start[0] || t >= q_start[batch]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kRopeThreads)
k_rope_append(const RopeArgs a, int tokens_per_cta)
{
    __shared__ float2 s_cs[kRopeMaxTokens][kMaxPairs];
    __shared__ int s_row[kRopeMaxTokens], s_left[kRopeMaxTokens];
    const int t0 = (int)blockIdx.x * tokens_per_cta, tn = min(tokens_per_cta, a.n_tokens - t0);
    const int pairs = a.rot_dim / 2;
    if (threadIdx.x < tn) {
        const int t = t0 + threadIdx.x;
        int b = row_of_token(a.q_start, a.batch, t), left = 0;
        if (b >= 0) {
            const int lo = a.q_start[b], hi = a.q_start[b + 1];
            left = hi - t;
            if (lo < 0 || hi < lo || hi > a.n_tokens || left <= 0 || t < lo) {
                atomicOr(a.status, MKV_DEV_BAD_TOKENS);
                b = -1;
            }
        }
        s_row[threadIdx.x] = b;
        s_left[threadIdx.x] = left;
    }
    for (int o = threadIdx.x; o < tn * pairs; o += kRopeThreads) {
        const int k = o / pairs, i = o - k * pairs;
        double turns = (double)a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= floor(turns);
        const unsigned long long frac = __double2ull_rn(turns * 18446744073709551616.0);  // 2^64
        const long long phase = (long long)(frac * (unsigned long long)(long long)a.positions[t0 + k]);
        float s, c;
        sincospif((float)phase * 1.0842021724855044e-19f, &s, &c);  // 2 x phase / 2^64 half turns
        s_cs[k][i] = make_float2(c * a.factor, s * a.factor);
    }
    __syncthreads();
    const int units = a.head_dim / 16;  // a unit: two groups of 8 dims that belong together
    const int all = a.q_heads + 2 * a.heads;
    const int work = tn * all * units;
    for (int o = threadIdx.x; o < work; o += kRopeThreads) {
        const int k = o / (all * units), hu = o - k * all * units, hh = hu / units, u = hu - hh * units;
        const int t = t0 + k, b = s_row[k];
        if (b < 0) continue;
        const bool is_q = hh < a.q_heads, is_k = !is_q && hh < a.q_heads + a.heads;
        const int j = is_q ? hh : is_k ? hh - a.q_heads : hh - a.q_heads - a.heads;
        const bool turn = (is_q || is_k) && u < a.rot_dim / 16;
        const bool half = turn && a.layout == MKV_ROPE_HALF;
        // dims [d0, d0 + 8) and [d1, d1 + 8)
        const int d0 = half ? 8 * u : 16 * u, d1 = half ? pairs + 8 * u : 16 * u + 8;
        const uint8_t *src = is_q   ? a.Q + 2 * ((int64_t)t * a.q_stride + (int64_t)j * a.head_dim)
                             : is_k ? a.K + 2 * ((int64_t)t * a.k_stride + (int64_t)j * a.head_dim)
                                    : a.V + 2 * ((int64_t)t * a.v_stride + (int64_t)j * a.head_dim);
        float x[8], y[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(src + 2 * d0), x);
        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(src + 2 * d1), y);
        if (half) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = s_cs[k][8 * u + e];
                const float p = x[e] * cs.x - y[e] * cs.y, q = x[e] * cs.y + y[e] * cs.x;
                x[e] = p;
                y[e] = q;
            }
        } else if (turn) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 c0 = s_cs[k][8 * u + e], c1 = s_cs[k][8 * u + 4 + e];
                const float p0 = x[2 * e] * c0.x - x[2 * e + 1] * c0.y, q0 = x[2 * e] * c0.y + x[2 * e + 1] * c0.x;
                const float p1 = y[2 * e] * c1.x - y[2 * e + 1] * c1.y, q1 = y[2 * e] * c1.y + y[2 * e + 1] * c1.x;
                x[2 * e] = p0;
                x[2 * e + 1] = q0;
                y[2 * e] = p1;
                y[2 * e + 1] = q1;
            }
        }
        if (is_q) {
            uint8_t *dst = a.Q_out + 2 * ((int64_t)t * a.q_heads + j) * a.head_dim;
            st_v4(dst + 2 * d0, pack8(x));
            st_v4(dst + 2 * d1, pack8(y));
            continue;
        }
        const int64_t list = (int64_t)b * a.heads + j;
        const int len = a.lens[list], slot = len - s_left[k];
        if (slot < 0 || len > (a.max_pages << a.page_shift)) {
            if (u == 0) atomicOr(a.status, MKV_DEV_BAD_SEQ_LEN);
            continue;
        }
        const int id = a.table[list * a.max_pages + (slot >> a.page_shift)];
        if ((uint32_t)id >= (uint32_t)a.n_pages) {
            if (u == 0) atomicOr(a.status, MKV_DEV_BAD_PAGE);
            continue;
        }
        const int64_t row = ((int64_t)id << a.page_shift) + (slot & (a.page_size - 1));
        uint8_t *dst = (is_k ? a.k : a.v) + row * a.head_dim * a.es;
        if (a.es == 2) {
            st_v4(dst + 2 * d0, pack8(x));
            st_v4(dst + 2 * d1, pack8(y));
        } else {
            const float sc = is_k ? a.k_scale : a.v_scale;
            *reinterpret_cast<uint2 *>(dst + d0) = quant8(x, sc);
            *reinterpret_cast<uint2 *>(dst + d1) = quant8(y, sc);
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t st)
{
    const int per = 1;
    k_rope_append<<<(unsigned)((a.n_tokens + per - 1) / per), kRopeThreads, 0, st>>>(a, per);
    return cudaGetLastError();
}

}  // namespace mkv
