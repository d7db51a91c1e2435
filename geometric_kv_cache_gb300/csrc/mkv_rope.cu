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
// Every element is read and written once (bytes: q twice, k and v and their
// stored form), so HBM is the floor. A warp takes one token (or, when there
// are few, a share of one token's heads) with no shared memory and no
// barrier: a lane always has the same 16 dims of a head, so the 8 pairs of
// sine and cosine that it needs stay in its registers for all heads. 16384
// tokens of 32 + 2 x 8 heads of 128 dims take 71 us, 5.7 TB/s, 0.83 of the
// measured copy peak; the form with a CTA per group of tokens and the angles in
// shared memory took 82 us, one without loads ahead of the angles 93.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "mkv_device.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// Head groups whose loads are in flight together, and CTAs per SM. Measured on
// 16384 tokens of 32 + 2 x 8 heads of 128 dims (floor 59 us): 2 groups and 3 CTAs
// 70 us, 4 and 2 73 us, 3 and 3 (spilling) 96 us, 2 and 4 (spilling) 101 us.
constexpr int kRopeBatch = 2;

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

// A row of D dims is D / 16 units, one lane each (two groups of 8 dims that
// belong together); the warp covers a group of 512 / D heads at a time: first
// the groups of query heads, then of key heads, then of value heads. `parts`
// warps share a token, group by group.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 3)
k_rope_append(const RopeArgs a, int parts)
{
    constexpr int UNITS = D / 16, HS = 32 / UNITS, OWN = 8 / HS;
    const int lane = threadIdx.x & 31, u = lane % UNITS, sub = lane / UNITS;
    const int pairs = a.rot_dim / 2;
    const int gq = (a.q_heads + HS - 1) / HS, gk = (a.heads + HS - 1) / HS, groups = gq + 2 * gk;
    const bool turned = u < a.rot_dim / 16;  // this lane's dims of a query or key rotate: pairs 8u .. 8u + 7
    // Every row's range, whether a token is found in it or not. (Here and not at
    // the end: the loop then keeps its registers. 16384 tokens 71.2 us, at the end
    // 74.1; 16 rows of one token 4.5 us, as without it.)
    for (int64_t i = (int64_t)(gridDim.x - 1 - blockIdx.x) * kRopeThreads + threadIdx.x; i < a.batch;
         i += (int64_t)gridDim.x * kRopeThreads) {
        const int lo = a.q_start[i], hi = a.q_start[i + 1];
        if (lo < 0 || hi < lo || hi > a.n_tokens) atomicOr(a.status, MKV_DEV_BAD_TOKENS);
    }
    // the fractions of a turn per position of the pairs whose angles this lane works out
    unsigned long long frac[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        frac[o] = 0;
        if (turned) {
            double turns = (double)a.inv_freq[8 * u + sub * OWN + o] * 0.15915494309189533577;  // 1 / (2 pi)
            turns -= floor(turns);
            frac[o] = __double2ull_rn(turns * 18446744073709551616.0);  // 2^64
        }
    }
    const int64_t warps = (int64_t)gridDim.x * kRopeWarps, items = (int64_t)a.n_tokens * parts;
    for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5); item < items; item += warps) {
        const int t = (int)(item / parts), part = (int)(item - (int64_t)t * parts);
        float2 cs[8];
        int b = -1, left = 0;
        for (int g0 = part; g0 < groups; g0 += parts * kRopeBatch) {
            uint4 xr[kRopeBatch], yr[kRopeBatch];
            int id[kRopeBatch], slot[kRopeBatch];
            // group g: 0 queries, 1 keys, 2 values, and this lane's head of it (-1: none)
            auto head_of = [&](int g, int &kind, int &head) {
                kind = g < gq ? 0 : g < gq + gk ? 1 : 2;
                head = (g - (kind == 0 ? 0 : kind == 1 ? gq : gq + gk)) * HS + sub;
                if (g >= groups || head >= (kind == 0 ? a.q_heads : a.heads)) head = -1;
            };
            auto dims = [&](int kind, int &d0, int &d1) {
                const bool half = turned && kind < 2 && a.layout == MKV_ROPE_HALF;
                d0 = half ? 8 * u : 16 * u;
                d1 = half ? pairs + 8 * u : 16 * u + 8;
            };
#pragma unroll
            for (int c = 0; c < kRopeBatch; ++c) {
                int kind, head, d0, d1;
                head_of(g0 + c * parts, kind, head);
                dims(kind, d0, d1);
                if (head >= 0) {
                    const uint8_t *src = (kind == 0 ? a.Q : kind == 1 ? a.K : a.V) +
                                         2 * (t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                                              (int64_t)head * D);
                    xr[c] = *reinterpret_cast<const uint4 *>(src + 2 * d0);
                    yr[c] = *reinterpret_cast<const uint4 *>(src + 2 * d1);
                }
            }
            if (g0 == part) {  // the token's row and angles, while its data is on the way
                const int position = a.positions[t];
                b = row_of_token(a.q_start, a.batch, t);
                if (b < 0) break;  // a token of no row
                const int lo = a.q_start[b], hi = a.q_start[b + 1];
                // (a refused row: no list is that long, so its queries alone are written)
                left = lo < 0 || hi > a.n_tokens ? INT_MAX : hi - t;
                float2 mine[OWN];
#pragma unroll
                for (int o = 0; o < OWN; ++o) {
                    const long long phase = (long long)(frac[o] * (unsigned long long)(long long)position);
                    float sn, cn;
                    sincospif((float)phase * 1.0842021724855044e-19f, &sn, &cn);  // 2 x phase / 2^64 half turns
                    mine[o] = make_float2(cn * a.factor, sn * a.factor);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    cs[e].x = __shfl_sync(kFull, mine[e % OWN].x, u + (e / OWN) * UNITS);
                    cs[e].y = __shfl_sync(kFull, mine[e % OWN].y, u + (e / OWN) * UNITS);
                }
            }
            // the pages of the batch's keys and values
#pragma unroll
            for (int c = 0; c < kRopeBatch; ++c) {
                int kind, head;
                head_of(g0 + c * parts, kind, head);
                slot[c] = -1;
                if (head < 0 || kind == 0) continue;
                const int len = a.lens[(int64_t)b * a.heads + head];
                if (len < left || len > (a.max_pages << a.page_shift)) {
                    if (u == 0 && left != INT_MAX) atomicOr(a.status, MKV_DEV_BAD_SEQ_LEN);
                } else {
                    slot[c] = len - left;
                }
            }
#pragma unroll
            for (int c = 0; c < kRopeBatch; ++c) {
                int kind, head;
                head_of(g0 + c * parts, kind, head);
                id[c] = -1;
                if (slot[c] < 0) continue;
                id[c] = a.table[((int64_t)b * a.heads + head) * a.max_pages + (slot[c] >> a.page_shift)];
                if ((uint32_t)id[c] >= (uint32_t)a.n_pages) {
                    if (u == 0) atomicOr(a.status, MKV_DEV_BAD_PAGE);
                    id[c] = -1;
                }
            }
#pragma unroll
            for (int c = 0; c < kRopeBatch; ++c) {
                int kind, head, d0, d1;
                head_of(g0 + c * parts, kind, head);
                dims(kind, d0, d1);
                if (head < 0 || (kind > 0 && id[c] < 0)) continue;
                float x[8], y[8];
                bf16x8_to_f32(xr[c], x);
                bf16x8_to_f32(yr[c], y);
                if (turned && kind < 2) {
                    if (a.layout == MKV_ROPE_HALF) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float p = x[e] * cs[e].x - y[e] * cs[e].y, q = x[e] * cs[e].y + y[e] * cs[e].x;
                            x[e] = p;
                            y[e] = q;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p0 = x[2 * e] * cs[e].x - x[2 * e + 1] * cs[e].y;
                            const float q0 = x[2 * e] * cs[e].y + x[2 * e + 1] * cs[e].x;
                            const float p1 = y[2 * e] * cs[4 + e].x - y[2 * e + 1] * cs[4 + e].y;
                            const float q1 = y[2 * e] * cs[4 + e].y + y[2 * e + 1] * cs[4 + e].x;
                            x[2 * e] = p0;
                            x[2 * e + 1] = q0;
                            y[2 * e] = p1;
                            y[2 * e + 1] = q1;
                        }
                    }
                }
                if (kind == 0) {
                    uint8_t *dst = a.Q_out + 2 * ((int64_t)t * a.q_heads + head) * D;
                    st_v4(dst + 2 * d0, pack8(x));
                    st_v4(dst + 2 * d1, pack8(y));
                    continue;
                }
                const int64_t row = ((int64_t)id[c] << a.page_shift) + (slot[c] & (a.page_size - 1));
                uint8_t *dst = (kind == 1 ? a.k : a.v) + row * D * a.es;
                if (a.es == 2) {
                    st_v4(dst + 2 * d0, pack8(x));
                    st_v4(dst + 2 * d1, pack8(y));
                } else {
                    const float sc = kind == 1 ? a.k_inv : a.v_inv;
                    *reinterpret_cast<uint2 *>(dst + d0) = quant8(x, sc);
                    *reinterpret_cast<uint2 *>(dst + d1) = quant8(y, sc);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t st)
{
    const void *fn = a.head_dim == 64    ? (const void *)k_rope_append<64>
                     : a.head_dim == 128 ? (const void *)k_rope_append<128>
                     : a.head_dim == 256 ? (const void *)k_rope_append<256>
                                         : nullptr;
    if (!fn) return cudaErrorInvalidValue;
    // a warp per token; with few tokens their heads are shared out
    int parts = 1;
    while (parts < kRopeWarps && (int64_t)a.n_tokens * parts < 152 * kRopeWarps) parts *= 2;
    RopeArgs args = a;
    void *p[] = {&args, &parts};
    const int grid = grid_for_items(fn, kRopeThreads, 0, ((int64_t)a.n_tokens * parts + kRopeWarps - 1) / kRopeWarps);
    const cudaError_t e = cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(kRopeThreads), p, 0, st);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace mkv
