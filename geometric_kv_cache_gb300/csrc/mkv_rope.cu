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
#include "mkv_e2m1.cuh"
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

// Sine and cosine, times `factor`, of the 64-bit product position * freq. The
// angle in turns is a product with 1 / (2 pi) of 106 bits, whose whole turns drop
// out exactly.
__device__ __forceinline__ double2 turn_exactly(int position, float freq, float factor)
{
    const double angle = (double)position * (double)freq;
    const double hi = angle * 0.15915494309189535, lo = fma(angle, 0.15915494309189535, -hi) + angle * -9.839338337591243e-18;
    const double turns = (hi - rint(hi)) + lo;
    double sn, cn;
    sincospi(2.0 * turns, &sn, &cn);
    return make_double2(cn * factor, sn * factor);
}

// The rotated values of this lane's 16 dims (x, y as loaded) as 64-bit
// arithmetic gives them, rounded once to fp32, for a whole warp: a lane works out
// the angles that it works out in 32 bits, and the others come from their lanes.
// Not inlined: 4-bit keys next to a border take it, one in a few hundred groups
// of heads. (64-bit operations are 1 / 64 of the 32-bit rate.)
template <int D>
__device__ __noinline__ void rotate_exactly(const RopeArgs &a, int t, uint4 xr, uint4 yr, float (&x)[8], float (&y)[8])
{
    constexpr int UNITS = D / 16, OWN = 8 * UNITS / 32;
    const int lane = threadIdx.x & 31, u = lane % UNITS, sub = lane / UNITS;
    double2 mine[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int pair = 8 * u + sub * OWN + o;
        mine[o] = make_double2(0.0, 0.0);
        if (u < a.rot_dim / 16) {
            int axis = a.n_axes > 0 ? a.axes[pair] : 0;
            if ((uint32_t)axis >= (uint32_t)a.n_axes) axis = 0;
            mine[o] = turn_exactly(a.positions[(int64_t)axis * a.n_tokens + t], a.inv_freq[pair], a.factor);
        }
    }
    float p[8], q[8];
    bf16x8_to_f32(xr, p);
    bf16x8_to_f32(yr, q);
    const bool half = a.layout == MKV_ROPE_HALF;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double cn = __shfl_sync(kFull, mine[e % OWN].x, u + (e / OWN) * UNITS);
        const double sn = __shfl_sync(kFull, mine[e % OWN].y, u + (e / OWN) * UNITS);
        // pairs (x[e], y[e]); neighbouring ones: x holds the lane's first four, y the others
        const int i = 2 * e & 7;
        const float c0 = half ? p[e] : e < 4 ? p[i] : q[i], c1 = half ? q[e] : e < 4 ? p[i + 1] : q[i + 1];
        const float r0 = (float)(c0 * cn - c1 * sn), r1 = (float)(c0 * sn + c1 * cn);
        if (half) {
            x[e] = r0;
            y[e] = r1;
        } else if (e < 4) {
            x[i] = r0;
            x[i + 1] = r1;
        } else {
            y[i] = r0;
            y[i + 1] = r1;
        }
    }
}

// Where the other eight dims of a group of 16 are, when the row is one of pairs
// (i, i + rot / 2) and its rotated part is `halves` times 8 pairs: eights are
// numbered along the row, a lane u < halves has numbers u (its x) and halves + u
// (its y). Lane in the lower bits, 32 for its y.
__device__ __forceinline__ int other_eight(int eight, int halves)
{
    const int o = eight ^ 1;
    return o < halves ? o : 32 + o - halves;
}

// Codes of a lane's eight values t = x r where x is known to +-err only: flags
// what another x within that could change.
__device__ __forceinline__ uint32_t codes8_within(const float (&x)[8], float r, float err, bool &unsure)
{
    // (2^-19: the roundings of x r and of the sums below, values up to 8)
    const float e = fmaf(err * 1.0001f, r, 1.9073486e-6f);
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __fmul_rn(x[i], r);
        lo[i] = t - e;
        hi[i] = t + e;
    }
    const uint32_t l = f32x8_to_e2m1(lo), h = f32x8_to_e2m1(hi);
    // (the ends of a small enough stretch have different signs only where both are zero; a large one is of groups whose
    // scale is saturated, or of infinities and NaN)
    unsure |= ((l ^ h) & 0x77777777u) != 0 || !(e < 0.125f);
    return plain_zeros(l);
}

// A row of D dims is D / 16 units, one lane each (two groups of 8 dims that
// belong together); the warp covers a group of 512 / D heads at a time: first
// the groups of query heads, then of key heads, then of value heads. `parts`
// warps share a token, group by group.
//
// FOUR: keys and values become 4-bit codes. A lane's two eights are one group of
// 16 dims or, where pairs lie half a row apart, one each of two groups, whose
// largest elements meet over shuffles. Codes of rotated keys have to be those of
// the exact rotation, whose fp32 form here is off by up to kOff times its
// operands (and 2^-50 of the angle, whose fraction of a turn comes from 64-bit
// floating point): where that could change a code or a scale (its lower and upper ends
// round differently) the warp works the rotation out in 64 bits.
// AXES: pairs turn by the position of their own axis.
constexpr float kOff = 1e-6f;

template <int D, bool FOUR, bool AXES>
__global__ void __launch_bounds__(kRopeThreads, FOUR ? 2 : 3)
k_rope_append(const __grid_constant__ RopeArgs a, int parts)
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
    const int32_t *place[AXES ? OWN : 1];  // and where those pairs' positions are
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        frac[o] = 0;
        if constexpr (AXES) {
            place[o] = a.positions;
            if (turned) {
                const int axis = a.axes[8 * u + sub * OWN + o];
                if ((uint32_t)axis < (uint32_t)a.n_axes) place[o] += (int64_t)axis * a.n_tokens;
                else atomicOr(a.status, MKV_DEV_BAD_AXIS);
            }
        }
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
        float off = kOff;
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
                int position[AXES ? OWN : 1];
#pragma unroll
                for (int o = 0; o < (AXES ? OWN : 1); ++o) position[o] = AXES ? place[o][t] : a.positions[t];
                b = row_of_token(a.q_start, a.batch, t);
                if (b < 0) break;  // a token of no row
                const int lo = a.q_start[b], hi = a.q_start[b + 1];
                // (a refused row: no list is that long, so its queries alone are written)
                left = lo < 0 || hi > a.n_tokens ? INT_MAX : hi - t;
                float2 mine[OWN];
#pragma unroll
                for (int o = 0; o < OWN; ++o) {
                    const long long phase = (long long)(frac[o] * (unsigned long long)(long long)position[AXES ? o : 0]);
                    float sn, cn;
                    sincospif((float)phase * 1.0842021724855044e-19f, &sn, &cn);  // 2 x phase / 2^64 half turns
                    mine[o] = make_float2(cn * a.factor, sn * a.factor);
                }
                if constexpr (FOUR) {  // the largest angle of the lane's pairs
                    float angle = 0.f;
#pragma unroll
                    for (int o = 0; o < OWN; ++o)
                        if (turned) angle = fmaxf(angle, fabsf(a.inv_freq[8 * u + sub * OWN + o] * (float)position[AXES ? o : 0]));
#pragma unroll
                    for (int y = UNITS; y < 32; y <<= 1) angle = fmaxf(angle, __shfl_xor_sync(kFull, angle, y));
                    off = kOff + angle * 8.9e-16f;
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
                // (rows that become codes: all lanes of the warp, which may have to work together)
                if constexpr (FOUR) {
                    if (!__any_sync(kFull, head >= 0 && (kind == 0 || id[c] >= 0))) continue;
                    if (head < 0 || (kind > 0 && id[c] < 0)) xr[c] = yr[c] = make_uint4(0u, 0u, 0u, 0u);
                } else if (head < 0 || (kind > 0 && id[c] < 0)) {
                    continue;
                }
                float x[8], y[8];
                bf16x8_to_f32(xr[c], x);
                bf16x8_to_f32(yr[c], y);
                float size = 0.f;  // of the lane's operands: pairs' |x| + |y| at most
                if constexpr (FOUR) {
                    if (turned && kind == 1) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) size = fmaxf(size, fabsf(x[e]) + fabsf(y[e]));
                        if (a.layout == MKV_ROPE_INTERLEAVED) size *= 2.f;  // (pairs lie within x and within y)
                    }
                }
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
                    if (FOUR && head < 0) continue;
                    uint8_t *dst = a.Q_out + 2 * ((int64_t)t * a.q_heads + head) * D;
                    st_v4(dst + 2 * d0, pack8(x));
                    st_v4(dst + 2 * d1, pack8(y));
                    continue;
                }
                if constexpr (FOUR) {
                    const float inv = kind == 1 ? a.k_inv : a.v_inv, inv6 = kind == 1 ? a.k_inv6 : a.v_inv6;
                    const int halves = a.rot_dim / 16;
                    const bool split = kind == 1 && turned && a.layout == MKV_ROPE_HALF;  // two eights, two groups
                    uint32_t sx, sy, wx, wy;
                    for (int exact = 0;; ++exact) {
                        const float mx = largest8(x), my = largest8(y);
                        float gx = max_nan(mx, my), gy = gx, ex = exact ? 0.f : size * fabsf(a.factor) * off, ey = ex;
                        if (kind == 1 && a.layout == MKV_ROPE_HALF) {
                            const int ox = other_eight(u, halves), oy = other_eight(halves + u, halves), at = lane - u;
                            const int lx = at + (ox & 31) % UNITS, ly = at + (oy & 31) % UNITS;
                            const float xx = __shfl_sync(kFull, mx, lx), xy = __shfl_sync(kFull, my, lx);
                            const float yx = __shfl_sync(kFull, mx, ly), yy = __shfl_sync(kFull, my, ly);
                            const float fx = __shfl_sync(kFull, ex, lx), fy = __shfl_sync(kFull, ex, ly);
                            if (split) {
                                gx = max_nan(mx, ox < 32 ? xx : xy);
                                gy = max_nan(my, oy < 32 ? yx : yy);
                                ey = fmaxf(ex, fy);
                                ex = fmaxf(ex, fx);
                            }
                        }
                        // (2^-21: the roundings of the product)
                        const uint32_t ends_x = f32x2_to_e4m3(max_nan(gx - ex, 0.f) * inv6, (gx + ex) * inv6);
                        const uint32_t ends_y = f32x2_to_e4m3(max_nan(gy - ey, 0.f) * inv6, (gy + ey) * inv6);
                        sx = ends_x & 0xFFu;
                        sy = ends_y & 0xFFu;
                        const float rx = code_factor(sx, inv), ry = code_factor(sy, inv);
                        if (kind == 2 || exact) {
                            wx = codes8(x, rx);
                            wy = codes8(y, ry);
                            break;
                        }
                        bool unsure = sx != ends_x >> 8 || sy != ends_y >> 8;
                        wx = codes8_within(x, rx, ex, unsure);
                        wy = codes8_within(y, ry, ey, unsure);
                        if (!__any_sync(kFull, turned && unsure)) {
                            if (!turned) {
                                wx = codes8(x, rx);
                                wy = codes8(y, ry);
                            }
                            break;
                        }
                        float p[8], q[8];
                        rotate_exactly<D>(a, t, xr[c], yr[c], p, q);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[e] = turned ? p[e] : x[e];
                            y[e] = turned ? q[e] : y[e];
                        }
                    }
                    if (head < 0 || id[c] < 0) continue;
                    uint8_t *page = (kind == 1 ? a.k : a.v) + (int64_t)id[c] * (D * 9 / 16 << a.page_shift);
                    const int row = slot[c] & (a.page_size - 1);
                    *reinterpret_cast<uint32_t *>(page + row * (D / 2) + d0 / 2) = wx;
                    *reinterpret_cast<uint32_t *>(page + row * (D / 2) + d1 / 2) = wy;
                    uint8_t *scales = page + (D / 2 << a.page_shift) + row * (D / 16);
                    if (d0 % 16 == 0) scales[d0 / 16] = (uint8_t)sx;
                    if (d1 % 16 == 0) scales[d1 / 16] = (uint8_t)sy;
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

template <bool FOUR, bool AXES>
const void *rope_fn(int head_dim)
{
    return head_dim == 64    ? (const void *)k_rope_append<64, FOUR, AXES>
           : head_dim == 128 ? (const void *)k_rope_append<128, FOUR, AXES>
           : head_dim == 256 ? (const void *)k_rope_append<256, FOUR, AXES>
                             : nullptr;
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t st)
{
    const bool axes = a.n_axes > 0;
    const void *fn = a.es ? (axes ? rope_fn<false, true>(a.head_dim) : rope_fn<false, false>(a.head_dim))
                          : (axes ? rope_fn<true, true>(a.head_dim) : rope_fn<true, false>(a.head_dim));
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
