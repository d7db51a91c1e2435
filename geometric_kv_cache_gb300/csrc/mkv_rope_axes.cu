// sm_103a rotary positions with several axes (mkv_rope_append_axes), and rotary
// appends into 4-bit pages (both calls).
//
// Pair i of a row turns by positions[axes[i]][t] * inv_freq[i]; everything else is
// as in mkv_rope.cu, whose angles -- 64-bit fractions of a turn -- and results these
// are. The arithmetic is less than the bytes only if little else is executed: a
// warp takes a token (or a share of its heads), walks its query, key and value
// heads in three loops with the next heads' rows on their way, two elements per
// floating-point instruction, and looks its 32 heads' places in the pages up at
// once, a lane each.
//
// 4-bit pages. A lane has two eights of a row's dims: one group of 16 or, where
// pairs lie half a row apart, one each of two groups, whose largest elements meet
// over shuffles. Codes of keys have to be those of the exact rotation. Its fp32
// form is off by up to kOff of a pair's |x| + |y| -- the angle's rounding pi 2^-24, its
// sine's and cosine's 2^-23, the products' and the sum's 3 2^-24, the exact value's
// own 2^-24 -- and 2^-50 of the angle, whose fraction of a turn comes from 64-bit
// floating point. (|x| + |y| is at most sqrt(2) times that of the rotated pair over
// |factor|, so rotated pairs tell it.) Where that could change a code or a scale,
// because the ends of the stretch round differently, the element (for a scale, those
// that can be the largest) is worked out in 64 bits, at 1 / 64 of the 32-bit rate.
//
// Measured (16384 tokens of 32 + 2 x 8 heads of 128 dims, three axes): bf16 68 us, 0.88 of
// the floor, E4M3 65 (54), 4-bit 72 (52): 36M instructions, where the form that mkv_rope.cu
// has, extended, took 107 us and 62M. Groups of query heads on their way together (bf16 /
// 4-bit, whose 64-bit work then took it 5 us longer): four 68 / 77 us, two 72 / 84, eight, which
// spill, 79 / 88; two with three CTAs per SM 84 / 85. Chunks of 7 rows, 2300 tokens, 4-bit: 20 us, of which 64-bit work costs 2; as one
// 64-bit rotation of all the warp's heads it cost 6, in a chain of 62 cycles per operation.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "mkv_device.cuh"
#include "mkv_e2m1.cuh"
#include "mkv_pages.h"
#include "mkv_rope.cuh"

namespace mkv {
namespace {

using namespace dev;

constexpr int kBatch = 4;  // groups of query heads on their way together
constexpr float kOff = 6.5e-7f, kOffRotated = 1.4143f;  // (the parts named above: 5.5e-7)

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c; "
        "mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 two(const float (&f)[8], int i) { return make_float2(f[2 * i], f[2 * i + 1]); }
__device__ __forceinline__ void put(float (&f)[8], int i, float2 v)
{
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
}

// This lane's 16 dims (x, y), eight pairs, turned: x c - y s and x s + y c, in this
// order of roundings. HALF: pairs (x[e], y[e]); else neighbours, x the first four.
template <bool HALF>
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8])
{
    if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 sn = two(s, i), cn = two(c, i), p = two(x, i), q = two(y, i);
            put(x, i, fma2(p, cn, mul2(q, make_float2(-sn.x, -sn.y))));
            put(y, i, fma2(p, sn, mul2(q, cn)));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float p0 = fmaf(x[2 * e], c[e], -(x[2 * e + 1] * s[e])), q0 = fmaf(x[2 * e], s[e], x[2 * e + 1] * c[e]);
            const float p1 = fmaf(y[2 * e], c[4 + e], -(y[2 * e + 1] * s[4 + e]));
            const float q1 = fmaf(y[2 * e], s[4 + e], y[2 * e + 1] * c[4 + e]);
            x[2 * e] = p0;
            x[2 * e + 1] = q0;
            y[2 * e] = p1;
            y[2 * e + 1] = q1;
        }
    }
}

// Cosine and sine, times `factor`, of the 64-bit product position * freq. The
// angle in turns is a product with 1 / (2 pi) of 106 bits, of which whole quarters
// drop out exactly; for what is left, at most pi / 4, the Taylor sums up to the 16th
// power (the next terms are below 2^-54), by pairs of terms: a 64-bit operation waits
// 62 cycles for the one before it, so the depth counts. 45 operations in a row
// (sincospi) take 2800 cycles for one element.
__device__ __forceinline__ double2 turn_exactly(int position, float freq, float factor)
{
    const double angle = (double)position * (double)freq;
    const double hi = angle * 0.15915494309189535, lo = fma(angle, 0.15915494309189535, -hi) + angle * -9.839338337591243e-18;
    const double quarters = rint(4.0 * hi);
    const double x = (fma(quarters, -0.25, hi) + lo) * 6.283185307179586477, z = x * x, z2 = z * z, z4 = z2 * z2;
    const double s = fma(z4, fma(z2, fma(z, 1.0 / 355687428096000.0, -1.0 / 1307674368000.0), fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0)),
                         fma(z2, fma(z, 1.0 / 362880.0, -1.0 / 5040.0), fma(z, 1.0 / 120.0, -1.0 / 6.0)));
    const double c = fma(z4, fma(z2, fma(z, 1.0 / 20922789888000.0, -1.0 / 87178291200.0), fma(z, 1.0 / 479001600.0, -1.0 / 3628800.0)),
                         fma(z2, fma(z, 1.0 / 40320.0, -1.0 / 720.0), fma(z, 1.0 / 24.0, -1.0 / 2.0)));
    const double sn = fma(x * z, s, x), cn = fma(z, c, 1.0);
    const int q = (int)(long long)quarters & 3;
    const double cq = q & 1 ? sn : cn, sq = q & 1 ? cn : sn;
    return make_double2((q == 1 || q == 2 ? -cq : cq) * factor, (q >= 2 ? -sq : sq) * factor);
}

// One rotated element as 64-bit arithmetic gives it, rounded once to fp32: of pair
// (c0, c1), the first or second. Not inlined: it is rare.
__device__ __noinline__ float exact_element(const RopeArgs &a, int t, int pair, float c0, float c1, bool second)
{
    int axis = a.n_axes > 0 ? a.axes[pair] : 0;
    if ((uint32_t)axis >= (uint32_t)a.n_axes) axis = 0;
    const double2 turn = turn_exactly(a.positions[(int64_t)axis * a.n_tokens + t], a.inv_freq[pair], a.factor);
    return (float)(second ? c0 * turn.y + c1 * turn.x : c0 * turn.x - c1 * turn.y);
}

// Element i of eight bf16.
__device__ __forceinline__ float element(uint4 v, int i)
{
    const uint32_t w = i < 4 ? (i < 2 ? v.x : v.y) : (i < 6 ? v.z : v.w);
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
}

// Element i of a lane's rotated x or y, worked out exactly.
template <bool HALF>
__device__ __forceinline__ float exact_of(const RopeArgs &a, int t, int u, uint4 xr, uint4 yr, bool is_y, int i)
{
    const uint4 row = is_y ? yr : xr;
    const int pair = HALF ? 8 * u + i : 8 * u + (is_y ? 4 : 0) + (i >> 1);
    const float c0 = HALF ? element(xr, i) : element(row, i & 6), c1 = HALF ? element(yr, i) : element(row, i | 1);
    return exact_element(a, t, pair, c0, c1, HALF ? is_y : (i & 1) != 0);
}

// The codes w of a lane's x or y with those of the elements that `unsure` marks, in
// the lowest bits of their codes, settled.
template <bool HALF>
__device__ __forceinline__ uint32_t settle(const RopeArgs &a, int t, int u, uint4 xr, uint4 yr, bool is_y, float r,
                                           uint32_t w, uint32_t unsure)
{
    for (; unsure; unsure &= unsure - 1) {
        const int bit = __ffs(unsure) - 1;
        const float f[8] = {__fmul_rn(exact_of<HALF>(a, t, u, xr, yr, is_y, bit >> 2), r)};
        w = (w & ~(15u << bit)) | (plain_zeros(f32x8_to_e2m1(f)) & 15u) << bit;
    }
    return w;
}

// The largest magnitude of a lane's x or y (v, as rotated in fp32), worked out
// exactly; only elements from `least` on can be it.
template <bool HALF>
__device__ __forceinline__ float exact_largest(const RopeArgs &a, int t, int u, uint4 xr, uint4 yr, bool is_y,
                                               const float (&v)[8], float least)
{
    uint32_t can = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) can |= fabsf(v[i]) >= least ? 1u << i : 0u;
    float m = 0.f;
    for (; can; can &= can - 1) m = fmaxf(m, fabsf(exact_of<HALF>(a, t, u, xr, yr, is_y, __ffs(can) - 1)));
    return m;
}

// The rotated values of this lane's 16 dims (x, y as loaded) as 64-bit
// arithmetic gives them, rounded once to fp32, for a whole warp: a lane works out
// the angles that it works out in 32 bits, the others come from their lanes. For
// groups far beyond the largest scale, infinities and NaN; not inlined.
template <int D, bool HALF>
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
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double cn = __shfl_sync(kFull, mine[e % OWN].x, u + (e / OWN) * UNITS);
        const double sn = __shfl_sync(kFull, mine[e % OWN].y, u + (e / OWN) * UNITS);
        const int i = 2 * e & 7;
        const float c0 = HALF ? p[e] : e < 4 ? p[i] : q[i], c1 = HALF ? q[e] : e < 4 ? p[i + 1] : q[i + 1];
        const float r0 = (float)(c0 * cn - c1 * sn), r1 = (float)(c0 * sn + c1 * cn);
        if (HALF) {
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

// Eight values x, times r.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float r)
{
    float t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) put(t, i, mul2(two(x, i), make_float2(r, r)));
    return plain_zeros(f32x8_to_e2m1(t));
}

// Codes of a lane's eight rotated values t = x r, each known to within `off` times
// its pair's |x| + |other|. unsure: the lowest bits of the codes that another x
// within that could change.
__device__ __forceinline__ uint32_t codes_within(const float (&x)[8], const float (&other)[8], float r, float off, uint32_t &unsure)
{
    float lo[8], hi[8];
    const float o = off * r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = two(x, i), w = two(other, i), t = mul2(v, make_float2(r, r));
        const float2 size = add2(make_float2(fabsf(v.x), fabsf(v.y)), make_float2(fabsf(w.x), fabsf(w.y)));
        // (2^-20: the roundings of x r and of the sums below, values up to 8)
        const float2 e = fma2(size, make_float2(o, o), make_float2(9.5367432e-7f, 9.5367432e-7f));
        put(lo, i, add2(t, make_float2(-e.x, -e.y)));
        put(hi, i, add2(t, e));
    }
    const uint32_t l = f32x8_to_e2m1(lo), h = f32x8_to_e2m1(hi);
    const uint32_t d = l ^ h;  // (ends with different signs are both zero: see small enough, below)
    unsure = (d | d >> 1 | d >> 2) & 0x11111111u;
    return plain_zeros(l);
}

template <int D, int ES, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 2)
k_rope_axes(const __grid_constant__ RopeArgs a, int parts)
{
    constexpr int UNITS = D / 16, HS = 32 / UNITS, OWN = 8 / HS;
    const int lane = threadIdx.x & 31, u = lane % UNITS, sub = lane / UNITS;
    const int halves = a.rot_dim / 16;
    const int gq = (a.q_heads + HS - 1) / HS, gk = (a.heads + HS - 1) / HS;  // groups of HS heads
    const bool turned = u < halves;  // this lane's dims of a query or key rotate: pairs 8u .. 8u + 7
    const bool apart = HALF && turned;
    const int d0 = apart ? 8 * u : 16 * u, d1 = apart ? 8 * halves + 8 * u : 16 * u + 8;
    // Every row's range, whether a token is found in it or not.
    for (int64_t i = (int64_t)(gridDim.x - 1 - blockIdx.x) * kRopeThreads + threadIdx.x; i < a.batch;
         i += (int64_t)gridDim.x * kRopeThreads) {
        const int lo = a.q_start[i], hi = a.q_start[i + 1];
        if (lo < 0 || hi < lo || hi > a.n_tokens) atomicOr(a.status, MKV_DEV_BAD_TOKENS);
    }
    // the pairs whose angles this lane works out: fractions of a turn per position, and where their positions are
    unsigned long long frac[OWN];
    const int32_t *place[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        frac[o] = 0;
        place[o] = a.positions;
        if (turned) {
            const int pair = 8 * u + sub * OWN + o, axis = a.n_axes > 0 ? a.axes[pair] : 0;
            if ((uint32_t)axis < (uint32_t)max(a.n_axes, 1)) place[o] += (int64_t)axis * a.n_tokens;
            else atomicOr(a.status, MKV_DEV_BAD_AXIS);
            double turns = (double)a.inv_freq[pair] * 0.15915494309189533577;  // 1 / (2 pi)
            turns -= floor(turns);
            frac[o] = __double2ull_rn(turns * 18446744073709551616.0);  // 2^64
        }
    }
    const int64_t warps = (int64_t)gridDim.x * kRopeWarps, items = (int64_t)a.n_tokens * parts;
    for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5); item < items; item += warps) {
        const int t = (int)(item / parts), part = (int)(item - (int64_t)t * parts);
        // groups are numbered queries, keys, values; this warp has every parts-th
        const int k0 = part + (max(gq - part, 0) + parts - 1) / parts * parts - gq;
        const int v0 = part + (max(gq + gk - part, 0) + parts - 1) / parts * parts - gq - gk;
        const uint8_t *q_row = a.Q + 2 * ((int64_t)t * a.q_stride + (int64_t)sub * D);
        const uint8_t *k_row = a.K + 2 * ((int64_t)t * a.k_stride + (int64_t)sub * D);
        const uint8_t *v_row = a.V + 2 * ((int64_t)t * a.v_stride + (int64_t)sub * D);
        struct Rows {
            uint4 x, y;
        };
        // two eights of head g HS + sub; zeros where there is none
        auto load = [&](const uint8_t *row, int g, int heads, int e0, int e1) -> Rows {
            Rows r = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
            if (g * HS + sub < heads) {
                const uint8_t *src = row + (int64_t)g * (2 * HS * D);
                r.x = *reinterpret_cast<const uint4 *>(src + 2 * e0);
                r.y = *reinterpret_cast<const uint4 *>(src + 2 * e1);
            }
            return r;
        };
        Rows q_rows[kBatch];
        auto load_queries = [&](int g) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) q_rows[i] = load(q_row, g + i * parts, a.q_heads, d0, d1);
        };
        load_queries(part);
        Rows k_next = load(k_row, k0, a.heads, d0, d1), v_next = load(v_row, v0, a.heads, 16 * u, 16 * u + 8);

        // the token's row, places and angles, while its data is on the way
        int position[OWN];
#pragma unroll
        for (int o = 0; o < OWN; ++o) position[o] = place[o][t];
        const int b = row_of_token(a.q_start, a.batch, t);
        if (b < 0) continue;  // a token of no row
        const int lo = a.q_start[b], hi = a.q_start[b + 1];
        // (a refused row: no list is that long, so its queries alone are written)
        const int left = lo < 0 || hi > a.n_tokens ? INT_MAX : hi - t;
        const bool stores = k0 < gk || v0 < gk;  // of keys or values
        // lane y's spot (row of the pool, -1: none) of head base + y
        const int32_t *lens = a.lens + (int64_t)b * a.heads;
        int base = 0, spot = -1, len = stores && lane < a.heads ? lens[lane] : 0;
        auto find_spots = [&]() {
            spot = -1;
            if (base + lane >= a.heads) return;
            if (len < left || len > (a.max_pages << a.page_shift)) {
                if (left != INT_MAX) atomicOr(a.status, MKV_DEV_BAD_SEQ_LEN);
                return;
            }
            const int slot = len - left;
            const int id = a.table[((int64_t)b * a.heads + base + lane) * a.max_pages + (slot >> a.page_shift)];
            if ((uint32_t)id >= (uint32_t)a.n_pages) atomicOr(a.status, MKV_DEV_BAD_PAGE);
            else spot = (id << a.page_shift) + (slot & (a.page_size - 1));
        };
        float cs[OWN], sn[OWN], angle = 0.f;
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const long long phase = (long long)(frac[o] * (unsigned long long)(long long)position[o]);
            sincospif((float)phase * 1.0842021724855044e-19f, &sn[o], &cs[o]);  // 2 x phase / 2^64 half turns
            cs[o] *= a.factor;
            sn[o] *= a.factor;
            if (ES == 0 && turned) angle = fmaxf(angle, fabsf(a.inv_freq[8 * u + sub * OWN + o] * (float)position[o]));
        }
        if (stores) find_spots();
        float c[8], s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] = __shfl_sync(kFull, cs[e % OWN], u + (e / OWN) * UNITS);
            s[e] = __shfl_sync(kFull, sn[e % OWN], u + (e / OWN) * UNITS);
        }
        // head g HS + sub's spot, for the whole warp (32 heads at a time: their groups never straddle)
        auto spot_of = [&](int g) -> int {
            if ((g * HS & ~31) != base) {
                base = g * HS & ~31;
                len = base + lane < a.heads ? lens[base + lane] : 0;
                find_spots();
            }
            const int at = __shfl_sync(kFull, spot, (g * HS + sub) & 31);
            return g * HS + sub < a.heads ? at : -1;
        };

        uint8_t *q_out = a.Q_out + 2 * ((int64_t)t * a.q_heads + sub) * D;
        for (int g0 = part; g0 < gq; g0 += kBatch * parts) {
            if (g0 > part) load_queries(g0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int g = g0 + i * parts;
                if (g * HS + sub >= a.q_heads) continue;
                float x[8], y[8];
                bf16x8_to_f32(q_rows[i].x, x);
                bf16x8_to_f32(q_rows[i].y, y);
                if (turned) rotate<HALF>(x, y, c, s);
                uint8_t *dst = q_out + (int64_t)g * (2 * HS * D);
                st_v4(dst + 2 * d0, pack8(x));
                st_v4(dst + 2 * d1, pack8(y));
            }
        }

        // a row of a key or value (e0, e1: its dims) as the pages hold it
        auto store = [&](uint8_t *pool, int at, const float (&x)[8], const float (&y)[8], int e0, int e1, float inv) {
            if (at < 0) return;
            uint8_t *dst = pool + (int64_t)at * (D * ES);
            if constexpr (ES == 2) {
                st_v4(dst + 2 * e0, pack8(x));
                st_v4(dst + 2 * e1, pack8(y));
            } else {
                *reinterpret_cast<uint2 *>(dst + e0) = quant8(x, inv);
                *reinterpret_cast<uint2 *>(dst + e1) = quant8(y, inv);
            }
        };
        auto store4 = [&](uint8_t *pool, int at, uint32_t wx, uint32_t wy, uint32_t sx, uint32_t sy, int e0, int e1) {
            if (at < 0) return;
            const int row = at & (a.page_size - 1);
            uint8_t *page = pool + (int64_t)(at >> a.page_shift) * (D * 9 / 16 << a.page_shift), *codes = page + row * (D / 2);
            uint8_t *scales = page + (D / 2 << a.page_shift) + row * (D / 16);
            if (e1 == e0 + 8) {
                *reinterpret_cast<uint2 *>(codes + e0 / 2) = make_uint2(wx, wy);
                scales[e0 / 16] = (uint8_t)sx;
                return;
            }
            *reinterpret_cast<uint32_t *>(codes + e0 / 2) = wx;
            *reinterpret_cast<uint32_t *>(codes + e1 / 2) = wy;
            if (e0 % 16 == 0) scales[e0 / 16] = (uint8_t)sx;
            if (e1 % 16 == 0) scales[e1 / 16] = (uint8_t)sy;
        };

        float off = 0.f;  // how far a rotated value may be off, of its rotated pair
        int lx = 0, ly = 0, ox = 0, oy = 0;
        if constexpr (ES == 0) {
            // the largest angle of the lane's pairs
#pragma unroll
            for (int y = UNITS; y < 32; y <<= 1) angle = fmaxf(angle, __shfl_xor_sync(kFull, angle, y));
            off = (kOff + angle * 8.9e-16f) * kOffRotated;
            if constexpr (HALF) {
                ox = other_eight(u, halves);
                oy = other_eight(halves + u, halves);
                lx = lane - u + (ox & 31) % UNITS;
                ly = lane - u + (oy & 31) % UNITS;
            }
        }
        for (int g = k0; g < gk; g += parts) {
            const Rows r = k_next;
            k_next = load(k_row, g + parts, a.heads, d0, d1);
            const int at = spot_of(g);
            float x[8], y[8];
            bf16x8_to_f32(r.x, x);
            bf16x8_to_f32(r.y, y);
            if (turned) rotate<HALF>(x, y, c, s);
            if constexpr (ES != 0) {
                store(a.k, at, x, y, d0, d1, a.k_inv);
            } else {
                uint32_t sx, sy, wx, wy;
                for (int exact = 0;; ++exact) {
                    // largest elements of the two groups, and by how much they may be off
                    const float mx = largest8(x), my = largest8(y);
                    float gx = max_nan(mx, my), gy = gx, ex = turned && !exact ? 2.f * gx * off : 0.f, ey = ex;
                    // (x and y: two eights of one group, or of two whose other eights lie in other lanes)
                    auto others = [&](float p, float q, float &of_x, float &of_y) {
                        const float xx = __shfl_sync(kFull, p, lx), xy = __shfl_sync(kFull, q, lx);
                        const float yx = __shfl_sync(kFull, p, ly), yy = __shfl_sync(kFull, q, ly);
                        of_x = ox < 32 ? xx : xy;
                        of_y = oy < 32 ? yx : yy;
                    };
                    if constexpr (HALF) {
                        float of_x, of_y;
                        others(mx, my, of_x, of_y);
                        const float fx = __shfl_sync(kFull, ex, lx), fy = __shfl_sync(kFull, ex, ly);
                        if (apart) {
                            gx = max_nan(mx, of_x);
                            gy = max_nan(my, of_y);
                            ey = fmaxf(ex, fy);
                            ex = fmaxf(ex, fx);
                        }
                    }
                    const uint32_t ends_x = f32x2_to_e4m3(max_nan(gx - ex, 0.f) * a.k_inv6, (gx + ex) * a.k_inv6);
                    const uint32_t ends_y = f32x2_to_e4m3(max_nan(gy - ey, 0.f) * a.k_inv6, (gy + ey) * a.k_inv6);
                    sx = ends_x & 0xFFu;
                    sy = ends_y & 0xFFu;
                    const bool doubt_x = sx != ends_x >> 8, doubt_y = sy != ends_y >> 8;
                    float rx = code_factor(sx, a.k_inv), ry = apart ? code_factor(sy, a.k_inv) : rx;
                    if (exact || !__any_sync(kFull, turned)) {
                        wx = codes_of(x, rx);
                        wy = codes_of(y, ry);
                        break;
                    }
                    // Stretches of less than a quarter of a code's least border are told apart below. (Larger ones are of groups
                    // far beyond the largest scale, or of infinities and NaN.)
                    if (!__any_sync(kFull, turned && (!(ex * rx < 0.06f) || !(ey * ry < 0.06f)))) {
                        if (__any_sync(kFull, doubt_x || doubt_y)) {  // scales first
                            float px = doubt_x ? exact_largest<HALF>(a, t, u, r.x, r.y, false, x, gx - 2.f * ex) : 0.f;
                            float py = doubt_y ? exact_largest<HALF>(a, t, u, r.x, r.y, true, y, gy - 2.f * ey) : 0.f;
                            if constexpr (HALF) {
                                float of_x, of_y;
                                others(px, py, of_x, of_y);
                                px = fmaxf(px, apart ? of_x : py);
                                py = fmaxf(py, apart ? of_y : px);
                            } else {
                                px = py = fmaxf(px, py);
                            }
                            if (doubt_x) sx = f32x2_to_e4m3(px * a.k_inv6, 0.f) & 0xFFu;
                            if (doubt_y) sy = f32x2_to_e4m3(py * a.k_inv6, 0.f) & 0xFFu;
                            rx = code_factor(sx, a.k_inv);
                            ry = code_factor(sy, a.k_inv);
                        }
                        uint32_t x_unsure, y_unsure;
                        if constexpr (HALF) {
                            wx = codes_within(x, y, rx, off, x_unsure);
                            wy = codes_within(y, x, ry, off, y_unsure);
                        } else {
                            float x1[8], y1[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                x1[e] = x[e ^ 1];
                                y1[e] = y[e ^ 1];
                            }
                            wx = codes_within(x, x1, rx, off, x_unsure);
                            wy = codes_within(y, y1, ry, off, y_unsure);
                        }
                        if (!turned) {  // (nothing is off)
                            wx = codes_of(x, rx);
                            wy = codes_of(y, ry);
                        } else if (x_unsure | y_unsure) {
                            wx = settle<HALF>(a, t, u, r.x, r.y, false, rx, wx, x_unsure);
                            wy = settle<HALF>(a, t, u, r.x, r.y, true, ry, wy, y_unsure);
                        }
                        break;
                    }
                    float p[8], q[8];
                    rotate_exactly<D, HALF>(a, t, r.x, r.y, p, q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = turned ? p[e] : x[e];
                        y[e] = turned ? q[e] : y[e];
                    }
                }
                store4(a.k, at, wx, wy, sx, sy, d0, d1);
            }
        }
        for (int g = v0; g < gk; g += parts) {
            const Rows r = v_next;
            v_next = load(v_row, g + parts, a.heads, 16 * u, 16 * u + 8);
            const int at = spot_of(g);
            float x[8], y[8];
            bf16x8_to_f32(r.x, x);
            bf16x8_to_f32(r.y, y);
            if constexpr (ES != 0) {
                store(a.v, at, x, y, 16 * u, 16 * u + 8, a.v_inv);
            } else {
                const uint32_t sc = f32x2_to_e4m3(max_nan(largest8(x), largest8(y)) * a.v_inv6, 0.f) & 0xFFu;
                const float f = code_factor(sc, a.v_inv);
                store4(a.v, at, codes_of(x, f), codes_of(y, f), sc, sc, 16 * u, 16 * u + 8);
            }
        }
    }
}

template <int D>
const void *rope_fn(int es, bool half)
{
    return es == 2   ? (half ? (const void *)k_rope_axes<D, 2, true> : (const void *)k_rope_axes<D, 2, false>)
           : es == 1 ? (half ? (const void *)k_rope_axes<D, 1, true> : (const void *)k_rope_axes<D, 1, false>)
                     : (half ? (const void *)k_rope_axes<D, 0, true> : (const void *)k_rope_axes<D, 0, false>);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeArgs &a, cudaStream_t st)
{
    const bool half = a.layout == MKV_ROPE_HALF;
    const void *fn = a.head_dim == 64    ? rope_fn<64>(a.es, half)
                     : a.head_dim == 128 ? rope_fn<128>(a.es, half)
                     : a.head_dim == 256 ? rope_fn<256>(a.es, half)
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
