// What the two forms of mkv_paged_attention share (internal): tiles of packed
// rows, the line of key blocks and its cut into one part per CTA, and the
// bookkeeping that lets the parts of a cut tile be joined.
//
// The rows (new token, query head of the KV head's group) of a list are packed
// token by token into tiles; a tile walks the blocks of KEYS keys that any of
// its rows sees. The blocks of all tiles of all lists form one line, cut into
// one part per CTA (mkv_line.h: equal parts, or nearly equal ones of whole
// tiles): no CTA idles behind a long list or an uneven number of tiles. A tile
// that is cut leaves its parts (O before the division, m, l) in the workspace,
// at most two per CTA, and they are joined in order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "mkv_device.cuh"
#include "mkv_line.h"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

__device__ __forceinline__ uint32_t saddr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Next to E4M3 keys the queries run as fp16, which takes one conversion per two
// codes where bf16 would take five instructions: a row of queries is scaled by
// the power of two that brings its largest magnitude into [1, 2). Elements
// from 2^-14 of that on keep all their bits; smaller ones are off by at most
// 2^-25 of the largest. E: the biased exponent of the largest magnitude (at
// least 2^-63: smaller queries make no difference to any score, and the
// factor that takes the scaling back stays far from the smallest numbers).
__device__ __forceinline__ int row_exponent(float largest)
{
    return min(max((int)(__float_as_uint(largest) >> 23), 64), 253);
}
__device__ __forceinline__ float down_by(int E) { return __uint_as_float((uint32_t)(254 - E) << 23); }  // 2^(127 - E)
__device__ __forceinline__ float up_by(int E) { return __uint_as_float((uint32_t)E << 23); }            // 2^(E - 127)

struct Tile {
    int b, j, n, L, row0, rows;  // batch row, head, new tokens, list length, first packed row, rows
    int end;                     // keys from here on are visible to no row
    int sink_blocks, win_block, blocks;  // blocks of keys: [0, sink_blocks) and from win_block on; in all
};

// Tile `at` (list-major); rows 0 where there is nothing to do.
template <int KEYS>
__device__ __forceinline__ Tile make_tile(const AttnArgs &a, int at, int tile_rows, bool report)
{
    Tile t;
    const int list = a.by_tiles(at), tile = at - list * a.tiles;
    t.b = a.by_heads(list);
    t.j = list - t.b * a.heads;
    t.row0 = tile * tile_rows;
    t.rows = t.blocks = t.sink_blocks = t.win_block = t.end = 0;
    const int lo = a.q_start[t.b], hi = a.q_start[t.b + 1];
    t.n = hi - lo;
    t.L = a.lens[list];
    if (lo < 0 || hi < lo || hi > a.n_tokens || t.n > a.max_q) {
        if (report) atomicOr(a.status, MKV_DEV_BAD_TOKENS);
        return t;
    }
    if (t.L < 0 || t.L > a.max_len) {
        if (report) atomicOr(a.status, MKV_DEV_BAD_SEQ_LEN);
        return t;
    }
    t.rows = max(0, min(tile_rows, t.n * a.group - t.row0));
    if (t.rows == 0) return t;
    const int p_lo = t.L - t.n + a.by_group(t.row0), p_hi = t.L - t.n + a.by_group(t.row0 + t.rows - 1);
    t.end = max(0, p_hi + 1);
    const int all = (t.end + KEYS - 1) / KEYS;
    if (a.window > 0) {
        const int start = max(0, p_lo - a.window + 1);  // the first key inside any row's window
        t.win_block = min(start / KEYS, all);
        t.sink_blocks = min((min(a.sinks, t.end) + KEYS - 1) / KEYS, t.win_block);
    }
    t.blocks = t.sink_blocks + all - t.win_block;
    return t;
}

template <int KEYS>
__device__ __forceinline__ int block_key(const Tile &t, int blk)
{
    return (blk < t.sink_blocks ? blk : blk - t.sink_blocks + t.win_block) * KEYS;
}

// Units of a tile on the line: its blocks; one for a tile whose rows see nothing.
__device__ __forceinline__ int units_of(const Tile &t) { return t.rows > 0 ? max(t.blocks, 1) : 0; }

// The reference point m of a row's weights 2^(x - m): its running maximum,
// which may lag by 2^8 (weights stay below 256, and rescaling O is rare), less
// kBase. Weights next to E4M3 values are fp16, which rounds what is below 2^-25
// to 0: put 2^7 higher they are at most 2^15, still in range, and what is lost,
// while the sum l in fp32 keeps it, is below 2^-32 of the maximum each (without,
// a flat tail of a million keys could lose 3% of the output).
template <int ES>
constexpr float kBase = ES == 1 ? 7.f : 0.f;
template <int ES>
constexpr float kLag = 8.f + kBase<ES>;

// Two weights rounded for the product with V: to bf16, the MMA's type next to
// bf16 values; to fp16 (11 bits) next to E4M3 ones, which fp16 holds exactly.
// (Scores from 2^24 on, whose steps are whole powers of two, may come out above
// 2^16: they saturate, so that nothing turns infinite that was not.)
template <int ES>
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi)
{
    if constexpr (ES == 2) return pack_bf16(lo, hi);
    uint32_t v;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}

// What a row's sum l of weights makes of it. l is 0 only for a row that has seen
// nothing (or scores of -inf alone); a NaN among its scores (queries may hold
// anything) makes l NaN, also where the maximum, which passes over NaN, is
// still -inf. Such a row's O and lse are NaN; no part of it may pass as empty.
__device__ __forceinline__ float inverse_sum(float l, float v_scale) { return l == 0.f ? 0.f : v_scale / l; }
__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * CUDART_LN2_F;
}

// A CTA's walk over its part of the line.
struct Walk {
    int tile, left;  // the next tile, units left
    int skip;        // units of that tile that belong to the CTA before
    int begin;       // the unit of the line that this CTA's part begins with
    bool have;       // t is that tile already
    Tile t;
    int first, last, units;  // units [first, last) of the tile's
    template <int KEYS>
    __device__ __forceinline__ bool next(const AttnArgs &a, int tile_rows)
    {
        if (left <= 0) return false;
        const int n_tiles = a.batch * a.heads * a.tiles;
        for (;; ++tile) {
            if (tile >= n_tiles) return false;
            if (!have) t = make_tile<KEYS>(a, tile, tile_rows, false);
            have = false;
            units = units_of(t);
            if (units > skip) break;
            skip -= units;  // (0 units: nothing to do)
        }
        first = skip;
        last = min(units, first + left);
        left -= last - first;
        skip = 0;
        ++tile;
        return true;
    }
    __device__ __forceinline__ bool whole() const { return first == 0 && last == units; }
    // blocks [from(), to()) of the segment
    __device__ __forceinline__ int from() const { return min(first, t.blocks); }
    __device__ __forceinline__ int to() const { return min(last, t.blocks); }
};

// This CTA's part of the line; every thread of the CTA must call it. (The host
// has checked that the line's length fits 32 bits.) mkv_line.h has the rule.
struct LineScratch {
    int sum[32], rest[32], live[32];
    LineCut cut;
    int off;   // where the tile begins that holds the first unit of this CTA's equal part
    Walk walk;
};
constexpr int kLineShifts = kPlanSms + 1;
// shift: kLineShifts integers of shared memory, by how much each part's begin
// would move; free again after the caller's next barrier.
template <int KEYS, int THREADS>
__device__ __forceinline__ Walk cut_line(const AttnArgs &a, int tile_rows, LineRule rule, LineScratch &s, int *shift)
{
    constexpr int WARPS = THREADS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tiles = a.batch * a.heads * a.tiles;
    for (int x = threadIdx.x; x < kLineShifts; x += THREADS) shift[x] = 0;
    // the first THREADS tiles, one per thread, and the sum of the others
    Tile t;
    int mine = 0, rest = 0, live = 0;
    if ((int)threadIdx.x < n_tiles) {
        t = make_tile<KEYS>(a, threadIdx.x, tile_rows, blockIdx.x == 0);
        mine = units_of(t);
        live = mine > 0;
    }
    for (int x = threadIdx.x + THREADS; x < n_tiles; x += THREADS) {
        const int u = units_of(make_tile<KEYS>(a, x, tile_rows, blockIdx.x == 0));
        rest += u;
        live += u > 0;
    }
    auto scan = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    int upto = scan(mine);
    if (n_tiles > THREADS) rest = __reduce_add_sync(kFull, rest);
    live = __reduce_add_sync(kFull, live);
    if (lane == 31) {
        s.sum[warp] = upto;
        s.rest[warp] = rest;
        s.live[warp] = live;
    }
    __syncthreads();
    int before = 0, units = 0, tiles = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        before += i < warp ? s.sum[i] : 0;
        units += s.sum[i];
        tiles += s.live[i];
    }
    int seen = units;  // in the tiles looked at so far
    if (n_tiles > THREADS)
        for (int i = 0; i < WARPS; ++i) units += s.rest[i];
    const LineCut cut = LineCut::make(units, tiles, (int)gridDim.x, rule);
    const int me = (int)blockIdx.x, u0 = cut.begin(me), u1 = cut.begin(me + 1);
    const bool move = cut.hopeful();
    if (threadIdx.x == 0) s.cut = cut;
    // The thread whose tile holds the part's first unit, and those whose tiles hold cuts that may move.
    auto look = [&](int x, int off) {
        if (mine == 0) return;
        if (off <= u0 && u0 < off + mine) {
            s.off = off;
            s.walk.tile = x;
            s.walk.t = t;
        }
        if (move && cut.movable(mine))
            for (int c = cut.part_from(off); c < cut.parts; ++c) {
                const int u = cut.begin(c);
                if (u >= off + mine) break;
                shift[c] = LineCut::moved(u, off, mine) - u;
            }
    };
    look(threadIdx.x, before + upto - mine);
    for (int x0 = THREADS; x0 < n_tiles && (move ? seen < units : seen <= u0); x0 += THREADS) {
        const int x = x0 + threadIdx.x;
        mine = 0;
        if (x < n_tiles) {
            t = make_tile<KEYS>(a, x, tile_rows, false);
            mine = units_of(t);
        }
        upto = scan(mine);
        __syncthreads();
        if (lane == 31) s.sum[warp] = upto;
        __syncthreads();
        before = seen;
        for (int i = 0; i < WARPS; ++i) {
            before += i < warp ? s.sum[i] : 0;
            seen += s.sum[i];
        }
        look(x, before + upto - mine);
    }
    __syncthreads();
    int begin = u0, end = u1;
    if (move) {
        int longest = 0;
        for (int c = lane; c < cut.parts; c += 32)
            longest = max(longest, cut.begin(c + 1) + shift[c + 1] - cut.begin(c) - shift[c]);
        if (cut.fits(__reduce_max_sync(kFull, longest))) {
            begin += shift[me];
            end += shift[me + 1];
        }
    }
    Walk w = s.walk;  // (of no use where the part is empty)
    w.have = begin < s.off + units_of(w.t);
    w.tile += w.have ? 0 : 1;
    w.skip = w.have ? begin - s.off : 0;
    w.begin = begin;
    w.left = end - begin;
    return w;
}

// The CTA whose part holds the first or last unit of a cut tile: the one whose
// equal part does. (A cut that moves goes no further than the ends of its tile,
// which is not cut then.)
__device__ __forceinline__ int cta_of(int unit, const LineScratch &s) { return s.cut.part_of(unit); }

// What the joining kernel needs of each CTA.
struct LineInfo {
    int32_t open_tile;  // the tile whose first part is this CTA's last segment, -1: none
    int32_t ends;       // this CTA's first segment continues a tile and ends it
};

// The workspace's part of a segment that is not a whole tile, of `rows` rows.
__device__ __forceinline__ int64_t part_row(const Walk &w, int rows)
{
    return ((int64_t)blockIdx.x * 2 + (w.first > 0 ? 0 : 1)) * rows;
}

// Notes a segment in the CTA's entry (one thread).
__device__ __forceinline__ void note_segment(const Walk &w, LineInfo &info)
{
    if (w.first > 0 && w.last == w.units) info.ends = 1;
    if (w.first == 0 && w.last < w.units) info.open_tile = w.tile - 1;
}

// The tile that CTA c0 opened, -1 when none; c1 is the last CTA with a part of
// it. For a whole warp. The parts: c0's second, then the first of c0 + 1 .. c1.
__device__ __forceinline__ int opened_tile(const LineInfo *__restrict__ info, int c0, int ctas, int &c1)
{
    const int lane = threadIdx.x & 31;
    // this CTA's entry and, in the same round trip, those of the 32 after it
    const int tile = info[c0].open_tile;
    int ends = c0 + 1 + lane < ctas ? info[c0 + 1 + lane].ends : 1;
    if (tile < 0) return -1;
    c1 = c0 + 1;
    for (;;) {
        const unsigned hit = __ballot_sync(kFull, ends != 0);
        if (hit) {
            c1 += __ffs(hit) - 1;
            break;
        }
        c1 += 32;
        ends = c1 + lane < ctas ? info[c1 + lane].ends : 1;
    }
    c1 = min(c1, ctas - 1);
    return tile;
}

// Rows r0 .. r0 + J - 1 of a tile (of ROWS rows) whose parts the CTAs c0 .. c1
// left (c0's second, the first of the others): a warp, the loads of U parts in
// flight. Other CTAs wrote them, maybe in this launch: loads through L2.
template <int D, int ROWS, int J, int U>
__device__ __forceinline__ void join_rows(const AttnArgs &a, const Tile &t, int c0, int c1, int r0)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float sum[J][E], l[J], M[J];
#pragma unroll
    for (int x = 0; x < J; ++x) {
        l[x] = 0.f;
        M[x] = -CUDART_INF_F;
#pragma unroll
        for (int e = 0; e < E; ++e) sum[x][e] = 0.f;
    }
    for (int s0 = c0; s0 <= c1; s0 += U) {
        float2 ml[U][J], v[U][J][E / 2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u;
#pragma unroll
            for (int x = 0; x < J; ++x) {
                ml[u][x] = make_float2(-CUDART_INF_F, 0.f);
                if (s > c1 || r0 + x >= t.rows) continue;
                const int64_t at = ((int64_t)s * 2 + (s == c0 ? 1 : 0)) * ROWS + r0 + x;
                ml[u][x] = __ldcg(a.part_ml + at);
                const float2 *src = reinterpret_cast<const float2 *>(a.part_o + at * D + lane * E);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) v[u][x][e] = __ldcg(src + e);
            }
        }
#pragma unroll
        for (int x = 0; x < J; ++x) {
            float best = M[x];
#pragma unroll
            for (int u = 0; u < U; ++u) best = fmaxf(best, ml[u][x].x);
            const float f0 = M[x] == -CUDART_INF_F ? 0.f : exp2_approx(M[x] - best);
            M[x] = best;
            l[x] *= f0;
#pragma unroll
            for (int e = 0; e < E; ++e) sum[x][e] *= f0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (ml[u][x].y == 0.f) continue;  // none, or it saw nothing
                const float f = exp2_approx(ml[u][x].x - M[x]);
                l[x] += f * ml[u][x].y;
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    sum[x][2 * e] += f * v[u][x][e].x;
                    sum[x][2 * e + 1] += f * v[u][x][e].y;
                }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < J; ++x) {
        if (r0 + x >= t.rows) break;
        const float inv = inverse_sum(l[x], a.v_scale);
        const int R = t.row0 + r0 + x, i = a.by_group(R), head = t.j * a.group + R - i * a.group;
        const int64_t token = (int64_t)a.q_start[t.b] + i;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.O + 2 * (token * a.o_stride + (int64_t)head * D + lane * E));
#pragma unroll
        for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16(sum[x][2 * e] * inv, sum[x][2 * e + 1] * inv);
        if (lane == 0 && a.lse) a.lse[token * a.q_heads + head] = log_sum(M[x], l[x]);
    }
}

}  // namespace
}  // namespace mkv
