// sm_103a attention of a step's few new tokens over 4-bit pages (the form of
// mkv_paged_attention for lists with few query rows; see mkv_attention.cu for
// the definition, mkv_attention_chunk.cu for the form for many).
//
// A cached element is code * scale, exact in fp16, so the arithmetic is that of
// E4M3 caches: queries as fp16 scaled by a power of two per row, fp16 weights,
// fp32 sums. What is new is the work per byte: 1 KB of HBM holds 1820 elements,
// each to be expanded (a conversion for two codes, a product with the scale for
// two) before a tensor core can take it. So the cached side is the MMA's A
// operand, 16 keys or 16 dims per instruction, and the rows are its 8 columns:
//     S^T = K Q^T   (16 keys x 8 rows),   O^T += V^T P^T   (16 dims x 8 rows):
// a tile of 8 rows takes half the instructions that 16 rows would, and a tile of
// 16 expands every element once for both halves. Keys of a lane's fragment are
// the bytes that it loads: dims may be contracted in any order, so a lane's dims
// are those of one 16-byte load and the queries follow; likewise a lane's dims
// of V are consecutive ones, all under one scale per key.
//
// The split of work is that of the other form: tiles of packed rows, the line of
// key blocks cut over 152 CTAs, a ring of cp.async stages per warp, the parts of
// cut tiles joined by the CTA that comes last (mkv_attention.cuh).
//
// Measured (128 dims, group 4): 64 rows x 8 heads of 4K-16K tokens 143 us (floor 111),
// two rows of 120K-131K tokens x 10 heads 69 (53), one row of 2K tokens x 8 heads 9. 64
// dims: the 64 rows 92 (56), the two rows 47 (27); 256 dims, 32 rows 132 (111). Group 16: 64
// rows 193 at 128 dims, 122 at 64, 32 rows 183 at 256. 128 rows x 8 heads of 200-300 tokens
// 31, 35 and 51 at 64, 128 and 256 dims (floors 3, 6, 11). At 128 dims the
// copies alone take 117 us of the 143, the arithmetic alone 129. What bounds the
// arithmetic: 16 keys are 225 instructions without their copies -- 64 conversions
// and 64 products at two a cycle and SM, 16 MMAs -- and of their mix an SM executes 2.1
// a cycle, with 12 warps or with 16 (4 conversions, 4 products and an MMA that depends on
// them take 5 cycles by themselves); 108 cycles where the bytes of the 16 keys take
// 102. Steps on the way (64 rows): 16 keys per step and lookups and
// addresses for each, 199 us, of its 410 instructions 107 for the copies; 32 keys, pages looked
// up for 16 steps at once, one address per lane 154; a lane's places computed once 146; 12
// warps instead of 16 143. 64 keys per step 142 (and one row of 2K tokens 10 instead of 9);
// 14 warps, which share the SM's four parts unevenly, 157; 8 warps 157.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include "mkv_attention.cuh"
#include "mkv_device.cuh"
#include "mkv_e2m1.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kKeys = 16;  // keys of an MMA's rows: they lie in one page
constexpr float kTop = 32768.f;        // 2^kLag<1>
constexpr float kNothing = -3e38f;  // the reference point of a row that has seen nothing (finite: no case of its own)
// Cuts move to tiles' ends for a slack of 3 blocks (of 256 to 512 keys; see mkv_line.h).
// Measured (us, cuts never move / slack 1 / 3 / 6), 128 dims: 384 lists of 1536 keys 32.1 /
// 32.4 / 29.4 / 28.9, 228 of 1536 19.9 / 19.7 / 21.3 / 21.1, lists of 192-768 keys: 152 of them
// 16.3 / 17.1 / 14.1 / 14.1, 456 28.1 / 29.2 / 25.9 / 25.8; 256 dims, 228 lists of 4 blocks 30.9 /
// 30.4 / 33.6 / 33.6, 152 of 2 to 8 blocks 32.9 / 33.1 / 33.6 / 36.1. Where lists are even and fill the
// CTAs as they are, looking for moves costs 0.5 to 1 us. Over 125 mixes of 152 to 608 lists the
// four take 1.4, 3.8, 2.8 and 3.1% more than the best of them: 3 is for short lists of
// uneven length, which compressed caches have.
constexpr LineRule kLine = {1, 3, 3};

// Shape of one instantiation: head dims, rows of a tile.
template <int D, int R>
struct Attend4 {
    static constexpr int WARPS = D == 256 ? (R == 8 ? 12 : 8) : D == 128 ? 12 : 16;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int NK = 2;                   // groups of 16 keys of a warp's step
    static constexpr int KT = NK * kKeys;          // its keys
    static constexpr int KEYS = WARPS * KT;        // keys per block of the CTA
    static constexpr int CB = D / 2, SB = D / 16;  // bytes of a row's codes and scales
    static constexpr int CODES = kKeys * CB, SCALES = kKeys * SB;  // ... of 16 keys
    static constexpr int HALF = CODES + SCALES, GROUP = 2 * HALF, STAGE = NK * GROUP;
    static constexpr int STAGES = D == 256 && R == 8 ? 2 : 3;
    static constexpr int RING = STAGES * STAGE;    // per warp
    static constexpr int OS = D + 4;               // floats between a result's rows
    static constexpr int MERGE = WARPS * R * OS * 4;
    static constexpr int SMEM = WARPS * RING > MERGE ? WARPS * RING : MERGE;
    static constexpr int NR = R / 8;               // column tiles of rows
    static constexpr bool EARLY = R == 8 && D <= 128;  // queries of the next tile loaded ahead: else registers spill
    static constexpr int KW = D / 32;              // 32-bit words of codes per lane and key, K
    static constexpr int VW = D / 64 ? D / 64 : 1; // ... V: 8 dims to a word
};

// 16 bytes to shared memory, if `real`.
__device__ __forceinline__ void cp16_if(bool real, uint32_t dst, const void *src)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %2, 0; @p cp.async.cg.shared.global [%0], [%1], 16; }" ::"r"(dst), "l"(src),
                 "r"((uint32_t)real)
                 : "memory");
}
// 16 bytes, of which the first n come from src, the others are zeros.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr)
{
    uint32_t v;
    asm volatile("{ .reg .u16 h; ld.shared.u16 h, [%1]; cvt.u32.u16 %0, h; }" : "=r"(v) : "r"(addr));
    return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w)
{
    if constexpr (N == 1) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
        const uint4 v = lds16(addr);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

// Where 16-byte chunk c of row r of a step's codes lies. K: a quarter-warp reads
// two rows of 64 bytes, or half of two rows of 128, one of which has its halves
// exchanged. V: the lanes that load together have the rows 0, 2, 4, 6 (or the
// odd ones) and the same quarter of each, which have to be 8 distinct chunks
// modulo 128 bytes.
template <int D>
__device__ __forceinline__ uint32_t k_at(int r, int c)
{
    return (uint32_t)(r * (D / 32) + (D == 256 ? c ^ (r & 1) << 2 : c)) * 16u;
}
template <int D>
__device__ __forceinline__ uint32_t v_at(int r, int c)
{
    if constexpr (D == 64) return (uint32_t)((r ^ (r >> 2 & 1)) * 2 + c) * 16u;
    if constexpr (D == 128) return (uint32_t)((r * 4 ^ (r >> 1 & 1) << 2) + (c ^ (r >> 2 & 1) << 1)) * 16u;
    return (uint32_t)(r * 8 + (c ^ (r >> 1 & 3) << 1)) * 16u;
}

template <int D, int R>
__global__ void __launch_bounds__(Attend4<D, R>::THREADS, 1)
k_attend_e2m1(const __grid_constant__ AttnArgs a)
{
    using A = Attend4<D, R>;
    constexpr int NR = A::NR, KW = A::KW, VW = A::VW;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineScratch s_line;
    __shared__ int s_shift[kLineShifts];
    __shared__ int4 s_join[2];  // tiles to join: tile, first and last CTA with a part
    __shared__ Walk s_next;     // after the next step of the walk, and whether it found a tile
    __shared__ bool s_more;
    __shared__ float2 s_ml[A::WARPS][R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
    Walk w = cut_line<A::KEYS, A::THREADS>(a, R, kLine, s_line, s_shift);
    int at_unit = w.begin;  // of the line
    if (threadIdx.x < 2) s_join[threadIdx.x].x = -1;
    // this lane's dims of a key: word x holds 8 of them
    auto k_dim = [&](int x) -> int {
        return D == 64 ? 16 * tq + 8 * x : D == 128 ? 32 * tq + 8 * x : 128 * (x / 4) + 32 * tq + 8 * (x % 4);
    };
    // What this lane copies of every step: chunks of one group's codes, and one chunk of its keys' or values' scales.
    // Groups of 16 rows of the pool are numbered: number x has its codes at x CODES + (its page) PS SB, its scales at
    // x SCALES + (its page + 1) PS CB, with PS rows in a page.
    constexpr int LG = 32 / A::NK, PER_LANE = A::CODES / 16 / LG, SC = A::SCALES / 16;
    constexpr int SC_ROUNDS = (2 * SC * A::NK + 31) / 32, SC_STEP = 32 / (2 * SC);  // copies of scales, and groups of one
    const int own = lane / LG, chunk0 = lane % LG, sc_own = lane / (2 * SC), sc_kv = lane / SC % 2, sc_chunk = lane % SC;
    const uint8_t *k_lane = a.k + chunk0 * 16, *v_lane = a.v + chunk0 * 16;
    const uint8_t *sc_lane = (sc_kv ? a.v : a.k) + (A::CB << a.page_shift) + sc_chunk * 16;
    const int group_shift = a.page_shift - 4;  // groups of a page
    const uint32_t page_scales = A::SB << a.page_shift, page_codes = A::CB << a.page_shift;
    // Offsets in a stage of what it copies, and of what it loads (a key's or value's words, its scales). A copy's
    // further chunks follow at fixed distances, those of V from one of a few places in turn; so do the keys of a load.
    constexpr int STEP_ROWS = LG / (D / 32), TURNS = D == 64 ? 1 : 8 / STEP_ROWS < PER_LANE ? 8 / STEP_ROWS : PER_LANE;
    const uint32_t k_to = own * A::GROUP + k_at<D>(chunk0 / (D / 32), chunk0 % (D / 32));
    const uint32_t sc_to = sc_own * A::GROUP + sc_kv * A::HALF + A::CODES + sc_chunk * 16;
    uint32_t v_to[TURNS], v_from[2];
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
        v_to[i] = own * A::GROUP + A::HALF + v_at<D>(chunk0 / (D / 32) + STEP_ROWS * i, chunk0 % (D / 32)) - i * LG * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v_from[i] = A::HALF + (D == 64    ? v_at<D>(2 * tq + i, gr >> 2) + 4 * (gr & 3)
                               : D == 128 ? v_at<D>(2 * tq + i, gr >> 1) + 8 * (gr & 1)
                                          : v_at<D>(2 * tq + i, gr));
    const uint32_t k_from = D == 64 ? k_at<D>(gr, tq >> 1) + 8 * (tq & 1) : k_at<D>(gr, tq);
    const uint32_t k_from2 = D == 256 ? k_at<D>(gr, tq + 4) : 0u;
    const uint32_t ks_from = A::CODES + gr * A::SB + (D == 64 ? tq : 2 * tq);
    const uint32_t vs_from = A::HALF + A::CODES + 2 * tq * A::SB + (D == 64 ? gr >> 1 : D == 128 ? gr : 2 * gr);
    // The tile at hand: its blocks, its first and last row's places in the list, its queries as loaded, the groups of
    // keys to copy next. All of it is fetched before the last tile's results are put together.
    int first = 0, last = 0, qrow0 = 0, p_lo = 0, p_hi = 0;
    const int32_t *table = nullptr;
    uint4 raw[NR][KW];
    uint32_t groups = 0, next = 0;
    constexpr int STEPS = 32 / A::NK;  // groups are looked up for so many steps at once
    const uint32_t ring = saddr(smem) + warp * A::RING;
    auto key0 = [&](int blk) -> int { return block_key<A::KEYS>(w.t, blk) + warp * A::KT; };
    // Lane y: the group that it numbers, y groups on from block blk0 -- its number in the pool and, above bit 26, how
    // many of its keys there are: none where no row sees any of them, or where the page is outside the pool.
    auto lookup = [&](int blk0) -> uint32_t {
        const int blk = blk0 + lane / A::NK;
        if (blk >= last) return 0u;
        const int s = key0(blk) + lane % A::NK * kKeys;
        if (s >= w.t.end || (a.window > 0 && s + kKeys - 1 <= p_lo - a.window && s >= a.sinks)) return 0u;
        const int id = table[s >> a.page_shift];
        if ((uint32_t)id >= (uint32_t)a.n_pages) {
            atomicOr(a.status, MKV_DEV_BAD_PAGE);
            return 0u;
        }
        return (uint32_t)((id << group_shift) + ((s & (a.page_size - 1)) >> 4)) | (uint32_t)min(kKeys, w.t.end - s) << 26;
    };
    // The copies of a step whose groups are `at` lanes on. Scales of keys that
    // are not there arrive as zeros, which makes their elements zeros: nothing
    // else has to be told apart, codes are finite whatever they are.
    auto issue = [&](uint32_t dst, uint32_t groups, int at) {
        const uint32_t mine = __shfl_sync(kFull, groups, at + own), x = mine & 0x3FFFFFFu;
        const uint64_t off = (uint64_t)x * A::CODES + (uint64_t)(x >> group_shift) * page_scales;
        const uint8_t *ks = k_lane + off, *vs = v_lane + off;
        const bool real = mine >> 26 != 0;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            cp16_if(real, dst + k_to + i * LG * 16, ks + i * LG * 16);
            cp16_if(real, dst + v_to[i % TURNS] + i * LG * 16, vs + i * LG * 16);
        }
#pragma unroll
        for (int i = 0; i < SC_ROUNDS; ++i) {
            const uint32_t sc = __shfl_sync(kFull, groups, (at + sc_own + i * SC_STEP) & 31), y = sc & 0x3FFFFFFu;
            if (SC * 2 * A::NK >= 32 || sc_own < A::NK)
                cp16(dst + sc_to + i * SC_STEP * A::GROUP,
                     sc_lane + ((uint64_t)y * A::SCALES + (uint64_t)(y >> group_shift) * page_codes),
                     min(max((int)(sc >> 26) * A::SB - 16 * sc_chunk, 0), 16));
        }
    };

    auto load_queries = [&]() {  // column gr of each column tile, this lane's dims
        const Tile &t = w.t;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int Rq = t.row0 + min(8 * n + gr, t.rows - 1), i = a.by_group(Rq), g = Rq - i * a.group;
            const uint8_t *src = a.Q + 2 * ((int64_t)(qrow0 + i) * a.q_stride + (int64_t)(t.j * a.group + g) * D);
#pragma unroll
            for (int x = 0; x < KW; ++x) raw[n][x] = *reinterpret_cast<const uint4 *>(src + 2 * k_dim(x));
        }
    };
    auto begin_tile = [&]() {
        const Tile &t = w.t;
        first = w.from();
        last = w.to();
        table = a.table + ((int64_t)t.b * a.heads + t.j) * a.max_pages;
        qrow0 = a.q_start[t.b];
        p_lo = t.L - t.n + a.by_group(t.row0);
        p_hi = t.L - t.n + a.by_group(t.row0 + t.rows - 1);
        if (A::EARLY) load_queries();
        groups = lookup(first);
        next = lookup(first + STEPS);
    };
    bool more = w.next<A::KEYS>(a, R);
    if (more) begin_tile();
    while (more) {
        const Tile &t = w.t;
        if (!A::EARLY) load_queries();

        // queries: column gr of each column tile, this lane's dims, as fp16 with a power of two taken out. (They take
        // the scale's sign, and a factor of zero becomes the smallest normal number: zero times a masked score's
        // -inf would be NaN.)
        uint32_t q[NR][2 * KW][2];
        float sc[NR][2];  // of this lane's columns of scores, 2 tq and 2 tq + 1
        int p[NR][2];     // their places in the list
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float m = 0.f;
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                float f[8];
                bf16x8_to_f32(raw[n][x], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
            }
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
            const int E = row_exponent(m);
            const float down = a.scale_log2 < 0.f ? -down_by(E) : down_by(E);
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                float f[8];
                bf16x8_to_f32(raw[n][x], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) q[n][2 * x + (e >> 1)][e & 1] = pack_f16(f[2 * e] * down, f[2 * e + 1] * down);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sc[n][c] = fmaxf(fabsf(a.scale_log2) * up_by(__shfl_sync(kFull, E, (2 * tq + c) * 4)), FLT_MIN);
                p[n][c] = t.L - t.n + a.by_group(t.row0 + min(8 * n + 2 * tq + c, t.rows - 1));
            }
        }
        float o[D / 16][NR][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int n = 0; n < NR; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m[n][0] = m[n][1] = kNothing;
            l[n][0] = l[n][1] = 0.f;
        }

        int at = 0;  // the next step to copy: its place among `groups`
        auto copy_step = [&](uint32_t dst) {
            issue(dst, groups, at);
            cp_commit();
            at += A::NK;
        };
        const uint32_t ring_end = ring + A::RING;
#pragma unroll
        for (int s = 0; s < A::STAGES - 1; ++s) copy_step(ring + s * A::STAGE);  // (past the last block: zeros alone)
        if (warp == 0) {  // where the walk goes on, while the first keys are on their way
            Walk x = w;
            const bool found = x.next<A::KEYS>(a, R);
            if (lane == 0) {
                s_next = x;
                s_more = found;
            }
        }
        uint32_t stage = ring, fill = ring_end - A::STAGE;
        for (int blk = first; blk < last; ++blk, fill = stage, stage = stage + A::STAGE == ring_end ? ring : stage + A::STAGE) {
            copy_step(fill);
            if (at == 32) {
                at = 0;
                groups = next;
                next = lookup(blk + A::STAGES + STEPS);
            }
            cp_wait<A::STAGES - 1>();
            __syncwarp();

            // scores: rows of an MMA are the keys gr and gr + 8 of a group
            float s[A::NK][NR][4];
            constexpr int WB = KW < 4 ? KW : 4;  // words of a load
#pragma unroll
            for (int g = 0; g < A::NK; ++g) {
                const uint32_t group = stage + g * A::GROUP;
#pragma unroll
                for (int n = 0; n < NR; ++n) s[g][n][0] = s[g][n][1] = s[g][n][2] = s[g][n][3] = 0.f;
#pragma unroll
                for (int x0 = 0; x0 < KW; x0 += WB) {
                    uint32_t kw[2][WB], sk[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        lds_words<WB>(group + (x0 ? k_from2 : k_from) + 8 * h * A::CB, kw[h]);
                        const uint32_t sc_at = group + ks_from + 8 * h * A::SB + 2 * x0;
                        if constexpr (D == 64) {
                            const uint32_t f = e4m3x2_to_f16x2(lds_u8(sc_at));
                            sk[h][0] = sk[h][1] = __byte_perm(f, 0, 0x1010);
                        } else {
                            const uint32_t f = e4m3x2_to_f16x2(lds_u16(sc_at));
                            sk[h][0] = __byte_perm(f, 0, 0x1010);
                            sk[h][1] = __byte_perm(f, 0, 0x3232);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < WB; ++x) {
                        uint32_t f[2][4];
                        e2m1x8_to_f16(kw[0][x], f[0]);
                        e2m1x8_to_f16(kw[1][x], f[1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t k[4] = {mul_f16x2(f[0][2 * e], sk[0][x >> 1]), mul_f16x2(f[1][2 * e], sk[1][x >> 1]),
                                                   mul_f16x2(f[0][2 * e + 1], sk[0][x >> 1]),
                                                   mul_f16x2(f[1][2 * e + 1], sk[1][x >> 1])};
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                const uint32_t(&b)[2] = q[n][2 * (x0 + x) + e];
                                mma_f16(s[g][n], k, b[0], b[1]);
                            }
                        }
                    }
                }
            }

            // Weights 2^(s c - m) of the visible keys. Where a lane's sum of a row's is
            // above 2^kLag, a score may be that far above the row's reference point.
            const int k0 = key0(blk), k1 = k0 + A::KT - 1;
            const bool whole = k1 <= p_lo && (a.window <= 0 || k0 > p_hi - a.window || k1 < a.sinks);
            float d[A::NK][NR][4], sum[NR][2];
            auto weights = [&]() {
                float top = 0.f;
#pragma unroll
                for (int n = 0; n < NR; ++n) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        sum[n][c] = 0.f;
#pragma unroll
                        for (int x = 0; x < 2 * A::NK; ++x) {
                            const int g = x >> 1, e = 2 * (x & 1) + c;
                            d[g][n][e] = exp2_approx(fmaf(s[g][n][e], sc[n][c], -m[n][c]));
                            sum[n][c] += d[g][n][e];
                        }
                        top = fmaxf(top, sum[n][c]);
                    }
                }
                return top;
            };
            if (!whole)
#pragma unroll
                for (int g = 0; g < A::NK; ++g)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = k0 + g * kKeys + gr + 8 * (e >> 1), at_key = p[n][e & 1];
                            const bool seen = (key <= at_key) & ((a.window <= 0) | (key > at_key - a.window) | (key < a.sinks));
                            s[g][n][e] = seen ? s[g][n][e] : -CUDART_INF_F;
                        }
            if (__any_sync(kFull, weights() > kTop)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x = -CUDART_INF_F;
#pragma unroll
                        for (int g = 0; g < A::NK; ++g) x = fmaxf(x, fmaxf(s[g][n][c] * sc[n][c], s[g][n][2 + c] * sc[n][c]));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                        const float to = fmaxf(m[n][c], x - kBase<1>);
                        const float f = exp2_approx(m[n][c] - to);  // (0 for a row that had seen nothing)
                        m[n][c] = to;
                        l[n][c] *= f;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[i][n][c] *= f;
                            o[i][n][2 + c] *= f;
                        }
                    }
                weights();
            }
            uint32_t pw[A::NK][NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                l[n][0] += sum[n][0];
                l[n][1] += sum[n][1];
#pragma unroll
                for (int g = 0; g < A::NK; ++g) {
                    pw[g][n][0] = transpose8(pack_weights<1>(d[g][n][0], d[g][n][1]));
                    pw[g][n][1] = transpose8(pack_weights<1>(d[g][n][2], d[g][n][3]));
                }
            }

            // O^T: rows of an MMA are two of this lane's D / 8 consecutive dims, its contraction 16 keys
#pragma unroll
            for (int g = 0; g < A::NK; ++g) {
                const uint32_t group = stage + g * A::GROUP;
                uint32_t vw[4][VW], sv[2][2], sb[4];  // keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    lds_words<VW>(group + v_from[y & 1] + 8 * (y >> 1) * A::CB, vw[y]);
                    const uint32_t sc_at = group + vs_from + ((y & 1) + 8 * (y >> 1)) * A::SB;
                    sb[y] = D == 256 ? lds_u16(sc_at) : lds_u8(sc_at);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sv[h][0] = e4m3x2_to_f16x2(__byte_perm(sb[2 * h], sb[2 * h + 1], 0x40));
                    sv[h][1] = D == 256 ? e4m3x2_to_f16x2(__byte_perm(sb[2 * h], sb[2 * h + 1], 0x51)) : sv[h][0];
                }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    uint32_t ev[2][4], od[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // two keys' codes of the same dim side by side: even dims, odd dims
                        const uint32_t u = vw[2 * h][x], v = vw[2 * h + 1][x];
                        e2m1x8_to_f16((u & 0x0F0F0F0Fu) | (v << 4 & 0xF0F0F0F0u), ev[h]);
                        e2m1x8_to_f16((u >> 4 & 0x0F0F0F0Fu) | (v & 0xF0F0F0F0u), od[h]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int hf = x * 8 + 2 * e >= 16 ? 1 : 0;  // the second scale of a lane's 32 dims
                        const uint32_t f[4] = {mul_f16x2(ev[0][e], sv[0][hf]), mul_f16x2(od[0][e], sv[0][hf]),
                                               mul_f16x2(ev[1][e], sv[1][hf]), mul_f16x2(od[1][e], sv[1][hf])};
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma_f16(o[4 * x + e][n], f, pw[g][n][0], pw[g][n][1]);
                    }
                }
            }
            __syncwarp();  // the stage is free for the next copies
        }
        cp_wait<0>();
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[n][c] += __shfl_xor_sync(kFull, l[n][c], 4);
                l[n][c] += __shfl_xor_sync(kFull, l[n][c], 8);
                l[n][c] += __shfl_xor_sync(kFull, l[n][c], 16);
            }
        __syncthreads();  // every ring is done with: the warps' results take its place
        float *mine = reinterpret_cast<float *>(smem) + warp * R * A::OS;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * n + 2 * tq + c;
                if (gr == 0) s_ml[warp][r] = make_float2(m[n][c], l[n][c]);
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
                    *reinterpret_cast<float4 *>(mine + r * A::OS + gr * (D / 8) + 2 * i) =
                        make_float4(o[i][n][c], o[i][n][2 + c], o[i + 1][n][c], o[i + 1][n][2 + c]);
            }
        struct {
            int rows, row0, j, qrow0, first, last, units, tile;
            int64_t part;
            bool whole;
        } const done = {t.rows, t.row0, t.j, qrow0, w.first, w.last, w.units, w.tile - 1, part_row(w, R), w.whole()};
        more = s_more;
        w = s_next;
        if (more) begin_tile();
        __syncthreads();
        for (int x = threadIdx.x; x < done.rows * (D / 4); x += A::THREADS) {
            const int r = x / (D / 4), c = x % (D / 4);
            float M = -CUDART_INF_F;
#pragma unroll
            for (int y = 0; y < A::WARPS; ++y) M = fmaxf(M, s_ml[y][r].x);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float total = 0.f;
#pragma unroll
            for (int y = 0; y < A::WARPS; ++y) {
                const float2 ml = s_ml[y][r];
                const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - M);
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + (y * R + r) * A::OS + 4 * c);
                sum.x += f * v.x;
                sum.y += f * v.y;
                sum.z += f * v.z;
                sum.w += f * v.w;
                total += f * ml.y;
            }
            if (!done.whole) {
                const int64_t part = done.part + r;
                reinterpret_cast<float4 *>(a.part_o)[part * (D / 4) + c] = sum;
                if (c == 0) a.part_ml[part] = make_float2(M, total);
                continue;
            }
            const float inv = inverse_sum(total, a.v_scale);
            const int Rq = done.row0 + r, i = a.by_group(Rq), head = done.j * a.group + Rq - i * a.group;
            *reinterpret_cast<uint2 *>(a.O + 2 * ((int64_t)(done.qrow0 + i) * a.o_stride + (int64_t)head * D + 4 * c)) =
                make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
            if (c == 0 && a.lse) a.lse[(int64_t)(done.qrow0 + i) * a.q_heads + head] = log_sum(M, total);
        }
        __syncthreads();  // the next segment's copies may overwrite the results
        if (!done.whole && threadIdx.x == 0) {
            // Parts of a tile count themselves in a byte of the workspace's head,
            // which the last one takes back to zero; it joins the parts below.
            const int unit0 = at_unit - done.first, c0 = cta_of(unit0, s_line), c1 = cta_of(unit0 + done.units - 1, s_line);
            uint32_t *word = a.counts + c0 / 4;
            const int shift = c0 % 4 * 8;
            __threadfence();
            if ((int)(atomicAdd(word, 1u << shift) >> shift & 255u) == c1 - c0) {
                atomicSub(word, (uint32_t)(c1 - c0 + 1) << shift);
                s_join[done.first > 0 ? 0 : 1] = make_int4(done.tile, c0, c1, 0);
            }
        }
        at_unit += done.last - done.first;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {  // (a CTA's first segment and its last one)
        const int4 j = s_join[k];
        if (j.x < 0) continue;
        __threadfence();
        const Tile t = make_tile<A::KEYS>(a, j.x, R, false);
        for (int r = warp; r < t.rows; r += A::WARPS) join_rows<D, R, 1, 8>(a, t, j.y, j.z, r);
    }
}

template <int D, int R>
cudaError_t launch_one(const AttnArgs &a, cudaStream_t st)
{
    using A = Attend4<D, R>;
    cudaError_t e = cudaFuncSetAttribute(k_attend_e2m1<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
    if (e != cudaSuccess) return e;
    k_attend_e2m1<D, R><<<a.ctas, A::THREADS, A::SMEM, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Rows of a tile: 8 where a list has no more (a decode step of up to 8 query
// heads per KV head), else 16.
int e2m1_tile_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_attend_e2m1(const AttnArgs &a, cudaStream_t st)
{
    const bool small = a.tile_rows == 8;
    switch (a.head_dim) {
    case 64: return small ? launch_one<64, 8>(a, st) : launch_one<64, 16>(a, st);
    case 128: return small ? launch_one<128, 8>(a, st) : launch_one<128, 16>(a, st);
    case 256: return small ? launch_one<256, 8>(a, st) : launch_one<256, 16>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace mkv
