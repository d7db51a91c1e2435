// sm_103a attention of a step's new tokens over a paged cache
// (mkv_paged_attention): the consumer of the compacted cache ("ManifoldKV:
// Training-Free KV Cache Compression via Euclidean Outlier Detection", ICML
// 2026 poster 62526, abstract: the tokens the cache retains are what later
// queries see).
//
// For the rows (new token i, query head g of the KV head's group) of one list,
// packed 16 to a tile, with scores x_s = scale q.k_s over the visible tokens:
//     m = max x, l = sum 2^(x - m), O = sum 2^(x - m) v / l
// kept as running values over blocks of keys (m, l and O in fp32; a new maximum
// multiplies l and O by 2^(m_old - m_new); any m near the maximum will do, see
// kBase).
//
// This file: the form for few rows, whose bound is the bytes of K and V. A
// tile is 16 rows (the M of mma.sync m16n8k16; a decode step of a group of 4
// fills 4), a block WARPS x KT keys, KT for each warp of the CTA. Every warp
// has its own ring of cp.async stages (16 bytes per lane, the block's page
// entries read one block ahead), so the walk over a tile has no CTA barrier;
// the warps' (m, l, O) meet in shared memory at its end. The line of blocks is
// cut over 152 CTAs (mkv_attention.cuh); of the CTAs with a part of a cut tile
// the one that comes last joins the parts, always in the same order.
//
// Measured: 32 rows of 4K-16K bf16 tokens (8 KV heads of 128 dims, group 4) 200 us,
// 6.4 TB/s, 0.95 of the measured copy rate, 19 such rows 130 us; two rows of 60K-65K
// E4M3 tokens (10 KV heads) 64 us, 5.0 TB/s (55 us without any arithmetic: start,
// first and last copies); one row of 2K tokens 9 us, latency. The first form, with a
// fixed number of parts per list, took 213 us for the 32 rows, 101 for the two and 7
// for the one, which pays for the cut of the line and the join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "mkv_attention.cuh"
#include "mkv_device.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kRows = 16;  // rows per tile (the MMA's M)
constexpr double kAgainBytes = 80e6;  // see takes_chunks
constexpr LineRule kLine = {1, 3, 3};  // see mkv_line.h

// Shape of one instantiation.
template <int D, int ES>
struct Attend {
    // keys per block and warp, and warps: E4M3 blocks have half the bytes for the
    // same arithmetic, which takes more warps to hide (two rows of 60K-65K tokens, 128
    // dims: 12 x 16 keys 63.5 us, 8 x 32 65.1, 16 x 16 64.3; the copies alone take 55)
    static constexpr int KT = ES == 1 || D == 256 ? 16 : 32;
    static constexpr int WARPS = ES == 2 ? 4 : D == 256 ? 8 : 12;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int KEYS = WARPS * KT;            // keys per block of the CTA
    static constexpr int RB = D * ES;                  // bytes per cached row
    static constexpr int CPR = RB / 16;                // 16-byte chunks per row
    static constexpr int HALF = KT * RB;               // bytes of a block's keys
    static constexpr int STAGE = 2 * HALF;
    static constexpr int STAGES = 4 * WARPS * STAGE <= 200 * 1024 ? 4 : 3;  // what shared memory holds
    static constexpr int RING = STAGES * STAGE;        // per warp
    static constexpr int MERGE = WARPS * kRows * D * 4;
    static constexpr int SMEM = WARPS * RING > MERGE ? WARPS * RING : MERGE;
};

// 16 bytes to shared memory; zeros when !real.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Where 16-byte chunk c of row r of a block lies: rows of CPR chunks, chunks
// exchanged so that the eight rows (ldmatrix) or the two rows (16-byte loads
// of E4M3 keys) that one access reads fall into distinct banks.
template <int CPR>
__device__ __forceinline__ uint32_t at_rows8(int r, int c)
{
    return (uint32_t)(r * CPR + (c ^ (CPR >= 8 ? r & 7 : (r >> 1) & 3))) * 16u;
}
template <int CPR>
__device__ __forceinline__ uint32_t at_rows2(int r, int c)
{
    return (uint32_t)(r * CPR + (c ^ (CPR >= 8 ? (r & 1) << 2 : 0))) * 16u;
}

template <int D, int ES>
__global__ void __launch_bounds__(Attend<D, ES>::THREADS, 1)
k_attend(const AttnArgs a)
{
    using A = Attend<D, ES>;
    constexpr int KT = A::KT, NT = KT / 8, KS = D / 16;  // key tiles of 8, dim steps of 16
    constexpr bool Q_REGS = ES == 2 && D <= 128;  // the queries' fragments: in registers, or read from shared memory
    constexpr int QS = D * 2 + 16;                // bytes between rows there: rows fall into distinct banks
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) uint8_t s_q[Q_REGS ? 16 : kRows * QS];
    __shared__ float s_up[kRows];
    __shared__ LineScratch s_line;
    __shared__ int s_shift[kLineShifts];
    __shared__ int4 s_join[2];  // tiles to join: tile, first and last CTA with a part
    __shared__ float2 s_ml[A::WARPS][kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
    Walk w = cut_line<A::KEYS, A::THREADS>(a, kRows, kLine, s_line, s_shift);
    int at_unit = w.begin;  // of the line
    if (threadIdx.x < 2) s_join[threadIdx.x].x = -1;
    while (w.next<A::KEYS>(a, kRows)) {
        const Tile &t = w.t;
        const int first = w.from(), last = w.to();
        const int64_t list = (int64_t)t.b * a.heads + t.j;
        const int32_t *table = a.table + list * a.max_pages;
        const int page_mask = a.page_size - 1;

        // the two rows of this lane: packed row -> (new token, query head)
        const int qrow0 = a.q_start[t.b];
        auto q_row = [&](int r) -> const uint8_t * {
            const int R = t.row0 + min(r, t.rows - 1);
            const int i = a.by_group(R), g = R - i * a.group;
            return a.Q + 2 * ((int64_t)(qrow0 + i) * a.q_stride + (int64_t)(t.j * a.group + g) * D);
        };
        // dims of an A fragment: pairs (2t, 2t + 1) and (2t + 8, 2t + 9) of a step,
        // for E4M3 keys the dims that the lane's 16-byte load holds
        auto q_dim = [&](int k, int hi) -> int {
            return ES == 2 ? k * 16 + 2 * tq + 8 * hi : (k / 4) * 64 + 16 * tq + (k % 4) * 4 + 2 * hi;
        };
        uint32_t q[Q_REGS ? KS : 1][4];
        float sc0 = a.scale_log2, sc1 = a.scale_log2;  // of this lane's two rows of scores
        if constexpr (Q_REGS) {
            const uint8_t *q0 = q_row(gr), *q1 = q_row(gr + 8);
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    q[k][2 * hi] = *reinterpret_cast<const uint32_t *>(q0 + 2 * q_dim(k, hi));
                    q[k][2 * hi + 1] = *reinterpret_cast<const uint32_t *>(q1 + 2 * q_dim(k, hi));
                }
        } else {
            constexpr int LANES = D / 8, PASS = 32 / LANES;  // lanes of a row, rows of a warp's pass
            for (int r0 = warp * PASS; r0 < kRows; r0 += A::WARPS * PASS) {
                const int r = r0 + lane / LANES, x = lane % LANES;
                uint4 v = reinterpret_cast<const uint4 *>(q_row(r))[x];
                if constexpr (ES == 1) {
                    uint32_t w8[4] = {v.x, v.y, v.z, v.w};
                    float m = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(lo_bf16(w8[e])), fabsf(hi_bf16(w8[e]))));
#pragma unroll
                    for (int y = LANES / 2; y; y >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, y));
                    const int E = row_exponent(m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w8[e] = pack_f16(lo_bf16(w8[e]) * down_by(E), hi_bf16(w8[e]) * down_by(E));
                    v = make_uint4(w8[0], w8[1], w8[2], w8[3]);
                    if (x == 0) s_up[r] = up_by(E);
                }
                *reinterpret_cast<uint4 *>(s_q + r * QS + 16 * x) = v;
            }
            __syncthreads();
            if constexpr (ES == 1) {
                sc0 *= s_up[gr];
                sc1 *= s_up[gr + 8];
            }
        }
        // places of the tile's first and last row, and of this lane's two
        const int p_lo = t.L - t.n + a.by_group(t.row0), p_hi = t.L - t.n + a.by_group(t.row0 + t.rows - 1);
        const int p0 = t.L - t.n + a.by_group(t.row0 + min(gr, t.rows - 1));
        const int p1 = t.L - t.n + a.by_group(t.row0 + min(gr + 8, t.rows - 1));

        const uint32_t ring = saddr(smem) + warp * A::RING;
        auto key0 = [&](int blk) -> int { return block_key<A::KEYS>(t, blk) + warp * KT; };
        // the pool row of this lane's key of a block, -1 where no row sees it
        auto lookup = [&](int blk) -> int {
            if (blk >= last || lane >= KT) return -1;
            const int s = key0(blk) + lane;
            if (s >= t.end || (a.window > 0 && s <= p_lo - a.window && s >= a.sinks)) return -1;
            const int id = table[s >> a.page_shift];
            if ((uint32_t)id >= (uint32_t)a.n_pages) {
                atomicOr(a.status, MKV_DEV_BAD_PAGE);
                return -1;
            }
            return (id << a.page_shift) + (s & page_mask);
        };
        auto issue = [&](int stage, int blk, int row) {
            if (blk < last) {
                const uint32_t dst = ring + stage * A::STAGE;
#pragma unroll
                for (int i = 0; i < KT * A::CPR / 32; ++i) {
                    const int o = lane + 32 * i, r = o / A::CPR, c = o % A::CPR;
                    const int src = __shfl_sync(kFull, row, r);
                    const size_t off = (size_t)max(src, 0) * A::RB + c * 16;
                    cp16(dst + (ES == 2 ? at_rows8<A::CPR>(r, c) : at_rows2<A::CPR>(r, c)), a.k + off, src >= 0);
                    cp16(dst + A::HALF + at_rows8<A::CPR>(r, c), a.v + off, src >= 0);
                }
            }
            cp_commit();
        };

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;

        int row = lookup(first);
#pragma unroll
        for (int s = 0; s < A::STAGES - 1; ++s) {
            const int next = lookup(first + s + 1);
            issue(s, first + s, row);
            row = next;
        }
        for (int blk = first, it = 0; blk < last; ++blk, ++it) {
            {
                const int ahead = blk + A::STAGES - 1, next = lookup(ahead + 1);
                issue((it + A::STAGES - 1) % A::STAGES, ahead, row);
                row = next;
            }
            cp_wait<A::STAGES - 1>();
            __syncwarp();
            const uint32_t kb = ring + (it % A::STAGES) * A::STAGE, vb = kb + A::HALF;

            // scores
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
            auto q_frag = [&](int k, uint32_t (&f)[4]) {
                if constexpr (Q_REGS) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = q[k][e];
                } else {
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) {
                        f[2 * hi] = *reinterpret_cast<const uint32_t *>(s_q + gr * QS + 2 * q_dim(k, hi));
                        f[2 * hi + 1] = *reinterpret_cast<const uint32_t *>(s_q + (gr + 8) * QS + 2 * q_dim(k, hi));
                    }
                }
            };
            if constexpr (ES == 2) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t f[4];
                    q_frag(k, f);
#pragma unroll
                    for (int i = 0; i < NT / 2; ++i) {
                        uint32_t b[4];
                        ldsm4(kb + at_rows8<A::CPR>(i * 16 + (lane >> 4) * 8 + (lane & 7), 2 * k + ((lane >> 3) & 1)), b);
                        mma_bf16(s[2 * i], f, b[0], b[1]);
                        mma_bf16(s[2 * i + 1], f, b[2], b[3]);
                    }
                }
            } else {
#pragma unroll
                for (int k4 = 0; k4 < KS / 4; ++k4) {
                    uint32_t kw[NT][4];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 v = lds16(kb + at_rows2<A::CPR>(i * 8 + gr, 4 * k4 + tq));
                        kw[i][0] = v.x;
                        kw[i][1] = v.y;
                        kw[i][2] = v.z;
                        kw[i][3] = v.w;
                    }
                    // four steps' fragments are 32 bytes of each of the lane's rows
                    uint32_t f4[4][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint4 v = lds16(saddr(s_q) + (gr + 8 * h) * QS + 2 * q_dim(4 * k4, 0) + 16 * x);
                            f4[2 * x][h] = v.x;
                            f4[2 * x][2 + h] = v.y;
                            f4[2 * x + 1][h] = v.z;
                            f4[2 * x + 1][2 + h] = v.w;
                        }
                    // (consecutive MMAs add to different tiles of scores)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t(&f)[4] = f4[e];
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            mma_f16(s[i], f, e4m3x2_to_f16x2(kw[i][e] & 0xFFFFu), e4m3x2_to_f16x2(kw[i][e] >> 16));
                    }
                }
            }

            // mask, running maximum, weights
            const int k0 = key0(blk), k1 = k0 + KT - 1;
            const bool whole = k1 <= p_lo && (a.window <= 0 || k0 > p_hi - a.window || k1 < a.sinks);
            float x0 = -CUDART_INF_F, x1 = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = s[i][e] * (e < 2 ? sc0 : sc1);
                    if (!whole) {
                        const int key = k0 + i * 8 + 2 * tq + (e & 1), p = e < 2 ? p0 : p1;
                        const bool seen = (key <= p) & ((a.window <= 0) | (key > p - a.window) | (key < a.sinks));
                        x = seen ? x : -CUDART_INF_F;
                    }
                    s[i][e] = x;
                    if (e < 2) x0 = fmaxf(x0, x);
                    else x1 = fmaxf(x1, x);
                }
            x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, 1));
            x0 = fmaxf(x0, __shfl_xor_sync(kFull, x0, 2));
            x1 = fmaxf(x1, __shfl_xor_sync(kFull, x1, 2));
            if (__any_sync(kFull, x0 - m0 > kLag<ES> || x1 - m1 > kLag<ES>)) {
                const float n0 = fmaxf(m0, x0 - kBase<ES>), n1 = fmaxf(m1, x1 - kBase<ES>);
                // (a row that has seen nothing yet has l = 0 and O = 0: any finite factor)
                const float f0 = m0 == -CUDART_INF_F ? 0.f : exp2_approx(m0 - n0);
                const float f1 = m1 == -CUDART_INF_F ? 0.f : exp2_approx(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= f0;
                    o[i][1] *= f0;
                    o[i][2] *= f1;
                    o[i][3] *= f1;
                }
            }
            const float b0 = m0 == -CUDART_INF_F ? 0.f : m0, b1 = m1 == -CUDART_INF_F ? 0.f : m1;
            uint32_t p[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const float e0 = exp2_approx(s[i][0] - b0), e1 = exp2_approx(s[i][1] - b0);
                const float e2 = exp2_approx(s[i][2] - b1), e3 = exp2_approx(s[i][3] - b1);
                l0 += e0 + e1;
                l1 += e2 + e3;
                p[i][0] = pack_weights<ES>(e0, e1);
                p[i][1] = pack_weights<ES>(e2, e3);
            }
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
                const uint32_t f[4] = {p[2 * kk][0], p[2 * kk][1], p[2 * kk + 1][0], p[2 * kk + 1][1]};
                if constexpr (ES == 2) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t b[4];
                        ldsm4_t(vb + at_rows8<A::CPR>(kk * 16 + (lane & 15), 2 * c + (lane >> 4)), b);
                        mma_bf16(o[2 * c], f, b[0], b[1]);
                        mma_bf16(o[2 * c + 1], f, b[2], b[3]);
                    }
                } else {
                    // a 16-byte chunk holds 16 dims: even dims to one column tile, odd to the next
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t b[4];
                        ldsm4_t(vb + at_rows8<A::CPR>(kk * 16 + (lane & 15), 2 * c + (lane >> 4)), b);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            // (key, dim) bytes 00 01 10 11 to 00 10 | 01 11: the two dims' key pairs
                            const uint32_t v0 = __byte_perm(b[2 * hf], 0, 0x3120), v1 = __byte_perm(b[2 * hf + 1], 0, 0x3120);
                            mma_f16(o[4 * c + 2 * hf], f, e4m3x2_to_f16x2(v0 & 0xFFFFu), e4m3x2_to_f16x2(v1 & 0xFFFFu));
                            mma_f16(o[4 * c + 2 * hf + 1], f, e4m3x2_to_f16x2(v0 >> 16), e4m3x2_to_f16x2(v1 >> 16));
                        }
                    }
                }
            }
            __syncwarp();  // the stage is free for the next copies
        }
        cp_wait<0>();
        l0 += __shfl_xor_sync(kFull, l0, 1);
        l1 += __shfl_xor_sync(kFull, l1, 1);
        l0 += __shfl_xor_sync(kFull, l0, 2);
        l1 += __shfl_xor_sync(kFull, l1, 2);
        __syncthreads();  // every ring is done with: the warps' results take its place
        float *mine = reinterpret_cast<float *>(smem) + warp * kRows * D;
        if (tq == 0) {
            s_ml[warp][gr] = make_float2(m0, l0);
            s_ml[warp][gr + 8] = make_float2(m1, l1);
        }
        if constexpr (ES == 2) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                *reinterpret_cast<float2 *>(mine + gr * D + i * 8 + 2 * tq) = make_float2(o[i][0], o[i][1]);
                *reinterpret_cast<float2 *>(mine + (gr + 8) * D + i * 8 + 2 * tq) = make_float2(o[i][2], o[i][3]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                *reinterpret_cast<float4 *>(mine + gr * D + c * 16 + 4 * tq) =
                    make_float4(o[2 * c][0], o[2 * c + 1][0], o[2 * c][1], o[2 * c + 1][1]);
                *reinterpret_cast<float4 *>(mine + (gr + 8) * D + c * 16 + 4 * tq) =
                    make_float4(o[2 * c][2], o[2 * c + 1][2], o[2 * c][3], o[2 * c + 1][3]);
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < t.rows * (D / 4); x += A::THREADS) {
            const int r = x / (D / 4), c = x % (D / 4);
            float M = -CUDART_INF_F;
#pragma unroll
            for (int y = 0; y < A::WARPS; ++y) M = fmaxf(M, s_ml[y][r].x);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int y = 0; y < A::WARPS; ++y) {
                const float2 ml = s_ml[y][r];
                const float f = ml.y == 0.f ? 0.f : exp2_approx(ml.x - M);
                const float4 v = reinterpret_cast<const float4 *>(smem)[(y * kRows + r) * (D / 4) + c];
                sum.x += f * v.x;
                sum.y += f * v.y;
                sum.z += f * v.z;
                sum.w += f * v.w;
                l += f * ml.y;
            }
            if (!w.whole()) {
                const int64_t part = part_row(w, kRows) + r;
                reinterpret_cast<float4 *>(a.part_o)[part * (D / 4) + c] = sum;
                if (c == 0) a.part_ml[part] = make_float2(M, l);
                continue;
            }
            const float inv = inverse_sum(l, a.v_scale);
            const int R = t.row0 + r, i = a.by_group(R), head = t.j * a.group + R - i * a.group;
            *reinterpret_cast<uint2 *>(a.O + 2 * ((int64_t)(qrow0 + i) * a.o_stride + (int64_t)head * D + 4 * c)) =
                make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
            if (c == 0 && a.lse) a.lse[(int64_t)(qrow0 + i) * a.q_heads + head] = log_sum(M, l);
        }
        __syncthreads();  // the next segment's copies may overwrite the results
        if (!w.whole() && threadIdx.x == 0) {
            // Parts of a tile count themselves in a byte of the workspace's head,
            // which the last one takes back to zero; it joins the parts below.
            const int unit0 = at_unit - w.first, c0 = cta_of(unit0, s_line), c1 = cta_of(unit0 + w.units - 1, s_line);
            uint32_t *word = a.counts + c0 / 4;
            const int shift = c0 % 4 * 8;
            __threadfence();
            if ((int)(atomicAdd(word, 1u << shift) >> shift & 255u) == c1 - c0) {
                atomicSub(word, (uint32_t)(c1 - c0 + 1) << shift);
                s_join[w.first > 0 ? 0 : 1] = make_int4(w.tile - 1, c0, c1, 0);
            }
        }
        at_unit += w.last - w.first;
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {  // (a CTA's first segment and its last one)
        const int4 j = s_join[k];
        if (j.x < 0) continue;
        __threadfence();
        const Tile t = make_tile<A::KEYS>(a, j.x, kRows, false);
        for (int r = warp; r < t.rows; r += A::WARPS) join_rows<D, kRows, 1, 8>(a, t, j.y, j.z, r);
    }
}

template <int D, int ES>
cudaError_t launch_one(const AttnArgs &a, cudaStream_t st)
{
    using A = Attend<D, ES>;
    cudaError_t e = cudaFuncSetAttribute(k_attend<D, ES>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM);
    if (e != cudaSuccess) return e;
    k_attend<D, ES><<<a.ctas, A::THREADS, A::SMEM, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Which form: this file's reads K and V once per 16 rows, the other once per
// 128 or 256, but takes 4 to 9 us more from launch to end. Up to 16 rows this
// one always; beyond, while what its further tiles cost is less: bytes that are
// read again, 128 operations' worth per key, and 1024 keys' worth of start and
// end per tile. (Rows are a bound, so the tiles are too: every new token's, and
// one begun per list.) Over 350 mixes of 32 to 256 rows, 8 to 384 lists of 64 to
// 4096 keys, all dims and types, the rule takes 1.5% more time than the better
// form of each; bytes alone took 7%. Measured (us, this form / the other, 128
// dims, bf16): 8 lists of 1024 keys, 32 rows 12 / 16, 128 rows 17.5 / 19; 32 lists
// of 4096 keys, 32 rows 29 / 27, 64 rows 44 / 29; 128 lists of 1024 keys, 32 rows
// 28 / 21, 128 rows 87 / 23; E4M3, 128 lists of 4096 keys, 32 rows 65 / 70, 48 rows
// 89 / 70.
bool takes_chunks(int64_t batch, int64_t heads, int32_t group, int64_t n_tokens, int64_t max_q, int64_t max_len,
                  int32_t head_dim, int32_t es)
{
    const int64_t per_list = (max_q * group + kRows - 1) / kRows - 1, in_all = n_tokens * group / kRows;
    const int64_t again = heads * std::min(batch * per_list, in_all);
    return (double)again * (double)(max_len + 1024) * (head_dim * es + 128) > kAgainBytes;
}

AttnPlan attention_plan(int32_t batch, int32_t heads, int32_t group, int32_t n_tokens, int32_t max_q, int32_t max_len,
                        int32_t head_dim, int32_t es, int ctas)
{
    AttnPlan p;
    const int64_t rows = (int64_t)max_q * group;
    p.chunked = takes_chunks(batch, heads, group, n_tokens, max_q, max_len, head_dim, es);
    const int tile = p.chunked ? chunk_tile_rows(head_dim) : kRows;
    p.tiles = (int32_t)((rows + tile - 1) / tile);
    p.ctas = ctas;
    p.part_rows = (int64_t)ctas * 2 * tile;
    p.bytes = (size_t)p.part_rows * (head_dim * sizeof(float) + sizeof(float2)) + ctas * sizeof(LineInfo);
    return p;
}

cudaError_t launch_paged_attention(const AttnArgs &a, cudaStream_t st)
{
    if (a.chunked) return launch_attend_chunk(a, st);
    if (a.es == 2) {
        switch (a.head_dim) {
        case 64: return launch_one<64, 2>(a, st);
        case 128: return launch_one<128, 2>(a, st);
        case 256: return launch_one<256, 2>(a, st);
        }
    } else {
        switch (a.head_dim) {
        case 64: return launch_one<64, 1>(a, st);
        case 128: return launch_one<128, 1>(a, st);
        case 256: return launch_one<256, 1>(a, st);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace mkv
