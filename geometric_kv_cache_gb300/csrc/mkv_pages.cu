// sm_103a page lists of a paged cache: fork, copy, free and extend
// (mkv_page_update), and compaction into new pages (mkv_page_compact).
//
// The ManifoldKV path ends with a compacted cache whose heads differ in
// length ("ManifoldKV: Training-Free KV Cache Compression via Euclidean
// Outlier Detection", ICML 2026 poster 62526, abstract: which past tokens the
// cache retains). A serving engine keeps it in pages, one list per head.
//
// A call is three launches, each a programmatic dependent of the one before
// (small problems do the first two in one, k_page_plan, and small updates all three):
//  1. k_page_count: per chunk of rows the pages its lists need, per chunk of
//     the pool the free pages (refs 0);
//  2. k_page_assign: every CTA sums the chunk totals before its own (a few KB
//     from L2), so that lists get their first rank among the new pages and
//     the lowest free pages land in free_ids[rank]; every CTA also comes to the
//     same verdict (enough pages, every device argument valid), which CTA 0
//     writes down;
//  3. k_page_update / k_page_compact: tables, counts and rows. On a bad
//     verdict they write the input's lists.
// Measured: the update of 512 rows of 8 lists (4096 lists, 350K pages, a quarter of
// the rows moved) 12 us, of 8 rows 9 us: round trips of latency each; the
// compaction of 64 lists of 8K-32K tokens to half 119 us, 107 of it the copy, 6.3
// TB/s, 0.93 of the measured copy peak. 4-bit pages of as many tokens 45 us (floor 28):
// planned in the same 9, and every second row of 64 bytes is copied at 0.6 of memory's
// rate; a bf16 cache into 4-bit pages (mkv_page_quantize) 83 us (64), into E4M3 pages 89
// (75). Very many lists: 140000 of 20-40 tokens halved 1.16 ms in bf16, 0.97 in 4 bits.
// Integers only decide, and every rank is a prefix sum: nothing depends on
// the order of the atomics (counts are sums).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mkv_device.cuh"
#include "mkv_e2m1.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kPageThreads = 256;
// Problems of up to 8 chunks (of 8 rows or runs of lists, of 4096 pages) are planned by one
// cluster, a chunk per CTA, in one launch; larger ones in two. The update of 16 rows x
// 8 heads of 500-2048 tokens (5 chunks): planned in one launch 13.1 us per call from
// Python and 8.8 us in a graph, in two 15 and 9.1; 32 rows (10 chunks, two per CTA) took
// 16.4 and 14.7 against 15.2 and 11.6. Updates of no more lists than the cluster has
// warps come along in the same launch. That is for the host's sake: from Python, 8 to 64
// lists of 500-2048 tokens take 12 us, with a launch of their own 14, but in a graph 7.3 to
// 10.4 against 6.9 to 9.9 (8 rows x 8 heads, a quarter moved 10.3 / 9.9; 4 rows, nearly
// all moved 10.4 / 9.5): the second barrier of the cluster costs 0.1 to 0.9 us more than
// a dependent launch.
static_assert(kPlanCluster <= 8, "a portable cluster");
// Tokens per item of the compaction: a page holds a whole number of them, and
// small items even out the warps' shares. With 4 rows of K and of V in flight
// per lane and 3 CTAs per SM, 8 rows of 8K-32K tokens halved take 119 us (107 us
// of it the copy, 0.93 of the copy peak); 8 in flight and 2 CTAs take 4 us more, items
// of 32 tokens 5.
constexpr int kItem = 16;

__device__ __forceinline__ int pages_of(int len, const PageArgs &a)
{
    return (len + a.page_size - 1) >> a.page_shift;
}

__device__ __forceinline__ bool len_ok(int len, const PageArgs &a)
{
    return len >= 0 && len <= (a.max_pages << a.page_shift);
}

// What one list of `out` becomes (update): its length, how many of the
// parent's pages it shares, and its pages in all.
struct ListPlan {
    int old_len, len, shared, total;
};

__device__ __forceinline__ ListPlan plan_list(const PageArgs &a, int b, int j, int src, bool keeps)
{
    ListPlan p = {0, 0, 0, 0};
    if (src < 0) return p;
    p.old_len = a.lens[(int64_t)src * a.heads + j];
    p.len = p.old_len + (a.n_new ? a.n_new[b] : 0);
    p.shared = keeps ? pages_of(p.old_len, a) : p.old_len >> a.page_shift;
    p.total = pages_of(p.len, a);
    return p;
}

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The holders of this thread's pages of a chunk, consecutive ones; -1 past the pool.
constexpr int kThreadPages = kPlanPages / kPageThreads;
__device__ __forceinline__ void load_refs(const PageArgs &a, int chunk, int (&r)[kThreadPages])
{
    constexpr int N = kThreadPages;
    const int64_t p0 = (int64_t)chunk * kPlanPages + threadIdx.x * N;
    if (p0 + N <= a.n_pages && (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const int4 v = *reinterpret_cast<const int4 *>(a.refs + p0 + i);
            r[i] = v.x;
            r[i + 1] = v.y;
            r[i + 2] = v.z;
            r[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = p0 + i < a.n_pages ? a.refs[p0 + i] : -1;
    }
}

// Chunk c of the lists, or after them of the pool: what the lists need, what is
// free. A warp has `run` lists, those of a row in an update, whose parents count.
// Each list's need goes into list_off, and into `pages` that of this lane's first
// one; r: the chunk's holders (of the pool's chunks).
template <bool COMPACT>
__device__ __forceinline__ void count_chunk(const PageArgs &a, int c, int (&r)[kThreadPages], int &pages)
{
    __shared__ long long s_need[kPlanRows];
    __shared__ uint32_t s_bits[kPlanRows];
    __shared__ int s_free[kPageThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (c < a.row_chunks) {
        const int w = c * kPlanRows + warp, b = w;
        long long need = 0;
        uint32_t bits = 0;
        pages = 0;
        if constexpr (COMPACT) {
            const int lists = a.batch * a.heads, h0 = w * a.run, n = min(a.run, lists - h0);
            for (int j = lane; j < n; j += 32) {
                const int h = h0 + j, own_len = a.lens[h], kept = a.kept[h];
                const int T = !a.K ? own_len : a.seq_lens ? a.seq_lens[h / a.heads] : a.t_max;
                if (!len_ok(own_len, a) || (a.K && (T < 0 || T > a.t_max))) bits |= MKV_DEV_BAD_SEQ_LEN;
                // (without indices tokens 0 .. kept-1 must be there)
                if (!len_ok(kept, a) || kept > (a.idx ? a.idx_stride : T)) {
                    bits |= MKV_DEV_BAD_N_KEEP;
                    continue;
                }
                const int p = pages_of(kept, a);
                a.list_off[h] = p;
                if (j == lane) pages = p;
                need += p;
            }
        } else if (b < a.batch) {
            int src = b;
            bool keeps = true;
            if (a.parent) {
                src = a.parent[b];
                if (src < -1 || src >= a.batch) {
                    bits |= MKV_DEV_BAD_PARENT;
                    src = -1;
                }
                // the row that keeps the parent's partly filled last pages:
                // the parent itself if it goes on, else its lowest child
                if (src >= 0 && src != b) {
                    keeps = a.parent[src] != src;
                    for (int64_t i = 0; keeps && i < b; i += 256) {
                        bool hit = false;
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int64_t x = i + 32 * u + lane;
                            hit |= x < b && a.parent[x] == src;
                        }
                        keeps = !__any_sync(kFull, hit);
                    }
                }
            }
            if (lane == 0) a.row_src[b] = make_int2(src, keeps ? 1 : 0);
            const int add = a.n_new && src >= 0 ? a.n_new[b] : 0;
            if (add < 0) bits |= MKV_DEV_BAD_PARENT;
            for (int j = lane; j < a.heads; j += 32) {
                const int h = b * a.heads + j;
                if (!len_ok(a.lens[h], a)) bits |= MKV_DEV_BAD_SEQ_LEN;
                if (src >= 0) {
                    const int L = a.lens[(int64_t)src * a.heads + j];
                    if (!len_ok(L, a)) continue;  // reported by its own row
                    if (add < 0 || (long long)L + add > ((long long)a.max_pages << a.page_shift)) {
                        bits |= MKV_DEV_BAD_PARENT;
                        continue;
                    }
                }
                const ListPlan p = plan_list(a, b, j, src, keeps);
                a.list_off[h] = p.total - p.shared;
                if (j == lane) pages = p.total - p.shared;
                need += p.total - p.shared;
            }
        }
        need = warp_sum(need);
        bits = __reduce_or_sync(kFull, bits);
        if (lane == 0) {
            s_need[warp] = need;
            s_bits[warp] = bits;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            long long n = 0;
            uint32_t x = 0;
            for (int i = 0; i < kPlanRows; ++i) {
                n += s_need[i];
                x |= s_bits[i];
            }
            a.row_need[c] = n;
            a.row_bits[c] = x;
        }
    } else {
        const int chunk = c - a.row_chunks;
        int n = 0;
        load_refs(a, chunk, r);
#pragma unroll
        for (int i = 0; i < kThreadPages; ++i) n += r[i] == 0;
        n = __reduce_add_sync(kFull, n);
        if (lane == 0) s_free[warp] = n;
        __syncthreads();
        if (threadIdx.x == 0) {
            int t = 0;
            for (int i = 0; i < kPageThreads / 32; ++i) t += s_free[i];
            a.page_free[chunk] = t;
        }
    }
}

// Sums over the CTA of three values at once.
__device__ __forceinline__ void block_sums(long long &x, long long &y, long long &z, uint32_t &bits)
{
    __shared__ long long s[3][kPageThreads / 32];
    __shared__ uint32_t sb[kPageThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_sum(x);
    y = warp_sum(y);
    z = warp_sum(z);
    bits = __reduce_or_sync(kFull, bits);
    if (lane == 0) {
        s[0][warp] = x;
        s[1][warp] = y;
        s[2][warp] = z;
        sb[warp] = bits;
    }
    __syncthreads();
    x = y = z = 0;
    bits = 0;
    for (int i = 0; i < kPageThreads / 32; ++i) {
        x += s[0][i];
        y += s[1][i];
        z += s[2][i];
        bits |= sb[i];
    }
    __syncthreads();
}

// The same chunk, once all are counted: its lists' first ranks among the new
// pages, or its free pages by rank. Chunk 0 writes the verdict. r, pages: as counted.
template <bool COMPACT>
__device__ __forceinline__ void assign_chunk(const PageArgs &a, int c, const int (&r)[kThreadPages], int pages)
{
    __shared__ uint32_t scratch[kPageThreads / 32];
    __shared__ long long s_row[kPlanRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool rows = c < a.row_chunks;
    const int chunk = rows ? c : c - a.row_chunks;
    // pages needed and free in all, and (rows: needed, pages: free) in the chunks before this one
    long long need = 0, free_pages = 0, before = 0;
    uint32_t bits = 0;
    for (int i = threadIdx.x; i < a.row_chunks; i += kPageThreads) {
        const long long n = a.row_need[i];
        need += n;
        bits |= a.row_bits[i];
        if (rows && i < chunk) before += n;
    }
    for (int i = threadIdx.x; i < a.page_chunks; i += kPageThreads) {
        const int n = a.page_free[i];
        free_pages += n;
        if (!rows && i < chunk) before += n;
    }
    block_sums(need, free_pages, before, bits);
    if (need > free_pages) bits |= MKV_DEV_NO_PAGES;
    if (c == 0 && threadIdx.x == 0) {
        a.verdict[0] = bits;
        a.verdict[1] = bits ? 0u : (uint32_t)need;  // pages taken
        if (bits) atomicOr(a.status, bits);
    }
    if (rows) {
        if (bits) return;  // no list gets a page
        const int h0 = (chunk * kPlanRows + warp) * a.run, lists = min(a.run, a.batch * a.heads - h0);
        int32_t *offs = a.list_off + h0;
        long long row = pages;
        for (int j = 32 + lane; j < lists; j += 32) row += offs[j];
        row = warp_sum(row);
        if (lane == 0) s_row[warp] = row;
        __syncthreads();
        int off = (int)before;  // at most n_pages: the verdict was good
        for (int i = 0; i < warp; ++i) off += (int)s_row[i];
        for (int j0 = 0; j0 < lists; j0 += 32) {
            const int j = j0 + lane, n = j0 == 0 ? pages : j < lists ? offs[j] : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            if (j < lists) offs[j] = off + x - n;
            if constexpr (COMPACT)  // whose each new page is
                for (int k = 0; k < min(32, lists - j0); ++k) {
                    const int m = __shfl_sync(kFull, n, k), at = off + __shfl_sync(kFull, x, k) - m;
                    for (int q = lane; q < m; q += 32) a.owners[at + q] = make_int2(h0 + j0 + k, q);
                }
            off += __shfl_sync(kFull, x, 31);
        }
    } else {
        constexpr int N = kThreadPages;
        const int64_t p0 = (int64_t)chunk * kPlanPages + threadIdx.x * N;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) n += r[i] == 0;
        if (a.refs_out != a.refs) {
            if (p0 + N <= a.n_pages && (reinterpret_cast<uintptr_t>(a.refs_out) & 15) == 0) {
#pragma unroll
                for (int i = 0; i < N; i += 4)
                    *reinterpret_cast<int4 *>(a.refs_out + p0 + i) = make_int4(r[i], r[i + 1], r[i + 2], r[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (p0 + i < a.n_pages) a.refs_out[p0 + i] = r[i];
            }
        }
        if (bits || before >= need) return;  // no page of this chunk is taken
        long long rank = before + block_exclusive_scan<kPageThreads>((uint32_t)n, scratch, nullptr);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (r[i] == 0) {
                if (rank < need) a.free_ids[rank] = (int32_t)(p0 + i);
                ++rank;
            }
    }
}

template <bool COMPACT>
__global__ void __launch_bounds__(kPageThreads)
k_page_count(const PageArgs a)
{
    pdl_trigger();
    int r[kThreadPages], pages;
    count_chunk<COMPACT>(a, (int)blockIdx.x, r, pages);
}

// (The call's inputs are there before k_page_count starts, which is nobody's
// programmatic dependent: the launches after it read them before they wait.)
template <bool COMPACT>
__global__ void __launch_bounds__(kPageThreads)
k_page_assign(const PageArgs a)
{
    pdl_trigger();
    int r[kThreadPages];
    if ((int)blockIdx.x >= a.row_chunks) load_refs(a, (int)blockIdx.x - a.row_chunks, r);
    pdl_wait();
    int pages = 0;
    const int h0 = ((int)blockIdx.x * kPlanRows + ((int)threadIdx.x >> 5)) * a.run, j = threadIdx.x & 31;
    if ((int)blockIdx.x < a.row_chunks && j < min(a.run, a.batch * a.heads - h0)) pages = a.list_off[h0 + j];
    assign_chunk<COMPACT>(a, (int)blockIdx.x, r, pages);
}

__device__ __forceinline__ void add_ref(const PageArgs &a, int page, int by)
{
    if ((uint32_t)page < (uint32_t)a.n_pages)
        atomicAdd(a.refs_out + page, by);
    else
        atomicOr(a.status, MKV_DEV_BAD_PAGE);
}

// What an update reads of its list h before it has the plan: its length, the list
// that it goes on with (src -1: none), that one's length and last page, the new tokens,
// and this lane's first pages of that list and, where they are given up, of its own
// (kAhead of each; a loop of single ones waits for memory at every step).
constexpr int kAhead = 4;
struct ListInputs {
    int own_len, src, old_len, add, last;
    int from[kAhead], own[kAhead];
};
__device__ __forceinline__ void load_ids(const int32_t *ids, int p0, int n, int (&id)[kAhead])
{
#pragma unroll
    for (int i = 0; i < kAhead; ++i) id[i] = p0 + 32 * i < n ? ids[p0 + 32 * i] : -1;
}

__device__ __forceinline__ ListInputs update_inputs(const PageArgs &a, int64_t h)
{
    const int b = (int)(h / a.heads), j = (int)(h - (int64_t)b * a.heads);
    ListInputs in;
    in.own_len = a.lens[h];
    in.add = a.n_new ? a.n_new[b] : 0;
    in.src = b;
    if (a.parent) {
        in.src = a.parent[b];
        if (in.src < -1 || in.src >= a.batch) in.src = -1;
    }
    const int64_t s = (int64_t)max(in.src, 0) * a.heads + j;
    in.old_len = in.src == b ? in.own_len : in.src >= 0 ? a.lens[s] : 0;
    const int lane = threadIdx.x & 31;
    const bool good = len_ok(in.old_len, a);
    in.last = in.src != b && good && (in.old_len & (a.page_size - 1)) ? a.table[s * a.max_pages + (in.old_len >> a.page_shift)] : -1;
    load_ids(a.table + s * a.max_pages, lane, good && a.lens_out != a.lens ? pages_of(in.old_len, a) : 0, in.from);
    load_ids(a.table + h * a.max_pages, lane, in.src != b && len_ok(in.own_len, a) ? pages_of(in.own_len, a) : 0, in.own);
    return in;
}

// List h by one warp, once all chunks are assigned.
__device__ __forceinline__ void update_list(const PageArgs &a, int64_t h, const ListInputs &in)
{
    const int lane = threadIdx.x & 31;
    const int b = (int)(h / a.heads), j = (int)(h - (int64_t)b * a.heads);
    const bool in_place = a.lens_out == a.lens;  // (lists without capacity may have no tables at all)
    const int32_t *mine = a.table + h * a.max_pages;
    int32_t *out = a.table_out + h * a.max_pages;
    // (read together; the last two mean nothing after a bad verdict)
    const uint32_t verdict = a.verdict[0];
    const int2 src = a.row_src[b];
    const int first = a.list_off[h];
    if (verdict) {  // the lists stay as they were
        if (in_place) return;
        if (lane == 0) a.lens_out[h] = in.own_len;
        if (len_ok(in.own_len, a))
            for (int p = lane; p < pages_of(in.own_len, a); p += 32) out[p] = mine[p];
        return;
    }
    const bool keeps = src.y != 0, moved = in.src != b;
    const int len = in.src < 0 ? 0 : in.old_len + in.add;
    const int shared = keeps ? pages_of(in.old_len, a) : in.old_len >> a.page_shift, total = pages_of(len, a);
    const int32_t *from = a.table + ((int64_t)(in.src < 0 ? b : in.src) * a.heads + j) * a.max_pages;
    __syncwarp();
    if (!in_place)
        for (int p0 = lane; p0 < shared; p0 += 32 * kAhead) {
            int id[kAhead];
            if (p0 == lane) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) id[i] = in.from[i];
            } else {
                load_ids(from, p0, shared, id);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (p0 + 32 * i < shared) {
                    out[p0 + 32 * i] = id[i];
                    if (moved) add_ref(a, id[i], 1);
                }
        }
    for (int p = shared + lane; p < total; p += 32) {
        const int id = a.free_ids[first + p - shared];
        out[p] = id;
        atomicAdd(a.refs_out + id, 1);
    }
    if (moved)  // nobody continues this list under its own row: its holder goes
        for (int p0 = lane, n = pages_of(in.own_len, a); p0 < n; p0 += 32 * kAhead) {
            int id[kAhead];
            if (p0 == lane) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) id[i] = in.own[i];
            } else {
                load_ids(mine, p0, n, id);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (p0 + 32 * i < n) add_ref(a, id[i], -1);
        }
    if (lane == 0) a.lens_out[h] = len;
    const int rest = in.old_len & (a.page_size - 1);
    if (!keeps && rest > 0) {  // a copy of the partly filled last page
        const int s = in.last, d = a.free_ids[first];
        if ((uint32_t)s >= (uint32_t)a.n_pages) {
            if (lane == 0) atomicOr(a.status, MKV_DEV_BAD_PAGE);
            return;
        }
        const int64_t n = rest * a.row_bytes;
        const uint8_t *ks = a.k + s * a.page_bytes, *vs = a.v + s * a.page_bytes;
        uint8_t *kd = a.k + d * a.page_bytes, *vd = a.v + d * a.page_bytes;
        // 4-bit pages: the rows' scales, behind the codes of the whole page
        const int64_t sc = a.row_bytes << a.page_shift;
        for (int o = lane * 4; o < rest * a.scale_bytes; o += 128) {
            const uint32_t x = *reinterpret_cast<const uint32_t *>(ks + sc + o);
            const uint32_t y = *reinterpret_cast<const uint32_t *>(vs + sc + o);
            *reinterpret_cast<uint32_t *>(kd + sc + o) = x;
            *reinterpret_cast<uint32_t *>(vd + sc + o) = y;
        }
        // one round trip for 16 rows of 256 bytes
        constexpr int U = 8;
        for (int64_t o = lane * 16; o < n; o += 512 * U) {
            uint4 x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (o + 512 * u < n) {
                    x[u] = ld_stream(ks + o + 512 * u);
                    y[u] = ld_stream(vs + o + 512 * u);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (o + 512 * u < n) {
                    st_v4(kd + o + 512 * u, x[u]);
                    st_v4(vd + o + 512 * u, y[u]);
                }
        }
    }
}

// One warp per list.
__global__ void __launch_bounds__(kPageThreads)
k_page_update(const PageArgs a)
{
    const int64_t h = ((int64_t)blockIdx.x * kPageThreads + threadIdx.x) >> 5;
    const bool some = h < (int64_t)a.batch * a.heads;
    ListInputs in;
    if (some) in = update_inputs(a, h);
    pdl_wait();
    if (some) update_list(a, h, in);
}

// What every CTA of the cluster wrote is there for all.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Counts and places in one launch of one cluster, for problems of few chunks. UPDATE:
// the lists as well, one per warp (they would be as many warps in a launch of their own).
template <bool COMPACT, bool UPDATE>
__global__ void __launch_bounds__(kPageThreads)
k_page_plan(const PageArgs a)
{
    if (!UPDATE) pdl_trigger();
    const bool mine = (int)blockIdx.x < a.row_chunks + a.page_chunks;
    const int64_t h = ((int64_t)blockIdx.x * kPageThreads + threadIdx.x) >> 5;
    const bool some = UPDATE && h < (int64_t)a.batch * a.heads;
    ListInputs in;
    if (some) in = update_inputs(a, h);
    int r[kThreadPages], pages = 0;
    if (mine) count_chunk<COMPACT>(a, (int)blockIdx.x, r, pages);
    __syncthreads();
    cluster_sync();
    if (mine) assign_chunk<COMPACT>(a, (int)blockIdx.x, r, pages);
    if (UPDATE) {
        __syncthreads();
        cluster_sync();
        if (some) update_list(a, h, in);
    }
}

// The first `list_ctas` CTAs write tables and counts, list by list; the warps
// of the others copy rows. Item = 16 tokens of a new page, one lane per token
// for its places; owners[rank] names a new page's list and place in it,
// so the items are the pages taken, whatever the lists' lengths and capacities.
// An item's owner is read three items ahead, its indices two and its page
// entries one, so that every row copy (groups of LPR lanes, 16 bytes each, 4
// rows of K and of V in flight per lane) finds its addresses in registers.
// ROWS: what a row is. Rows of 4-bit pages are short: a warp takes two items at
// once, and a lane also copies the scales of its own token, with one load of each. Rows that become codes are 32 bytes of bf16 per
// lane, one group of 16 dims: its largest element never leaves the lane.
template <int BYTES>
struct ScaleWord {
    using type = uint32_t;
};
template <>
struct ScaleWord<8> {
    using type = uint2;
};
template <>
struct ScaleWord<16> {
    using type = uint4;
};
enum Rows { kCopy, kCopyCodes, kToE4m3, kToE2m1 };

// A group of 16 bf16 as E4M3 codes (16 bytes), or as 4-bit codes (8 bytes) and their scale.
__device__ __forceinline__ uint4 group_to_e4m3(uint4 lo, uint4 hi, Rounding r)
{
    float x[8], y[8];
    bf16x8_to_f32(lo, x);
    bf16x8_to_f32(hi, y);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float *f = i < 2 ? x + 4 * i : y + 4 * (i - 2);
        w[i] = f32x2_to_e4m3(f[0] * r.inv, f[1] * r.inv) | f32x2_to_e4m3(f[2] * r.inv, f[3] * r.inv) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 group_to_e2m1(uint4 lo, uint4 hi, Rounding r, uint32_t &scale)
{
    float x[8], y[8];
    bf16x8_to_f32(lo, x);
    bf16x8_to_f32(hi, y);
    scale = f32x2_to_e4m3(max_nan(largest8(x), largest8(y)) * r.inv6, 0.f) & 0xFFu;
    const float f = code_factor(scale, r.inv);
    return make_uint2(codes8(x, f), codes8(y, f));
}

// 16 bytes of a short row, of which memory is to bring no more than 64: by itself it
// brings 128, and of every second row kept 151 MB instead of 108 (64 lists of
// 8K-32K 4-bit tokens of 128 dims halved: 4 us more of 45).
__device__ __forceinline__ uint4 ld_short(const void *p)
{
    uint4 r;
    asm("ld.global.nc.L1::no_allocate.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

template <int LPR, Rows ROWS>
__global__ void __launch_bounds__(kPageThreads, 3)
k_page_compact(const PageArgs a, int list_ctas)
{
    constexpr bool ROUND = ROWS == kToE4m3 || ROWS == kToE2m1;
    constexpr int RB = LPR * (ROUND ? 32 : 16), RPS = 32 / LPR;  // bytes of a row (read), rows per step
    constexpr int ITEMS = ROWS == kCopyCodes ? 2 : 1;  // at once: half a warp each
    constexpr int MOST = ROUND ? 2 : 4;
    constexpr int STEPS = ITEMS * kItem / RPS, B = STEPS < MOST ? STEPS : MOST;  // steps, and of a batch
    constexpr int SB = ROWS == kCopyCodes ? LPR * 2 : ROWS == kToE2m1 ? LPR : 0;  // bytes of a row's scales
    constexpr int WB = ROWS == kToE2m1 ? LPR * 8 : LPR * 16;                      // bytes of a row written, without them
    pdl_wait();
    const bool bad = a.verdict[0] != 0;
    const int64_t lists = (int64_t)a.batch * a.heads;
    if ((int)blockIdx.x < list_ctas) {
        for (int64_t h = blockIdx.x; h < lists; h += list_ctas) {
            // (read together; the last means nothing after a bad verdict)
            const int own_len = a.lens[h], kept = a.kept[h], first = a.list_off[h], n = bad ? 0 : kept;
            const int32_t *mine = a.table + h * a.max_pages;
            int32_t *out = a.table_out + h * a.max_pages;
            if (threadIdx.x == 0) a.lens_out[h] = bad ? own_len : n;
            if (bad && !len_ok(own_len, a)) continue;
            for (int p = threadIdx.x; p < pages_of(n, a); p += kPageThreads) {
                const int id = a.free_ids[first + p];
                out[p] = id;
                atomicAdd(a.refs_out + id, 1);
            }
            for (int p = threadIdx.x; p < pages_of(own_len, a); p += kPageThreads) {
                if (bad) out[p] = mine[p];  // the lists stay as they were
                else add_ref(a, mine[p], -1);
            }
        }
        return;
    }
    const int lane = threadIdx.x & 31, g = lane / LPR, lr = lane % LPR;
    const int per_shift = a.page_shift - 4;  // items of a page
    const int64_t warps = (int64_t)(gridDim.x - list_ctas) * (kPageThreads / 32);
    const int64_t warp = (int64_t)(blockIdx.x - list_ctas) * (kPageThreads / 32) + (threadIdx.x >> 5);
    // a page that is taken: its list, its place in it, its number (list -1: none)
    struct Owner {
        int h, at, page;
    };
    // (of item x of the warps' count this lane has item x ITEMS + lane / kItem, which lanes of no item do not look up)
    auto owner = [&](int64_t x, int64_t pages) -> Owner {
        const int64_t page = (ITEMS == 1 ? x : x * ITEMS + lane / kItem) >> per_shift;
        if (page >= pages) return {-1, 0, 0};
        const int2 o = a.owners[page];
        return {o.x, o.y, a.free_ids[page]};
    };
    // (the first ones come with the verdict; what lies behind the pages taken is dropped)
    const int64_t room = min((int64_t)a.n_pages, lists * a.max_pages);
    Owner first = owner(warp, room), second = owner(warp + warps, room);
    const int64_t taken = a.verdict[1], items = taken << per_shift;
    if (bad) return;
    auto drop = [&](int64_t x, Owner &o) {
        if ((ITEMS == 1 ? x : x * ITEMS + lane / kItem) >= items) o = {-1, 0, 0};
    };
    drop(warp, first);
    drop(warp + warps, second);
    // an item: its list, its new page, and this lane's token of it with its source (-1: none)
    struct Item {
        int h, page, i, s;
    };
    auto source = [&](int64_t x, Owner own) -> Item {
        const int64_t item = ITEMS == 1 ? x : x * ITEMS + lane / kItem;
        Item it = {own.h, own.page, -1, -1};
        if (own.h < 0 || lane >= ITEMS * kItem) return it;
        const int64_t h = own.h;
        const int i = (own.at << a.page_shift) + (int)(item & ((1 << per_shift) - 1)) * kItem + lane % kItem;
        // (read together: an index behind the kept ones is not looked at)
        const int kept = a.kept[h], s = !a.idx ? i : i < a.idx_stride ? a.idx[h * a.idx_stride + i] : -1;
        if (i >= kept) return it;
        const int T = !a.K ? a.lens[h] : a.seq_lens ? a.seq_lens[own.h / a.heads] : a.t_max;
        it.i = i;
        if (s < 0 || s >= T) atomicOr(a.status, MKV_DEV_BAD_INDEX);
        else it.s = s;
        return it;
    };
    // the rows of the pool (or the contiguous cache) it is copied from and to
    auto places = [&](const Item &it, int64_t &from, int &to) {
        from = to = -1;
        if (it.s < 0) return;
        if (a.K) {
            from = (int64_t)it.h * a.t_max + it.s;
        } else {
            const int id = a.table[(int64_t)it.h * a.max_pages + (it.s >> a.page_shift)];
            if ((uint32_t)id >= (uint32_t)a.n_pages) {
                atomicOr(a.status, MKV_DEV_BAD_PAGE);
                return;
            }
            from = (id << a.page_shift) + (it.s & (a.page_size - 1));
        }
        to = (it.page << a.page_shift) + (it.i & (a.page_size - 1));
    };
    const uint8_t *ks = (a.K ? a.K : a.k) + lr * (RB / LPR), *vs = (a.K ? a.V : a.v) + lr * (RB / LPR);
    uint8_t *kd = a.k + lr * (WB / LPR), *vd = a.v + lr * (WB / LPR);
    // where a row of the pool's codes, and of its scales, lies: each page has both
    auto codes_at = [&](int64_t row) -> int64_t {
        return row * WB + (SB ? (row >> a.page_shift << a.page_shift) * SB : 0);
    };
    auto scales_at = [&](int64_t row) -> int64_t {
        return ((row >> a.page_shift) + 1 << a.page_shift) * WB + row * SB;
    };
    int64_t from;
    int to;
    Item ahead = source(warp, first);
    const Item next = source(warp + warps, second);
    Owner own = owner(warp + 2 * warps, taken);
    places(ahead, from, to);
    ahead = next;
    for (int64_t item = warp; item * ITEMS < items; item += warps) {
        constexpr int N = ROUND ? 2 : 1;
        uint4 kr[B][N], vr[B][N];
        int dst[B];
        auto load = [&](int b0) {
#pragma unroll
            for (int u = 0; u < B; ++u) {
                const int row = (b0 + u) * RPS + g;
                const int64_t src = __shfl_sync(kFull, from, row);
                dst[u] = __shfl_sync(kFull, to, row);
                if (dst[u] >= 0) {
                    const int64_t at = ROWS == kCopyCodes ? codes_at(src) : src * RB;
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        kr[u][x] = RB <= 64 && ROWS == kCopyCodes ? ld_short(ks + at) : ld_stream(ks + at + 16 * x);
                        vr[u][x] = RB <= 64 && ROWS == kCopyCodes ? ld_short(vs + at) : ld_stream(vs + at + 16 * x);
                    }
                }
            }
        };
        // short rows: the first ones are on their way while the next items' places are waited for (bf16 and E4M3 rows
        // are not faster for it)
        using S = typename ScaleWord<SB>::type;
        S k_scales, v_scales;  // of this lane's token
        if constexpr (ROWS == kCopyCodes)
            if (to >= 0) {
                const int64_t s = scales_at(from);
                k_scales = *reinterpret_cast<const S *>(a.k + s);
                v_scales = *reinterpret_cast<const S *>(a.v + s);
            }
        if constexpr (ROWS != kCopy) load(0);
        int64_t next_from;
        int next_to;
        places(ahead, next_from, next_to);
        ahead = source(item + 2 * warps, own);
        own = owner(item + 3 * warps, taken);
#pragma unroll
        for (int b0 = 0; b0 < STEPS; b0 += B) {
            if (ROWS == kCopy || b0 > 0) load(b0);
#pragma unroll
            for (int u = 0; u < B; ++u)
                if (dst[u] >= 0) {
                    const int64_t at = codes_at(dst[u]);
                    if constexpr (ROWS == kToE4m3) {
                        st_v4(kd + at, group_to_e4m3(kr[u][0], kr[u][N - 1], a.k_round));
                        st_v4(vd + at, group_to_e4m3(vr[u][0], vr[u][N - 1], a.v_round));
                    } else if constexpr (ROWS == kToE2m1) {
                        uint32_t s, z;
                        *reinterpret_cast<uint2 *>(kd + at) = group_to_e2m1(kr[u][0], kr[u][N - 1], a.k_round, s);
                        *reinterpret_cast<uint2 *>(vd + at) = group_to_e2m1(vr[u][0], vr[u][N - 1], a.v_round, z);
                        const int64_t to_scales = scales_at(dst[u]) + lr;
                        a.k[to_scales] = (uint8_t)s;
                        a.v[to_scales] = (uint8_t)z;
                    } else {
                        st_v4(kd + at, kr[u][0]);
                        st_v4(vd + at, vr[u][0]);
                    }
                }
        }
        if constexpr (ROWS == kCopyCodes)
            if (to >= 0) {
                const int64_t d = scales_at(to);
                *reinterpret_cast<S *>(a.k + d) = k_scales;
                *reinterpret_cast<S *>(a.v + d) = v_scales;
            }
        from = next_from;
        to = next_to;
    }
}

template <Rows ROWS>
const void *compact_lanes(int64_t lanes)
{
    if constexpr (ROWS == kCopyCodes)
        if (lanes == 2) return (const void *)k_page_compact<2, ROWS>;
    if constexpr (ROWS != kCopyCodes)
        if (lanes == 16) return (const void *)k_page_compact<16, ROWS>;
    if constexpr (ROWS == kCopy)
        if (lanes == 32) return (const void *)k_page_compact<32, ROWS>;
    return lanes == 4 ? (const void *)k_page_compact<4, ROWS> : lanes == 8 ? (const void *)k_page_compact<8, ROWS> : nullptr;
}

const void *compact_fn(const PageArgs &a)
{
    if (a.quantize == 1) return compact_lanes<kToE4m3>(a.row_bytes / 16);
    if (a.quantize == 2) return compact_lanes<kToE2m1>(a.row_bytes / 8);
    return a.scale_bytes ? compact_lanes<kCopyCodes>(a.row_bytes / 16) : compact_lanes<kCopy>(a.row_bytes / 16);
}

cudaError_t launch_dependent(const void *fn, int64_t grid, void **args, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kPageThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_page_call(const PageArgs &pa, cudaStream_t st)
{
    PageArgs a = pa;
    const int64_t lists = (int64_t)a.batch * a.heads;
    const unsigned plan = (unsigned)(a.row_chunks + a.page_chunks);
    void *args[] = {&a};
    cudaError_t e;
    if (plan <= kPlanCluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kPlanCluster);
        cfg.blockDim = dim3(kPageThreads);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kPlanCluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        // (as many warps as there are lists: their update comes along)
        const bool update = !a.kept && lists <= kPlanCluster * (kPageThreads / 32);
        const void *fn = a.kept   ? (const void *)k_page_plan<true, false>
                         : update ? (const void *)k_page_plan<false, true>
                                  : (const void *)k_page_plan<false, false>;
        if ((e = cudaLaunchKernelExC(&cfg, fn, args)) != cudaSuccess || update) return e;
    } else {
        if (a.kept) k_page_count<true><<<plan, kPageThreads, 0, st>>>(a);
        else k_page_count<false><<<plan, kPageThreads, 0, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const void *assign = a.kept ? (const void *)k_page_assign<true> : (const void *)k_page_assign<false>;
        if ((e = launch_dependent(assign, plan, args, st)) != cudaSuccess) return e;
    }
    if (!a.kept)
        return launch_dependent((const void *)k_page_update, (lists * 32 + kPageThreads - 1) / kPageThreads, args, st);
    const void *fn = compact_fn(a);
    if (!fn) return cudaErrorInvalidValue;
    // no more items than the pages that can be taken have
    const int64_t most = a.idx ? std::min((int64_t)a.idx_stride, (int64_t)a.max_pages << a.page_shift)
                               : std::min((int64_t)(a.K ? a.t_max : INT32_MAX), (int64_t)a.max_pages << a.page_shift);
    const int64_t pages = std::min((int64_t)a.n_pages, lists * ((most + a.page_size - 1) >> a.page_shift));
    const int64_t items = pages << (a.page_shift - 4);
    int list_ctas = (int)std::min<int64_t>(lists, 152);
    const int64_t copy_ctas = grid_for_items(fn, kPageThreads, 0, (items + kPageThreads / 32 - 1) / (kPageThreads / 32));
    void *cargs[] = {&a, &list_ctas};
    return launch_dependent(fn, list_ctas + copy_ctas, cargs, st);
}

}  // namespace mkv
