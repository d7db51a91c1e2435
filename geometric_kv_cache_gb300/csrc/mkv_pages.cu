// sm_103a page lists of a paged cache: fork, copy, free and extend
// (mkv_page_update), and compaction into new pages (mkv_page_compact).
//
// The ManifoldKV path ends with a compacted cache whose heads differ in
// length ("ManifoldKV: Training-Free KV Cache Compression via Euclidean
// Outlier Detection", ICML 2026 poster 62526, abstract: which past tokens the
// cache retains). A serving engine keeps it in pages, one list per head.
//
// A call is three launches, each a programmatic dependent of the one before
// (small problems do the first two in one, k_page_plan):
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
// the rows moved) 15 us, of 8 rows 11 us: three round trips of latency each; the
// compaction of 64 lists of 8K-32K tokens to half 122 us, 107 of it the copy, 6.3
// TB/s, 0.93 of the measured copy peak.
// Integers only decide, and every rank is a prefix sum: nothing depends on
// the order of the atomics (counts are sums).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mkv_device.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kPageThreads = 256;
// Problems of up to 8 chunks (of 8 rows, of 4096 pages) are planned by one
// cluster, a chunk per CTA, in one launch; larger ones in two. 16 rows x 8 heads of
// 500-2048 tokens (5 chunks): one launch 13.1 us per call from Python and 11.4 us
// in a graph, two 15.2 and 11.1; 32 rows (10 chunks, two per CTA): 16.4 and 14.7
// against 15.2 and 11.6.
constexpr int kPlanCluster = 8;
// Tokens per item of the compaction: a page holds a whole number of them, and
// small items even out the warps' shares. With 4 rows of K and of V in flight
// per lane and 3 CTAs per SM, 8 rows of 8K-32K tokens halved take 123 us (107 us
// of it the copy, 0.93 of the copy peak); 8 in flight and 2 CTAs 127 us, with
// items of 32 tokens 128 us.
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
    if (a.kept) {
        p.len = a.kept[(int64_t)b * a.heads + j];
        p.total = pages_of(p.len, a);
        return p;
    }
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
__device__ __forceinline__ void load_refs(const PageArgs &a, int chunk, int (&r)[kPlanPages / kPageThreads])
{
    constexpr int N = kPlanPages / kPageThreads;
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

// Chunk c of the rows, or after them of the pool: what its lists need, what is
// free.
__device__ __forceinline__ void count_chunk(const PageArgs &a, int c)
{
    __shared__ long long s_need[kPlanRows];
    __shared__ uint32_t s_bits[kPlanRows];
    __shared__ int s_free[kPageThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (c < a.row_chunks) {
        const int64_t b = (int64_t)c * kPlanRows + warp;
        long long need = 0;
        uint32_t bits = 0;
        if (b < a.batch) {
            int src = (int)b;
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
            const int add = a.n_new && src >= 0 && !a.kept ? a.n_new[b] : 0;
            if (add < 0) bits |= MKV_DEV_BAD_PARENT;
            for (int j = lane; j < a.heads; j += 32) {
                const int64_t h = b * a.heads + j;
                if (!len_ok(a.lens[h], a)) bits |= MKV_DEV_BAD_SEQ_LEN;
                if (a.kept) {
                    const int n = a.kept[h];
                    bool ok = len_ok(n, a) && (!a.idx || n <= a.idx_stride);
                    if (ok && !a.idx) {  // tokens 0 .. n-1 must be there
                        const int T = !a.K ? a.lens[h] : a.seq_lens ? a.seq_lens[b] : a.t_max;
                        ok = n <= T;
                    }
                    if (!ok) {
                        bits |= MKV_DEV_BAD_N_KEEP;
                        continue;
                    }
                } else if (src >= 0) {
                    const int L = a.lens[(int64_t)src * a.heads + j];
                    if (!len_ok(L, a)) continue;  // reported by its own row
                    if (add < 0 || (long long)L + add > ((long long)a.max_pages << a.page_shift)) {
                        bits |= MKV_DEV_BAD_PARENT;
                        continue;
                    }
                }
                const ListPlan p = plan_list(a, (int)b, j, src, keeps);
                need += p.total - p.shared;
            }
            if (a.kept && a.K && a.seq_lens && (a.seq_lens[b] < 0 || a.seq_lens[b] > a.t_max))
                bits |= MKV_DEV_BAD_SEQ_LEN;
            need = warp_sum(need);
            bits = __reduce_or_sync(kFull, bits);
        }
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
        int r[kPlanPages / kPageThreads], n = 0;
        load_refs(a, chunk, r);
#pragma unroll
        for (int i = 0; i < kPlanPages / kPageThreads; ++i) n += r[i] == 0;
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
// pages, or its free pages by rank. Chunk 0 writes the verdict.
__device__ __forceinline__ void assign_chunk(const PageArgs &a, int c)
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
        const int64_t b = (int64_t)chunk * kPlanRows + warp;
        const int2 src = b < a.batch ? a.row_src[b] : make_int2(-1, 0);
        long long row = 0;
        if (b < a.batch)
            for (int j = lane; j < a.heads; j += 32) {
                const ListPlan p = plan_list(a, (int)b, j, src.x, src.y != 0);
                row += p.total - p.shared;
            }
        row = warp_sum(row);
        if (lane == 0) s_row[warp] = row;
        __syncthreads();
        int off = (int)before;  // at most n_pages: the verdict was good
        for (int i = 0; i < warp; ++i) off += (int)s_row[i];
        if (b >= a.batch) return;
        for (int j0 = 0; j0 < a.heads; j0 += 32) {
            const int j = j0 + lane;
            int n = 0;
            if (j < a.heads) {
                const ListPlan p = plan_list(a, (int)b, j, src.x, src.y != 0);
                n = p.total - p.shared;
            }
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            if (j < a.heads) a.list_off[b * a.heads + j] = off + x - n;
            if (a.kept)  // whose each new page is
                for (int k = 0; k < min(32, a.heads - j0); ++k) {
                    const int m = __shfl_sync(kFull, n, k), at = off + __shfl_sync(kFull, x, k) - m;
                    for (int q = lane; q < m; q += 32) a.owners[at + q] = make_int2((int)(b * a.heads) + j0 + k, q);
                }
            off += __shfl_sync(kFull, x, 31);
        }
    } else {
        constexpr int N = kPlanPages / kPageThreads;
        const int64_t p0 = (int64_t)chunk * kPlanPages + threadIdx.x * N;
        int r[N], n = 0;
        load_refs(a, chunk, r);
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

__global__ void __launch_bounds__(kPageThreads)
k_page_count(const PageArgs a)
{
    pdl_trigger();
    count_chunk(a, (int)blockIdx.x);
}

__global__ void __launch_bounds__(kPageThreads)
k_page_assign(const PageArgs a)
{
    pdl_trigger();
    pdl_wait();
    assign_chunk(a, (int)blockIdx.x);
}

// Both in one launch of one cluster, for problems of few chunks.
__global__ void __launch_bounds__(kPageThreads)
k_page_plan(const PageArgs a)
{
    pdl_trigger();
    const bool mine = (int)blockIdx.x < a.row_chunks + a.page_chunks;
    if (mine) count_chunk(a, (int)blockIdx.x);
    __syncthreads();
    // every CTA's counts are there
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (mine) assign_chunk(a, (int)blockIdx.x);
}

__device__ __forceinline__ void add_ref(const PageArgs &a, int page, int by)
{
    if ((uint32_t)page < (uint32_t)a.n_pages)
        atomicAdd(a.refs_out + page, by);
    else
        atomicOr(a.status, MKV_DEV_BAD_PAGE);
}

// One warp per list.
__global__ void __launch_bounds__(kPageThreads)
k_page_update(const PageArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t h = ((int64_t)blockIdx.x * kPageThreads + threadIdx.x) >> 5;
    if (h >= (int64_t)a.batch * a.heads) return;
    const int b = (int)(h / a.heads), j = (int)(h - (int64_t)b * a.heads);
    const bool in_place = a.lens_out == a.lens;  // (lists without capacity may have no tables at all)
    const int32_t *mine = a.table + h * a.max_pages;
    int32_t *out = a.table_out + h * a.max_pages;
    // (read together; the last two mean nothing after a bad verdict)
    const int own_len = a.lens[h];
    const uint32_t verdict = a.verdict[0];
    const int2 src = a.row_src[b];
    const int first = a.list_off[h];
    if (verdict) {  // the lists stay as they were
        if (in_place) return;
        if (lane == 0) a.lens_out[h] = own_len;
        if (len_ok(own_len, a))
            for (int p = lane; p < pages_of(own_len, a); p += 32) out[p] = mine[p];
        return;
    }
    const bool keeps = src.y != 0, moved = src.x != b;
    const ListPlan lp = plan_list(a, b, j, src.x, keeps);
    const int32_t *from = a.table + ((int64_t)(src.x < 0 ? b : src.x) * a.heads + j) * a.max_pages;
    __syncwarp();
    if (!in_place)
        for (int p = lane; p < lp.shared; p += 32) {
            const int id = from[p];
            out[p] = id;
            if (moved) add_ref(a, id, 1);
        }
    for (int p = lp.shared + lane; p < lp.total; p += 32) {
        const int id = a.free_ids[first + p - lp.shared];
        out[p] = id;
        atomicAdd(a.refs_out + id, 1);
    }
    if (moved)  // nobody continues this list under its own row: its holder goes
        for (int p = lane; p < pages_of(own_len, a); p += 32) add_ref(a, mine[p], -1);
    if (lane == 0) a.lens_out[h] = lp.len;
    const int rest = lp.old_len & (a.page_size - 1);
    if (!keeps && rest > 0) {  // a copy of the partly filled last page
        const int s = from[lp.shared], d = a.free_ids[first];
        if ((uint32_t)s >= (uint32_t)a.n_pages) {
            if (lane == 0) atomicOr(a.status, MKV_DEV_BAD_PAGE);
            return;
        }
        const int64_t page_bytes = a.row_bytes << a.page_shift, n = rest * a.row_bytes;
        const uint8_t *ks = a.k + s * page_bytes, *vs = a.v + s * page_bytes;
        uint8_t *kd = a.k + d * page_bytes, *vd = a.v + d * page_bytes;
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

// The first `list_ctas` CTAs write tables and counts, list by list; the warps
// of the others copy rows. Item = 16 tokens of a new page, one lane per token
// for its places; owners[rank] names a new page's list and place in it,
// so the items are the pages taken, whatever the lists' lengths and capacities.
// An item's owner is read three items ahead, its indices two and its page
// entries one, so that every row copy (groups of LPR lanes, 16 bytes each, 4
// rows of K and of V in flight per lane) finds its addresses in registers.
template <int LPR>
__global__ void __launch_bounds__(kPageThreads, 3)
k_page_compact(const PageArgs a, int list_ctas)
{
    constexpr int RB = LPR * 16, RPS = 32 / LPR;  // bytes of a row, rows per step
    constexpr int STEPS = kItem / RPS, B = STEPS < 4 ? STEPS : 4;  // steps, and of a batch
    pdl_wait();
    const bool bad = a.verdict[0] != 0;
    const int64_t lists = (int64_t)a.batch * a.heads;
    if ((int)blockIdx.x < list_ctas) {
        for (int64_t h = blockIdx.x; h < lists; h += list_ctas) {
            const int own_len = a.lens[h], n = bad ? 0 : a.kept[h], first = bad ? 0 : a.list_off[h];
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
    if (bad) return;
    const int lane = threadIdx.x & 31, g = lane / LPR, lr = lane % LPR;
    const int per_shift = a.page_shift - 4;  // items of a page
    const int64_t warps = (int64_t)(gridDim.x - list_ctas) * (kPageThreads / 32);
    const int64_t warp = (int64_t)(blockIdx.x - list_ctas) * (kPageThreads / 32) + (threadIdx.x >> 5);
    const int64_t items = (int64_t)a.verdict[1] << per_shift;  // pages taken
    auto owner = [&](int64_t item) -> int2 {
        return item < items ? a.owners[item >> per_shift] : make_int2(-1, 0);
    };
    // an item: its list, its new page's rank, and this lane's token of it with its source (-1: none)
    struct Item {
        int h, rank, i, s;
    };
    auto source = [&](int64_t item, int2 own) -> Item {
        Item it = {own.x, (int)(item >> per_shift), -1, -1};
        if (own.x < 0 || lane >= kItem) return it;
        const int64_t h = own.x;
        const int i = (own.y << a.page_shift) + (int)(item & ((1 << per_shift) - 1)) * kItem + lane;
        // (read together: an index behind the kept ones is not looked at)
        const int kept = a.kept[h], s = !a.idx ? i : i < a.idx_stride ? a.idx[h * a.idx_stride + i] : -1;
        if (i >= kept) return it;
        const int T = !a.K ? a.lens[h] : a.seq_lens ? a.seq_lens[own.x / a.heads] : a.t_max;
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
        to = (a.free_ids[it.rank] << a.page_shift) + (it.i & (a.page_size - 1));
    };
    const uint8_t *ks = (a.K ? a.K : a.k) + lr * 16, *vs = (a.K ? a.V : a.v) + lr * 16;
    uint8_t *kd = a.k + lr * 16, *vd = a.v + lr * 16;
    int64_t from;
    int to;
    Item ahead = source(warp, owner(warp));
    int2 own = owner(warp + warps);
    places(ahead, from, to);
    ahead = source(warp + warps, own);
    own = owner(warp + 2 * warps);
    for (int64_t item = warp; item < items; item += warps) {
        int64_t next_from;
        int next_to;
        places(ahead, next_from, next_to);
        ahead = source(item + 2 * warps, own);
        own = owner(item + 3 * warps);
#pragma unroll
        for (int b0 = 0; b0 < STEPS; b0 += B) {
            uint4 kr[B], vr[B];
            int dst[B];
#pragma unroll
            for (int u = 0; u < B; ++u) {
                const int row = (b0 + u) * RPS + g;
                const int64_t src = __shfl_sync(kFull, from, row);
                dst[u] = __shfl_sync(kFull, to, row);
                if (dst[u] >= 0) {
                    kr[u] = ld_stream(ks + src * RB);
                    vr[u] = ld_stream(vs + src * RB);
                }
            }
#pragma unroll
            for (int u = 0; u < B; ++u)
                if (dst[u] >= 0) {
                    st_v4(kd + (int64_t)dst[u] * RB, kr[u]);
                    st_v4(vd + (int64_t)dst[u] * RB, vr[u]);
                }
        }
        from = next_from;
        to = next_to;
    }
}

const void *compact_fn(int64_t row_bytes)
{
    switch (row_bytes) {
    case 64: return (const void *)k_page_compact<4>;
    case 128: return (const void *)k_page_compact<8>;
    case 256: return (const void *)k_page_compact<16>;
    case 512: return (const void *)k_page_compact<32>;
    default: return nullptr;
    }
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
        if ((e = cudaLaunchKernelExC(&cfg, (const void *)k_page_plan, args)) != cudaSuccess) return e;
    } else {
        k_page_count<<<plan, kPageThreads, 0, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_dependent((const void *)k_page_assign, plan, args, st)) != cudaSuccess) return e;
    }
    if (!a.kept)
        return launch_dependent((const void *)k_page_update, (lists * 32 + kPageThreads - 1) / kPageThreads, args, st);
    const void *fn = compact_fn(a.row_bytes);
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
