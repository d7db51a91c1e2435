// C ABI of the paged-cache calls (declared in include/mkv.h): host-side
// argument checks, workspace carving and the launches. Nothing here allocates
// device memory or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "mkv_pages.h"

namespace mkv {

namespace {

constexpr size_t kAlign = 256;
// Where the workspace's head holds the counts of cut tiles' parts.
constexpr size_t kCounts = 64;
static_assert(kCounts + kPlanSms <= kAlign && kPlanSms < 256, "a byte per CTA");

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename T>
T *region(void *ws, size_t off)
{
    return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}

mkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MKV_OK : MKV_ERR_CUDA; }

int page_shift(int32_t page_size)
{
    for (int s = 4; s <= 7; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Sizes of a pool and its lists (no pointers).
mkv_status check_sizes(const mkv_page_pool &p, const mkv_page_lists &l)
{
    if (p.n_pages < 0 || p.page_size <= 0 || p.head_dim <= 0) return MKV_ERR_INVALID_ARG;
    if (l.batch < 0 || l.heads < 0 || l.max_pages < 0) return MKV_ERR_INVALID_ARG;
    if (!supported_head_dim(p.head_dim) || elem_bytes(p.dtype) == 0) return MKV_ERR_UNSUPPORTED;
    if (page_shift(p.page_size) < 0) return MKV_ERR_UNSUPPORTED;
    if ((int64_t)p.n_pages * p.page_size > (1 << 30) || (int64_t)l.max_pages * p.page_size > (1 << 30))
        return MKV_ERR_UNSUPPORTED;
    if (l.batch > 65536 || (int64_t)l.batch * l.heads > (1 << 24)) return MKV_ERR_UNSUPPORTED;
    return MKV_OK;
}

bool no_lists(const mkv_page_lists &l) { return l.batch == 0 || l.heads == 0; }

mkv_status check_pointers(const mkv_page_pool &p, const mkv_page_lists &l)
{
    if (p.n_pages > 0 && (!p.k_pages || !p.v_pages || p.k_pages == p.v_pages)) return MKV_ERR_INVALID_ARG;
    if (!aligned(p.k_pages, 16) || !aligned(p.v_pages, 16)) return MKV_ERR_INVALID_ARG;
    if (!no_lists(l) && ((l.max_pages > 0 && !l.table) || !l.lens)) return MKV_ERR_INVALID_ARG;
    if (!aligned(l.table, 4) || !aligned(l.lens, 4)) return MKV_ERR_INVALID_ARG;
    return MKV_OK;
}

mkv_status check_tokens(const mkv_new_tokens &t, const mkv_page_lists &l)
{
    if (t.n_tokens < 0 || t.q_heads <= 0) return MKV_ERR_INVALID_ARG;
    if (l.heads > 0 && t.q_heads % l.heads != 0) return MKV_ERR_INVALID_ARG;
    if (t.q_heads > 1024) return MKV_ERR_UNSUPPORTED;
    return MKV_OK;
}

// Tokens of `heads` rows of head_dim bf16 elements, `stride` elements apart.
bool rows_ok(const void *p, int64_t stride, int32_t heads, int32_t head_dim)
{
    return p && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * head_dim && stride <= (1 << 30);
}

PageLayout make_page_layout(const mkv_page_pool &p, const mkv_page_lists &l)
{
    const size_t lists = (size_t)l.batch * l.heads;
    const size_t row_chunks = ((size_t)l.batch + kPlanRows - 1) / kPlanRows;
    const size_t page_chunks = ((size_t)p.n_pages + kPlanPages - 1) / kPlanPages;
    // no call takes more pages than the pool has, nor more than its lists hold
    const size_t taken = std::min((size_t)p.n_pages, lists * (size_t)l.max_pages);
    PageLayout L;
    size_t at = kAlign;  // the status word
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round_up(bytes, kAlign);
        return here;
    };
    L.verdict = take(2 * sizeof(uint32_t));
    L.row_src = take((size_t)l.batch * sizeof(int2));
    L.row_need = take(row_chunks * sizeof(long long));
    L.row_bits = take(row_chunks * sizeof(uint32_t));
    L.page_free = take(page_chunks * sizeof(int32_t));
    L.list_off = take(lists * sizeof(int32_t));
    L.free_ids = take(taken * sizeof(int32_t));
    L.owners = take(taken * sizeof(int2));
    L.total = at;
    return L;
}

mkv_status check_ws(size_t need, void *ws, size_t ws_bytes)
{
    if (!ws || !aligned(ws, kAlign) || ws_bytes < need) return MKV_ERR_WORKSPACE;
    return MKV_OK;
}

// Checks and arguments that the update and the compaction share.
mkv_status page_call(const mkv_page_pool &p, const mkv_page_lists &in, const int32_t *refs, const mkv_page_lists &out,
                     int32_t *refs_out, bool may_be_in_place, void *ws, size_t ws_bytes, PageArgs *a)
{
    mkv_status rc = check_sizes(p, in);
    if (rc != MKV_OK) return rc;
    if (out.batch != in.batch || out.heads != in.heads || out.max_pages != in.max_pages) return MKV_ERR_INVALID_ARG;
    if ((rc = check_pointers(p, in)) != MKV_OK || (rc = check_pointers(p, out)) != MKV_OK) return rc;
    if (p.n_pages > 0 && (!refs || !refs_out)) return MKV_ERR_INVALID_ARG;
    if (!aligned(refs, 4) || !aligned(refs_out, 4)) return MKV_ERR_INVALID_ARG;
    if (!no_lists(in)) {
        const bool same_table = in.max_pages > 0 ? in.table == out.table : in.lens == out.lens;
        const bool same_lens = in.lens == out.lens;
        if (same_table != same_lens || (same_lens && !may_be_in_place)) return MKV_ERR_INVALID_ARG;
    }
    const PageLayout L = make_page_layout(p, in);
    if ((rc = check_ws(L.total, ws, ws_bytes)) != MKV_OK) return rc;
    a->n_pages = p.n_pages;
    a->page_size = p.page_size;
    a->page_shift = page_shift(p.page_size);
    a->batch = in.batch;
    a->heads = in.heads;
    a->max_pages = in.max_pages;
    a->row_bytes = (int64_t)p.head_dim * elem_bytes(p.dtype);
    a->k = static_cast<uint8_t *>(p.k_pages);
    a->v = static_cast<uint8_t *>(p.v_pages);
    a->table = in.table;
    a->lens = in.lens;
    a->refs = refs;
    a->table_out = out.table;
    a->lens_out = out.lens;
    a->refs_out = refs_out;
    a->status = region<uint32_t>(ws, L.status);
    a->verdict = region<uint32_t>(ws, L.verdict);
    a->row_src = region<int2>(ws, L.row_src);
    a->row_need = region<long long>(ws, L.row_need);
    a->row_bits = region<uint32_t>(ws, L.row_bits);
    a->page_free = region<int32_t>(ws, L.page_free);
    a->list_off = region<int32_t>(ws, L.list_off);
    a->free_ids = region<int32_t>(ws, L.free_ids);
    a->owners = region<int2>(ws, L.owners);
    a->row_chunks = (in.batch + kPlanRows - 1) / kPlanRows;
    a->page_chunks = (p.n_pages + kPlanPages - 1) / kPlanPages;
    return MKV_OK;
}

}  // namespace
}  // namespace mkv

using namespace mkv;

extern "C" {

size_t mkv_page_workspace_size(mkv_page_pool pool, mkv_page_lists lists)
{
    return check_sizes(pool, lists) == MKV_OK ? make_page_layout(pool, lists).total : 0;
}

mkv_status mkv_page_update(mkv_page_pool pool, mkv_page_lists in, const int32_t *refs, const int32_t *parent,
                           const int32_t *n_new, mkv_page_lists out, int32_t *refs_out, void *workspace,
                           size_t workspace_bytes, mkv_stream_t stream)
{
    PageArgs a = {};
    const mkv_status rc = page_call(pool, in, refs, out, refs_out, parent == nullptr, workspace, workspace_bytes, &a);
    if (rc != MKV_OK) return rc;
    if (!aligned(parent, 4) || !aligned(n_new, 4)) return MKV_ERR_INVALID_ARG;
    if (no_lists(in)) {
        // no list: the counts alone carry over
        if (refs_out != refs && pool.n_pages > 0)
            return cuda_status(cudaMemcpyAsync(refs_out, refs, (size_t)pool.n_pages * sizeof(int32_t),
                                               cudaMemcpyDeviceToDevice, reinterpret_cast<cudaStream_t>(stream)));
        return MKV_OK;
    }
    a.parent = parent;
    a.n_new = n_new;
    return cuda_status(launch_page_call(a, reinterpret_cast<cudaStream_t>(stream)));
}

mkv_status mkv_page_compact(mkv_page_pool pool, mkv_page_lists in, const int32_t *refs, const int32_t *idx,
                            int32_t idx_stride, const int32_t *kept, const void *K, const void *V, int32_t t_max,
                            const int32_t *seq_lens, mkv_page_lists out, int32_t *refs_out, void *workspace,
                            size_t workspace_bytes, mkv_stream_t stream)
{
    PageArgs a = {};
    const mkv_status rc = page_call(pool, in, refs, out, refs_out, false, workspace, workspace_bytes, &a);
    if (rc != MKV_OK) return rc;
    if ((K == nullptr) != (V == nullptr) || !aligned(K, 16) || !aligned(V, 16)) return MKV_ERR_INVALID_ARG;
    if (K && t_max < 0) return MKV_ERR_INVALID_ARG;
    if (K && t_max > (1 << 30)) return MKV_ERR_UNSUPPORTED;
    if (idx && idx_stride < 0) return MKV_ERR_INVALID_ARG;
    if (!aligned(idx, 4) || !aligned(kept, 4) || !aligned(seq_lens, 4)) return MKV_ERR_INVALID_ARG;
    if (no_lists(in)) {
        if (refs_out != refs && pool.n_pages > 0)
            return cuda_status(cudaMemcpyAsync(refs_out, refs, (size_t)pool.n_pages * sizeof(int32_t),
                                               cudaMemcpyDeviceToDevice, reinterpret_cast<cudaStream_t>(stream)));
        return MKV_OK;
    }
    if (!kept) return MKV_ERR_INVALID_ARG;
    a.idx = idx;
    a.idx_stride = idx_stride;
    a.kept = kept;
    a.K = static_cast<const uint8_t *>(K);
    a.V = static_cast<const uint8_t *>(V);
    a.t_max = t_max;
    a.seq_lens = seq_lens;
    return cuda_status(launch_page_call(a, reinterpret_cast<cudaStream_t>(stream)));
}

mkv_status mkv_rope_append(const void *Q, int64_t q_stride, const void *K, int64_t k_stride, const void *V,
                           int64_t v_stride, mkv_new_tokens tokens, const int32_t *positions, const float *inv_freq,
                           int32_t rot_dim, mkv_rope_layout layout, float factor, void *Q_out, mkv_page_pool pool,
                           mkv_page_lists lists, float k_scale, float v_scale, void *workspace, size_t workspace_bytes,
                           mkv_stream_t stream)
{
    mkv_status rc = check_sizes(pool, lists);
    if (rc != MKV_OK || (rc = check_tokens(tokens, lists)) != MKV_OK) return rc;
    if ((rc = check_pointers(pool, lists)) != MKV_OK) return rc;
    const int d = pool.head_dim, es = elem_bytes(pool.dtype);
    if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0) return MKV_ERR_INVALID_ARG;
    if (layout != MKV_ROPE_HALF && layout != MKV_ROPE_INTERLEAVED) return MKV_ERR_INVALID_ARG;
    if (!isfinite(factor) || !isfinite(k_scale) || !isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f) ||
        !isfinite(1.f / k_scale) || !isfinite(1.f / v_scale))
        return MKV_ERR_INVALID_ARG;
    if (es == 2 && (k_scale != 1.f || v_scale != 1.f)) return MKV_ERR_INVALID_ARG;
    const bool none = tokens.n_tokens == 0 || no_lists(lists);
    if (!none) {
        if (!rows_ok(Q, q_stride, tokens.q_heads, d) || !rows_ok(K, k_stride, lists.heads, d) ||
            !rows_ok(V, v_stride, lists.heads, d) || !rows_ok(Q_out, (int64_t)tokens.q_heads * d, tokens.q_heads, d))
            return MKV_ERR_INVALID_ARG;
        if (Q_out == Q && q_stride != (int64_t)tokens.q_heads * d) return MKV_ERR_INVALID_ARG;
        if (!tokens.q_start || !positions || !inv_freq) return MKV_ERR_INVALID_ARG;
        if (!aligned(tokens.q_start, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4)) return MKV_ERR_INVALID_ARG;
    }
    if ((rc = check_ws(make_page_layout(pool, lists).total, workspace, workspace_bytes)) != MKV_OK) return rc;
    if (none) return MKV_OK;
    RopeArgs a = {};
    a.Q = static_cast<const uint8_t *>(Q);
    a.K = static_cast<const uint8_t *>(K);
    a.V = static_cast<const uint8_t *>(V);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.Q_out = static_cast<uint8_t *>(Q_out);
    a.positions = positions;
    a.q_start = tokens.q_start;
    a.table = lists.table;
    a.lens = lists.lens;
    a.inv_freq = inv_freq;
    a.k = static_cast<uint8_t *>(pool.k_pages);
    a.v = static_cast<uint8_t *>(pool.v_pages);
    a.n_tokens = tokens.n_tokens;
    a.q_heads = tokens.q_heads;
    a.batch = lists.batch;
    a.heads = lists.heads;
    a.max_pages = lists.max_pages;
    a.n_pages = pool.n_pages;
    a.page_size = pool.page_size;
    a.page_shift = page_shift(pool.page_size);
    a.head_dim = d;
    a.es = es;
    a.rot_dim = rot_dim;
    a.layout = layout;
    a.factor = factor;
    a.k_inv = 1.f / k_scale;
    a.v_inv = 1.f / v_scale;
    a.status = region<uint32_t>(workspace, 0);
    return cuda_status(launch_rope_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t mkv_rope_frequencies(int32_t rot_dim, double theta, mkv_rope_scaling scaling, double scale,
                             int32_t original_len, double low_turns, double high_turns, float *inv_freq)
{
    if (rot_dim <= 0 || rot_dim % 16 != 0 || !(theta > 1.0) || !isfinite(theta) || !(scale >= 1.0) || !isfinite(scale) ||
        !inv_freq)
        return -1;
    if (scaling != MKV_ROPE_PLAIN && scaling != MKV_ROPE_LINEAR && scaling != MKV_ROPE_BY_PARTS) return -1;
    if (scaling == MKV_ROPE_BY_PARTS &&
        (original_len < 1 || !(low_turns > 0.0) || !(high_turns > low_turns) || !isfinite(high_turns)))
        return -1;
    for (int32_t i = 0; i < rot_dim / 2; ++i) {
        double f = pow(theta, -2.0 * i / rot_dim);
        if (scaling == MKV_ROPE_LINEAR) f /= scale;
        if (scaling == MKV_ROPE_BY_PARTS) {
            const double turns = original_len * f / (2.0 * M_PI);
            const double g = fmin(fmax((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0);
            f *= g + (1.0 - g) / scale;
        }
        inv_freq[i] = (float)f;
    }
    return 0;
}

// Status, then the parts of the key axis.
static mkv_status attention_sizes(const mkv_page_pool &pool, const mkv_page_lists &lists, const mkv_new_tokens &tokens,
                                  int32_t max_q, int32_t max_len, AttnPlan *plan)
{
    mkv_status rc = check_sizes(pool, lists);
    if (rc != MKV_OK || (rc = check_tokens(tokens, lists)) != MKV_OK) return rc;
    if (max_q < 0 || max_len < 0 || max_len > (int64_t)lists.max_pages * pool.page_size) return MKV_ERR_INVALID_ARG;
    if (max_q > (1 << 20)) return MKV_ERR_UNSUPPORTED;
    *plan = AttnPlan();
    if (no_lists(lists) || max_q == 0) return MKV_OK;
    const int64_t n = (int64_t)lists.batch * lists.heads;
    *plan = attention_plan(lists.batch, lists.heads, tokens.q_heads / lists.heads, tokens.n_tokens, max_q, max_len,
                           pool.head_dim, elem_bytes(pool.dtype), kPlanSms);
    // blocks of at least 64 keys of all tiles are counted in 32 bits
    if (n * plan->tiles > (int64_t)INT32_MAX / ((int64_t)max_len / 64 + 2))
        return MKV_ERR_UNSUPPORTED;
    return MKV_OK;
}

size_t mkv_attention_workspace_size(mkv_page_pool pool, mkv_page_lists lists, mkv_new_tokens tokens, int32_t max_q,
                                    int32_t max_len)
{
    AttnPlan plan;
    if (attention_sizes(pool, lists, tokens, max_q, max_len, &plan) != MKV_OK) return 0;
    return kAlign + round_up(plan.bytes, kAlign);
}

mkv_status mkv_paged_attention(const void *Q, int64_t q_stride, mkv_new_tokens tokens, int32_t max_q,
                               mkv_page_pool pool, mkv_page_lists lists, int32_t max_len, float scale, float k_scale,
                               float v_scale, int32_t window, int32_t sinks, void *O, int64_t o_stride, float *lse,
                               void *workspace, size_t workspace_bytes, mkv_stream_t stream)
{
    AttnPlan plan;
    mkv_status rc = attention_sizes(pool, lists, tokens, max_q, max_len, &plan);
    if (rc != MKV_OK || (rc = check_pointers(pool, lists)) != MKV_OK) return rc;
    if (window < 0 || sinks < 0) return MKV_ERR_INVALID_ARG;
    if (!isfinite(scale) || !isfinite(k_scale) || !isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f))
        return MKV_ERR_INVALID_ARG;
    if (elem_bytes(pool.dtype) == 2 && (k_scale != 1.f || v_scale != 1.f)) return MKV_ERR_INVALID_ARG;
    const float scale_log2 = (float)((double)scale * (double)k_scale * M_LOG2E);
    if (!isfinite(scale_log2)) return MKV_ERR_INVALID_ARG;  // (infinity times a score of 0 would be NaN)
    const int d = pool.head_dim;
    const bool none = tokens.n_tokens == 0 || no_lists(lists) || max_q == 0;
    if (!none) {
        if (pool.n_pages == 0) return MKV_ERR_INVALID_ARG;
        if (!rows_ok(Q, q_stride, tokens.q_heads, d) || !rows_ok(O, o_stride, tokens.q_heads, d) || O == Q)
            return MKV_ERR_INVALID_ARG;
        if (!tokens.q_start || !aligned(tokens.q_start, 4) || !aligned(lse, 4)) return MKV_ERR_INVALID_ARG;
    }
    if ((rc = check_ws(kAlign + round_up(plan.bytes, kAlign), workspace, workspace_bytes)) != MKV_OK) return rc;
    if (none) return MKV_OK;
    AttnArgs a = {};
    a.Q = static_cast<const uint8_t *>(Q);
    a.O = static_cast<uint8_t *>(O);
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.q_start = tokens.q_start;
    a.table = lists.table;
    a.lens = lists.lens;
    a.k = static_cast<const uint8_t *>(pool.k_pages);
    a.v = static_cast<const uint8_t *>(pool.v_pages);
    a.n_tokens = tokens.n_tokens;
    a.q_heads = tokens.q_heads;
    a.group = tokens.q_heads / lists.heads;
    a.batch = lists.batch;
    a.heads = lists.heads;
    a.max_pages = lists.max_pages;
    a.n_pages = pool.n_pages;
    a.page_size = pool.page_size;
    a.page_shift = page_shift(pool.page_size);
    a.head_dim = d;
    a.es = elem_bytes(pool.dtype);
    a.max_q = max_q;
    a.max_len = max_len;
    a.window = std::min(window, std::max(max_len, 1));  // no list is longer
    a.sinks = sinks;
    a.scale_log2 = scale_log2;
    a.v_scale = v_scale;
    a.tiles = plan.tiles;
    a.ctas = plan.ctas;
    a.by_tiles = FastDiv(plan.tiles);
    a.by_heads = FastDiv(lists.heads);
    a.by_group = FastDiv(a.group);
    a.chunked = plan.chunked;
    a.part_o = region<float>(workspace, kAlign);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + plan.part_rows * d);
    a.status = region<uint32_t>(workspace, 0);
    a.counts = region<uint32_t>(workspace, kCounts);
    return cuda_status(launch_paged_attention(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
