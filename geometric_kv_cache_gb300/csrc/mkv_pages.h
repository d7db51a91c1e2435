// Internal declarations of the paged-cache kernels (mkv_pages.cu,
// mkv_rope.cu, mkv_attention.cu) and their C ABI (mkv_pages_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mkv_internal.h"

namespace mkv {

// The launches are planned for the 152 SMs of a GB300, so that workspace sizes
// need no device and results do not depend on one.
constexpr int kPlanSms = 152;
constexpr int kPlanPages = 4096;  // pages of refs per CTA of the plan kernels (256 threads x 16)
constexpr int kPlanRows = 8;      // rows, or runs of lists, per CTA of the plan kernels (one warp each)
constexpr int kPlanCluster = 8;   // chunks that one launch of the plan takes
constexpr int kPlanRuns = 4096;   // runs of a compaction's lists

// What a pool's rows are made of. es: bytes per element, 0 for 4-bit codes with
// an E4M3 scale per 16 dims (a page is its rows' codes, then its rows' scales).
constexpr bool pool_dtype(int32_t dtype) { return elem_bytes(dtype) != 0 || dtype == MKV_DTYPE_E2M1; }
constexpr int code_row_bytes(int32_t dtype, int d) { return dtype == MKV_DTYPE_E2M1 ? d / 2 : d * elem_bytes(dtype); }
constexpr int scale_row_bytes(int32_t dtype, int d) { return dtype == MKV_DTYPE_E2M1 ? d / 16 : 0; }

// How values become codes (mkv_rope_append, mkv_page_quantize): E4M3 takes value *
// inv, 4-bit groups inv6 = 1 / (6 scale) for their scale and inv = 1 / scale for
// their codes; each rounded once to fp32.
struct Rounding {
    float inv, inv6;
    Rounding() = default;
    explicit Rounding(float scale) : inv((float)(1.0 / scale)), inv6((float)(1.0 / (6.0 * scale))) {}
};

// Byte offsets of the page workspace (each 256-byte aligned).
struct PageLayout {
    size_t status = 0, verdict = 0, row_src = 0, row_need = 0, row_bits = 0, page_free = 0, list_off = 0, free_ids = 0,
           owners = 0, total = 0;
};

// What the page calls share. Pointers of `in` and `out` lists; in place when
// lens_out == lens (and then table_out == table).
struct PageArgs {
    int32_t n_pages, page_size, page_shift, batch, heads, max_pages;
    int64_t row_bytes;    // of a row's elements or codes
    int32_t scale_bytes;  // of a row's scales (4-bit pages)
    int64_t page_bytes;
    uint8_t *k, *v;
    const int32_t *table, *lens, *refs;
    int32_t *table_out, *lens_out, *refs_out;
    // update
    const int32_t *parent, *n_new;
    // compact (kept != NULL)
    const int32_t *idx, *kept, *seq_lens;
    const uint8_t *K, *V;
    int32_t idx_stride, t_max;
    int32_t quantize;  // K and V are bf16, the pages E4M3 (1) or 4-bit (2); 0: rows are copied
    Rounding k_round, v_round;
    // workspace
    uint32_t *status, *verdict;  // verdict: status bits (0: the call goes through), pages taken
    int2 *row_src;
    long long *row_need;
    uint32_t *row_bits;
    int32_t *page_free, *list_off, *free_ids;
    int2 *owners;  // compact: list and place in it of each page taken
    int32_t row_chunks, page_chunks;
    int32_t run;  // lists of a warp of the plan: those of a row, or in a compaction any
};

cudaError_t launch_page_call(const PageArgs &a, cudaStream_t st);

struct RopeArgs {
    const uint8_t *Q, *K, *V;
    int64_t q_stride, k_stride, v_stride;  // elements
    uint8_t *Q_out;
    const int32_t *positions, *q_start, *table, *lens;
    const float *inv_freq;
    uint8_t *k, *v;
    int32_t n_tokens, q_heads, batch, heads, max_pages, n_pages, page_size, page_shift, head_dim, es, rot_dim, layout;
    float factor, k_inv, v_inv;  // (E4M3 pools: the scales' reciprocals)
    float k_inv6, v_inv6;        // (4-bit pools: see Rounding)
    int32_t n_axes;              // positions [n_axes, n_tokens]; 0: one axis
    const int32_t *axes;         // of each pair
    uint32_t *status;
};
cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t st);
cudaError_t launch_rope_axes(const RopeArgs &a, cudaStream_t st);  // several axes, or 4-bit pages

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiplication (Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication", PLDI 1994,
// figure 4.1): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d is
// the high word of m n, plus n, shifted right by l.
struct FastDiv {
    uint32_t d = 1, m = 1, l = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div)
    {
        while ((1ull << l) < d) ++l;
        m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> l); }
#endif
};

struct AttnArgs {
    const uint8_t *Q;
    uint8_t *O;
    float *lse;
    int64_t q_stride, o_stride;  // elements
    const int32_t *q_start, *table, *lens;
    const uint8_t *k, *v;
    int32_t n_tokens, q_heads, group, batch, heads, max_pages, n_pages, page_size, page_shift, head_dim, es;
    int32_t max_q, max_len, window, sinks;
    float scale_log2;  // scale * k_scale * log2(e)
    float v_scale;
    int32_t chunked;   // the form for many rows (mkv_attention_chunk.cu)
    int32_t tiles;     // tiles of tile_rows rows per list (of max_q * group rows)
    FastDiv by_tiles, by_heads, by_group;
    int32_t ctas;      // CTAs that the line of key blocks is cut over
    float *part_o;     // [2 ctas, rows of a tile, head_dim]: parts of cut tiles, before the division
    float2 *part_ml;   // [2 ctas, rows of a tile]: running maximum (log2 units) and sum; the CTAs' LineInfo follows
    uint32_t *status;
    uint32_t *counts;  // a byte per CTA in the workspace's head, zero between calls: parts of the tile that it opened
    int32_t tile_rows;
};
// The launch of a shape, and the workspace bytes behind the status word.
struct AttnPlan {
    int32_t chunked = 0, tile_rows = 0, tiles = 0, ctas = 0;
    int64_t part_rows = 0;  // rows of part_o
    size_t bytes = 0;
};
AttnPlan attention_plan(int32_t batch, int32_t heads, int32_t group, int32_t n_tokens, int32_t max_q, int32_t max_len,
                        int32_t head_dim, int32_t es, int ctas);
int chunk_tile_rows(int head_dim);
cudaError_t launch_attend_chunk(const AttnArgs &a, cudaStream_t st);
int e2m1_tile_rows(int64_t rows);
cudaError_t launch_attend_e2m1(const AttnArgs &a, cudaStream_t st);  // few rows, 4-bit pages
cudaError_t launch_paged_attention(const AttnArgs &a, cudaStream_t st);

}  // namespace mkv
