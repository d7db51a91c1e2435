// sm_103a attention of chunks of new tokens over a paged cache, on the
// 5th-generation tensor cores (the form of mkv_paged_attention for lists with
// many query rows; see mkv_attention.cu for the definition and the form for
// few).
//
// A tile is NSUB x 128 packed rows (new token, query head of the KV head's
// group) of one list; a block is 128 keys (64 at 256 dims). Per block and sub-tile
//     S = Q K^T          tcgen05.mma, M = 128, N = 128, fp32 in TMEM
//     P = 2^(S c - m)    one thread per row, P rounded to 16 bits over S in TMEM
//     O += P V           tcgen05.mma with P as the A operand from TMEM
// with the row's maximum m allowed to lag: O is multiplied by 2^(m_old - m_new)
// only when the maximum has grown by more than 2^8, so weights stay below 256
// (next to E4M3 values 2^15, see kBase) and the rescaling, which has to wait for
// the tensor core, is rare.
//
// Roles (one CTA per SM): warps 0 and 3 bring the pages of K and of V blocks
// into a ring of shared-memory slots (TMA, 128-byte swizzle, one box of 64 dims
// per page, page entries read a block ahead); warps 1 and 2 issue the MMAs of
// sub-tile 0 and 1, so that the tensor core works on one while the other waits
// for its softmax or its operands; warps 4-7 and 8-11 are the softmax of
// sub-tile 0 and 1 (they also load its queries and write its output). E4M3
// pages land as codes in a ring of their own; warps 12-15 expand them into the
// slots as fp16, which holds every code exactly, and the queries are fp16 too,
// each row scaled by a power of two (mkv_attention.cuh). 4-bit pages are copied as
// they lie, codes and scales, and expanded to fp16 products of both.
//
// The line of blocks is cut over 152 CTAs (mkv_attention.cuh);
// k_chunk_combine joins the parts of cut tiles.
//
// Measured: 2048 new tokens of 32 query heads (8 KV heads of 128 dims) over 32768
// bf16 tokens 0.72 ms, 1.48 PFLOP/s, 0.77 of the measured cuBLAS rate; the tensor
// pipe is busy 67% of the time. Without the softmax (weights left as they are)
// the same loop takes 0.63 ms, without copies too 0.57: what is left is the chain
// scores -> weights -> product of each sub-tile, of which two overlap. E4M3 at
// the same size 0.86 ms (0.99 with three slots and three blocks of codes instead
// of four and two); the conversions themselves cost nothing, the traffic of
// codes and their expansion through shared memory does. 4-bit pages 0.81 ms: 0.90
// with E4M3's way of expanding, 0.85 with places that are fixed per thread, and the
// rest by giving the softmax the registers that its loop spilled.
//
// Every wait is bounded (1 s); when one runs out the CTA reports
// MKV_DEV_TIMEOUT, its roles leave their loops, the copies and MMAs in flight
// are waited for (bounded) and the TMEM is freed.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "mkv_attention.cuh"
#include "mkv_device.cuh"
#include "mkv_e2m1.cuh"
#include "mkv_pages.h"

namespace mkv {
namespace {

using namespace dev;

constexpr int kSubRows = 128;                // rows per sub-tile: the MMA's M, the TMEM lanes
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kSlackKeys = 768, kUnevenKeys = 4096;  // see mkv_line.h
constexpr int kMinBlocks = 4;                // least blocks of a CTA's part: fewer make more parts to join, not less time

template <int D, int ES>
struct Chunk {
    static constexpr int NSUB = D == 256 ? 1 : 2;  // O of two sub-tiles fits the 512 TMEM columns up to D = 128
    static constexpr int ROWS = NSUB * kSubRows;
    // Keys per block: 128; 64 at 256 dims, where shared memory then holds five
    // blocks instead of two and the copies run ahead.
    static constexpr int KEYS = D == 256 ? 64 : 128;
    static constexpr int BOXES = D / 64;
    static constexpr int BOX = KEYS * 128;          // 64 dims of a block: rows of 128 bytes
    static constexpr int SLOT = BOXES * BOX;        // one block of K or of V as the MMA reads it
    static constexpr int CODES_BYTES = ES == 0 ? KEYS * D / 2 : KEYS * D;   // ... as E4M3 or 4-bit codes
    static constexpr int RAW = CODES_BYTES + (ES == 0 ? KEYS * D / 16 : 0);  // (and their scales)
    static constexpr int RAWS = ES == 2 ? 0 : D == 64 ? 3 : 2;
    static constexpr int SLOTS = ES == 2 ? (D == 64 ? 8 : D == 128 ? 4 : 5) : (D == 64 ? 9 : 4);
    // The next tile's queries go to the MMAs before this one's output is written
    // (384 lists of 64 keys, 256 rows: E4M3 at 128 dims 43.5 us, else 44.7; bf16 at 256
    // dims 63 / 66; 160 lists of 2048, 1024 rows, E4M3 at 64 dims 148 / 153). Of bf16 at 64
    // and 128 dims it takes registers from the loop: 8192 rows over 32768 keys 725 / 712.
    static constexpr bool EARLY = ES != 2 || D == 256;
    static constexpr int QBOX = kSubRows * 128;
    static constexpr int QBYTES = BOXES * QBOX;     // one sub-tile of queries
    static constexpr int SMEM = NSUB * QBYTES + SLOTS * SLOT + RAWS * RAW + 1024;
    static constexpr int SOFT = NSUB * 4;                     // softmax warps, from warp 4 on
    static constexpr int CODES = ES == 2 ? 0 : 4;             // warps that expand codes, after them
    static constexpr int THREADS = (4 + SOFT + CODES) * 32;   // 256, 384 or 512
    // Registers per thread of warps 0-3, the softmax warps and the expanding
    // ones: at most what the launch has (256 x 224, 384 x 168 or 512 x 128).
    // 512 threads, 4-bit pages (128 dims, 2048 tokens over 32768): 64 / 192 / 64 819 us, the 80 / 176 / 80 of E4M3 pages
    // 856. (E4M3's loop spills with its 176 too, 20 bytes at 128 dims and 16 at 64; it keeps them, no other split of it
    // has been timed.) 384 threads with codes (256 dims): 88 / 208 / 80; 240 for the softmax is no faster (2048 tokens
    // over 16384, 4-bit 1375 us, E4M3 1419 with both), and the 4-bit loop spills a little more.
    static constexpr int REGS_FEED = THREADS == 256 ? 168 : THREADS == 384 ? 88 : ES == 0 ? 64 : 80;
    static constexpr int REGS_SOFT = THREADS == 256 ? 240 : THREADS == 384 ? 208 : ES == 0 ? 192 : 176;
    static constexpr int REGS_CODES = THREADS == 512 && ES == 0 ? 64 : 80;
    static constexpr int REGS_LAUNCH = THREADS == 256 ? 224 : THREADS == 384 ? 168 : 128;
    static_assert(4 * REGS_FEED + SOFT * REGS_SOFT + CODES * REGS_CODES <= THREADS / 32 * REGS_LAUNCH, "register split");
    static constexpr int TMEM = 512;
    static constexpr int O_COL = NSUB * KEYS;      // S of the sub-tiles, then O
};

__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}

// Bounded wait for a phase; false on a timeout (reported, the CTA's abort flag
// raised) or, when abortable, as soon as another role raised the flag.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, uint32_t *status, volatile uint32_t *abort_flag,
                                         bool abortable = true)
{
    const uint32_t a = saddr(b);
    uint64_t t0 = 0;
    for (uint32_t spin = 0;; ++spin) {
        uint32_t done;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(done)
                     : "r"(a), "r"(parity)
                     : "memory");
        if (done) return true;
        if ((spin & 63u) == 63u) {
            if (abortable && *abort_flag) return false;
            if (t0 == 0) t0 = global_ns();
            else if (global_ns() - t0 > kWaitNs) {
                atomicOr(status, MKV_DEV_TIMEOUT);
                *abort_flag = 1u;
                return false;
            }
        }
    }
}

// The same for a whole warp: all lanes get one answer.
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, uint32_t *status, volatile uint32_t *abort_flag)
{
    return __all_sync(kFull, bar_wait(b, parity, status, abort_flag));
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *b)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(saddr(b))
        : "memory");
}

// `bytes` consecutive ones (a multiple of 16, as are both addresses).
__device__ __forceinline__ void bulk_load(uint32_t dst, const uint8_t *src, uint32_t bytes, uint64_t *b)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(saddr(b))
                 : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle (layout type 2, version
// 1), 8-row groups 1024 bytes apart. Keys and queries are K-major (the
// contraction runs along the 128-byte rows; leading offset unused). Values
// are MN-major (the contraction runs over the rows): the leading offset is
// the distance of the 64-dim boxes.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
template <int BOX>
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(BOX >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16, fp32 accumulator, both operands bf16 or both fp16, M = 128, N = n;
// bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_16bit(bool bf16, int n, bool b_mn)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kSubRows >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *b)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(b))
                 : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// One lane of the converged warp. (Issued under this the MMAs go out back to
// back; under a test of the lane number they took 90 cycles each, more than
// the 64 that the tensor core needs for one.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v)
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// Two fp32 operations in one instruction: (a.x b.x + c.x, a.y b.y + c.y).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c; "
        "mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
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
// Not inlined: the kernel's loops are then compiled with fewer spills (2048
// tokens of 32 query heads over 32768 bf16 tokens 712 us, inlined 755; a call with nearly
// nothing to do takes 0.7 us more).
template <int KEYS, int THREADS>
__device__ __noinline__ void cut_for_warps(const AttnArgs &a, int tile_rows, LineRule rule, LineScratch &s, int *shift,
                                           Walk *walks)
{
    const Walk start = cut_line<KEYS, THREADS>(a, tile_rows, rule, s, shift);
    if ((threadIdx.x & 31) == 0) walks[threadIdx.x >> 5] = start;
}

template <int D, int ES>
__global__ void __launch_bounds__(Chunk<D, ES>::THREADS, 1)
k_attend_chunk(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ AttnArgs a, LineInfo *info)
{
    using C = Chunk<D, ES>;
    constexpr int NSUB = C::NSUB, SLOTS = C::SLOTS, RAWS = C::RAWS, kKeys = C::KEYS, kBoxBytes = C::BOX;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *q_smem = smem;                      // NSUB x [D / 64 boxes][128 rows x 128 B]
    uint8_t *ring = smem + NSUB * C::QBYTES;     // SLOTS blocks: K, V, K, V, ...
    uint8_t *raws = ring + SLOTS * C::SLOT;      // RAWS blocks of codes, in the same order
    __shared__ __align__(8) uint64_t full[SLOTS], empty[SLOTS], raw_full[RAWS + 1], raw_empty[RAWS + 1], s_full[2],
        p_ready[2], o_done[2], o_free[2], q_full[2], drain[2];
    __shared__ uint32_t tmem_base;
    __shared__ volatile uint32_t abort_flag;
    __shared__ Walk s_walk[C::THREADS / 32];
    __shared__ LineScratch s_line;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();

    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            bar_init(&full[s], ES == 2 ? 1 : 4);
            bar_init(&empty[s], NSUB);
        }
        for (int s = 0; s < RAWS; ++s) {
            bar_init(&raw_full[s], 1);
            bar_init(&raw_empty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(&s_full[s], 1);
            bar_init(&p_ready[s], 4);
            bar_init(&o_done[s], 1);
            bar_init(&o_free[s], 4);
            bar_init(&q_full[s], 4);
        }
        bar_init(&drain[0], 1);
        bar_init(&drain[1], 1);
        abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_base)),
                     "n"(C::TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // (the queries' place lends its memory: nothing is there before the barrier below)
    cut_for_warps<kKeys, C::THREADS>(a, C::ROWS, {kMinBlocks, kSlackKeys / kKeys, kUnevenKeys / kKeys}, s_line,
                                     reinterpret_cast<int *>(q_smem), s_walk);
    // A warp's walk lies in shared memory: registers are for the loops.
    const Walk &w = s_walk[warp];
    auto next_segment = [&]() -> bool {
        __syncwarp();
        Walk x = w;
        __syncwarp();
        const bool more = x.next<kKeys>(a, C::ROWS);
        if (lane == 0) s_walk[warp] = x;
        __syncwarp();
        return more;
    };
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_FEED));
        if (warp == 0 || warp == 3) {
            // -------------------------- pages of K (warp 0) and of V (warp 3) --
            const int kv = warp == 0 ? 0 : 1;
            const CUtensorMap *map = kv ? &map_v : &map_k;
            // boxes of a page's rows, or of a block's if that is less: one lane each
            const int box_shift = min(a.page_shift, kKeys == 64 ? 6 : 7), per_block = kKeys >> box_shift;
            // the ring that the copies land in: the MMAs' slots, or the codes
            constexpr int N = ES == 2 ? SLOTS : RAWS;
            uint64_t *landed = ES == 2 ? full : raw_full, *taken = ES == 2 ? empty : raw_empty;
            LineInfo ci = {-1, 0};
            uint32_t seq = kv;  // K blocks take the even places of the ring's order, V blocks the odd ones
            bool ok = true;
            while (next_segment()) {
                note_segment(w, ci);
                const int32_t *table = a.table + ((int64_t)w.t.b * a.heads + w.t.j) * a.max_pages;
                const int from = w.from(), to = w.to(), end = w.t.end;
                const int sink_blocks = w.t.sink_blocks, past_sinks = w.t.win_block - w.t.sink_blocks;
                // the pool row of this lane's box of a block; past every row (zero fill) for a bad page, -1: none
                auto lookup = [&](int blk) -> int {
                    const int key = (blk + (blk < sink_blocks ? 0 : past_sinks)) * kKeys + (lane << box_shift);
                    if (blk >= to || lane >= per_block || key >= end) return -1;
                    const int id = table[key >> a.page_shift];
                    if ((uint32_t)id >= (uint32_t)a.n_pages) {
                        atomicOr(a.status, MKV_DEV_BAD_PAGE);
                        return a.n_pages << a.page_shift;
                    }
                    return (id << a.page_shift) + (key & (a.page_size - 1));
                };
                int row = lookup(from);
                for (int blk = from; ok && blk < to; ++blk, seq += 2) {
                    const int next = lookup(blk + 1), s = (int)(seq % N);
                    bool copied = row >= 0;
                    // (4-bit pages are copied as they lie, with no tensor map that would fill in for a bad one)
                    if constexpr (ES == 0) copied = copied && row < a.n_pages << a.page_shift;
                    const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(kFull, copied)) * (ES ? D * ES : D * 9 / 16)) << box_shift;
                    ok = seq < N || warp_wait(&taken[s], ((seq / N) - 1) & 1u, a.status, &abort_flag);
                    if (!ok) break;
                    if constexpr (ES == 0) {
                        if (row >= 0 && !copied) {  // a bad page's elements are zeros: all its scales
                            const uint32_t dst = saddr(raws + s * C::RAW + C::CODES_BYTES) + ((uint32_t)lane * (D / 16) << box_shift);
                            for (int o = 0; o < D / 16 << box_shift; o += 16) sts16(dst + o, make_uint4(0u, 0u, 0u, 0u));
                            fence_async();
                        }
                        __syncwarp();
                    }
                    if (lane == 0) bar_expect(&landed[s], bytes);
                    __syncwarp();
                    if (copied) {
                        if constexpr (ES == 0) {
                            const int in_page = row & (a.page_size - 1);
                            const uint8_t *page = (kv ? a.v : a.k) + (int64_t)(row >> a.page_shift) * (D * 9 / 16 << a.page_shift);
                            const uint32_t dst = saddr(raws + s * C::RAW);
                            bulk_load(dst + ((uint32_t)lane * (D / 2) << box_shift), page + in_page * (D / 2),
                                      (uint32_t)(D / 2) << box_shift, &landed[s]);
                            bulk_load(dst + C::CODES_BYTES + ((uint32_t)lane * (D / 16) << box_shift),
                                      page + (D / 2 << a.page_shift) + in_page * (D / 16), (uint32_t)(D / 16) << box_shift,
                                      &landed[s]);
                        } else if constexpr (ES == 2) {
                            const uint32_t dst = saddr(ring + s * C::SLOT) + ((uint32_t)lane * 128u << box_shift);
#pragma unroll
                            for (int x = 0; x < C::BOXES; ++x)
                                tma_load_2d(dst + x * kBoxBytes, map, x * 64, row, &landed[s]);
                        } else {
                            tma_load_2d(saddr(raws + s * C::RAW) + ((uint32_t)lane * D << box_shift), map, 0, row, &landed[s]);
                        }
                    }
                    row = next;
                }
                if (!ok) break;
            }
            if (warp == 0 && lane == 0) info[blockIdx.x] = ci;
            // every copy issued lands before the CTA may exit (the last uses of the ring's places)
            for (int x = (int)seq - 2; x >= 0 && x >= (int)seq - kv - N; x -= 2)
                bar_wait(&landed[x % N], (uint32_t)(x / N) & 1u, a.status, &abort_flag, false);
        } else if (warp <= NSUB) {
            // ----------------------------- MMAs of sub-tile 0 (warp 1), 1 (warp 2) --
            constexpr uint32_t id_qk = idesc_16bit(ES == 2, kKeys, false), id_pv = idesc_16bit(ES == 2, D, true);
            const int t = warp - 1;
            const uint32_t s_col = tmem + t * kKeys, o_col = tmem + C::O_COL + t * D;
            uint32_t seq = 0, n_p = 0, n_seg = 0;  // slots, blocks and segments so far
            bool ok = true;
            auto qk = [&](int slot) {
                const uint64_t qd = desc_k(saddr(q_smem + t * C::QBYTES)), kd = desc_k(saddr(ring + slot * C::SLOT));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t in_row = (k & 3) * 32;
                    mma_ss(s_col, qd + (uint64_t)(((k >> 2) * C::QBOX + in_row) >> 4),
                           kd + (uint64_t)(((k >> 2) * kBoxBytes + in_row) >> 4), id_qk, k > 0);
                }
                mma_commit(&s_full[t]);
            };
            while (ok && next_segment()) {
                const int nb = w.to() - w.from();
                if (nb == 0) continue;
                if (t * kSubRows >= w.t.rows) {
                    // no rows for this warp: it keeps step (a slot is free when both warps have let it go)
                    for (int x = 0; ok && x < 2 * nb; ++x, ++seq) {
                        ok = warp_wait(&full[seq % SLOTS], (seq / SLOTS) & 1u, a.status, &abort_flag);
                        if (ok && lane == 0) bar_arrive(&empty[seq % SLOTS]);
                    }
                    continue;
                }
                const int first = w.from();
                const int ks = (int)(seq % SLOTS);
                ok = warp_wait(&full[ks], (seq / SLOTS) & 1u, a.status, &abort_flag) &&
                     warp_wait(&q_full[t], n_seg & 1u, a.status, &abort_flag);
                fence_after();
                if (ok && elect_one()) {
                    qk(ks);
                    mma_commit(&empty[ks]);
                }
                __syncwarp();
                for (int blk = 0; ok && blk < nb; ++blk, seq += 2) {
                    // values of this block, keys of the next
                    const int vs = (int)((seq + 1) % SLOTS), kn = (int)((seq + 2) % SLOTS);
                    const bool more = blk + 1 < nb;
                    ok = warp_wait(&full[vs], ((seq + 1) / SLOTS) & 1u, a.status, &abort_flag);
                    if (more) ok = ok && warp_wait(&full[kn], ((seq + 2) / SLOTS) & 1u, a.status, &abort_flag);
                    if (!ok) break;
                    // values behind the list's end may be anything, also NaN: zero them, their weights are zero too
                    // (both warps write the same zeros, each before its own MMAs; codes are zeroed when converted)
                    const int live = w.t.end - block_key<kKeys>(w.t, first + blk);
                    if (ES == 2 && live < kKeys) {
                        const uint32_t base = saddr(ring + vs * C::SLOT);
                        for (int o = max(live, 0) * 8 + lane; o < kKeys * 8; o += 32)
#pragma unroll
                            for (int x = 0; x < C::BOXES; ++x)
                                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + x * kBoxBytes + o * 16),
                                             "r"(0u)
                                             : "memory");
                        fence_async();
                        __syncwarp();
                    }
                    if (blk == 0) ok = n_seg == 0 || warp_wait(&o_free[t], (n_seg - 1) & 1u, a.status, &abort_flag);
                    ok = ok && warp_wait(&p_ready[t], n_p & 1u, a.status, &abort_flag);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
                        const uint64_t vd = desc_mn<kBoxBytes>(saddr(ring + vs * C::SLOT));
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            mma_ts(o_col, s_col + k * 8, vd + (uint64_t)(k * 2048 >> 4), id_pv, blk > 0 || k > 0);
                        // one thread's MMAs run in order: the next scores are complete only after this block's O
                        if (more) qk(kn);
                        else mma_commit(&o_done[t]);
                        mma_commit(&empty[vs]);
                        if (more) mma_commit(&empty[kn]);
                    }
                    __syncwarp();
                    ++n_p;
                }
                ++n_seg;
            }
            // the tensor core is done with shared memory and TMEM
            if (n_seg > 0 || !ok) {
                if (elect_one()) mma_commit(&drain[t]);
                bar_wait(&drain[t], 0, a.status, &abort_flag, false);
            }
        }
    } else if (warp >= 4 + C::SOFT) {
        // ------------------------------------------------- codes to fp16 (exact) --
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CODES));
        if constexpr (ES != 2) {
            const int quarter = warp - 4 - C::SOFT;
            uint32_t seq = 0;
            bool ok = true;
            while (ok && next_segment()) {
                for (int blk = w.from(); ok && blk < w.to(); ++blk) {
                    // codes behind the list's end may be anything: zeros (see the MMAs)
                    const int live = w.t.end - block_key<kKeys>(w.t, blk);
                    for (int kv = 0; ok && kv < 2; ++kv, ++seq) {
                        const int s = (int)(seq % SLOTS), q = (int)(seq % RAWS);
                        ok = warp_wait(&raw_full[q], (seq / RAWS) & 1u, a.status, &abort_flag) &&
                             (seq < SLOTS || warp_wait(&empty[s], ((seq / SLOTS) - 1) & 1u, a.status, &abort_flag));
                        if (!ok) break;
                        const uint32_t from = saddr(raws + q * C::RAW), to = saddr(ring + s * C::SLOT);
                        constexpr int CPR = D / 16;  // groups of 16 codes per row
                        if constexpr (ES == 0) {
                            // A thread's groups are the same one of rows STEP apart, so its places are one of each kind and
                            // fixed distances. (Eight lanes store into two rows of one box, whose swizzle gives them all chunks.)
                            constexpr int STEP = 128 / CPR, ROUNDS = kKeys / STEP;
                            const int o = quarter * 32 + lane, c = (o & 3) | (o >> 3 & (CPR / 4 - 1)) << 2;
                            const int key = (o >> 2 & 1) | o / (2 * CPR) << 1;
                            const uint32_t codes = from + (key * CPR + c) * 8, scales = from + C::CODES_BYTES + key * CPR + c;
                            const uint32_t row = to + (c >> 2) * kBoxBytes + key * 128, x = (uint32_t)(c & 3) * 2;
                            const uint32_t lo = row + ((x ^ (key & 7)) << 4), hi = row + (((x + 1) ^ (key & 7)) << 4);
                            static_assert(STEP % 8 == 0, "rows a step apart have one swizzle");
#pragma unroll 4
                            for (int i = 0; i < ROUNDS; ++i) {
                                const uint2 v = lds8(codes + i * 1024);
                                uint32_t sc = lds1(scales + i * 128);
                                if (live < kKeys && key + STEP * i >= live) sc = 0u;
                                sc = e4m3x2_to_f16x2(sc | sc << 8);
                                uint32_t h[2][4];
                                e2m1x8_to_f16(v.x, h[0]);
                                e2m1x8_to_f16(v.y, h[1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    h[0][e] = mul_f16x2(h[0][e], sc);
                                    h[1][e] = mul_f16x2(h[1][e], sc);
                                }
                                sts16(lo + i * STEP * 128, make_uint4(h[0][0], h[0][1], h[0][2], h[0][3]));
                                sts16(hi + i * STEP * 128, make_uint4(h[1][0], h[1][1], h[1][2], h[1][3]));
                            }
                        } else {
#pragma unroll 4
                            for (int o = quarter * 32 + lane; o < kKeys * CPR; o += 128) {
                                const int key = o / CPR, c = o % CPR;
                                uint4 v = lds16(from + o * 16);
                                if (key >= live) v = make_uint4(0u, 0u, 0u, 0u);
                                const uint32_t row = to + (c >> 2) * kBoxBytes + key * 128, x = (uint32_t)(c & 3) * 2;
                                sts16(row + ((x ^ (key & 7)) << 4),
                                      make_uint4(e4m3x2_to_f16x2(v.x & 0xFFFFu), e4m3x2_to_f16x2(v.x >> 16),
                                                 e4m3x2_to_f16x2(v.y & 0xFFFFu), e4m3x2_to_f16x2(v.y >> 16)));
                                sts16(row + (((x + 1) ^ (key & 7)) << 4),
                                      make_uint4(e4m3x2_to_f16x2(v.z & 0xFFFFu), e4m3x2_to_f16x2(v.z >> 16),
                                                 e4m3x2_to_f16x2(v.w & 0xFFFFu), e4m3x2_to_f16x2(v.w >> 16)));
                            }
                        }
                        fence_async();
                        __syncwarp();
                        if (lane == 0) {
                            bar_arrive(&raw_empty[q]);
                            bar_arrive(&full[s]);
                        }
                    }
                }
            }
        }
    } else {
        // ------------------------------------------ softmax, queries, output --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFT));
        const int t = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;  // sub-tile, row of it
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + t * kKeys, o_addr = tmem + lanes + C::O_COL + t * D;
        // scores c x_s with c > 0: the queries take the sign, and a factor of zero
        // becomes the smallest normal number, which makes every score as good as zero
        // (zero times a masked score's -inf would be NaN)
        const float c_all = fmaxf(fabsf(a.scale_log2), FLT_MIN);
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
        uint32_t n_s = 0, n_o = 0;  // blocks, segments with blocks so far
        bool ok = true;
        // The next segment with rows for this sub-tile, its queries on their way
        // to the MMAs. (Every wait for the last block of the segment before has
        // ended: Q is free.)
        float c_row = c_all;
        auto begin = [&]() -> bool {
            do {
                if (!next_segment()) return false;
            } while (t * kSubRows >= w.t.rows);
            const bool real = t * kSubRows + row < w.t.rows;
            if (w.to() > w.from()) {
                const int R = w.t.row0 + t * kSubRows + row, i = a.by_group(R), head = w.t.j * a.group + R - i * a.group;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.Q + 2 * (((int64_t)a.q_start[w.t.b] + i) * a.q_stride + (int64_t)head * D));
                const uint32_t dst = saddr(q_smem + t * C::QBYTES) + row * 128;
                float down = 1.f;
                if constexpr (ES != 2) {  // fp16 next to codes, the row scaled by a power of two
                    float largest = 0.f;
                    if (real)
#pragma unroll 8
                        for (int x = 0; x < D / 8; ++x) {
                            float f[8];
                            bf16x8_to_f32(src[x], f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) largest = fmaxf(largest, fabsf(f[e]));
                        }
                    const int E = row_exponent(largest);
                    down = down_by(E);
                    c_row = fmaxf(c_all * up_by(E), FLT_MIN);
                }
#pragma unroll 8
                for (int x = 0; x < D / 8; ++x) {
                    uint4 v = real ? src[x] : make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (ES != 2) {
                        float f[8];
                        bf16x8_to_f32(v, f);
                        v = make_uint4(pack_f16(f[0] * down, f[1] * down), pack_f16(f[2] * down, f[3] * down),
                                       pack_f16(f[4] * down, f[5] * down), pack_f16(f[6] * down, f[7] * down));
                    }
                    v.x ^= flip;
                    v.y ^= flip;
                    v.z ^= flip;
                    v.w ^= flip;
                    sts16(dst + (x >> 3) * C::QBOX + (((x & 7) ^ (row & 7)) << 4), v);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(&q_full[t]);
            }
            return true;
        };
        bool have = C::EARLY && begin();
        while (C::EARLY ? have : begin()) {
            const bool real = t * kSubRows + row < w.t.rows;
            const int first = w.from(), nb = w.to() - first;
            const float c = ES != 2 ? c_row : c_all;
            // the row's own key (of rows that are not there: the first row's)
            const int p = w.t.L - w.t.n + a.by_group(w.t.row0 + t * kSubRows + (real ? row : 0));
            const int sink_blocks = w.t.sink_blocks, past_sinks = w.t.win_block - w.t.sink_blocks;
            // the first and last place that is visible to every row: blocks inside need no mask
            const int r_last = min(w.t.rows, (t + 1) * kSubRows) - 1;
            const int whole_to = w.t.L - w.t.n + a.by_group(w.t.row0 + t * kSubRows);
            const int whole_from = a.window > 0 ? w.t.L - w.t.n + a.by_group(w.t.row0 + r_last) - a.window : -1;
            float m = -CUDART_INF_F, l = 0.f;
            for (int blk = 0; blk < nb; ++blk, ++n_s) {
                ok = warp_wait(&s_full[t], n_s & 1u, a.status, &abort_flag);
                if (!ok) break;
                fence_after();
                float s[kKeys];
#pragma unroll
                for (int x = 0; x < kKeys; x += 32) tmem_ld32(s_addr + x, s + x);
                wait_ld();
                const int k0 = (first + blk + (first + blk < sink_blocks ? 0 : past_sinks)) * kKeys, k1 = k0 + kKeys - 1;
                if (!(k1 <= whole_to && (k0 > whole_from || k1 < a.sinks))) {
                    // bit x: key k0 + x is visible -- up to the row's own, and in its window or the first tokens
                    const int seen = p - k0, from = a.window > 0 ? seen - a.window : -1, sinks = a.sinks - k0;
#pragma unroll
                    for (int x = 0; x < kKeys; x += 32) {
                        const uint32_t vis = low_bits(seen + 1 - x) & (~low_bits(from + 1 - x) | low_bits(sinks - x));
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[x + e] = vis >> e & 1u ? s[x + e] : -CUDART_INF_F;
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int x = 4; x < kKeys; ++x) mx[x & 3] = fmaxf(mx[x & 3], s[x]);
                const float best = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                uint32_t pk[16];
                const bool grow = best - m > kLag<ES>;
                if (blk == 0) {
                    m = best - kBase<ES>;
                } else if (__any_sync(kFull, grow)) {
                    const float to = best - kBase<ES>;
                    const float f = !grow ? 1.f : m == -CUDART_INF_F ? 0.f : exp2_approx(m - to);
                    if (grow) m = to;
                    l *= f;
                    // (O is complete up to the block before: its MMAs came before the ones of these scores)
#pragma unroll
                    for (int x = 0; x < D; x += 16) {
                        tmem_ld16(o_addr + x, pk);
                        wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) pk[e] = __float_as_uint(__uint_as_float(pk[e]) * f);
                        tmem_st16(o_addr + x, pk);
                    }
                }
                // the weights above the reference point m
                const float base = m == -CUDART_INF_F ? 0.f : m;
                const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int x = 0; x < kKeys; x += 32) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 v = fma2(make_float2(s[x + e], s[x + e + 1]), c2, b2);
                        v.x = exp2_approx(v.x);
                        v.y = exp2_approx(v.y);
                        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], v);
                        pk[e >> 1] = pack_weights<ES>(v.x, v.y);
                    }
                    tmem_st16(s_addr + (x >> 1), pk);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&p_ready[t]);
            }
            if (!ok) break;
            if (nb > 0) {
                ok = warp_wait(&o_done[t], n_o++ & 1u, a.status, &abort_flag);
                if (!ok) break;
                fence_after();
            }
            const int R = w.t.row0 + t * kSubRows + row, i = a.by_group(R), head = w.t.j * a.group + R - i * a.group;
            const int64_t token = (int64_t)a.q_start[w.t.b] + i;
            const bool whole = w.whole();
            const int64_t part = part_row(w, C::ROWS) + t * kSubRows + row;
            const float inv = inverse_sum(l, a.v_scale);
            uint4 *dst = reinterpret_cast<uint4 *>(a.O + 2 * (token * a.o_stride + (int64_t)head * D));
            float4 *dst_part = reinterpret_cast<float4 *>(a.part_o + part * D);
            if (real && whole && a.lse) a.lse[token * a.q_heads + head] = log_sum(m, l);
            if (real && !whole) a.part_ml[part] = make_float2(m, l);
            const bool write = real, seen = nb > 0;
            if (C::EARLY) have = begin();
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float o[32];
                if (seen) {
                    tmem_ld32(o_addr + x, o);
                    wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (write && whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        dst[(x + e) >> 3] =
                            make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                       pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
                } else if (write) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) dst_part[(x + e) >> 2] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                __syncwarp();
            }
            if (seen) {
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&o_free[t]);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::TMEM) : "memory");
    }
}

// Joins the parts of the tile that CTA blockIdx.y opened, if it did: a warp per
// J rows, eight of their parts in flight. Four rows; one where few tiles are
// cut into many parts each, whose joining is a chain of round trips (two lists
// of 32768 keys, 256 rows: 35 us, with four rows 55), at the price of four times
// the blocks, of which most find nothing to join (2.5 us).
template <int D, int ES, int J>
__global__ void __launch_bounds__(256)
k_chunk_combine(const AttnArgs a, const LineInfo *__restrict__ info)
{
    using C = Chunk<D, ES>;
    pdl_wait();
    const int c0 = (int)blockIdx.y;
    int c1;
    const int tile = opened_tile(info, c0, (int)gridDim.y, c1);
    if (tile < 0) return;
    const Tile t = make_tile<C::KEYS>(a, tile, C::ROWS, false);
    const int row0 = ((int)blockIdx.x * 8 + (threadIdx.x >> 5)) * J;
    if (row0 < t.rows) join_rows<D, C::ROWS, J, 8 / J>(a, t, c0, c1, row0);
}

// --------------------------------------------------------------- host side --

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// The pool as rows of head_dim elements; boxes of one page (of a block's keys
// if that is less) x 64 bf16 dims (swizzled) or all the codes of a row.
bool make_map(CUtensorMap *map, const void *base, const AttnArgs &a, int32_t keys)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const bool bf16 = a.es == 2;
    const cuuint64_t dims[2] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_pages * a.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)a.head_dim * a.es};
    const cuuint32_t box[2] = {bf16 ? 64u : (cuuint32_t)a.head_dim, (cuuint32_t)std::min(a.page_size, keys)};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int ES>
cudaError_t launch_one(const AttnArgs &a, cudaStream_t st)
{
    using C = Chunk<D, ES>;
    CUtensorMap mk = {}, mv = {};  // (4-bit pages are copied without)
    if (ES != 0 && (!make_map(&mk, a.k, a, C::KEYS) || !make_map(&mv, a.v, a, C::KEYS))) return cudaErrorUnknown;
    cudaError_t e = cudaFuncSetAttribute(k_attend_chunk<D, ES>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    LineInfo *info = reinterpret_cast<LineInfo *>(a.part_ml + (int64_t)a.ctas * 2 * C::ROWS);
    k_attend_chunk<D, ES><<<a.ctas, C::THREADS, C::SMEM, st>>>(mk, mv, a, info);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    // tiles of eight parts and more
    const bool few = (int64_t)a.batch * a.heads * a.tiles * 8 <= a.ctas && a.max_len >= 8 * kMinBlocks * C::KEYS;
    cfg.gridDim = dim3((unsigned)(C::ROWS / 8 / (few ? 1 : 4)), (unsigned)a.ctas);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, k_chunk_combine<D, ES, 1>, a, (const LineInfo *)info)
               : cudaLaunchKernelEx(&cfg, k_chunk_combine<D, ES, 4>, a, (const LineInfo *)info);
}

}  // namespace

int chunk_tile_rows(int head_dim) { return head_dim == 256 ? kSubRows : 2 * kSubRows; }

cudaError_t launch_attend_chunk(const AttnArgs &a, cudaStream_t st)
{
    const int es = a.es;
    switch (a.head_dim) {
    case 64: return es == 2 ? launch_one<64, 2>(a, st) : es == 1 ? launch_one<64, 1>(a, st) : launch_one<64, 0>(a, st);
    case 128: return es == 2 ? launch_one<128, 2>(a, st) : es == 1 ? launch_one<128, 1>(a, st) : launch_one<128, 0>(a, st);
    case 256: return es == 2 ? launch_one<256, 2>(a, st) : es == 1 ? launch_one<256, 1>(a, st) : launch_one<256, 0>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace mkv
