// latent_prefill.cuh -- prompt attention over the paged latent pool with
// keys and values expanded (sm_100a tensor cores), in two launches:
//
//   latent_expand_kernel   K_h = C W_h^K, V_h = C W_h^V for every token of
//                          every context: a product of 128 tokens x 256
//                          columns (one head's key and value) over L, rounded
//                          once to 16 bits and kept in the workspace.  The
//                          tokens' rows stay in shared memory while the heads'
//                          weights stream past them.
//   latent_attend_kernel   causal attention of 256 queries of one head:
//                          S = Q K^T over 128 + 64 elements (the rotated part
//                          is shared by the heads), P V over 128.
//
// The expansion costs 2 L 256 operations a token and head, the attention 2 (192
// + 128) a query, visible token and head.  Measured at 4096 new tokens, 32
// heads, L 512: 39.4 us (0.87 PFLOP/s) and 165 us (1.04 PFLOP/s), of 1.64 that
// products alone reach here; 226 us a call, under the power limit.  The
// attention's products take 3480 of its 3700 cycles a step, as scores of 64 keys
// at a time read shared memory at its rate.
//
// Roundings: sums and softmax are fp32.  K goes to the pool's type, as the
// queries are of it and the operands of a product are of one type.  V and the
// weights P go to fp16, with a power of two a head and 32 tokens: bf16 for them
// added as much error each as the output's own rounding (0.0027 of the output
// in all, its own 0.0017; with fp16 0.0020, for 1 % of the time), and no finite
// value passes the type.  A token whose values are 2^14 below the largest of its
// 32 begins to lose bits.  So does a weight whose product with that largest value is
// 2^21 below the row's largest such product; below 2^32 it is gone from the output
// (not from the weights' sum).  Long prompts have such: a first token that takes
// most of the mass and has a small value.  With weights of at most 2^8, not 2^15,
// those bounds were 2^14 and 2^25: at 32768 tokens and 2^24 a weight 4 % of the output.
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "pa_common.cuh"
#include "tcgen05.cuh"

namespace pa {

constexpr int kNope = 128;                      // unrotated elements of a head's key
constexpr int kValue = 128;                     // elements of a head's value
constexpr int kRot = 64;                        // rotated elements, shared by the heads
constexpr int kKvTile = 128;                    // tokens of a tile of keys
constexpr int kQueryTile = 128;                 // queries of a tile; a CTA takes two

struct LatentPrefillArgs {
    void* out;
    const void* cache;
    const int32_t* block_tables;
    const int32_t* query_starts;
    const int32_t* context_lens;
    void* ws_k;                 // [S][H][rows][128]
    void* ws_v;                 // [S][H][rows][128]
    void* ws_rot;               // [S][rows][64]
    uint32_t* ws_mask;          // [S][rows / 32]: tokens that count
    float* ws_exp;              // [S][H][rows / 32]: V of 32 tokens is kept times 2^-this
    int32_t rows;               // max_context_len rounded up to whole tiles
    int32_t num_seqs, num_tokens, num_heads, heads_per_cta, block_size, max_blocks_per_seq;
    int64_t num_blocks;
    int32_t max_query_len, max_context_len;
    int32_t pairs, sorted;      // pairs of query tiles a sequence; whether the grid takes them by size
    float scale_log2;
    int32_t* d_status;
};

// A sequence's rows of the batch and its context.  `first` < 0: the starts are
// bad and its rows are left alone; `context` < 0: its rows are zeroed.
struct PromptSpan {
    int32_t first, count, context;
};

__device__ __forceinline__ PromptSpan prompt_span(const LatentPrefillArgs& a, int s)
{
    PromptSpan p;
    p.first = a.query_starts[s];
    const int32_t end = a.query_starts[s + 1];
    p.count = end - p.first;
    if (p.first < 0 || end < p.first || end > a.num_tokens || p.count > a.max_query_len) {
        p.first = -1;
        p.count = 0;
    }
    p.context = a.context_lens[s];
    if (p.context < p.count || p.context > a.max_context_len ||
        static_cast<int64_t>(p.context) > static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size)
        p.context = -1;
    return p;
}

// ---------------------------------------------------------------------------
// Expansion
// ---------------------------------------------------------------------------

template <int L>
struct ExpandShape {
    static constexpr int kChunks = L / 64;
    static constexpr int kRowsBytes = kChunks * kKvTile * 128;
    static constexpr int kStageBytes = 128 * 128;   // 64 columns of a head's key or value weights
    static constexpr int kStages = L == 512 ? 5 : 8;
    static constexpr int kOutBytes = 32 * 64;       // 32 tokens x 32 columns on their way out
    static constexpr int kSmem = 1024 + kRowsBytes + kStages * kStageBytes + 8 * kOutBytes + 512;
};

constexpr int kExpandThreads = 192;
constexpr int kLeastExp = -60;                  // values below 2^-60 are kept as if they were that large

// The larger magnitude, or NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// Grid (group of heads, tile of 128 tokens, sequence).  Warps: 0-3 store, 4
// copies, 5 products; two accumulators of 256 columns (key, value) alternate.
// Results leave through shared memory by TMA: stored from the registers, a
// row a thread, the 32 lines that each store touches took as long as the
// products.  Each warp has two boxes of its own for it, so it waits for no other
// and for the last box but one (4096 tokens, 32 heads, 512 elements: 66.6 k
// cycles, with one box for all warps 70.8 k).  Without the stores, the products
// or the weights' copies it is 58 to 62 k each, 34 k being the products' own:
// the start, with rows from memory, is about 15 k.
template <typename T, int L>
__global__ void __launch_bounds__(kExpandThreads, 1)
    latent_expand_kernel(const __grid_constant__ CUtensorMap tm_cache,
                         const __grid_constant__ CUtensorMap tm_weights,
                         const __grid_constant__ CUtensorMap tm_key,
                         const __grid_constant__ CUtensorMap tm_value,
                         const __grid_constant__ LatentPrefillArgs a)
{
    using S = ExpandShape<L>;
    constexpr int CH = S::kChunks;
    constexpr int ST = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* s_rows = smem;
    uint8_t* s_weights = smem + S::kRowsBytes;
    uint8_t* s_out = s_weights + ST * S::kStageBytes;
    uint64_t* r_full = reinterpret_cast<uint64_t*>(s_out + 8 * S::kOutBytes);   // [CH]
    uint64_t* w_full = r_full + CH;        // [ST]
    uint64_t* w_empty = w_full + ST;       // [ST]
    uint64_t* o_full = w_empty + ST;       // [2]
    uint64_t* o_empty = o_full + 2;        // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_empty + 2);

    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int s = blockIdx.z, t0 = blockIdx.y * kKvTile;
    const int h0 = blockIdx.x * a.heads_per_cta;
    const int heads = min(a.heads_per_cta, a.num_heads - h0);
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tm_cache);
        prefetch_tensor_map(&tm_weights);
        prefetch_tensor_map(&tm_key);
        prefetch_tensor_map(&tm_value);
    }
    grid_dependency_wait();
    const PromptSpan span = prompt_span(a, s);
    allow_dependents();
    if (span.count == 0 || t0 >= span.context) return;    // (a bad context is negative)

    if (threadIdx.x == 0) {
        for (int i = 0; i < CH; ++i) mbar_init(r_full + i, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(w_full + i, 1);
            mbar_init(w_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(o_full + i, 1);
            mbar_init(o_empty + i, 128);
        }
        fence_barrier_init();
    }
    if (warp == 5) tmem_alloc(tmem_slot, 512);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_slot, 0);
    const uint32_t leader = elect_lane() ? 1u : 0u;
    bool ok = true;

    if (warp == 4) {
        const int valid = min(kKvTile, span.context - t0);
        const int blocks = (valid + a.block_size - 1) / a.block_size;
        const int block_bytes = a.block_size * 128;
        int32_t page = 0;
        if (lane < blocks) {
            page = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + t0 / a.block_size + lane];
            // a block outside the pool reads as zeros, beyond the map's end
            if (page < 0 || page >= a.num_blocks) {
                page = static_cast<int32_t>(a.num_blocks);
                if (blockIdx.x == 0) status_or(a.d_status, PA_STATUS_BAD_BLOCK);
            }
        }
        int32_t it = 0;
        for (int h = 0; h < heads && ok; ++h) {
            for (int c = 0; c < 2 * CH && ok; ++c, ++it) {       // key and value of each chunk
                const int st = it % ST;
                if (it >= ST) ok = mbar_poll_warp(w_empty + st, (it / ST - 1) & 1);
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(w_full + st, S::kStageBytes);
                    tma_load_3d(s_weights + st * S::kStageBytes, &tm_weights, (c >> 1) * 64,
                                (h0 + h) * (kNope + kValue) + (c & 1) * kNope, 0, w_full + st);
                }
                if (h == 0 && (c & 1) == 0) {             // the rows, with the first head's weights
                    const int rc = c >> 1;
                    if (leader) mbar_arrive_expect_tx(r_full + rc, blocks * block_bytes);
                    for (int b = 0; b < blocks; ++b) {
                        const int32_t pg = __shfl_sync(kFullMask, page, b);
                        if (leader)
                            tma_load_3d(s_rows + rc * kKvTile * 128 + b * block_bytes, &tm_cache,
                                        rc * 64, 0, pg, r_full + rc);
                    }
                }
            }
        }
        if (!ok) {                                        // let the copies in flight land
            if (lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
            for (int k = max(0, it - ST); k < it; ++k) mbar_poll_warp(w_full + k % ST, (k / ST) & 1);
            for (int c = 0; c < min(CH, (it + 1) / 2); ++c) mbar_poll_warp(r_full + c, 0);
        }
    } else if (warp == 5) {
        const uint32_t idesc = mma_desc<T>(kKvTile, kNope);
        const uint32_t r_addr = smem_u32(s_rows), w_addr = smem_u32(s_weights);
        int32_t it = 0;
        for (int h = 0; h < heads && ok; ++h) {
            const int b = h & 1;
            if (h >= 2) ok = mbar_poll_warp(o_empty + b, (h / 2 - 1) & 1);
            tmem_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2 * CH && ok; ++c, ++it) {
                const int st = it % ST;
                ok = mbar_poll_warp(w_full + st, (it / ST) & 1) &&
                     (h > 0 || (c & 1) != 0 || mbar_poll_warp(r_full + (c >> 1), 0));
                if (!ok) break;
                const uint64_t da = desc_k_major(r_addr + (c >> 1) * kKvTile * 128);
                const uint64_t db = desc_k_major(w_addr + st * S::kStageBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss(tmem + b * 256 + (c & 1) * kNope, da + 2 * k, db + 2 * k, idesc,
                           (c >> 1) + k > 0, leader);
                if (leader) mma_commit(w_empty + st);
            }
            if (leader && ok) mma_commit(o_full + b);
        }
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    } else {
        // A thread has one token's row.
        const int r = threadIdx.x;
        const int32_t t = t0 + r;
        bool counts = t < span.context;
        int32_t page = 0;
        if (counts) {
            page = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + t / a.block_size];
            counts = page >= 0 && page < a.num_blocks;
        }
        const int64_t srow = static_cast<int64_t>(s) * a.rows + t;
        if (blockIdx.x == 0) {
            const uint32_t word = __ballot_sync(kFullMask, counts);
            if (lane == 0) a.ws_mask[srow >> 5] = word;
            // the rotated part, the same for every head
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.cache) +
                (static_cast<int64_t>(page) * a.block_size + t % a.block_size) * (L + kRot) + L);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.ws_rot) + srow * kRot);
            uint4 v[kRot / 8];
#pragma unroll
            for (int i = 0; i < kRot / 8; ++i) v[i] = counts ? ld_nc_v4(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kRot / 8; ++i) dst[i] = v[i];
        }
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        for (int h = 0; h < heads; ++h) {
            const int b = h & 1;
            // a wait that gave up is not repeated (PA_STATUS_TIMEOUT)
            if (ok) ok = mbar_poll_warp(o_full + b, (h / 2) & 1);
            tmem_fence_after();
            // V is kept in fp16 whatever the pool's type, the 32 tokens of a warp
            // times a power of two that brings their largest element below 1.
            float high = 0.f;
#pragma unroll 1
            for (int c = 4; c < 8; ++c) {
                uint32_t o[32];
                tmem_ld32(o, lanes + b * 256 + c * 32);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) high = max_abs_nan(high, __uint_as_float(o[i]));
            }
            // A token that does not count is a row of zeros: 0 times what its place
            // holds may not be 0.  So is a value that is not finite, for the queries
            // before its token, whose weight of it is 0; its key is NaN instead,
            // which those that see the token take over.
            const bool odd = !(high < INFINITY);
            const uint32_t most = __reduce_max_sync(kFullMask, counts && !odd ? __float_as_uint(high) : 0u);
            const int ex = min(max(static_cast<int>(most >> 23) - 126, kLeastExp), 126);
            const float unit = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            if (lane == 0)
                a.ws_exp[((static_cast<int64_t>(s) * a.num_heads + h0 + h) * a.rows + t) >> 5] =
                    static_cast<float>(ex);
#pragma unroll 1
            for (int turn = 0; turn < 8; ++turn) {        // 32 columns each: four of V, four of K
                const int c = turn ^ 4;
                uint32_t o[32];
                tmem_ld32(o, lanes + b * 256 + c * 32);
                tmem_wait_ld();
                if (turn == 7) {
                    tmem_fence_before();
                    mbar_arrive(o_empty + b);
                }
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float lo = __uint_as_float(o[2 * i]), hi = __uint_as_float(o[2 * i + 1]);
                    p[i] = c >= 4 ? Elem<__half>::from_float2(lo * unit, hi * unit)
                                  : Elem<T>::from_float2(lo, hi);
                }
                const bool keep = counts && !odd;
                const uint32_t other = counts && c < 4 ? 0x7fff7fffu : 0u;      // NaN in both types
                // the last box but one has been read out of shared memory
                uint8_t* box = s_out + (2 * warp + (turn & 1)) * S::kOutBytes;
                if (lane == 0) tma_store_wait_read<1>();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4*>(box + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) =
                        keep ? make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3])
                             : make_uint4(other, other, other, other);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(c < 4 ? &tm_key : &tm_value, (c & 3) * 32, t0 + warp * 32,
                                 s * a.num_heads + h0 + h, box);
                    tma_store_commit();
                }
            }
        }
        if (lane == 0) tma_store_wait_all();
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 5) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------

struct AttendShape {
    static constexpr int kChunks = (kNope + kRot) / 64;
    static constexpr int kQueryBytes = kChunks * kQueryTile * 128;
    static constexpr int kSlotBytes = kKvTile * 128;           // 64 columns of a tile of keys or values
    static constexpr int kKeySlots = kChunks, kValueSlots = kValue / 64;
    static constexpr int kSlots = 8;                           // of a ring of K and V by turns
    static constexpr int kSmem = 1024 + 2 * kQueryBytes + kSlots * kSlotBytes + 512;
    // TMEM: S of the two query tiles (P takes the first half of its S), O of both
    static constexpr int kOCol = 256;
};

constexpr int kAttendThreads = 352;
constexpr int kHalf = kKvTile / 2;              // keys whose scores and weights are under way at once
constexpr float kFaint = -40.0f;                // log2 of products of no account
constexpr float kHeadroom = 7.0f;               // weights are kept times 2^7, up to 2^15: what fp16 has room for
constexpr int kSortItems = 128;                 // pairs of query tiles at most that are sorted

// How long pair `item` of the query tiles takes, about: a step of both tiles
// costs about 41, of one alone 29.
__device__ __forceinline__ int32_t attend_size(const LatentPrefillArgs& a, int32_t item)
{
    const PromptSpan p = prompt_span(a, item / a.pairs);
    const int32_t row0 = (a.pairs - 1 - item % a.pairs) * 2 * kQueryTile;
    if (row0 >= p.count || p.context < 0) return 0;
    const int32_t before = p.context - p.count;
    const int32_t one = (before + min(p.count, row0 + kQueryTile) + kKvTile - 1) / kKvTile;
    if (row0 + kQueryTile >= p.count) return 29 * one;
    const int32_t all = (before + min(p.count, row0 + 2 * kQueryTile) + kKvTile - 1) / kKvTile;
    return 41 * one + 29 * (all - one);
}

// Grid (head, pair of query tiles of a sequence), the longest pairs first: by
// size over all sequences where they are few enough to rank (7 prompts of 1 to
// 700 tokens behind up to 2300, 20 heads: 97 us, in the sequences' order 107, both
// before tiles went in halves; now 87), else within a sequence.  Warps:
// 0-3 and 4-7 softmax of one query tile each, a thread a query; 8 copies; 9
// and 10 the products of one query tile each (with one warp for both the tensor
// cores stood still 480 cycles a step).
//
// A tile of keys goes through in two halves of 64: while the softmax has one,
// the scores of the other are made, so that it never waits for them.  Weights
// take the first half of their scores' place, and the scores of the next half
// but one follow them there.  (4096 tokens, 32 heads: 264 k cycles; 128 keys at
// once, whose scores have no second place in TMEM, 290 k, though products of 64
// columns take 50 cycles and of 128 only 66.)
//
// Tile i of the keys takes slots 5 i .. 5 i + 2 of the ring (modulo 8), its
// values the two after them.  So K_i follows K_{i-2} and V_{i-2}, and V_i
// follows K_{i-1}, which is free as soon as its scores are made: the values
// lie there when their weights are ready.  (With two buffers for K and one for
// V every step waited 700 cycles for its values.)
template <typename T>
__global__ void __launch_bounds__(kAttendThreads, 1)
    latent_attend_kernel(const __grid_constant__ CUtensorMap tm_query,
                         const __grid_constant__ CUtensorMap tm_key,
                         const __grid_constant__ CUtensorMap tm_value,
                         const __grid_constant__ CUtensorMap tm_rot,
                         const __grid_constant__ LatentPrefillArgs a)
{
    using S = AttendShape;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* s_query = smem;
    uint8_t* s_ring = s_query + 2 * S::kQueryBytes;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(s_ring + S::kSlots * S::kSlotBytes);    // [2]
    uint64_t* k_full = q_full + 2;         // [2], of even and odd tiles
    uint64_t* k_empty = k_full + 2;        // [2]
    uint64_t* v_full = k_empty + 2;        // [2]
    uint64_t* v_empty = v_full + 2;        // [2]
    uint64_t* s_full = v_empty + 2;        // [2][2], of a query tile's halves
    uint64_t* p_full = s_full + 4;         // [2][2]
    uint64_t* pv_done = p_full + 4;        // [2][2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pv_done + 4);
    int32_t* begun = reinterpret_cast<int32_t*>(tmem_slot + 1);   // the first tile's first weights

    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int h = blockIdx.x;
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tm_query);
        prefetch_tensor_map(&tm_key);
        prefetch_tensor_map(&tm_value);
        prefetch_tensor_map(&tm_rot);
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 2);                    // both tiles' products
            mbar_init(v_full + i, 1);
            mbar_init(v_empty + i, 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 128);
            mbar_init(pv_done + i, 1);
        }
        *begun = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    allow_dependents();
    int32_t item = blockIdx.z * a.pairs + blockIdx.y;
    if (a.sorted) {
        // The item whose size has this block's rank among them all.
        int32_t* sizes = reinterpret_cast<int32_t*>(smem);
        const int32_t n = gridDim.y, i = threadIdx.x;
        if (i < n) sizes[i] = attend_size(a, i);
        __syncthreads();
        if (i < n) {
            const int32_t mine = sizes[i];
            int32_t rank = 0;
            for (int32_t k = 0; k < n; ++k) rank += sizes[k] > mine || (sizes[k] == mine && k < i);
            if (rank == item) sizes[n] = i;
        }
        __syncthreads();
        item = __shfl_sync(kFullMask, sizes[n], 0);
        fence_proxy_async_smem();                         // the queries' copies take this place
        __syncthreads();
    }
    const int s = item / a.pairs;
    const int row0 = (a.pairs - 1 - item % a.pairs) * 2 * kQueryTile;
    const PromptSpan span = prompt_span(a, s);
    if (threadIdx.x == 0 && h == 0 && row0 == 0 && (span.first < 0 || span.context < 0))
        status_or(a.d_status, PA_STATUS_BAD_CONTEXT);
    if (row0 >= span.count) return;
    if (span.context < 0) {                               // zero rows
        const int n = min(2 * kQueryTile, span.count - row0);
        for (int i = threadIdx.x; i < n * (kValue / 8); i += kAttendThreads) {
            const int64_t row = static_cast<int64_t>(span.first + row0 + i / (kValue / 8)) * a.num_heads + h;
            reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * kValue)[i % (kValue / 8)] =
                make_uint4(0, 0, 0, 0);
        }
        return;
    }
    // Tiles of keys each query tile sees: up to its last query's position.
    const int32_t before = span.context - span.count;     // tokens before the first query
    int32_t steps[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int32_t r = row0 + t * kQueryTile;
        steps[t] = r >= span.count ? 0
                                   : (before + min(span.count, r + kQueryTile) + kKvTile - 1) / kKvTile;
        steps[t] = __shfl_sync(kFullMask, steps[t], 0);
    }
    const int32_t total = max(steps[0], steps[1]);

    if (warp == 9) tmem_alloc(tmem_slot, 512);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_slot, 0);
    const uint32_t leader = elect_lane() ? 1u : 0u;
    bool ok = true;

    if (warp == 8) {
        auto queries = [&](int t) {
            if (steps[t] == 0 || !leader) return;
            mbar_arrive_expect_tx(q_full + t, S::kQueryBytes);
#pragma unroll
            for (int c = 0; c < S::kChunks; ++c)
                tma_load_3d(s_query + t * S::kQueryBytes + c * kQueryTile * 128, &tm_query, c * 64,
                            span.first + row0 + t * kQueryTile, h, q_full + t);
        };
        queries(0);                                       // the second tile's after the first keys
        int32_t keys = 0, values = 0;                     // tiles copied
        const int32_t plane = s * a.num_heads + h;
        for (int32_t i = 0; i < total; ++i) {
            const int b = i & 1;
            if (i >= 2)
                ok = mbar_poll_warp(k_empty + b, (i / 2 - 1) & 1) &&
                     mbar_poll_warp(v_empty + b, (i / 2 - 1) & 1);
            if (!ok) break;
            if (leader) {
                mbar_arrive_expect_tx(k_full + b, S::kKeySlots * S::kSlotBytes);
#pragma unroll
                for (int c = 0; c < S::kKeySlots; ++c)
                    tma_load_3d(s_ring + (5 * i + c) % S::kSlots * S::kSlotBytes,
                                c < 2 ? &tm_key : &tm_rot, c < 2 ? c * 64 : 0, i * kKvTile,
                                c < 2 ? plane : s, k_full + b);
            }
            ++keys;
            if (i == 0) queries(1);
            if (i >= 1) ok = mbar_poll_warp(k_empty + (b ^ 1), ((i - 1) / 2) & 1);
            if (!ok) break;
            if (leader) {
                mbar_arrive_expect_tx(v_full + b, S::kValueSlots * S::kSlotBytes);
#pragma unroll
                for (int c = 0; c < S::kValueSlots; ++c)
                    tma_load_3d(s_ring + (5 * i + 3 + c) % S::kSlots * S::kSlotBytes, &tm_value, c * 64,
                                i * kKvTile, plane, v_full + b);
            }
            ++values;
        }
        if (!ok) {                                        // let the copies in flight land
            if (lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
            for (int t = 0; t < 2; ++t)
                if (steps[t] > 0) mbar_poll_warp(q_full + t, 0);
            for (int k = max(0, keys - 2); k < keys; ++k) mbar_poll_warp(k_full + (k & 1), (k / 2) & 1);
            for (int k = max(0, values - 2); k < values; ++k) mbar_poll_warp(v_full + (k & 1), (k / 2) & 1);
        }
    } else if (warp >= 9) {
        const int t = warp - 9;
        const int32_t n = steps[t];
        const uint32_t idesc_s = mma_desc<T>(kQueryTile, kHalf);
        const uint32_t idesc_o = mma_desc<__half>(kQueryTile, 64, false, true);
        const uint32_t query = smem_u32(s_query) + t * S::kQueryBytes, ring = smem_u32(s_ring);
        // Scores of half j of the keys (of tile j / 2, which has arrived).
        auto scores = [&](int32_t j) {
            const int half = j & 1;
#pragma unroll
            for (int c = 0; c < S::kChunks; ++c) {
                const uint64_t da = desc_k_major(query + c * kQueryTile * 128);
                const uint64_t db = desc_k_major(ring + (5 * (j >> 1) + c) % S::kSlots * S::kSlotBytes +
                                                 half * kHalf * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss(tmem + t * kKvTile + half * kHalf, da + 2 * k, db + 2 * k, idesc_s, c + k > 0,
                           leader);
            }
            if (leader) {
                mma_commit(s_full + 2 * t + half);
                if (half) mma_commit(k_empty + ((j >> 1) & 1));
            }
        };
        // The weights of half j times its values.
        auto values = [&](int32_t j) {
            const int half = j & 1;
#pragma unroll
            for (int c = 0; c < S::kValueSlots; ++c) {
                const uint64_t db = desc_mn_major(
                    ring + (5 * (j >> 1) + 3 + c) % S::kSlots * S::kSlotBytes + half * kHalf * 128,
                    S::kSlotBytes);
#pragma unroll
                for (int k = 0; k < kHalf / 16; ++k)
                    mma_ts(tmem + S::kOCol + t * kValue + c * 64, tmem + t * kKvTile + half * kHalf + k * 8,
                           db + k * (2048 >> 4), idesc_o, j + k > 0, leader);
            }
            if (leader) {
                mma_commit(pv_done + 2 * t + half);
                if (half) mma_commit(v_empty + ((j >> 1) & 1));
            }
        };
        ok = (n == 0 || mbar_poll_warp(q_full + t, 0)) && mbar_poll_warp(k_full, 0);
        // The second tile starts when the first one's weights are out: apart,
        // their softmax and products alternate.
        if (t == 1 && n > 0)
            for (int i = 0; i < 4096 && !__all_sync(kFullMask, *static_cast<volatile int32_t*>(begun) != 0); ++i)
                __nanosleep(20);
        if (ok && n > 0) {
            scores(0);
            scores(1);
        } else if (ok && leader) {
            mbar_arrive(k_empty);
        }
        // Past the tile's last step the room is let go of all the same (not
        // before the copies are there: a release a step, or they would run ahead).
        for (int32_t i = 0; i < total; ++i) {
            ok = ok && mbar_poll_warp(v_full + (i & 1), (i / 2) & 1) &&
                 (i >= n || mbar_poll_warp(p_full + 2 * t, i & 1));
            if (!ok) break;
            tmem_fence_after();
            // S of the next half in the same place takes that of P: products run in order
            if (i < n) values(2 * i);
            if (i + 1 < total) {
                ok = mbar_poll_warp(k_full + ((i + 1) & 1), ((i + 1) / 2) & 1);
                if (!ok) break;
                if (i + 1 < n)
                    scores(2 * i + 2);
                else if (leader)
                    mbar_arrive(k_empty + ((i + 1) & 1));
            }
            if (i < n) {
                ok = mbar_poll_warp(p_full + 2 * t + 1, i & 1);
                if (!ok) break;
                tmem_fence_after();
                values(2 * i + 1);
                if (i + 1 < n) scores(2 * i + 3);
            } else if (leader) {
                mbar_arrive(v_empty + (i & 1));
            }
        }
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    } else {
        const int t = warp >> 2;
        const int32_t n = steps[t];
        const int32_t r = row0 + t * kQueryTile + (threadIdx.x & 127);          // the thread's query
        // the last token it sees; rows past the queries see what the last one does
        const int32_t last = before + min(r, span.count - 1);
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + quarter + t * kKvTile;
        const uint32_t o_tmem = tmem + quarter + S::kOCol + t * kValue;
        float m = -INFINITY, l = 0.f;
        for (int32_t j = 0; j < 2 * n; ++j) {
            const int half = j & 1;
            const int32_t t0 = j * kHalf;
            const uint2 word = *reinterpret_cast<const uint2*>(a.ws_mask +
                                                               ((static_cast<int64_t>(s) * a.rows + t0) >> 5));
            const float2 ex = *reinterpret_cast<const float2*>(
                a.ws_exp + (((static_cast<int64_t>(s) * a.num_heads + h) * a.rows + t0) >> 5));
            ok = mbar_poll_warp(s_full + 2 * t + half, (j >> 1) & 1);
            if (!ok) break;
            tmem_fence_after();
            uint32_t x[kHalf];
#pragma unroll
            for (int c = 0; c < kHalf / 32; ++c)
                tmem_ld32(*reinterpret_cast<uint32_t(*)[32]>(x + 32 * c), s_tmem + half * kHalf + 32 * c);
            tmem_wait_ld();
            float unit = a.scale_log2;
            const bool whole = (word.x & word.y) == ~0u && last - t0 >= kHalf - 1;
            if (!__all_sync(kFullMask, whole) || unit < 0.f) {
                // scaled here: a masked score is -inf whatever the scale
                const uint32_t words[2] = {word.x, word.y};
#pragma unroll
                for (int e = 0; e < kHalf; ++e) {
                    const bool sees = e <= last - t0 && (words[e >> 5] >> (e & 31) & 1);
                    x[e] = __float_as_uint(sees ? __uint_as_float(x[e]) * unit : -INFINITY);
                }
                unit = 1.f;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < kHalf; e += 2)
                top[(e >> 1 & 1) + 2 * (e >> 5)] =
                    max3(top[(e >> 1 & 1) + 2 * (e >> 5)], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            // Weights take the powers of two of their values along: w = 2^(x + ex - m),
            // so m follows the largest product of a weight and a value, and
            //   out = sum w V' / l,  l = sum w 2^-ex = sum 2^(x - m).
            const float peaks[2] = {fmaf(fmaxf(top[0], top[1]), unit, ex.x),
                                    fmaf(fmaxf(top[2], top[3]), unit, ex.y)};
            const float peak = fmaxf(peaks[0], peaks[1]);
            // The reference moves where it is unset or passed by 2^8.  32 tokens whose
            // products all lie 2^-40 below it are faint: their weights are 0 in fp16, but
            // in l they count (zeros beside values of 2^70).  2^(x + ex - m) may be below
            // what fp32 has, 2^(x - m) is not where it matters, so they go without ex.
            const bool moves = peak > m + 8.0f;
            bool faint[2] = {false, false}, any_faint = false;
            if (__any_sync(kFullMask, moves || fminf(peaks[0], peaks[1]) < m + kFaint)) {
                if (__any_sync(kFullMask, moves)) {
                    const float f = moves ? exp2_fast(m - peak) : 1.f;
                    // l may be held by tokens of small values: its factor, 2^-186 at the
                    // least for equal scores, is applied as two that fp32 has
                    const float root = moves ? exp2_fast(0.5f * (m - peak)) : 1.f;
                    if (moves) m = peak;
                    l = l * root * root;
                    if (j > 0) {
                        ok = mbar_poll_warp(pv_done + 2 * t + (half ^ 1), ((j - 1) >> 1) & 1);
                        if (!ok) break;
                        tmem_fence_after();
#pragma unroll 1
                        for (int c = 0; c < kValue; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(o, o_tmem + c);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(o_tmem + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                faint[0] = peaks[0] < m + kFaint;
                faint[1] = peaks[1] < m + kFaint;
                any_faint = __any_sync(kFullMask, faint[0] || faint[1]);
            }
            const float sub = (m == -INFINITY ? 0.f : m) - kHeadroom;
            const float shift[2] = {faint[0] ? 0.f : ex.x, faint[1] ? 0.f : ex.y};
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 unit2 = make_float2(unit, unit);
            const float2 add[2] = {make_float2(shift[0] - sub, shift[0] - sub),
                                   make_float2(shift[1] - sub, shift[1] - sub)};
            uint32_t p[kHalf / 2];
#pragma unroll
            for (int e = 0; e < kHalf / 2; ++e) {
                const float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                      unit2, add[e >> 4]);
                const float2 w = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                sum[e >> 4] = add2(sum[e >> 4], w);
                p[e] = Elem<__half>::from_float2(w.x, w.y);
            }
            if (any_faint) {
#pragma unroll
                for (int e = 0; e < kHalf / 2; ++e) p[e] = faint[e >> 4] ? 0u : p[e];
            }
            tmem_st32(s_tmem + half * kHalf, p);
            l += (sum[0].x + sum[0].y) * exp2_fast(-shift[0]) + (sum[1].x + sum[1].y) * exp2_fast(-shift[1]);
            tmem_wait_st();
            tmem_fence_before();
            mbar_arrive(p_full + 2 * t + half);
            if (j == 0 && threadIdx.x == 0) *static_cast<volatile int32_t*>(begun) = 1;
        }
        if (ok && n > 0) ok = mbar_poll_warp(pv_done + 2 * t + 1, (n - 1) & 1);
        if (ok && n > 0) {
            tmem_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;      // (NaN where a score was)
            // Through shared memory (the tile's queries have been used), 8 KB a
            // warp: stored a row a thread, the 32 lines that each store touches
            // took 9000 cycles.  16-byte chunk j of row r lies at j ^ (r % 8).
            uint8_t* mine = s_query + t * S::kQueryBytes + (warp & 3) * 8192;
#pragma unroll
            for (int c = 0; c < kValue; c += 32) {
                uint32_t o[32];
                tmem_ld32(o, o_tmem + c);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[e] = Elem<T>::from_float2(__uint_as_float(o[8 * j + 2 * e]) * inv,
                                                    __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
                    *reinterpret_cast<uint4*>(mine + lane * 256 + ((c / 8 + j) ^ (lane & 7)) * 16) =
                        make_uint4(p[0], p[1], p[2], p[3]);
                }
            }
            __syncwarp();
            const int32_t first = row0 + t * kQueryTile + (warp & 3) * 32;      // the warp's first query
            T* dst = static_cast<T*>(a.out) +
                     (static_cast<int64_t>(span.first + first) * a.num_heads + h) * kValue + (lane & 15) * 8;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int row = 2 * k + (lane >> 4);
                const uint4 v =
                    *reinterpret_cast<const uint4*>(mine + row * 256 + ((lane & 15) ^ (row & 7)) * 16);
                if (first + row < span.count)
                    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(row) * a.num_heads * kValue) = v;
            }
        }
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace pa
