// latent_decode.cuh -- single-query attention over the paged latent pool
// with absorbed projections (sm_100a tensor cores).
//
// For a sequence with rows r_t = (c_t, k_t) of W = L + 64 elements and heads
// h with queries q_h:  x_ht = scale q_h . r_t,  o_h = softmax(x_h) C.  All
// heads share the rows, so a row is read once for up to 64 heads and serves
// both products from the same place in shared memory:
//   S [64 heads x 64 tokens] = Q R^T       rows as the K-major operand
//   O^T [L x heads] += C^T P^T             rows as the MN-major operand
// Heads run along the columns of O^T, so few heads waste no tensor time:
// the 128 lanes of each accumulator are latent elements.
//
// Work split: the 64-token tiles of all sequences form one list, cut into
// equal runs, one a CTA (one CTA an SM: two stages of 72 KB and the query
// fill its shared memory).  A run that cuts a sequence leaves unnormalised
// partial sums; latent_combine_kernel adds them up in tile order, so results
// depend on the batch's lengths and the SM count only.
//
// Warps: 0-3 softmax and epilogue, 4 copies (TMA, one box of a block and 64
// columns each), 5 products.  The softmax keeps a reference m a head; O^T is
// rescaled only when a maximum passes m by more than 2^8, so p <= 2^8 (exact
// in 16 bits up to the rounding every p has).
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "pa_common.cuh"
#include "tcgen05.cuh"

namespace pa {

constexpr int kTile = 64;                       // tokens of a tile
constexpr int kLatentThreads = 192;
constexpr int kMaxGroupHeads = 64;              // heads a CTA serves
constexpr float kRescaleAbove = 8.0f;           // log2 of how far p may pass 1

struct LatentDecodeArgs {
    void* out;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float* ws_o;                // [CTA][2][H][L] unnormalised partial sums
    float2* ws_ml;              // [CTA][2][H] (m, l)
    int32_t* ws_meta;           // [0]: tiles a CTA, [1 + s]: first tile of sequence s
    int32_t num_seqs, num_heads, group_heads, block_size, max_blocks_per_seq;
    int64_t num_blocks;
    int32_t max_context_len, min_tiles;
    float scale_log2;
    int32_t* d_status;
};

// The context of sequence s, or -1 where it is not one.
__device__ __forceinline__ int32_t checked_context(const int32_t* lens, int s, int32_t max_context,
                                                   int32_t max_blocks, int32_t block_size)
{
    const int32_t c = lens[s];
    return c >= 0 && c <= max_context &&
                   static_cast<int64_t>(c) <= static_cast<int64_t>(max_blocks) * block_size
               ? c
               : -1;
}

template <int L>
struct LatentDecodeShape {
    static constexpr int kChunks = L / 64 + 1;                 // 64-column chunks of a row
    static constexpr int kStageBytes = kChunks * kTile * 128;
    static constexpr int kStages = L == 512 ? 2 : 4;
    static constexpr int kQueryBytes = kChunks * kMaxGroupHeads * 128;
    static constexpr int kWeightBytes = kMaxGroupHeads * 128;  // P: heads x 64 tokens
    static constexpr int kSmem = 1024 + kQueryBytes + kStages * kStageBytes + kWeightBytes + 1024;
    static constexpr int kOCol = 128;                          // TMEM: S 2 x 64, then O^T
};

// The CTA's tiles, in order: tile `tile` of sequence s with context ctx.
// Every warp walks the same list.
struct TileWalk {
    const LatentDecodeArgs* a;
    int32_t s, tile, tiles, ctx, left;

    __device__ __forceinline__ void load()
    {
        ctx = checked_context(a->context_lens, s, a->max_context_len, a->max_blocks_per_seq,
                              a->block_size);
        tiles = ctx > 0 ? (ctx + kTile - 1) / kTile : 0;
    }
    __device__ __forceinline__ void start(const LatentDecodeArgs& args, int32_t s0, int32_t t0,
                                          int32_t count)
    {
        a = &args;
        s = s0;
        tile = t0;
        left = count;
        if (left > 0) load();
    }
    __device__ __forceinline__ bool last() const { return left == 1 || tile + 1 == tiles; }
    __device__ __forceinline__ void next()
    {
        --left;
        if (++tile < tiles || left == 0) return;
        tile = 0;
        do {
            ++s;
            load();
        } while (tiles == 0);              // left > 0: a further tile exists
    }
};

template <typename T, int L>
__global__ void __launch_bounds__(kLatentThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap tm_query,
                         const __grid_constant__ CUtensorMap tm_cache,
                         const __grid_constant__ LatentDecodeArgs a)
{
    using S = LatentDecodeShape<L>;
    constexpr int CH = S::kChunks;
    constexpr int ST = S::kStages;
    constexpr int NB = L / 128;            // 128-lane blocks of O^T
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* s_query = smem;
    uint8_t* s_rows = s_query + S::kQueryBytes;
    uint8_t* s_p = s_rows + ST * S::kStageBytes;
    uint8_t* s_misc = s_p + S::kWeightBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_misc);
    uint64_t* q_full = bars;
    uint64_t* q_empty = bars + 1;
    uint64_t* pv_done = bars + 2;
    uint64_t* p_full = bars + 3;
    uint64_t* o_empty = bars + 4;
    uint64_t* s_full = bars + 5;           // [2]
    uint64_t* s_empty = bars + 7;          // [2]
    uint64_t* k_full = bars + 9;           // [ST]
    uint64_t* k_empty = bars + 9 + ST;     // [ST]
    uint64_t* masks = bars + 9 + 2 * ST;   // [ST]: which tokens of the tile count
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 9 + 3 * ST);
    int32_t* run = reinterpret_cast<int32_t*>(tmem_slot + 1);     // s0, t0, count
    int32_t* scan = run + 3;                                      // [6] warp totals
    float* factors = reinterpret_cast<float*>(s_misc + 256);      // [64]
    float* inv_l = factors + kMaxGroupHeads;                      // [64]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x;
    const int h0 = group * a.group_heads;
    const int heads = min(a.group_heads, a.num_heads - h0);
    const int n_cols = (heads + 15) / 16 * 16;                    // columns of O^T
    const int q_rows = (a.group_heads + 7) / 8 * 8;               // rows of a query chunk and box

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(pv_done, 1);
        mbar_init(p_full, 128);
        mbar_init(o_empty, 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, 128);
        }
        for (int i = 0; i < ST; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
        }
        fence_barrier_init();
    }
    if (warp == 5) tmem_alloc(tmem_slot, 512);
    grid_dependency_wait();
    allow_dependents();

    // The CTA's run of tiles: every thread counts the tiles of a slice of the
    // sequences, a scan over the threads gives each slice's first tile.
    {
        const int per = (a.num_seqs + kLatentThreads - 1) / kLatentThreads;
        const int first = min(a.num_seqs, static_cast<int>(threadIdx.x) * per);
        const int last = min(a.num_seqs, first + per);
        int32_t mine = 0;
        for (int s = first; s < last; ++s) {
            const int32_t c = checked_context(a.context_lens, s, a.max_context_len,
                                              a.max_blocks_per_seq, a.block_size);
            if (c > 0) mine += (c + kTile - 1) / kTile;
        }
        int32_t incl = mine;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int32_t v = __shfl_up_sync(kFullMask, incl, k);
            if (lane >= k) incl += v;
        }
        if (lane == 31) scan[warp] = incl;
        if (threadIdx.x == 0) run[2] = 0;
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
        int32_t base = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kLatentThreads / 32; ++w) {
            if (w < warp) base += scan[w];
            total += scan[w];
        }
        const int32_t ctas = static_cast<int32_t>(gridDim.y);
        const int32_t per_cta = max(a.min_tiles, (total + ctas - 1) / ctas);
        const int32_t begin = min(static_cast<int64_t>(blockIdx.y) * per_cta, static_cast<int64_t>(total));
        const int32_t end = min(begin + per_cta, total);
        int32_t at = base + incl - mine;                  // first tile of the slice
        if (begin < end && at <= end) {
            for (int s = first; s < last; ++s) {
                const int32_t c = checked_context(a.context_lens, s, a.max_context_len,
                                                  a.max_blocks_per_seq, a.block_size);
                const int32_t n = c > 0 ? (c + kTile - 1) / kTile : 0;
                if (n > 0) {
                    if (at <= begin && begin < at + n) {
                        run[0] = s;
                        run[1] = begin - at;
                        run[2] = end - begin;
                    }
                    // sequences that begin in this run: where, for the sum of the partials
                    if (group == 0 && a.ws_meta != nullptr && at >= begin && at < end) {
                        a.ws_meta[1 + s] = at;
                        a.ws_meta[0] = per_cta;
                    }
                }
                at += n;
            }
        }
        __syncthreads();
    }
    const uint32_t tmem = *tmem_slot;
    TileWalk w;
    w.start(a, run[0], run[1], run[2]);
    bool ok = true;

    if (warp == 4) {
        // Copies.  Lane l holds the page of the tile's block l.
        const int per_tile = kTile / a.block_size;
        int32_t it = 0, seg = 0;
        bool fresh = true;                                // first tile of a segment
        while (w.left > 0 && ok) {
            const int st = it % ST;
            const int32_t t0 = w.tile * kTile;
            const int32_t valid = min(kTile, w.ctx - t0);
            const int blocks = (valid + a.block_size - 1) / a.block_size;
            int32_t page = 0;
            bool bad = false;
            if (lane < blocks) {
                page = a.block_tables[static_cast<int64_t>(w.s) * a.max_blocks_per_seq +
                                      t0 / a.block_size + lane];
                bad = page < 0 || page >= a.num_blocks;
                // a block outside the pool reads as zeros, beyond the map's end
                if (bad) page = static_cast<int32_t>(a.num_blocks);
            }
            uint64_t mask = valid == 64 ? ~0ull : (1ull << valid) - 1;
            const uint32_t bad_blocks = __ballot_sync(kFullMask, bad);
            if (bad_blocks != 0) {
                if (lane == 0 && group == 0) status_or(a.d_status, PA_STATUS_BAD_BLOCK);
                for (int b = 0; b < blocks; ++b)
                    if (bad_blocks >> b & 1)
                        mask &= ~((a.block_size == 64 ? ~0ull : (1ull << a.block_size) - 1)
                                  << (b * a.block_size));
            }
            if (it >= ST) ok = mbar_wait_warp(k_empty + st, (it / ST - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                masks[st] = mask;
                mbar_arrive_expect_tx(k_full + st, blocks * a.block_size * 128 * CH);
            }
            __syncwarp();
            uint8_t* stage = s_rows + st * S::kStageBytes;
            for (int i0 = 0; i0 < per_tile * CH; i0 += 32) {
                const int i = i0 + lane;
                const int b = i % per_tile, c = i / per_tile;
                const int32_t pg = __shfl_sync(kFullMask, page, b);
                if (c < CH && b < blocks)
                    tma_load_3d(stage + c * kTile * 128 + b * a.block_size * 128, &tm_cache, c * 64,
                                0, pg, k_full + st);
            }
            ++it;
            if (fresh) {
                if (seg > 0) ok = mbar_wait_warp(q_empty, (seg - 1) & 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(q_full, CH * q_rows * 128);
                __syncwarp();
                if (lane < CH)
                    tma_load_3d(s_query + lane * q_rows * 128, &tm_query, lane * 64,
                                w.s * a.num_heads + h0, 0, q_full);
                ++seg;
            }
            fresh = w.last();
            w.next();
        }
        if (!ok) {                                        // let the copies in flight land
            if (lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
            for (int k = max(0, it - ST); k < it; ++k) mbar_wait_warp(k_full + k % ST, (k / ST) & 1);
            if (seg > 0) mbar_wait_warp(q_full, (seg - 1) & 1);
        }
    } else if (warp == 5) {
        // Products, one thread.  S of the next tile goes ahead of O^T of this one.
        if (lane == 0) {
            const uint32_t idesc_s = mma_desc<T>(64, kTile);
            const uint32_t idesc_o = mma_desc<T>(128, n_cols, true, false);
            const uint32_t q_addr = smem_u32(s_query), r_addr = smem_u32(s_rows), p_addr = smem_u32(s_p);
            TileWalk nx = w;
            int32_t nseg = 0, seg = 0;
            bool nfresh = true, fresh = true;
            auto scores = [&](int32_t it) {
                const int st = it % ST, b = it & 1;
                if (nfresh && !mbar_wait_bounded(q_full, nseg & 1)) return false;
                if (!mbar_wait_bounded(k_full + st, (it / ST) & 1)) return false;
                if (it >= 2 && !mbar_wait_bounded(s_empty + b, (it / 2 - 1) & 1)) return false;
                tmem_fence_after();
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    const uint64_t da = desc_k_major(q_addr + c * q_rows * 128);
                    const uint64_t db = desc_k_major(r_addr + st * S::kStageBytes + c * kTile * 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem + b * kTile, da + 2 * k, db + 2 * k, idesc_s, c + k > 0);
                }
                mma_commit(s_full + b);
                nfresh = nx.last();
                if (nfresh) {
                    mma_commit(q_empty);
                    ++nseg;
                }
                nx.next();
                return true;
            };
            int32_t it = 0;
            if (w.left > 0) ok = scores(0);
            while (w.left > 0 && ok) {
                if (nx.left > 0) ok = scores(it + 1);
                if (!ok) break;
                const int st = it % ST;
                ok = mbar_wait_bounded(p_full, it & 1) &&
                     (!(fresh && seg > 0) || mbar_wait_bounded(o_empty, (seg - 1) & 1));
                if (!ok) break;
                tmem_fence_after();
#pragma unroll 1
                for (int b = 0; b < NB; ++b) {
                    const uint64_t da = desc_mn_major(
                        r_addr + st * S::kStageBytes + 2 * b * kTile * 128, kTile * 128);
                    const uint64_t db = desc_k_major(p_addr);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem + S::kOCol + b * n_cols, da + k * (2048 >> 4), db + 2 * k,
                               idesc_o, !fresh || k > 0);
                }
                mma_commit(k_empty + st);
                mma_commit(pv_done);
                fresh = w.last();
                if (fresh) ++seg;
                ++it;
                w.next();
            }
            if (!ok) status_or(a.d_status, PA_STATUS_TIMEOUT);
        }
    } else {
        // A wait that gave up is not repeated: the warps walk on together, so
        // that none is left alone at a barrier, and what they store is not
        // specified (PA_STATUS_TIMEOUT).
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = mbar_wait_warp(bar, parity);
        };
        // Softmax and epilogue.  Head r of the group is lane 32 (r / 16) + r % 16
        // of S (rows of a 64-row product use 16 lanes of each warp's 32).
        const int head = warp * 16 + lane;                // of the group, lanes 0-15
        const bool mine = lane < 16 && head < heads;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        // empty and bad contexts: zero rows
        for (int s = blockIdx.y; s < a.num_seqs; s += gridDim.y) {
            const int32_t c = checked_context(a.context_lens, s, a.max_context_len,
                                              a.max_blocks_per_seq, a.block_size);
            if (c > 0) continue;
            if (c < 0 && threadIdx.x == 0 && group == 0) status_or(a.d_status, PA_STATUS_BAD_CONTEXT);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) +
                                                  (static_cast<int64_t>(s) * a.num_heads + h0) * L);
            for (int i = threadIdx.x; i < heads * L / 8; i += 128) dst[i] = make_uint4(0, 0, 0, 0);
        }
        float m = -INFINITY, l = 0.f;
        int32_t it = 0;
        bool fresh = true;
        bool first_seg = true;
        bool cut = w.tile > 0;                            // the segment began in another run
        while (w.left > 0) {
            const int st = it % ST, b = it & 1;
            wait(k_full + st, (it / ST) & 1);
            wait(s_full + b, (it / 2) & 1);
            tmem_fence_after();
            const uint64_t mask = masks[st];
            const bool whole = mask == ~0ull;
            uint32_t x[kTile];
            if (warp * 16 < heads) {
                tmem_ld32(*reinterpret_cast<uint32_t(*)[32]>(x), lanes + b * kTile);
                tmem_ld32(*reinterpret_cast<uint32_t(*)[32]>(x + 32), lanes + b * kTile + 32);
                tmem_wait_ld();
            }
            tmem_fence_before();
            mbar_arrive(s_empty + b);
            float top = -INFINITY;
            if (mine) {
#pragma unroll
                for (int i = 0; i < kTile; ++i) {
                    float v = __uint_as_float(x[i]) * a.scale_log2;
                    if (!whole && !(mask >> i & 1)) v = -INFINITY;
                    x[i] = __float_as_uint(v);
                    top = fmaxf(top, v);
                }
            }
            // The reference moves when it is unset or passed by 2^8.
            const bool moves = mine && top > m + kRescaleAbove;
            float f = 1.f;
            if (fresh) {
                m = top;
                l = 0.f;
            } else if (moves) {
                f = exp2_fast(m - top);
                m = top;
                l *= f;
            }
            if (lane < 16 && head < kMaxGroupHeads) factors[head] = f;
            const bool rescale = named_barrier_or(1, 128, !fresh && moves);
            if (it > 0) {
                wait(pv_done, (it - 1) & 1);
                tmem_fence_after();
            }
            if (rescale) {
#pragma unroll 1
                for (int c = 0; c < NB * n_cols; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(o, lanes + S::kOCol + c);
                    tmem_wait_ld();
                    const float* fc = factors + c % n_cols;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * fc[i]);
                    tmem_st16(lanes + S::kOCol + c, o);
                }
                tmem_wait_st();
                tmem_fence_before();
            }
            if (!whole) {
                // rows that do not count are zeroed: 0 times what they hold may not be 0
                uint8_t* stage = s_rows + st * S::kStageBytes;
                for (int i = threadIdx.x; i < kTile * (L / 64) * 8; i += 128) {
                    const int t = (i >> 3) % kTile, c = (i >> 3) / kTile;
                    if (!(mask >> t & 1))
                        *reinterpret_cast<uint4*>(stage + (c * kTile + t) * 128 + (i & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
            }
            if (lane < 16 && warp * 16 < n_cols) {
                const float sub = m == -INFINITY ? 0.f : m;
                uint8_t* row = s_p + (head >> 3) * 1024 + (head & 7) * 128;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p0 = mine ? exp2_fast(__uint_as_float(x[j * 8 + 2 * e]) - sub) : 0.f;
                        const float p1 = mine ? exp2_fast(__uint_as_float(x[j * 8 + 2 * e + 1]) - sub) : 0.f;
                        sum += p0 + p1;
                        pk[e] = Elem<T>::from_float2(p0, p1);
                    }
                    *reinterpret_cast<uint4*>(row + ((j ^ (head & 7)) << 4)) =
                        make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                l += sum;
            }
            fence_proxy_async_smem();
            mbar_arrive(p_full);
            fresh = w.last();
            if (fresh) {
                // The segment is complete: normalise and store, or leave a partial.
                const bool split = cut || w.tile + 1 < w.tiles;
                if (mine) inv_l[head] = split ? 1.f : (l > 0.f ? 1.f / l : 0.f);
                const int64_t slot = static_cast<int64_t>(blockIdx.y) * 2 + (first_seg ? 0 : 1);
                if (split && mine) a.ws_ml[slot * a.num_heads + h0 + head] = make_float2(m, l);
                named_barrier(1, 128);
                wait(pv_done, it & 1);
                tmem_fence_after();
                const int d0 = warp * 32 + lane;
#pragma unroll 1
                for (int c = 0; c < NB * n_cols; c += 16) {
                    const int blk = c / n_cols, n0 = c % n_cols;
                    uint32_t o[16];
                    tmem_ld16(o, lanes + S::kOCol + c);
                    tmem_wait_ld();
                    const int d = blk * 128 + d0;
                    if (split) {
                        float* dst = a.ws_o + (slot * a.num_heads + h0 + n0) * L + d;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < heads) dst[static_cast<int64_t>(i) * L] = __uint_as_float(o[i]);
                    } else {
                        T* dst = static_cast<T*>(a.out) +
                                 (static_cast<int64_t>(w.s) * a.num_heads + h0 + n0) * L + d;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < heads)
                                dst[static_cast<int64_t>(i) * L] =
                                    T(__uint_as_float(o[i]) * inv_l[n0 + i]);
                    }
                }
                tmem_fence_before();
                mbar_arrive(o_empty);
                named_barrier(1, 128);                    // inv_l and factors are free again
                first_seg = cut = false;
            }
            ++it;
            w.next();
        }
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 5) tmem_dealloc(tmem, 512);
}

// Adds up the partials of the sequences that a cut of the work list split:
// with M = max_p m_p and w_p = 2^(m_p - M),  out = sum w_p O_p / sum w_p l_p,
// in the order of the CTAs.  With WPR = 1 a warp takes a row of L elements;
// with eight (few rows of many partials) a CTA takes 128 elements of a row
// (blockIdx.y) and each warp every eighth partial.
constexpr int kCombineWarps = 8;

template <typename T, int L, int WPR>
__global__ void __launch_bounds__(kCombineWarps * 32)
    latent_combine_kernel(const __grid_constant__ LatentDecodeArgs a)
{
    grid_dependency_wait();
    constexpr int PER = WPR == 1 ? L / 128 : 1;           // float4s a lane holds
    __shared__ float4 s_acc[WPR][WPR == 1 ? 1 : 32];
    __shared__ float s_sum[kCombineWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kCombineWarps / WPR) + (WPR == 1 ? warp : 0);
    if (row >= static_cast<int64_t>(a.num_seqs) * a.num_heads) return;
    const int s = static_cast<int>(row / a.num_heads), h = static_cast<int>(row % a.num_heads);
    const int32_t ctx = checked_context(a.context_lens, s, a.max_context_len, a.max_blocks_per_seq,
                                        a.block_size);
    if (ctx <= 0) return;
    const int32_t per_cta = a.ws_meta[0];
    const int32_t begin = a.ws_meta[1 + s];
    const int32_t end = begin + (ctx + kTile - 1) / kTile;
    const int32_t c0 = begin / per_cta, c1 = (end - 1) / per_cta;
    if (c0 == c1) return;                                 // written by the decode kernel
    const int d0 = WPR == 1 ? 0 : blockIdx.y * 128;
    // A CTA's second slot is its last segment when that is not its first.
    auto slot_of = [&](int32_t c) {
        return (static_cast<int64_t>(c) * 2 + (begin > c * per_cta ? 1 : 0)) * a.num_heads + h;
    };
    float M = -INFINITY;
    for (int32_t c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, a.ws_ml[slot_of(c)].x);
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, k));
    const float sub = M == -INFINITY ? 0.f : M;
    float4 acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int32_t c = c0 + (WPR == 1 ? 0 : warp); c <= c1; c += WPR) {
        const int64_t slot = slot_of(c);
        const float2 ml = a.ws_ml[slot];
        const float w = exp2f(ml.x - sub);
        sum = fmaf(w, ml.y, sum);
        const float4* src = reinterpret_cast<const float4*>(a.ws_o + slot * L + d0) + lane;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float4 v = src[i * 32];
            acc[i].x = fmaf(w, v.x, acc[i].x);
            acc[i].y = fmaf(w, v.y, acc[i].y);
            acc[i].z = fmaf(w, v.z, acc[i].z);
            acc[i].w = fmaf(w, v.w, acc[i].w);
        }
    }
    if constexpr (WPR > 1) {
        s_acc[warp][lane] = acc[0];
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp != 0) return;
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            const float4 v = s_acc[i][lane];
            r.x += v.x; r.y += v.y; r.z += v.z; r.w += v.w;
            sum += s_sum[i];
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * L + d0 + lane * 4) =
            make_uint2(Elem<T>::from_float2(r.x * inv, r.y * inv),
                       Elem<T>::from_float2(r.z * inv, r.w * inv));
    } else {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * L + (i * 32 + lane) * 4) =
                make_uint2(Elem<T>::from_float2(acc[i].x * inv, acc[i].y * inv),
                           Elem<T>::from_float2(acc[i].z * inv, acc[i].w * inv));
    }
}

}  // namespace pa
