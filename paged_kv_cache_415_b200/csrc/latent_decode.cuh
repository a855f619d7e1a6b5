// latent_decode.cuh -- single-query attention over the paged latent pool
// with absorbed projections (sm_100a tensor cores).
//
// For a sequence with rows r_t = (c_t, k_t) of W = L + 64 elements and heads
// h with queries q_h:  x_ht = scale q_h . r_t,  o_h = softmax(x_h) C.  All
// heads share the rows, so a row is read once for up to 64 heads and serves
// both products from the same place in shared memory:
//   S^T [64 tokens x heads] = R Q^T      rows as the K-major operand
//   O^T [L x heads] += C^T P^T           rows as the MN-major operand
// Tokens and latent elements take the rows of the products, heads their
// columns, so no product is wider than the heads need: with the heads in the
// rows of S (64 at least) a batch of 16 heads drew the power of eight times
// its products and the SM clock fell from 1.97 to 1.69 GHz.
//
// Work split: the 64-token tiles of all sequences form one list, cut into
// equal runs, one a CTA (one CTA an SM: two stages of 72 KB fill its shared
// memory).  A run that cuts a sequence leaves unnormalised partial sums;
// latent_combine_kernel adds them up in tile order, so results depend on the
// batch's lengths and the SM count only.
//
// Warps: 0-3 softmax and epilogue, 4 and 7 copies (TMA, one box of a block and
// 64 columns each, 50 cycles to issue one: blocks of 16 tokens make 36 a tile,
// so two warps share a tile's parts), 5 the products for S, 6 those for O^T
// (apart, so that neither waits in line behind the other).  A stage is filled in parts of 128 columns
// and S starts with the first that has arrived.
//
// Softmax: a thread has two tokens of N / 4 heads.  It keeps a reference m a
// head and takes p = 2^(x - m) at once; only if some x passes m by more than 8
// (or m is not set yet) do the warps put their maxima together, move m and
// rescale O^T.  So p <= 2^8, exact in 16 bits up to the rounding every p has.
// For fp16, whose smallest numbers are near, m lies another 2^7 lower: p <= 2^15,
// and weights down to 2^-21 of the reference keep all their bits (2^-14 without).
//
// Measured: 256 sequences of 3500 to 4500 tokens, 16 heads, in 203 us of this
// kernel (1.20 GB, 5.9 TB/s: memory); 64 sequences to 4096 tokens, 128 heads,
// in 93 us, 97 a call with the sum (0.42 PFLOP/s: the chain of a tile's copies,
// scores, softmax and sums, with room for two tiles).
#pragma once

#include <cuda.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "pa_common.cuh"
#include "tcgen05.cuh"

namespace pa {

constexpr int kTile = 64;                       // tokens of a tile
constexpr int kLatentThreads = 256;
constexpr int kMaxGroupHeads = 64;              // heads a CTA serves
constexpr int kAhead = 3;                       // tiles whose pages are looked up ahead
constexpr float kRescaleAbove = 8.0f;           // log2 of how far p may pass the reference's
// log2 of the reference token's own p: up to 2^15 fit into fp16, bf16 has the
// exponents of fp32
template <typename T>
constexpr float kHeadroom = 0.0f;
template <>
constexpr float kHeadroom<__half> = 7.0f;

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

// N: columns for heads (a multiple of 16, at most 64).
template <int L, int N>
struct LatentDecodeShape {
    static constexpr int kChunks = L / 64 + 1;                 // 64-column chunks of a row
    static constexpr int kParts = L / 128 + 1;                 // of a stage: the last is the rotated chunk
    static constexpr int kStageBytes = kChunks * kTile * 128;
    static constexpr int kQueryChunk = N * 128;
    static constexpr int kQueryBytes = kChunks * kQueryChunk;
    // P^T [heads][64 tokens]; the epilogue stages 1 KB a warp in it
    static constexpr int kWeightBytes = N * 128 > 4096 ? N * 128 : 4096;
    static constexpr int kFixed = 1024 + kQueryBytes + kWeightBytes + 2048;
    static constexpr int kStages = (227 * 1024 - kFixed) / kStageBytes < 5
                                       ? (227 * 1024 - kFixed) / kStageBytes : 5;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    // TMEM columns: S^T (two buffers), O^T (L / 128 blocks of 128 lanes)
    static constexpr int kOCol = 2 * N;
    static constexpr int kColumns = (2 + L / 128) * N;
    static constexpr int kAlloc = kColumns <= 64 ? 64 : kColumns <= 128 ? 128 : kColumns <= 256 ? 256 : 512;
};

// The CTA's tiles, in order: tile `tile` of sequence s with context ctx.
// Every warp walks the same list.
struct TileWalk {
    const LatentDecodeArgs* a;
    int32_t s, tile, tiles, ctx, left;

    __device__ __forceinline__ void load()
    {
        // from one lane: what the loops count is then in uniform registers
        ctx = __shfl_sync(kFullMask, checked_context(a->context_lens, s, a->max_context_len,
                                                     a->max_blocks_per_seq, a->block_size), 0);
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

__device__ __forceinline__ void load16(float (&f)[16], const float* src)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4*>(src)[i];
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
}

template <typename T, int L, int N>
__global__ void __launch_bounds__(kLatentThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap tm_query,
                         const __grid_constant__ CUtensorMap tm_cache,
                         const __grid_constant__ LatentDecodeArgs a)
{
    using S = LatentDecodeShape<L, N>;
    constexpr int CH = S::kChunks;
    constexpr int ST = S::kStages;
    constexpr int PT = S::kParts;
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
    uint64_t* masks = bars + 9;            // [ST]: which tokens of the tile count
    uint64_t* k_empty = masks + ST;        // [ST]
    uint64_t* k_full = k_empty + ST;       // [ST][PT]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + ST * PT);
    int32_t* run = reinterpret_cast<int32_t*>(tmem_slot + 1);     // s0, t0, count
    int32_t* scan = run + 3;                                      // [8] warp totals
    float* factors = reinterpret_cast<float*>(s_misc + 512);      // [64]
    float* tops = factors + kMaxGroupHeads;                       // [4][64]: of a warp's tokens

    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int group = blockIdx.x;
    const int h0 = group * a.group_heads;
    const int heads = min(a.group_heads, a.num_heads - h0);

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
            for (int p = 0; p < PT; ++p) mbar_init(k_full + i * PT + p, 1);
            mbar_init(k_empty + i, 1);
        }
        fence_barrier_init();
    }
    if (warp == 5) tmem_alloc(tmem_slot, S::kAlloc);
    if (warp == 4 && lane == 0) {
        prefetch_tensor_map(&tm_query);
        prefetch_tensor_map(&tm_cache);
    }
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
    const uint32_t tmem = __shfl_sync(kFullMask, *tmem_slot, 0);
    TileWalk w;
    w.start(a, __shfl_sync(kFullMask, run[0], 0), __shfl_sync(kFullMask, run[1], 0),
            __shfl_sync(kFullMask, run[2], 0));
    const uint32_t leader = elect_lane() ? 1u : 0u;
    bool ok = true;

    if (warp == 4 || warp == 7) {
        // Copies.  Lane l looks up the page of a tile's block l, kAhead tiles in
        // front of the one being copied, so that no copy waits for its table.
        // Warp 4 takes the even parts and the rotated one, warp 7 the odd ones
        // and the queries.
        const bool odd = warp == 7;
        const int block_bytes = a.block_size * 128;       // of one chunk
        int32_t it = 0, seg = 0;
        bool fresh = true;                                // first tile of a segment
        int32_t page[kAhead + 1];                         // as the table has them
        TileWalk ahead = w;
        auto look = [&](int32_t& pg) {
            const int32_t t0 = ahead.tile * kTile;
            const int32_t blocks = (min(kTile, ahead.ctx - t0) + a.block_size - 1) / a.block_size;
            pg = 0;
            if (lane < blocks)
                pg = a.block_tables[static_cast<int64_t>(ahead.s) * a.max_blocks_per_seq +
                                    t0 / a.block_size + lane];
            ahead.next();
        };
        auto queries = [&]() {
            if (leader) {
                mbar_arrive_expect_tx(q_full, S::kQueryBytes);
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    tma_load_3d(s_query + c * S::kQueryChunk, &tm_query, c * 64,
                                w.s * a.num_heads + h0, 0, q_full);
            }
            ++seg;
        };
        if (odd && w.left > 0) queries();                 // the first ones before any rows
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (ahead.left > 0) look(page[i]);
        while (w.left > 0 && ok) {
            const int st = it % ST;
            const int32_t valid = min(kTile, w.ctx - w.tile * kTile);
            const int blocks = (valid + a.block_size - 1) / a.block_size;
            if (ahead.left > 0) look(page[kAhead]);
            uint64_t mask = valid == 64 ? ~0ull : (1ull << valid) - 1;
            const bool bad = lane < blocks && (page[0] < 0 || page[0] >= a.num_blocks);
            // a block outside the pool reads as zeros, beyond the map's end
            const int32_t mine = bad ? static_cast<int32_t>(a.num_blocks) : page[0];
            const uint32_t bad_blocks = __ballot_sync(kFullMask, bad);
            if (bad_blocks != 0) {
                if (lane == 0 && group == 0 && !odd) status_or(a.d_status, PA_STATUS_BAD_BLOCK);
                for (int b = 0; b < blocks; ++b)
                    if (bad_blocks >> b & 1)
                        mask &= ~((a.block_size == 64 ? ~0ull : (1ull << a.block_size) - 1)
                                  << (b * a.block_size));
            }
            int32_t pages[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) pages[b] = __shfl_sync(kFullMask, mine, b);
            uint8_t* stage = s_rows + st * S::kStageBytes;
            if (it >= ST) ok = mbar_poll_warp(k_empty + st, (it / ST - 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < PT; ++i) {                // the rotated chunk first, as S takes it
                const int p = i == 0 ? PT - 1 : i - 1;
                const int n = i == 0 ? 1 : 2;             // chunks
                if ((i > 0 && (p & 1) != 0) != odd) continue;
                uint64_t* bar = k_full + st * PT + p;
                if (leader) {
                    // the mask is written before this arrival, its readers wait for it
                    if (i == 0) masks[st] = mask;
                    mbar_arrive_expect_tx(bar, blocks * block_bytes * n);
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (b >= blocks) break;
#pragma unroll
                        for (int c = 2 * p; c < 2 * p + n; ++c)
                            tma_load_3d(stage + c * kTile * 128 + b * block_bytes, &tm_cache, c * 64, 0,
                                        pages[b], bar);
                    }
                }
            }
            ++it;
            if (fresh && it > 1 && odd) {
                ok = mbar_poll_warp(q_empty, (seg - 1) & 1);
                if (!ok) break;
                queries();
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) page[i] = page[i + 1];
            fresh = w.last();
            w.next();
        }
        if (!ok) {                                        // let the copies in flight land
            if (lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
            for (int k = max(0, it - ST); k < it; ++k)
                for (int p = 0; p < PT; ++p)
                    if ((p < PT - 1 && (p & 1) != 0) == odd)
                        mbar_poll_warp(k_full + k % ST * PT + p, (k / ST) & 1);
            if (odd && seg > 0) mbar_poll_warp(q_full, (seg - 1) & 1);
        }
    } else if (warp == 5) {
        // S^T = R Q^T
        const uint32_t idesc = mma_desc<T>(64, N);
        const uint32_t q_addr = smem_u32(s_query), r_addr = smem_u32(s_rows);
        int32_t it = 0, seg = 0;
        bool fresh = true;
        while (w.left > 0) {
            const int st = it % ST, b = it & 1;
            ok = (!fresh || mbar_poll_warp(q_full, seg & 1)) &&
                 (it < 2 || mbar_poll_warp(s_empty + b, (it / 2 - 1) & 1));
            if (!ok) break;
            tmem_fence_after();
            const uint32_t rows = r_addr + st * S::kStageBytes;
            bool ready = mbar_poll_warp(k_full + st * PT + PT - 1, (it / ST) & 1);
            ok = ready;
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const int p = i == 0 ? PT - 1 : i - 1;
                const int n = i == 0 ? 1 : 2;
                if (!ready) ok = ok && mbar_poll_warp(k_full + st * PT + p, (it / ST) & 1);
                // look for the next part while this one's products go out
                if (i + 1 < PT) ready = mbar_try_wait(k_full + st * PT + i, (it / ST) & 1);
#pragma unroll
                for (int c = 2 * p; c < 2 * p + n; ++c) {
                    const uint64_t da = desc_k_major(rows + c * kTile * 128);
                    const uint64_t db = desc_k_major(q_addr + c * S::kQueryChunk);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem + b * N, da + 2 * k, db + 2 * k, idesc, i + k > 0 || c > 2 * p,
                               leader);
                }
                ready = __all_sync(kFullMask, ready);
            }
            if (!ok) break;
            fresh = w.last();
            if (leader) {
                mma_commit(s_full + b);
                if (fresh) mma_commit(q_empty);
            }
            if (fresh) ++seg;
            ++it;
            w.next();
        }
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    } else if (warp == 6) {
        // O^T += C^T P^T
        const uint32_t idesc = mma_desc<T>(128, N, true, false);
        const uint32_t r_addr = smem_u32(s_rows);
        const uint64_t db = desc_k_major(smem_u32(s_p));
        int32_t it = 0, seg = 0;
        bool fresh = true;
        while (w.left > 0) {
            const int st = it % ST;
            ok = mbar_poll_warp(p_full, it & 1) &&
                 (!(fresh && seg > 0) || mbar_poll_warp(o_empty, (seg - 1) & 1));
            if (!ok) break;
            tmem_fence_after();
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint64_t da = desc_mn_major(
                    r_addr + st * S::kStageBytes + 2 * b * kTile * 128, kTile * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss(tmem + S::kOCol + b * N, da + k * (2048 >> 4), db + 2 * k, idesc,
                           !fresh || k > 0, leader);
            }
            if (leader) {
                mma_commit(k_empty + st);
                mma_commit(pv_done);
            }
            fresh = w.last();
            if (fresh) ++seg;
            ++it;
            w.next();
        }
        if (!ok && lane == 0) status_or(a.d_status, PA_STATUS_TIMEOUT);
    } else {
        // A wait that gave up is not repeated: the warps walk on together, so
        // that none is left alone at a barrier, and what they store is not
        // specified (PA_STATUS_TIMEOUT).
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = mbar_poll_warp(bar, parity);
        };
        // Softmax and epilogue.  Rows of a 64-row product use 16 lanes of each
        // warp's 32: the warp has tokens 16 warp .. + 15 of the tile, a lane
        // those at lane / 4 and 8 further, of heads 8 j + 2 (lane % 4) and the
        // next:  x[4 j + 2 (token / 8) + head % 2],  m and l [2 j + head % 2].
        constexpr int J = N / 8;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const int tok = warp * 16 + (lane >> 2);
        const int head0 = 2 * (lane & 3);
        // stmatrix: lane l gives head l % 8 of matrix l / 8 = (token half, j)
        const uint32_t p_addr = smem_u32(s_p) + (lane >> 4) * 1024 + (lane & 7) * 128 +
                                (((warp * 2 + (lane >> 3 & 1)) ^ (lane & 7)) << 4);
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
        float m[2 * J], l[2 * J];
        int32_t it = 0;
        bool fresh = true;
        bool first_seg = true;
        bool cut = w.tile > 0;                            // the segment began in another run
        while (w.left > 0) {
            const int st = it % ST, b = it & 1;
            wait(k_full + st * PT + PT - 1, (it / ST) & 1);
            const uint64_t mask = masks[st];
            const bool whole = mask == ~0ull;
            if (fresh) {
                // Unset, a reference is the least finite value: any score passes it but
                // -inf, which less it is still -inf.  Columns past the heads: p = 0, and
                // their reference never moves.
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    m[i] = 8 * (i >> 1) + head0 + (i & 1) < heads ? -FLT_MAX : INFINITY;
                    l[i] = 0.f;
                }
            }
            wait(s_full + b, (it / 2) & 1);
            tmem_fence_after();
            uint32_t x[4 * J];
            tmem_ld_heads<N>(x, lanes + b * N);
            tmem_wait_ld();
            tmem_fence_before();
            mbar_arrive(s_empty + b);
            // looked at early, used where P^T is written
            const bool pv_ready = it == 0 || mbar_test(pv_done, (it - 1) & 1);
            const bool on[2] = {(mask >> tok & 1) != 0, (mask >> (tok + 8) & 1) != 0};
            if (fresh && mask != 0) {
                // The segment's references: the scores of its first token that
                // counts.  (Its maxima would do as well, for three shuffles and
                // an exchange more a head: p may pass 1 by 2^8.)  Not below the
                // least finite value: a score of -inf less itself would be NaN.
                const int f = __ffsll(static_cast<long long>(mask)) - 1;
                if ((tok & ~8) == (f & ~8)) {
                    const int half = f >> 3 & 1;
#pragma unroll
                    for (int k = 0; k < J; ++k)
                        *reinterpret_cast<float2*>(tops + 8 * k + head0) = make_float2(
                            __uint_as_float(half ? x[4 * k + 2] : x[4 * k]) * a.scale_log2,
                            __uint_as_float(half ? x[4 * k + 3] : x[4 * k + 1]) * a.scale_log2);
                }
                named_barrier(1, 128);
#pragma unroll
                for (int k = 0; k < J; ++k) {
                    const float2 v = *reinterpret_cast<const float2*>(tops + 8 * k + head0);
                    if (8 * k + head0 < heads) m[2 * k] = fmaxf(v.x, -FLT_MAX) - kHeadroom<T>;
                    if (8 * k + head0 + 1 < heads) m[2 * k + 1] = fmaxf(v.y, -FLT_MAX) - kHeadroom<T>;
                }
            }
            float y[4 * J];
            auto shift = [&]() {                          // y = log2 of the weights
#pragma unroll
                for (int i = 0; i < 4 * J; ++i) {
                    y[i] = fmaf(__uint_as_float(x[i]), a.scale_log2, -m[2 * (i >> 2) + (i & 1)]);
                    if (!whole && !on[i >> 1 & 1]) y[i] = -INFINITY;
                }
            };
            shift();
            float high[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 4 * J; ++i) high[i & 1] = fmaxf(high[i & 1], y[i]);
            const bool move = named_barrier_or(1, 128, fmaxf(high[0], high[1]) > kRescaleAbove + kHeadroom<T>);
            if (move) {
                // Maxima of the tile: over the lane's tokens, the warp's, the warps'.
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    float top = -INFINITY;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (on[t])
                            top = fmaxf(top, __uint_as_float(x[4 * (i >> 1) + 2 * t + (i & 1)]) *
                                                 a.scale_log2);
#pragma unroll
                    for (int k = 4; k <= 16; k <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, k));
                    if (lane < 4) tops[warp * kMaxGroupHeads + 8 * (i >> 1) + head0 + (i & 1)] = top;
                }
                named_barrier(1, 128);
                float f[2 * J];
#pragma unroll
                for (int k = 0; k < J; ++k) {
                    float2 top = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 v = *reinterpret_cast<const float2*>(
                            tops + q * kMaxGroupHeads + 8 * k + head0);
                        top.x = fmaxf(top.x, v.x);
                        top.y = fmaxf(top.y, v.y);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float t = (e ? top.y : top.x) - kHeadroom<T>;
                        f[2 * k + e] = 1.f;
                        if (t > m[2 * k + e] + kRescaleAbove) {   // (never past the heads)
                            f[2 * k + e] = exp2_fast(m[2 * k + e] - t);
                            m[2 * k + e] = t;
                            l[2 * k + e] *= f[2 * k + e];
                        }
                    }
                }
                // A segment's last tile: its sums take the place of the maxima,
                // which every warp has to have read.  (Elsewhere the next tile's
                // barriers lie between.)
                if (w.last()) named_barrier(1, 128);
                // every warp writes the same factors, and reads its own
                if (lane < 4) {
#pragma unroll
                    for (int k = 0; k < J; ++k)
                        *reinterpret_cast<float2*>(factors + 8 * k + head0) =
                            make_float2(f[2 * k], f[2 * k + 1]);
                }
                __syncwarp();
                if (!fresh) {
                    wait(pv_done, (it - 1) & 1);
                    tmem_fence_after();
#pragma unroll 1
                    for (int c = 0; c < NB * N; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o, lanes + S::kOCol + c);
                        tmem_wait_ld();
                        float fc[16];
                        load16(fc, factors + c % N);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * fc[i]);
                        tmem_st16(lanes + S::kOCol + c, o);
                    }
                    tmem_wait_st();
                    tmem_fence_before();
                }
                shift();
            }
            // The weights, rounded in pairs; where every score so far is masked
            // (m not set) all of them are 0.
            uint32_t pk[2 * J];
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
                const float p0 = exp2_fast(y[2 * i]), p1 = exp2_fast(y[2 * i + 1]);
                l[2 * (i >> 1)] += p0;
                l[2 * (i >> 1) + 1] += p1;
                pk[i] = Elem<T>::from_float2(p0, p1);
            }
            if (!__all_sync(kFullMask, pv_ready)) wait(pv_done, (it - 1) & 1);
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
#pragma unroll
            for (int j = 0; j < J; j += 2)                // heads 8 j .. 8 j + 15, the warp's 16 tokens
                stmatrix_x4_trans(p_addr + j * 1024, pk[2 * j], pk[2 * j + 1], pk[2 * j + 2],
                                  pk[2 * j + 3]);
            fence_proxy_async_smem();
            mbar_arrive(p_full);
            fresh = w.last();
            if (fresh) {
                // The segment is complete: normalise and store, or leave a partial.
                const bool split = cut || w.tile + 1 < w.tiles;
                const int64_t slot = static_cast<int64_t>(blockIdx.y) * 2 + (first_seg ? 0 : 1);
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1)
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) l[i] += __shfl_xor_sync(kFullMask, l[i], k);
                if (lane < 4) {
#pragma unroll
                    for (int k = 0; k < J; ++k) {
                        const int head = 8 * k + head0;
                        *reinterpret_cast<float2*>(tops + warp * kMaxGroupHeads + head) =
                            make_float2(l[2 * k], l[2 * k + 1]);
                        if (split && warp == 0) {
                            float2* ml = a.ws_ml + slot * a.num_heads + h0 + head;
                            if (head < heads) ml[0].x = m[2 * k];
                            if (head + 1 < heads) ml[1].x = m[2 * k + 1];
                        }
                    }
                }
                named_barrier(1, 128);
                for (int head = lane; head < N; head += 32) {
                    float sum = tops[head];
#pragma unroll
                    for (int q = 1; q < 4; ++q) sum += tops[q * kMaxGroupHeads + head];
                    // every warp writes the same factors, and reads its own
                    factors[head] = sum > 0.f ? 1.f / sum : 0.f;
                    if (split && warp == 0 && head < heads)
                        a.ws_ml[slot * a.num_heads + h0 + head].y = sum;
                }
                __syncwarp();
                wait(pv_done, it & 1);
                tmem_fence_after();
                uint8_t* mine = s_p + warp * 1024;        // P^T has been used
                // two groups of 16 columns at a time
#pragma unroll 1
                for (int c2 = 0; c2 < NB * N; c2 += 32) {
                    uint32_t o[2][16];
                    tmem_ld16(o[0], lanes + S::kOCol + c2);
                    tmem_ld16(o[1], lanes + S::kOCol + c2 + 16);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int c = c2 + 16 * q;
                        const int n0 = c % N, d0 = c / N * 128 + warp * 32;
                        const int left = heads - n0;      // heads of this group
                        if (left <= 0) continue;
                        if (split) {
                            float* dst = a.ws_o + (slot * a.num_heads + h0 + n0) * L + d0 + lane;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i < left) dst[i * L] = __uint_as_float(o[q][i]);
                        } else {
                            // through shared memory: 16 heads x 32 elements, then 16 bytes a lane
                            float fc[16];
                            load16(fc, factors + n0);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                reinterpret_cast<T*>(mine)[i * 32 + lane] =
                                    T(__uint_as_float(o[q][i]) * fc[i]);
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int i = k * 8 + (lane >> 2);
                                const uint4 v =
                                    *reinterpret_cast<const uint4*>(mine + i * 64 + (lane & 3) * 16);
                                if (i < left)
                                    *reinterpret_cast<uint4*>(
                                        static_cast<T*>(a.out) +
                                        (static_cast<int64_t>(w.s) * a.num_heads + h0 + n0 + i) * L + d0 +
                                        (lane & 3) * 8) = v;
                            }
                            __syncwarp();
                        }
                    }
                }
                tmem_fence_before();
                mbar_arrive(o_empty);
                named_barrier(1, 128);                    // the sums and the staging are free again
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
    if (warp == 5) tmem_dealloc(tmem, S::kAlloc);
}

// Adds up the partials of the sequences that a cut of the work list split:
// with M = max_p m_p and w_p = 2^(m_p - M),  out = sum w_p O_p / sum w_p l_p,
// in the order of the CTAs.  Where a row has many partials a CTA takes 128
// elements of one row (DEEP: blockIdx.y), weighs all partials at once and each
// warp adds up every eighth; else a warp takes a row.
constexpr int kCombineWarps = 8;
constexpr int kMaxPartials = 256;                         // of a row: CTAs of the decode kernel

template <typename T, int L, bool DEEP>
__global__ void __launch_bounds__(kCombineWarps * 32)
    latent_combine_kernel(const __grid_constant__ LatentDecodeArgs a)
{
    constexpr int PER = DEEP ? 1 : L / 128;               // float4s a lane holds
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = DEEP ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * kCombineWarps + warp;
    const bool inside = row < static_cast<int64_t>(a.num_seqs) * a.num_heads;
    const int s = inside ? static_cast<int>(row / a.num_heads) : 0;
    const int h = inside ? static_cast<int>(row % a.num_heads) : 0;
    grid_dependency_wait();
    const int32_t ctx = checked_context(a.context_lens, s, a.max_context_len, a.max_blocks_per_seq,
                                        a.block_size);
    if (!inside || ctx <= 0) return;
    const int32_t per_cta = a.ws_meta[0];
    const int32_t begin = a.ws_meta[1 + s];
    const int32_t end = begin + (ctx + kTile - 1) / kTile;
    const int32_t c0 = begin / per_cta, c1 = (end - 1) / per_cta;
    if (c0 == c1) return;                                 // written by the decode kernel
    // A CTA's second slot is its last segment when that is not its first.
    auto slot_of = [&](int32_t c) {
        return (static_cast<int64_t>(c) * 2 + (begin > c * per_cta ? 1 : 0)) * a.num_heads + h;
    };
    float4 acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4* src) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float4 v = src[i * 32];
            acc[i].x = fmaf(w, v.x, acc[i].x);
            acc[i].y = fmaf(w, v.y, acc[i].y);
            acc[i].z = fmaf(w, v.z, acc[i].z);
            acc[i].w = fmaf(w, v.w, acc[i].w);
        }
    };
    float sum = 0.f;
    if constexpr (DEEP) {
        __shared__ float s_w[kMaxPartials], s_top[kCombineWarps], s_sum[kCombineWarps];
        __shared__ float4 s_acc[kCombineWarps][32];
        const int n = c1 - c0 + 1;                        // at most one a thread
        float2 ml = make_float2(-INFINITY, 0.f);
        if (static_cast<int>(threadIdx.x) < n) ml = a.ws_ml[slot_of(c0 + threadIdx.x)];
        float top = ml.x;
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, k));
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCombineWarps; ++i) top = fmaxf(top, s_top[i]);
        const float w = exp2f(ml.x - (top == -INFINITY ? 0.f : top));
        s_w[threadIdx.x] = w;
        float part = w * ml.y;
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) part += __shfl_xor_sync(kFullMask, part, k);
        if (lane == 0) s_sum[warp] = part;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCombineWarps; ++i) sum += s_sum[i];
        const int d0 = blockIdx.y * 128;
#pragma unroll 8
        for (int p = warp; p < n; p += kCombineWarps)
            add(s_w[p], reinterpret_cast<const float4*>(a.ws_o + slot_of(c0 + p) * L + d0) + lane);
        s_acc[warp][lane] = acc[0];
        __syncthreads();
        if (warp != 0) return;
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kCombineWarps; ++i) {
            const float4 v = s_acc[i][lane];
            r.x += v.x; r.y += v.y; r.z += v.z; r.w += v.w;
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * L + d0 + lane * 4) =
            make_uint2(Elem<T>::from_float2(r.x * inv, r.y * inv),
                       Elem<T>::from_float2(r.z * inv, r.w * inv));
    } else {
        float top = -INFINITY;
        for (int32_t c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, a.ws_ml[slot_of(c)].x);
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, k));
        const float sub = top == -INFINITY ? 0.f : top;
#pragma unroll 4
        for (int32_t c = c0; c <= c1; ++c) {
            const int64_t slot = slot_of(c);
            const float2 ml = a.ws_ml[slot];
            const float w = exp2f(ml.x - sub);
            sum = fmaf(w, ml.y, sum);
            add(w, reinterpret_cast<const float4*>(a.ws_o + slot * L) + lane);
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * L + (i * 32 + lane) * 4) =
                make_uint2(Elem<T>::from_float2(acc[i].x * inv, acc[i].y * inv),
                           Elem<T>::from_float2(acc[i].z * inv, acc[i].w * inv));
    }
}

}  // namespace pa
