// latent_decode.cu -- host entry points of single-query attention over the
// paged latent pool: argument checks, the work split and the launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_host.h"
#include "pa_tensor_map.h"
#include "latent_decode.cuh"

namespace pa {

// How the heads and the tiles are split: groups of at most 64 heads, each
// served by `ctas` CTAs, one an SM over all groups.
struct LatentSplit {
    int32_t groups, group_heads, ctas;
    int64_t max_tiles;          // upper bound of the batch's tiles
    bool partials;              // whether a sequence may be cut
};

// Tiles a CTA takes at least: shorter runs cost more in partial sums than they
// save (33 sequences to 700 tokens, 40 heads: 16.0 us a call with 2, 16.2 to 16.6
// with 1, 20 to 22 with 3, 4 or 6; one sequence of 32773: 20.6 with 1 or 2).
constexpr int32_t kMinTiles = 2;

static LatentSplit latent_split(int32_t num_seqs, int32_t num_heads, int32_t max_context_len)
{
    LatentSplit s;
    s.groups = (num_heads + kMaxGroupHeads - 1) / kMaxGroupHeads;
    s.group_heads = (num_heads + s.groups - 1) / s.groups;
    const int64_t per_seq = (static_cast<int64_t>(max_context_len) + kTile - 1) / kTile;
    s.max_tiles = per_seq * num_seqs;
    const int64_t useful = (s.max_tiles + kMinTiles - 1) / kMinTiles;
    // (a combining thread weighs one partial)
    const int64_t sms = sm_count() < kMaxPartials ? sm_count() : kMaxPartials;
    const int64_t fill = sms / s.groups;
    s.ctas = static_cast<int32_t>(useful < 1 ? 1 : useful < fill ? useful : fill);
    s.partials = per_seq > 1 && s.ctas > 1;
    return s;
}

static size_t latent_partial_rows(const LatentSplit& s, int32_t num_heads)
{
    return static_cast<size_t>(s.ctas) * 2 * num_heads;
}

template <typename T, int L, int N>
static pa_status launch_latent_heads(const LatentDecodeArgs& a, const LatentSplit& sp,
                                      const void* query, const void* cache, cudaStream_t stream)
{
    using S = LatentDecodeShape<L, N>;
    static std::atomic<uint64_t> attr_done{0};
    auto kernel = latent_decode_kernel<T, L, N>;
    if (!ensure_smem_attr(kernel, S::kSmem, attr_done)) return PA_ERR_CUDA;
    constexpr uint64_t kRowBytes = (L + 64) * 2;
    CUtensorMap tm_query, tm_cache;
    const uint64_t rows = static_cast<uint64_t>(a.num_seqs) * a.num_heads;
    if (!encode_rows_map(&tm_query, query, L + 64, rows, 1, kRowBytes, kRowBytes * rows,
                         N) ||
        !encode_rows_map(&tm_cache, cache, L + 64, a.block_size, a.num_blocks, kRowBytes,
                         kRowBytes * a.block_size, a.block_size))
        return PA_ERR_CUDA;
    pa_status st = launch_overlapped(kernel, dim3(sp.groups, sp.ctas), dim3(kLatentThreads), S::kSmem,
                                     stream, tm_query, tm_cache, a);
    if (st != PA_OK || !sp.partials) return st;
    // Few rows of many partials: a CTA of eight warps for 128 elements of a
    // row; else a warp for a row.
    const bool deep = sp.ctas / a.num_seqs >= 2 * kCombineWarps;
    if (deep)
        return launch_overlapped(latent_combine_kernel<T, L, true>,
                                 dim3(static_cast<unsigned>(rows), L / 128), dim3(kCombineWarps * 32),
                                 0, stream, a);
    return launch_overlapped(latent_combine_kernel<T, L, false>,
                             dim3(static_cast<unsigned>((rows + kCombineWarps - 1) / kCombineWarps)),
                             dim3(kCombineWarps * 32), 0, stream, a);
}

// Columns for the heads of a group, rounded up to what a product takes.
template <typename T, int L>
static pa_status launch_latent_decode(const LatentDecodeArgs& a, const LatentSplit& sp,
                                      const void* query, const void* cache, cudaStream_t stream)
{
    switch ((sp.group_heads + 15) / 16) {
    case 1: return launch_latent_heads<T, L, 16>(a, sp, query, cache, stream);
    case 2: return launch_latent_heads<T, L, 32>(a, sp, query, cache, stream);
    case 3: return launch_latent_heads<T, L, 48>(a, sp, query, cache, stream);
    default: return launch_latent_heads<T, L, 64>(a, sp, query, cache, stream);
    }
}

}  // namespace pa

extern "C" size_t pa_latent_decode_workspace_size(int32_t num_seqs, int32_t num_heads,
                                                  int32_t latent_dim, int32_t block_size,
                                                  int32_t max_context_len)
{
    using namespace pa;
    if (bad_latent_shape(num_seqs, num_heads, latent_dim, block_size, max_context_len) ||
        !supported_latent(latent_dim, 64) || !supported_latent_block(block_size) ||
        num_heads > kMaxLatentHeads || num_seqs > 65535)
        return 0;
    const LatentSplit sp = latent_split(num_seqs, num_heads, max_context_len);
    if (!sp.partials) return 0;
    const size_t rows = latent_partial_rows(sp, num_heads);
    return rows * (static_cast<size_t>(latent_dim) * 4 + 8) + (static_cast<size_t>(num_seqs) + 1) * 4;
}

extern "C" pa_status pa_latent_decode(void* out, const void* query, const void* cache,
                                      const int32_t* block_tables, const int32_t* context_lens,
                                      int32_t num_seqs, int32_t num_heads, int32_t latent_dim,
                                      int32_t rope_dim, int32_t block_size,
                                      int32_t max_blocks_per_seq, int64_t num_blocks,
                                      int32_t max_context_len, float scale, void* workspace,
                                      size_t workspace_bytes, pa_dtype dtype, int32_t* d_status,
                                      pa_stream_t stream)
{
    using namespace pa;
    if (bad_latent_shape(num_seqs, num_heads, latent_dim, block_size, max_context_len) || rope_dim <= 0 ||
        max_blocks_per_seq <= 0 || num_blocks <= 0 || !isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (!supported_dtype(dtype) || !supported_latent(latent_dim, rope_dim) ||
        !supported_latent_block(block_size) || num_heads > kMaxLatentHeads || num_seqs > 65535)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(cache) || !aligned4(block_tables) ||
        !aligned4(context_lens) || (d_status && !aligned4(d_status)))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa_latent_decode_workspace_size(num_seqs, num_heads, latent_dim, block_size,
                                                        max_context_len);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
        return PA_ERR_INVALID_ARG;
    const LatentSplit sp = latent_split(num_seqs, num_heads, max_context_len);
    if (sp.max_tiles > (1 << 30) || max_context_len > 0x7fffffff - kTile || num_blocks > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    LatentDecodeArgs a = {};
    a.out = out;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    if (sp.partials) {
        const size_t rows = latent_partial_rows(sp, num_heads);
        a.ws_o = static_cast<float*>(workspace);
        a.ws_ml = reinterpret_cast<float2*>(a.ws_o + rows * latent_dim);
        a.ws_meta = reinterpret_cast<int32_t*>(a.ws_ml + rows);
    }
    a.num_seqs = num_seqs;
    a.num_heads = num_heads;
    a.group_heads = sp.group_heads;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.max_context_len = max_context_len;
    a.min_tiles = kMinTiles;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.d_status = d_status;
    if (dtype == PA_DTYPE_F16)
        return latent_dim == 512 ? launch_latent_decode<__half, 512>(a, sp, query, cache, stream)
                                 : launch_latent_decode<__half, 256>(a, sp, query, cache, stream);
    return latent_dim == 512
               ? launch_latent_decode<__nv_bfloat16, 512>(a, sp, query, cache, stream)
               : launch_latent_decode<__nv_bfloat16, 256>(a, sp, query, cache, stream);
}
