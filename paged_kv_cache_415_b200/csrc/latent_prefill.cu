// latent_prefill.cu -- host entry points of prompt attention over the paged
// latent pool: argument checks, the workspace and the two launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_host.h"
#include "pa_tensor_map.h"
#include "latent_prefill.cuh"

namespace pa {

// The workspace: K and V of every head, the rotated part, one mask bit a
// token and one exponent a head and 32 tokens; a sequence's rows are whole tiles
// of keys.
struct PrefillSpace {
    int64_t rows;
    size_t key_bytes, rot_bytes, mask_bytes, exp_bytes;
    size_t total() const { return 2 * key_bytes + rot_bytes + mask_bytes + exp_bytes; }
};

static PrefillSpace prefill_space(int32_t num_seqs, int32_t num_heads, int32_t max_context_len)
{
    PrefillSpace s;
    s.rows = (static_cast<int64_t>(max_context_len > 0 ? max_context_len : 1) + kKvTile - 1) / kKvTile * kKvTile;
    const size_t all = static_cast<size_t>(s.rows) * num_seqs;
    s.key_bytes = all * num_heads * kNope * 2;
    s.rot_bytes = all * kRot * 2;
    s.mask_bytes = all / 8;
    s.exp_bytes = all / 32 * num_heads * 4;
    return s;
}

// Heads a CTA of the expansion takes.  Its rows are loaded once for all of
// them; a wave of CTAs costs its heads and about 1.5 more of start and end, so
// the number that makes waves x (heads + 1.5) least is taken.
static int32_t expand_heads(int64_t tiles, int32_t num_heads)
{
    int32_t best = 1;
    double least = 0.0;
    for (int32_t n = 1; n <= num_heads; ++n) {
        const int64_t ctas = tiles * ((num_heads + n - 1) / n);
        const double cost = static_cast<double>((ctas + sm_count() - 1) / sm_count()) * (n + 1.5);
        if (n == 1 || cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

template <typename T, int L>
static pa_status launch_prefill(LatentPrefillArgs& a, const void* query, const void* w_kv,
                                cudaStream_t stream)
{
    using E = ExpandShape<L>;
    using S = AttendShape;
    static std::atomic<uint64_t> expand_done{0}, attend_done{0};
    auto expand = latent_expand_kernel<T, L>;
    auto attend = latent_attend_kernel<T>;
    if (!ensure_smem_attr(expand, E::kSmem, expand_done) || !ensure_smem_attr(attend, S::kSmem, attend_done))
        return PA_ERR_CUDA;
    const uint64_t row_bytes = (L + kRot) * 2;
    const uint64_t kv_rows = static_cast<uint64_t>(a.rows);
    const uint64_t heads = static_cast<uint64_t>(a.num_heads);
    const uint64_t w_rows = heads * (kNope + kValue);
    const uint64_t q_bytes = (kNope + kRot) * 2;
    const uint64_t planes = static_cast<uint64_t>(a.num_seqs) * heads;
    CUtensorMap tm_cache, tm_w, tm_q, tm_k, tm_v, tm_r, tm_k_out, tm_v_out;
    if (!encode_rows_map(&tm_cache, a.cache, L + kRot, a.block_size, a.num_blocks, row_bytes,
                         row_bytes * a.block_size, a.block_size) ||
        !encode_rows_map(&tm_w, w_kv, L, w_rows, 1, L * 2, L * 2 * w_rows, 128) ||
        !encode_rows_map(&tm_q, query, kNope + kRot, a.num_tokens, heads, q_bytes * heads, q_bytes,
                         kQueryTile) ||
        !encode_rows_map(&tm_k, a.ws_k, kNope, kv_rows, planes, kNope * 2, kNope * 2 * kv_rows, kKvTile) ||
        !encode_rows_map(&tm_v, a.ws_v, kValue, kv_rows, planes, kValue * 2, kValue * 2 * kv_rows, kKvTile) ||
        !encode_rows_map(&tm_k_out, a.ws_k, kNope, kv_rows, planes, kNope * 2, kNope * 2 * kv_rows, 32, 32) ||
        !encode_rows_map(&tm_v_out, a.ws_v, kValue, kv_rows, planes, kValue * 2, kValue * 2 * kv_rows, 32, 32) ||
        !encode_rows_map(&tm_r, a.ws_rot, kRot, kv_rows, a.num_seqs, kRot * 2, kRot * 2 * kv_rows, kKvTile))
        return PA_ERR_CUDA;
    const int64_t tiles = a.rows / kKvTile;
    a.heads_per_cta = expand_heads(tiles * a.num_seqs, a.num_heads);
    pa_status st = launch_overlapped(
        expand,
        dim3((a.num_heads + a.heads_per_cta - 1) / a.heads_per_cta, static_cast<unsigned>(tiles), a.num_seqs),
        dim3(kExpandThreads), E::kSmem, stream, tm_cache, tm_w, tm_k_out,
        tm_v_out, a);
    if (st != PA_OK) return st;
    a.pairs = (a.max_query_len + 2 * kQueryTile - 1) / (2 * kQueryTile);
    const int64_t items = static_cast<int64_t>(a.pairs) * a.num_seqs;
    // (where all blocks run at once their order does not matter)
    a.sorted = a.num_seqs > 1 && items <= kSortItems && items * a.num_heads > sm_count();
    const dim3 grid = a.sorted ? dim3(a.num_heads, static_cast<unsigned>(items))
                               : dim3(a.num_heads, a.pairs, a.num_seqs);
    return launch_overlapped(attend, grid, dim3(kAttendThreads), S::kSmem, stream, tm_q, tm_k, tm_v, tm_r, a);
}

}  // namespace pa

extern "C" size_t pa_latent_prefill_workspace_size(int32_t num_seqs, int32_t num_heads,
                                                   int32_t latent_dim, int32_t block_size,
                                                   int32_t max_context_len)
{
    using namespace pa;
    if (bad_latent_shape(num_seqs, num_heads, latent_dim, block_size, max_context_len) ||
        !supported_latent(latent_dim, 64) || !supported_latent_block(block_size) ||
        num_heads > kMaxLatentHeads || num_seqs > 65535)
        return 0;
    return prefill_space(num_seqs, num_heads, max_context_len).total();
}

extern "C" pa_status pa_latent_prefill(
    void* out, const void* query, const void* cache, const void* w_kv, const int32_t* block_tables,
    const int32_t* query_starts, const int32_t* context_lens, int32_t num_seqs, int32_t num_tokens,
    int32_t num_heads, int32_t latent_dim, int32_t rope_dim, int32_t nope_dim, int32_t value_dim,
    int32_t block_size, int32_t max_blocks_per_seq, int64_t num_blocks, int32_t max_query_len,
    int32_t max_context_len, float scale, void* workspace, size_t workspace_bytes, pa_dtype dtype,
    int32_t* d_status, pa_stream_t stream)
{
    using namespace pa;
    if (bad_latent_shape(num_seqs, num_heads, latent_dim, block_size, max_context_len) || rope_dim <= 0 ||
        nope_dim <= 0 || value_dim <= 0 || num_tokens < 0 || max_query_len < 0 ||
        max_blocks_per_seq <= 0 || num_blocks <= 0 || !isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (!supported_dtype(dtype) || !supported_latent(latent_dim, rope_dim) || nope_dim != kNope ||
        value_dim != kValue || !supported_latent_block(block_size) || num_heads > kMaxLatentHeads ||
        num_seqs > 65535)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!out || !query || !cache || !w_kv || !block_tables || !query_starts || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(cache) || !aligned16(w_kv) ||
        !aligned4(block_tables) || !aligned4(query_starts) || !aligned4(context_lens) ||
        (d_status && !aligned4(d_status)))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa_latent_prefill_workspace_size(num_seqs, num_heads, latent_dim,
                                                         block_size, max_context_len);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)))
        return PA_ERR_INVALID_ARG;
    const PrefillSpace sp = prefill_space(num_seqs, num_heads, max_context_len);
    if (sp.rows > 65535LL * kKvTile || num_blocks > 0x7fffffff ||
        max_query_len > 65535LL * 2 * kQueryTile)
        return PA_ERR_UNSUPPORTED;
    LatentPrefillArgs a = {};
    a.out = out;
    a.cache = cache;
    a.block_tables = block_tables;
    a.query_starts = query_starts;
    a.context_lens = context_lens;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.ws_k = ws;
    a.ws_v = ws + sp.key_bytes;
    a.ws_rot = ws + 2 * sp.key_bytes;
    a.ws_mask = reinterpret_cast<uint32_t*>(ws + 2 * sp.key_bytes + sp.rot_bytes);
    a.ws_exp = reinterpret_cast<float*>(ws + 2 * sp.key_bytes + sp.rot_bytes + sp.mask_bytes);
    a.rows = static_cast<int32_t>(sp.rows);
    a.num_seqs = num_seqs;
    a.num_tokens = num_tokens;
    a.num_heads = num_heads;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.max_query_len = max_query_len;
    a.max_context_len = max_context_len;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.d_status = d_status;
    if (dtype == PA_DTYPE_F16)
        return latent_dim == 512 ? launch_prefill<__half, 512>(a, query, w_kv, stream)
                                 : launch_prefill<__half, 256>(a, query, w_kv, stream);
    return latent_dim == 512 ? launch_prefill<__nv_bfloat16, 512>(a, query, w_kv, stream)
                             : launch_prefill<__nv_bfloat16, 256>(a, query, w_kv, stream);
}
