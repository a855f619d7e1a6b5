// latent_prefill.cu -- prompt attention over the paged latent pool with keys
// and values expanded for each head.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_host.h"

namespace pa {

constexpr int kRowWarps4 = 4;
constexpr int kNope = 128;
constexpr int kValue = 128;

struct LatentArgs {
    void* out;
    const void* query;
    const void* cache;
    const void* w_kv;
    const int32_t* block_tables;
    const int32_t* query_starts;
    const int32_t* context_lens;
    int32_t num_seqs, num_tokens, num_heads, block_size, max_blocks_per_seq;
    int64_t num_blocks;
    int32_t max_query_len, max_context_len;
    float scale_log2;
    int32_t* d_status;
};

__device__ __forceinline__ float lat_to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float lat_to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void lat_store(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void lat_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ bool good_context(const LatentArgs& a, int32_t ctx)
{
    return ctx >= 0 && ctx <= a.max_context_len &&
           static_cast<int64_t>(ctx) <= static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
}

// Attention of one query (fp32 [L + 64] in shared memory) over the first
// `seen` rows of sequence s, by the CTA's four warps, a token a warp at a
// time; the normalised sum of the latent parts goes to `result` [L].
template <typename T, int L>
__device__ void attend_rows(const LatentArgs& a, int s, int32_t seen, const float* q, float* result,
                            float* merge)
{
    constexpr int W = L + 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f, acc[L / 32];
#pragma unroll
    for (int i = 0; i < L / 32; ++i) acc[i] = 0.f;
    for (int32_t t = warp; t < seen; t += kRowWarps4) {
        const int32_t page = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + t / a.block_size];
        if (page < 0 || page >= a.num_blocks) {
            if (lane == 0) status_or(a.d_status, PA_STATUS_BAD_BLOCK);
            continue;
        }
        const T* row = static_cast<const T*>(a.cache) +
                       (static_cast<int64_t>(page) * a.block_size + t % a.block_size) * W;
        float x[W / 32];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < W / 32; ++i) {
            x[i] = lat_to_float(row[i * 32 + lane]);
            dot = fmaf(x[i], q[i * 32 + lane], dot);
        }
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) dot += __shfl_xor_sync(kFullMask, dot, k);
        dot *= a.scale_log2;
        const float mn = fmaxf(m, dot);
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float p = exp2f(dot - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < L / 32; ++i) acc[i] = acc[i] * f + p * x[i];
    }
    float* mine = merge + warp * (L + 2);
#pragma unroll
    for (int i = 0; i < L / 32; ++i) mine[i * 32 + lane] = acc[i];
    if (lane == 0) {
        mine[L] = m;
        mine[L + 1] = l;
    }
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
    for (int w = 0; w < kRowWarps4; ++w) M = fmaxf(M, merge[w * (L + 2) + L]);
    const float msub = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kRowWarps4; ++w)
        sum += merge[w * (L + 2) + L + 1] * exp2f(merge[w * (L + 2) + L] - msub);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    for (int i = threadIdx.x; i < L; i += blockDim.x) {
        float o = 0.f;
        for (int w = 0; w < kRowWarps4; ++w)
            o += merge[w * (L + 2) + i] * exp2f(merge[w * (L + 2) + L] - msub);
        result[i] = o * inv;
    }
    __syncthreads();
}

template <typename T, int L>
__global__ void __launch_bounds__(128) latent_prefill_simple_kernel(const LatentArgs a)
{
    __shared__ float qin[kNope], q[L + 64], result[L], merge[kRowWarps4 * (L + 2)];
    grid_dependency_wait();
    const int h = blockIdx.x, s = blockIdx.z, i = blockIdx.y;
    const int32_t first = a.query_starts[s], last = a.query_starts[s + 1];
    if (first < 0 || last < first || last > a.num_tokens || last - first > a.max_query_len) {
        if (threadIdx.x == 0) status_or(a.d_status, PA_STATUS_BAD_CONTEXT);
        return;
    }
    if (i >= last - first) return;
    int32_t ctx = a.context_lens[s];
    const bool ok = good_context(a, ctx) && ctx >= last - first;
    if (!ok && threadIdx.x == 0) status_or(a.d_status, PA_STATUS_BAD_CONTEXT);
    const int32_t seen = ok ? ctx - (last - first) + i + 1 : 0;
    const int64_t row = static_cast<int64_t>(first + i) * a.num_heads + h;
    const T* w = static_cast<const T*>(a.w_kv) + static_cast<int64_t>(h) * (kNope + kValue) * L;
    const T* qr = static_cast<const T*>(a.query) + row * (kNope + 64);
    for (int e = threadIdx.x; e < kNope; e += blockDim.x) qin[e] = lat_to_float(qr[e]);
    if (threadIdx.x < 64) q[L + threadIdx.x] = lat_to_float(qr[kNope + threadIdx.x]);
    __syncthreads();
    for (int c = threadIdx.x; c < L; c += blockDim.x) {
        float v = 0.f;
        for (int e = 0; e < kNope; ++e) v = fmaf(qin[e], lat_to_float(w[e * L + c]), v);
        q[c] = v;
    }
    __syncthreads();
    attend_rows<T, L>(a, s, seen, q, result, merge);
    for (int e = threadIdx.x; e < kValue; e += blockDim.x) {
        float v = 0.f;
        for (int c = 0; c < L; ++c) v = fmaf(result[c], lat_to_float(w[(kNope + e) * L + c]), v);
        lat_store(static_cast<T*>(a.out) + row * kValue + e, v);
    }
}

}  // namespace pa

extern "C" size_t pa_latent_prefill_workspace_size(int32_t num_seqs, int32_t num_heads,
                                                   int32_t latent_dim, int32_t block_size,
                                                   int32_t max_context_len)
{
    using namespace pa;
    if (bad_latent_shape(num_seqs, num_heads, latent_dim, block_size, max_context_len) ||
        !supported_latent(latent_dim, 64) || !supported_latent_block(block_size) ||
        num_heads > kMaxLatentHeads)
        return 0;
    const size_t rows = (static_cast<size_t>(max_context_len) + 127) / 128 * 128 * num_seqs;
    return rows * (static_cast<size_t>(num_heads) * (kNope + kValue) + 64) * 2;
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
    if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) return PA_OK;
    LatentArgs a = {};
    a.out = out;
    a.query = query;
    a.cache = cache;
    a.w_kv = w_kv;
    a.block_tables = block_tables;
    a.query_starts = query_starts;
    a.context_lens = context_lens;
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
    auto kernel = dtype == PA_DTYPE_F16
                      ? (latent_dim == 512 ? latent_prefill_simple_kernel<__half, 512>
                                           : latent_prefill_simple_kernel<__half, 256>)
                      : (latent_dim == 512 ? latent_prefill_simple_kernel<__nv_bfloat16, 512>
                                           : latent_prefill_simple_kernel<__nv_bfloat16, 256>);
    return launch_overlapped(kernel, dim3(num_heads, max_query_len, num_seqs), dim3(128), 0, stream, a);
}
