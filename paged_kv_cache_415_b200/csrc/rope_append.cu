// rope_append.cu -- appends to a paged cache that normalise and rotate on
// the way:
//   rope_append_kernel    queries and keys of each head normalised (optional)
//                         and rotated by position; queries to query_out, keys
//                         and values to their slots of the K / V pools
//                         (16-bit, or one-byte codes)
//   latent_append_kernel  the latent vector of each token normalised
//                         (optional) and its key part rotated, both to their
//                         slot of the latent pool; the queries' rotated part
//                         to query_out
// Each reads its inputs once and writes its outputs once: both are bound by
// memory for prompts and by launch and load latency for decode steps.
// Measured, a call: 8192 tokens, 32 + 32 heads of 128 in 81.6 us (5.0 TB/s; the
// kernel alone 75.5), 8191 latent rows of 576 with 32 heads in 21.1 us (4.2 TB/s;
// 16.5), 64 tokens of 32 + 8 heads in 2.05 us from a graph.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "pa.h"
#include "pa_codes.cuh"
#include "pa_common.cuh"
#include "pa_host.h"
#include "rope.cuh"

namespace pa {

constexpr int kRopeThreads = 128;


struct RopeArgs {
    void* query_out;
    const void* query;
    const void* key;
    const void* value;
    void* k_cache;
    void* v_cache;
    float* k_scales;                  // one scale a row of one-byte pools, or null
    float* v_scales;
    const int64_t* slot_mapping;
    const int64_t* positions;
    const float* cos_sin;
    const void* q_weight;             // norm weights [D], or null: no norm
    const void* k_weight;
    float eps;
    uint32_t num_tokens, per_token;   // lane groups a token
    int32_t num_q_heads, num_kv_heads, rot_dim;
    int64_t max_position;
    int32_t interleaved;
    int64_t query_out_stride, query_stride, key_stride, value_stride;   // elements a token
    int32_t block_size;
    int64_t num_slots;
    float k_inv, v_inv;
    int32_t* d_status;
};

struct PlainRows {};                  // pools of the input's own 16-bit type

// The rows of all tokens, Hq + 2 Hkv each, are shared out over lane groups of
// D / 8 lanes: `per_token` groups a token, group g taking its rows g, g +
// per_token, ... (ROWS of them, all loads issued first, the angles loaded once).
// Neighbouring groups take neighbouring rows, and a warp may hold groups of
// several tokens, so no lane is idle whatever the head counts.
template <typename T, typename Store, int D, int ROWS>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a)
{
    constexpr int LANES = D / 8;
    grid_dependency_wait();
    allow_dependents();
    const int hq = a.num_q_heads, hkv = a.num_kv_heads;
    const int rows = hq + 2 * hkv;
    const int j = threadIdx.x % LANES;            // place in the row
    const int e0 = j * 8;
    const uint32_t group = (blockIdx.x * kRopeThreads + threadIdx.x) / LANES;
    const uint32_t token = group / a.per_token;
    const int g = static_cast<int>(group - token * a.per_token);
    const bool inside = token < a.num_tokens;
    const int64_t t = inside ? token : 0;
    const int64_t pos = a.positions[t];
    const int64_t slot = a.slot_mapping[t];
    uint4 x[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = inside ? g + i * static_cast<int>(a.per_token) : rows;
        x[i] = make_uint4(0, 0, 0, 0);
        if (r < hq)
            x[i] = ld_stream_v4(static_cast<const T*>(a.query) + t * a.query_stride +
                                static_cast<int64_t>(r) * D + e0);
        else if (r < hq + hkv)
            x[i] = ld_stream_v4(static_cast<const T*>(a.key) + t * a.key_stride +
                                static_cast<int64_t>(r - hq) * D + e0);
        else if (r < rows)
            x[i] = ld_stream_v4(static_cast<const T*>(a.value) + t * a.value_stride +
                                static_cast<int64_t>(r - hq - hkv) * D + e0);
    }
    // nothing of a padding token (pos < 0) or one past the table is written
    const bool live = inside && pos >= 0 && pos < a.max_position;
    const bool cached = live && slot >= 0 && slot < a.num_slots;
    if (inside && g == 0 && j == 0) {
        if (pos >= a.max_position) status_or(a.d_status, PA_STATUS_BAD_POSITION);
        if (live && slot >= a.num_slots) status_or(a.d_status, PA_STATUS_BAD_SLOT);
    }
    Angles ang;
    if (live && e0 < a.rot_dim)
        load_angles(ang, a.cos_sin + pos * a.rot_dim, e0, a.rot_dim, a.interleaved != 0);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = g + i * static_cast<int>(a.per_token);
        const bool is_q = r < hq;
        const bool is_k = !is_q && r < hq + hkv;
        float f[8];
        unpack8<T>(x[i], f);
        if (__any_sync(kFullMask, is_q || is_k)) {
            if (a.q_weight != nullptr || a.k_weight != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
                ss = row_sum<LANES>(ss);
                const T* w = static_cast<const T*>(is_q ? a.q_weight : is_k ? a.k_weight : nullptr);
                if (w != nullptr) {
                    const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
                    float wf[8];
                    unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w + e0)), wf);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = f[e] * rs * wf[e];
                }
            }
            float g8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) g8[e] = f[e];
            rotate8(g8, ang, e0, a.rot_dim, a.interleaved != 0);
            if (is_q || is_k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = g8[e];
            }
        }
        if (is_q && live)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.query_out) + t * a.query_out_stride +
                                      static_cast<int64_t>(r) * D + e0) = pack8<T>(f);
        const bool store = !is_q && r < rows && cached;
        const int h = is_k ? r - hq : r - hq - hkv;
        const int64_t dst = (slot * hkv + h) * D + e0;      // used only where `store`
        if constexpr (std::is_same<Store, PlainRows>::value) {
            if (store)
                *reinterpret_cast<uint4*>(static_cast<T*>(is_k ? a.k_cache : a.v_cache) + dst) =
                    pack8<T>(f);
        } else {
            float inv = is_k ? a.k_inv : a.v_inv;
            if (a.k_scales != nullptr) {          // a scale for this row, from its own values
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
                m = row_max<LANES>(m);
                const float s = m / Store::kMax;
                const bool tiny = !(s >= FLT_MIN);
                inv = tiny ? 0.f : 1.0f / s;
                if (tiny) {                       // zero codes, whatever the values are
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = 0.f;
                }
                if (store && j == 0)
                    (is_k ? a.k_scales : a.v_scales)[((slot / a.block_size) * hkv + h) *
                                                         a.block_size + slot % a.block_size] =
                        tiny ? 0.f : s;
            }
            if (store) {
                uint32_t c[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = Store::encode2(f[2 * e] * inv, f[2 * e + 1] * inv);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) + dst) =
                    make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
            }
        }
    }
}

// Rows a lane group takes: as many (1, 2 or 4) as leave enough warps to fill
// the GPU, kFillWarps.  (8192 tokens, 32 + 32 heads: 131 us with 1, 87 with 2,
// 76 with 4, more with 6 or 8; where the warps are few, more rows a group only
// lengthen its chain.)
constexpr int64_t kFillWarps = 148 * 32;

template <typename T, typename Store, int D, int ROWS>
static pa_status launch_rope_rows(RopeArgs& a, pa_stream_t stream)
{
    const int64_t rows = static_cast<int64_t>(a.num_q_heads) + 2 * a.num_kv_heads;
    const int64_t per_token = (rows + ROWS - 1) / ROWS;
    const int64_t groups = per_token * a.num_tokens;
    const int64_t ctas = (groups * (D / 8) + kRopeThreads - 1) / kRopeThreads;
    // (thread numbers stay below 2^32)
    if (ctas > 0xffffffffLL / kRopeThreads) return PA_ERR_UNSUPPORTED;
    a.per_token = static_cast<uint32_t>(per_token);
    return launch_overlapped(rope_append_kernel<T, Store, D, ROWS>, dim3(static_cast<unsigned>(ctas)),
                             dim3(kRopeThreads), 0, stream, a);
}

template <typename T, typename Store, int D>
static pa_status launch_rope(RopeArgs& a, pa_stream_t stream)
{
    const int64_t rows = static_cast<int64_t>(a.num_q_heads) + 2 * a.num_kv_heads;
    const int64_t warps = a.num_tokens * rows * (D / 8) / 32;
    if (warps >= 4 * kFillWarps) return launch_rope_rows<T, Store, D, 4>(a, stream);
    if (warps >= 2 * kFillWarps) return launch_rope_rows<T, Store, D, 2>(a, stream);
    return launch_rope_rows<T, Store, D, 1>(a, stream);
}

template <typename T, typename Store>
static pa_status launch_rope_dim(RopeArgs& a, int32_t head_dim, pa_stream_t stream)
{
    return head_dim == 128 ? launch_rope<T, Store, 128>(a, stream)
                           : launch_rope<T, Store, 64>(a, stream);
}

template <typename T>
static pa_status launch_rope_store(RopeArgs& a, pa_dtype pool, int32_t head_dim, pa_stream_t stream)
{
    if (pool == PA_DTYPE_FP8_E4M3)
        return launch_rope_dim<T, E4m3Codes>(a, head_dim, stream);
    if (pool == PA_DTYPE_INT8) return launch_rope_dim<T, Int8Codes>(a, head_dim, stream);
    return launch_rope_dim<T, PlainRows>(a, head_dim, stream);
}

// A stride in elements between `count` rows: whole 16-byte vectors, at least
// `need`.  That of a single row is never used and may be anything.
static bool good_stride(int64_t stride, int64_t need, int32_t count)
{
    return count <= 1 || (stride % 8 == 0 && stride >= need);
}

// ---------------------------------------------------------------------------
// Latent pool
// ---------------------------------------------------------------------------

constexpr int kLatentRope = 64;       // rotated key elements of a latent row

struct LatentAppendArgs {
    void* query_out;
    const void* query_rope;
    const void* latent;
    void* cache;
    const int64_t* slot_mapping;
    const int64_t* positions;
    const float* cos_sin;
    const void* weight;
    float eps;
    uint32_t num_tokens, units;       // units a token
    int32_t num_heads;
    int64_t max_position;
    int32_t interleaved;
    int64_t query_out_stride, query_out_head_stride, query_stride, query_head_stride;
    int64_t latent_stride;
    int64_t num_slots;
    int32_t* d_status;
};

// A warp a unit, `units` units a token: unit 0 takes its latent row, L
// elements over 32 lanes (L / 256 vectors each) and the 64 rotated ones over
// the first 8 lanes; every further one rotates 4 * STEPS heads of the query, 8
// lanes a head, all loads first.
template <typename T, int L, int STEPS>
__global__ void __launch_bounds__(kRopeThreads) latent_append_kernel(const LatentAppendArgs a)
{
    constexpr int VECS = L / 256;
    grid_dependency_wait();
    allow_dependents();
    const uint32_t item = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const uint32_t token = item / a.units;
    if (token >= a.num_tokens) return;
    const int unit = static_cast<int>(item - token * a.units);
    const int64_t t = token;
    const int lane = threadIdx.x & 31;
    const int e0 = (lane & 7) * 8;
    const int64_t pos = a.positions[t];
    if (unit == 0) {
        const T* row = static_cast<const T*>(a.latent) + t * a.latent_stride;
        const int64_t slot = a.slot_mapping[t];
        uint4 x[VECS], xr = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < VECS; ++v) x[v] = ld_stream_v4(row + v * 256 + lane * 8);
        if (lane < 8) xr = ld_stream_v4(row + L + e0);
        if (pos < 0) return;
        if (pos >= a.max_position) {
            if (lane == 0) status_or(a.d_status, PA_STATUS_BAD_POSITION);
            return;
        }
        if (slot < 0) return;
        if (slot >= a.num_slots) {
            if (lane == 0) status_or(a.d_status, PA_STATUS_BAD_SLOT);
            return;
        }
        Angles ang;
        load_angles(ang, a.cos_sin + pos * kLatentRope, e0, kLatentRope, a.interleaved != 0);
        T* dst = static_cast<T*>(a.cache) + slot * (L + kLatentRope);
        if (a.weight != nullptr) {
            float f[VECS][8];
            float ss = 0.f;
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                unpack8<T>(x[v], f[v]);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[v][e], f[v][e], ss);
            }
            const float rs = rsqrtf(row_sum<32>(ss) * (1.0f / L) + a.eps);
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                float wf[8];
                unpack8<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.weight) +
                                                                v * 256 + lane * 8)), wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[v][e] = f[v][e] * rs * wf[e];
                x[v] = pack8<T>(f[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < VECS; ++v)
            *reinterpret_cast<uint4*>(dst + v * 256 + lane * 8) = x[v];
        float r[8];
        unpack8<T>(xr, r);
        rotate8(r, ang, e0, kLatentRope, a.interleaved != 0);
        if (lane < 8) *reinterpret_cast<uint4*>(dst + L + e0) = pack8<T>(r);
        return;
    }
    const int h0 = (unit - 1) * 4 * STEPS + (lane >> 3);
    uint4 x[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int h = h0 + 4 * i;
        x[i] = make_uint4(0, 0, 0, 0);
        if (h < a.num_heads)
            x[i] = ld_stream_v4(static_cast<const T*>(a.query_rope) + t * a.query_stride +
                                h * a.query_head_stride + e0);
    }
    if (pos < 0 || pos >= a.max_position) return;
    Angles ang;
    load_angles(ang, a.cos_sin + pos * kLatentRope, e0, kLatentRope, a.interleaved != 0);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int h = h0 + 4 * i;
        float f[8];
        unpack8<T>(x[i], f);
        rotate8(f, ang, e0, kLatentRope, a.interleaved != 0);
        if (h < a.num_heads)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.query_out) + t * a.query_out_stride +
                                      h * a.query_out_head_stride + e0) = pack8<T>(f);
    }
}

template <typename T, int L, int STEPS>
static pa_status launch_latent_append(LatentAppendArgs& a, pa_stream_t stream)
{
    constexpr int kWarpsPerCta = kRopeThreads / 32;
    const int64_t units = 1 + (static_cast<int64_t>(a.num_heads) + 4 * STEPS - 1) / (4 * STEPS);
    const int64_t items = units * a.num_tokens;
    if (items > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    a.units = static_cast<uint32_t>(units);
    return launch_overlapped(latent_append_kernel<T, L, STEPS>,
                             dim3(static_cast<unsigned>((items + kWarpsPerCta - 1) / kWarpsPerCta)),
                             dim3(kRopeThreads), 0, stream, a);
}

template <typename T>
static pa_status dispatch_latent_append(LatentAppendArgs& a, int32_t latent_dim, pa_stream_t stream)
{
    // several heads a lane group where the grid fills the GPU without them
    const bool many = static_cast<int64_t>(a.num_tokens) * (1 + a.num_heads / 4) >= 4 * kFillWarps;
    if (latent_dim == 512)
        return many ? launch_latent_append<T, 512, 4>(a, stream) : launch_latent_append<T, 512, 1>(a, stream);
    return many ? launch_latent_append<T, 256, 4>(a, stream) : launch_latent_append<T, 256, 1>(a, stream);
}

}  // namespace pa

extern "C" pa_status pa_rope_append(
    void* query_out, const void* query, const void* key, const void* value, void* k_cache,
    void* v_cache, float* k_scales, float* v_scales, const int64_t* slot_mapping,
    const int64_t* positions, const float* cos_sin, const void* q_weight, const void* k_weight,
    float eps, int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t rot_dim, int64_t max_position, int32_t interleaved, int64_t query_out_stride,
    int64_t query_stride, int64_t key_stride, int64_t value_stride, int32_t block_size,
    int64_t num_blocks, pa_dtype dtype, pa_dtype pool_dtype, float k_scale, float v_scale,
    int32_t* d_status, pa_stream_t stream)
{
    using namespace pa;
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || rot_dim < 0 || max_position <= 0)
        return PA_ERR_INVALID_ARG;
    if (!supported_dtype(dtype) || !supported_head_dim(head_dim) || !supported_block_size(block_size))
        return PA_ERR_UNSUPPORTED;
    const bool codes = code_dtype(pool_dtype);
    if (!codes && pool_dtype != dtype) return PA_ERR_UNSUPPORTED;
    if (rot_dim > head_dim) return PA_ERR_INVALID_ARG;
    if (rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !isfinite(eps)) return PA_ERR_INVALID_ARG;
    const bool row_scaled = k_scales != nullptr || v_scales != nullptr;
    if (row_scaled && (!codes || !k_scales || !v_scales || !aligned16(k_scales) ||
                       !aligned16(v_scales)))
        return PA_ERR_INVALID_ARG;
    if (codes && !row_scaled &&
        (!(k_scale > 0.f) || !(v_scale > 0.f) || !isfinite(k_scale) || !isfinite(v_scale)))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!query_out || !query || !key || !value || !k_cache || !v_cache || !slot_mapping ||
        !positions || (rot_dim > 0 && !cos_sin))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query_out) || !aligned16(query) || !aligned16(key) || !aligned16(value) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !aligned8(slot_mapping) ||
        !aligned8(positions) || (cos_sin && !aligned16(cos_sin)) ||
        (q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) ||
        (d_status && !aligned4(d_status)))
        return PA_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!good_stride(query_out_stride, q_row, num_tokens) ||
        !good_stride(query_stride, q_row, num_tokens) ||
        !good_stride(key_stride, kv_row, num_tokens) ||
        !good_stride(value_stride, kv_row, num_tokens))
        return PA_ERR_INVALID_ARG;
    RopeArgs a;
    a.query_out = query_out;
    a.query = query;
    a.key = key;
    a.value = value;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.num_tokens = static_cast<uint32_t>(num_tokens);
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.rot_dim = rot_dim;
    a.max_position = max_position;
    a.interleaved = interleaved;
    a.query_out_stride = query_out_stride;
    a.query_stride = query_stride;
    a.key_stride = key_stride;
    a.value_stride = value_stride;
    a.block_size = block_size;
    a.num_slots = num_blocks * block_size;
    a.k_inv = codes && !row_scaled ? 1.0f / k_scale : 1.f;
    a.v_inv = codes && !row_scaled ? 1.0f / v_scale : 1.f;
    a.d_status = d_status;
    return dtype == PA_DTYPE_F16
               ? launch_rope_store<__half>(a, pool_dtype, head_dim, stream)
               : launch_rope_store<__nv_bfloat16>(a, pool_dtype, head_dim, stream);
}

extern "C" pa_status pa_latent_append(
    void* query_out, const void* query_rope, const void* latent, void* cache,
    const int64_t* slot_mapping, const int64_t* positions, const float* cos_sin,
    const void* weight, float eps, int32_t num_tokens, int32_t num_heads, int32_t latent_dim,
    int32_t rope_dim, int64_t max_position, int32_t interleaved, int64_t query_out_stride,
    int64_t query_out_head_stride, int64_t query_stride, int64_t query_head_stride,
    int64_t latent_stride, int32_t block_size, int64_t num_blocks, pa_dtype dtype,
    int32_t* d_status, pa_stream_t stream)
{
    using namespace pa;
    if (num_tokens < 0 || num_heads < 0 || latent_dim <= 0 || rope_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || max_position <= 0)
        return PA_ERR_INVALID_ARG;
    if (!supported_dtype(dtype) || !supported_latent(latent_dim, rope_dim) ||
        !supported_latent_block(block_size))
        return PA_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !isfinite(eps)) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!latent || !cache || !slot_mapping || !positions || !cos_sin ||
        (num_heads > 0 && (!query_out || !query_rope)))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(query_out) || !aligned16(query_rope) || !aligned16(latent) ||
        !aligned16(cache) || !aligned8(slot_mapping) || !aligned8(positions) ||
        !aligned16(cos_sin) || (weight && !aligned16(weight)) || (d_status && !aligned4(d_status)))
        return PA_ERR_INVALID_ARG;
    if (!good_stride(latent_stride, latent_dim + rope_dim, num_tokens)) return PA_ERR_INVALID_ARG;
    if (num_heads > 0) {
        // the rows of different heads and tokens must not overlap
        const int64_t out_row = (num_heads - 1) * query_out_head_stride + rope_dim;
        const int64_t in_row = (num_heads - 1) * query_head_stride + rope_dim;
        if (!good_stride(query_out_head_stride, rope_dim, num_heads) ||
            !good_stride(query_head_stride, rope_dim, num_heads) ||
            !good_stride(query_out_stride, out_row, num_tokens) ||
            !good_stride(query_stride, in_row, num_tokens))
            return PA_ERR_INVALID_ARG;
    }
    LatentAppendArgs a;
    a.query_out = query_out;
    a.query_rope = query_rope;
    a.latent = latent;
    a.cache = cache;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.weight = weight;
    a.eps = eps;
    a.num_tokens = static_cast<uint32_t>(num_tokens);
    a.num_heads = num_heads;
    a.max_position = max_position;
    a.interleaved = interleaved;
    a.query_out_stride = query_out_stride;
    a.query_out_head_stride = query_out_head_stride;
    a.query_stride = query_stride;
    a.query_head_stride = query_head_stride;
    a.latent_stride = latent_stride;
    a.num_slots = num_blocks * block_size;
    a.d_status = d_status;
    return dtype == PA_DTYPE_F16 ? dispatch_latent_append<__half>(a, latent_dim, stream)
                                 : dispatch_latent_append<__nv_bfloat16>(a, latent_dim, stream);
}
