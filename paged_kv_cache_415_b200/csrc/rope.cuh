// rope.cuh -- the position rotation and the norm of a head's row, for the
// kernels that append rotated rows to a cache (sm_100a).
//
// A row of D elements is held by D / 8 neighbouring lanes, 8 consecutive
// elements (one 16-byte vector) each.  Its first `rot` elements are rotated
// in rot / 2 pairs by the angles of the token's position,
//   (a, b) -> (a cos - b sin, b cos + a sin),
// the pair of angle i being elements (i, i + rot / 2), or (2i, 2i + 1) when
// interleaved.  Angles come from a table of fp32 cosines and sines (the
// caller's: angles of far positions need more than 32 bits to form), one row
// [cos 0 .. cos rot/2 - 1, sin 0 .. sin rot/2 - 1] a position.
//
// Everything is computed in fp32; a row is rounded once, when it is stored.
#pragma once

#include <stdint.h>

#include "pa_common.cuh"

namespace pa {

// The angles a lane needs: of its 8 elements, or (interleaved) of its 4
// pairs, in entries 0 .. 3.
struct Angles {
    float c[8], s[8];
};

// `e0`: the lane's first element; the caller checks e0 < rot.  rot is a
// multiple of 16, so a lane's elements lie in one half of the rotated part
// and their angles are whole float4s of the table row.
__device__ __forceinline__ void load_angles(Angles& a, const float* __restrict__ table_row,
                                            int e0, int rot, bool interleaved)
{
    const int half = rot >> 1;
    const int i0 = interleaved ? e0 >> 1 : (e0 < half ? e0 : e0 - half);
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(table_row + i0));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(table_row + half + i0));
    a.c[0] = c0.x; a.c[1] = c0.y; a.c[2] = c0.z; a.c[3] = c0.w;
    a.s[0] = s0.x; a.s[1] = s0.y; a.s[2] = s0.z; a.s[3] = s0.w;
    if (!interleaved) {
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(table_row + i0 + 4));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(table_row + half + i0 + 4));
        a.c[4] = c1.x; a.c[5] = c1.y; a.c[6] = c1.z; a.c[7] = c1.w;
        a.s[4] = s1.x; a.s[5] = s1.y; a.s[6] = s1.z; a.s[7] = s1.w;
    }
}

// Rotates the lane's 8 elements in place.  Every lane of the warp calls it
// (the half-split pairs exchange elements by shuffle); lanes with
// e0 >= rot keep theirs.
__device__ __forceinline__ void rotate8(float (&f)[8], const Angles& a, int e0, int rot,
                                        bool interleaved)
{
    if (interleaved) {
        if (e0 < rot) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float x = f[2 * p], y = f[2 * p + 1];
                f[2 * p] = x * a.c[p] - y * a.s[p];
                f[2 * p + 1] = y * a.c[p] + x * a.s[p];
            }
        }
        return;
    }
    const int half = rot >> 1;
    const int lane = threadIdx.x & 31;
    const bool low = e0 < half;
    const int partner = e0 < rot ? (low ? lane + (half >> 3) : lane - (half >> 3)) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(kFullMask, f[i], partner);
        if (e0 < rot) f[i] = f[i] * a.c[i] + (low ? -y : y) * a.s[i];
    }
}

// Sum over the LANES neighbouring lanes that hold a row (a power of two).
template <int LANES>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int k = LANES / 2; k >= 1; k >>= 1) v += __shfl_xor_sync(kFullMask, v, k);
    return v;
}

template <int LANES>
__device__ __forceinline__ float row_max(float v)
{
#pragma unroll
    for (int k = LANES / 2; k >= 1; k >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, k));
    return v;
}

// 16 bytes that another thread of this grid may overwrite after they are
// read (an in-place rotation): a plain load, not the read-only path.
__device__ __forceinline__ uint4 ld_stream_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

}  // namespace pa
