// ra_head_rows.cuh -- one head's row of d channels (d = 64 or 128) spread over
// d / 8 lanes, eight channels (16 bytes of bf16) a lane, and what the kernels
// around the attention do with it: the RMS norm of the row and the rotation of
// its channel pairs by the token's position in time, height and width.
//
//   norm    u = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)   (fp32; w may be absent: u = x)
//   rotate  channel pair (2 i, 2 i + 1): (u0 c - u1 s, u0 s + u1 c) with the cosine
//           and sine of pair i, read from the table of the axis that pair i belongs
//           to: the first t_pairs pairs follow the frame, the next h_pairs the row
//           in the frame, the next w_pairs the column; the rest are not rotated.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ra_bounds.cuh"

namespace ra {

// Position tables: fp32 (cos, sin) pairs, [len][pairs][2] for each axis.
struct RopeArgs {
    const float2* t;  // null: no rotation
    const float2* h;
    const float2* w;
    int t_pairs, h_pairs, w_pairs;
    int grid_h, grid_w;  // token i of a call: frame first + i / (grid_h * grid_w), row-major within it
    int first;           // frame of the call's first token
    int frames;          // rows of t
    int* err;            // debug build: see ra_bounds.cuh
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The lane's eight norm weights (bf16 or fp32 in memory).
__device__ __forceinline__ void load_weight(const void* weight, int fp32, int lane_in_row, float (&w)[8])
{
    if (fp32) {
        const float4* p = reinterpret_cast<const float4*>(weight) + 2 * lane_in_row;
        const float4 a = p[0], b = p[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
        unpack_bf16x8(reinterpret_cast<const uint4*>(weight)[lane_in_row], w);
    }
}

// Cosines and sines of the lane's four channel pairs at token `i`.
__device__ __forceinline__ void load_rope(const RopeArgs& a, int i, int lane_in_row, float2 (&cs)[4])
{
    const int s = a.grid_h * a.grid_w;
    const int f = i / s, pos = i - f * s;
    const int row = pos / a.grid_w, col = pos - row * a.grid_w;
    const float2* t = a.t + static_cast<size_t>(a.first + f) * a.t_pairs;
    const float2* h = a.h + static_cast<size_t>(row) * a.h_pairs - a.t_pairs;
    const float2* w = a.w + static_cast<size_t>(col) * a.w_pairs - (a.t_pairs + a.h_pairs);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = lane_in_row * 4 + j;
        const float2* at = p < a.t_pairs ? t : (p < a.t_pairs + a.h_pairs ? h : w);
        if (!inside(a.err, p < a.t_pairs ? a.first + f : p < a.t_pairs + a.h_pairs ? row : col, 1,
                    p < a.t_pairs ? a.frames : p < a.t_pairs + a.h_pairs ? a.grid_h : a.grid_w, SITE_I_ROPE)) {
            cs[j] = make_float2(1.f, 0.f);
            continue;
        }
        cs[j] = p < a.t_pairs + a.h_pairs + a.w_pairs ? __ldg(at + p) : make_float2(1.f, 0.f);
    }
}

// Sum over the LPR lanes that hold one row (every lane gets it).
template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// How many of the lane's four pairs are turned.
__device__ __forceinline__ int turned_pairs(const RopeArgs& a, int lane_in_row)
{
    return a.t_pairs + a.h_pairs + a.w_pairs - 4 * lane_in_row;
}

// Pairs that are not turned (their angles are 1, 0) are left alone, not multiplied
// through: an infinity or a NaN would reach the channel beside it.
__device__ __forceinline__ void keep_unturned(const float (&before)[8], int turned, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j >= turned) {
            x[2 * j] = before[2 * j];
            x[2 * j + 1] = before[2 * j + 1];
        }
}

__device__ __forceinline__ void rotate(const float2 (&cs)[4], float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = a * cs[j].x - b * cs[j].y;
        x[2 * j + 1] = a * cs[j].y + b * cs[j].x;
    }
}

// The transpose of rotate: turns back by the same angles.
__device__ __forceinline__ void rotate_back(const float2 (&cs)[4], float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = a * cs[j].x + b * cs[j].y;
        x[2 * j + 1] = b * cs[j].x - a * cs[j].y;
    }
}

// x -> x * r * w over the row; every lane of the warp takes part.
template <int D>
__device__ __forceinline__ void rms_norm(float (&x)[8], const float (&w)[8], float eps)
{
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        ss = fmaf(x[j], x[j], ss);
    const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] *= r * w[j];
}

}  // namespace ra
