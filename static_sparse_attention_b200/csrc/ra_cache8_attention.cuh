// ra_cache8_attention.cuh -- what the kernels of attention over the 8-bit ring
// share: their arguments and where a key's scale lies.
#pragma once
#include <cuda_runtime.h>

#include "ra_bounds.cuh"
#include "ra_cache8.cuh"
#include "ra_internal.h"

namespace ra {

constexpr float LN2 = 0.69314718055994530942f;

struct AttnParams {
    const __nv_bfloat16* Q;  // [B, H, nq, d]
    const uint8_t* k8;       // [B, H, W * s, d]
    const uint8_t* v8;
    const float* k_scale;    // [B, H, W, blocks]
    const float* v_scale;
    const int* counts;       // [B] keys of each batch element, or null: nk
    __nv_bfloat16* O;        // [B, H, nq, d]
    float* lse;              // [B, H, nq] or null
    float* part_o;           // [B, H, nq, splits, d], when splits > 1
    float2* part_ml;         // [B, H, nq, splits]: maximum (base 2) and sum
    int H, nq, s, W, blocks, nk;
    uint32_t per_s;          // floor(2^32 / s) (2^32 - 1 for s = 1): see scale_index
    int q_tiles, splits, chunk;  // tiles of queries; ranges of keys, each of `chunk` keys
    float scale_log2;        // scale * log2(e)
    int B;
    int* err;                // the library's device error word (few-query kernel: debug build only)
    bool skip_on_error;      // the kernel before the join may have given up
    unsigned long long timeout_ns;
};

__device__ __forceinline__ int key_count(const AttnParams& p, int b)
{
    return p.counts ? min(max(p.counts[b], 0), p.nk) : p.nk;
}

// Index of key's scale: slot = key / s by a multiplication, floor(2^32 / s) for which
// key * floor(2^32 / s) / 2^32 is less than key / 2^32 < 1 below key / s: at most one off.
__device__ __forceinline__ long long scale_index(const AttnParams& p, long long bh, int key)
{
    int slot = static_cast<int>(__umulhi(static_cast<uint32_t>(key), p.per_s));
    int at = key - slot * p.s;
    if (at >= p.s) {
        ++slot;
        at -= p.s;
    }
    return (bh * p.W + slot) * p.blocks + at / CACHE8_BLOCK;
}

// Bounds checks of the debug build (see ra_bounds.cuh): `n` keys of head bh from `key`
// on, their scale's index, a query's row, a partial result's.
__device__ __forceinline__ bool keys_inside(const AttnParams& p, long long bh, long long key, long long n)
{
    return inside(p.err, key, n, p.nk, SITE_I_CODE) &&
           inside(p.err, bh * p.W * p.s + key, n, static_cast<long long>(p.B) * p.H * p.W * p.s, SITE_I_CODE);
}
__device__ __forceinline__ bool scale_inside(const AttnParams& p, long long at)
{
    return inside(p.err, at, 1, static_cast<long long>(p.B) * p.H * p.W * p.blocks, SITE_I_SCALE);
}
__device__ __forceinline__ bool row_inside(const AttnParams& p, long long row, int site)
{
    return inside(p.err, row, 1, static_cast<long long>(p.B) * p.H * p.nq, site);
}
__device__ __forceinline__ bool part_inside(const AttnParams& p, long long at)
{
    return inside(p.err, at, 1, static_cast<long long>(p.B) * p.H * p.nq * p.splits, SITE_I_PART);
}

// The many-query kernel (256 queries a block, or 128 if `one`; P as a pair of bf16
// numbers if `pair`), writing O and lse, or partial results when p.splits > 1.
ra_status cache8_tiles(const AttnParams& p, int B, int d, bool one, bool pair, cudaStream_t cs);

}  // namespace ra
