// ra_cache8.cu -- new frames into the 8-bit key/value ring (ra_cache8.cuh), the
// keys normed and rotated on the way.
//
// One thread block per (head, 64-token block of a frame, K or V): its rows are
// read from the projection's token-major layout, normed and rotated in fp32 (K),
// and kept in registers; the block's largest magnitude fixes the scale, the least
// power of two that brings it to at most 448, and the codes are rounded once, to
// nearest even, from fp32.  Bound by memory: 3 bytes a value (2 read, 1 written).
//
// The scale's power of two costs no precision against amax / 448: e4m3 is a
// floating format, so only the numbers near its subnormals (2^-15 of the largest
// and below) see the difference.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "ra_cache8.cuh"
#include "ra_head_rows.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int PASSES = 4;         // row groups of a block held in registers
constexpr int ROWS_PER_PASS = 16; // so that PASSES * ROWS_PER_PASS rows make a block
static_assert(PASSES * ROWS_PER_PASS == CACHE8_BLOCK, "a block of tokens is held whole");

struct AppendParams {
    const __nv_bfloat16* x[2];  // K, V [B, frames * s, H, d] by strides (elements)
    long long sb[2], sn[2], sh[2];
    uint8_t* code[2];           // [B, H, W * s, d]
    float* scale[2];            // [B, H, W, blocks]
    const void* weight;         // norm of K, or null
    int weight_fp32;
    int H, s, W, blocks, slot0;
    RopeArgs rope;
    float eps;
};

template <int D>
__global__ void __launch_bounds__(ROWS_PER_PASS * D / 8) cache8_append_kernel(const AppendParams p)
{
    constexpr int LPR = D / 8;
    const int which = blockIdx.y, b = blockIdx.z;
    const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.H));
    const int fb = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.H));
    const int frame = fb / p.blocks, blk = fb - frame * p.blocks;
    const int rows = min(CACHE8_BLOCK, p.s - blk * CACHE8_BLOCK);
    const int sub = threadIdx.x % LPR, row0 = threadIdx.x / LPR, step = blockDim.x / LPR;
    const int token0 = frame * p.s + blk * CACHE8_BLOCK;  // among the call's tokens
    const __nv_bfloat16* x = p.x[which] + b * p.sb[which] + h * p.sh[which] + sub * 8;
    uint4 v[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = row0 + i * step;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < rows)
            v[i] = __ldcs(reinterpret_cast<const uint4*>(x + static_cast<long long>(token0 + r) * p.sn[which]));
    }
    float f[PASSES][8];
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
        unpack_bf16x8(v[i], f[i]);
    if (which == 0) {
        if (p.weight) {
            float w[8];
            load_weight(p.weight, p.weight_fp32, sub, w);
#pragma unroll
            for (int i = 0; i < PASSES; ++i)
                rms_norm<D>(f[i], w, p.eps);
        }
        if (p.rope.t) {
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                if (row0 + i * step < rows) {
                    float2 cs[4];
                    load_rope(p.rope, token0 + row0 + i * step, sub, cs);
                    rotate(cs, f[i]);
                }
            }
        }
    }
    // the largest magnitude as bits: above every finite number for infinities and NaN
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    __shared__ uint32_t tops[ROWS_PER_PASS * LPR / 32];
    if (blockDim.x > 32) {
        if (threadIdx.x % 32 == 0)
            tops[threadIdx.x / 32] = top;
        __syncthreads();
        for (unsigned k = 0; k < blockDim.x / 32; ++k)
            top = max(top, tops[k]);
    }
    // scale = 2^k: largest = 1.m * 2^e, k = e - 8, one more above 448 = 1.75 * 2^8
    float scale = 1.f, inverse = 1.f;
    if (top >= 0x7F800000u) {
        scale = __uint_as_float(0x7FFFFFFFu);
        inverse = 0.f;  // codes of such a block are zero or, from infinities and NaN, the format's largest
    } else if (top > 0) {
        int k = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        k = max(k, -126);
        scale = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
        inverse = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    }
    const int slot = (p.slot0 + frame) % p.W;
    const long long slot_of_head = (static_cast<long long>(b) * p.H + h) * p.W + slot;
    uint8_t* code = p.code[which] + (slot_of_head * p.s + blk * CACHE8_BLOCK) * D + sub * 8;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = row0 + i * step;
        if (r >= rows)
            continue;
        uint32_t word[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t half[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                half[e] = __nv_cvt_float2_to_fp8x2(make_float2(f[i][4 * j + 2 * e] * inverse,
                                                               f[i][4 * j + 2 * e + 1] * inverse),
                                                   __NV_SATFINITE, __NV_E4M3);
            word[j] = top >= 0x7F800000u ? 0u : half[0] | (half[1] << 16);
        }
        *reinterpret_cast<uint2*>(code + static_cast<size_t>(r) * D) = make_uint2(word[0], word[1]);
    }
    if (threadIdx.x == 0)
        p.scale[which][slot_of_head * p.blocks + blk] = scale;
}

}  // namespace

ra_status check_cache8(const void* k8, const void* v8, const float* k_scale, const float* v_scale, int B, int H, int d,
                       int s, int W)
{
    if (!k8 || !v8 || !k_scale || !v_scale)
        return fail(RA_ERR_INVALID_ARG, "NULL ring pointer");
    if (!aligned16(k8) || !aligned16(v8))
        return fail(RA_ERR_INVALID_ARG, "the rings must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(k_scale) % 4 || reinterpret_cast<uintptr_t>(v_scale) % 4)
        return fail(RA_ERR_INVALID_ARG, "the scales must be 4-byte aligned");
    if (B < 1 || H < 1 || B > 65535 || H > 65535)
        return fail(RA_ERR_INVALID_ARG, "B and H must be in [1, 65535] (B=%d, H=%d)", B, H);
    if (d != 64 && d != 128)
        return fail(RA_ERR_UNSUPPORTED, "head dim %d is not supported (64 or 128)", d);
    if (s < 1 || W < 1)
        return fail(RA_ERR_INVALID_ARG, "s and window_frames must be >= 1");
    if (static_cast<long long>(s) * W > (1LL << 31) - 1)
        return fail(RA_ERR_UNSUPPORTED, "window of %lld tokens is too long", static_cast<long long>(s) * W);
    return RA_OK;
}

}  // namespace ra

using namespace ra;

extern "C" ra_status ra_cache8_append(const ra_head_rows* k, const ra_head_rows* v, int B, int frames, int d, int s,
                                      int window_frames, long long frame, const ra_rope* rope, float eps, void* k8,
                                      void* v8, float* k_scale, float* v_scale, ra_stream stream)
{
    if (!k || !v)
        return fail(RA_ERR_INVALID_ARG, "NULL argument");
    if (k->heads != v->heads)
        return fail(RA_ERR_INVALID_ARG, "k and v must have the same heads (%d, %d)", k->heads, v->heads);
    if (v->weight)
        return fail(RA_ERR_INVALID_ARG, "v is not normed: its weight must be NULL");
    const int H = k->heads, W = window_frames;
    ra_status st = check_cache8(k8, v8, k_scale, v_scale, B, H, d, s, W);
    if (st != RA_OK)
        return st;
    if (frames < 1 || frames > W)
        return fail(RA_ERR_INVALID_ARG, "frames must be in [1, window_frames] (%d of %d): each takes a slot of its own",
                    frames, W);
    if (frame < 0)
        return fail(RA_ERR_INVALID_ARG, "frame must be >= 0");
    if (!(eps > 0.f) || !std::isfinite(eps))
        return fail(RA_ERR_INVALID_ARG, "eps must be finite and > 0");
    const int n = frames * s;
    AppendParams p;
    std::memset(&p, 0, sizeof p);
    if (rope) {
        if (static_cast<long long>(rope->grid_h) * rope->grid_w != s)
            return fail(RA_ERR_INVALID_ARG, "the rope's grid of %d x %d is not a frame of %d tokens", rope->grid_h,
                        rope->grid_w, s);
        if (frame > (1LL << 31) - 1)
            return fail(RA_ERR_INVALID_ARG, "frame %lld is outside the time table", frame);
    }
    if ((st = rope_args(rope, static_cast<int>(rope ? frame : 0), n, d, &p.rope)) != RA_OK ||
        (st = head_rows_args("k", k, B, n, d, &p.sb[0], &p.sn[0], &p.sh[0])) != RA_OK ||
        (st = head_rows_args("v", v, B, n, d, &p.sb[1], &p.sn[1], &p.sh[1])) != RA_OK)
        return st;
    p.x[0] = static_cast<const __nv_bfloat16*>(k->x);
    p.x[1] = static_cast<const __nv_bfloat16*>(v->x);
    p.weight = k->weight;
    p.weight_fp32 = k->weight_fp32;
    p.code[0] = static_cast<uint8_t*>(k8);
    p.code[1] = static_cast<uint8_t*>(v8);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.H = H;
    p.s = s;
    p.W = W;
    p.blocks = cache8_blocks(s);
    p.slot0 = static_cast<int>(frame % W);
    p.eps = eps;
    const long long heads = static_cast<long long>(B) * H;
    const Span out[4] = {span(k8, heads * W * s * d), span(v8, heads * W * s * d),
                         span(k_scale, heads * W * p.blocks * 4), span(v_scale, heads * W * p.blocks * 4)};
    const Span in[3] = {span(k->x, extent(p.sb[0], p.sn[0], p.sh[0], B, n, H, d)),
                        span(v->x, extent(p.sb[1], p.sn[1], p.sh[1], B, n, H, d)),
                        span(k->weight, d * (k->weight_fp32 ? 4 : 2))};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(out[i], in[j]))
                return fail(RA_ERR_INVALID_ARG, "the rings may not alias an input");
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i], out[j]))
                return fail(RA_ERR_INVALID_ARG, "the rings and scales may not alias one another");
    }
    const long long blocks = static_cast<long long>(frames) * p.blocks * H;
    if (blocks > (1LL << 31) - 1)
        return fail(RA_ERR_UNSUPPORTED, "too many blocks in one call (%lld)", blocks);
    const dim3 grid(static_cast<unsigned>(blocks), 2, B);
    const int rows = s < ROWS_PER_PASS ? s : ROWS_PER_PASS;
    const int threads = (rows * (d / 8) + 31) / 32 * 32;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64)
        cache8_append_kernel<64><<<grid, threads, 0, cs>>>(p);
    else
        cache8_append_kernel<128><<<grid, threads, 0, cs>>>(p);
    return cuda_fail(cudaGetLastError(), "cache8_append_kernel launch");
}
