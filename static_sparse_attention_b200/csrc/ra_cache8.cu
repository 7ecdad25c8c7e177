// ra_cache8.cu -- new frames into the 8-bit key/value ring (ra_cache8.cuh), the
// keys normed and rotated on the way.
//
// A thread block takes one 64-token block of a frame, K or V, and walks a group of
// heads: its threads stay with their rows, so a row's cosines and sines and the
// norm's weights are loaded once for all of them.  Each head's rows are read from
// the projection's token-major layout one head ahead, normed and rotated in fp32
// (K), and kept in registers; the block's largest magnitude fixes the scale, the
// least power of two that brings it to at most 448, and the codes are rounded once,
// to nearest even, from fp32.  Bound by memory: 3 bytes a value (2 read, 1 written).
// 12 frames of 3555 tokens, 24 heads of 128: 155 us, 77 % of the measured copy rate
// (120 us); issue slots 58 %, DRAM 59 % busy, the rest is the barrier that fixes a
// block's scale.  (80 registers a thread, three blocks an SM of 128 channels, leave 28
// bytes of spills.)  With a thread block for each head the position look-up was a third
// of the instructions: 247 us.
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
// Heads of a thread block, at most (12 frames of 3555 tokens, 24 heads: 157 us, with 8 heads
// 162; more than 24 not measured).
constexpr int HEADS_MAX = 24;
constexpr int SLOTS = 148 * 3;  // blocks of 128 channels that run at once (of 64: twice as many, not counted)
constexpr double START = 1.5;   // of a block, in heads
static_assert(PASSES * ROWS_PER_PASS == CACHE8_BLOCK, "a block of tokens is held whole");

struct AppendParams {
    const __nv_bfloat16* x[2];  // K, V [B, frames * s, H, d] by strides (elements)
    long long sb[2], sn[2], sh[2];
    uint8_t* code[2];           // [B, H, W * s, d]
    float* scale[2];            // [B, H, W, blocks]
    const void* weight;         // norm of K, or null
    int weight_fp32;
    int H, s, W, blocks, slot0;
    int groups, heads;          // groups of heads, heads of a group
    RopeArgs rope;
    float eps;
    long long x_size[2], code_size, scale_size;  // elements that x spans, of a ring, of its scales
    int* err;                   // debug build: see ra_bounds.cuh
};

// The larger magnitude; NaN if one is.
__device__ __forceinline__ float max_abs(float m, float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
}

template <int D>
struct Shared {
    uint32_t tops[2][ROWS_PER_PASS * D / 256];  // each warp's largest magnitude
    // Cosines and sines, [row][lane of the row]: each thread's own, here rather than
    // in 32 of its registers.
    float4 turns[CACHE8_BLOCK][D / 8][2];
};

// FULL: a block of 64 tokens and all threads.
template <int D, bool KEYS, bool FULL>
__device__ __forceinline__ void append_block(const AppendParams& p, Shared<D>& shared)
{
    constexpr int LPR = D / 8, WHICH = KEYS ? 0 : 1, WARPS = ROWS_PER_PASS * LPR / 32;
    const int b = blockIdx.z;
    const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.groups));
    const int fb = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.groups));
    const int frame = fb / p.blocks, blk = fb - frame * p.blocks;
    const int rows = FULL ? CACHE8_BLOCK : min(CACHE8_BLOCK, p.s - blk * CACHE8_BLOCK);
    const int step = FULL ? ROWS_PER_PASS : blockDim.x / LPR;
    const int sub = threadIdx.x % LPR, row0 = threadIdx.x / LPR;
    const int token0 = frame * p.s + blk * CACHE8_BLOCK;  // among the call's tokens
    const int h0 = group * p.heads, h1 = min(h0 + p.heads, p.H);
    const __nv_bfloat16* x =
        p.x[WHICH] + b * p.sb[WHICH] + h0 * p.sh[WHICH] + (token0 + row0) * p.sn[WHICH] + sub * 8;
    const long long row_step = step * p.sn[WHICH];
    auto in = [&](int i) { return FULL || row0 + i * step < rows; };
    auto load = [&](uint4 (&v)[PASSES]) {  // the head that x stands at
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (in(i) && inside(p.err, x + i * row_step - p.x[WHICH], 8, p.x_size[WHICH], SITE_I_IN))
                v[i] = __ldcs(reinterpret_cast<const uint4*>(x + i * row_step));
        }
        x += p.sh[WHICH];
    };
    uint4 next[PASSES];
    load(next);
    float w[8];
    if (KEYS) {
        if (p.weight)
            load_weight(p.weight, p.weight_fp32, sub, w);
        if (p.rope.t) {
            for (int r = row0; r < rows; r += step) {
                float2 cs[4];
                load_rope(p.rope, token0 + r, sub, cs);
                shared.turns[r][sub][0] = make_float4(cs[0].x, cs[0].y, cs[1].x, cs[1].y);
                shared.turns[r][sub][1] = make_float4(cs[2].x, cs[2].y, cs[3].x, cs[3].y);
            }
        }
    }
    long long head = static_cast<long long>(b) * p.H + h0;
    const int slot = (p.slot0 + frame) % p.W;
    const long long first = (head * p.W + slot) * p.s + blk * CACHE8_BLOCK + row0, next_head = static_cast<long long>(p.W) * p.s;
    uint8_t* code = p.code[WHICH] + first * D + sub * 8;
    for (int h = h0; h < h1; ++h) {
        // f: the row before the norm's factor r, which joins the scale's below
        float f[PASSES][8], r[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i)
            unpack_bf16x8(next[i], f[i]);
        if (h + 1 < h1)
            load(next);
        if (KEYS && p.weight) {
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss = fmaf(f[i][j], f[i][j], ss);
                r[i] = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[i][j] *= w[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < PASSES; ++i)
                r[i] = 1.f;
        }
        if (KEYS && p.rope.t) {
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                if (in(i)) {
                    const float4 a = shared.turns[row0 + i * step][sub][0], c = shared.turns[row0 + i * step][sub][1];
                    const float2 cs[4] = {{a.x, a.y}, {a.z, a.w}, {c.x, c.y}, {c.z, c.w}};
                    rotate(cs, f[i]);
                }
            }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            float m = max_abs(0.f, f[i][0], f[i][1]);
#pragma unroll
            for (int j = 2; j < 8; j += 2)
                m = max_abs(m, f[i][j], f[i][j + 1]);
            top = max_abs(top, m * r[i], 0.f);
        }
        // as bits, magnitudes compare like numbers, infinities and NaN above the finite ones
        uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
        if (FULL || blockDim.x > 32) {
            uint32_t(&tops)[WARPS] = shared.tops[h & 1];  // two sets: the last head's may still be read
            const int lane = threadIdx.x & 31;
            if (lane == 0)
                tops[threadIdx.x / 32] = bits;
            __syncthreads();
            bits = __reduce_max_sync(0xFFFFFFFFu, lane < (FULL ? WARPS : static_cast<int>(blockDim.x) / 32) ? tops[lane] : 0u);
        }
        // scale = 2^k: largest = 1.m * 2^e, k = e - 8, one more above 448 = 1.75 * 2^8
        const bool finite = bits < 0x7F800000u;
        int k = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        k = bits == 0 || !finite ? 0 : max(k, -126);
        if (threadIdx.x == 0 && inside(p.err, (head * p.W + slot) * p.blocks + blk, 1, p.scale_size, SITE_I_SCALE))
            p.scale[WHICH][(head * p.W + slot) * p.blocks + blk] =
                __uint_as_float(finite ? static_cast<uint32_t>(k + 127) << 23 : 0x7FFFFFFFu);
        // 1 / scale, joined to the norm's factor: r is below 2^75 (1 / sqrt of the least eps),
        // so that r / scale stays finite down to scales of 2^-50, and is taken in three
        // factors below.
        const int k1 = max(k, -50);
        const float inverse = __uint_as_float(static_cast<uint32_t>(127 - k1) << 23);
        if (k1 != k) {
            const float rest = __uint_as_float(static_cast<uint32_t>(127 + k1 - k) << 23);
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[i][j] = f[i][j] * r[i] * rest;
                r[i] = 1.f;
            }
        }
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const float by = r[i] * inverse;
            uint32_t half[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                half[e] = __nv_cvt_float2_to_fp8x2(make_float2(f[i][2 * e] * by, f[i][2 * e + 1] * by), __NV_SATFINITE,
                                                   __NV_E4M3);
            uint2 word = make_uint2(__byte_perm(half[0], half[1], 0x5410), __byte_perm(half[2], half[3], 0x5410));
            if (!finite)
                word = make_uint2(0, 0);
            if (in(i) && inside(p.err, code + static_cast<long long>(i) * step * D - p.code[WHICH], 8, p.code_size, SITE_I_CODE))
                *reinterpret_cast<uint2*>(code + static_cast<size_t>(i) * step * D) = word;
        }
        ++head;
        code += next_head * D;
    }
}

template <int D>
__global__ void __launch_bounds__(ROWS_PER_PASS * D / 8, 3 * 128 / D) cache8_append_kernel(const AppendParams p)
{
    __shared__ Shared<D> shared;
    const int blk = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.groups)) % p.blocks;
    const bool full = p.s - blk * CACHE8_BLOCK >= CACHE8_BLOCK;
    if (blockIdx.y == 0) {
        if (full)
            append_block<D, true, true>(p, shared);
        else
            append_block<D, true, false>(p, shared);
    } else {
        if (full)
            append_block<D, false, true>(p, shared);
        else
            append_block<D, false, false>(p, shared);
    }
}

}  // namespace

namespace {

// Heads of a thread block: least rounds of the SLOTS blocks (fractions counted, so that
// 500 blocks are 1.13 rounds) times the heads of one and START more for its start; at
// most HEADS_MAX.
int heads_per_block(long long units, int H)
{
    int best = 1;
    double least = 0;
    for (int heads = 1; heads <= H && heads <= HEADS_MAX; ++heads) {
        const double rounds = static_cast<double>(units * ((H + heads - 1) / heads)) / SLOTS;
        const double cost = (rounds > 1 ? rounds : 1) * (heads + START);
        if (heads == 1 || cost < least) {
            least = cost;
            best = heads;
        }
    }
    return best;
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
    if (static_cast<long long>(s) * W > CACHE8_MAX_ROWS)
        return fail(RA_ERR_UNSUPPORTED, "window of %lld tokens is too long", static_cast<long long>(s) * W);
    if (static_cast<long long>(B) * H > (1LL << 40) / (static_cast<long long>(s) * W))
        return fail(RA_ERR_UNSUPPORTED, "ring too large");
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
    p.code_size = heads * W * s * d;
    p.scale_size = heads * W * p.blocks;
    for (int i = 0; i < 2; ++i)
        p.x_size[i] = extent(p.sb[i], p.sn[i], p.sh[i], B, n, H, d) / 2;
    if ((st = bounds_word(&p.err)) != RA_OK)
        return st;
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
    const long long units = static_cast<long long>(frames) * p.blocks;
    p.heads = heads_per_block(units * B * 2, H);
    p.groups = (H + p.heads - 1) / p.heads;
    const long long blocks = units * p.groups;
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
