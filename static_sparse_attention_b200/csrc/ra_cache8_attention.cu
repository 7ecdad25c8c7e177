// ra_cache8_attention.cu -- attention of a few or many queries over the 8-bit
// key/value ring (ra_cache8.cuh):
//     O = softmax(scale * Q K^T) V over the first count keys of each head.
//
// Few-query kernel: one block per (head, 16 queries, range of keys), four warps
// that take groups of 16 keys in turn.  Codes go from memory to registers and are
// turned to bf16 there; both products are 16 x 8 x 16 warp products with fp32
// sums.  The order of channels and keys inside a product is free, so it is chosen
// by what a lane loads: 16 contiguous bytes of a key's row for S, and of a
// value's row for P V.  Ranges of keys leave partial (maximum, sum, O) to a
// second kernel that joins them.  Bound by memory for few queries (one byte a
// value of K and V).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "ra_cache8_attention.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int ROWS = 16;   // queries of a block
constexpr int WARPS = 4;
constexpr int GROUP = 16;  // keys that a warp takes at a time
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// D += A B: A 16 x 16 (row), B 16 x 8 (column), bf16, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes and scales of one group of keys, as a lane (r = lane / 4, c = lane % 4) holds them.
template <int D>
struct Group {
    static constexpr int KP = D / 64;   // 16-byte pieces of a key's row a lane holds
    static constexpr int VW = D / 32;   // 4-byte words of a value's row a lane holds
    uint4 k[2][KP];                     // keys 8 t + r: channels 64 p + 16 c .. + 15
    uint32_t v[4][VW];                  // keys 2 c + {0, 1, 8, 9}: channels (D / 8) r .. + D / 8 - 1
    float scale;                        // lanes 0-15: of key lane, 16-31: of value lane - 16 (0 behind the range)
};

template <int D>
__device__ __forceinline__ void load_group(Group<D>& g, const AttnParams& p, long long bh, int key0, int end)
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const long long head = bh * p.W * p.s;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int key = key0 + 8 * t + r;
#pragma unroll
        for (int i = 0; i < Group<D>::KP; ++i) {
            g.k[t][i] = make_uint4(0, 0, 0, 0);
            if (key < end)
                g.k[t][i] = __ldcs(reinterpret_cast<const uint4*>(p.k8 + (head + key) * D + 64 * i + 16 * c));
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int key = key0 + 2 * c + (t & 1) + 8 * (t >> 1);
#pragma unroll
        for (int i = 0; i < Group<D>::VW; ++i)
            g.v[t][i] = 0;
        if (key < end) {
            const uint8_t* at = p.v8 + (head + key) * D + r * (D / 8);
            if (D == 128) {
                const uint4 w = __ldcs(reinterpret_cast<const uint4*>(at));
                g.v[t][0] = w.x, g.v[t][1] = w.y, g.v[t][Group<D>::VW - 2] = w.z, g.v[t][Group<D>::VW - 1] = w.w;
            } else {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(at));
                g.v[t][0] = w.x, g.v[t][1] = w.y;
            }
        }
    }
    const int key = key0 + (lane & 15);
    g.scale = 0.f;
    if (key < end) {
        const long long at = scale_index(p, bh, key);
        g.scale = lane < 16 ? p.k_scale[at] : p.v_scale[at];
    }
}

// The running state of 16 queries in one warp: rows r and r + 8 of the tile.
template <int D>
struct State {
    uint32_t q[D / 16][4];  // A operands of S
    float o[D / 8][4];
    float m[2], l[2];       // l: this lane's keys only
};

// TWO: some scale of the group needs its second factor.
template <int D, bool TWO>
__device__ __forceinline__ void group_step(State<D>& st, const Group<D>& g, int key0, int end, float scale_log2)
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const CodeScale mine = code_scale(g.scale);
    const uint32_t both = mine.first | (mine.second << 16);
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t f = __shfl_sync(0xFFFFFFFFu, both, 8 * t + r);
        const uint32_t f1 = __byte_perm(f, 0, 0x1010), f2 = __byte_perm(f, 0, 0x3232);
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int i = 0; i < Group<D>::KP; ++i) {
            const uint32_t w[4] = {g.k[t][i].x, g.k[t][i].y, g.k[t][i].z, g.k[t][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t b0 = mul_bf16x2(e4m3x2_small(w[j] << 8), f1);
                uint32_t b1 = mul_bf16x2(e4m3x2_small(w[j]), f1);
                if (TWO) {
                    b0 = mul_bf16x2(b0, f2);
                    b1 = mul_bf16x2(b1, f2);
                }
                mma16816(s[t], st.q[4 * i + j], b0, b1);
            }
        }
    }
    // online softmax in base 2, keys behind the range masked
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[t][e] = key0 + 8 * t + 2 * c + (e & 1) < end ? __fmul_rn(s[t][e], scale_log2) : -INFINITY;
            top[e >> 1] = fmaxf(top[e >> 1], s[t][e]);
        }
    bool grew = false;
    float use[2], alpha[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        top[y] = fmaxf(top[y], __shfl_xor_sync(0xFFFFFFFFu, top[y], 1));
        top[y] = fmaxf(top[y], __shfl_xor_sync(0xFFFFFFFFu, top[y], 2));
        const float m = fmaxf(st.m[y], top[y]);
        alpha[y] = m == -INFINITY ? 1.f : exp2_fast(st.m[y] - m);
        grew |= m > st.m[y];
        st.m[y] = m;
        use[y] = m == -INFINITY ? 0.f : m;  // no finite score yet: 2^(-inf) = 0, and a NaN stays one
    }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            st.o[j][0] *= alpha[0];
            st.o[j][1] *= alpha[0];
            st.o[j][2] *= alpha[1];
            st.o[j][3] *= alpha[1];
        }
        st.l[0] *= alpha[0];
        st.l[1] *= alpha[1];
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[t][e] = exp2_fast(s[t][e] - use[e >> 1]);
            st.l[e >> 1] += s[t][e];
        }
    const uint32_t a[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]),
                           pack2(s[1][2], s[1][3])};
    uint32_t f1[2], f2[2];  // of the value pairs 2 c, 2 c + 1 and 8 + 2 c, 9 + 2 c
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t x = __shfl_sync(0xFFFFFFFFu, both, 16 + 8 * t + 2 * c);
        const uint32_t y = __shfl_sync(0xFFFFFFFFu, both, 17 + 8 * t + 2 * c);
        f1[t] = __byte_perm(x, y, 0x5410);
        f2[t] = __byte_perm(x, y, 0x7632);
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
        // byte j of each pair of keys, to bytes 1 and 3 (the others are masked out)
        const uint32_t pick = static_cast<uint32_t>(((4 + j % 4) << 12) | ((j % 4) << 4));
        uint32_t b0 = mul_bf16x2(e4m3x2_small(__byte_perm(g.v[0][j / 4], g.v[1][j / 4], pick)), f1[0]);
        uint32_t b1 = mul_bf16x2(e4m3x2_small(__byte_perm(g.v[2][j / 4], g.v[3][j / 4], pick)), f1[1]);
        if (TWO) {
            b0 = mul_bf16x2(b0, f2[0]);
            b1 = mul_bf16x2(b1, f2[1]);
        }
        mma16816(st.o[j], a, b0, b1);
    }
}

template <int D>
__global__ void __launch_bounds__(WARPS * 32) cache8_rows_kernel(const AttnParams p)
{
    __shared__ float sm_o[WARPS][ROWS][D + 4];
    __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int split = static_cast<int>(blockIdx.x) % p.splits, q_tile = static_cast<int>(blockIdx.x) / p.splits;
    const int h = blockIdx.y, b = blockIdx.z;
    const long long bh = static_cast<long long>(b) * p.H + h;
    const int count = key_count(p, b);
    const int begin = split * p.chunk;
    if (p.splits > 1 && begin >= count)
        return;  // the join does not read this split
    const int end = min(begin + p.chunk, count);
    const int q0 = q_tile * ROWS;

    State<D> st;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            uint2 w = make_uint2(0, 0);
            const int q = q0 + r + 8 * y;
            if (q < p.nq)
                w = *reinterpret_cast<const uint2*>(p.Q + (bh * p.nq + q) * D + 64 * (i / 4) + 16 * c + 4 * (i % 4));
            st.q[i][y] = __byte_perm(w.x, w.y, 0x5410);      // channels 0, 2 of the four
            st.q[i][2 + y] = __byte_perm(w.x, w.y, 0x7632);  // channels 1, 3
        }
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
        st.o[j][0] = st.o[j][1] = st.o[j][2] = st.o[j][3] = 0.f;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;

    Group<D> g;
    int key = begin + warp * GROUP;
    if (key < end)
        load_group(g, p, bh, key, end);
    for (; key < end; key += WARPS * GROUP) {
        const Group<D> now = g;
        if (key + WARPS * GROUP < end)
            load_group(g, p, bh, key + WARPS * GROUP, end);
        if (__any_sync(0xFFFFFFFFu, !(now.scale <= 128.f)))
            group_step<D, true>(st, now, key, end, p.scale_log2);
        else
            group_step<D, false>(st, now, key, end, p.scale_log2);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        st.l[y] += __shfl_xor_sync(0xFFFFFFFFu, st.l[y], 1);
        st.l[y] += __shfl_xor_sync(0xFFFFFFFFu, st.l[y], 2);
        if (c == 0) {
            sm_m[warp][r + 8 * y] = st.m[y];
            sm_l[warp][r + 8 * y] = st.l[y];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            sm_o[warp][r + 8 * y][(D / 8) * (2 * c) + j] = st.o[j][2 * y];
            sm_o[warp][r + 8 * y][(D / 8) * (2 * c + 1) + j] = st.o[j][2 * y + 1];
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < ROWS * D; k += WARPS * 32) {
        const int row = k / D, ch = k % D, q = q0 + row;
        if (q >= p.nq)
            break;
        float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            m = fmaxf(m, sm_m[w][row]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = sm_m[w][row] == -INFINITY ? 1.f : exp2_fast(sm_m[w][row] - m);  // 1: its sums are 0 or NaN
            l += sm_l[w][row] * f;
            o += sm_o[w][row][ch] * f;
        }
        const long long at = bh * p.nq + q;
        if (p.splits > 1) {
            p.part_o[(at * p.splits + split) * D + ch] = o;
            if (ch == 0)
                p.part_ml[at * p.splits + split] = make_float2(m, l);
        } else {
            p.O[at * D + ch] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
            if (p.lse && ch == 0)
                p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
        }
    }
}

// Joins the splits of a query: one warp each.
template <int D>
__global__ void __launch_bounds__(128) cache8_join_kernel(const AttnParams p, long long rows)
{
    const long long at = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (at >= rows)
        return;
    const int b = static_cast<int>(at / (static_cast<long long>(p.H) * p.nq));
    const int n = (key_count(p, b) + p.chunk - 1) / p.chunk;
    const float2* ml = p.part_ml + at * p.splits;
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32)
        m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
    float l = 0.f, o[D / 32] = {};
    for (int k = 0; k < n; ++k) {
        const float2 x = ml[k];
        const float f = x.x == -INFINITY ? 1.f : exp2_fast(x.x - m);
        l += x.y * f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            o[i] += p.part_o[(at * p.splits + k) * D + i * 32 + lane] * f;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        p.O[at * D + i * 32 + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
    if (p.lse && lane == 0)
        p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

// How the work is cut.  Few queries: ranges of at least MIN_CHUNK keys, enough
// blocks for every SM.  Many: the number of ranges with the least estimated time,
// counted in steps of 64 keys of the 256-query kernel (one block an SM).
constexpr int MIN_CHUNK = 256;
constexpr int WHOLE = 512;  // as many keys as one block takes in less time than the join's launch
constexpr int SMS = 148;
constexpr int WANT_BLOCKS = SMS * 8;
constexpr int TILES_MIN_QUERIES = 33;  // more queries than this go to the many-query kernel
constexpr double STEP_US = 0.9;        // a step of 64 keys of 256 queries
constexpr double START_STEPS = 6;      // a block's start and epilogue, in steps
constexpr double JOIN_BYTES_PER_US = 5e6;

struct Plan {
    bool many;
    int q_tiles, splits, chunk;
    size_t bytes;
};

Plan plan_of(int B, int H, int d, int nq, int nk)
{
    Plan pl;
    pl.many = nq >= TILES_MIN_QUERIES;
    const int rows = pl.many ? 256 : ROWS, unit = pl.many ? 64 : GROUP * WARPS;
    pl.q_tiles = (nq + rows - 1) / rows;
    const long long tiles = static_cast<long long>(pl.q_tiles) * H * B;
    long long splits = 1;
    if (pl.many) {
        const long long steps = (static_cast<long long>(nk) + unit - 1) / unit;
        const double part = static_cast<double>(B) * H * nq * (d + 2) * 4 * 2 / JOIN_BYTES_PER_US / STEP_US;
        double best = 0;
        for (long long k = 1; k <= 32 && k * 4 <= (steps > 4 ? steps : 4); ++k) {
            const double rounds = static_cast<double>((tiles * k + SMS - 1) / SMS);
            const double cost = rounds * (static_cast<double>((steps + k - 1) / k) + START_STEPS) +
                                (k > 1 ? part * static_cast<double>(k) + 5 : 0);
            if (k == 1 || cost < best) {
                best = cost;
                splits = k;
            }
        }
    } else {
        splits = (WANT_BLOCKS + tiles - 1) / tiles;
        const long long most = nk <= WHOLE ? 1 : (static_cast<long long>(nk) + MIN_CHUNK - 1) / MIN_CHUNK;
        splits = splits < most ? splits : most;
        splits = splits < 1 ? 1 : splits;
    }
    const long long chunk = (nk + splits - 1) / splits;
    pl.chunk = static_cast<int>((chunk + unit - 1) / unit * unit);
    pl.chunk = pl.chunk < unit ? unit : pl.chunk;
    pl.splits = static_cast<int>((static_cast<long long>(nk) + pl.chunk - 1) / pl.chunk);
    pl.splits = pl.splits < 1 ? 1 : pl.splits;
    pl.bytes = pl.splits == 1 ? 0 : static_cast<size_t>(B) * H * nq * pl.splits * (d + 2) * sizeof(float);
    return pl;
}

ra_status check_attention(int B, int H, int d, int nq, int s, int W, int held)
{
    if (B < 1 || H < 1 || B > 65535 || H > 65535)
        return fail(RA_ERR_INVALID_ARG, "B and H must be in [1, 65535] (B=%d, H=%d)", B, H);
    if (d != 64 && d != 128)
        return fail(RA_ERR_UNSUPPORTED, "head dim %d is not supported (64 or 128)", d);
    if (s < 1 || W < 1)
        return fail(RA_ERR_INVALID_ARG, "s and window_frames must be >= 1");
    if (static_cast<long long>(s) * W > (1LL << 31) - 1 - 128)
        return fail(RA_ERR_UNSUPPORTED, "window of %lld tokens is too long", static_cast<long long>(s) * W);
    if (held < 0 || held > W)
        return fail(RA_ERR_INVALID_ARG, "frames held must be in [0, window_frames] (%d of %d)", held, W);
    if (nq < 1 || nq > (1 << 24))
        return fail(RA_ERR_INVALID_ARG, "nq must be in [1, 2^24] (%d)", nq);
    return RA_OK;
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" ra_status ra_cache8_attention_workspace_bytes(int B, int H, int d, int nq, int s, int window_frames,
                                                         int held, size_t* bytes)
{
    if (!bytes)
        return fail(RA_ERR_INVALID_ARG, "NULL output pointer");
    *bytes = 0;
    const ra_status st = check_attention(B, H, d, nq, s, window_frames, held);
    if (st == RA_OK)
        *bytes = plan_of(B, H, d, nq, held * s).bytes;
    return st;
}

extern "C" ra_status ra_cache8_attention(const void* Q, const void* k8, const void* v8, const float* k_scale,
                                         const float* v_scale, void* O, int B, int H, int d, int nq, int s,
                                         int window_frames, int held, const int* key_counts, float scale, float* lse,
                                         void* workspace, size_t workspace_bytes, ra_stream stream)
{
    ra_status st = check_attention(B, H, d, nq, s, window_frames, held);
    if (st != RA_OK || (st = check_cache8(k8, v8, k_scale, v_scale, B, H, d, s, window_frames)) != RA_OK)
        return st;
    if (!Q || !O)
        return fail(RA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned16(Q) || !aligned16(O) || reinterpret_cast<uintptr_t>(lse) % 4 ||
        reinterpret_cast<uintptr_t>(key_counts) % 4)
        return fail(RA_ERR_INVALID_ARG, "tensors must be 16-byte aligned (lse and key_counts 4)");
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(RA_ERR_INVALID_ARG, "scale must be finite and > 0");
    const Plan pl = plan_of(B, H, d, nq, held * s);
    if (pl.bytes && (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)))
        return fail(RA_ERR_INVALID_ARG, "the workspace needs %zu bytes, 16-byte aligned", pl.bytes);
    const long long heads = static_cast<long long>(B) * H, rows = heads * nq;
    const int blocks = cache8_blocks(s);
    const Span out[3] = {span(O, rows * d * 2), span(lse, rows * 4), span(pl.bytes ? workspace : nullptr, pl.bytes)};
    const Span in[6] = {span(Q, rows * d * 2),
                        span(k8, heads * window_frames * s * d),
                        span(v8, heads * window_frames * s * d),
                        span(k_scale, heads * window_frames * blocks * 4),
                        span(v_scale, heads * window_frames * blocks * 4),
                        span(key_counts, static_cast<long long>(B) * 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 6; ++j)
            if (overlap(out[i], in[j]))
                return fail(RA_ERR_INVALID_ARG, "an output may not alias another buffer of the call");
        for (int j = i + 1; j < 3; ++j)
            if (overlap(out[i], out[j]))
                return fail(RA_ERR_INVALID_ARG, "an output may not alias another buffer of the call");
    }
    AttnParams p;
    std::memset(&p, 0, sizeof p);
    p.Q = static_cast<const __nv_bfloat16*>(Q);
    p.k8 = static_cast<const uint8_t*>(k8);
    p.v8 = static_cast<const uint8_t*>(v8);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.counts = key_counts;
    p.O = static_cast<__nv_bfloat16*>(O);
    p.lse = lse;
    p.H = H;
    p.nq = nq;
    p.s = s;
    p.W = window_frames;
    p.blocks = blocks;
    p.nk = held * s;
    p.per_s = s == 1 ? 0xFFFFFFFFu : static_cast<uint32_t>((1ULL << 32) / static_cast<unsigned>(s));
    p.q_tiles = pl.q_tiles;
    p.splits = pl.splits;
    p.chunk = pl.chunk;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (pl.bytes) {
        p.part_o = static_cast<float*>(workspace);
        p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(rows) * pl.splits * d);
    }
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (pl.many) {
        p.timeout_ns = wait_timeout_ns();
        if ((st = device_error_word(&p.err)) != RA_OK || (st = cache8_tiles(p, B, d, cs)) != RA_OK)
            return st;
    } else {
        const dim3 grid(static_cast<unsigned>(pl.q_tiles) * pl.splits, H, B);
        if (d == 64)
            cache8_rows_kernel<64><<<grid, WARPS * 32, 0, cs>>>(p);
        else
            cache8_rows_kernel<128><<<grid, WARPS * 32, 0, cs>>>(p);
        RA_CUDA_TRY(cudaGetLastError());
    }
    if (pl.splits == 1)
        return RA_OK;
    const unsigned joins = static_cast<unsigned>((rows + 3) / 4);
    if (d == 64)
        cache8_join_kernel<64><<<joins, 128, 0, cs>>>(p, rows);
    else
        cache8_join_kernel<128><<<joins, 128, 0, cs>>>(p, rows);
    return cuda_fail(cudaGetLastError(), "cache8_join_kernel launch");
}
