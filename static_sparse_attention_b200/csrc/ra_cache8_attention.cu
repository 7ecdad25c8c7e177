// ra_cache8_attention.cu -- attention of a few or many queries over the 8-bit
// key/value ring (ra_cache8.cuh):
//     O = softmax(scale * Q K^T) V over the first count keys of each head.
//
// Few-query kernel: one block per (head, 8 or 16 queries, range of keys), four
// warps that take groups of 16 keys in turn; L2 is asked for them some rounds ahead.
// Both products are 16 x 8 x 16 warp products with fp32 sums that keep the queries as
// columns: S^T = K Q^T and O^T += V^T P^T, so that eight queries (or one) take half
// the registers that they would as rows.  The order of channels and keys inside a
// product is free and chosen by what a lane loads: 16 contiguous bytes of a key's
// row, and of a value's row.
//   S^T: the codes go to fp16 as they are (one instruction for two), Q is brought to
//        fp16 by a power of two for each query, and the key's scale multiplies the
//        score.
//   P V: the values go to bf16 code * scale (ra_cache8.cuh) and P to bf16, whose
//        range no mixture of scales leaves, with or without what the rounding leaves
//        (PForm).  For up to four queries the rests ride in the product's free
//        columns: the eight caches 182 us, without them 179; a second product 197.
//        For more it is a second product, asked for below 4096 keys.
// Ranges of keys leave partial (maximum, sum, O) to a second kernel that joins them.
// Few queries read one byte a value of K and V: one query on each of eight caches of
// 4096 to 32768 keys, 24 heads of 128, takes 182 us in a run of 30 calls = 5.1 TB/s, 78 %
// of the measured copy rate, and 194 with caches that change from call to call (DRAM
// traffic 0.939 GB of 0.934).  Nothing is at its limit: DRAM 65 % busy, the integer pipe,
// which turns the codes of V to bf16, 60 %, issue slots 54 %, with 14 warps an SM.  One
// launch of a few hundred keys: 7 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "ra_cache8_attention.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int COLS = 8;    // queries of a product
constexpr int WARPS = 4;
constexpr int GROUP = 16;  // keys that a warp takes at a time
constexpr int PREFETCH = 4;  // rounds of groups that L2 is asked for ahead
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

// What the rounding to the pair of bf16 numbers `rounded` leaves of lo and hi.
__device__ __forceinline__ uint32_t rest2(float lo, float hi, uint32_t rounded)
{
    return pack2(lo - __uint_as_float(rounded << 16), hi - __uint_as_float(rounded & 0xFFFF0000u));
}

// D += A B: A 16 x 16 (row), B 16 x 8 (column), fp32 sums.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit numbers spread over the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Codes 0, 1 and codes 2, 3 of a word as fp16 numbers.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
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

// Where a lane reads: its places in the rows of the group that starts at key 0 of
// the head.
struct Places {
    const uint8_t* k;     // row r
    const uint8_t* v;     // row 2 c
    const uint8_t* ahead; // row lane % 16 of K (lanes 0-15) or V, for the prefetch
    const float* scale;   // of K or V
};

template <int D>
__device__ __forceinline__ Places places_of(const AttnParams& p, long long bh)
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const long long head = bh * p.W * p.s * D;
    return Places{p.k8 + head + r * D + 16 * c, p.v8 + head + 2 * c * D + r * (D / 8),
                  (lane < 16 ? p.k8 : p.v8) + head + (lane & 15) * D, lane < 16 ? p.k_scale : p.v_scale};
}

template <int D, bool WHOLE_GROUP>
__device__ __forceinline__ void load_codes(Group<D>& g, const AttnParams& p, const Places& at, long long bh, int key0,
                                           int end)
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const uint8_t *k = at.k + static_cast<long long>(key0) * D, *v = at.v + static_cast<long long>(key0) * D;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < Group<D>::KP; ++i) {
            if (!WHOLE_GROUP)
                g.k[t][i] = make_uint4(0, 0, 0, 0);
            if ((WHOLE_GROUP || key0 + 8 * t + r < end) && keys_inside(p, bh, key0 + 8 * t + r, 1))
                g.k[t][i] = __ldcs(reinterpret_cast<const uint4*>(k + 8 * t * D + 64 * i));
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int row = (t & 1) + 8 * (t >> 1);  // behind 2 c
        if (!WHOLE_GROUP) {
#pragma unroll
            for (int i = 0; i < Group<D>::VW; ++i)
                g.v[t][i] = 0;
        }
        if ((WHOLE_GROUP || key0 + 2 * c + row < end) && keys_inside(p, bh, key0 + 2 * c + row, 1)) {
            if (D == 128) {
                const uint4 w = __ldcs(reinterpret_cast<const uint4*>(v + row * D));
                g.v[t][0] = w.x, g.v[t][1] = w.y, g.v[t][Group<D>::VW - 2] = w.z, g.v[t][Group<D>::VW - 1] = w.w;
            } else {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(v + row * D));
                g.v[t][0] = w.x, g.v[t][1] = w.y;
            }
        }
    }
}

// Ask L2 for a later group's codes and scales: one row of K or V a lane.
template <int D>
__device__ __forceinline__ void prefetch_group(const AttnParams& p, const Places& at, long long bh, int key0, int end)
{
    const int key = key0 + static_cast<int>(threadIdx.x & 15);
    if (key < end && keys_inside(p, bh, key, 1) && scale_inside(p, scale_index(p, bh, key))) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at.ahead + static_cast<long long>(key0) * D));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at.scale + scale_index(p, bh, key)));
    }
}

// The group that starts at key0: its codes (zeros behind `end`) and scales; and the
// prefetch of one PREFETCH rounds later.
template <int D>
__device__ __forceinline__ void load_group(Group<D>& g, const AttnParams& p, const Places& at, long long bh, int key0,
                                           int end)
{
    if (key0 + GROUP <= end)
        load_codes<D, true>(g, p, at, bh, key0, end);
    else
        load_codes<D, false>(g, p, at, bh, key0, end);
    const int key = key0 + static_cast<int>(threadIdx.x & 15);
    g.scale = key < end && scale_inside(p, scale_index(p, bh, key)) ? at.scale[scale_index(p, bh, key)] : 0.f;
    prefetch_group<D>(p, at, bh, key0 + PREFETCH * WARPS * GROUP, end);
}

// The running state of 8 NT queries in one warp: a lane holds queries 8 t + 2 c and
// 8 t + 2 c + 1.
template <int D, int NT>
struct State {
    uint32_t q[D / 16][NT][2];  // B operands of S^T
    float unit[NT][2];          // scale * log2(e) * the query's power of two
    float o[D / 16][NT][4];     // O^T: channels (D / 8) r + 2 i and the next
    float m[NT][2], l[NT][2];   // l: this lane's keys only
};

// How P reaches its product with V: rounded to bf16; as that and what the rounding
// leaves (to 2^-16 of a weight), in two products; or, for up to four queries, in one,
// whose columns 4-7 are free for the rests of columns 0-3.
enum PForm { P_BF16, P_PAIR, P_COLUMNS };

// TWO: some scale of the group needs its second factor.
template <int D, int NT, PForm P, bool TWO>
__device__ __forceinline__ void group_step(State<D, NT>& st, const Group<D>& g, int key0, int end)
{
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int i = 0; i < Group<D>::KP; ++i) {
        const uint32_t w0[4] = {g.k[0][i].x, g.k[0][i].y, g.k[0][i].z, g.k[0][i].w};
        const uint32_t w1[4] = {g.k[1][i].x, g.k[1][i].y, g.k[1][i].z, g.k[1][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a[4];
            codes_to_f16(w0[j], a[0], a[2]);
            codes_to_f16(w1[j], a[1], a[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                mma_f16(s[t], a, st.q[4 * i + j][t][0], st.q[4 * i + j][t][1]);
        }
    }
    // online softmax in base 2: rows r and r + 8 are keys, those behind the range masked
    const float k0 = __shfl_sync(0xFFFFFFFFu, g.scale, r), k1 = __shfl_sync(0xFFFFFFFFu, g.scale, 8 + r);
    const bool in0 = key0 + r < end, in1 = key0 + 8 + r < end;
    bool grew = false;
    float alpha[NT][2], use[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            s[t][y] = in0 ? __fmul_rn(s[t][y] * st.unit[t][y], k0) : -INFINITY;
            s[t][2 + y] = in1 ? __fmul_rn(s[t][2 + y] * st.unit[t][y], k1) : -INFINITY;
            float top = fmaxf(s[t][y], s[t][2 + y]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            const float m = fmaxf(st.m[t][y], top);
            alpha[t][y] = m == -INFINITY ? 1.f : exp2_fast(st.m[t][y] - m);
            grew |= m > st.m[t][y];
            st.m[t][y] = m;
            use[t][y] = m == -INFINITY ? 0.f : m;  // no finite score yet: 2^(-inf) = 0, and a NaN stays one
        }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                st.o[i][t][0] *= alpha[t][0];
                st.o[i][t][1] *= alpha[t][1];
                st.o[i][t][2] *= alpha[t][0];
                st.o[i][t][3] *= alpha[t][1];
            }
            st.l[t][0] *= alpha[t][0];
            st.l[t][1] *= alpha[t][1];
        }
    }
    uint32_t b0[NT], b1[NT];  // P^T: keys 2 c, 2 c + 1 (b0) and 8 more (b1) of query r
    uint32_t l0[NT], l1[NT];  // P_PAIR: the rests
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[t][e] = exp2_fast(s[t][e] - use[t][e & 1]);
            st.l[t][e & 1] += s[t][e];
        }
        uint32_t x0 = pack2(s[t][0], s[t][1]), x1 = pack2(s[t][2], s[t][3]);
        if (P != P_BF16) {
            const uint32_t y0 = rest2(s[t][0], s[t][1], x0), y1 = rest2(s[t][2], s[t][3], x1);
            if (P == P_PAIR) {
                l0[t] = transpose8x8(y0);
                l1[t] = transpose8x8(y1);
            } else {  // queries 4-7, a lane's from c = 2 on, are queries 0-3 again
                x0 = c < 2 ? x0 : y0;
                x1 = c < 2 ? x1 : y1;
            }
        }
        b0[t] = transpose8x8(x0);
        b1[t] = transpose8x8(x1);
    }
    const CodeScale mine = code_scale(g.scale);
    const uint32_t both = mine.first | (mine.second << 16);
    uint32_t f1[2], f2[2];  // of the value pairs 2 c, 2 c + 1 and 8 + 2 c, 9 + 2 c
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t x = __shfl_sync(0xFFFFFFFFu, both, 16 + 8 * t + 2 * c);
        const uint32_t y = __shfl_sync(0xFFFFFFFFu, both, 17 + 8 * t + 2 * c);
        f1[t] = __byte_perm(x, y, 0x5410);
        f2[t] = __byte_perm(x, y, 0x7632);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // byte 2 i + e of each pair of keys, to bytes 1 and 3 (the others are masked out)
            const int word = (2 * i + e) / 4, byte = (2 * i + e) % 4;
            const uint32_t pick = static_cast<uint32_t>(((4 + byte) << 12) | (byte << 4));
            a[e] = mul_bf16x2(e4m3x2_small(__byte_perm(g.v[0][word], g.v[1][word], pick)), f1[0]);
            a[2 + e] = mul_bf16x2(e4m3x2_small(__byte_perm(g.v[2][word], g.v[3][word], pick)), f1[1]);
            if (TWO) {
                a[e] = mul_bf16x2(a[e], f2[0]);
                a[2 + e] = mul_bf16x2(a[2 + e], f2[1]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mma_bf16(st.o[i][t], a, b0[t], b1[t]);
            if (P == P_PAIR)
                mma_bf16(st.o[i][t], a, l0[t], l1[t]);
        }
    }
}

// AHEAD: a second group is on its way in registers while one is computed; else the
// next one is loaded behind it (L2 has been asked for it), and more warps fit.  Blocks
// an SM of either (128 and 64 channels):
__host__ __device__ constexpr int rows_blocks(int D, int NT, bool ahead) { return NT > 1 ? 2 : ahead ? 3 : D == 64 ? 5 : 4; }

template <int D, int NT, bool AHEAD, PForm P>
__global__ void __launch_bounds__(WARPS * 32, rows_blocks(D, NT, AHEAD)) cache8_rows_kernel(const AttnParams p)
{
    constexpr int ROWS = COLS * NT;
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
    if (p.splits > 1)
        let_next_launch();

    // AHEAD: two groups, taken in turn
    Group<D> even, odd;
    const Places at = places_of<D>(p, bh);
    int key = begin + warp * GROUP;
    if (key < end)
        load_group(even, p, at, bh, key, end);
#pragma unroll
    for (int i = 1; i < PREFETCH; ++i)
        prefetch_group<D>(p, at, bh, key + i * WARPS * GROUP, end);

    State<D, NT> st;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // query 8 t + r: a quarter of its channels in each of four lanes
        uint2 w[D / 16];
        uint32_t top = 0;
        const int q = q0 + 8 * t + (P == P_COLUMNS ? r & 3 : r);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            w[i] = make_uint2(0, 0);
            if (q < p.nq && row_inside(p, bh * p.nq + q, SITE_I_QUERY))
                w[i] = *reinterpret_cast<const uint2*>(p.Q + (bh * p.nq + q) * D + 64 * (i / 4) + 16 * c + 4 * (i % 4));
            top = max(top, max(max(w[i].x & 0x7FFFu, (w[i].x >> 16) & 0x7FFFu),
                               max(w[i].y & 0x7FFFu, (w[i].y >> 16) & 0x7FFFu)));
        }
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^k brings the largest magnitude to [2^14, 2^15) (less below 2^-86)
        const int k = min(14 + 127 - static_cast<int>(top >> 7), 100);
        const float by = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t x = y ? w[i].y : w[i].x;
                const __half2 v = __floats2half2_rn(__uint_as_float(x << 16) * by,
                                                    __uint_as_float(x & 0xFFFF0000u) * by);
                st.q[i][t][y] = *reinterpret_cast<const uint32_t*>(&v);
            }
        const float unit = __uint_as_float(static_cast<uint32_t>(127 - k) << 23) * p.scale_log2;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            st.unit[t][y] = __shfl_sync(0xFFFFFFFFu, unit, 4 * (2 * c + y));
            st.m[t][y] = -INFINITY;
            st.l[t][y] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            st.o[i][t][0] = st.o[i][t][1] = st.o[i][t][2] = st.o[i][t][3] = 0.f;
    }

    auto step = [&](const Group<D>& now, Group<D>& next) {
        const int ahead = key + WARPS * GROUP;
        if (AHEAD && ahead < end)
            load_group(next, p, at, bh, ahead, end);
        if (__any_sync(0xFFFFFFFFu, lane >= 16 && !(now.scale <= 128.f)))
            group_step<D, NT, P, true>(st, now, key, end);
        else
            group_step<D, NT, P, false>(st, now, key, end);
        if (!AHEAD && ahead < end)
            load_group(next, p, at, bh, ahead, end);
        key = ahead;
    };
    while (key < end) {
        if (!AHEAD) {
            step(even, even);
        } else {
            step(even, odd);
            if (key < end)
                step(odd, even);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int q = 8 * t + 2 * c + y;
            st.l[t][y] += __shfl_xor_sync(0xFFFFFFFFu, st.l[t][y], 4);
            st.l[t][y] += __shfl_xor_sync(0xFFFFFFFFu, st.l[t][y], 8);
            st.l[t][y] += __shfl_xor_sync(0xFFFFFFFFu, st.l[t][y], 16);
            if (r == 0) {
                sm_m[warp][q] = st.m[t][y];
                sm_l[warp][q] = st.l[t][y];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float2*>(&sm_o[warp][q][(D / 8) * r + 2 * i]) =
                    make_float2(st.o[i][t][y], st.o[i][t][2 + y]);
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
            o += (P == P_COLUMNS ? sm_o[w][row][ch] + sm_o[w][row + 4][ch] : sm_o[w][row][ch]) * f;
        }
        const long long row_at = bh * p.nq + q;
        if (!row_inside(p, row_at, SITE_I_RESULT) || (p.splits > 1 && !part_inside(p, row_at * p.splits + split)))
            break;
        if (p.splits > 1) {
            p.part_o[(row_at * p.splits + split) * D + ch] = o;
            if (ch == 0)
                p.part_ml[row_at * p.splits + split] = make_float2(m, l);
        } else {
            p.O[row_at * D + ch] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
            if (p.lse && ch == 0)
                p.lse[row_at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
        }
    }
}

using RowsKernel = void (*)(const AttnParams);
template <int D>
RowsKernel rows_kernel(bool one, bool ahead, PForm form)
{
    if (!one)
        return form == P_PAIR ? cache8_rows_kernel<D, 2, true, P_PAIR> : cache8_rows_kernel<D, 2, true, P_BF16>;
    if (form == P_COLUMNS)
        return ahead ? cache8_rows_kernel<D, 1, true, P_COLUMNS> : cache8_rows_kernel<D, 1, false, P_COLUMNS>;
    if (form == P_PAIR)
        return ahead ? cache8_rows_kernel<D, 1, true, P_PAIR> : cache8_rows_kernel<D, 1, false, P_PAIR>;
    return ahead ? cache8_rows_kernel<D, 1, true, P_BF16> : cache8_rows_kernel<D, 1, false, P_BF16>;
}
RowsKernel rows_kernel(int d, bool one, bool ahead, PForm form)
{
    return d == 64 ? rows_kernel<64>(one, ahead, form) : rows_kernel<128>(one, ahead, form);
}

// Joins the splits of a query: one warp each.
template <int D>
__global__ void __launch_bounds__(128) cache8_join_kernel(const AttnParams p, long long rows)
{
    wait_for_previous();
    if (p.skip_on_error && *reinterpret_cast<volatile int*>(p.err) != 0)
        return;  // a block gave up: the parts are not whole
    const long long at = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (at >= rows)
        return;
    const int b = static_cast<int>(at / (static_cast<long long>(p.H) * p.nq));
    const int n = (key_count(p, b) + p.chunk - 1) / p.chunk;
    if (!row_inside(p, at, SITE_I_RESULT) || (n && !part_inside(p, at * p.splits + n - 1)))
        return;
    const float2* ml = p.part_ml + at * p.splits;
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32)
        m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
    // 32 splits' factors at a time, one a lane; then their O, several loads in flight
    float l = 0.f, o[D / 32] = {};
    for (int k0 = 0; k0 < n; k0 += 32) {
        float f = 0.f;
        if (k0 + lane < n) {
            const float2 x = ml[k0 + lane];
            f = x.x == -INFINITY ? 1.f : exp2_fast(x.x - m);  // 1: its sums are 0 or NaN
            l += x.y * f;
        }
        const float* part = p.part_o + (at * p.splits + k0) * D + lane;
        const int here = min(32, n - k0);
#pragma unroll 8
        for (int k = 0; k < here; ++k) {
            const float by = __shfl_sync(0xFFFFFFFFu, f, k);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                o[i] = fmaf(part[k * D + i * 32], by, o[i]);
        }
    }
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1)
        l += __shfl_xor_sync(0xFFFFFFFFu, l, i);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        p.O[at * D + i * 32 + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
    if (p.lse && lane == 0)
        p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

// How the work is cut.  Few queries: ranges of at least MIN_CHUNK keys, as many as
// fill the SMs once (counted at the three blocks an SM of up to 8 queries; 9 to 16 have
// two), or several times where the ranges stay above LONG_CHUNK (batches of unequal
// lengths balance better).  Many: the tiles a block (two, or one) and the number of
// ranges, up to 32, with the least estimated time, one block an SM.  (With one or two
// heads more ranges would fill more SMs: 17 queries over 200000 keys of one head are an
// estimated 92 us with 32 and 28 with 143.)
constexpr int MIN_CHUNK = 256, LONG_CHUNK = 1024;
constexpr int WHOLE = 512;  // as many keys as one block takes in less time than the join's launch
constexpr int SMS = 148;
constexpr int ONE_WAVE = SMS * 3;
constexpr int WANT_BLOCKS = SMS * 16;
// More than 16 queries go to the many-query kernel (24 heads of 128, 2048 keys: 24 us
// against 19 at 17 queries; at 16 the two are equal), except over so few keys that
// the few-query kernel takes them in one go with blocks to spare (256 keys, 24 heads
// of 64, 128 queries: 9.5 against 10.4 us; twice the blocks: 14.5 against 20.7).
constexpr int FEW_BLOCKS = 192;
// A step of 64 keys, and a block's start and epilogue, as measured with a block on
// each SM (12480 keys: two tiles 197 us with 64 channels and 231 with 128, one 113 and
// 171; P as one number); the join.  One tile a block wins where blocks are scarce or the last tile is
// alone: 300 queries, 80 heads of 64, 12480 keys 253 -> 214 us; 256 queries, 24 heads
// of 128, 512 keys 18.7 -> 14.6, but 12480 keys 62 -> 73.
struct TileCost {
    int rows;
    double step64_us, step128_us, start_us;
};
constexpr TileCost TILE_COSTS[2] = {{128, 0.55, 0.85, 4}, {256, 1.0, 1.15, 6}};
constexpr double JOIN_US = 5, JOIN_BYTES_PER_US = 5e6;

struct Plan {
    bool many, one;
    bool ahead;  // few-query kernel: see AHEAD
    int q_tiles, splits, chunk;
    size_t bytes;
};

Plan plan_of(int B, int H, int d, int nq, int nk)
{
    Plan pl;
    pl.many = nq > 2 * COLS && !(nk <= WHOLE && static_cast<long long>((nq + 2 * COLS - 1) / (2 * COLS)) * H * B <= FEW_BLOCKS);
    pl.one = pl.ahead = false;
    const int unit = pl.many ? 64 : GROUP * WARPS;
    long long splits = 1;
    if (pl.many) {
        const long long steps = (static_cast<long long>(nk) + unit - 1) / unit;
        const double part = static_cast<double>(B) * H * nq * (d + 2) * 4 * 2 / JOIN_BYTES_PER_US;
        double best = -1;
        for (const TileCost& c : TILE_COSTS) {
            const int q_tiles = (nq + c.rows - 1) / c.rows;
            const long long tiles = static_cast<long long>(q_tiles) * H * B;
            if (c.rows == 256 && nq <= 128)
                break;
            for (long long k = 1; k <= 32 && k * 4 <= (steps > 4 ? steps : 4); ++k) {
                const double rounds = static_cast<double>((tiles * k + SMS - 1) / SMS);
                const double step = d == 64 ? c.step64_us : c.step128_us;
                const double cost = rounds * (static_cast<double>((steps + k - 1) / k) * step + c.start_us) +
                                    (k > 1 ? part * static_cast<double>(k) + JOIN_US : 0);
                if (best < 0 || cost < best) {
                    best = cost;
                    splits = k;
                    pl.q_tiles = q_tiles;
                    pl.one = c.rows == 128;
                }
            }
        }
    } else {
        const int rows = nq <= COLS ? COLS : 2 * COLS;
        pl.q_tiles = (nq + rows - 1) / rows;
        const long long tiles = static_cast<long long>(pl.q_tiles) * H * B;
        const long long one_wave = (ONE_WAVE + tiles - 1) / tiles, waves = (WANT_BLOCKS + tiles - 1) / tiles;
        const long long long_chunks = nk / LONG_CHUNK;
        splits = waves < long_chunks ? waves : long_chunks;
        splits = splits > one_wave ? splits : one_wave;
        const long long most = nk <= WHOLE ? 1 : (static_cast<long long>(nk) + MIN_CHUNK - 1) / MIN_CHUNK;
        splits = splits < most ? splits : most;
        splits = splits < 1 ? 1 : splits;
    }
    const long long chunk = (nk + splits - 1) / splits;
    pl.chunk = static_cast<int>((chunk + unit - 1) / unit * unit);
    pl.chunk = pl.chunk < unit ? unit : pl.chunk;
    pl.splits = static_cast<int>((static_cast<long long>(nk) + pl.chunk - 1) / pl.chunk);
    pl.splits = pl.splits < 1 ? 1 : pl.splits;
    // One wave of blocks waits for its loads: the second group hides them (12480 keys, 24
    // heads of 128: 25 us, without it 27-29).  Several waves want more warps (eight caches
    // of up to 32768 keys, P as one number: 179 us, with it 189).  Sixteen queries need the
    // registers for two groups either way (250 us; one group and 12 warps 273).
    pl.ahead = nq > COLS || static_cast<long long>(pl.q_tiles) * pl.splits * H * B <= 2 * ONE_WAVE;
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
    if (static_cast<long long>(s) * W > CACHE8_MAX_ROWS)
        return fail(RA_ERR_UNSUPPORTED, "window of %lld tokens is too long", static_cast<long long>(s) * W);
    if (held < 0 || held > W)
        return fail(RA_ERR_INVALID_ARG, "frames held must be in [0, window_frames] (%d of %d)", held, W);
    if (nq < 1 || nq > (1 << 24))
        return fail(RA_ERR_INVALID_ARG, "nq must be in [1, 2^24] (%d)", nq);
    if (static_cast<long long>(B) * H > (1LL << 32) / nq)
        return fail(RA_ERR_UNSUPPORTED, "tensor too large");
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

extern "C" ra_status ra_cache8_attention_plan(int B, int H, int d, int nq, int s, int window_frames, int held,
                                              int* kernel, int* ranges)
{
    const ra_status st = check_attention(B, H, d, nq, s, window_frames, held);
    if (st != RA_OK)
        return st;
    if (!kernel || !ranges)
        return fail(RA_ERR_INVALID_ARG, "NULL output pointer");
    const Plan pl = plan_of(B, H, d, nq, held * s);
    *kernel = pl.many ? (pl.one ? RA_CACHE8_ONE_TILE : RA_CACHE8_TWO_TILES) : (pl.ahead ? RA_CACHE8_ROWS_AHEAD : RA_CACHE8_ROWS);
    *ranges = pl.splits;
    return RA_OK;
}

extern "C" ra_status ra_cache8_attention_check(const void* Q, const void* k8, const void* v8, const float* k_scale,
                                               const float* v_scale, const void* O, int B, int H, int d, int nq, int s,
                                               int window_frames, int held, const int* key_counts, float scale,
                                               const float* lse, const void* workspace, size_t workspace_bytes)
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
    return RA_OK;
}

extern "C" ra_status ra_cache8_attention(const void* Q, const void* k8, const void* v8, const float* k_scale,
                                         const float* v_scale, void* O, int B, int H, int d, int nq, int s,
                                         int window_frames, int held, const int* key_counts, float scale, float* lse,
                                         void* workspace, size_t workspace_bytes, ra_stream stream)
{
    ra_status st = ra_cache8_attention_check(Q, k8, v8, k_scale, v_scale, O, B, H, d, nq, s, window_frames, held,
                                             key_counts, scale, lse, workspace, workspace_bytes);
    if (st != RA_OK)
        return st;
    const Plan pl = plan_of(B, H, d, nq, held * s);
    const bool pair = split_p(held * s);
    const long long rows = static_cast<long long>(B) * H * nq;
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
    p.B = B;
    p.H = H;
    p.nq = nq;
    p.s = s;
    p.W = window_frames;
    p.blocks = cache8_blocks(s);
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
        p.skip_on_error = true;
        if ((st = device_error_word(&p.err)) != RA_OK || (st = cache8_tiles(p, B, d, pl.one, pair, cs)) != RA_OK)
            return st;
    } else {
        if ((st = bounds_word(&p.err)) != RA_OK)
            return st;
        const dim3 grid(static_cast<unsigned>(pl.q_tiles) * pl.splits, H, B);
        auto kernel = rows_kernel(d, nq <= COLS, pl.ahead, nq <= COLS / 2 ? P_COLUMNS : pair ? P_PAIR : P_BF16);
        kernel<<<grid, WARPS * 32, 0, cs>>>(p);
        RA_CUDA_TRY(cudaGetLastError());
    }
    if (pl.splits == 1)
        return RA_OK;
    const dim3 joins(static_cast<unsigned>((rows + 3) / 4));
    return launch_behind("cache8_join_kernel launch", d == 64 ? cache8_join_kernel<64> : cache8_join_kernel<128>, joins,
                         dim3(128), cs, p, rows);
}
