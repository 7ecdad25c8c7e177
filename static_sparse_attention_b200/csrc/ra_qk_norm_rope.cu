// ra_qk_norm_rope.cu -- what stands between the Q and K projections and the
// attention: the RMS norm of every head's row and its rotation by the token's
// position in time, height and width, in one pass that also turns the
// projection's token-major rows into the attention's [B, H, n, d]; and the
// gradient of that pass.
//
// Forward, per row x of d channels:  y = R(position) (x * r * w),  r = 1 / sqrt(mean(x^2) + eps).
// Backward, per row:  g = R^T dy;  xh = x * r;  a = g * w;
//   dx = r * (a - xh * mean(a * xh)),   dw = sum over batch, tokens and heads of g * xh.
// Nothing is kept from the forward: r is recomputed from x, which the backward
// has to read anyway.  Both are bound by memory: 4 bytes a value forward (read
// x, write y), 6 backward (read x and dy, write dx).
//
// A row is held by d / 8 lanes, 16 bytes each (ra_head_rows.cuh).  A lane stays
// with its token and walks heads, so the cosines and sines of a token are
// loaded once for many rows, which are fetched HEADS_IN_FLIGHT at a time.
//
// Measured: 108000 tokens, q and k of 24 heads of 128, 428 us = 6.2 TB/s, 95 % of the
// measured copy rate (DRAM traffic 2.60 GB of 2.65); backward of 63960 tokens, 40 heads
// of 128, 702 us = 5.6 TB/s, 85 % (24 warps an SM; issue slots 68 % busy).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "ra_head_rows.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int THREADS = 256;
constexpr int HEADS_IN_FLIGHT = 4;  // rows loaded before the first is used
// The backward keeps 24 warps an SM: at 16 (122 registers a thread, nothing asked of
// the compiler) 63960 tokens of 40 heads of 128 take 778 us, at 24 (85 registers)
// 690, at 32 (64 registers, spills) 830.
constexpr int BWD_BLOCKS_PER_SM = 3;
constexpr int BWD_BLOCKS = 148 * BWD_BLOCKS_PER_SM;  // and as many partial sums of a weight's gradient
constexpr int FWD_SLOTS = 148 * 5;

// One of the two tensors (q or k) of a call.
struct Rows {
    const __nv_bfloat16* x;  // [B, n, H, d] by strides (elements), channels contiguous
    long long sb, sn, sh;
    const void* weight;  // [d], null: no norm
    int weight_fp32;
    int H;
    int chunks;              // ceil(H / heads per chunk)
    __nv_bfloat16* y;        // forward: [B, H, n, d]
    const __nv_bfloat16* dy; // backward: [B, H, n, d]
    __nv_bfloat16* dx;       // backward: [B, n, H, d] by strides
    long long gb, gn, gh;
    float* dw_part;          // backward: [blocks][d], null: no weight
    float* dw;               // [d]
    long long x_size, y_size, dx_size;  // elements that x, y (and dy) and dx span
};

struct Params {
    Rows t[2];
    RopeArgs rope;
    int n, B, tiles;  // tiles: token tiles of one batch element
    int heads;        // heads per chunk
    float eps;
    int* err;         // debug build: see ra_bounds.cuh
};

// Which of a row's channel pairs are rotated: an instance each, since the third costs
// registers (108000 tokens, 24 heads of 128 take 48 a thread with all pairs turned, 58
// with a choice in the loop: one block an SM less).
enum class Turn { NONE, ALL, SOME };

// Turns a lane's eight channels; in the third form those of its first `turned` pairs.
template <Turn T, typename Rotate>
__device__ __forceinline__ void turn_pairs(Rotate&& rotate_by, int turned, float (&x)[8])
{
    if (T == Turn::NONE)
        return;
    float before[8];
    if (T == Turn::SOME) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            before[j] = x[j];
    }
    rotate_by(x);
    if (T == Turn::SOME)
        keep_unturned(before, turned, x);
}

template <int D, Turn T>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const Params p)
{
    constexpr int LPR = D / 8, TOKENS = THREADS / LPR;
    const int which = blockIdx.y >= static_cast<unsigned>(p.t[0].chunks) ? 1 : 0;
    const Rows& t = p.t[which];
    const int h0 = (static_cast<int>(blockIdx.y) - (which ? p.t[0].chunks : 0)) * p.heads;
    const int h1 = min(h0 + p.heads, t.H);
    const int b = blockIdx.z;
    const int sub = threadIdx.x % LPR;
    const int i = static_cast<int>(blockIdx.x) * TOKENS + static_cast<int>(threadIdx.x) / LPR;
    const bool live = i < p.n;
    const bool norm = t.weight != nullptr;
    const int turned = turned_pairs(p.rope, sub);
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (norm)
        load_weight(t.weight, t.weight_fp32, sub, w);
    float2 cs[4] = {{1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}};
    if (T != Turn::NONE && live)
        load_rope(p.rope, i, sub, cs);
    const __nv_bfloat16* x = t.x + b * t.sb + (live ? i : 0) * t.sn + sub * 8;
    __nv_bfloat16* y = t.y + (static_cast<long long>(b) * t.H * p.n + (live ? i : 0)) * D + sub * 8;
    for (int h = h0; h < h1; h += HEADS_IN_FLIGHT) {
        uint4 v[HEADS_IN_FLIGHT];
#pragma unroll
        for (int u = 0; u < HEADS_IN_FLIGHT; ++u) {
            v[u] = make_uint4(0, 0, 0, 0);
            if (live && h + u < h1 && inside(p.err, x + (h + u) * t.sh - t.x, 8, t.x_size, SITE_I_IN))
                v[u] = __ldcs(reinterpret_cast<const uint4*>(x + (h + u) * t.sh));
        }
#pragma unroll
        for (int u = 0; u < HEADS_IN_FLIGHT; ++u) {
            if (h + u >= h1)  // the same for the whole block
                break;
            float f[8];
            unpack_bf16x8(v[u], f);
            if (norm)
                rms_norm<D>(f, w, p.eps);
            turn_pairs<T>([&](float (&u)[8]) { rotate(cs, u); }, turned, f);
            if (live && inside(p.err, y + static_cast<long long>(h + u) * p.n * D - t.y, 8, t.y_size, SITE_I_OUT))
                *reinterpret_cast<uint4*>(y + static_cast<long long>(h + u) * p.n * D) = pack_bf16x8(f);
        }
    }
}

template <int D, Turn T>
__global__ void __launch_bounds__(THREADS, BWD_BLOCKS_PER_SM) qk_norm_rope_bwd_kernel(const Params p)
{
    constexpr int LPR = D / 8, TOKENS = THREADS / LPR;
    const Rows& t = p.t[blockIdx.y];
    if (t.dw_part)  // the sum of the blocks' parts is launched behind this kernel
        let_next_launch();
    const int sub = threadIdx.x % LPR;
    const int tok = static_cast<int>(threadIdx.x) / LPR;
    const bool norm = t.weight != nullptr;
    const int turned = turned_pairs(p.rope, sub);
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (norm)
        load_weight(t.weight, t.weight_fp32, sub, w);
    // work item: (batch element, token tile, head chunk), head chunks innermost
    const long long items = static_cast<long long>(p.B) * p.tiles * t.chunks;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int chunk = static_cast<int>(it % t.chunks);
        const long long bt = it / t.chunks;
        const int tile = static_cast<int>(bt % p.tiles), b = static_cast<int>(bt / p.tiles);
        const int h0 = chunk * p.heads, h1 = min(h0 + p.heads, t.H);
        const int i = tile * TOKENS + tok;
        const bool live = i < p.n;
        float2 cs[4] = {{1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}, {1.f, 0.f}};
        if (T != Turn::NONE && live)
            load_rope(p.rope, i, sub, cs);
        const long long row = live ? i : 0;
        const __nv_bfloat16* x = t.x + b * t.sb + row * t.sn + sub * 8;
        const __nv_bfloat16* dy = t.dy + (static_cast<long long>(b) * t.H * p.n + row) * D + sub * 8;
        __nv_bfloat16* dx = t.dx + b * t.gb + row * t.gn + sub * 8;
        for (int h = h0; h < h1; h += HEADS_IN_FLIGHT) {
            uint4 vx[HEADS_IN_FLIGHT], vg[HEADS_IN_FLIGHT];
#pragma unroll
            for (int u = 0; u < HEADS_IN_FLIGHT; ++u) {
                vx[u] = vg[u] = make_uint4(0, 0, 0, 0);
                if (live && h + u < h1 &&
                    inside(p.err, dy + static_cast<long long>(h + u) * p.n * D - t.dy, 8, t.y_size, SITE_I_GRAD_IN) &&
                    (!norm || inside(p.err, x + (h + u) * t.sh - t.x, 8, t.x_size, SITE_I_IN))) {
                    vg[u] = __ldcs(reinterpret_cast<const uint4*>(dy + static_cast<long long>(h + u) * p.n * D));
                    if (norm)
                        vx[u] = __ldcs(reinterpret_cast<const uint4*>(x + (h + u) * t.sh));
                }
            }
#pragma unroll
            for (int u = 0; u < HEADS_IN_FLIGHT; ++u) {
                if (h + u >= h1)  // the same for the whole block
                    break;
                float g[8];
                unpack_bf16x8(vg[u], g);
                turn_pairs<T>([&](float (&u)[8]) { rotate_back(cs, u); }, turned, g);
                if (norm) {
                    float f[8], ss = 0.f, ax = 0.f;
                    unpack_bf16x8(vx[u], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        ss = fmaf(f[j], f[j], ss);
                        ax = fmaf(g[j] * w[j], f[j], ax);
                    }
                    ss = row_sum<LPR>(ss);
                    ax = row_sum<LPR>(ax);
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
                    const float c = r * (r * (ax * (1.f / D)));  // dx = r * (a - x * c); r^2 alone may overflow
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dw[j] = fmaf(g[j], f[j] * r, dw[j]);
                        g[j] = r * fmaf(-f[j], c, g[j] * w[j]);
                    }
                }
                if (live && inside(p.err, dx + (h + u) * t.gh - t.dx, 8, t.dx_size, SITE_I_GRAD_OUT))
                    *reinterpret_cast<uint4*>(dx + (h + u) * t.gh) = pack_bf16x8(g);
            }
        }
    }
    if (!t.dw_part)
        return;
    // the block's sum of dw: over its TOKENS rows in shared memory, in a fixed order
    __shared__ float part[TOKENS][D];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        part[tok][sub * 8 + j] = dw[j];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < TOKENS; ++r)
            s += part[r][threadIdx.x];
        if (inside(p.err, static_cast<long long>(blockIdx.x) * D + threadIdx.x, 1, BWD_BLOCKS * D, SITE_I_PART))
            t.dw_part[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = s;
    }
}

// dw[c] = sum over the blocks' partial sums, in a fixed order (deterministic, no atomics).
template <int D>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const Params p, int blocks)
{
    constexpr int G = 1024 / D;
    wait_for_previous();
    const Rows& t = p.t[blockIdx.x];
    if (!t.dw_part)
        return;
    __shared__ float part[G][D];
    const int c = threadIdx.x % D, g = threadIdx.x / D;
    float s = 0.f;
    for (int k = g; k < blocks; k += G)
        if (inside(p.err, static_cast<long long>(k) * D + c, 1, BWD_BLOCKS * D, SITE_I_PART))
            s += t.dw_part[static_cast<size_t>(k) * D + c];
    part[g][c] = s;
    __syncthreads();
    if (g == 0) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < G; ++k)
            s += part[k][c];
        t.dw[c] = s;
    }
}

// cos and sin of position * base^(-2 i / dim), the angle in 64 bits: at position
// 10^5 an fp32 angle would be off by up to 2^-8.
__global__ void rope_table_kernel(float2* table, int start, int length, int pairs, double log2_base)
{
    const long long k = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (k >= static_cast<long long>(length) * pairs)
        return;
    const int i = static_cast<int>(k % pairs);
    const double pos = static_cast<double>(start) + static_cast<double>(k / pairs);
    double sn, cs;
    sincos(pos * exp2(-log2_base * i / pairs), &sn, &cs);
    table[k] = make_float2(static_cast<float>(cs), static_cast<float>(sn));
}

ra_status check_strides(const char* what, long long* sb, long long* sn, long long* sh, int B, int n, int H)
{
    long long* s[3] = {sb, sn, sh};
    const int size[3] = {B, n, H};
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 1)
            *s[i] = 0;  // never used
        if (*s[i] < 0 || *s[i] % 8 != 0 || *s[i] > (1LL << 46) / (size[i] > 1 ? size[i] : 1))
            return fail(RA_ERR_INVALID_ARG,
                        "%s strides must be multiples of 8 elements, >= 0, and span at most 2^46 elements", what);
    }
    return RA_OK;
}

// Whether blocks of `row` contiguous elements, one for each index of up to four
// dimensions, certainly share none: sorted by stride, each dimension steps over the
// whole of the ones below it.
struct Dim {
    long long stride;
    int size;
};
template <int N>
bool blocks_disjoint(Dim (&dims)[N], long long row)
{
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j)
            if (dims[j].stride < dims[i].stride ||
                (dims[j].stride == dims[i].stride && dims[j].size < dims[i].size)) {
                const Dim a = dims[i];
                dims[i] = dims[j];
                dims[j] = a;
            }
    long long below = row;
    for (const Dim& dim : dims) {
        if (dim.size == 1)
            continue;
        if (dim.stride < below)
            return false;
        below = dim.stride * (dim.size - 1) + below;
    }
    return true;
}

// The rows of a strided output.
bool rows_disjoint(const Rows& t, int B, int n, int d)
{
    Dim dims[3] = {{t.gb, B}, {t.gn, n}, {t.gh, t.H}};
    return blocks_disjoint(dims, d);
}

// Whether the strided tensors dq and dk (bf16 elements), the rows of each disjoint,
// certainly share none: apart altogether, or slots of one packed buffer -- of each
// token's row (the output of a fused projection, [B, n, Hq + Hk + .., d]), or with as
// many heads of the same stride, dk as dq's second index ([B, n, H, 2 or 3, d],
// [B, 2 H, n, d] and the like).
bool grads_disjoint(const Rows& q, const Rows& k, int B, int n, int d)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(q.dx), c = reinterpret_cast<uintptr_t>(k.dx);
    if (!overlap(span(q.dx, extent(q.gb, q.gn, q.gh, B, n, q.H, d)), span(k.dx, extent(k.gb, k.gn, k.gh, B, n, k.H, d))))
        return true;
    if (q.gb != k.gb || q.gn != k.gn)
        return false;
    const long long apart = static_cast<long long>(a < c ? c - a : a - c) / 2;
    const Rows &lo = a < c ? q : k, &hi = a < c ? k : q;
    // a token's slots as one block, from the first one's start to the second one's end
    Dim tokens[2] = {{q.gb, B}, {q.gn, n}};
    if (apart >= (lo.H - 1) * lo.gh + d && blocks_disjoint(tokens, apart + (hi.H - 1) * hi.gh + d))
        return true;
    Dim rows[4] = {{q.gb, B}, {q.gn, n}, {q.gh, q.H}, {apart, 2}};
    return q.gh == k.gh && q.H == k.H && blocks_disjoint(rows, d);
}

}  // namespace

ra_status rope_args(const ra_rope* rope, int frame0, int n, int d, RopeArgs* out)
{
    std::memset(out, 0, sizeof *out);
    out->grid_h = out->grid_w = 1;
    if (!rope)
        return RA_OK;
    const int pairs[3] = {rope->t_pairs, rope->h_pairs, rope->w_pairs};
    const float* tables[3] = {rope->t, rope->h, rope->w};
    long long total = 0;
    for (int i = 0; i < 3; ++i) {
        if (pairs[i] < 0 || pairs[i] > d / 2)
            return fail(RA_ERR_INVALID_ARG, "channel pairs of an axis must be in [0, d / 2]");
        if (pairs[i] && (!tables[i] || reinterpret_cast<uintptr_t>(tables[i]) % 8))
            return fail(RA_ERR_INVALID_ARG, "a rope table is NULL or not 8-byte aligned");
        total += pairs[i];
    }
    if (total < 1 || total > d / 2)
        return fail(RA_ERR_INVALID_ARG, "the axes' channel pairs must add up to 1 .. d / 2 (%lld of %d)", total, d / 2);
    if (rope->frames < 1 || rope->grid_h < 1 || rope->grid_w < 1 ||
        static_cast<long long>(rope->grid_h) * rope->grid_w > (1LL << 31) - 1)
        return fail(RA_ERR_INVALID_ARG, "rope grid sizes must be >= 1 and grid_h * grid_w below 2^31");
    const long long s = static_cast<long long>(rope->grid_h) * rope->grid_w;
    if (frame0 < 0 || frame0 + (n + s - 1) / s > rope->frames)
        return fail(RA_ERR_INVALID_ARG, "frames %d .. %lld are outside the time table of %d frames", frame0,
                    frame0 + (n + s - 1) / s - 1, rope->frames);
    // an axis without pairs never reads its table; a non-null t says that there is a rotation
    const float* any = tables[0] ? tables[0] : (tables[1] ? tables[1] : tables[2]);
    out->t = reinterpret_cast<const float2*>(tables[0] ? tables[0] : any);
    out->h = reinterpret_cast<const float2*>(tables[1] ? tables[1] : any);
    out->w = reinterpret_cast<const float2*>(tables[2] ? tables[2] : any);
    out->t_pairs = pairs[0];
    out->h_pairs = pairs[1];
    out->w_pairs = pairs[2];
    out->grid_h = rope->grid_h;
    out->grid_w = rope->grid_w;
    out->first = frame0;
    out->frames = rope->frames;
    return bounds_word(&out->err);
}

ra_status head_rows_args(const char* what, const ra_head_rows* r, int B, int n, int d, long long* sb, long long* sn,
                         long long* sh)
{
    if (!r->x)
        return fail(RA_ERR_INVALID_ARG, "NULL %s pointer", what);
    if (r->heads < 1 || r->heads > 65535)
        return fail(RA_ERR_INVALID_ARG, "%s heads must be in [1, 65535] (%d)", what, r->heads);
    if (!aligned16(r->x) || (r->weight && !aligned16(r->weight)))
        return fail(RA_ERR_INVALID_ARG, "%s and its weight must be 16-byte aligned", what);
    *sb = r->stride_b;
    *sn = r->stride_n;
    *sh = r->stride_h;
    (void)d;
    return check_strides(what, sb, sn, sh, B, n, r->heads);
}

namespace {

ra_status check_sizes(int B, int n, int d, float eps)
{
    if (B < 1 || B > 65535)
        return fail(RA_ERR_INVALID_ARG, "B must be in [1, 65535] (B=%d)", B);
    if (n < 0)
        return fail(RA_ERR_INVALID_ARG, "n must be >= 0");
    if (d != 64 && d != 128)
        return fail(RA_ERR_UNSUPPORTED, "head dim %d is not supported (64 or 128)", d);
    if (!(eps > 0.f) || !std::isfinite(eps))
        return fail(RA_ERR_INVALID_ARG, "eps must be finite and > 0");
    return RA_OK;
}

// Heads that a lane walks for one token: all of them when there are tokens enough (a
// token's rows are then read in one stretch: 63960 tokens of 40 heads of 128 backward
// 704 us against 758 with 8 heads at a time), else as many as cost least, in rounds
// of the `slots` blocks that run at once (whole rounds where the blocks stay and take
// several items each) times the batches of loads that a lane waits for, with a
// quarter of one for the look-up of its angles.  (The backward plans each of its two
// tensors as if it had all BWD_BLOCKS places, which the two share: one frame's rows, 792
// blocks on 444 places, take 28.6 us of 14.8.)
int heads_per_chunk(long long tiles, int B, int H, int slots, bool whole_rounds)
{
    int best = H;
    double least = 0;
    for (int c = 1; c <= H && c <= 64; ++c) {
        const int heads = (H + c - 1) / c;
        const long long blocks = tiles * B * ((H + heads - 1) / heads);
        double rounds = static_cast<double>(blocks) / slots;
        rounds = whole_rounds ? std::ceil(rounds) : (rounds > 1 ? rounds : 1);
        const double cost = rounds * ((heads + HEADS_IN_FLIGHT - 1) / HEADS_IN_FLIGHT + 0.25);
        if (c == 1 || cost < least) {
            least = cost;
            best = heads;
        }
    }
    return best;
}

ra_status fill(Params* p, const ra_head_rows* q, const ra_head_rows* k, int B, int n, int d, const ra_rope* rope,
               int frame0, float eps, int slots, bool whole_rounds)
{
    std::memset(p, 0, sizeof *p);
    ra_status st = rope_args(rope, frame0, n, d, &p->rope);
    if (st != RA_OK)
        return st;
    const ra_head_rows* in[2] = {q, k};
    const char* name[2] = {"q", "k"};
    const int tokens = THREADS / (d / 8);
    p->n = n;
    p->B = B;
    p->tiles = (n + tokens - 1) / tokens;
    p->eps = eps;
    int H = 0;
    for (int i = 0; i < 2; ++i) {
        if (!in[i])
            continue;
        Rows& t = p->t[i];
        if ((st = head_rows_args(name[i], in[i], B, n, d, &t.sb, &t.sn, &t.sh)) != RA_OK)
            return st;
        if (!in[i]->weight && !rope)
            return fail(RA_ERR_INVALID_ARG, "%s has neither a norm weight nor a rotation", name[i]);
        t.x = static_cast<const __nv_bfloat16*>(in[i]->x);
        t.weight = in[i]->weight;
        t.weight_fp32 = in[i]->weight_fp32;
        t.H = in[i]->heads;
        t.x_size = extent(t.sb, t.sn, t.sh, B, n, t.H, d) / 2;
        t.y_size = static_cast<long long>(B) * t.H * n * d;
        H = t.H > H ? t.H : H;
    }
    if (static_cast<long long>(B) * H * n > (1LL << 40))
        return fail(RA_ERR_UNSUPPORTED, "tensor too large");
    p->heads = heads_per_chunk(p->tiles, B, H, slots, whole_rounds);
    for (int i = 0; i < 2; ++i)
        p->t[i].chunks = (p->t[i].H + p->heads - 1) / p->heads;
    return bounds_word(&p->err);
}

using Kernel = void (*)(const Params);
template <int D>
Turn turn_of(const RopeArgs& r)
{
    return !r.t ? Turn::NONE : r.t_pairs + r.h_pairs + r.w_pairs == D / 2 ? Turn::ALL : Turn::SOME;
}
template <int D>
Kernel forward_kernel(const RopeArgs& r)
{
    const Turn t = turn_of<D>(r);
    return t == Turn::NONE  ? qk_norm_rope_kernel<D, Turn::NONE>
           : t == Turn::ALL ? qk_norm_rope_kernel<D, Turn::ALL>
                            : qk_norm_rope_kernel<D, Turn::SOME>;
}
template <int D>
Kernel backward_kernel(const RopeArgs& r)
{
    const Turn t = turn_of<D>(r);
    return t == Turn::NONE  ? qk_norm_rope_bwd_kernel<D, Turn::NONE>
           : t == Turn::ALL ? qk_norm_rope_bwd_kernel<D, Turn::ALL>
                            : qk_norm_rope_bwd_kernel<D, Turn::SOME>;
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" ra_status ra_rope_table(float* table, int start, int length, int pairs, double base, ra_stream stream)
{
    if (!table || reinterpret_cast<uintptr_t>(table) % 8)
        return fail(RA_ERR_INVALID_ARG, "the table is NULL or not 8-byte aligned");
    if (start < 0 || length < 1 || pairs < 1 || pairs > 64)
        return fail(RA_ERR_INVALID_ARG, "start >= 0, length >= 1 and pairs in [1, 64] are required");
    if (static_cast<long long>(start) + length > (1LL << 31) - 1)
        return fail(RA_ERR_INVALID_ARG, "positions must stay below 2^31");
    if (!(base > 1.0) || !std::isfinite(base))
        return fail(RA_ERR_INVALID_ARG, "base must be finite and > 1");
    const long long blocks = (static_cast<long long>(length) * pairs + 255) / 256;
    rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<float2*>(table), start, length, pairs, std::log2(base));
    return cuda_fail(cudaGetLastError(), "rope_table_kernel launch");
}

extern "C" ra_status ra_qk_norm_rope(const ra_head_rows* q, const ra_head_rows* k, void* q_out, void* k_out, int B,
                                     int n, int d, const ra_rope* rope, int frame0, float eps, ra_stream stream)
{
    if (!q)
        return fail(RA_ERR_INVALID_ARG, "NULL q");
    if (!q_out || (k && !k_out))
        return fail(RA_ERR_INVALID_ARG, "NULL output pointer");
    if (!aligned16(q_out) || !aligned16(k_out))
        return fail(RA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    ra_status st = check_sizes(B, n, d, eps);
    if (st != RA_OK)
        return st;
    Params p;
    if ((st = fill(&p, q, k, B, n, d, rope, frame0, eps, k ? FWD_SLOTS / 2 : FWD_SLOTS, false)) != RA_OK)
        return st;
    if (n == 0)
        return RA_OK;
    void* out[2] = {q_out, k ? k_out : nullptr};
    Span out_span[2];
    for (int i = 0; i < 2; ++i) {
        out_span[i] = span(out[i], static_cast<long long>(B) * p.t[i].H * n * d * 2);
        p.t[i].y = static_cast<__nv_bfloat16*>(out[i]);
    }
    bool bad = overlap(out_span[0], out_span[1]);
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) {
            const Rows& t = p.t[j];
            bad |= overlap(out_span[i], span(t.x, t.x ? extent(t.sb, t.sn, t.sh, B, n, t.H, d) : 0)) ||
                   overlap(out_span[i], span(t.weight, d * (t.weight_fp32 ? 4 : 2)));
        }
    if (bad)
        return fail(RA_ERR_INVALID_ARG, "an output may not alias another buffer of the call");
    const dim3 grid(p.tiles, p.t[0].chunks + p.t[1].chunks, B);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    auto kernel = d == 64 ? forward_kernel<64>(p.rope) : forward_kernel<128>(p.rope);
    kernel<<<grid, THREADS, 0, cs>>>(p);
    return cuda_fail(cudaGetLastError(), "qk_norm_rope_kernel launch");
}

extern "C" size_t ra_qk_norm_rope_bwd_workspace_bytes(int d)
{
    return d == 64 || d == 128 ? static_cast<size_t>(2) * BWD_BLOCKS * d * sizeof(float) : 0;
}

extern "C" ra_status ra_qk_norm_rope_bwd(const ra_head_rows* q, const ra_head_rows* k, const ra_head_grads* dq,
                                         const ra_head_grads* dk, int B, int n, int d, const ra_rope* rope, int frame0,
                                         float eps, void* workspace, size_t workspace_bytes, ra_stream stream)
{
    if (!q || !dq || (k && !dk))
        return fail(RA_ERR_INVALID_ARG, "NULL argument");
    ra_status st = check_sizes(B, n, d, eps);
    if (st != RA_OK)
        return st;
    Params p;
    if ((st = fill(&p, q, k, B, n, d, rope, frame0, eps, BWD_BLOCKS, true)) != RA_OK)
        return st;
    const ra_head_grads* grads[2] = {dq, k ? dk : nullptr};
    const char* name[2] = {"dq", "dk"};
    Span outs[5], ins[6];
    int n_out = 0, n_in = 0;
    bool weights = false;
    for (int i = 0; i < 2; ++i) {
        if (!grads[i])
            continue;
        Rows& t = p.t[i];
        const ra_head_grads* g = grads[i];
        if (!g->dy || !g->dx)
            return fail(RA_ERR_INVALID_ARG, "NULL %s pointer", name[i]);
        if (!aligned16(g->dy) || !aligned16(g->dx))
            return fail(RA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
        if ((t.weight != nullptr) != (g->dweight != nullptr))
            return fail(RA_ERR_INVALID_ARG, "%s: a weight and its gradient's pointer go together", name[i]);
        if (reinterpret_cast<uintptr_t>(g->dweight) % 4)
            return fail(RA_ERR_INVALID_ARG, "%s: the weight's gradient must be 4-byte aligned", name[i]);
        t.gb = g->stride_b;
        t.gn = g->stride_n;
        t.gh = g->stride_h;
        if ((st = check_strides(name[i], &t.gb, &t.gn, &t.gh, B, n, t.H)) != RA_OK)
            return st;
        if (n > 0 && !rows_disjoint(t, B, n, d))
            return fail(RA_ERR_INVALID_ARG, "%s: rows of an output overlap", name[i]);
        t.dy = static_cast<const __nv_bfloat16*>(g->dy);
        t.dx = static_cast<__nv_bfloat16*>(g->dx);
        t.dw = g->dweight;
        t.dx_size = extent(t.gb, t.gn, t.gh, B, n, t.H, d) / 2;
        weights |= t.dw != nullptr;
        if (n > 0) {
            outs[n_out++] = span(t.dx, extent(t.gb, t.gn, t.gh, B, n, t.H, d));
            ins[n_in++] = span(t.x, extent(t.sb, t.sn, t.sh, B, n, t.H, d));
            ins[n_in++] = span(t.dy, static_cast<long long>(B) * t.H * n * d * 2);
        }
        ins[n_in++] = span(t.weight, d * (t.weight_fp32 ? 4 : 2));
    }
    if (weights) {
        if (!workspace || workspace_bytes < ra_qk_norm_rope_bwd_workspace_bytes(d) || !aligned16(workspace))
            return fail(RA_ERR_INVALID_ARG, "the workspace needs %zu bytes, 16-byte aligned",
                        ra_qk_norm_rope_bwd_workspace_bytes(d));
        outs[n_out++] = span(workspace, static_cast<long long>(ra_qk_norm_rope_bwd_workspace_bytes(d)));
    }
    // dq and dk may be slots of one packed buffer (their spans interleave), but
    // not the same rows; everything else is apart.
    bool bad = k && n > 0 && !grads_disjoint(p.t[0], p.t[1], B, n, d);
    Span small[2] = {span(p.t[0].dw, d * 4), span(p.t[1].dw, d * 4)};
    bad |= overlap(small[0], small[1]);
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            bad |= overlap(outs[i], ins[j]);
        bad |= overlap(outs[i], small[0]) || overlap(outs[i], small[1]);
        if (weights && i + 1 < n_out)
            bad |= overlap(outs[i], outs[n_out - 1]);
    }
    for (int j = 0; j < n_in; ++j)
        bad |= overlap(ins[j], small[0]) || overlap(ins[j], small[1]);
    if (bad)
        return fail(RA_ERR_INVALID_ARG, "an output may not alias another buffer of the call");
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) {  // no rows: the weights' gradients are zero
        for (int i = 0; i < 2; ++i)
            if (p.t[i].dw)
                RA_CUDA_TRY(cudaMemsetAsync(p.t[i].dw, 0, d * sizeof(float), cs));
        return RA_OK;
    }
    long long items = 0;
    for (int i = 0; i < 2; ++i) {
        const long long mine = static_cast<long long>(B) * p.tiles * p.t[i].chunks;
        items = mine > items ? mine : items;
        if (p.t[i].dw)
            p.t[i].dw_part = static_cast<float*>(workspace) + static_cast<size_t>(i) * BWD_BLOCKS * d;
    }
    const int blocks = static_cast<int>(items < BWD_BLOCKS ? items : BWD_BLOCKS);
    const dim3 grid(blocks, k ? 2 : 1);
    auto kernel = d == 64 ? backward_kernel<64>(p.rope) : backward_kernel<128>(p.rope);
    kernel<<<grid, THREADS, 0, cs>>>(p);
    RA_CUDA_TRY(cudaGetLastError());
    if (!weights)
        return RA_OK;
    return launch_behind("weight_grad_kernel launch", d == 64 ? weight_grad_kernel<64> : weight_grad_kernel<128>,
                         dim3(k ? 2 : 1), dim3(1024), cs, p, blocks);
}
