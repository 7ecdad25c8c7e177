// ra_cache8_tiles.cu -- attention of many queries over the 8-bit key/value ring
// on the tensor cores (tcgen05, accumulators in TMEM).
//
// One CTA per (head, 256 queries, range of keys), or 128 queries (see ONE below), one
// CTA per SM, keys in steps of 64.  Five warpgroups in fixed roles:
//   warps 0-3, 4-7  softmax of query tile 0 and 1 (128 rows each): thread t of the
//                   group owns row t (TMEM lane t); per step reads S, keeps the
//                   running maximum and sum, writes P (bf16) back over S; at the end
//                   the epilogue.
//   warps 18, 19    fetch, a step each in turn: bulk copies of a step's codes (its 64
//                   rows of K, and of V, are contiguous) into a ring of shared memory,
//                   RAW steps ahead; the lanes turn the rows' scales into the factors
//                   of the conversion.
//   warps 8-15      convert: codes become code * scale in bf16 -- exactly, see
//                   ra_cache8.cuh -- in the MMA's 128-byte swizzle, in a ring of K
//                   stages and one of V stages.
//   warps 16, 17    MMA of tile 0 and 1 (16 allocates TMEM): one elected lane issues
//                   S_h = Q K_h^T (N = 64) into S buffer h % 2 and O += P_h V_h, in
//                   the order S_0, S_1, PV_0, S_2, PV_1, S_3, ...
// Two query tiles share one conversion: 4.5 integer and multiply instructions for two
// codes, 1400 warp instructions for a step of 64 keys of 128 channels, beside 2900 for
// the softmax of 2 x 128 x 64 scores and 1280 clocks of the tensor pipe.
//
// Measured: 1560 queries, 24960 keys, 40 heads of 128 (280 CTAs, two rounds of SMs)
// 895 us in a run of 30 calls = 891 TFLOP/s, 55 % of the measured bf16 burst (921 with
// rings that change from call to call; 827 on another GPU); 2000 clocks a step, issue
// slots 67 %, exp2 and tensor pipes half busy each.  What a step waits for is the
// softmax warps' own chain (1500 clocks of exponentials with the convert warps beside
// them, 400 of barriers and TMEM).  On the way: one MMA warp for both tiles 1134 us (its
// waits, 100-200 clocks each, stood between one tile's products and the other's), four
// convert warps 918.
//
// Up to 128 queries, and more where that is sooner done, are one tile a block (ONE).
// Its steps are taken in turn by the two
// softmax groups and MMA warps, each with its own maximum, sum and O, which group 0
// joins to its own at the end.  With one group at work and one fetch warp a step took
// 1700 clocks; turns alone changed nothing, a fetch warp's own chain (waits, indexes,
// factors) being as long.  With both, a step is 1000 clocks at 64 channels (issue
// slots 67 %) and 1500 at 128, where the conversion is the longest (without it 1150).
// 32 queries, 12480 keys: 80 heads of 64 113 -> 88 us, 192 heads of 128 269 -> 247.
// All 128 rows of the tile are computed, however few of them are queries.
//
// A word of four codes is turned into two pairs, channels (0, 2) and (1, 3), which
// saves the byte permutes.  So channels lie in the order 0, 2, 1, 3 within every
// four in shared memory: Q is stored in the same order (S does not depend on it),
// and the epilogue puts O's columns, which follow V's, back.
//
// S_{h+2} overwrites the TMEM columns whose P the P V of step h reads.  The PTX
// ISA executes two tcgen05 operations of a thread in order for the pairs that it
// lists as pipelined; MMA -> shift and shift -> MMA are such pairs for any two of
// the same cta_group, so a tcgen05.shift of columns that S_{h+2} overwrites anyway
// orders it behind that P V.  O is rescaled only after the step before has
// completed.  Every wait is bounded (ra_sm100.cuh).
//
// The convert warps write K and V through the generic proxy and the MMA reads them
// through the async proxy: the proxy fence between the two stands in the MMA warp,
// behind its wait for the writers' barrier.
//
// (With the codes fetched by the convert warps' own loads, two steps ahead, these
// waited for their loads.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "ra_cache8_attention.cuh"
#include "ra_internal.h"
#include "ra_sm100.cuh"

namespace ra {
namespace {

constexpr int STEP = 64;           // keys of a step
constexpr int TILE_ROWS = 128;     // queries of a tile
constexpr int THREADS = 640;
constexpr int CONVERT_WARP = 8, MMA_WARP = 16, FETCH_WARP = 18;  // two warps each of MMA and fetch
// Registers a thread of each warpgroup keeps of the 96 that the block is launched
// with: the softmax holds 64 scores, P and its sums.
constexpr int SOFTMAX_REGS = 152, CONVERT_REGS = 56, MMA_REGS = 64;
static_assert(2 * SOFTMAX_REGS + 2 * CONVERT_REGS + MMA_REGS <= 5 * 96, "the split draws on the block's own registers");
constexpr uint32_t TMEM_COLS = 512;
// TMEM columns of a tile: S / P buffers 0 and 1 (64 fp32 columns each), then O.
__host__ __device__ constexpr uint32_t tile_col(int t) { return 256u * static_cast<uint32_t>(t); }
__host__ __device__ constexpr uint32_t s_col(int t, int buf) { return tile_col(t) + 64u * static_cast<uint32_t>(buf); }
__host__ __device__ constexpr uint32_t o_col(int t) { return tile_col(t) + 128u; }
// The running maximum (base 2) is raised only when a step exceeds it by more: P
// stays below 2^8, which fp32 and bf16 hold as precisely as values below 1.
constexpr float RAISE = 8.0f;

enum : int {
    SITE_RAW_EMPTY = 60, SITE_RAW_FULL, SITE_K_EMPTY, SITE_V_EMPTY, SITE_K_FULL, SITE_V_FULL, SITE_P_FULL, SITE_S_FULL,
    SITE_PV_DONE, SITE_O_FINAL, SITE_SMEM_ALIGN, SITE_B_KEYS
};

// ONE: a single tile of queries (see Turns).
template <int D, bool ONE>
struct Layout {
    static constexpr int CHUNKS = D / 64;                       // 128-byte swizzle atoms across d
    static constexpr int Q_CHUNK = TILE_ROWS * 128;             // bytes of 128 rows x 64 channels
    static constexpr int Q_TILE = CHUNKS * Q_CHUNK;
    static constexpr int KV_CHUNK = STEP * 128;
    static constexpr int KV_TILE = CHUNKS * KV_CHUNK;           // K or V of a step
    static constexpr int STAGES = ONE ? 4 : 3;                  // of K, and of V
    static constexpr int RAW = 4;                               // steps of codes
    static constexpr int RAW_TILE = STEP * D;                   // bytes of K's or V's codes of a step
    static constexpr int K_OFF = (ONE ? 1 : 2) * Q_TILE;
    static constexpr int V_OFF = K_OFF + STAGES * KV_TILE;
    static constexpr int RAW_OFF = V_OFF + STAGES * KV_TILE;    // [RAW][K, V]
    static constexpr int FACTOR_OFF = RAW_OFF + RAW * 2 * RAW_TILE;
    static constexpr int FACTORS = 2 * STEP + 4;                // words: of K's rows, of V's rows, the TWO flag
    static constexpr int BAR_OFF = FACTOR_OFF + RAW * FACTORS * 4;
    static constexpr int SMEM = BAR_OFF + 304;                  // barriers, the TMEM address, the abort flag
    static_assert(SMEM <= 227 * 1024, "one block's shared memory");
};

enum : int {
    B_K_FULL = 0,      // + stage (up to 4)
    B_V_FULL = 4,      // + stage
    B_K_EMPTY = 8,     // + stage
    B_V_EMPTY = 12,    // + stage
    B_RAW_FULL = 16,   // + raw stage
    B_RAW_EMPTY = 20,  // + raw stage
    B_S_FULL = 24,     // + 2 * tile + buffer
    B_P_FULL = 28,     // + 2 * tile + buffer
    B_PV_DONE = 32,    // + tile
    B_O_FINAL = 34,    // + tile
    B_COUNT = 36
};
constexpr int CONVERT_WARPS = 8;

// Arrivals that complete a phase of barrier i: the convert warps, a commit for each
// tile, the threads of a softmax warpgroup, or one thread (a tile's commit, the fetch).
__device__ __forceinline__ uint32_t arrivals(int i, int tiles)
{
    return i < B_K_EMPTY || (i >= B_RAW_EMPTY && i < B_S_FULL) ? CONVERT_WARPS
           : i < B_RAW_FULL                                    ? tiles
           : i >= B_P_FULL && i < B_PV_DONE                    ? 128u
                                                               : 1u;
}

// Contiguous copy of `bytes` (a multiple of 16) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// ---- packed fp32 pairs -------------------------------------------------------
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// p = 2^(s * c - m) of 32 columns, packed to bf16, summed into four pairs of
// accumulators; MAX also tracks the largest s, PAIR also returns what the rounding leaves.
template <bool MAX, bool PAIR>
__device__ __forceinline__ void exp_columns(const uint32_t (&s)[32], float c, float negm, uint64_t (&sum)[4],
                                            float (&top)[4], uint32_t (&p)[16], uint32_t (&rest)[16])
{
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float s0 = __uint_as_float(s[e]), s1 = __uint_as_float(s[e + 1]);
        if (MAX)
            top[(e >> 1) & 3] = max3(top[(e >> 1) & 3], s0, s1);
        float x0, x1;
        unpair(pair_fma(pair(s0, s1), pair(c, c), pair(negm, negm)), x0, x1);
        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
        sum[(e >> 1) & 3] = pair_add(sum[(e >> 1) & 3], pair(p0, p1));
        p[e >> 1] = pack_bf16(p0, p1);
        if (PAIR)
            rest[e >> 1] = pack_bf16(p0 - __uint_as_float(p[e >> 1] << 16),
                                     p1 - __uint_as_float(p[e >> 1] & 0xFFFF0000u));
    }
}

// Four codes to bf16 code * factor: channels (0, 2) in x, (1, 3) in y.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t factor, uint32_t& x, uint32_t& y)
{
    x = mul_bf16x2(e4m3x2_small(w << 8), factor);
    y = mul_bf16x2(e4m3x2_small(w), factor);
}

// What a convert thread takes of a step's K or V: 16 codes of row `row` and of every
// ROW_STEP-th behind it, and the rows' factors.
template <int D>
struct Codes {
    static constexpr int PER_ROW = D / 16;  // threads a row
    static constexpr int ROW_STEP = CONVERT_WARPS * 32 / PER_ROW;
    static constexpr int N = STEP / ROW_STEP;
    uint4 x[N];
    uint32_t f[N];
};

template <int D>
__device__ __forceinline__ void load_codes(Codes<D>& c, const uint8_t* raw, const uint32_t* factors, int row, int part)
{
#pragma unroll
    for (int i = 0; i < Codes<D>::N; ++i) {
        c.x[i] = *reinterpret_cast<const uint4*>(raw + (row + i * Codes<D>::ROW_STEP) * D + part * 16);
        c.f[i] = factors[row + i * Codes<D>::ROW_STEP];
    }
}

// Convert them into a stage.  TWO: some scale of the step needs its second factor.
template <int D, bool TWO>
__device__ __forceinline__ void store_codes(const Codes<D>& c, uint8_t* stage, int row, int part)
{
    using C = Codes<D>;
    // 16-byte units 2 part and 2 part + 1 of the row.  With eight threads a row the
    // upper four store theirs in the other order, so that the eight of a store fall
    // on different banks.  row and row + i * ROW_STEP have the same swizzle.
    static_assert(C::ROW_STEP % 8 == 0, "one swizzle for all rows of a thread");
    const int swap = D == 128 ? part >> 2 : 0;
    uint8_t* base = stage + (part >> 2) * (STEP * 128) + row * 128;
    uint8_t* at0 = base + (((2 * (part & 3) + swap) ^ (row & 7)) << 4);
    uint8_t* at1 = base + (((2 * (part & 3) + 1 - swap) ^ (row & 7)) << 4);
#pragma unroll
    for (int i = 0; i < C::N; ++i) {
        const uint32_t f = __byte_perm(c.f[i], 0, 0x1010);
        const uint32_t w[4] = {c.x[i].x, c.x[i].y, c.x[i].z, c.x[i].w};
        uint32_t out[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            codes4(w[j], f, out[2 * j], out[2 * j + 1]);
        if (TWO) {
            const uint32_t f2 = __byte_perm(c.f[i], 0, 0x3232);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                out[j] = mul_bf16x2(out[j], f2);
        }
        const uint4 lo = make_uint4(out[0], out[1], out[2], out[3]), hi = make_uint4(out[4], out[5], out[6], out[7]);
        *reinterpret_cast<uint4*>(at0 + i * C::ROW_STEP * 128) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(at1 + i * C::ROW_STEP * 128) = swap ? lo : hi;
    }
}

// The steps of the key range that tile t's softmax group and MMA warp take: all; or,
// with one tile of queries (ONE), every second one, so that both groups have work.
struct Turns {
    int first, stride, n;
    __device__ __forceinline__ int step(int i) const { return first + i * stride; }
};
template <bool ONE>
__device__ __forceinline__ Turns turns_of(int t, int n)
{
    return ONE ? Turns{t, 2, (n - t + 1) / 2} : Turns{0, 1, n};
}

template <int REGS>
__device__ __forceinline__ void shed_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}

// PAIR: P is kept as a pair of bf16 numbers, P = hi + lo to 2^-16 of a weight, and P V
// runs as two products (S is 64 fp32 columns, hi and lo 32 each).  1560 queries, 3120
// keys, 40 heads of 128: 150 us, with P as one number 128.
template <int D, bool ONE, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1) cache8_tiles_kernel(const AttnParams p)
{
    using L = Layout<D, ONE>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bars = sbase + L::BAR_OFF;
    auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::BAR_OFF + 8 * B_COUNT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::BAR_OFF + 8 * B_COUNT + 4);

    const int warp = threadIdx.x >> 5;
    const int split = static_cast<int>(blockIdx.x) % p.splits, q_tile = static_cast<int>(blockIdx.x) / p.splits;
    const int h = blockIdx.y, b = blockIdx.z;
    const long long bh = static_cast<long long>(b) * p.H + h;
    const int count = key_count(p, b);
    const int begin = split * p.chunk;
    if (p.splits > 1 && begin >= count)
        return;  // the join does not read this split
    const int end = min(begin + p.chunk, count);
    const int q0 = q_tile * (ONE ? 1 : 2) * TILE_ROWS;
    const int tiles = !ONE && p.nq - q0 > TILE_ROWS ? 2 : 1;
    WaitCtl wc{abort_flag, p.err, p.timeout_ns};
    if (p.splits > 1)
        let_next_launch();

    if (threadIdx.x == 0) {
        *abort_flag = *reinterpret_cast<volatile int*>(p.err) != 0 ? 1 : 0;
        if (sbase & 1023u)  // the swizzled tiles need 1024-byte alignment: record it, run nothing
            report_timeout(wc, SITE_SMEM_ALIGN);
        for (int i = 0; i < B_COUNT; ++i)
            mbar_init(bar(i), arrivals(i, tiles));
        fence_barrier_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    // Q, zeros behind the last query, in the order of channels that K has
    constexpr int UNITS = D / 8, LOADS = 4;  // 16-byte units of a row; loads in flight
    for (int i0 = threadIdx.x; i0 < tiles * TILE_ROWS * UNITS; i0 += THREADS * LOADS) {
        uint4 v[LOADS];
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int i = i0 + THREADS * j, row = i / UNITS;
            v[j] = make_uint4(0, 0, 0, 0);
            if (row < tiles * TILE_ROWS && q0 + row < p.nq && row_inside(p, bh * p.nq + q0 + row, SITE_I_QUERY))
                v[j] = *reinterpret_cast<const uint4*>(p.Q + (bh * p.nq + q0 + row) * D + i % UNITS * 8);
        }
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int i = i0 + THREADS * j, row = i / UNITS, unit = i % UNITS;
            uint8_t* at = smem + (row / TILE_ROWS) * L::Q_TILE + (unit / 8) * L::Q_CHUNK + (row % TILE_ROWS) * 128;
            if (row < tiles * TILE_ROWS)
                *reinterpret_cast<uint4*>(at + (((unit % 8) ^ (row & 7)) << 4)) =
                    make_uint4(__byte_perm(v[j].x, v[j].y, 0x5410), __byte_perm(v[j].x, v[j].y, 0x7632),
                               __byte_perm(v[j].z, v[j].w, 0x5410), __byte_perm(v[j].z, v[j].w, 0x7632));
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool skip = *abort_flag != 0;  // an earlier kernel gave up: do nothing
    const int n = skip || end <= begin ? 0 : (end - begin + STEP - 1) / STEP;

    if (warp >= MMA_WARP) {
        // ----------------------------------------------------------------- MMA
        shed_registers<MMA_REGS>();
        const int t = warp - MMA_WARP;
        const Turns turns = turns_of<ONE>(t, n);
        if (warp < FETCH_WARP && (ONE || t < tiles) && turns.n > 0) {
            const bool leader = elect_one();
            constexpr uint32_t idesc_s = idesc_bf16_f32(TILE_ROWS, STEP, 0, 0);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(TILE_ROWS, D, 0, 1);
            const uint64_t q_desc = smem_desc_sw128(sbase + (ONE ? 0 : t) * L::Q_TILE, 16, 1024);
            const uint64_t k_desc = smem_desc_sw128(sbase + L::K_OFF, 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(sbase + L::V_OFF, L::KV_CHUNK, 1024);  // V as MN-major B
            auto wait_all = [&](uint32_t bb, uint32_t parity, int site) {
                return __all_sync(0xFFFFFFFFu, mbar_wait(bb, parity, wc, site)) != 0;
            };
            // S of this warp's step i, whose K has been waited for
            auto issue_s = [&](int i) {
                const int st = turns.step(i) % L::STAGES;
                // behind the P V of its step i - 2, which reads this buffer (see the header)
                if (i >= 2 && leader)
                    tmem_shift_down(tmem + s_col(t, i & 1));
                const uint64_t kd = desc_add(k_desc, st * L::KV_TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t ad = desc_add(q_desc, (kk >> 2) * L::Q_CHUNK + (kk & 3) * 32);
                    const uint64_t bd = desc_add(kd, (kk >> 2) * L::KV_CHUNK + (kk & 3) * 32);
                    mma_ss(leader, tmem + s_col(t, i & 1), ad, bd, idesc_s, kk > 0 ? 1u : 0u);
                }
                if (leader) {
                    mma_commit(bar(B_S_FULL + 2 * t + (i & 1)));
                    mma_commit(bar(B_K_EMPTY + st));
                }
            };
            auto wait_k = [&](int i) {
                const int h = turns.step(i);
                return wait_all(bar(B_K_FULL + h % L::STAGES), (h / L::STAGES) & 1, SITE_K_FULL);
            };
            bool ok = true;
            for (int i = 0; ok && i < min(turns.n, 2); ++i) {
                if (!(ok = wait_k(i)))
                    break;
                fence_proxy_async_smem();
                tc_fence_after();
                issue_s(i);
            }
            for (int i = 0; ok && i < turns.n; ++i) {
                // V of this step and K of the step after next first, so that nothing
                // stands between P and the two products behind it.  (With the steps
                // taken in turn that K is four steps on: the convert warps reach it
                // only when this step's P V has left its stage of V.)
                const int h = turns.step(i), st = h % L::STAGES, buf = i & 1;
                const bool more = i + 2 < turns.n;
                ok = wait_all(bar(B_V_FULL + st), (h / L::STAGES) & 1, SITE_V_FULL);
                if (!ONE && ok && more)
                    ok = wait_k(i + 2);
                if (!ok)
                    break;
                fence_proxy_async_smem();
                if (!(ok = wait_all(bar(B_P_FULL + 2 * t + buf), (i >> 1) & 1, SITE_P_FULL)))
                    break;
                tc_fence_after();
                const uint64_t vd = desc_add(v_desc, st * L::KV_TILE);
#pragma unroll
                for (int kk = 0; kk < STEP / 16; ++kk)
                    mma_ts(leader, tmem + o_col(t), tmem + s_col(t, buf) + kk * 8, desc_add(vd, kk * 2048), idesc_pv,
                           (i > 0 || kk > 0) ? 1u : 0u);
                if (PAIR) {
#pragma unroll
                    for (int kk = 0; kk < STEP / 16; ++kk)
                        mma_ts(leader, tmem + o_col(t), tmem + s_col(t, buf) + STEP / 2 + kk * 8,
                               desc_add(vd, kk * 2048), idesc_pv, 1u);
                }
                if (leader) {
                    mma_commit(bar(B_PV_DONE + t));
                    mma_commit(bar(B_V_EMPTY + st));
                }
                if (more) {
                    if (ONE) {
                        if (!(ok = wait_k(i + 2)))
                            break;
                        fence_proxy_async_smem();
                        tc_fence_after();
                    }
                    issue_s(i + 2);
                }
            }
            if (leader)
                mma_commit(bar(B_O_FINAL + t));
            // Every MMA issued by the elected lane has completed once O_FINAL fires.
            drain_wait(bar(B_O_FINAL + t), 0, p.timeout_ns);
        } else if (warp >= FETCH_WARP && n > 0) {
            // ----------------------------------------------------------- fetch
            const int lane = threadIdx.x & 31;
            const long long first = (bh * p.W * p.s + begin) * D;
            // the scales of rows lane and lane + 32 of K and of V, one step ahead
            float scale[4];
            auto load_scales = [&](int hh) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = begin + hh * STEP + lane + 32 * (i & 1);
                    scale[i] = 0.f;
                    if (key < end && scale_inside(p, scale_index(p, bh, key)))
                        scale[i] = __ldg((i < 2 ? p.k_scale : p.v_scale) + scale_index(p, bh, key));
                }
            };
            const int mine = warp - FETCH_WARP;  // the two fetch warps take the steps in turn
            load_scales(mine);
            int last = mine - 2;
            for (int hh = mine; hh < n; hh += 2) {
                const int rs = hh % L::RAW;
                if (hh >= L::RAW && !__all_sync(0xFFFFFFFFu, mbar_wait(bar(B_RAW_EMPTY + rs), ((hh / L::RAW) - 1) & 1,
                                                                       wc, SITE_RAW_EMPTY)))
                    break;
                uint32_t* factors = reinterpret_cast<uint32_t*>(smem + L::FACTOR_OFF) + rs * L::FACTORS;
                bool two = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const CodeScale cs = code_scale(scale[i]);
                    factors[32 * i + lane] = cs.first | (cs.second << 16);
                    two |= cs.second != 0x3F80u;
                }
                two = __any_sync(0xFFFFFFFFu, two);
                if (lane == 0) {
                    factors[2 * STEP] = two ? 1u : 0u;
                }
                __syncwarp();
                // (debug build: nothing is copied, and the other roles leave their waits)
                const int keys = min(STEP, end - begin - hh * STEP);
                if (!in_bounds(wc, keys_inside(p, bh, begin + hh * STEP, keys), SITE_B_KEYS))
                    break;
                if (lane == 0) {
                    const uint32_t bytes = static_cast<uint32_t>(keys) * D;
                    const uint32_t raw = sbase + L::RAW_OFF + rs * 2 * L::RAW_TILE;
                    const long long at = first + static_cast<long long>(hh) * L::RAW_TILE;
                    mbar_arrive_expect_tx(bar(B_RAW_FULL + rs), 2 * bytes);
                    bulk_load(raw, p.k8 + at, bytes, bar(B_RAW_FULL + rs));
                    bulk_load(raw + L::RAW_TILE, p.v8 + at, bytes, bar(B_RAW_FULL + rs));
                }
                last = hh;
                if (hh + 2 < n)
                    load_scales(hh + 2);
            }
            // Let the copies in flight land before the block can exit: at most the last
            // one of each stage is.
            static_assert(L::RAW == 4, "two stages a fetch warp");
            for (int j = max(mine, last - 2); j <= last; j += 2)
                drain_wait(bar(B_RAW_FULL + j % L::RAW), (j / L::RAW) & 1, p.timeout_ns);
        }
    } else if (warp >= CONVERT_WARP) {
        // ------------------------------------------------------------- convert
        shed_registers<CONVERT_REGS>();
        using C = Codes<D>;
        const int thread = threadIdx.x - CONVERT_WARP * 32, lane = thread & 31;
        const int part = thread % C::PER_ROW, row = thread / C::PER_ROW;
        for (int hh = 0; hh < n; ++hh) {
            const int st = hh % L::STAGES, rs = hh % L::RAW;
            const uint32_t freed = ((hh / L::STAGES) - 1) & 1;
            auto wait_empty = [&](int kv) {
                return hh < L::STAGES ||
                       __all_sync(0xFFFFFFFFu, mbar_wait(bar((kv ? B_V_EMPTY : B_K_EMPTY) + st), freed, wc,
                                                         kv ? SITE_V_EMPTY : SITE_K_EMPTY));
            };
            const uint8_t* raw = smem + L::RAW_OFF + rs * 2 * L::RAW_TILE;
            const uint32_t* factors =
                reinterpret_cast<const uint32_t*>(smem + L::FACTOR_OFF) + rs * L::FACTORS;
            auto store = [&](const Codes<D>& c, int kv) {
                uint8_t* stage = smem + (kv ? L::V_OFF : L::K_OFF) + st * L::KV_TILE;
                if (factors[2 * STEP])
                    store_codes<D, true>(c, stage, row, part);
                else
                    store_codes<D, false>(c, stage, row, part);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar((kv ? B_V_FULL : B_K_FULL) + st));
            };
            bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(B_RAW_FULL + rs), (hh / L::RAW) & 1, wc, SITE_RAW_FULL));
            if (ONE) {  // K and V together: the step is as long as this takes
                if (!(ok = ok && wait_empty(0) && wait_empty(1)))
                    break;
                Codes<D> k, v;
                load_codes<D>(k, raw, factors, row, part);
                load_codes<D>(v, raw + L::RAW_TILE, factors + STEP, row, part);
                store(k, 0);
                store(v, 1);
            } else {
#pragma unroll 1
                for (int kv = 0; ok && kv < 2; ++kv) {
                    if (!(ok = wait_empty(kv)))
                        break;
                    Codes<D> c;
                    load_codes<D>(c, raw + kv * L::RAW_TILE, factors + kv * STEP, row, part);
                    store(c, kv);
                }
                if (!ok)
                    break;
            }
            if (lane == 0)
                mbar_arrive(bar(B_RAW_EMPTY + rs));
        }
    } else if (ONE || warp < 4 * tiles) {
        // ------------------------------------------------------------- softmax
        take_registers<SOFTMAX_REGS>();
        const int t = warp >> 2;
        const Turns turns = turns_of<ONE>(t, n);
        const int row = q0 + (ONE ? 0 : t) * TILE_ROWS + (threadIdx.x & 127);
        const bool row_valid = row < p.nq;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const float c = p.scale_log2;
        float m_run = -INFINITY, l_run = 0.f;
        bool ok = true;
        for (int i = 0; i < turns.n; ++i) {
            const uint32_t col = s_col(t, i & 1);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(B_S_FULL + 2 * t + (i & 1)), (i >> 1) & 1, wc, SITE_S_FULL));
            if (!ok)
                break;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(lanes + col, s[0]);
            tmem_ld32(lanes + col + 32, s[1]);
            tmem_wait_ld();
            const int valid = end - (begin + turns.step(i) * STEP);  // keys of this step
            if (valid < STEP) {
#pragma unroll
                for (int e = 0; e < STEP; ++e)
                    if (e >= valid)
                        s[e / 32][e % 32] = __float_as_uint(-INFINITY);
            }
            auto exp_pass = [&](float m_use, bool with_max, float& top) -> float {
                uint64_t sum[4] = {0, 0, 0, 0};
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t pk[16], rest[16];
                    if (with_max)
                        exp_columns<true, PAIR>(s[k], c, -m_use, sum, mx, pk, rest);
                    else
                        exp_columns<false, PAIR>(s[k], c, -m_use, sum, mx, pk, rest);
                    tmem_st16(lanes + col + k * 16, pk);
                    if (PAIR)
                        tmem_st16(lanes + col + STEP / 2 + k * 16, rest);
                }
                top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                float lo, hi;
                unpair(pair_add(pair_add(sum[0], sum[1]), pair_add(sum[2], sum[3])), lo, hi);
                return lo + hi;
            };
            // Raise the running maximum (for the whole warp) and rescale O and l, once
            // the P V of the step before has completed.
            bool raised = true;
            auto raise_max = [&](float m_step) {
                const float m_new = fmaxf(m_run, m_step);
                const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m_run - m_new);
                if (i > 0) {
                    raised = __all_sync(0xFFFFFFFFu, mbar_wait(bar(B_PV_DONE + t), (i - 1) & 1, wc, SITE_PV_DONE));
                    if (!raised)
                        return;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tmem_ld32(lanes + o_col(t) + k * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(lanes + o_col(t) + k * 32, o);
                    }
                }
                l_run *= alpha;
                m_run = m_new;
            };
            float sum, top;
            if (__any_sync(0xFFFFFFFFu, m_run == -INFINITY)) {
                // no reference maximum yet in this warp: the maximum first
                float mx[8];
#pragma unroll
                for (int a = 0; a < 8; ++a)
                    mx[a] = -INFINITY;
#pragma unroll
                for (int e = 0; e < STEP; ++e)
                    mx[e % 8] = fmaxf(mx[e % 8], __uint_as_float(s[e / 32][e % 32]));
#pragma unroll
                for (int w = 4; w >= 1; w /= 2)
#pragma unroll
                    for (int a = 0; a < w; ++a)
                        mx[a] = fmaxf(mx[a], mx[a + w]);
                const float m_step = mx[0] * c;  // c > 0
                if (__any_sync(0xFFFFFFFFu, m_step > m_run + RAISE))
                    raise_max(m_step);
                sum = exp_pass(m_run == -INFINITY ? 0.f : m_run, false, top);
            } else {
                // one pass against the running maximum; redone in the rare step that exceeds it by more than RAISE
                sum = exp_pass(m_run, true, top);
                const float m_step = top * c;
                if (__any_sync(0xFFFFFFFFu, m_step > m_run + RAISE)) {
                    raise_max(m_step);
                    sum = exp_pass(m_run, false, top);
                }
            }
            if (!(ok = raised))
                break;
            l_run += sum;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(B_P_FULL + 2 * t + (i & 1)));
        }

        // ------------------------------------------------------------ epilogue
        if (turns.n > 0 && ok)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(B_O_FINAL + t), 0, wc, SITE_O_FINAL));
        // With the steps taken in turn, group 1 leaves its maximum, sum and O
        // ([column][row]) in the stages, and group 0 joins them to its own.
        float* other_o = reinterpret_cast<float*>(smem + L::K_OFF) + (threadIdx.x & 127);
        float* other_ml = reinterpret_cast<float*>(smem + L::RAW_OFF) + (threadIdx.x & 127);
        const bool join = ONE && n > 1;  // group 1 has had a step
        if (join) {
            if (ok)  // the other's products read the stages
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(B_O_FINAL + 1 - t), 0, wc, SITE_O_FINAL));
            tc_fence_after();
            if (t == 1 && ok) {
                static_assert(!ONE || D * TILE_ROWS * 4 <= 2 * L::STAGES * L::KV_TILE, "O fits the stages");
                other_ml[0] = m_run;
                other_ml[TILE_ROWS] = l_run;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(lanes + o_col(1) + k * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        other_o[(k * 32 + e) * TILE_ROWS] = __uint_as_float(o[e]);
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");  // the two groups, whatever became of them
        }
        tc_fence_after();
        // one answer a warp: the flag may rise between two lanes' looks at it
        if (__all_sync(0xFFFFFFFFu, ok && !*abort_flag) && (!ONE || t == 0)) {
            const long long at = bh * p.nq + row;
            float mine = 1.f, others = 0.f;  // factors of the joined O
            if (join) {
                const float m1 = other_ml[0], m = fmaxf(m_run, m1);
                mine = m_run == -INFINITY ? 1.f : fast_exp2(m_run - m);  // 1: its sums are 0 or NaN
                others = m1 == -INFINITY ? 1.f : fast_exp2(m1 - m);
                l_run = l_run * mine + other_ml[TILE_ROWS] * others;
                m_run = m;
            }
            if (p.splits == 1) {
                const float f = l_run == 0.f ? 0.f : 1.f / l_run;
                mine *= f;
                others *= f;
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                // The stores of the round before part the lanes of a tile's last, ragged warp; the
                // load is warp-collective (.sync.aligned) and undefined in a warp that is not whole.
                __syncwarp();
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(lanes + o_col(t) + k * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0u;
                }
                float x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {  // columns 1 and 2 of every four hold channels 2 and 1
                    const int from = (e & 3) == 1 ? e + 1 : ((e & 3) == 2 ? e - 1 : e);
                    x[e] = __uint_as_float(o[from]) * mine;
                    if (join)
                        x[e] = fmaf(other_o[(k * 32 + from) * TILE_ROWS], others, x[e]);
                }
                if (!row_valid)
                    continue;
                if (!row_inside(p, at, SITE_I_RESULT) || (p.splits > 1 && !part_inside(p, at * p.splits + split)))
                    continue;
                if (p.splits > 1) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (at * p.splits + split) * D + k * 32);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        dst[u] = make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.O + at * D + k * 32);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        dst[u] = make_uint4(pack_bf16(x[8 * u], x[8 * u + 1]), pack_bf16(x[8 * u + 2], x[8 * u + 3]),
                                            pack_bf16(x[8 * u + 4], x[8 * u + 5]),
                                            pack_bf16(x[8 * u + 6], x[8 * u + 7]));
                }
            }
            if (row_valid && row_inside(p, at, SITE_I_RESULT)) {
                if (p.splits > 1)
                    p.part_ml[at * p.splits + split] = make_float2(m_run, l_run);
                else if (p.lse)
                    p.lse[at] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * LN2;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP) {
        __syncwarp();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int D, bool ONE, bool PAIR>
ra_status launch(const AttnParams& p, int B, cudaStream_t cs)
{
    // the attribute belongs to the function on one device
    static std::atomic<unsigned long long> set{0};
    int dev = 0;
    RA_CUDA_TRY(cudaGetDevice(&dev));
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev >= 64 || !(set.load(std::memory_order_acquire) & bit)) {
        RA_CUDA_TRY(cudaFuncSetAttribute(cache8_tiles_kernel<D, ONE, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Layout<D, ONE>::SMEM));
        if (dev < 64)
            set.fetch_or(bit, std::memory_order_release);
    }
    const dim3 grid(static_cast<unsigned>(p.q_tiles) * p.splits, p.H, B);
    cache8_tiles_kernel<D, ONE, PAIR><<<grid, THREADS, Layout<D, ONE>::SMEM, cs>>>(p);
    return cuda_fail(cudaGetLastError(), "cache8_tiles_kernel launch");
}

}  // namespace

ra_status cache8_tiles(const AttnParams& p, int B, int d, bool one, bool pair, cudaStream_t cs)
{
    auto run = [&](auto D, auto ONE) {
        return pair ? launch<D(), ONE(), true>(p, B, cs) : launch<D(), ONE(), false>(p, B, cs);
    };
    using std::integral_constant;
    using One = std::true_type;
    using Two = std::false_type;
    if (d == 64)
        return one ? run(integral_constant<int, 64>{}, One{}) : run(integral_constant<int, 64>{}, Two{});
    return one ? run(integral_constant<int, 128>{}, One{}) : run(integral_constant<int, 128>{}, Two{});
}

}  // namespace ra
