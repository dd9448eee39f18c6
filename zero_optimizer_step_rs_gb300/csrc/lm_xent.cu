// lm_xent.cu - softmax cross entropy of activations against a (tied)
// embedding table, in pieces of the vocabulary and without kept logits, and
// its gradients (declared in include/zero_step.h).
//
//   l = h E^T (bf16 products, fp32 sums), lse_t = log sum_v exp(l_tv),
//   loss_t = lse_t - l_{t, y_t}                       (0 for an ignored token)
//   P_tv = (exp(l_tv - lse_t) - [v = y_t]) * dloss_t / u   (0 in an ignored row)
//   dh = u (P E + e_t E_y),  dE = u P^T h,  u = max_t |dloss_t|
// with e_t what the rounding of P_ty to bf16 lost.
//
// Forward is one matrix product whose epilogue keeps, per row and tile of up to
// 256 vocabulary rows, a maximum and the sum of exponentials relative to it; a
// small second kernel joins the tiles.  Backward keeps nothing but lse: for a
// piece of the vocabulary at a time it makes the logits again, turns them into P
// in bf16 (an operand of the tensor cores, and the one rounding before the
// sums), and multiplies P with both operands.  A row's entry at the target,
// exp - 1, outweighs all others together, so its rounding would be the error of the
// row of dh (0.0023 of it, where rounding the result takes 0.0017): what it lost is
// kept as one fp32 number a token, and its product with the target's row of the
// table is added in fp32 before dh is rounded.  The gradient of the table has P's
// rounding: a token's terms go to as many rows as the vocabulary has, so adding
// the lost parts there would take the tokens sorted by target.  Where all tokens
// weigh the same, as in a mean, dloss / u is exactly 1 and the entry near -1 loses
// next to nothing (0.0017); with other weights it is off by 0.0022 to 0.0024, two
// roundings.  The gradient of the table's piece is final and written once; dh is
// summed over the pieces in fp32 and rounded once at the end.
//
// Floor: 2*T*D*V operations forward, 6*T*D*V backward (the logits are needed
// again), on the tensor cores; with few tokens the table's 2*V*D bytes.
// Measured, one GB300: 8192 x 128256 x 2048 forward 2.05 ms in a short burst
// (2.1 PFLOP/s, tensor pipe 98 % busy at the 1.75 GHz that the power limit
// leaves) and 2.3 ms sustained; backward 7.1 and 7.6 to 7.7 ms (1.82 and 1.67 to
// 1.69).  17 x 50257 x 768 forward 25 us for the table's 77 MB (11.4 us at the copy
// rate): two launches, a pipeline to fill, and three rounds of tiles for 76 CTA
// pairs; backward 72 us (23).
//
// The product kernel (k_mma): a pair of CTAs (cta_group::2) owns a 256 x 256
// tile of fp32 sums in tensor memory, 128 rows in each CTA, two tiles deep, so
// that one tile's epilogue runs under the next tile's products.  Warp 0 of each
// CTA brings its half of both operands into shared memory with TMA (64 wide
// along the summed dimension, 128-byte swizzle, 6 stages: 32 KB a CTA for 512
// cycles of products), warp 1 of the first CTA issues the products, warps 4-11
// run the epilogue.  An operand may be contiguous along the summed dimension or
// along the other one; both are read as they lie in memory, nothing is
// transposed.  The grid is one CTA pair for every two SMs, each walking over its
// units of work.
//
// What was measured and not kept: pieces of the vocabulary small enough for P to
// stay in L2 (4 to 15 % slower than 512 MiB of P: more, shorter launches);
// tiles ordered in blocks of 2 to 16 token tiles (2 to 14 % slower than all
// token tiles of a vocabulary tile at a time); the table brought into L2 ahead
// by bulk prefetches (17 x 128256 x 2048: 97 -> 146 us); four epilogue warps, bulk
// tensor stores and pauses between the stores (the same within 1 %).
//
// Every wait is bounded.  When one runs out the CTA sets ZERO_DEV_TIMEOUT, all
// of its roles leave their loops, copies and products in flight are waited
// for (again bounded, ZERO_DEV_DRAIN_FAILED if that runs out), the tensor
// memory is freed and the kernel returns.
#include <cuda.h>

#include "lm_common.cuh"

namespace {

using namespace lm;

constexpr float kLog2e = 1.4426950408889634f;
// 1 / kLog2e (the fp32 number, not log2 e), in two parts: maxima are kept as x * kLog2e,
// and the fp32 constant alone would be off by 1e-5 at logits of some hundreds
constexpr float kUnLog2e = (float)(1.0 / (double)kLog2e);
constexpr float kUnLog2eRest = (float)(1.0 / (double)kLog2e - (double)kUnLog2e);

constexpr int BM = 256, BN = 256, BK = 64;         // a CTA pair's largest tile, a stage's depth
constexpr int kEpilogueWarps = 8;                  // two for each quarter of the tensor memory
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kStageBytes = 2 * 128 * BK * 2;      // per CTA: 128 rows of each operand
constexpr int kPieceAlign = 256;
constexpr int64_t kMostP = 1ll << 28;              // elements of a piece's P, unless asked for
constexpr uint64_t kWaitLimit = 2000000000;        // ns that a wait may take
constexpr uint64_t kDrainLimit = 200000000;
constexpr int kWarpStage = 4096;                   // an epilogue warp's output buffer
constexpr int kStaging = kEpilogueWarps * kWarpStage;

// The loss; a piece's P; both gradients of a piece (two products in one launch).
enum Kind { kLse, kP, kGrads };

constexpr int kShares = 2 * 128 * 8;               // kLse: the second half's (maximum, sum)

constexpr int kStages = 6;

template <Kind K>
constexpr int smem_bytes()
{
    return 1024 + kStages * kStageBytes + (K == kLse ? kShares : kStaging) + 256;
}

// One product: its operands, its result and how it is cut into units of work.
struct Product {
    CUtensorMap a, b;
    void* out;                         // bf16; dh's sums: fp32
    int64_t out_ld;
    int32_t m_tiles, n_tiles, bn;      // tiles of 256 x bn
    int32_t k_blocks, splits;          // blocks of 64 along the summed dimension; its splits
    int32_t m_fast;                    // which tile coordinate runs fastest
    // Rows of a box of `a` where it is contiguous along the sum, and how many of
    // the pair's CTAs load one: filling the rest of a mostly empty tile with
    // zeros took longer than reading it (17 tokens longer than 256), and what
    // stands in rows past the last goes nowhere.
    int32_t a_box, a_ctas;
    // Along the sum, the last stage's steps of 16, and the rows of its boxes
    // where an operand is contiguous the other way (one stage only, else 64).
    int32_t last_steps, k_box;
    int64_t rows, cols;                // of the result (of the piece)
    int32_t units() const { return m_tiles * n_tiles * splits; }
};

struct MmaArgs {
    Product x, y;                      // kGrads: dh (x) and the table's gradient (y); else x
    int32_t x_units, y_units;
    // y's units beyond x's: the pairs from `light` on have one unit of x less and
    // first take `extra` of y's units among themselves
    int32_t light, extra;
    int64_t out_split_rows;            // kGrads: rows between the splits of dh
    int32_t add;                       // kGrads: dh's sums are added to what is there
    int32_t token_bytes;
    const void* targets;
    int64_t V, v0;                     // the vocabulary, and where the piece starts
    const float* lse;
    const float* dloss;
    const float* unit;                 // u
    float* lost;                       // kP: e_t, of the rows whose target is in the piece
    float2* part;                      // kLse: [n_tiles][part_ld] (maximum, sum)
    int64_t part_ld;
    float* at_target;                  // kLse: the target's logit
    int32_t* status;
    uint64_t wait_limit;               // ns
};

// ------------------------------------------------------------ PTX pieces --

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}
// True in one lane of a converged warp.  The compiler knows that what it guards
// runs in a single lane: with `lane == 0` instead, and one thread in the loops that
// feed the tensor cores, these were busy for 83 % of the time and not 98 %.
__device__ __forceinline__ bool elect()
{
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// the same address in the pair's first CTA
__device__ __forceinline__ uint32_t in_leader(uint32_t addr)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// One thread waits for a phase; gives up after `limit` ns (at once if that is 0), or once
// another role of the CTA has given up.  False: the caller leaves its loop.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit,
                                          volatile int* dead)
{
    if (limit != 0) {
        if (mbar_try(bar, parity)) return true;
        const uint64_t start = now_ns();
        do {
#pragma unroll 1
            for (int i = 0; i < 16; ++i)
                if (mbar_try(bar, parity)) return true;
        } while (!*dead && now_ns() - start < limit);
    }
    *dead = 1;
    return false;
}
// The same by a whole warp, whose lanes stay together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit,
                                          volatile int* dead)
{
    if (limit != 0) {
        if (__all_sync(0xFFFFFFFFu, mbar_try(bar, parity))) return true;
        const uint64_t start = now_ns();
        do {
#pragma unroll 1
            for (int i = 0; i < 16; ++i)
                if (__all_sync(0xFFFFFFFFu, mbar_try(bar, parity))) return true;
        } while (!__any_sync(0xFFFFFFFFu, *dead || now_ns() - start >= limit));
    }
    *dead = 1;
    return false;
}
// One box into this CTA's shared memory; the bytes count on the leader's barrier.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t leader_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(leader_bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; "
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}
// Arrive at the barrier at this offset in both CTAs once the products issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&x)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How an operand lies in shared memory (128-byte swizzle).  Contiguous along
// the summed dimension: rows of 128 bytes, 1024 bytes between groups of 8 rows.
// Contiguous along the other one: two chunks of 64 x 64, 8192 bytes apart,
// 1024 bytes between groups of 8 along the summed dimension.
template <bool K_MAJOR>
struct Layout {
    static __device__ __forceinline__ uint64_t descriptor(uint32_t addr)
    {
        const uint64_t lead = K_MAJOR ? 1 : 8192 >> 4;
        return (uint64_t)((addr >> 4) & 0x3FFF) | lead << 16 | (uint64_t)(1024 >> 4) << 32 |
               1ull << 46 | 2ull << 61;
    }
    static constexpr uint64_t step = (K_MAJOR ? 32 : 2048) >> 4;     // 16 along the sum
    // 128 rows of a stage
    static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, int row, int k,
                                                uint32_t bar)
    {
        if constexpr (K_MAJOR) {
            tma_load(dst, map, k, row, bar);
        } else {
            tma_load(dst, map, row, k, bar);
            tma_load(dst + 8192, map, row + 64, k, bar);
        }
    }
};
// fp32 sums, bf16 operands, 256 x bn
template <bool A_K, bool B_K>
__device__ __forceinline__ uint32_t instruction(int bn)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (A_K ? 0u : 1u << 15) | (B_K ? 0u : 1u << 16) |
           (uint32_t)(bn >> 3) << 17 | (uint32_t)(BM >> 4) << 24;
}
// One stage's products.
template <bool A_K, bool B_K>
__device__ __forceinline__ void products(uint32_t d, uint32_t at, int bn, bool add)
{
    const uint64_t da = Layout<A_K>::descriptor(at);
    const uint64_t db = Layout<B_K>::descriptor(at + kStageBytes / 2);
    const uint32_t idesc = instruction<A_K, B_K>(bn);
#pragma unroll
    for (int q = 0; q < BK / 16; ++q)
        mma(d, da + q * Layout<A_K>::step, db + q * Layout<B_K>::step, idesc, add || q > 0);
}
// The first `steps` of them, where the sum ends in the stage.
template <bool A_K, bool B_K>
__device__ __forceinline__ void products_end(uint32_t d, uint32_t at, int bn, bool add, int steps)
{
    const uint64_t da = Layout<A_K>::descriptor(at);
    const uint64_t db = Layout<B_K>::descriptor(at + kStageBytes / 2);
#pragma unroll 1
    for (int q = 0; q < steps; ++q)
        mma(d, da + q * Layout<A_K>::step, db + q * Layout<B_K>::step, instruction<A_K, B_K>(bn),
            add || q > 0);
}

// The i-th unit of work of a CTA pair, or -1: x's units by turns, then (for
// the pairs that got one less) the extra ones of y, then the rest of y by turns.
__device__ __forceinline__ int unit_of(const MmaArgs& a, int pair, int pairs, int i)
{
    const int nx = pair < a.x_units ? (a.x_units - pair + pairs - 1) / pairs : 0;
    if (i < nx) return pair + i * pairs;
    i -= nx;
    if (pair >= a.light) {
        const int lights = pairs - a.light, q = pair - a.light;
        const int ne = q < a.extra ? (a.extra - q + lights - 1) / lights : 0;
        if (i < ne) return a.x_units + q + i * lights;
        i -= ne;
    }
    const int j = a.extra + pair + i * pairs;
    return j < a.y_units ? a.x_units + j : -1;
}

struct Unit {
    int m, n, k0, k1, split;
};

__device__ __forceinline__ Unit unit_at(const Product& p, int u)
{
    Unit t;
    const int tiles = p.m_tiles * p.n_tiles;
    t.split = u / tiles;
    const int q = u - t.split * tiles;
    const int fast = p.m_fast ? p.m_tiles : p.n_tiles;
    const int hi = q / fast, lo = q - hi * fast;
    t.m = p.m_fast ? lo : hi;
    t.n = p.m_fast ? hi : lo;
    t.k0 = 0;
    t.k1 = p.k_blocks;
    if (p.splits > 1) {
        t.k0 = (int)((int64_t)p.k_blocks * t.split / p.splits);
        t.k1 = (int)((int64_t)p.k_blocks * (t.split + 1) / p.splits);
    }
    return t;
}

// ---------------------------------------------------------- the epilogues --

// What an epilogue needs to know of its row; asked for while the tile's
// products still run (after them it is a good part of a short tile's time).
struct Row {
    int64_t y = -1;                    // the target, or -1 where the row takes part in nothing
    float lse2 = 0.0f;                 // kP: lse in units of log 2
    float g = 0.0f;                    // kP: dloss / u; kGrads: u
};

template <Kind K>
__device__ __forceinline__ Row row_of(const MmaArgs& a, int64_t row, float unit)
{
    Row r;
    if constexpr (K != kGrads) {
        if (row >= a.x.rows) return r;
        r.y = token_at(a.targets, a.token_bytes, row);
        if (r.y >= a.V) r.y = -1;
        if constexpr (K == kP) {
            const float lse = a.lse[row], g = a.dloss[row];
            if (r.y >= 0) {
                r.lse2 = lse * kLog2e;
                r.g = g / unit;
            }
        }
    } else {
        r.g = unit;
    }
    return r;
}

// The joint (maximum, sum) of two parts of a row; maxima in units of log 2.
__device__ __forceinline__ void join(float& m, float& s, float2 x)
{
    const float top = fmaxf(m, x.x);
    const float ref = top == -INFINITY ? 0.0f : top;
    s = s * exp2_fast(m - ref) + x.y * exp2_fast(x.x - ref);
    m = top;
}

// The row's running maximum and sum over the tile's columns, 128 of them by
// each of two warps: the second leaves its part in `share` and arrives at
// `ready`, the first joins the two.  There are two of both, used by turns; a
// tile's are free again once the first warp has given up the tile's sums, without
// which the products two tiles on do not start.
__device__ __forceinline__ bool epilogue_lse(const MmaArgs& a, const Unit& t, uint32_t tmem,
                                             int64_t row, const Row& info, int half,
                                             float2* share, uint32_t ready, uint32_t parity,
                                             volatile int* dead)
{
    const int64_t c0 = (int64_t)t.n * a.x.bn;
    const int live = (int)min((int64_t)a.x.bn, a.V - c0);
    const int64_t y = info.y - c0;                           // of the tile, if in it
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int c = half * 128; c < half * 128 + 128; c += 32) {
        if (c >= live) break;
        float x[32];
        tmem_load32(tmem + c, x);
        if (c + 32 > live) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i >= live) x[i] = -INFINITY;
        }
        const int at = (int)(y - c);
        if (y >= c && y < min(c + 32, live)) {        // not the next tile's first columns
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i == at) v = x[i];
            a.at_target[row] = v;
        }
        __syncwarp();                                        // together at the next load
        float m = x[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) m = fmaxf(m, x[i]);
        m = fmaxf(top, m * kLog2e);
        const float ref = m == -INFINITY ? 0.0f : m;         // nothing but -Inf so far
        sum *= exp2_fast(top - ref);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i & 3] += exp2_fast(fmaf(x[i], kLog2e, -ref));
        sum += (s[0] + s[1]) + (s[2] + s[3]);
        top = m;
    }
    if (half == 1) {
        *share = make_float2(top, sum);
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(ready) : "memory");
        return true;
    }
    const bool ok = warp_wait(ready, parity, a.wait_limit, dead);
    if (ok && row < a.x.rows) {
        join(top, sum, *share);
        a.part[(int64_t)t.n * a.part_ld + row] = make_float2(top, sum);
    }
    return ok;
}

// 16 bytes at (row, chunk) of a 32-row buffer of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ void stage16(uint32_t buf, int row, int chunk, uint32_t x, uint32_t y,
                                        uint32_t z, uint32_t w)
{
    const uint32_t p = buf + row * 128 + ((chunk ^ (row & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(x), "r"(y), "r"(z),
                 "r"(w)
                 : "memory");
}

// Writes a staged buffer out, 8 lanes to a 128-byte row.
template <typename Store>
__device__ __forceinline__ void write_rows(uint32_t buf, int lane, Store&& store)
{
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = j * 4 + (lane >> 3), chunk = lane & 7;
        const uint32_t p = buf + row * 128 + ((chunk ^ (row & 7)) << 4);
        uint4 x;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(p)
                     : "memory");
        store(row, chunk, x);
    }
    __syncwarp();
}

// The tile's 128 rows of this CTA in bf16 (P, or the table's gradient): 64
// columns at a time through the warp's buffer, 128 columns a warp.
template <bool P>
__device__ __forceinline__ void epilogue_bf16(const MmaArgs& a, const Product& p, const Unit& t,
                                              uint32_t tmem, int64_t row0, const Row& info,
                                              int lane, int half, uint32_t to)
{
    const int64_t c0 = (int64_t)t.n * p.bn;
    if (row0 >= p.rows) return;
    const bool live = !P || info.y >= 0;
    const float lse2 = info.lse2, g = info.g;
    const int64_t y = info.y - (a.v0 + c0);
#pragma unroll 1
    for (int c = half * 128; c < min(p.bn, half * 128 + 128); c += 64) {
        if (c0 + c >= p.cols) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[32];
            tmem_load32(tmem + c + 32 * h, x);
            if constexpr (P) {
                const int at = (int)(y - (c + 32 * h));
                const bool here = live && y >= c + 32 * h && y < c + 32 * h + 32;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    x[i] = live ? exp2_fast(fmaf(x[i], kLog2e, -lse2)) : 0.0f;
                }
                if (here) {
                    float v = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i == at) {
                            x[i] -= 1.0f;
                            v = x[i] * g;
                        }
                    const float e = v - bf_lo(bf_pack(v, 0.0f));
                    a.lost[row0 + lane] = fabsf(e) < INFINITY ? e : 0.0f;
                }
                __syncwarp();
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= g;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                stage16(to, lane, 4 * h + j, bf_pack(x[8 * j], x[8 * j + 1]),
                        bf_pack(x[8 * j + 2], x[8 * j + 3]), bf_pack(x[8 * j + 4], x[8 * j + 5]),
                        bf_pack(x[8 * j + 6], x[8 * j + 7]));
        }
        uint16_t* out = static_cast<uint16_t*>(p.out) + row0 * p.out_ld + c0 + c;
        write_rows(to, lane, [&](int r, int chunk, const uint4& x) {
            // 8 columns at once: P's rows are padded to whole pieces, D is a multiple of 8
            if (row0 + r < p.rows && c0 + c + chunk * 8 < p.cols) {
                if constexpr (P) st16(out + r * p.out_ld + chunk * 8, x);
                else st16_stream(out + r * p.out_ld + chunk * 8, x);
            }
        });
    }
}

// dh's partial sums in fp32, 32 columns at a time; each element gets one
// addition per launch, so the order of the sum is the order of the pieces.
__device__ __forceinline__ void epilogue_f32(const MmaArgs& a, const Unit& t, uint32_t tmem,
                                             int64_t row0, int lane, int half, uint32_t to)
{
    const Product& p = a.x;
    const int64_t c0 = (int64_t)t.n * p.bn;
    if (row0 >= p.rows) return;
#pragma unroll 1
    for (int c = half * 128; c < min(p.bn, half * 128 + 128); c += 32) {
        if (c0 + c >= p.cols) break;
        float x[32];
        tmem_load32(tmem + c, x);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            stage16(to, lane, j, __float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                    __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
        float* out = static_cast<float*>(p.out) + (t.split * a.out_split_rows + row0) * p.out_ld +
                     c0 + c;
        write_rows(to, lane, [&](int r, int chunk, uint4 x) {
            if (row0 + r >= p.rows || c0 + c + chunk * 4 >= p.cols) return;
            float4* at = reinterpret_cast<float4*>(out + r * p.out_ld + chunk * 4);
            float4 f = make_float4(__uint_as_float(x.x), __uint_as_float(x.y),
                                   __uint_as_float(x.z), __uint_as_float(x.w));
            if (a.add) {
                const float4 g = *at;
                f.x += g.x; f.y += g.y; f.z += g.z; f.w += g.w;
            }
            *at = f;
        });
    }
}

// ------------------------------------------------------------ the product --

template <Kind K>
__global__ void __launch_bounds__(kThreads, 1) k_mma(const __grid_constant__ MmaArgs a)
{
    constexpr int S = kStages;
    extern __shared__ uint8_t raw[];
    // the swizzle pattern needs 1024-byte aligned stages, at the same place in both CTAs
    const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t staging = smem + S * kStageBytes;
    const uint32_t bars = staging + (K == kLse ? kShares : kStaging);
    const uint32_t full = bars, empty = bars + 8 * S;
    const uint32_t sums_full = empty + 8 * S, sums_empty = sums_full + 16;
    const uint32_t drained = sums_empty + 16;
    const uint32_t shared_full = drained + 8;            // kLse: [2][4], a quarter's second half
    const uint32_t slot = shared_full + 64;
    volatile int* dead = reinterpret_cast<volatile int*>(raw + (slot + 4 - smem_u32(raw)));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sums_full + 8 * b, 1);
            mbar_init(sums_empty + 8 * b, 2 * kEpilogueWarps);    // of both CTAs
        }
        mbar_init(drained, 1);
        for (int q = 0; q < 8; ++q) mbar_init(shared_full + 8 * q, 1);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            slot));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    asm volatile("fence.proxy.async.global;" ::: "memory");

    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    bool drain_failed = false;

    if (warp == 0) {                                     // ---- loads
        uint32_t s = 0, ph = 0, issued = 0;              // stage, its phase, loads so far
        bool ok = true;
        const uint32_t leader_full = in_leader(full);
        for (int i = 0, u; ok && (u = unit_of(a, pair, pairs, i)) >= 0; ++i) {
            const bool first = K != kGrads || u < a.x_units;
            const Product& p = first ? a.x : a.y;
            const Unit t = unit_at(p, first ? u : u - a.x_units);
            const int ra = t.m * BM + (int)rank * 128, rb = t.n * p.bn + (int)rank * (p.bn / 2);
            // both CTAs' boxes of a stage (a box always counts in full)
            const uint32_t stage_tx = (first ? p.a_ctas * p.a_box : 4 * p.k_box) * 128 +
                                      (K == kGrads ? 4 * p.k_box : p.bn) * 128;
            // (a loop for each way to load `a`: any condition inside it is paid for
            // by the tensor cores)
            auto stages = [&](auto load_a) {
                for (int kb = t.k0; kb < t.k1; ++kb) {
                    if (!(ok = warp_wait(empty + 8 * s, ph ^ 1, a.wait_limit, dead))) break;
                    if (elect()) {
                        if (leader) mbar_expect(full + 8 * s, stage_tx);
                        const uint32_t dst = smem + s * kStageBytes, bar = leader_full + 8 * s;
                        load_a(dst, kb * BK, bar);
                        Layout<K != kGrads>::load(dst + kStageBytes / 2, &p.b, rb, kb * BK, bar);
                    }
                    __syncwarp();
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            };
            if (!first)
                stages([&](uint32_t dst, int k, uint32_t bar) {
                    Layout<false>::load(dst, &p.a, ra, k, bar);
                });
            else if ((int)rank < p.a_ctas)
                stages([&](uint32_t dst, int k, uint32_t bar) {
                    Layout<true>::load(dst, &p.a, ra, k, bar);
                });
            else
                stages([](uint32_t, int, uint32_t) {});
        }
        // Before this CTA may leave: the products' last arrivals at its
        // barriers; or, after a wait ran out, the copies that were issued.  Both
        // CTAs' copies count on the leader's barriers, so the other CTA knows of its
        // own only by the products that have read them; one without is reported.
        const uint32_t from = issued > (uint32_t)S ? issued - S : 0;
        if (ok) {
            for (uint32_t j = from; j < issued && ok; ++j)
                ok = warp_wait(empty + 8 * (j % S), (j / S) & 1, a.wait_limit, dead);
        }
        if (!ok && lane == 0) {
            const uint32_t bar = leader ? full : empty;
            for (uint32_t j = from; j < issued; ++j) {
                int none = 0;
                drain_failed |= !mbar_wait(bar + 8 * (j % S), (j / S) & 1, kDrainLimit, &none);
            }
        }
    } else if (warp == 1 && leader) {                    // ---- products
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (int i = 0, u; ok && (u = unit_of(a, pair, pairs, i)) >= 0; ++i) {
            const bool first = K != kGrads || u < a.x_units;
            const Product& p = first ? a.x : a.y;
            const Unit t = unit_at(p, first ? u : u - a.x_units);
            const int b = i & 1, nk = t.k1 - t.k0, bn = p.bn;
            // a last stage that the sum ends in
            const int end = t.k1 == p.k_blocks && p.last_steps < BK / 16 ? nk - 1 : nk;
            if (!(ok = warp_wait(sums_empty + 8 * b, ((i >> 1) & 1) ^ 1, a.wait_limit, dead)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            // the next stage is looked at before this one's products are issued
            bool ready = __all_sync(0xFFFFFFFFu, mbar_try(full + 8 * s, ph));
            auto stages = [&](int from, int to, auto issue) {
                for (int k = from; k < to; ++k) {
                    if (!ready && !(ok = warp_wait(full + 8 * s, ph, a.wait_limit, dead))) return;
                    const uint32_t at = smem + s * kStageBytes, done = empty + 8 * s;
                    if (++s == S) { s = 0; ph ^= 1; }
                    if (k + 1 < nk) ready = __all_sync(0xFFFFFFFFu, mbar_try(full + 8 * s, ph));
                    if (elect()) {
                        issue(at, k > 0);
                        mma_commit(done);
                    }
                    __syncwarp();
                }
            };
            const uint32_t d = tmem + b * BN;
            if (first) {
                stages(0, end, [&](uint32_t at, bool add) {
                    products<true, K != kGrads>(d, at, bn, add);
                });
                if (ok) stages(end, nk, [&](uint32_t at, bool add) {
                    products_end<true, K != kGrads>(d, at, bn, add, p.last_steps);
                });
            } else {
                stages(0, end, [&](uint32_t at, bool add) {
                    products<false, false>(d, at, bn, add);
                });
                if (ok) stages(end, nk, [&](uint32_t at, bool add) {
                    products_end<false, false>(d, at, bn, add, p.last_steps);
                });
            }
            if (ok && elect()) mma_commit(sums_full + 8 * b);
            __syncwarp();
        }
        if (!ok) {                                       // products in flight
            if (elect()) mma_commit(drained);
            __syncwarp();
            int none = 0;
            if (lane == 0) drain_failed |= !mbar_wait(drained, 0, kDrainLimit, &none);
        }
    } else if (warp >= 4) {                              // ---- epilogue
        const int q = warp & 3;                          // the warp's quarter of the lanes
        const int half = (warp - 4) >> 2;                // and half of the columns
        const uint32_t buf = staging + (warp - 4) * kWarpStage;
        float2* share = reinterpret_cast<float2*>(raw + (staging - smem_u32(raw))) + q * 32 + lane;
        const float unit = K == kLse ? 1.0f : *a.unit;
        for (int i = 0, u; (u = unit_of(a, pair, pairs, i)) >= 0; ++i) {
            const bool first = K != kGrads || u < a.x_units;
            const Product& p = first ? a.x : a.y;
            const Unit t = unit_at(p, first ? u : u - a.x_units);
            const int b = i & 1;
            const int64_t row0 = (int64_t)t.m * BM + rank * 128 + q * 32;
            const Row info = row_of<K>(a, row0 + lane, unit);
            if (!warp_wait(sums_full + 8 * b, (i >> 1) & 1, a.wait_limit, dead)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t from = tmem + b * BN + ((uint32_t)(q * 32) << 16);
            if constexpr (K == kLse) {
                if (!epilogue_lse(a, t, from, row0 + lane, info, half, share + b * 128,
                                  shared_full + 8 * (4 * b + q), (i >> 1) & 1, dead))
                    break;
            } else if constexpr (K == kP) {
                epilogue_bf16<true>(a, p, t, from, row0, info, lane, half, buf);
            } else if (first) {
                epilogue_f32(a, t, from, row0, lane, half, buf);
            } else {
                epilogue_bf16<false>(a, p, t, from, row0, info, lane, half, buf);
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(in_leader(sums_empty + 8 * b));
        }
    }
    __syncwarp();
    if (drain_failed && a.status) atomicOr(a.status, ZERO_DEV_DRAIN_FAILED);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0 && *dead && a.status) atomicOr(a.status, ZERO_DEV_TIMEOUT);
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------ small parts --

// Joins a row's tiles: a block takes 32 rows, its 32 warps every 32nd tile.
struct JoinArgs {
    const float2* part;
    const float* at_target;
    const void* targets;
    int64_t part_ld, T, V;
    int32_t n_tiles, token_bytes;
    float* loss;
    float* lse;
    int32_t* status;
};

__global__ void __launch_bounds__(1024) k_xent_join(const __grid_constant__ JoinArgs a)
{
    pdl_enter();
    __shared__ float2 all[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + lane;
    // what the end needs, asked for first
    const int64_t r = (int64_t)blockIdx.x * 32 + warp;
    const bool last = lane == 0 && r < a.T;
    const int64_t y = last ? token_at(a.targets, a.token_bytes, r) : -1;
    const float at_target = last ? a.at_target[r] : 0.0f;      // meaningless without a target
    float m = -INFINITY, s = 0.0f;
    if (row < a.T) {
#pragma unroll 8
        for (int n = warp; n < a.n_tiles; n += 32) join(m, s, a.part[n * a.part_ld + row]);
    }
    all[lane][warp] = make_float2(m, s);
    __syncthreads();
    float2 x = all[warp][lane];                            // a row's 32 shares in a warp
    m = x.x;
    s = x.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float2 z = make_float2(__shfl_down_sync(0xFFFFFFFFu, m, o),
                                     __shfl_down_sync(0xFFFFFFFFu, s, o));
        join(m, s, z);
    }
    if (last) {
        // log s plus the distance from the target's logit to the maximum: the
        // difference of lse and the logit would carry lse's rounding (3e-5 at 500)
        const float log_s = logf(s);
        const float rest = fabsf(m) < INFINITY ? fmaf(m, kUnLog2eRest, log_s) : log_s;
        a.lse[r] = fmaf(m, kUnLog2e, rest);
        if (y >= a.V && a.status) atomicOr(a.status, ZERO_DEV_BAD_TOKEN);
        a.loss[r] = y >= 0 && y < a.V ? fmaf(m, kUnLog2e, -at_target) + rest : 0.0f;
    }
}

// h with the ignored rows zeroed: their P is zero, but zero times an Inf or a
// NaN that such a row may hold would reach every row of the table's gradient.
// Block 0 also finds u, the largest finite |dloss| of the tokens that count.
struct CleanArgs {
    const uint16_t* h;
    uint16_t* out;
    const float* dloss;
    float* unit;
    const void* targets;
    int64_t T, V, h_ld;
    int32_t D, token_bytes;
    int32_t* status;
};

__global__ void __launch_bounds__(256) k_clean(const __grid_constant__ CleanArgs a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31, nv = a.D >> 3;
    if (blockIdx.x == 0) {
        __shared__ float best[8];
        float u = 0.0f;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < a.T; i += 256) {
            const int64_t y = token_at(a.targets, a.token_bytes, i);
            const float g = fabsf(a.dloss[i]);
            if (y >= 0 && y < a.V && g < INFINITY) u = fmaxf(u, g);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) u = fmaxf(u, __shfl_xor_sync(0xFFFFFFFFu, u, o));
        if (lane == 0) best[threadIdx.x >> 5] = u;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int k = 1; k < 8; ++k) u = fmaxf(u, best[k]);
            *a.unit = u > 0.0f ? u : 1.0f;
        }
    }
    const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    if (t >= a.T) return;
    const int64_t y = token_at(a.targets, a.token_bytes, t);
    if (y >= a.V && lane == 0 && a.status) atomicOr(a.status, ZERO_DEV_BAD_TOKEN);
    const bool live = y >= 0 && y < a.V;
#pragma unroll 4
    for (int c = lane; c < nv; c += 32)
        st16(a.out + t * a.D + c * 8, live ? ld16(a.h + t * a.h_ld + c * 8) : make_uint4(0, 0, 0, 0));
}

// dh from its splits' sums, added in order, and what the target's entry lost.
// Rows of no token are zeros whatever the sums hold: their P is zero, but zero
// times an Inf or a NaN of the table is not.
struct FinishArgs {
    const float* sums;
    const float* unit;
    const float* lost;
    const uint16_t* table;
    const void* targets;
    uint16_t* dh;
    int64_t T, V, split_rows, dh_ld;
    int32_t D, splits, token_bytes;
};

// G threads share a vector of 8 columns (many splits: few tokens), each with every
// G-th split; their sums are added in order.
template <int G>
__global__ void __launch_bounds__(256) k_finish(const __grid_constant__ FinishArgs a)
{
    pdl_enter();
    constexpr int VECS = 256 / G;
    __shared__ float share[G > 1 ? G : 1][8][G > 1 ? VECS : 1];
    const int nv = a.D >> 3, lane = threadIdx.x % VECS, group = threadIdx.x / VECS;
    const int64_t i = (int64_t)blockIdx.x * VECS + lane;
    const int64_t t = i / nv;
    const int c = (int)(i - t * nv) * 8;
    const bool in = t < a.T;
    const float unit = *a.unit;
    float f[8] = {};
    const int64_t target = in && group == 0 ? token_at(a.targets, a.token_bytes, t) : -1;
    const bool live = target >= 0 && target < a.V;
    const float lost = live ? a.lost[t] : 0.0f;
    const uint4 row = live ? ld16(a.table + target * a.D + c) : make_uint4(0, 0, 0, 0);
    if (in) {
#pragma unroll 4
        for (int s = group; s < a.splits; s += G) {
            const float* p = a.sums + (s * a.split_rows + t) * a.D + c;
            const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
            const float4 y = __ldcs(reinterpret_cast<const float4*>(p + 4));
            f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
            f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
        }
    }
    if constexpr (G > 1) {
#pragma unroll
        for (int q = 0; q < 8; ++q) share[group][q][lane] = f[q];
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int k = 1; k < G; ++k)
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] += share[k][q][lane];
    }
    if (!in) return;
    if (lost != 0.0f) {
        float e[8];
        bf_unpack8(row, e);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = fmaf(lost, e[q], f[q]);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = live ? f[q] * unit : 0.0f;
    st16_stream(a.dh + t * a.dh_ld + c, bf_pack8(f));
}

// ------------------------------------------------------------------- host --

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// A row-major bf16 matrix (row stride `ld` elements), in boxes of 64 columns.
bool encode(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t steps[2] = {1, 1};
    const EncodeFn fn = encoder();
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides,
                    box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tiles(int64_t n, int width = 256) { return (int)((n + width - 1) / width); }

// The tile width along n (a multiple of `step`, 128 to 256): the one for which
// the CTA pair with the most tiles has the least to do, a tile's time being
// taken as that of its columns and 64 more (it reads the same 256 rows of the
// other operand however narrow it is: without the 64, tiles of 128 and 192
// were chosen at 8192 x 128256 x 2048 and made the gradient 40 % slower).  With
// many tiles that is 256; with few it evens out the last round.
int tile_width(int64_t n, int64_t m_tiles, int64_t splits, int step)
{
    const int64_t pairs = std::max(1, device_sms() / 2);
    int best = 256;
    int64_t least = INT64_MAX;
    for (int w = 256; w >= 128; w -= step) {
        const int64_t cost = (m_tiles * tiles(n, w) * splits + pairs - 1) / pairs * (w + 64);
        if (cost < least) {
            least = cost;
            best = w;
        }
    }
    return best;
}

// Where the sum of length `k` and the rows of `a` end.
void set_boxes(Product& p, int64_t k)
{
    p.k_blocks = (int32_t)((k + BK - 1) / BK);
    p.last_steps = (int32_t)((k - (int64_t)(p.k_blocks - 1) * BK + 15) / 16);
    p.k_box = p.k_blocks == 1 ? 16 * p.last_steps : BK;
    p.a_box = (int32_t)std::min<int64_t>(128, up(p.rows, 8));
    p.a_ctas = p.rows <= 128 ? 1 : 2;
}

template <Kind K>
cudaError_t run_mma(MmaArgs& a, cudaStream_t st)
{
    static std::atomic<uint64_t> smem_set;
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void*>(&k_mma<K>), smem_bytes<K>(), smem_set);
    if (e != cudaSuccess) return e;
    const int pairs = std::max(1, std::min(a.x.units() + (K == kGrads ? a.y.units() : 0),
                                           device_sms() / 2));
    a.x_units = a.x.units();
    a.y_units = K == kGrads ? a.y.units() : 0;
    a.light = pairs;
    if (K == kGrads && a.x_units % pairs != 0) {
        // Units of x are long and do not come out even over the pairs; those that
        // got one less take as many of y's as last as long.
        a.light = a.x_units % pairs;
        // (A unit takes no less than its epilogue, about 12 stages' time.)
        const auto cost = [](const Product& p) {
            return (int64_t)std::max(12, (p.k_blocks + p.splits - 1) / p.splits) * (p.bn + 64);
        };
        const int64_t each = (cost(a.x) + cost(a.y) / 2) / cost(a.y);
        a.extra = (int32_t)std::min<int64_t>(a.y_units, each * (pairs - a.light));
    }
    return launch_clusters(k_mma<K>, dim3((unsigned)(2 * pairs)), kThreads, smem_bytes<K>(), 2, st,
                           a);
}

struct LossScratch {
    int64_t part_ld, part, at_target, bytes;
};

LossScratch loss_scratch(int64_t T, int64_t V)
{
    LossScratch s;
    s.part_ld = up(T, 32);
    s.part = 0;
    s.at_target = up(8 * s.part_ld * (int64_t)tiles(V, 128), 256);      // of the narrowest tiles
    s.bytes = s.at_target + up(4 * T, 256);
    return s;
}

// The backward pass's plan: the piece, the splits of dh's sum, the scratch.
struct GradPlan {
    int64_t piece, p, clean, sums, lost, unit, split_rows, bytes;
    int32_t splits;
};

GradPlan grad_plan(int64_t T, int64_t V, int32_t D, int64_t piece)
{
    GradPlan g;
    if (piece == 0) {
        // P of a piece is at most 512 MiB; equal pieces
        const int64_t most = std::max<int64_t>(kPieceAlign, kMostP / std::max<int64_t>(T, 1) /
                                                                kPieceAlign * kPieceAlign);
        const int64_t n = (V + most - 1) / most;
        piece = (V + n - 1) / n;
    }
    g.piece = std::min(up(piece, kPieceAlign), up(V, kPieceAlign));
    const int64_t t = (int64_t)tiles(T) * tiles(D);
    const int64_t k_blocks = (std::min(V, g.piece) + BK - 1) / BK;
    // few tokens: the sum over the piece is split so that every CTA pair has a part
    g.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(device_sms() / 2 / std::max<int64_t>(t, 1),
                                                              k_blocks));
    g.p = 0;
    g.clean = up(2 * T * g.piece, 256);
    g.sums = g.clean + up(2 * T * D, 256);
    g.split_rows = T;
    g.lost = g.sums + up(4 * g.split_rows * D * g.splits, 256);
    g.unit = g.lost + up(4 * T, 256);
    g.bytes = g.unit + 256;
    return g;
}

// What grad_plan() asks for at any number of tokens up to T: fewer tokens may
// take a larger piece, and split the sum of dh more often.
int64_t grad_bytes(int64_t T, int64_t V, int32_t D, int64_t piece)
{
    const int64_t all = up(V, kPieceAlign), longest = piece ? std::min(piece, all) : all;
    int64_t p = T * longest;                             // elements of P
    if (piece == 0) p = std::min(p, std::max<int64_t>(kMostP, T * kPieceAlign));
    // t tokens are split at most pairs / (tiles(t) tiles(D)) times
    const int64_t pairs = device_sms() / 2, d = tiles(D);
    const int64_t most = std::max<int64_t>(
        1, std::min<int64_t>(pairs / d, (std::min(V, longest) + BK - 1) / BK));
    const int64_t rows = std::max(T, std::min(T * most, BM * (pairs / d)));
    return up(2 * p, 256) + up(2 * T * D, 256) + up(4 * rows * D, 256) + up(4 * T, 256) + 256;
}

zero_status check_units(int64_t T, int64_t V, int32_t D)
{
    LM_CHECK(check_sizes(T, V, D));
    // the units of a launch are counted in 32 bits
    const int64_t t = tiles(T, 128), v = tiles(V, 128), d = tiles(D, 128);
    if (t * v > INT32_MAX / 2 || v * d > INT32_MAX / 2 || t * d > INT32_MAX / 2)
        return ZERO_ERR_SIZE;
    return ZERO_OK;
}

zero_status check_xent(int64_t T, int64_t V, int32_t D, int32_t target_bytes, int32_t flags,
                       const int32_t* dev_status)
{
    LM_CHECK(check_units(T, V, D));
    if (target_bytes != 4 && target_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (flags & ~ZERO_FLAG_DEBUG_EXPIRE_WAITS) return ZERO_ERR_INVALID_ARG;
    if (flags && !dev_status) return ZERO_ERR_NULL;
    return check_status(dev_status);
}

}  // namespace

extern "C" int64_t zero_xent_scratch_bytes(int64_t T, int64_t V, int32_t D)
{
    if (check_units(T, V, D) != ZERO_OK) return -1;
    return loss_scratch(T, V).bytes;
}

extern "C" zero_status zero_xent(const uint16_t* h, int64_t h_ld, const uint16_t* table, int64_t V,
                                 int32_t D, const void* targets, int32_t target_bytes, int64_t T,
                                 float* loss, float* lse, void* scratch, int64_t scratch_bytes,
                                 int32_t flags, int32_t* dev_status, void* stream)
{
    LM_CHECK(check_xent(T, V, D, target_bytes, flags, dev_status));
    LM_CHECK(check_ld(h_ld, D));
    if (T == 0) return ZERO_OK;
    LM_CHECK(check_ptr(h));
    LM_CHECK(check_ptr(table));
    LM_CHECK(check_tokens(targets, target_bytes));
    LM_CHECK(check_ptr(loss, 4));
    LM_CHECK(check_ptr(lse, 4));
    LM_CHECK(check_ptr(scratch));
    const LossScratch s = loss_scratch(T, V);
    if (scratch_bytes < s.bytes) return ZERO_ERR_SIZE;
    Spans sp;
    sp.rows(h, T, h_ld, D, 2, false);
    sp.add(table, 2 * V * D, false);
    sp.add(targets, T * target_bytes, false);
    sp.add(loss, 4 * T, true);
    sp.add(lse, 4 * T, true);
    sp.add(scratch, s.bytes, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    uint8_t* base = static_cast<uint8_t*>(scratch);
    MmaArgs a{};
    Product& x = a.x;
    x.m_tiles = tiles(T);
    x.bn = tile_width(V, x.m_tiles, 1, 16);
    x.n_tiles = tiles(V, x.bn);
    x.splits = 1;
    x.m_fast = 1;
    x.rows = T;
    x.cols = V;
    set_boxes(x, D);
    if (!encode(&x.a, h, D, T, h_ld, x.a_box) || !encode(&x.b, table, D, V, D, x.bn / 2))
        return ZERO_ERR_CUDA;
    a.token_bytes = target_bytes;
    a.targets = targets;
    a.V = V;
    a.part = reinterpret_cast<float2*>(base + s.part);
    a.part_ld = s.part_ld;
    a.at_target = reinterpret_cast<float*>(base + s.at_target);
    a.status = dev_status;
    a.wait_limit = flags & ZERO_FLAG_DEBUG_EXPIRE_WAITS ? 0 : kWaitLimit;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = run_mma<kLse>(a, st);
    if (e == cudaSuccess) {
        const JoinArgs j{a.part, a.at_target, targets, s.part_ld, T, V, x.n_tiles, target_bytes,
                         loss, lse, dev_status};
        e = launch(k_xent_join, dim3((unsigned)((T + 31) / 32)), 1024, 0, st, j);
    }
    return status_of(e);
}

extern "C" int64_t zero_xent_grad_scratch_bytes(int64_t T, int64_t V, int32_t D, int64_t piece)
{
    if (check_units(T, V, D) != ZERO_OK || piece < 0 || piece % kPieceAlign != 0) return -1;
    return grad_bytes(T, V, D, piece);
}

extern "C" zero_status zero_xent_grad(const uint16_t* h, int64_t h_ld, const uint16_t* table,
                                      int64_t V, int32_t D, const void* targets,
                                      int32_t target_bytes, int64_t T, const float* lse,
                                      const float* dloss, uint16_t* dh, int64_t dh_ld,
                                      uint16_t* dtable, int64_t piece, void* scratch,
                                      int64_t scratch_bytes, int32_t flags, int32_t* dev_status,
                                      void* stream)
{
    LM_CHECK(check_xent(T, V, D, target_bytes, flags, dev_status));
    LM_CHECK(check_ld(h_ld, D));
    LM_CHECK(check_ld(dh_ld, D));
    if (piece < 0 || piece % kPieceAlign != 0) return ZERO_ERR_INVALID_ARG;
    LM_CHECK(check_ptr(dtable));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return status_of(cudaMemsetAsync(dtable, 0, (size_t)(2 * V * D), st));
    LM_CHECK(check_ptr(h));
    LM_CHECK(check_ptr(table));
    LM_CHECK(check_tokens(targets, target_bytes));
    LM_CHECK(check_ptr(lse, 4));
    LM_CHECK(check_ptr(dloss, 4));
    LM_CHECK(check_ptr(dh));
    LM_CHECK(check_ptr(scratch));
    const GradPlan g = grad_plan(T, V, D, piece);
    if (scratch_bytes < g.bytes) return ZERO_ERR_SIZE;
    Spans sp;
    sp.rows(h, T, h_ld, D, 2, false);
    sp.add(table, 2 * V * D, false);
    sp.add(targets, T * target_bytes, false);
    sp.add(lse, 4 * T, false);
    sp.add(dloss, 4 * T, false);
    sp.rows(dh, T, dh_ld, D, 2, true);
    sp.add(dtable, 2 * V * D, true);
    sp.add(scratch, g.bytes, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    uint8_t* base = static_cast<uint8_t*>(scratch);
    uint16_t* P = reinterpret_cast<uint16_t*>(base + g.p);
    uint16_t* clean = reinterpret_cast<uint16_t*>(base + g.clean);
    float* sums = reinterpret_cast<float*>(base + g.sums);
    const unsigned row_blocks = (unsigned)((T + 7) / 8);
    float* unit = reinterpret_cast<float*>(base + g.unit);
    float* lost = reinterpret_cast<float*>(base + g.lost);
    const CleanArgs ca{h, clean, dloss, unit, targets, T, V, h_ld, D, target_bytes, dev_status};
    cudaError_t e = launch(k_clean, dim3(row_blocks), 256, 0, st, ca);

    MmaArgs common{};
    common.token_bytes = target_bytes;
    common.targets = targets;
    common.V = V;
    common.lse = lse;
    common.dloss = dloss;
    common.unit = unit;
    common.lost = lost;
    common.status = dev_status;
    common.wait_limit = flags & ZERO_FLAG_DEBUG_EXPIRE_WAITS ? 0 : kWaitLimit;
    for (int64_t v0 = 0; v0 < V && e == cudaSuccess; v0 += g.piece) {
        const int64_t n = std::min(g.piece, V - v0);
        const uint16_t* rows = table + v0 * D;

        MmaArgs first = common;                             // P = f(h E^T)
        first.v0 = v0;
        Product& p = first.x;
        p.m_tiles = tiles(T);
        p.bn = tile_width(n, p.m_tiles, 1, 64);
        p.n_tiles = tiles(n, p.bn);
        p.out = P;
        p.out_ld = g.piece;
        p.splits = 1;
        p.m_fast = 1;
        p.rows = T;
        p.cols = n;
        set_boxes(p, D);
        if (!encode(&p.a, h, D, T, h_ld, p.a_box) || !encode(&p.b, rows, D, n, D, p.bn / 2))
            return ZERO_ERR_CUDA;
        if ((e = run_mma<kP>(first, st)) != cudaSuccess) break;

        MmaArgs second = common;
        Product& d = second.x;                              // dh += P E
        d.out = sums;
        d.out_ld = D;
        d.rows = T;
        d.cols = D;
        set_boxes(d, n);
        if (!encode(&d.a, P, n, T, g.piece, d.a_box) || !encode(&d.b, rows, D, n, D, d.k_box))
            return ZERO_ERR_CUDA;
        d.splits = std::min(g.splits, d.k_blocks);
        d.m_tiles = tiles(T);
        d.bn = tile_width(D, d.m_tiles, d.splits, 64);
        d.n_tiles = tiles(D, d.bn);
        second.out_split_rows = g.split_rows;
        second.add = v0 > 0;

        Product& w = second.y;                              // dE = P^T h
        w.rows = n;
        w.cols = D;
        set_boxes(w, T);
        if (!encode(&w.a, P, n, T, g.piece, w.k_box) || !encode(&w.b, clean, D, T, D, w.k_box))
            return ZERO_ERR_CUDA;
        w.out = dtable + v0 * D;
        w.out_ld = D;
        w.m_tiles = tiles(n);
        w.bn = tile_width(D, w.m_tiles, 1, 64);
        w.n_tiles = tiles(D, w.bn);
        w.splits = 1;
        e = run_mma<kGrads>(second, st);
    }
    if (e == cudaSuccess) {
        const FinishArgs f{sums, unit,         lost,  table, targets,  dh,          T,
                           V,    g.split_rows, dh_ld, D,     g.splits, target_bytes};
        const int64_t vecs = T * (D / 8);
        if (g.splits >= 8)
            e = launch(k_finish<8>, dim3((unsigned)((vecs + 31) / 32)), 256, 0, st, f);
        else
            e = launch(k_finish<1>, dim3((unsigned)((vecs + 255) / 256)), 256, 0, st, f);
    }
    return status_of(e);
}
