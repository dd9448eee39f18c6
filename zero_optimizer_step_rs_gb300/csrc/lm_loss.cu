// lm_loss.cu - losses of packed sequences from their tokens' losses, and the
// gradients of the tokens' losses: pairs of a chosen and a rejected sequence
// (zero_preference), and the clipped policy loss with a KL term (zero_policy).
// Declared in include/zero_step.h.
//
// Both are a sum per sequence of a term per token, and a gradient per token from a
// number per sequence.  The tokens are cut into tiles, one warp's each, whatever the
// sequences' lengths are.  A tile meets the sequences s0, s0 + 1, ...; going
// along the tokens either the tile or the sequence steps on, so that tile + s is a
// slot of its own for every pair that meets, the slots of a sequence lie one behind
// the other, and no slot needs clearing.  The sequence's slots are then joined, with what
// the additions round away kept beside the sum: no atomics, the same bits in every call.
//
// A token is 16 to 24 bytes read and 4 written in the gradient, which reads them once more.
// Measured, one GB300, with the gradient: 2^20 tokens of 256 pairs 9.5 us, of 512 sequences of the
// policy 15.0 us (2.2 and 2.0 TB/s of what they cannot do without).  About 5 us of each are three
// launches and their first loads' way; each half million tokens of the policy more takes 4.9 us,
// 5.4 TB/s of what both passes read, with half of the issue slots full.  999 tokens of 4 pairs take
// 5.2 us, 1501 of 16 sequences of the policy 6.6: two launches.
#include "lm_common.cuh"

#include <math.h>

namespace {

using namespace lm;

// Tokens of a lane.  A warp with 8 of the policy's takes over 1000 instructions one after the
// other, several us of a call of few tokens; with 1 it does less work per instruction (the
// search for its sequences, the sums' halvings), which costs where there are many: 2^20 tokens
// of the policy 15.8 us with 4 and 16.2 with 8, of preferences 11.0 and 9.7; 30000 of the policy
// 6.8 us with 1 and 7.5 with 2.
//
// The limit between few and many is the same for both kinds.  Batches of even lengths of the policy
// would take 1 for longer (of 512 sequences, 1 / 4 a lane: 65535 tokens 7.5 / 10.5 us, 200000 9.0 /
// 10.3, 300000 10.6 / 10.7), but where one sequence has most of the tokens its join has four times as
// many parts (the others 4 tokens each: 65535 25 / 33, 100000 35 / 34, 200000 62 / 42).
// Preferences, 1 / 8 a lane: 65535 tokens of 512 sequences 7.3 / 8.3, of 16 7.1 / 6.6, 200000 9.1 /
// 8.8 and 9.3 / 9.1; with one long sequence 65535 13 / 24, 200000 24 / 26.
constexpr int kFewItems = 1;
constexpr int many_items(int kind) { return kind == 0 ? 8 : 4; }
constexpr int64_t kFew = 1 << 16;                    // tokens from which on a lane takes several
constexpr int kThreads = 128;
constexpr int kAloneTiles = 48, kAloneSequences = 16;    // the most that one block takes alone
constexpr int kWideThreads = 512;                    // of a block that joins one result's parts
constexpr int64_t kWideTiles = 128;                  // parts a result from which on it does
constexpr unsigned kAll = 0xFFFFFFFFu;

template <int ITEMS>
constexpr int kTile = 32 * ITEMS;                    // tokens of a warp

enum Kind { kPreference, kPolicy };

// What a tile adds to a sequence.
struct __align__(16) Part {
    float a, k;                                      // the terms' sum, the KL estimates' sum
    int32_t count, clipped;
};

struct LossArgs {
    const float* nll;
    const float* old;                                // may be null
    const float* ref;                                // may be null
    const float* adv;
    const void* targets;
    const void* offsets;
    Part* parts;                                     // [tiles + S]
    int32_t* status;                                 // may be null
    float* loss;
    float* slope;
    float* ratios;
    float* kl;
    int32_t* counts;
    int32_t* clipped;
    const int32_t* counts_in;                        // gradients: what the forward call gave
    const float* slope_in;
    const float* dloss;
    float* dnll;
    int32_t T, S, tiles;                             // (tiles + S slots: below 2^31 as well)
    int32_t target_bytes, offset_bytes, per_token, average, kind;
    float kl_coef;
    float bound_lo, bound_hi;                        // 1 - clip_low, 1 + clip_high
    float edge_lo, edge_hi;                          // their logarithms, rounded
    float rest_lo, rest_hi;                          // and what that lost
    double beta, margin;
    float smoothing;
};

__device__ __forceinline__ int64_t raw_offset(const LossArgs& a, int i)
{
    return token_at(a.offsets, a.offset_bytes, i);
}

// The number of offsets (of S + 1) that are at most t, by a search in 32 parts.
__device__ __forceinline__ int offsets_up_to(const LossArgs& a, int t, int lane)
{
    int lo = 0, hi = a.S + 1;
    while (lo < hi) {
        const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
        const bool below = i < hi && raw_offset(a, i) <= t;
        const int n = __popc(__ballot_sync(kAll, below));
        if (n == 0) break;
        hi = min(hi, lo + n * step);
        lo += (n - 1) * step + 1;
    }
    return lo;
}

// exp(d) - d - 1 for |d| <= 1, where the three cancel: the exponential's series from its
// third term on.  The first term left out, d^13 / 13!, is under 2^-30 of the sum.
__device__ __forceinline__ float drift_series(float d)
{
    float p = 1.0f / 479001600.0f;
    p = fmaf(p, d, 1.0f / 39916800.0f);
    p = fmaf(p, d, 1.0f / 3628800.0f);
    p = fmaf(p, d, 1.0f / 362880.0f);
    p = fmaf(p, d, 1.0f / 40320.0f);
    p = fmaf(p, d, 1.0f / 5040.0f);
    p = fmaf(p, d, 1.0f / 720.0f);
    p = fmaf(p, d, 1.0f / 120.0f);
    p = fmaf(p, d, 1.0f / 24.0f);
    p = fmaf(p, d, 1.0f / 6.0f);
    p = fmaf(p, d, 0.5f);
    return p * d * d;
}

// What old - nll lost in its rounding (Knuth's two-sum).
__device__ __forceinline__ float lost(float old, float nll, float change)
{
    const float back = __fsub_rn(change, old);
    return __fsub_rn(__fsub_rn(old, __fsub_rn(change, back)), __fadd_rn(nll, back));
}

// A lane's tokens of a tile: t = base + 32 j + lane.
template <int ITEMS>
struct Tokens {
    float nll[ITEMS], old[ITEMS], ref[ITEMS], adv[ITEMS];
    unsigned live;                                   // bit j: token j counts
};

// FULL: the whole tile lies below T.
template <Kind K, bool GRAD, int ITEMS, bool FULL>
__device__ __forceinline__ void load_some(const LossArgs& a, int base, int lane,
                                          Tokens<ITEMS>& x)
{
    const int at = base + lane, n = a.T - at;        // the lane's first token, tokens from there on
    int id[ITEMS];                                   // (only the sign is looked at)
    if (a.target_bytes == 8) {
        const auto* p = static_cast<const long long*>(a.targets) + at;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) id[j] = FULL || j * 32 < n ? (int)(p[j * 32] >> 32) : -1;
    } else {
        const auto* p = static_cast<const int*>(a.targets) + at;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) id[j] = FULL || j * 32 < n ? p[j * 32] : -1;
    }
    const auto values = [&](float (&v)[ITEMS], const float* p) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) v[j] = p && (FULL || j * 32 < n) ? (p + at)[j * 32] : 0.0f;
    };
    if (K == kPolicy || !GRAD) {
        values(x.nll, a.nll);
        values(x.ref, a.ref);
    }
    if (K == kPolicy) {
        values(x.old, a.old);
        values(x.adv, a.per_token ? a.adv : nullptr);
    }
    x.live = 0;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) x.live |= (~(unsigned)id[j] >> 31) << j;
}

template <Kind K, bool GRAD, int ITEMS>
__device__ __forceinline__ void load_tokens(const LossArgs& a, int base, int lane,
                                            Tokens<ITEMS>& x)
{
    if (kTile<ITEMS> <= a.T - base) load_some<K, GRAD, ITEMS, true>(a, base, lane, x);
    else load_some<K, GRAD, ITEMS, false>(a, base, lane, x);
}

// The policy's tokens by themselves, whatever their advantage is: the ratios r, exp(d) - d -
// 1 or (GRAD) exp(d) - 1 of d = nll - ref, and which tokens have r above the upper and below
// the lower bound (bit j: token j).
//
// The bounds are compared as logarithms, old - nll with log(bound), and as exact numbers:
// rounding keeps the order, so only a difference that rounds to the same fp32 value as the logarithm
// needs what both roundings lost.  Such tokens, and those with |d| > 1, are few: the warp
// looks for them once and takes them by themselves.  (Made for every token these took a third of
// the time; the comparison in 64 bits, half.)
template <int ITEMS>
struct Ratios {
    float r[ITEMS], k[ITEMS];
    unsigned high, low;
};
template <bool GRAD, int ITEMS>
__device__ __forceinline__ Ratios<ITEMS> ratios_of(const LossArgs& a, const Tokens<ITEMS>& x)
{
    Ratios<ITEMS> v;
    v.high = v.low = 0;
    bool tie = false, far = false;
    const bool drifts = GRAD ? a.kl_coef != 0.0f : a.ref != nullptr;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const float change = a.old ? x.old[j] - x.nll[j] : 0.0f;
        v.r[j] = expf(change);
        v.high |= (change > a.edge_hi ? 1u : 0u) << j;
        v.low |= (change < a.edge_lo ? 1u : 0u) << j;
        tie |= change == a.edge_hi || change == a.edge_lo;
        v.k[j] = 0.0f;
        if (drifts) {
            const float d = x.nll[j] - x.ref[j], k = drift_series(d);
            v.k[j] = GRAD ? d + k : k;
            far |= !(fabsf(d) <= 1.0f);
        }
    }
    if (__any_sync(kAll, tie) && a.old) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const float change = x.old[j] - x.nll[j], rest = lost(x.old[j], x.nll[j], change);
            if (change == a.edge_hi && rest > a.rest_hi) v.high |= 1u << j;
            if (change == a.edge_lo && rest < a.rest_lo) v.low |= 1u << j;
        }
    }
    if (__any_sync(kAll, far)) {
#pragma unroll 1
        for (int j = 0; j < ITEMS; ++j) {
            float d = 0.0f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (i == j) d = x.nll[i] - x.ref[i];
            if (!__any_sync(kAll, !(fabsf(d) <= 1.0f))) continue;
            const float e = expf(d) - 1.0f, k = GRAD ? e : e - d;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (i == j && !(fabsf(d) <= 1.0f)) v.k[i] = k;
        }
    }
    return v;
}

// A lane's tokens of [lo, hi) of a tile, as bits.
template <int ITEMS>
__device__ __forceinline__ unsigned tokens_in(int lo, int hi, int lane)
{
    const int from = (max(lo - lane, 0) + 31) >> 5, to = (max(hi - lane, 0) + 31) >> 5;
    return (1u << to) - (1u << from);
}

// The advantages above and below 0 of a lane's tokens, as bits.
template <int ITEMS>
__device__ __forceinline__ void signs_of(const float (&A)[ITEMS], unsigned& pos, unsigned& neg)
{
    pos = neg = 0;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        pos |= (A[j] > 0.0f ? 1u : 0u) << j;
        neg |= (A[j] < 0.0f ? 1u : 0u) << j;
    }
}

// How many sequences from s on begin at `at` or before, rounded down to a power of two.  A call of its
// own: inside of the gradient it takes registers from the common way (2^20 tokens of the policy 8.0 us
// instead of 7.6).
__device__ __noinline__ int passed_over(const LossArgs& a, int s, int64_t at)
{
    const unsigned far = (unsigned)s + (1u << (threadIdx.x & 31));
    const bool before = far <= (unsigned)a.S && raw_offset(a, (int)far) <= at;
    const int lanes = __popc(__ballot_sync(kAll, before));
    return lanes ? 1 << (lanes - 1) : 0;
}

// Calls f(s, lo, hi, of(s)) for every sequence from s0 on that the tile at base meets, with the
// part [base + lo, base + hi) of it that lies inside.  The bounds and of(s) of 32 sequences are
// fetched at once, one a lane.  Where none of these has a token in the tile, the lanes look 2^lane
// sequences further on and the warp goes where still none had one: what a buffer of a fixed size has
// left over ends in one tile, and 31 at a time 2^20 empty sequences would take 34000 rounds (2^30,
// ten seconds and more).  Offsets that fall end it.
template <int ITEMS, typename Of, typename F>
__device__ __forceinline__ void for_sequences(const LossArgs& a, int base, int s0, int lane,
                                              Of&& of, F&& f)
{
    const int n = min(kTile<ITEMS>, a.T - base);
    for (int s = max(s0, 0); s < a.S;) {
        const int64_t bound = raw_offset(a, min(s + lane, a.S));
        const int lo = bound <= base ? 0 : (int)min(bound - base, (int64_t)n);
        const float2 about = of(min(s + lane, a.S - 1));
        const int hi = __shfl_down_sync(kAll, lo, 1);
        // (the last lane's sequence is the next round's first; past the last one none begins)
        unsigned left = __ballot_sync(kAll, lane < 31 && s + lane < a.S && lo < hi);
        while (left) {
            const int k = __ffs(left) - 1;
            left &= left - 1;
            f(s + k, __shfl_sync(kAll, lo, k), __shfl_sync(kAll, hi, k),
              make_float2(__shfl_sync(kAll, about.x, k), __shfl_sync(kAll, about.y, k)));
        }
        const int end = __shfl_sync(kAll, lo, 31);
        if (end >= n || __any_sync(kAll, lane < 31 && lo > hi)) return;
        s += 31;
        if (__shfl_sync(kAll, lo, 0) == end) s += passed_over(a, s, base + end);
    }
}

// The terms of a tile, summed for each sequence that it meets.
template <Kind K, int ITEMS>
__device__ __forceinline__ void tile_parts(const LossArgs& a, Part* parts, int tile, int lane)
{
    const int base = tile * kTile<ITEMS>;
    Tokens<ITEMS> x;
    load_tokens<K, false, ITEMS>(a, base, lane, x);
    const int s0 = offsets_up_to(a, base, lane) - 1;     // while the tokens are on their way
    Ratios<ITEMS> v;
    if (K == kPolicy) {
        v = ratios_of<false>(a, x);
    } else {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) v.r[j] = x.ref[j] - x.nll[j];
    }
    const auto about = [&](int s) {
        return make_float2(K == kPolicy && !a.per_token ? a.adv[s] : 0.0f, 0.0f);
    };
    for_sequences<ITEMS>(a, base, s0, lane, about, [&](int s, int lo, int hi, float2 of_s) {
        const unsigned mine = tokens_in<ITEMS>(lo, hi, lane) & x.live;
        float sum = 0.0f, ksum = 0.0f;
        int both = __popc(mine);                     // clipped tokens above bit 16, all below
        if (K == kPreference) {
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) sum += mine >> j & 1 ? v.r[j] : 0.0f;
        } else {
            if (!a.per_token)
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) x.adv[j] = of_s.x;
            unsigned pos, neg;
            signs_of(x.adv, pos, neg);
            both += __popc(mine & (v.high & pos | v.low & neg)) << 16;
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) {
                // -min(r A, bounded r A); where A is 0 no r, Inf among them, counts
                const float A = x.adv[j];
                // (comparisons that a NaN fails, so that it stays)
                const float r = A > 0.0f ? (v.r[j] > a.bound_hi ? a.bound_hi : v.r[j])
                                         : (v.r[j] < a.bound_lo ? a.bound_lo : v.r[j]);
                float term = A == 0.0f ? 0.0f : -(r * A);
                if (a.kl_coef != 0.0f) term = fmaf(a.kl_coef, v.k[j], term);
                sum += mine >> j & 1 ? term : 0.0f;
                ksum += mine >> j & 1 ? v.k[j] : 0.0f;
            }
        }
        sum = warp_sum(sum);
        if (K == kPolicy) ksum = warp_sum(ksum);
        both = __reduce_add_sync(kAll, both);
        if (lane == 0) parts[tile + s] = Part{sum, ksum, both & 0xFFFF, both >> 16};
    });
}

// A sum in two parts, of which the second holds what the roundings lost (up to its own).
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair plus(Pair x, float y)
{
    const float s = x.hi + y, back = s - x.hi;
    return {s, x.lo + ((x.hi - (s - back)) + (y - back))};
}
__device__ __forceinline__ Pair warp_pair(Pair x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(kAll, x.hi, o), lo = __shfl_xor_sync(kAll, x.lo, o);
        // both lanes of a pair add the same two numbers in the same order
        const bool upper = threadIdx.x & o;
        x = plus(Pair{upper ? hi : x.hi, x.lo + lo}, upper ? x.hi : hi);
    }
    return x;
}
__device__ __forceinline__ double whole(Pair x)
{
    // (Inf and NaN have no rest)
    return fabsf(x.hi) <= 3.0e38f ? (double)x.hi + (double)x.lo : (double)x.hi;
}
// x / n for a count n: the quotient, and that of what it leaves.
__device__ __forceinline__ Pair share(Pair x, int32_t n)
{
    if (n <= 1 || !(fabsf(x.hi) <= 3.0e38f)) return n > 1 ? Pair{x.hi / (float)n, 0.0f} : x;
    const float d = (float)n, more = (float)(n - (int32_t)d);
    const float q = x.hi / d;
    return {q, (fmaf(-q, more, fmaf(-q, d, x.hi)) + x.lo) / d};
}

struct Sums {
    Pair a, k;
    int32_t count, clipped;
};

// The parts of sequence s = [from, to), each of n threads taking every n-th; joined over the
// warp's lanes.
template <Kind K, int ITEMS>
__device__ __forceinline__ Sums join_parts(const LossArgs& a, const Part* parts, int s, int64_t from,
                                           int64_t to, int thread, int n)
{
    Sums r{{0.0f, 0.0f}, {0.0f, 0.0f}, 0, 0};
    if (from < 0 || to < from || to > a.T) {
        if (thread == 0 && a.status) atomicOr(a.status, ZERO_DEV_BAD_OFFSETS);
        return r;
    }
    if (from == to) return r;
    const int first = (int)from / kTile<ITEMS> + s, last = ((int)to - 1) / kTile<ITEMS> + s;
#pragma unroll 8
    for (int i = first + thread; i <= last; i += n) {
        const Part p = parts[i];
        r.a = plus(r.a, p.a);
        if (K == kPolicy) r.k = plus(r.k, p.k);
        r.count += p.count;
        r.clipped += p.clipped;
    }
    r.a = warp_pair(r.a);
    if (K == kPolicy) r.k = warp_pair(r.k);
    r.count = __reduce_add_sync(kAll, r.count);
    if (K == kPolicy) r.clipped = __reduce_add_sync(kAll, r.clipped);
    return r;
}

// The same over the warps of a block that has one result.
__device__ __forceinline__ Sums join_warps(Sums r)
{
    __shared__ Sums all[kWideThreads / 32];
    __syncthreads();                                 // (a pair's two sequences use it in turn)
    if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = r;
    __syncthreads();
    r = all[0];
    for (int w = 1; w < kWideThreads / 32; ++w) {
        const Sums x = all[w];
        r.a = plus(Pair{r.a.hi, r.a.lo + x.a.lo}, x.a.hi);
        r.k = plus(Pair{r.k.hi, r.k.lo + x.k.lo}, x.k.hi);
        r.count += x.count;
        r.clipped += x.clipped;
    }
    return r;
}

__device__ __forceinline__ float softplus(float x)
{
    return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// Pair p's loss from its two sequences, or sequence p's, by a warp or (WIDE) a block.
template <Kind K, int ITEMS, bool WIDE>
__device__ __forceinline__ void finish(const LossArgs& a, const Part* parts, int p)
{
    const int thread = WIDE ? threadIdx.x : threadIdx.x & 31, n = WIDE ? kWideThreads : 32;
    if (K == kPolicy) {
        const int64_t from = raw_offset(a, p), to = raw_offset(a, p + 1);
        Sums r = join_parts<K, ITEMS>(a, parts, p, from, to, thread, n);
        if (WIDE) r = join_warps(r);
        if (thread) return;
        if (a.average) {
            r.a = share(r.a, r.count);
            r.k = share(r.k, r.count);
        }
        a.loss[p] = (float)whole(r.a);
        a.kl[p] = (float)whole(r.k);
        a.counts[p] = r.count;
        a.clipped[p] = r.clipped;
        return;
    }
    const int64_t from = raw_offset(a, 2 * p), mid = raw_offset(a, 2 * p + 1),
                  to = raw_offset(a, 2 * p + 2);
    Sums c = join_parts<K, ITEMS>(a, parts, 2 * p, from, mid, thread, n);
    Sums r = join_parts<K, ITEMS>(a, parts, 2 * p + 1, mid, to, thread, n);
    if (WIDE) {
        c = join_warps(c);
        r = join_warps(r);
    }
    if (thread) return;
    if (a.average) {
        c.a = share(c.a, c.count);
        r.a = share(r.a, r.count);
    }
    const double chosen = whole(c.a), rejected = whole(r.a);
    a.ratios[2 * p] = (float)chosen;
    a.ratios[2 * p + 1] = (float)rejected;
    a.counts[2 * p] = c.count;
    a.counts[2 * p + 1] = r.count;
    const double d = chosen - rejected;
    float loss, slope;
    if (a.kind == ZERO_PREF_IPO) {
        const double e = d - a.margin;                     // (margin + 1/(2 beta))
        loss = (float)(e * e);
        slope = (float)(2.0 * e);
    } else {
        const double z = a.beta * d - a.margin;
        if (a.kind == ZERO_PREF_HINGE) {
            loss = z >= 1.0 ? 0.0f : (float)(1.0 - z);     // NaN stays NaN
            slope = z >= 1.0 ? 0.0f : z < 1.0 ? (float)-a.beta : (float)z;
        } else {
            const float f = (float)z, e = a.smoothing;
            loss = (1.0f - e) * softplus(-f);
            if (e != 0.0f) loss = fmaf(e, softplus(f), loss);
            // d/dz: e sigmoid(z) - (1 - e) sigmoid(-z)
            const float q = expf(-fabsf(f)), big = 1.0f / (1.0f + q), small = q / (1.0f + q);
            const float up = f >= 0.0f ? big : small, down = f >= 0.0f ? small : big;
            slope = (float)a.beta * (e * up - (1.0f - e) * down);
        }
    }
    a.loss[p] = loss;
    a.slope[p] = slope;
}

template <Kind K, int ITEMS>
__global__ void __launch_bounds__(kThreads) k_loss_parts(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int tile = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile < a.tiles) tile_parts<K, ITEMS>(a, a.parts, tile, threadIdx.x & 31);
}

template <Kind K, int ITEMS, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kWideThreads : kThreads)
    k_loss_join(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int p = WIDE ? blockIdx.x : blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (p < (K == kPreference ? a.S / 2 : a.S)) finish<K, ITEMS, WIDE>(a, a.parts, p);
}

// Few tokens: one block does both, and the parts stay in its shared memory.  Calls this small keep
// the host longer than the GPU (about 5.1 us with the gradient, 6.7 with a launch more), so the limits are
// where a call with its gradient, one behind the other from the host, takes as long in either
// form.  us in one block / in two launches, in brackets the same in a graph, where the host's time
// does not count and up to 32 tiles, one a warp, are the limit:
//   policy, sequences     1000 tokens             1536                    1750           2048
//      4            5.2 / 6.8 (4.9, 4.9)   6.0 / 6.9 (5.7, 4.9)   6.2 / 6.9        6.4 / 7.0
//     16            6.0 / 6.8 (5.7, 5.4)   6.9 / 6.9 (6.6, 5.4)   7.0 / 6.7        7.2 / 7.1
//   preferences, pairs    1000                    1536
//      4            5.7 / 6.6 (5.4, 5.8)   6.3 / 6.6 (6.0, 5.7)
//      8            5.8 / 6.2 (5.6, 5.7)   at 1100: 6.2 / 6.2 (6.0, 5.6)
//     12            6.4 / 6.1 (6.2, 5.7)   at 200:  6.6 / 6.8 (6.4, 6.4)
//     16            7.4 / 6.7 (7.1, 6.2)   at 200:  7.7 / 7.6 (7.4, 7.2)
template <Kind K>
__global__ void __launch_bounds__(1024) k_loss_alone(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    __shared__ Part parts[kAloneTiles + kAloneSequences];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    for (int tile = warp; tile < a.tiles; tile += warps)
        tile_parts<K, kFewItems>(a, parts, tile, threadIdx.x & 31);
    __syncthreads();
    for (int p = warp; p < (K == kPreference ? a.S / 2 : a.S); p += warps)
        finish<K, kFewItems, false>(a, parts, p);
}

// The gradient of each token's loss.
template <Kind K, int ITEMS>
__global__ void __launch_bounds__(kThreads) k_loss_grad(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int tile = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile >= a.tiles) return;
    const int base = tile * kTile<ITEMS>;
    Tokens<ITEMS> x;
    load_tokens<K, true, ITEMS>(a, base, lane, x);
    const int s0 = offsets_up_to(a, base, lane) - 1;
    Ratios<ITEMS> v;
    if (K == kPolicy) {
        v = ratios_of<true>(a, x);
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) v.k[j] *= a.kl_coef;
    }
    // the advantage, where it is the sequence's, and the upstream gradient of its tokens
    const auto about = [&](int s) {
        float back = a.dloss[K == kPolicy ? s : s >> 1];
        if (K == kPreference) {
            back *= a.slope_in[s >> 1];
            if (!(s & 1)) back = -back;
        }
        if (a.average) back /= (float)max(a.counts_in[s], 1);
        return make_float2(K == kPolicy && !a.per_token ? a.adv[s] : 0.0f, back);
    };
    for_sequences<ITEMS>(a, base, s0, lane, about, [&](int s, int lo, int hi, float2 of_s) {
        const unsigned in = tokens_in<ITEMS>(lo, hi, lane);
        const float back = of_s.y;
        float* out = a.dnll + base + lane;
        unsigned over = 0;
        if (K == kPolicy) {
            if (!a.per_token)
#pragma unroll
                for (int j = 0; j < ITEMS; ++j) x.adv[j] = of_s.x;
            unsigned pos, neg;
            signs_of(x.adv, pos, neg);
            // clipped, or an advantage of 0, which makes no ratio count, Inf among them
            over = v.high & pos | v.low & neg | ~(pos | neg);
        }
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            float g = back;
            if (K == kPolicy) g = fmaf(over >> j & 1 ? 0.0f : v.r[j], x.adv[j], v.k[j]) * back;
            if (in >> j & 1) out[j * 32] = x.live >> j & 1 ? g : 0.0f;
        }
    });
}

template <Kind K>
int64_t tiles_of(int64_t T)
{
    const int64_t tile = 32 * (T < kFew ? kFewItems : many_items(K));
    return (T + tile - 1) / tile;
}

constexpr int64_t kMaxSequences = 1ll << 30;

zero_status check_packed(int64_t T, int64_t S)
{
    if (T < 0 || S < 0) return ZERO_ERR_INVALID_ARG;
    return T > kMaxRows || S > kMaxSequences ? ZERO_ERR_SIZE : ZERO_OK;
}

zero_status check_offsets(const void* offsets, int32_t bytes)
{
    if (bytes != 4 && bytes != 8) return ZERO_ERR_INVALID_ARG;
    return check_ptr(offsets, (unsigned)bytes);
}

unsigned blocks_of(int64_t warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); }

template <Kind K, int ITEMS>
zero_status forward_in(const LossArgs& a, int64_t results, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;                     // (no tokens: no parts)
    if (a.tiles) e = launch(k_loss_parts<K, ITEMS>, dim3(blocks_of(a.tiles)), kThreads, 0, st, a);
    if (e != cudaSuccess) return status_of(e);
    // a warp takes a result unless it would have to fetch many parts (one sequence of 10^6
    // tokens: 41 us by a warp, 17 by a block).  The host knows only their mean: where one of 502
    // sequences has all but 2000 of 2^20 tokens, a warp joins its 8192 parts, and a call of the policy
    // with its gradient takes 106 us (even lengths 17), of preferences 37 (11).
    return status_of(a.tiles >= kWideTiles * results
                         ? launch(k_loss_join<K, ITEMS, true>, dim3((unsigned)results),
                                  kWideThreads, 0, st, a)
                         : launch(k_loss_join<K, ITEMS, false>, dim3(blocks_of(results)), kThreads,
                                  0, st, a));
}

template <Kind K>
zero_status forward(LossArgs& a, int64_t results, cudaStream_t st)
{
    a.tiles = (int32_t)tiles_of<K>(a.T);
    // (nor without tokens more: 2^30 results would take one block's warps ten seconds and more)
    if (a.tiles <= kAloneTiles && a.S <= kAloneSequences) {
        const int warps = (int)std::min<int64_t>(32, std::max<int64_t>(a.tiles, results));
        return status_of(launch(k_loss_alone<K>, dim3(1), 32 * warps, 0, st, a));
    }
    return a.T < kFew ? forward_in<K, kFewItems>(a, results, st)
                      : forward_in<K, many_items(K)>(a, results, st);
}

template <Kind K>
zero_status backward(LossArgs& a, cudaStream_t st)
{
    a.tiles = (int32_t)tiles_of<K>(a.T);
    return status_of(launch(a.T < kFew ? k_loss_grad<K, kFewItems> : k_loss_grad<K, many_items(K)>,
                            dim3(blocks_of(a.tiles)), kThreads, 0, st, a));
}

template <Kind K>
int64_t scratch_for(int64_t T, int64_t S)
{
    if (check_packed(T, S) != ZERO_OK) return -1;
    // (the longest of few tokens have more tiles than somewhat more tokens)
    const int64_t tiles = std::max(tiles_of<K>(T), tiles_of<K>(std::min(T, kFew - 1)));
    return up((int64_t)sizeof(Part) * (tiles + S), 256);
}

// The bounds of the policy's ratio, and their logarithms as the kernels compare with them.
zero_status policy_bounds(LossArgs& a, double clip_low, double clip_high, double kl_coef)
{
    if (!(clip_low >= 0.0) || clip_low > 1.0) return ZERO_ERR_INVALID_ARG;
    if (!(clip_high >= 0.0) || clip_high > 3.0e38) return ZERO_ERR_INVALID_ARG;
    if (!(kl_coef >= 0.0) || kl_coef > 3.0e38) return ZERO_ERR_INVALID_ARG;
    a.bound_lo = (float)(1.0 - clip_low);
    a.bound_hi = (float)(1.0 + clip_high);
    const double lo = log1p(-clip_low), hi = log1p(clip_high);       // lo: -Inf for 1
    a.edge_lo = (float)lo;
    a.edge_hi = (float)hi;
    a.rest_lo = clip_low < 1.0 ? (float)(lo - (double)a.edge_lo) : 0.0f;
    a.rest_hi = (float)(hi - (double)a.edge_hi);
    a.kl_coef = (float)kl_coef;
    return ZERO_OK;
}

}  // namespace

extern "C" int64_t zero_preference_scratch_bytes(int64_t T, int64_t P)
{
    return P < 0 || P > kMaxSequences / 2 ? -1 : scratch_for<kPreference>(T, 2 * P);
}

extern "C" zero_status zero_preference(const float* nll, const float* ref_nll, const void* targets,
                                       int32_t target_bytes, int64_t T, const void* offsets,
                                       int32_t offset_bytes, int64_t P, int32_t kind, double beta,
                                       double smoothing, double margin, int32_t average,
                                       float* loss, float* slope, float* ratios, int32_t* counts,
                                       void* scratch, int64_t scratch_bytes, int32_t* dev_status,
                                       void* stream)
{
    if (P < 0) return ZERO_ERR_INVALID_ARG;
    if (P > kMaxSequences / 2) return ZERO_ERR_SIZE;
    LM_CHECK(check_packed(T, 2 * P));
    if (target_bytes != 4 && target_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (offset_bytes != 4 && offset_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (kind < ZERO_PREF_SIGMOID || kind > ZERO_PREF_IPO) return ZERO_ERR_INVALID_ARG;
    if (!(beta > 0.0) || beta > 3.0e38) return ZERO_ERR_INVALID_ARG;
    if (!(smoothing >= 0.0) || smoothing >= 0.5) return ZERO_ERR_INVALID_ARG;
    if (kind != ZERO_PREF_SIGMOID && smoothing != 0.0) return ZERO_ERR_INVALID_ARG;
    if (!(fabs(margin) <= 3.0e38)) return ZERO_ERR_INVALID_ARG;
    if (average != 0 && average != 1) return ZERO_ERR_INVALID_ARG;
    LM_CHECK(check_status(dev_status));
    if (P == 0) return ZERO_OK;
    if (T > 0) {
        LM_CHECK(check_ptr(nll, 4));
        if (ref_nll) LM_CHECK(check_ptr(ref_nll, 4));
        LM_CHECK(check_tokens(targets, target_bytes));
    }
    LM_CHECK(check_offsets(offsets, offset_bytes));
    LM_CHECK(check_ptr(loss, 4));
    LM_CHECK(check_ptr(slope, 4));
    LM_CHECK(check_ptr(ratios, 4));
    LM_CHECK(check_ptr(counts, 4));
    LM_CHECK(check_ptr(scratch));
    const int64_t need = zero_preference_scratch_bytes(T, P);
    if (scratch_bytes < need) return ZERO_ERR_SIZE;
    Spans sp;
    sp.add(nll, 4 * T, false);
    sp.add(ref_nll, 4 * T, false);
    sp.add(targets, target_bytes * T, false);
    sp.add(offsets, offset_bytes * (2 * P + 1), false);
    sp.add(loss, 4 * P, true);
    sp.add(slope, 4 * P, true);
    sp.add(ratios, 8 * P, true);
    sp.add(counts, 8 * P, true);
    sp.add(scratch, need, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    LossArgs a{};
    a.nll = nll;
    a.ref = ref_nll;
    a.targets = targets;
    a.offsets = offsets;
    a.parts = static_cast<Part*>(scratch);
    a.status = dev_status;
    a.loss = loss;
    a.slope = slope;
    a.ratios = ratios;
    a.counts = counts;
    a.T = (int32_t)T;
    a.S = (int32_t)(2 * P);
    a.target_bytes = target_bytes;
    a.offset_bytes = offset_bytes;
    a.average = average;
    a.kind = kind;
    a.beta = beta;
    a.margin = kind == ZERO_PREF_IPO ? margin + 0.5 / beta : margin;
    a.smoothing = (float)smoothing;
    return forward<kPreference>(a, P, static_cast<cudaStream_t>(stream));
}

extern "C" zero_status zero_preference_grad(const void* targets, int32_t target_bytes, int64_t T,
                                            const void* offsets, int32_t offset_bytes, int64_t P,
                                            int32_t average, const float* slope,
                                            const int32_t* counts, const float* dloss,
                                            float* dnll, void* stream)
{
    if (P < 0) return ZERO_ERR_INVALID_ARG;
    if (P > kMaxSequences / 2) return ZERO_ERR_SIZE;
    LM_CHECK(check_packed(T, 2 * P));
    if (target_bytes != 4 && target_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (offset_bytes != 4 && offset_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (average != 0 && average != 1) return ZERO_ERR_INVALID_ARG;
    if (P == 0 || T == 0) return ZERO_OK;
    LM_CHECK(check_tokens(targets, target_bytes));
    LM_CHECK(check_offsets(offsets, offset_bytes));
    LM_CHECK(check_ptr(slope, 4));
    LM_CHECK(check_ptr(counts, 4));
    LM_CHECK(check_ptr(dloss, 4));
    LM_CHECK(check_ptr(dnll, 4));
    Spans sp;
    sp.add(targets, target_bytes * T, false);
    sp.add(offsets, offset_bytes * (2 * P + 1), false);
    sp.add(slope, 4 * P, false);
    sp.add(counts, 8 * P, false);
    sp.add(dloss, 4 * P, false);
    sp.add(dnll, 4 * T, true);
    LM_CHECK(sp.check());

    LossArgs a{};
    a.targets = targets;
    a.offsets = offsets;
    a.slope_in = slope;
    a.counts_in = counts;
    a.dloss = dloss;
    a.dnll = dnll;
    a.T = (int32_t)T;
    a.S = (int32_t)(2 * P);
    a.target_bytes = target_bytes;
    a.offset_bytes = offset_bytes;
    a.average = average;
    return backward<kPreference>(a, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t zero_policy_scratch_bytes(int64_t T, int64_t S) { return scratch_for<kPolicy>(T, S); }

// What the two calls of the policy loss have in common; nothing of a call that has
// nothing to write is looked at but its numbers.
static zero_status policy_args(LossArgs& a, Spans& sp, bool grad, const float* nll, const float* old_nll,
                               const float* ref_nll, const float* advantages, int32_t per_token,
                               const void* targets, int32_t target_bytes, int64_t T,
                               const void* offsets, int32_t offset_bytes, int64_t S,
                               double clip_low, double clip_high, double kl_coef, int32_t average,
                               int32_t* dev_status)
{
    LM_CHECK(check_packed(T, S));
    if (target_bytes != 4 && target_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (offset_bytes != 4 && offset_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (per_token != 0 && per_token != 1) return ZERO_ERR_INVALID_ARG;
    if (average != 0 && average != 1) return ZERO_ERR_INVALID_ARG;
    LM_CHECK(policy_bounds(a, clip_low, clip_high, kl_coef));
    LM_CHECK(check_status(dev_status));
    if (S == 0 || (grad && T == 0)) return ZERO_OK;
    if (T > 0) {
        LM_CHECK(check_ptr(nll, 4));
        if (old_nll) LM_CHECK(check_ptr(old_nll, 4));
        if (!ref_nll && kl_coef != 0.0) return ZERO_ERR_NULL;
        if (ref_nll) LM_CHECK(check_ptr(ref_nll, 4));
        LM_CHECK(check_tokens(targets, target_bytes));
        LM_CHECK(check_ptr(advantages, 4));
    }
    LM_CHECK(check_offsets(offsets, offset_bytes));
    sp.add(nll, 4 * T, false);
    sp.add(old_nll, 4 * T, false);
    sp.add(ref_nll, 4 * T, false);
    sp.add(advantages, 4 * (per_token ? T : S), false);
    sp.add(targets, target_bytes * T, false);
    sp.add(offsets, offset_bytes * (S + 1), false);
    sp.add(dev_status, 4, true);
    a.nll = nll;
    a.old = old_nll;
    a.ref = ref_nll;
    a.adv = advantages;
    a.targets = targets;
    a.offsets = offsets;
    a.status = dev_status;
    a.T = (int32_t)T;
    a.S = (int32_t)S;
    a.target_bytes = target_bytes;
    a.offset_bytes = offset_bytes;
    a.per_token = per_token;
    a.average = average;
    return ZERO_OK;
}

extern "C" zero_status zero_policy(const float* nll, const float* old_nll, const float* ref_nll,
                                   const float* advantages, int32_t per_token,
                                   const void* targets, int32_t target_bytes, int64_t T,
                                   const void* offsets, int32_t offset_bytes, int64_t S,
                                   double clip_low, double clip_high, double kl_coef,
                                   int32_t average, float* loss, float* kl, int32_t* clipped,
                                   int32_t* counts, void* scratch, int64_t scratch_bytes,
                                   int32_t* dev_status, void* stream)
{
    LossArgs a{};
    Spans sp;
    LM_CHECK(policy_args(a, sp, false, nll, old_nll, ref_nll, advantages, per_token, targets,
                         target_bytes, T, offsets, offset_bytes, S, clip_low, clip_high, kl_coef,
                         average, dev_status));
    if (S == 0) return ZERO_OK;
    LM_CHECK(check_ptr(loss, 4));
    LM_CHECK(check_ptr(kl, 4));
    LM_CHECK(check_ptr(clipped, 4));
    LM_CHECK(check_ptr(counts, 4));
    LM_CHECK(check_ptr(scratch));
    const int64_t need = zero_policy_scratch_bytes(T, S);
    if (scratch_bytes < need) return ZERO_ERR_SIZE;
    sp.add(loss, 4 * S, true);
    sp.add(kl, 4 * S, true);
    sp.add(clipped, 4 * S, true);
    sp.add(counts, 4 * S, true);
    sp.add(scratch, need, true);
    LM_CHECK(sp.check());
    a.parts = static_cast<Part*>(scratch);
    a.loss = loss;
    a.kl = kl;
    a.clipped = clipped;
    a.counts = counts;
    return forward<kPolicy>(a, S, static_cast<cudaStream_t>(stream));
}

extern "C" zero_status zero_policy_grad(const float* nll, const float* old_nll,
                                        const float* ref_nll, const float* advantages,
                                        int32_t per_token, const void* targets,
                                        int32_t target_bytes, int64_t T, const void* offsets,
                                        int32_t offset_bytes, int64_t S, double clip_low,
                                        double clip_high, double kl_coef, int32_t average,
                                        const int32_t* counts, const float* dloss, float* dnll,
                                        void* stream)
{
    LossArgs a{};
    Spans sp;
    LM_CHECK(policy_args(a, sp, true, nll, old_nll, ref_nll, advantages, per_token, targets,
                         target_bytes, T, offsets, offset_bytes, S, clip_low, clip_high, kl_coef,
                         average, nullptr));
    if (S == 0 || T == 0) return ZERO_OK;
    LM_CHECK(check_ptr(counts, 4));
    LM_CHECK(check_ptr(dloss, 4));
    LM_CHECK(check_ptr(dnll, 4));
    sp.add(counts, 4 * S, false);
    sp.add(dloss, 4 * S, false);
    sp.add(dnll, 4 * T, true);
    LM_CHECK(sp.check());
    a.counts_in = counts;
    a.dloss = dloss;
    a.dnll = dnll;
    return backward<kPolicy>(a, static_cast<cudaStream_t>(stream));
}
