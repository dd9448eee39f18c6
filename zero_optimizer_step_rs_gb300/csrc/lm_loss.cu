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
// the other, and no slot needs clearing.  The sequence's slots are then joined in 64
// bits, in order of the lanes: no atomics, the same bits in every call.
#include "lm_common.cuh"

#include <math.h>

namespace {

using namespace lm;

// Tokens of a lane: a warp with 8 takes 1500 instructions one after the other, which is 7 us
// of a call of few tokens; one with 2 does less work per instruction (the search for its
// sequences, the sums' halvings), which costs where there are many.
constexpr int kFewItems = 2, kManyItems = 8;
constexpr int64_t kFew = 1 << 16;                    // tokens from which on a lane takes 8
constexpr int kThreads = 128;
constexpr int kAloneThreads = 1024;                  // of the one block that does it all
constexpr int64_t kAloneResults = 64;
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
    int64_t T, S, tiles;
    int32_t target_bytes, offset_bytes, per_token, average, kind;
    float kl_coef;
    float bound_lo, bound_hi;                        // 1 - clip_low, 1 + clip_high
    float edge_lo, edge_hi;                          // their logarithms, rounded
    float rest_lo, rest_hi;                          // and what that lost
    double beta, margin;
    float smoothing;
};

__device__ __forceinline__ int64_t raw_offset(const LossArgs& a, int64_t i)
{
    return token_at(a.offsets, a.offset_bytes, i);
}

// The number of offsets (of S + 1) that are at most t, by a search in 32 parts.
__device__ __forceinline__ int64_t offsets_up_to(const LossArgs& a, int64_t t, int lane)
{
    int64_t lo = 0, hi = a.S + 1;
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) >> 5;
        const int64_t i = lo + lane * step;
        const bool below = i < hi && raw_offset(a, i) <= t;
        const int n = __popc(__ballot_sync(kAll, below));
        if (n == 0) break;
        hi = min(hi, lo + n * step);
        lo += (n - 1) * step + 1;
    }
    return lo;
}

// exp(d) - d - 1 and exp(d) - 1.  Near 0 these cancel, so there they are the
// exponential's series from its third term on; at |d| <= 1 the first term left out, d^13 / 13!,
// is under 2^-30 of the sum.
struct Drift {
    float k, e;
};
__device__ __forceinline__ Drift drift(float d)
{
    if (fabsf(d) <= 1.0f) {
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
        const float k = p * d * d;
        return {k, d + k};
    }
    const float e = expf(d) - 1.0f;
    return {e - d, e};
}

// Where old - nll, as exact numbers, lies beside the bounds' logarithms: bit 0 above the
// upper, bit 1 below the lower one.  Rounding keeps the order, so only a difference that
// rounds to the same fp32 value as the logarithm needs what both roundings lost: the
// difference's by Knuth's two-sum.  (In 64 bits, and be it for those few tokens alone, the
// comparisons took 6 of 12 us of a call: the compiler makes them for all.)
__device__ __forceinline__ unsigned beyond(const LossArgs& a, float old, float nll, float change)
{
    const float back = __fsub_rn(change, old);
    const float lost = __fsub_rn(__fsub_rn(old, __fsub_rn(change, back)), __fadd_rn(nll, back));
    const bool high = change > a.edge_hi || (change == a.edge_hi && lost > a.rest_hi);
    const bool low = change < a.edge_lo || (change == a.edge_lo && lost < a.rest_lo);
    return (unsigned)high | (unsigned)low << 1;
}

// A lane's tokens of a tile: t = base + 32 j + lane.
template <int ITEMS>
struct Tokens {
    float nll[ITEMS], old[ITEMS], ref[ITEMS], adv[ITEMS];
    unsigned live;                                   // bit j: token j counts
};

template <Kind K, bool GRAD, int ITEMS>
__device__ __forceinline__ void load_tokens(const LossArgs& a, int64_t base, int lane,
                                            Tokens<ITEMS>& x)
{
    int64_t id[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const int64_t t = base + j * 32 + lane;
        const bool in = t < a.T;
        id[j] = in ? token_at(a.targets, a.target_bytes, t) : -1;
        if (K == kPolicy || !GRAD) {
            x.nll[j] = in ? a.nll[t] : 0.0f;
            x.ref[j] = in && a.ref ? a.ref[t] : 0.0f;
        }
        if (K == kPolicy) {
            x.old[j] = in && a.old ? a.old[t] : x.nll[j];
            x.adv[j] = in && a.per_token ? a.adv[t] : 0.0f;
        }
    }
    x.live = 0;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) x.live |= (id[j] >= 0 ? 1u : 0u) << j;
}

// Calls f(s, lo, hi, of(s)) for every sequence from s0 on that the tile at base meets, with the
// part [base + lo, base + hi) of it that lies inside.  The bounds and of(s) of 32 sequences are
// fetched at once, one a lane.
template <int ITEMS, typename Of, typename F>
__device__ __forceinline__ void for_sequences(const LossArgs& a, int64_t base, int64_t s0,
                                              int lane, Of&& of, F&& f)
{
    const int64_t n = min((int64_t)kTile<ITEMS>, a.T - base);
    for (int64_t s = max(s0, (int64_t)0); s < a.S; s += 31) {
        const int lo = (int)min(max(raw_offset(a, min(s + lane, a.S)) - base, (int64_t)0), n);
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
        if (__shfl_sync(kAll, lo, 31) >= n) return;
    }
}

// The terms of a tile, summed for each sequence that it meets.
template <Kind K, int ITEMS>
__device__ __forceinline__ void tile_parts(const LossArgs& a, int64_t tile, int lane)
{
    const int64_t base = tile * kTile<ITEMS>;
    Tokens<ITEMS> x;
    load_tokens<K, false, ITEMS>(a, base, lane, x);
    const int64_t s0 = offsets_up_to(a, base, lane) - 1;     // while the tokens are on their way
    float v[ITEMS], kk[ITEMS];
    unsigned side = 0;                               // beyond(), two bits a token
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        if (K == kPreference) {
            v[j] = x.ref[j] - x.nll[j];
        } else {
            const float change = x.old[j] - x.nll[j];
            v[j] = expf(change);
            kk[j] = a.ref ? drift(x.nll[j] - x.ref[j]).k : 0.0f;
            side |= beyond(a, x.old[j], x.nll[j], change) << 2 * j;
        }
    }
    const auto about = [&](int64_t s) {
        return make_float2(K == kPolicy && !a.per_token ? a.adv[s] : 0.0f, 0.0f);
    };
    for_sequences<ITEMS>(a, base, s0, lane, about, [&](int64_t s, int lo, int hi, float2 of_s) {
        const float shared = of_s.x;
        float sum = 0.0f, ksum = 0.0f;
        int both = 0;                                // clipped tokens above bit 16, all below
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const int t = j * 32 + lane;
            if (t < lo || t >= hi || !(x.live >> j & 1)) continue;
            ++both;
            if (K == kPreference) {
                sum += v[j];
            } else {
                const float A = a.per_token ? x.adv[j] : shared;
                const bool over = A > 0.0f ? side >> 2 * j & 1 : A < 0.0f && (side >> 2 * j & 2);
                const float r = over ? (A > 0.0f ? a.bound_hi : a.bound_lo) : v[j];
                float term = A == 0.0f ? 0.0f : -(r * A);
                if (a.kl_coef != 0.0f) term = fmaf(a.kl_coef, kk[j], term);
                sum += term;
                ksum += kk[j];
                both += over ? 1 << 16 : 0;
            }
        }
        sum = warp_sum(sum);
        if (K == kPolicy) ksum = warp_sum(ksum);
        both = __reduce_add_sync(kAll, both);
        if (lane == 0) a.parts[tile + s] = Part{sum, ksum, both & 0xFFFF, both >> 16};
    });
}

struct Sums {
    double a, k;
    int32_t count, clipped;
};

// x / n for a count n.  A 64-bit division takes 1 us of a call that takes 2; the quotient of
// the high parts and one of what it leaves are as good as 48 bits.
__device__ __forceinline__ double over(double x, int32_t n)
{
    if (n <= 1) return x;
    const float d = (float)n, hi = (float)x;
    if (n >= 1 << 24 || !(fabsf(hi) <= 3.0e38f)) return x / (double)n;
    const float q = hi / d, lo = (float)(x - (double)hi);
    return (double)q + (double)((fmaf(-q, d, hi) + lo) / d);
}

// The parts of sequence s = [from, to) over a warp's lanes, joined in every lane.
template <Kind K, int ITEMS>
__device__ __forceinline__ Sums join_parts(const LossArgs& a, int64_t s, int64_t from, int64_t to,
                                           int lane)
{
    Sums r{0.0, 0.0, 0, 0};
    if (from < 0 || to < from || to > a.T) {
        if (lane == 0 && a.status) atomicOr(a.status, ZERO_DEV_BAD_OFFSETS);
        return r;
    }
    if (from == to) return r;
    const int64_t first = from / kTile<ITEMS>, last = (to - 1) / kTile<ITEMS>;
#pragma unroll 4
    for (int64_t i = first + lane; i <= last; i += 32) {
        const Part p = a.parts[i + s];
        r.a += p.a;
        if (K == kPolicy) r.k += p.k;
        r.count += p.count;
        r.clipped += p.clipped;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.a += __shfl_xor_sync(kAll, r.a, o);
        if (K == kPolicy) r.k += __shfl_xor_sync(kAll, r.k, o);
    }
    r.count = __reduce_add_sync(kAll, r.count);
    if (K == kPolicy) r.clipped = __reduce_add_sync(kAll, r.clipped);
    return r;
}

__device__ __forceinline__ float softplus(float x)
{
    return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// Pair p's loss from its two sequences, or sequence p's.  `ready` is called once between the
// offsets' loads and the parts'.
template <Kind K, int ITEMS, typename Ready>
__device__ __forceinline__ void finish(const LossArgs& a, int64_t p, int lane, Ready&& ready)
{
    if (K == kPolicy) {
        const int64_t from = raw_offset(a, p), to = raw_offset(a, p + 1);
        ready();
        Sums r = join_parts<K, ITEMS>(a, p, from, to, lane);
        if (lane) return;
        if (a.average) {
            r.a = over(r.a, r.count);
            r.k = over(r.k, r.count);
        }
        a.loss[p] = (float)r.a;
        a.kl[p] = (float)r.k;
        a.counts[p] = r.count;
        a.clipped[p] = r.clipped;
        return;
    }
    const int64_t from = raw_offset(a, 2 * p), mid = raw_offset(a, 2 * p + 1),
                  to = raw_offset(a, 2 * p + 2);
    ready();
    Sums c = join_parts<K, ITEMS>(a, 2 * p, from, mid, lane);
    Sums r = join_parts<K, ITEMS>(a, 2 * p + 1, mid, to, lane);
    if (lane) return;
    if (a.average) {
        c.a = over(c.a, c.count);
        r.a = over(r.a, r.count);
    }
    a.ratios[2 * p] = (float)c.a;
    a.ratios[2 * p + 1] = (float)r.a;
    a.counts[2 * p] = c.count;
    a.counts[2 * p + 1] = r.count;
    const double d = c.a - r.a;
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
    pdl_let_in();
    const int64_t tile = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile < a.tiles) tile_parts<K, ITEMS>(a, tile, threadIdx.x & 31);
}

// Its blocks come in beside those of k_loss_parts, which have waited for what was before them:
// the offsets may be read before the parts are there.
template <Kind K, int ITEMS>
__global__ void __launch_bounds__(kThreads) k_loss_join(const __grid_constant__ LossArgs a)
{
    const int64_t p = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (p < (K == kPreference ? a.S / 2 : a.S))
        finish<K, ITEMS>(a, p, threadIdx.x & 31, [] { pdl_enter(); });
    else
        pdl_enter();
}

// Few tokens: one block does both, in one launch.
template <Kind K>
__global__ void __launch_bounds__(kAloneThreads) k_loss_alone(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < a.tiles) tile_parts<K, kFewItems>(a, warp, lane);
    __syncthreads();
    const int64_t results = K == kPreference ? a.S / 2 : a.S;
    for (int64_t p = warp; p < results; p += kAloneThreads / 32)
        finish<K, kFewItems>(a, p, lane, [] {});
}

// The gradient of each token's loss.
template <Kind K, int ITEMS>
__global__ void __launch_bounds__(kThreads) k_loss_grad(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t tile = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile >= a.tiles) return;
    const int64_t base = tile * kTile<ITEMS>;
    Tokens<ITEMS> x;
    load_tokens<K, true, ITEMS>(a, base, lane, x);
    const int64_t s0 = offsets_up_to(a, base, lane) - 1;
    float v[ITEMS], kk[ITEMS];
    unsigned side = 0;
    if (K == kPolicy) {
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const float change = x.old[j] - x.nll[j];
            v[j] = expf(change);
            kk[j] = a.kl_coef != 0.0f ? a.kl_coef * drift(x.nll[j] - x.ref[j]).e : 0.0f;
            side |= beyond(a, x.old[j], x.nll[j], change) << 2 * j;
        }
    }
    // the advantage, where it is the sequence's, and the upstream gradient of its tokens
    const auto about = [&](int64_t s) {
        float back = a.dloss[K == kPolicy ? s : s >> 1];
        if (K == kPreference) {
            back *= a.slope_in[s >> 1];
            if (!(s & 1)) back = -back;
        }
        if (a.average) back /= (float)max(a.counts_in[s], 1);
        return make_float2(K == kPolicy && !a.per_token ? a.adv[s] : 0.0f, back);
    };
    for_sequences<ITEMS>(a, base, s0, lane, about, [&](int64_t s, int lo, int hi, float2 of_s) {
        const float shared = of_s.x, back = of_s.y;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const int t = j * 32 + lane;
            if (t < lo || t >= hi) continue;
            float g = 0.0f;
            if (x.live >> j & 1) {
                if (K == kPreference) {
                    g = back;
                } else {
                    const float A = a.per_token ? x.adv[j] : shared;
                    const bool over = A > 0.0f ? side >> 2 * j & 1 : A < 0.0f && (side >> 2 * j & 2);
                    g = fmaf(over || A == 0.0f ? 0.0f : v[j], A, kk[j]) * back;
                }
            }
            a.dnll[base + t] = g;
        }
    });
}

int items_of(int64_t T) { return T < kFew ? kFewItems : kManyItems; }

int64_t tiles_of(int64_t T) { return (T + 32 * items_of(T) - 1) / (32 * items_of(T)); }

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
    cudaError_t e = launch(k_loss_parts<K, ITEMS>, dim3(blocks_of(a.tiles)), kThreads, 0, st, a);
    if (e == cudaSuccess)
        e = launch(k_loss_join<K, ITEMS>, dim3(blocks_of(results)), kThreads, 0, st, a);
    return status_of(e);
}

template <Kind K>
zero_status forward(LossArgs& a, int64_t results, cudaStream_t st)
{
    a.tiles = tiles_of(a.T);
    // (without tokens there is no first launch that waits for the offsets)
    if (a.tiles == 0 || (a.tiles <= kAloneThreads / 32 && results <= kAloneResults))
        return status_of(launch(k_loss_alone<K>, dim3(1), kAloneThreads, 0, st, a));
    return items_of(a.T) == kFewItems ? forward_in<K, kFewItems>(a, results, st)
                                      : forward_in<K, kManyItems>(a, results, st);
}

template <Kind K>
zero_status backward(LossArgs& a, cudaStream_t st)
{
    a.tiles = tiles_of(a.T);
    return status_of(launch(items_of(a.T) == kFewItems ? k_loss_grad<K, kFewItems>
                                                       : k_loss_grad<K, kManyItems>,
                            dim3(blocks_of(a.tiles)), kThreads, 0, st, a));
}

int64_t scratch_for(int64_t T, int64_t S)
{
    if (check_packed(T, S) != ZERO_OK) return -1;
    // (the longest of few tokens have more tiles than somewhat more tokens)
    const int64_t tiles = std::max(tiles_of(T), tiles_of(std::min(T, kFew - 1)));
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
    return P < 0 || P > kMaxSequences / 2 ? -1 : scratch_for(T, 2 * P);
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
    a.T = T;
    a.S = 2 * P;
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
    a.T = T;
    a.S = 2 * P;
    a.target_bytes = target_bytes;
    a.offset_bytes = offset_bytes;
    a.average = average;
    return backward<kPreference>(a, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t zero_policy_scratch_bytes(int64_t T, int64_t S) { return scratch_for(T, S); }

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
    a.T = T;
    a.S = S;
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
