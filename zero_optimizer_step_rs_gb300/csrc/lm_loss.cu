// lm_loss.cu - losses of packed sequences from their tokens' losses, and the
// gradients of the tokens' losses: pairs of a chosen and a rejected sequence
// (zero_preference), and the clipped policy loss with a KL term (zero_policy).
// Declared in include/zero_step.h.
//
// Both are a sum per sequence of a term per token, and a gradient per token from a
// number per sequence.  The tokens are cut into tiles of 256, one warp's, whatever
// the sequences' lengths are.  A tile meets the sequences s0, s0 + 1, ...; going
// along the tokens either the tile or the sequence steps on, so that tile + s is a
// slot of its own for every pair that meets, the slots of a sequence lie one behind
// the other, and no slot needs clearing.  The sequence's slots are then joined in 64
// bits, in order of the lanes: no atomics, the same bits in every call.
#include "lm_common.cuh"

#include <math.h>

namespace {

using namespace lm;

constexpr int kItems = 8;                            // tokens of a lane
constexpr int kTile = 32 * kItems;                   // tokens of a warp
constexpr int kThreads = 256;
constexpr int kAloneThreads = 1024;                  // of the one block that does it all
constexpr unsigned kAll = 0xFFFFFFFFu;

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
    double log_lo, log_hi;                           // and not
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

// exp(d) - d - 1.  Near 0 the three cancel, so there it is the exponential's series
// from its third term on; at |d| <= 1 the first one left out, 2 d^11 / 13!, is under
// 2^-30 of the sum.
__device__ __forceinline__ float kl_estimate(float d)
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
        return p * d * d;
    }
    return expm1f(d) - d;
}

// Whether old - nll, as exact numbers, is above (below) the logarithm of a bound.
// Rounding keeps the order, so only a difference that rounds to the same fp32 value as the
// logarithm needs 64 bits.
__device__ __forceinline__ bool above(float change, float old, float nll, float edge, double log)
{
    if (change != edge) return change > edge;
    return (double)old - (double)nll > log;
}
__device__ __forceinline__ bool below(float change, float old, float nll, float edge, double log)
{
    if (change != edge) return change < edge;
    return (double)old - (double)nll < log;
}

// A lane's tokens of a tile: t = base + 32 j + lane.
struct Tokens {
    float nll[kItems], old[kItems], ref[kItems], adv[kItems];
    unsigned live;                                   // bit j: token j counts
};

template <Kind K, bool GRAD>
__device__ __forceinline__ void load_tokens(const LossArgs& a, int64_t base, int lane, Tokens& x)
{
    int64_t id[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
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
    for (int j = 0; j < kItems; ++j) x.live |= (id[j] >= 0 ? 1u : 0u) << j;
}

// Calls f(s, lo, hi) for every sequence that the tile [base, base + kTile) meets,
// with the part of it that lies inside.
template <typename F>
__device__ __forceinline__ void for_sequences(const LossArgs& a, int64_t base, int lane, F&& f)
{
    const int64_t end = min(base + kTile, a.T);
    int64_t s = max(offsets_up_to(a, base, lane) - 1, (int64_t)0);
    while (s < a.S) {
        // the next 32 bounds, one a lane
        const int64_t i = min(s + lane, a.S);
        const int64_t mine = raw_offset(a, i);
        const int64_t after = __shfl_down_sync(kAll, mine, 1);
        int n = (int)min((int64_t)31, a.S - s);
        for (int k = 0; k < n; ++k) {
            const int64_t from = __shfl_sync(kAll, mine, k), to = __shfl_sync(kAll, after, k);
            if (from >= end) return;
            const int64_t lo = max(from, base), hi = min(to, end);
            if (lo < hi) f(s + k, lo, hi);
        }
        s += n;
    }
}

// The terms of a tile, summed for each sequence that it meets.
template <Kind K>
__device__ __forceinline__ void tile_parts(const LossArgs& a, int64_t tile, int lane)
{
    const int64_t base = tile * kTile;
    Tokens x;
    load_tokens<K, false>(a, base, lane, x);
    float v[kItems], kk[kItems];
    unsigned high = 0, low = 0;                      // tokens beyond either bound
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        if (K == kPreference) {
            v[j] = x.ref[j] - x.nll[j];
        } else {
            const float change = x.old[j] - x.nll[j];
            v[j] = expf(change);
            kk[j] = a.ref ? kl_estimate(x.nll[j] - x.ref[j]) : 0.0f;
            high |= (unsigned)above(change, x.old[j], x.nll[j], a.edge_hi, a.log_hi) << j;
            low |= (unsigned)below(change, x.old[j], x.nll[j], a.edge_lo, a.log_lo) << j;
        }
    }
    for_sequences(a, base, lane, [&](int64_t s, int64_t lo, int64_t hi) {
        const float shared = K == kPolicy && !a.per_token ? a.adv[s] : 0.0f;
        float sum = 0.0f, ksum = 0.0f;
        int count = 0, clipped = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t t = base + j * 32 + lane;
            const bool in = t >= lo && t < hi && (x.live >> j & 1);
            if (!in) continue;
            ++count;
            if (K == kPreference) {
                sum += v[j];
            } else {
                const float A = a.per_token ? x.adv[j] : shared;
                const bool over = A > 0.0f ? high >> j & 1 : A < 0.0f && (low >> j & 1);
                const float r = over ? (A > 0.0f ? a.bound_hi : a.bound_lo) : v[j];
                float term = A == 0.0f ? 0.0f : -(r * A);
                if (a.kl_coef != 0.0f) term = fmaf(a.kl_coef, kk[j], term);
                sum += term;
                ksum += kk[j];
                clipped += over;
            }
        }
        sum = warp_sum(sum);
        if (K == kPolicy) ksum = warp_sum(ksum);
        const int both = __reduce_add_sync(kAll, count | clipped << 16);
        if (lane == 0) a.parts[tile + s] = Part{sum, ksum, both & 0xFFFF, both >> 16};
    });
}

struct Sums {
    double a, k;
    int32_t count, clipped;
};

// The parts of sequence s over a warp's lanes, joined in every lane.
template <Kind K>
__device__ __forceinline__ Sums join_parts(const LossArgs& a, int64_t s, int lane)
{
    Sums r{0.0, 0.0, 0, 0};
    const int64_t from = raw_offset(a, s), to = raw_offset(a, s + 1);
    if (from < 0 || to < from || to > a.T) {
        if (lane == 0 && a.status) atomicOr(a.status, ZERO_DEV_BAD_OFFSETS);
        return r;
    }
    if (from == to) return r;
    const int64_t first = from / kTile, last = (to - 1) / kTile;
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

// Pair p's loss from its two sequences, or sequence p's.
template <Kind K>
__device__ __forceinline__ void finish(const LossArgs& a, int64_t p, int lane)
{
    if (K == kPolicy) {
        Sums r = join_parts<K>(a, p, lane);
        if (lane) return;
        if (a.average && r.count > 1) {
            r.a /= (double)r.count;
            r.k /= (double)r.count;
        }
        a.loss[p] = (float)r.a;
        a.kl[p] = (float)r.k;
        a.counts[p] = r.count;
        a.clipped[p] = r.clipped;
        return;
    }
    Sums c = join_parts<K>(a, 2 * p, lane), r = join_parts<K>(a, 2 * p + 1, lane);
    if (lane) return;
    if (a.average) {
        if (c.count > 1) c.a /= (double)c.count;
        if (r.count > 1) r.a /= (double)r.count;
    }
    a.ratios[2 * p] = (float)c.a;
    a.ratios[2 * p + 1] = (float)r.a;
    a.counts[2 * p] = c.count;
    a.counts[2 * p + 1] = r.count;
    const double d = c.a - r.a;
    float loss, slope;
    if (a.kind == ZERO_PREF_IPO) {
        const double e = d - a.margin - 0.5 / a.beta;
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

template <Kind K>
__global__ void __launch_bounds__(kThreads) k_loss_parts(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int64_t tile = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile < a.tiles) tile_parts<K>(a, tile, threadIdx.x & 31);
}

template <Kind K>
__global__ void __launch_bounds__(kThreads) k_loss_join(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int64_t p = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (p < (K == kPreference ? a.S / 2 : a.S)) finish<K>(a, p, threadIdx.x & 31);
}

// The gradient of each token's loss.
template <Kind K>
__global__ void __launch_bounds__(kThreads) k_loss_grad(const __grid_constant__ LossArgs a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t tile = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (tile >= a.tiles) return;
    const int64_t base = tile * kTile;
    Tokens x;
    load_tokens<K, true>(a, base, lane, x);
    float v[kItems], kk[kItems];
    unsigned high = 0, low = 0;
    if (K == kPolicy) {
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const float change = x.old[j] - x.nll[j];
            v[j] = expf(change);
            kk[j] = a.ref && a.kl_coef != 0.0f ? a.kl_coef * expm1f(x.nll[j] - x.ref[j]) : 0.0f;
            high |= (unsigned)above(change, x.old[j], x.nll[j], a.edge_hi, a.log_hi) << j;
            low |= (unsigned)below(change, x.old[j], x.nll[j], a.edge_lo, a.log_lo) << j;
        }
    }
    for_sequences(a, base, lane, [&](int64_t s, int64_t lo, int64_t hi) {
        const float shared = K == kPolicy && !a.per_token ? a.adv[s] : 0.0f;
        float back = a.dloss[K == kPolicy ? s : s >> 1];
        if (K == kPreference) {
            back *= a.slope_in[s >> 1];
            if (!(s & 1)) back = -back;
        }
        if (a.average) back /= (float)max(a.counts_in[s], 1);
        if (lane == 0 && a.status && (raw_offset(a, s + 1) > a.T || raw_offset(a, s) < 0))
            atomicOr(a.status, ZERO_DEV_BAD_OFFSETS);
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t t = base + j * 32 + lane;
            if (t < lo || t >= hi) continue;
            float g = 0.0f;
            if (x.live >> j & 1) {
                if (K == kPreference) {
                    g = back;
                } else {
                    const float A = a.per_token ? x.adv[j] : shared;
                    const bool over = A > 0.0f ? high >> j & 1 : A < 0.0f && (low >> j & 1);
                    g = (fmaf(over || A == 0.0f ? 0.0f : v[j], A, kk[j])) * back;
                }
            }
            a.dnll[t] = g;
        }
    });
}

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }

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

template <Kind K>
zero_status forward(LossArgs& a, int64_t results, cudaStream_t st)
{
    a.tiles = tiles_of(a.T);
    cudaError_t e = cudaSuccess;
    if (a.tiles) e = launch(k_loss_parts<K>, dim3(blocks_of(a.tiles)), kThreads, 0, st, a);
    if (e == cudaSuccess) e = launch(k_loss_join<K>, dim3(blocks_of(results)), kThreads, 0, st, a);
    return status_of(e);
}

template <Kind K>
zero_status backward(LossArgs& a, cudaStream_t st)
{
    a.tiles = tiles_of(a.T);
    return status_of(launch(k_loss_grad<K>, dim3(blocks_of(a.tiles)), kThreads, 0, st, a));
}

int64_t scratch_for(int64_t T, int64_t S)
{
    if (check_packed(T, S) != ZERO_OK) return -1;
    return up((int64_t)sizeof(Part) * (tiles_of(T) + S), 256);
}

// The bounds of the policy's ratio, and their logarithms as the kernels compare with them.
zero_status policy_bounds(LossArgs& a, double clip_low, double clip_high, double kl_coef)
{
    if (!(clip_low >= 0.0) || clip_low > 1.0) return ZERO_ERR_INVALID_ARG;
    if (!(clip_high >= 0.0) || clip_high > 3.0e38) return ZERO_ERR_INVALID_ARG;
    if (!(kl_coef >= 0.0) || kl_coef > 3.0e38) return ZERO_ERR_INVALID_ARG;
    a.bound_lo = (float)(1.0 - clip_low);
    a.bound_hi = (float)(1.0 + clip_high);
    a.log_lo = log1p(-clip_low);                         // -Inf for 1
    a.log_hi = log1p(clip_high);
    a.edge_lo = (float)a.log_lo;
    a.edge_hi = (float)a.log_hi;
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
    a.margin = margin;
    a.smoothing = (float)smoothing;
    return forward<kPreference>(a, P, static_cast<cudaStream_t>(stream));
}

extern "C" zero_status zero_preference_grad(const void* targets, int32_t target_bytes, int64_t T,
                                            const void* offsets, int32_t offset_bytes, int64_t P,
                                            int32_t average, const float* slope,
                                            const int32_t* counts, const float* dloss,
                                            float* dnll, int32_t* dev_status, void* stream)
{
    if (P < 0) return ZERO_ERR_INVALID_ARG;
    if (P > kMaxSequences / 2) return ZERO_ERR_SIZE;
    LM_CHECK(check_packed(T, 2 * P));
    if (target_bytes != 4 && target_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (offset_bytes != 4 && offset_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (average != 0 && average != 1) return ZERO_ERR_INVALID_ARG;
    LM_CHECK(check_status(dev_status));
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
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    LossArgs a{};
    a.targets = targets;
    a.offsets = offsets;
    a.status = dev_status;
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
                                        int32_t* dev_status, void* stream)
{
    LossArgs a{};
    Spans sp;
    LM_CHECK(policy_args(a, sp, true, nll, old_nll, ref_nll, advantages, per_token, targets,
                         target_bytes, T, offsets, offset_bytes, S, clip_low, clip_high, kl_coef,
                         average, dev_status));
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
