// lm_embed.cu - embedding lookup with scaling, and its gradient by sorted
// tokens (declared in include/zero_step.h).
//
//   out[t, :]  = bf16(scale * table[tok_t, :])            tok_t < 0: a row of zeros
//   grad[v, :] = bf16([grad[v, :] +] scale * sum_{t : tok_t = v} dy[t, :])
//
// with the sum in fp32.  Both are bound by HBM traffic: the lookup reads each
// row met (from L2 where a token repeats) and writes 2*T*D bytes; the
// gradient reads 2*T*D bytes and writes the table's 2*V*D (or, when it adds to
// a gradient that is there, reads and writes the rows met only).
//
// Measured, one GB300: the lookup of 65536 x 2048 from 128256 rows 54.7 us (6.4 TB/s
// of the bytes above; the copy rate is 6.77); the gradient of 1000 x 2048 into
// 128256 rows 75.7 us (7.0 TB/s, mostly zeros written), of 32768 x 2048 added to a
// tied table 72 us for 230 MB (34 us at the copy rate): 18 us of that are the sort,
// in which 8 SMs wait on latencies one after another, 37 the sums (bound by the
// instructions around each row's 512 bytes a warp, and by latency), 10 the join.
//
// The gradient's sums have one fixed order, so a step can be repeated bit for
// bit.  More than 1024 tokens are sorted by (id, position); a row's terms are
// added in that order, and a row with more terms than a chunk has places is the
// sum of its chunks' sums, in pieces that depend on the sizes and the tokens
// alone.  Up to 1024 tokens are not sorted: a block looks for its id's places and
// adds them in order.  No atomics touch a sum.
#include "lm_common.cuh"

namespace {

using namespace lm;

// ================================================================ lookup ==

struct LookupArgs {
    const uint16_t* table;
    const void* tokens;
    uint16_t* out;
    int64_t T, V, out_ld;
    int32_t D, token_bytes, lanes_log2;
    float scale;
    int32_t* status;
};

constexpr int kLookupThreads = 256;
constexpr int kLookupVecs = 8;       // 16-byte vectors a thread holds at once

// A group of 2^lanes_log2 threads (a warp, or less for narrow tables) takes a
// row: all of a 2048-wide row's loads are issued before the first store.
__global__ void __launch_bounds__(kLookupThreads) k_lookup(const __grid_constant__ LookupArgs a)
{
    pdl_enter();
    const int lanes = 1 << a.lanes_log2;
    const int64_t t =
        ((int64_t)blockIdx.x * kLookupThreads + threadIdx.x) >> a.lanes_log2;
    if (t >= a.T) return;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t v = token_at(a.tokens, a.token_bytes, t);
    if (v >= a.V && lane == 0 && a.status) atomicOr(a.status, ZERO_DEV_BAD_TOKEN);
    const bool row = v >= 0 && v < a.V;
    const uint16_t* src = a.table + (row ? v : 0) * (int64_t)a.D;
    uint16_t* dst = a.out + t * a.out_ld;
    const int nv = a.D >> 3;
    for (int base = lane; base < nv; base += lanes * kLookupVecs) {
        uint4 x[kLookupVecs];
#pragma unroll
        for (int k = 0; k < kLookupVecs; ++k) {
            const int c = base + k * lanes;
            x[k] = row && c < nv ? __ldg(reinterpret_cast<const uint4*>(src) + c)
                                 : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kLookupVecs; ++k) {
            const int c = base + k * lanes;
            if (c >= nv) break;
            if (row) {
                float f[8];
                bf_unpack8(x[k], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) f[q] *= a.scale;
                x[k] = bf_pack8(f);
            }
            st16_stream(dst + c * 8, x[k]);
        }
    }
}

// ================================================================== sort ==
// A stable least-significant-digit radix sort of (token, position) by ONE
// cluster of up to 8 blocks: a block owns a contiguous part of the list, and the
// cluster barrier orders the passes, so the whole sort is one launch.  Up to
// 32768 tokens a block's part is one round, and the blocks read each other's
// digit counts and pass items on in shared memory; above, through global memory
// (L2).  Ids that take part in nothing (negative, or past the table) get the key
// V and end up last.
//
// The rest of the grid, where there is one, fills the table's gradient with
// zeros meanwhile; the rows that are met are written by the next launch.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 4;                               // per thread and round
constexpr int kSortRound = kSortThreads * kSortItems;       // items of a block per round
constexpr int kMaxCluster = 8;
constexpr int kMaxBins = 512;
constexpr int kSortBins = kSortWarps * kMaxBins * 4;        // bytes: a warp's place in each digit
constexpr int kSortSmem = kSortBins + 2 * 4 * kSortRound;   // and one round's ids and places

struct SortArgs {
    const void* tokens;
    int32_t token_bytes;
    int64_t T, V;
    uint32_t* key0;                  // ping-pong lists; after an odd number of
    uint32_t* key1;                  // passes the result is in the second
    uint32_t* pos0;
    uint32_t* pos1;
    int32_t* long_runs;              // set to 0 for the next launch
    int32_t passes, bits;            // digits of `bits` bits
    int32_t cluster;
    uint4* zero;                     // the gradient to fill, or null
    int64_t zero_vecs;
    int32_t* status;
};

// This address in another block of the cluster.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(r)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_remote(uint32_t addr, uint32_t x)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t addr)
{
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::
                     : "memory");
}

__global__ void __launch_bounds__(kSortThreads) k_sort(const __grid_constant__ SortArgs a)
{
    extern __shared__ uint32_t warp_bins[];                 // [kSortWarps][bins]
    uint32_t* held_key = warp_bins + kSortBins / 4;         // one round: this block's part
    uint32_t* held_pos = held_key + kSortRound;             // between two passes
    __shared__ uint32_t base[kMaxBins], total[kMaxBins], counts[kMaxBins];
    __shared__ uint32_t warp_total[kMaxBins / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if ((int)blockIdx.x >= a.cluster) {                     // whole clusters of fillers
        const int64_t n = (int64_t)(gridDim.x - a.cluster) * kSortThreads;
        for (int64_t i = (int64_t)(blockIdx.x - a.cluster) * kSortThreads + tid; i < a.zero_vecs;
             i += n)
            st16_stream(a.zero + i, make_uint4(0, 0, 0, 0));
        return;
    }

    if (blockIdx.x == 0 && tid == 0) *a.long_runs = 0;
    const int bins = 1 << a.bits;
    const int64_t part = (a.T + a.cluster - 1) / a.cluster;
    const int64_t lo = min((int64_t)blockIdx.x * part, a.T), hi = min(lo + part, a.T);
    const bool one_round = part <= kSortRound;
    // items of a thread and round: as few as do, since each is a row of votes
    const int items = one_round ? (int)((part + kSortThreads - 1) / kSortThreads) : kSortItems;
    uint32_t* mine = warp_bins + warp * bins;
    for (int pass = 0; pass < a.passes; ++pass) {
        const uint32_t* key_in = pass & 1 ? a.key1 : a.key0;
        const uint32_t* pos_in = pass & 1 ? a.pos1 : a.pos0;
        uint32_t* key_out = pass & 1 ? a.key0 : a.key1;
        uint32_t* pos_out = pass & 1 ? a.pos0 : a.pos1;
        const int shift = pass * a.bits;
        auto load = [&](int64_t i, uint32_t& k, uint32_t& p) {
            if (pass > 0 && one_round) {                    // written by the other blocks
                k = held_key[i - lo];
                p = held_pos[i - lo];
                return;
            }
            if (pass > 0) {
                k = __ldcg(key_in + i);
                p = __ldcg(pos_in + i);
                return;
            }
            const int64_t v = token_at(a.tokens, a.token_bytes, i);
            if (v >= a.V && a.status) atomicOr(a.status, ZERO_DEV_BAD_TOKEN);
            k = v >= 0 && v < a.V ? (uint32_t)v : (uint32_t)a.V;
            p = (uint32_t)i;
        };
        uint32_t k[kSortItems], p[kSortItems], rank[kSortItems];
        // A round's items, a warp 32 * items consecutive ones in list order:
        // each item's rank in its warp, each warp's first place in the block's
        // items of a digit (in warp_bins), and the block's total of each digit.
        auto rank_round = [&](int64_t r0) {
            for (int b = tid; b < kSortWarps * bins; b += kSortThreads) warp_bins[b] = 0;
            const int64_t w0 = r0 + warp * 32 * items + lane;
#pragma unroll
            for (int q = 0; q < kSortItems; ++q) {
                k[q] = 0;
                if (q < items && w0 + q * 32 < hi) load(w0 + q * 32, k[q], p[q]);
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kSortItems; ++q) {
                if (q >= items) break;
                const bool in = w0 + q * 32 < hi;
                const uint32_t d = (k[q] >> shift) & (bins - 1);
                // the lanes with the same digit, a vote for each of its bits
                // (the match instruction took several times as long)
                uint32_t same = __ballot_sync(0xFFFFFFFFu, in);
                for (int b = 0; b < a.bits; ++b) {
                    const uint32_t set = __ballot_sync(0xFFFFFFFFu, d >> b & 1);
                    same &= d >> b & 1 ? set : ~set;
                }
                const uint32_t below = __popc(same & ((1u << lane) - 1));
                const uint32_t had = in ? mine[d] : 0;
                __syncwarp();
                if (in && below == 0) mine[d] = had + __popc(same);
                rank[q] = had + below;
                __syncwarp();
            }
            __syncthreads();
            for (int b = tid; b < bins; b += kSortThreads) {
                uint32_t sum = 0;
#pragma unroll 8
                for (int w = 0; w < kSortWarps; ++w) {
                    const uint32_t n = warp_bins[w * bins + b];
                    warp_bins[w * bins + b] = sum;
                    sum += n;
                }
                total[b] = sum;
            }
            __syncthreads();
        };

        // how many items of each digit this block has
        if (one_round) {
            rank_round(lo);
        } else {
            for (int b = tid; b < bins; b += kSortThreads) total[b] = 0;
            __syncthreads();
            for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
                uint32_t kk, pp;
                load(i, kk, pp);
                atomicAdd(&total[(kk >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
        }
        // where this block's first item of each digit goes: the smaller
        // digits of all blocks, then the same digit of the blocks before
        uint32_t before = 0, sum = 0;
        if (a.cluster > 1) {
            if (tid < bins) counts[tid] = total[tid];
            cluster_sync();
            if (tid < bins) {
                uint32_t n[kMaxCluster];
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    n[q] = q < a.cluster ? ld_remote(in_block(&counts[tid], q)) : 0;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q) {
                    sum += n[q];
                    if (q < (int)blockIdx.x) before += n[q];
                }
            }
        } else if (tid < bins) {
            sum = total[tid];
        }
        // the others have read this block's counts once all have arrived here:
        // waited for at the end, before the block leaves or counts again
        if (pass + 1 == a.passes)
            asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        if (tid < kMaxBins) {
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) warp_total[warp] = incl;
            before += incl - sum;
        }
        __syncthreads();
        if (tid < bins) {
            for (int w = 0; w < warp; ++w) before += warp_total[w];
            base[tid] = before;
        }
        __syncthreads();

        for (int64_t r0 = lo; r0 < hi; r0 += kSortRound) {
            if (!one_round) rank_round(r0);
            const int64_t w0 = r0 + warp * 32 * items + lane;
#pragma unroll
            for (int q = 0; q < kSortItems; ++q) {
                if (q < items && w0 + q * 32 < hi) {
                    const uint32_t d = (k[q] >> shift) & (bins - 1);
                    const uint32_t to = base[d] + mine[d] + rank[q];
                    if (one_round && pass + 1 < a.passes) {
                        const uint32_t block = to / (uint32_t)part, at = to - block * (uint32_t)part;
                        st_remote(in_block(held_key + at, block), k[q]);
                        st_remote(in_block(held_pos + at, block), p[q]);
                    } else {
                        __stcg(key_out + to, k[q]);
                        __stcg(pos_out + to, p[q]);
                    }
                }
            }
            if (!one_round) {
                __syncthreads();
                for (int b = tid; b < bins; b += kSortThreads) base[b] += total[b];
                __syncthreads();
            }
        }
        if (pass + 1 < a.passes) cluster_sync();
        else asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
}

// ============================================================== gradient ==
// The sorted list is cut into chunks of C places; a warp takes a chunk and
// 256 columns (16 bytes a lane).  A token's run of at most C places is summed
// by the warp of the chunk it starts in, which reads on into the next chunk
// where the run does; it is written once, already rounded.  A longer run
// leaves one fp32 part per chunk it meets, and k_embed_join adds those in
// order.  So a frequent token is spread over as many warps as it has chunks,
// and text's many rare tokens leave no parts at all.

constexpr int kColumns = 256;                // of a warp: 32 lanes x 8
constexpr int kGradThreads = 128;
constexpr int kJoinThreads = 256;
constexpr int kBatch = 8;                    // rows in flight
constexpr int64_t kFewWarps = 2432;          // 16 for each of 152 SMs

struct GradArgs {
    const uint16_t* dy;
    const uint32_t* key;
    const uint32_t* pos;
    uint16_t* grad;
    float* parts;                            // [2 * chunks][D]: a chunk's head and tail
    int32_t* long_runs;                      // their number; from the third word on, the
                                             // chunk each starts in and its key
    int64_t T, V, dy_ld;
    int32_t D, slices, chunks, accumulate;
    float scale;
};

// What a warp finds out about a chunk from the keys around it.
struct ChunkRuns {
    uint32_t cur, next;                      // lane i: the key at place i, and at place C + i
    int skip;                                // leading places that belong to an earlier chunk's run
    bool head_long, tail_long;               // a long run covers [0, skip) / [tail, C)
    int tail;                                // where the tail run starts, C if it ends in the chunk
    int n;                                   // places with a token, in the chunk
    int more;                                // places of the tail run after the chunk, if not long
};

template <int C>
__device__ __forceinline__ ChunkRuns chunk_runs(const uint32_t* key, int64_t T, int64_t V,
                                                int64_t c, int lane)
{
    constexpr uint32_t ALL = 0xFFFFFFFFu, PLACES = C == 32 ? ALL : (1u << (C & 31)) - 1;
    ChunkRuns r;
    const uint32_t none = (uint32_t)V;
    const int64_t i = c * C + lane;
    const uint32_t prev = c > 0 && lane < C ? key[i - C] : none;
    r.cur = lane < C && i < T ? key[i] : none;
    r.next = lane < C && i + C < T ? key[i + C] : none;
    const uint32_t first = __shfl_sync(ALL, r.cur, 0);
    const uint32_t last = __shfl_sync(ALL, r.cur, C - 1);
    r.n = __popc(__ballot_sync(ALL, r.cur != none) & PLACES);
    const uint32_t not_head = __ballot_sync(ALL, r.cur != first) & PLACES;
    const uint32_t not_tail = __ballot_sync(ALL, r.cur != last) & PLACES;
    const uint32_t prev_not = __ballot_sync(ALL, prev != first) & PLACES;
    const uint32_t next_not = __ballot_sync(ALL, r.next != last) & PLACES;
    const int lead = not_head ? __ffs(not_head) - 1 : C;         // of the first key
    const int before = prev_not ? C - 32 + __clz(prev_not) : C;  // places just before the chunk
    const int after = next_not ? __ffs(next_not) - 1 : C;        // places just after it
    r.skip = first != none && before > 0 ? lead : 0;
    r.head_long = r.skip > 0 && before + lead > C;
    // the tail run: starts in this chunk and goes on in the next
    const bool goes_on = last != none && after > 0;
    const int start = not_tail ? 32 - __clz(not_tail) : 0;
    r.tail = goes_on && !(start == 0 && r.skip > 0) ? start : C;
    r.tail_long = r.tail < C && (C - r.tail) + after > C;
    r.more = r.tail < C && !r.tail_long ? after : 0;
    return r;
}

__device__ __forceinline__ void add8(float (&acc)[8], const uint4& x)
{
    float f[8];
    bf_unpack8(x, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += f[q];
}

template <int C, bool ACC>
__global__ void __launch_bounds__(kGradThreads) k_embed_grad(const __grid_constant__ GradArgs a)
{
    pdl_enter();
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * kGradThreads + threadIdx.x) >> 5;
    const int64_t c = w / a.slices;
    if (c >= a.chunks) return;
    const int col = (int)(w % a.slices) * kColumns + lane * 8;
    const bool on = col < a.D;
    const int64_t i0 = c * C;
    const uint32_t pos_cur = lane < C && i0 + lane < a.T ? a.pos[i0 + lane] : 0;
    const uint32_t pos_next = lane < C && i0 + C + lane < a.T ? a.pos[i0 + C + lane] : 0;
    const ChunkRuns r = chunk_runs<C>(a.key, a.T, a.V, c, lane);
    if (r.n == 0) return;
    // (in any order: each run is joined by itself)
    const uint32_t last = __shfl_sync(ALL, r.cur, C - 1);
    if (r.tail_long && w % a.slices == 0 && lane == 0)
        reinterpret_cast<uint2*>(a.long_runs)[1 + atomicAdd(a.long_runs, 1)] =
            make_uint2((uint32_t)c, last);

    // places [from, to) of the chunk and the C after it, a batch of rows at a
    // time, all asked for before the first is added; what the gradient holds
    // where a run ends is brought into L2 meanwhile (registers for it would
    // halve the resident warps)
    const int from = r.head_long ? 0 : r.skip;
    const int to = r.n + r.more;
    // bit s: place s is the last of its run (or of what is summed here); and
    // place s is of a long run
    uint64_t ends, longs;
    {
        constexpr uint32_t PLACES = C == 32 ? ALL : (1u << (C & 31)) - 1;
        const uint32_t up = __shfl_down_sync(ALL, r.cur, 1), first_next = __shfl_sync(ALL, r.next, 0);
        ends = (__ballot_sync(ALL, r.cur != (lane == C - 1 ? first_next : up)) & PLACES) |
               1ull << (to - 1);
        longs = (r.head_long ? (1ull << r.skip) - 1 : 0) |
                (r.tail_long ? (1ull << C) - (1ull << r.tail) : 0);
    }
    const uint16_t* dy = a.dy + col;
    uint16_t* grad = a.grad + col;
    float acc[8] = {};
    for (int b = from; b < to; b += kBatch) {
        // the batch's places: bit q stands for place b + q
        const uint32_t in = to - b >= kBatch ? (1u << kBatch) - 1 : (1u << (to - b)) - 1;
        const uint32_t end = (uint32_t)(ends >> b) & in, part = (uint32_t)(longs >> b);
        uint4 x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const uint32_t t = __shfl_sync(ALL, b + q < C ? pos_cur : pos_next, b + q & (C - 1));
            x[q] = make_uint4(0, 0, 0, 0);
            if (on && (in >> q & 1)) x[q] = ld16_stream(dy + t * a.dy_ld);
        }
        if constexpr (ACC) {
            for (uint32_t m = end & ~part; m; m &= m - 1) {
                const int s = b + __ffs(m) - 1;
                const uint32_t v = __shfl_sync(ALL, s < C ? r.cur : r.next, s & (C - 1));
                if (on) asm volatile("prefetch.global.L2 [%0];" ::"l"(grad + (int64_t)v * a.D));
            }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            add8(acc, x[q]);
            if (!(end >> q & 1)) continue;                         // the same for the whole warp
            const int s = b + q;
            const uint32_t v = __shfl_sync(ALL, s < C ? r.cur : r.next, s & (C - 1));
            if (on && (part >> q & 1)) {
                float* to_part = a.parts + (2 * c + (s >= r.skip ? 1 : 0)) * a.D + col;
                *reinterpret_cast<float4*>(to_part) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                *reinterpret_cast<float4*>(to_part + 4) =
                    make_float4(acc[4], acc[5], acc[6], acc[7]);
            } else if (on) {
                float f[8] = {};
                if constexpr (ACC) bf_unpack8(ld16(grad + (int64_t)v * a.D), f);
#pragma unroll
                for (int z = 0; z < 8; ++z) f[z] += acc[z] * a.scale;
                st16(grad + (int64_t)v * a.D, bf_pack8(f));
            }
#pragma unroll
            for (int z = 0; z < 8; ++z) acc[z] = 0.0f;
        }
    }
}

// Joins the parts of each long run: the chunk where the run starts has a tail
// part, the next ones head parts.  A block takes a run and 256 columns: its 8
// warps add a consecutive share of the parts each, and the shares are added in
// order.
template <int C>
__global__ void __launch_bounds__(kJoinThreads) k_embed_join(const __grid_constant__ GradArgs a)
{
    pdl_enter();
    constexpr int W = kJoinThreads / 32;
    __shared__ float share[W][kColumns];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t items = (int64_t)a.long_runs[0] * a.slices;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint2 run = reinterpret_cast<const uint2*>(a.long_runs)[1 + item / a.slices];
        const int64_t c = run.x;
        const int col = (int)(item % a.slices) * kColumns + lane * 8;
        const uint32_t v = run.y;
        // the first place past the run, by 32 probes at a time
        int64_t lo = (c + 1) * C, hi = a.T;
        for (int64_t near = 32; lo < hi; near = hi) {          // most are found near the start
            const int64_t gap = min(near, (hi - lo + 31) / 32), at = lo + lane * gap;
            const uint32_t past =
                __ballot_sync(0xFFFFFFFFu, at >= hi || a.key[at < hi ? at : hi - 1] > v);
            const int k = past ? __ffs(past) - 1 : 32;         // probes before k are in the run
            if (past) hi = min(hi, lo + k * gap);
            if (k > 0) lo += (k - 1) * gap + 1;
        }
        const int64_t parts = (lo - 1) / C - c + 1;            // one of each chunk it meets
        const int64_t each = (parts + W - 1) / W;
        const int64_t p0 = min(warp * each, parts), p1 = min(p0 + each, parts);
        float acc[8] = {};
        if (col < a.D) {
#pragma unroll 4
            for (int64_t p = p0; p < p1; ++p) {
                const float* s = a.parts + (2 * (c + p) + (p == 0 ? 1 : 0)) * a.D + col;
                const float4 x = *reinterpret_cast<const float4*>(s);
                const float4 y = *reinterpret_cast<const float4*>(s + 4);
                acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
                acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) share[warp][q * 32 + lane] = acc[q];
        __syncthreads();
        if (warp == 0 && col < a.D) {
            for (int j = 1; j < W; ++j)
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] += share[j][q * 32 + lane];
            uint16_t* p = a.grad + (int64_t)v * a.D + col;
            float f[8] = {};
            if (a.accumulate) bf_unpack8(ld16(p), f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] += acc[q] * a.scale;
            st16(p, bf_pack8(f));
        }
        __syncthreads();
    }
}

// Chunks of 32 places leave the fewest parts; with few tokens chunks of 8
// give four times the warps, each with one batch of rows to wait for.
int chunk_places(int64_t T, int32_t D)
{
    const int64_t warps = (T + 31) / 32 * ((D + kColumns - 1) / kColumns);
    return warps >= kFewWarps ? 32 : 8;
}

template <int C>
cudaError_t launch_grad(GradArgs a, cudaStream_t st)
{
    a.chunks = (int32_t)((a.T + C - 1) / C);
    const int64_t warps = (int64_t)a.chunks * a.slices;
    const int per = kGradThreads / 32;
    const dim3 grid((unsigned)((warps + per - 1) / per));
    cudaError_t e = launch(a.accumulate ? k_embed_grad<C, true> : k_embed_grad<C, false>, grid,
                           kGradThreads, 0, st, a);
    if (e == cudaSuccess && a.T > C) {
        // a long run has more than C places, so there are fewer of them than chunks
        const int64_t blocks = std::min<int64_t>((int64_t)a.chunks * a.slices, 6 * device_sms());
        e = launch(k_embed_join<C>, dim3((unsigned)blocks), kJoinThreads, 0, st, a);
    }
    return e;
}

// ------------------------------------------------- the gradient, few tokens --
// Up to 1024 tokens need no sort: a block takes a token and 1024 columns (256 a
// warp), looks through all ids for its own, stops unless it is the first to
// have it, and adds the rows.  One launch instead of three; other blocks fill
// the rows that no token has with zeros (16 rows a block, after a look at the
// same ids).  Measured against the sort: 64 x 768 into a tied table 18 -> 3 us,
// 1023 x 768 into an untied one of 50257 rows 22.6 -> 14.8 us.

constexpr int kFew = 1024;
constexpr int kFewThreads = 128;
constexpr int kFewBatch = 8;                 // rows in flight
constexpr int kFillRows = 16;                // (32 and 64: 11.4 -> 12.2 and 16.8 us for 77 MB)

struct FewArgs {
    const uint16_t* dy;
    const void* tokens;
    uint16_t* grad;
    int64_t V, dy_ld;
    int32_t T, D, slices, token_bytes, accumulate;
    int32_t fills;                           // blocks that fill with zeros
    float scale;
    int32_t* status;
};

__global__ void __launch_bounds__(kFewThreads) k_embed_few(const __grid_constant__ FewArgs a)
{
    pdl_enter();
    constexpr int W = kFewThreads / 32, EACH = kFew / kFewThreads;
    __shared__ uint16_t list[kFew];
    __shared__ uint32_t found[W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i0 = tid * EACH;                               // this thread's ids
    if ((int)blockIdx.x < a.fills) {                         // zeros
        const int64_t v0 = (int64_t)blockIdx.x * kFillRows;
        const int n = (int)min((int64_t)kFillRows, a.V - v0);
        if (tid == 0) found[0] = 0;
        __syncthreads();
        for (int i = tid; i < a.T; i += kFewThreads) {
            const int64_t r = token_at(a.tokens, a.token_bytes, i) - v0;
            if (r >= 0 && r < n) atomicOr(&found[0], 1u << r);
        }
        __syncthreads();
        const uint32_t met = found[0];
        const int nv = a.D >> 3;
        for (int r = warp; r < n; r += W) {
            if (met >> r & 1) continue;
            uint16_t* row = a.grad + (v0 + r) * a.D;
            for (int c = lane; c < nv; c += 32) st16_stream(row + c * 8, make_uint4(0, 0, 0, 0));
        }
        return;
    }

    const int block = (int)blockIdx.x - a.fills;
    const int groups = (a.slices + W - 1) / W, t = block / groups;
    const int col = (block % groups * W + warp) * kColumns + lane * 8;
    const int64_t v = token_at(a.tokens, a.token_bytes, t);
    if (v < 0 || v >= a.V) {
        if (v >= a.V && a.status && tid == 0) atomicOr(a.status, ZERO_DEV_BAD_TOKEN);
        return;
    }
    uint32_t same = 0;                                       // bit q: id i0 + q is this one
#pragma unroll
    for (int q = 0; q < EACH; ++q)
        if (i0 + q < a.T && token_at(a.tokens, a.token_bytes, i0 + q) == v) same |= 1u << q;
    const uint32_t before = i0 >= t ? 0 : t - i0 >= EACH ? same : same & ((1u << (t - i0)) - 1);
    if (__syncthreads_or(before != 0)) return;               // another block's
    // the places of the id, in order
    int at = __popc(same);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (lane >= o) at += x;
    }
    if (lane == 31) found[warp] = at;
    at -= __popc(same);
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        if (k < warp) at += found[k];
        n += found[k];
    }
    for (uint32_t m = same; m; m &= m - 1) list[at++] = (uint16_t)(i0 + __ffs(m) - 1);
    __syncthreads();

    if (col - lane * 8 >= a.D) return;                       // a warp past the row's end
    const bool on = col < a.D;
    float acc[8] = {};
    // (no load depends on a condition, so that all are asked for at once: the
    // last row again past the list's end, the first columns past the row's)
    const uint16_t* dy = a.dy + (on ? col : 0);
    for (int b = 0; b < n; b += kFewBatch) {
        uint4 x[kFewBatch];
#pragma unroll
        for (int q = 0; q < kFewBatch; ++q)
            x[q] = ld16(dy + (int64_t)list[min(b + q, n - 1)] * a.dy_ld);
#pragma unroll
        for (int q = 0; q < kFewBatch; ++q)
            if (b + q < n) add8(acc, x[q]);
    }
    if (on) {
        uint16_t* p = a.grad + v * a.D + col;
        float f[8] = {};
        if (a.accumulate) bf_unpack8(ld16(p), f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] += acc[q] * a.scale;
        st16(p, bf_pack8(f));
    }
}

struct GradScratch {
    int64_t key0, key1, pos0, pos1, long_runs, parts, bytes;
};

GradScratch grad_scratch(int64_t T, int32_t D)
{
    GradScratch s{};
    if (T <= kFew) {
        s.bytes = 256;
        return s;
    }
    const int64_t list = up(4 * T, 256);
    s.key0 = 0;
    s.key1 = list;
    s.pos0 = 2 * list;
    s.pos1 = 3 * list;
    const int C = chunk_places(T, D);
    s.long_runs = 4 * list;
    s.parts = s.long_runs + up(8 * (1 + (T + C - 1) / C), 256);
    s.bytes = s.parts + 8 * ((T + C - 1) / C) * (int64_t)D;
    return s;
}

// What grad_scratch() asks for at any number of tokens up to T: fewer tokens
// may have more chunks, of 8 places.
int64_t grad_bytes(int64_t T, int32_t D)
{
    const int64_t slices = (D + kColumns - 1) / kColumns;
    const int64_t last8 = (kFewWarps - 1) / slices * 32;       // tokens with such chunks
    return std::max(T > last8 ? grad_scratch(last8, D).bytes : 0, grad_scratch(T, D).bytes);
}

zero_status check_grad(int64_t T, int64_t V, int32_t D)
{
    LM_CHECK(check_sizes(T, V, D));
    // a launch's warps
    const int64_t slices = (D + kColumns - 1) / kColumns;
    return (T + 31) / 32 * slices > INT32_MAX ? ZERO_ERR_SIZE : ZERO_OK;
}

}  // namespace

extern "C" zero_status zero_embed(const uint16_t* table, int64_t V, int32_t D, const void* tokens,
                                  int32_t token_bytes, int64_t T, float scale, uint16_t* out,
                                  int64_t out_ld, int32_t* dev_status, void* stream)
{
    LM_CHECK(check_sizes(T, V, D));
    LM_CHECK(check_ld(out_ld, D));
    if (token_bytes != 4 && token_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (T == 0) return ZERO_OK;
    LM_CHECK(check_ptr(table));
    LM_CHECK(check_tokens(tokens, token_bytes));
    LM_CHECK(check_ptr(out));
    LM_CHECK(check_status(dev_status));
    Spans sp;
    sp.add(table, 2 * V * D, false);
    sp.add(tokens, T * token_bytes, false);
    sp.rows(out, T, out_ld, D, 2, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    LookupArgs a{};
    a.table = table;
    a.tokens = tokens;
    a.out = out;
    a.T = T;
    a.V = V;
    a.out_ld = out_ld;
    a.D = D;
    a.token_bytes = token_bytes;
    a.scale = scale;
    a.status = dev_status;
    a.lanes_log2 = 0;
    while ((1 << a.lanes_log2) < 32 && (1 << a.lanes_log2) < D / 8) ++a.lanes_log2;
    const int rows = kLookupThreads >> a.lanes_log2;
    const int64_t blocks = (T + rows - 1) / rows;
    return status_of(launch(k_lookup, dim3((unsigned)blocks), kLookupThreads, 0,
                            static_cast<cudaStream_t>(stream), a));
}

extern "C" int64_t zero_embed_grad_scratch_bytes(int64_t T, int64_t V, int32_t D)
{
    if (check_grad(T, V, D) != ZERO_OK) return -1;
    return grad_bytes(T, D);
}

extern "C" zero_status zero_embed_grad(const uint16_t* dy, int64_t dy_ld, const void* tokens,
                                       int32_t token_bytes, int64_t T, float scale, int64_t V,
                                       int32_t D, uint16_t* grad, int32_t accumulate,
                                       void* scratch, int64_t scratch_bytes, int32_t* dev_status,
                                       void* stream)
{
    LM_CHECK(check_grad(T, V, D));
    LM_CHECK(check_ld(dy_ld, D));
    if (token_bytes != 4 && token_bytes != 8) return ZERO_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return ZERO_ERR_INVALID_ARG;
    LM_CHECK(check_ptr(grad));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (accumulate) return ZERO_OK;
        return status_of(cudaMemsetAsync(grad, 0, (size_t)(2 * V * D), st));
    }
    LM_CHECK(check_ptr(dy));
    LM_CHECK(check_tokens(tokens, token_bytes));
    LM_CHECK(check_ptr(scratch));
    LM_CHECK(check_status(dev_status));
    const int64_t slices = (D + kColumns - 1) / kColumns;
    const GradScratch g = grad_scratch(T, D);
    if (scratch_bytes < g.bytes) return ZERO_ERR_SIZE;
    Spans sp;
    sp.rows(dy, T, dy_ld, D, 2, false);
    sp.add(tokens, T * token_bytes, false);
    sp.add(grad, 2 * V * D, true);
    sp.add(scratch, g.bytes, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    if (T <= kFew) {
        const int32_t fills = accumulate ? 0 : (int32_t)((V + kFillRows - 1) / kFillRows);
        const FewArgs f{dy, tokens, grad, V, dy_ld, (int32_t)T, D, (int32_t)slices, token_bytes,
                        accumulate, fills, scale, dev_status};
        const int64_t groups = (slices + kFewThreads / 32 - 1) / (kFewThreads / 32);
        return status_of(launch(k_embed_few, dim3((unsigned)(fills + T * groups)), kFewThreads, 0,
                                st, f));
    }

    uint8_t* base = static_cast<uint8_t*>(scratch);
    SortArgs s{};
    s.tokens = tokens;
    s.token_bytes = token_bytes;
    s.T = T;
    s.V = V;
    s.key0 = reinterpret_cast<uint32_t*>(base + g.key0);
    s.key1 = reinterpret_cast<uint32_t*>(base + g.key1);
    s.pos0 = reinterpret_cast<uint32_t*>(base + g.pos0);
    s.pos1 = reinterpret_cast<uint32_t*>(base + g.pos1);
    s.long_runs = reinterpret_cast<int32_t*>(base + g.long_runs);
    int key_bits = 1;                                      // keys run to V itself
    while (key_bits < 32 && (V >> key_bits) != 0) ++key_bits;
    s.passes = (key_bits + 8) / 9;                         // digits of at most 9 bits
    s.bits = (key_bits + s.passes - 1) / s.passes;
    s.cluster = T <= 2 * kSortThreads ? 1 : kMaxCluster;      // (4000 tokens: 24.6 and 22 us)
    s.status = dev_status;
    int fillers = 0;
    if (!accumulate) {
        s.zero = reinterpret_cast<uint4*>(grad);
        s.zero_vecs = V * D / 8;
        const int64_t want = (s.zero_vecs + kSortThreads * 4 - 1) / (kSortThreads * 4);
        fillers = (int)std::min<int64_t>(want, 2 * device_sms());
        fillers = (int)up(fillers, s.cluster);
    }
    static std::atomic<uint64_t> smem_set;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&k_sort), kSortSmem, smem_set);
    if (e == cudaSuccess)
        e = launch_clusters(k_sort, dim3((unsigned)(s.cluster + fillers)), kSortThreads,
                            kSortSmem, s.cluster, st, s);
    if (e != cudaSuccess) return status_of(e);

    GradArgs a{};
    a.dy = dy;
    a.key = s.passes & 1 ? s.key1 : s.key0;
    a.pos = s.passes & 1 ? s.pos1 : s.pos0;
    a.grad = grad;
    a.parts = reinterpret_cast<float*>(base + g.parts);
    a.long_runs = s.long_runs;
    a.T = T;
    a.V = V;
    a.dy_ld = dy_ld;
    a.D = D;
    a.slices = (int32_t)slices;
    a.accumulate = accumulate;
    a.scale = scale;
    e = chunk_places(T, D) == 32 ? launch_grad<32>(a, st) : launch_grad<8>(a, st);
    return status_of(e);
}
