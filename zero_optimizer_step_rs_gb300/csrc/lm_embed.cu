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
// The gradient's sums have one fixed order, so a step can be repeated bit for
// bit: the tokens are sorted by (id, position) and each row's terms are
// added in that order, in pieces that depend on the tokens alone.  No
// atomics touch a sum.
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
// cluster of up to 8 blocks: a block owns a contiguous part of the list, the
// blocks exchange digit counts and items through global memory (L2), and the
// cluster barrier orders the passes, so the whole sort is one launch.  Ids
// that take part in nothing (negative, or past the table) get the key V and
// end up last.
//
// The rest of the grid, where there is one, fills the table's gradient with
// zeros meanwhile; the rows that are met are written by the next launch.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 4;                               // per thread and round
constexpr int kSortRound = kSortThreads * kSortItems;       // items of a block per round
constexpr int kMaxCluster = 8;
constexpr int kMaxBins = 512;
constexpr int kSortSmem = kSortWarps * kMaxBins * 4;

struct SortArgs {
    const void* tokens;
    int32_t token_bytes;
    int64_t T, V;
    uint32_t* key[2];                // ping-pong lists; the result is in key[passes & 1]
    uint32_t* pos[2];
    uint32_t* counts;                // [kMaxCluster][kMaxBins]
    int32_t passes, bits;            // digits of `bits` bits
    int32_t cluster;
    uint4* zero;                     // the gradient to fill, or null
    int64_t zero_vecs;
    int32_t* status;
};

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

__global__ void __launch_bounds__(kSortThreads) k_sort(const __grid_constant__ SortArgs a)
{
    pdl_enter();
    extern __shared__ uint32_t warp_bins[];                 // [kSortWarps][bins]
    __shared__ uint32_t base[kMaxBins], scan[kMaxBins];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if ((int)blockIdx.x >= a.cluster) {                     // whole clusters of fillers
        const int64_t n = (int64_t)(gridDim.x - a.cluster) * kSortThreads;
        for (int64_t i = (int64_t)(blockIdx.x - a.cluster) * kSortThreads + tid; i < a.zero_vecs;
             i += n)
            st16_stream(a.zero + i, make_uint4(0, 0, 0, 0));
        return;
    }

    const int bins = 1 << a.bits;
    const int64_t part = (a.T + a.cluster - 1) / a.cluster;
    const int64_t lo = min((int64_t)blockIdx.x * part, a.T), hi = min(lo + part, a.T);
    for (int pass = 0; pass < a.passes; ++pass) {
        const uint32_t* key_in = a.key[pass & 1];
        const uint32_t* pos_in = a.pos[pass & 1];
        uint32_t* key_out = a.key[(pass & 1) ^ 1];
        uint32_t* pos_out = a.pos[(pass & 1) ^ 1];
        const int shift = pass * a.bits;
        auto load = [&](int64_t i, uint32_t& k, uint32_t& p) {
            if (pass > 0) {                                 // written by the other blocks
                k = __ldcg(key_in + i);
                p = __ldcg(pos_in + i);
                return;
            }
            const int64_t v = token_at(a.tokens, a.token_bytes, i);
            if (v >= a.V && a.status) atomicOr(a.status, ZERO_DEV_BAD_TOKEN);
            k = v >= 0 && v < a.V ? (uint32_t)v : (uint32_t)a.V;
            p = (uint32_t)i;
        };

        // how many items of each digit this block has
        for (int b = tid; b < bins; b += kSortThreads) scan[b] = 0;
        __syncthreads();
        for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
            uint32_t k, p;
            load(i, k, p);
            atomicAdd(&scan[(k >> shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        for (int b = tid; b < bins; b += kSortThreads)
            __stcg(a.counts + blockIdx.x * kMaxBins + b, scan[b]);
        cluster_sync();

        // where this block's first item of each digit goes: the smaller
        // digits of all blocks, then the same digit of the blocks before
        uint32_t before = 0, total = 0;
        if (tid < bins) {
            for (int q = 0; q < a.cluster; ++q) {
                const uint32_t n = __ldcg(a.counts + q * kMaxBins + tid);
                total += n;
                if (q < (int)blockIdx.x) before += n;
            }
        }
        if (tid < kMaxBins) scan[tid] = tid < bins ? total : 0;
        __syncthreads();
        for (int o = 1; o < kMaxBins; o <<= 1) {
            uint32_t x = 0;
            if (tid < kMaxBins && tid >= o) x = scan[tid - o];
            __syncthreads();
            if (tid < kMaxBins) scan[tid] += x;
            __syncthreads();
        }
        if (tid < bins) base[tid] = scan[tid] - total + before;
        __syncthreads();

        for (int64_t r0 = lo; r0 < hi; r0 += kSortRound) {
            for (int b = tid; b < kSortWarps * bins; b += kSortThreads) warp_bins[b] = 0;
            __syncthreads();
            // a warp owns 32 * kSortItems consecutive items, in list order
            uint32_t k[kSortItems], p[kSortItems], rank[kSortItems];
            uint32_t* mine = warp_bins + warp * bins;
            const int64_t w0 = r0 + warp * 32 * kSortItems + lane;
#pragma unroll
            for (int q = 0; q < kSortItems; ++q) {
                const int64_t i = w0 + q * 32;
                if (i < hi) load(i, k[q], p[q]);
            }
#pragma unroll
            for (int q = 0; q < kSortItems; ++q) {
                const bool in = w0 + q * 32 < hi;
                const uint32_t d = in ? (k[q] >> shift) & (bins - 1) : 0xFFFFFFFFu;
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
                const int first = __ffs(same) - 1;
                const uint32_t below = __popc(same & ((1u << lane) - 1));
                uint32_t had = 0;
                if (in && lane == first) {
                    had = mine[d];
                    mine[d] = had + __popc(same);
                }
                rank[q] = __shfl_sync(0xFFFFFFFFu, had, first) + below;
                __syncwarp();
            }
            __syncthreads();
            for (int b = tid; b < bins; b += kSortThreads) {
                uint32_t at = base[b];
                for (int w = 0; w < kSortWarps; ++w) {
                    const uint32_t n = warp_bins[w * bins + b];
                    warp_bins[w * bins + b] = at;
                    at += n;
                }
                base[b] = at;
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kSortItems; ++q) {
                if (w0 + q * 32 < hi) {
                    const uint32_t to = mine[(k[q] >> shift) & (bins - 1)] + rank[q];
                    __stcg(key_out + to, k[q]);
                    __stcg(pos_out + to, p[q]);
                }
            }
            __syncthreads();
        }
        cluster_sync();
    }
}

// ============================================================== gradient ==
// The sorted list is cut into chunks of 32 places; a warp takes a chunk and
// 256 columns (16 bytes a lane).  A token's run of at most 32 places is summed
// by the warp of the chunk it starts in, which reads on into the next chunk
// where the run does; it is written once, already rounded.  A longer run
// leaves one fp32 part per chunk it meets, and k_embed_join adds those in
// order.  So a frequent token is spread over as many warps as it has chunks,
// and text's many rare tokens leave no parts at all.

constexpr int kChunk = 32;
constexpr int kColumns = 256;                // of a warp: 32 lanes x 8
constexpr int kGradThreads = 256;
constexpr int kGradBatch = 8;                // rows in flight

struct GradArgs {
    const uint16_t* dy;
    const uint32_t* key;
    const uint32_t* pos;
    uint16_t* grad;
    float* parts;                            // [2 * chunks][D]: a chunk's head and tail
    int64_t T, V, dy_ld;
    int32_t D, slices, accumulate;
    float scale;
};

__device__ __forceinline__ void add_row(float (&acc)[8], const uint4& x)
{
    float f[8];
    bf_unpack8(x, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += f[q];
}

__device__ __forceinline__ void write_row(const GradArgs& a, uint32_t v, int col, float (&acc)[8])
{
    uint16_t* p = a.grad + (int64_t)v * a.D + col;
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] *= a.scale;
    if (a.accumulate) {
        float f[8];
        bf_unpack8(ld16(p), f);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += f[q];
    }
    st16(p, bf_pack8(acc));
}

// What a warp finds out about a chunk from the keys around it.
struct ChunkRuns {
    uint32_t cur, next;                      // this lane's key in the chunk, and 32 places on
    int skip;                                // leading places that belong to an earlier chunk's run
    bool head_long, tail_long;               // a long run covers [0, skip) / [tail, 32)
    int tail;                                // where the tail run starts, 32 if it ends in the chunk
    int n;                                   // places with a token, in the chunk
    int more;                                // places of the tail run after the chunk, if not long
};

__device__ __forceinline__ ChunkRuns chunk_runs(const uint32_t* key, int64_t T, int64_t V,
                                                int64_t c, int lane)
{
    ChunkRuns r;
    const uint32_t none = (uint32_t)V;
    const int64_t i = c * kChunk + lane;
    const uint32_t prev = c > 0 ? key[i - kChunk] : none;
    r.cur = i < T ? key[i] : none;
    r.next = i + kChunk < T ? key[i + kChunk] : none;
    const uint32_t first = __shfl_sync(0xFFFFFFFFu, r.cur, 0);
    const uint32_t last = __shfl_sync(0xFFFFFFFFu, r.cur, 31);
    r.n = __popc(__ballot_sync(0xFFFFFFFFu, r.cur != none));
    const uint32_t not_head = __ballot_sync(0xFFFFFFFFu, r.cur != first);
    const uint32_t not_tail = __ballot_sync(0xFFFFFFFFu, r.cur != last);
    const uint32_t prev_not = __ballot_sync(0xFFFFFFFFu, prev != first);
    const uint32_t next_not = __ballot_sync(0xFFFFFFFFu, r.next != last);
    const int lead = not_head ? __ffs(not_head) - 1 : 32;        // of the first key
    const int before = prev_not ? __clz(prev_not) : 32;          // places just before the chunk
    const int after = next_not ? __ffs(next_not) - 1 : 32;       // places just after it
    r.skip = first != none && before > 0 ? lead : 0;
    r.head_long = r.skip > 0 && (before + lead > kChunk);
    // the tail run: starts in this chunk and goes on in the next
    const bool goes_on = last != none && after > 0;
    const int start = not_tail ? 32 - __clz(not_tail) : 0;
    r.tail = goes_on && !(start == 0 && r.skip > 0) ? start : 32;
    r.tail_long = r.tail < 32 && (32 - r.tail) + after > kChunk;
    r.more = r.tail < 32 && !r.tail_long ? after : 0;
    return r;
}

__global__ void __launch_bounds__(kGradThreads) k_embed_grad(const __grid_constant__ GradArgs a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * kGradThreads + threadIdx.x) >> 5;
    const int64_t c = w / a.slices;
    if (c * kChunk >= a.T) return;
    const int col = (int)(w % a.slices) * kColumns + lane * 8;
    const bool on = col < a.D;
    const ChunkRuns r = chunk_runs(a.key, a.T, a.V, c, lane);
    if (r.n == 0) return;
    const int64_t i0 = c * kChunk;
    const uint32_t pos_cur = i0 + lane < a.T ? a.pos[i0 + lane] : 0;
    const uint32_t pos_next = i0 + kChunk + lane < a.T ? a.pos[i0 + kChunk + lane] : 0;

    // places [from, to) of the chunk and the 32 after it, a run at a time
    const int from = r.head_long ? 0 : r.skip;
    const int to = r.n + r.more;
    float acc[8] = {};
    for (int b = from; b < to; b += kGradBatch) {
        uint4 x[kGradBatch];
#pragma unroll
        for (int q = 0; q < kGradBatch; ++q) {
            const int s = b + q;
            const uint32_t p0 = __shfl_sync(0xFFFFFFFFu, pos_cur, s & 31);
            const uint32_t p1 = __shfl_sync(0xFFFFFFFFu, pos_next, s & 31);
            const int64_t t = s < 32 ? p0 : p1;
            x[q] = on && s < to ? ld16_stream(a.dy + t * a.dy_ld + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < kGradBatch; ++q) {
            const int s = b + q;
            if (s >= to) break;
            add_row(acc, x[q]);
            const uint32_t k0 = __shfl_sync(0xFFFFFFFFu, r.cur, s & 31);
            const uint32_t k1 = __shfl_sync(0xFFFFFFFFu, r.next, s & 31);
            const uint32_t v = s < 32 ? k0 : k1;
            const uint32_t n0 = __shfl_sync(0xFFFFFFFFu, r.cur, (s + 1) & 31);
            const uint32_t n1 = __shfl_sync(0xFFFFFFFFu, r.next, (s + 1) & 31);
            const uint32_t after = s + 1 < 32 ? n0 : n1;
            const bool ends = s + 1 == to || after != v || (s + 1 == 32 && r.more == 0);
            if (!ends) continue;
            if (on) {
                const bool head = r.head_long && s < r.skip;
                const bool tail = r.tail_long && s >= r.tail;
                if (head || tail) {
                    float* to_part = a.parts + (2 * c + (tail ? 1 : 0)) * a.D + col;
                    *reinterpret_cast<float4*>(to_part) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    *reinterpret_cast<float4*>(to_part + 4) =
                        make_float4(acc[4], acc[5], acc[6], acc[7]);
                } else {
                    write_row(a, v, col, acc);
                }
            }
#pragma unroll
            for (int z = 0; z < 8; ++z) acc[z] = 0.0f;
        }
    }
}

// Joins the parts of each long run: the block of the chunk where the run
// starts adds the tail part of that chunk and the head parts of the next
// ones.  Each of its 8 warps adds a consecutive share of them, and the shares
// are added in order.
__global__ void __launch_bounds__(kGradThreads) k_embed_join(const __grid_constant__ GradArgs a)
{
    pdl_enter();
    constexpr int W = kGradThreads / 32;
    __shared__ float share[W][kColumns];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x / a.slices;
    const int col = (int)(blockIdx.x % a.slices) * kColumns + lane * 8;
    const ChunkRuns r = chunk_runs(a.key, a.T, a.V, c, lane);
    if (!r.tail_long) return;                                  // the same in every warp
    const uint32_t v = __shfl_sync(0xFFFFFFFFu, r.cur, 31);
    int64_t lo = (c + 1) * kChunk, hi = a.T;                   // the first place past the run
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.key[mid] > v) hi = mid;
        else lo = mid + 1;
    }
    const int64_t parts = (lo - 1) / kChunk - c + 1;           // one of each chunk it meets
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
    for (int q = 0; q < 8; ++q) share[warp][lane * 8 + q] = acc[q];
    __syncthreads();
    if (warp == 0 && col < a.D) {
        for (int k = 1; k < W; ++k)
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += share[k][lane * 8 + q];
        write_row(a, v, col, acc);
    }
}

struct GradScratch {
    int64_t key0, key1, pos0, pos1, counts, parts, bytes;
};

GradScratch grad_scratch(int64_t T, int32_t D)
{
    GradScratch s;
    const int64_t list = up(4 * T, 256);
    s.key0 = 0;
    s.key1 = list;
    s.pos0 = 2 * list;
    s.pos1 = 3 * list;
    s.counts = 4 * list;
    s.parts = s.counts + 4 * kMaxCluster * kMaxBins;
    s.bytes = s.parts + 8 * ((T + kChunk - 1) / kChunk) * (int64_t)D;
    return s;
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
    return status_of(launch(k_lookup, dim3((unsigned)blocks), kLookupThreads, 0, 1,
                            static_cast<cudaStream_t>(stream), a));
}

extern "C" int64_t zero_embed_grad_scratch_bytes(int64_t T, int64_t V, int32_t D)
{
    if (check_sizes(T, V, D) != ZERO_OK) return -1;
    return grad_scratch(T, D).bytes;
}

extern "C" zero_status zero_embed_grad(const uint16_t* dy, int64_t dy_ld, const void* tokens,
                                       int32_t token_bytes, int64_t T, float scale, int64_t V,
                                       int32_t D, uint16_t* grad, int32_t accumulate,
                                       void* scratch, int64_t scratch_bytes, int32_t* dev_status,
                                       void* stream)
{
    LM_CHECK(check_sizes(T, V, D));
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
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    const int64_t slices = (D + kColumns - 1) / kColumns;
    if (chunks * slices > INT32_MAX) return ZERO_ERR_SIZE;         // a launch's blocks
    const GradScratch g = grad_scratch(T, D);
    if (scratch_bytes < g.bytes) return ZERO_ERR_SIZE;
    Spans sp;
    sp.rows(dy, T, dy_ld, D, 2, false);
    sp.add(tokens, T * token_bytes, false);
    sp.add(grad, 2 * V * D, true);
    sp.add(scratch, g.bytes, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());

    uint8_t* base = static_cast<uint8_t*>(scratch);
    SortArgs s{};
    s.tokens = tokens;
    s.token_bytes = token_bytes;
    s.T = T;
    s.V = V;
    s.key[0] = reinterpret_cast<uint32_t*>(base + g.key0);
    s.key[1] = reinterpret_cast<uint32_t*>(base + g.key1);
    s.pos[0] = reinterpret_cast<uint32_t*>(base + g.pos0);
    s.pos[1] = reinterpret_cast<uint32_t*>(base + g.pos1);
    s.counts = reinterpret_cast<uint32_t*>(base + g.counts);
    int key_bits = 1;                                      // keys run to V itself
    while (key_bits < 32 && (V >> key_bits) != 0) ++key_bits;
    s.passes = (key_bits + 8) / 9;                         // digits of at most 9 bits
    s.bits = (key_bits + s.passes - 1) / s.passes;
    s.cluster = 1;
    while (s.cluster < kMaxCluster && s.cluster * (int64_t)kSortRound < T) s.cluster *= 2;
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
        e = launch(k_sort, dim3((unsigned)(s.cluster + fillers)), kSortThreads,
                   kSortWarps * (4 << s.bits), s.cluster, st, s);
    if (e != cudaSuccess) return status_of(e);

    GradArgs a{};
    a.dy = dy;
    a.key = s.key[s.passes & 1];
    a.pos = s.pos[s.passes & 1];
    a.grad = grad;
    a.parts = reinterpret_cast<float*>(base + g.parts);
    a.T = T;
    a.V = V;
    a.dy_ld = dy_ld;
    a.D = D;
    a.slices = (int32_t)slices;
    a.accumulate = accumulate;
    a.scale = scale;
    const int64_t warps = chunks * slices;
    const int per = kGradThreads / 32;
    e = launch(k_embed_grad, dim3((unsigned)((warps + per - 1) / per)), kGradThreads, 0, 1, st, a);
    if (e == cudaSuccess && T > kChunk)
        e = launch(k_embed_join, dim3((unsigned)warps), kGradThreads, 0, 1, st, a);
    return status_of(e);
}
