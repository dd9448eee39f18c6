// lm_clip.cu - the 2-norm of gradients that lie in many tensors, and their
// clipping (declared in include/zero_step.h).
//
//   norms[i] = sqrt(sum of g^2 over tensor i),  norm = sqrt(sum of norms[i]^2)
//   out = g * (float)(max_norm / (norm + 1e-6)) where that is below 1
//
// The tensors are cut into tiles of 8192 elements, no tile over two tensors, and a
// block takes a run of consecutive tiles.  Going along the tiles either the block
// or the tensor steps on, so block + tensor is a slot of its own for every pair that
// meets, the slots of a tensor lie one behind the other, and no slot needs
// clearing.  A tensor's tiles begin at its first 16-byte boundary, so that the order of the
// additions depends on the addresses modulo 16 too.  The table of tensors goes into the launch's arguments: nothing is copied to the
// device, and a captured graph holds it.
//
// Bound by HBM: the norm reads every element once, the clipping once more and writes it, since
// the first output depends on the last input.  Measured, one GB300, 146 tensors of 1.24 G
// elements: the norm of bf16 ones 344 to 350 us (7.1 TB/s), norm and clipping of fp32 ones into
// bf16 1763 to 1778 us (7.0 TB/s of the 10 bytes).  37 tensors of 10^6 elements: 4.4 and 7.7 us,
// two and three launches.
#include "lm_common.cuh"

#include <cuda_fp16.h>
#include <math.h>

#include <new>

namespace {

using namespace lm;

constexpr int kThreads = 256;
// Elements of a tile, 4 vectors of a thread: with 2 vectors the norm of 1.24 G bf16 elements takes
// 443 us, with 1 573 (350 with 4), since a block waits for a tile before it asks for the next.
constexpr int kTile = 8192;
// The most blocks of a launch, for each of 152 SMs 4, which are resident at once, and 8.  The norm
// of 30 M bf16 elements takes 14.5 us in 4 and 16.3 in 8, norm and clipping of 1.24 G fp32 ones 1763
// us with 8 for the clipping and 1787 with 4.
constexpr int kNormBlocks = 608, kClipBlocks = 1216;
constexpr int kJoinThreads = 128;
// A head: input and output have no boundary together, and go an element at a time (2^30 elements, fp32
// into bf16 3.38 ms instead of 0.95, bf16 3.33 instead of 0.64).
constexpr int kNoVectors = 255;
constexpr int64_t kMaxNumel = 1ll << 40, kMaxTotal = 1ll << 43;

struct Entry {
    const void* p;
    void* out;
    int64_t numel;
    int32_t tile;                                    // the tensor's first tile
    uint8_t type, out_type;
    uint8_t head;                                    // elements before the first 16-byte vector
    uint8_t pad;
};

// Entries of a launch: 2, 8, 30 KB of arguments.  A few hundred launches of 30 KB fill the queue, and
// the host waits for the GPU (146 tensors: 6.5 us a call of the norm in 8 KB, 200 in 30, behind a long
// kernel).  Without one a call of 256 tensors takes the host 8.2 us and the GPU 5.2, of 290 10.5 and
// 5.1, of 960 19.9 and 9.2.
constexpr int kFew = 64, kSome = 256, kMany = 960;

template <int N>
struct ClipArgs {
    const float* norm_in;
    float* norm;
    float* norms;
    double* parts;
    double* total;
    int32_t* status;
    int64_t tiles;
    int32_t count, per_block;
    int32_t slots;                                   // that the blocks fill
    int32_t first, last;                             // of the call's launches
    int32_t in_place;
    int32_t last_full;                               // the last tensor that is not empty
    float max_norm;
    Entry e[N];
};

// The types' vectors of 8 elements, at multiples of 16 bytes, and single elements.
template <int TYPE>
struct Elem {
    using E = uint16_t;
    struct Raw {
        uint4 a;
    };
    static __device__ __forceinline__ Raw load8(const E* p) { return {ld16(p)}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[8])
    {
        if constexpr (TYPE == ZERO_TYPE_BF16) {
            bf_unpack8(r.a, f);
        } else {
            const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                f[2 * k] = x.x;
                f[2 * k + 1] = x.y;
            }
        }
    }
    static __device__ __forceinline__ void store8(E* p, const float (&f)[8])
    {
        if constexpr (TYPE == ZERO_TYPE_BF16) {
            st16_stream(p, bf_pack8(f));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            st16_stream(p, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
    static __device__ __forceinline__ float load1(const E* p)
    {
        if constexpr (TYPE == ZERO_TYPE_BF16) return __uint_as_float((uint32_t)*p << 16);
        else return __half2float(*reinterpret_cast<const __half*>(p));
    }
    static __device__ __forceinline__ void store1(E* p, float x)
    {
        if constexpr (TYPE == ZERO_TYPE_BF16) *p = (uint16_t)bf_pack(x, 0.0f);
        else *p = __half_as_ushort(__float2half_rn(x));
    }
};
template <>
struct Elem<ZERO_TYPE_FP32> {
    using E = float;
    struct Raw {
        uint4 a, b;
    };
    static __device__ __forceinline__ Raw load8(const E* p) { return {ld16(p), ld16(p + 4)}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[8])
    {
        f[0] = __uint_as_float(r.a.x); f[1] = __uint_as_float(r.a.y);
        f[2] = __uint_as_float(r.a.z); f[3] = __uint_as_float(r.a.w);
        f[4] = __uint_as_float(r.b.x); f[5] = __uint_as_float(r.b.y);
        f[6] = __uint_as_float(r.b.z); f[7] = __uint_as_float(r.b.w);
    }
    static __device__ __forceinline__ void store8(E* p, const float (&f)[8])
    {
        st16_stream(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                                  __float_as_uint(f[2]), __float_as_uint(f[3])));
        st16_stream(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                      __float_as_uint(f[6]), __float_as_uint(f[7])));
    }
    static __device__ __forceinline__ float load1(const E* p) { return *p; }
    static __device__ __forceinline__ void store1(E* p, float x) { *p = x; }
};

// A tile of a tensor: kTile elements from the first vector on, the tensor's first one with
// the elements before that too.
struct Place {
    int64_t start;                                   // of its vectors
    int n, before;                                   // elements from there on, and from 0 on
};
__device__ __forceinline__ Place place_of(int64_t numel, int head, int64_t tile)
{
    Place p;
    p.start = head + tile * kTile;
    p.n = (int)min(max(numel - p.start, (int64_t)0), (int64_t)kTile);
    p.before = tile ? 0 : (int)min((int64_t)head, numel);
    return p;
}

constexpr int kVecs = kTile / 8 / kThreads;          // vectors of a thread

// Calls f(x) for a thread's elements of a tile; all loads are asked for before the first
// call.
template <int TYPE, typename F>
__device__ __forceinline__ void for_elements(const void* base, int64_t numel, int head,
                                             int64_t tile, F&& f)
{
    using X = Elem<TYPE>;
    const Place at = place_of(numel, head, tile);
    const auto* first = static_cast<const typename X::E*>(base);
    const auto* p = first + at.start;
    const int nv = at.n >> 3, rest = at.n & 7, tid = threadIdx.x;
    typename X::Raw r[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        // (a register that only a predicated load sets stays taken through the loop over
        // the tiles, for every type's case at once)
        r[u] = {};
        if (tid + u * kThreads < nv) r[u] = X::load8(p + (tid + u * kThreads) * 8);
    }
    if (tid < rest) f(X::load1(p + nv * 8 + tid));
    if (tid < at.before) f(X::load1(first + tid));
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        if (tid + u * kThreads < nv) {
            float x[8];
            X::unpack(r[u], x);
#pragma unroll
            for (int q = 0; q < 8; ++q) f(x[q]);
        }
    }
}

__device__ __forceinline__ double warp_sum64(double x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// The sum over the block's threads, in every thread.
__device__ __forceinline__ float block_sum(float x)
{
    __shared__ float slots[kThreads / 32];
    x = warp_sum(x);
    __syncthreads();                                 // the slots may be in use still
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) x += slots[k];
    return x;
}

__device__ __forceinline__ uint32_t block_max(uint32_t x)
{
    __shared__ uint32_t slots[kThreads / 32];
    x = __reduce_max_sync(0xFFFFFFFFu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) m = max(m, slots[k]);
    return m;
}

// A thread's sum of squares over tiles [lo, hi) of a tensor, each value times s1 and s2 first
// (SCALED).  A tile's squares are added by themselves, and what the tiles' addition rounds away
// is kept beside it: a block may have thousands of tiles.
template <int TYPE, bool SCALED>
__device__ __forceinline__ float thread_squares(const void* p, int64_t numel, int head, int64_t lo,
                                                int64_t hi, float s1, float s2)
{
    float sum = 0.0f, rest = 0.0f;
#pragma unroll 1
    for (int64_t t = lo; t < hi; ++t) {
        float part = 0.0f;
        for_elements<TYPE>(p, numel, head, t, [&](float x) {
            if (SCALED) x = x * s1 * s2;
            part = fmaf(x, x, part);
        });
        const float next = sum + part, back = next - sum;
        rest += (sum - (next - back)) + (part - back);
        sum = next;
    }
    return sum + rest;
}

// The block's sum of squares where fp32 squares overflow or vanish: relative to the largest
// value's power of two.
template <int TYPE>
__device__ __noinline__ double scaled_sum(const void* p, int64_t numel, int head, int64_t lo,
                                          int64_t hi)
{
    uint32_t m = 0;
#pragma unroll 1
    for (int64_t t = lo; t < hi; ++t)
        for_elements<TYPE>(p, numel, head, t,
                           [&](float x) { m = max(m, __float_as_uint(x) & 0x7FFFFFFFu); });
    m = block_max(m);
    if (m == 0) return 0.0;
    const double top = (double)__uint_as_float(m);
    if (m >= 0x7F800000u) return top * top;
    int power;
    frexp(top, &power);
    // in two steps: 2^-power alone may be past fp32
    const float s1 = ldexpf(1.0f, -power / 2), s2 = ldexpf(1.0f, -power - -power / 2);
    return ldexp((double)block_sum(thread_squares<TYPE, true>(p, numel, head, lo, hi, s1, s2)),
                 2 * power);
}

template <int TYPE>
__device__ __forceinline__ double sum_squares(const void* p, int64_t numel, int head, int64_t lo,
                                              int64_t hi)
{
    const float s =
        block_sum(thread_squares<TYPE, false>(p, numel, head, lo, hi, 1.0f, 1.0f));
    // (each of the sum's terms was off by at most 2^-150: under 2^-24 of it from here up; a sum of 0
    // may be of zeros or of values whose squares vanish, so a run of zeros is read twice: 2^30 bf16
    // elements 309 us, 605 if all are 0, of fp32 594 and 1180)
    if (s >= 0x1p-80f && s <= 0x1p120f) return (double)s;
    return scaled_sum<TYPE>(p, numel, head, lo, hi);
}

// The tensor that holds a tile: the last whose first tile is at most that (empty
// tensors share theirs with the next one).
template <int N>
__device__ __forceinline__ int tensor_of(const ClipArgs<N>& a, int64_t tile)
{
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.e[mid].tile <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) k_grad_norm(const __grid_constant__ ClipArgs<N> a)
{
    pdl_enter();
    int64_t tile = (int64_t)blockIdx.x * a.per_block;
    const int64_t end = min(tile + a.per_block, a.tiles);
    int i = tensor_of(a, tile);
    // Slots that no pair has, beside empty tensors and where a block and a tensor end together,
    // become 0 by the block that comes after them: the sum of all slots is that of all tensors.
    int slot = blockIdx.x == 0 ? 0 : (int)blockIdx.x + tensor_of(a, tile - 1);
    while (tile < end) {
        const int64_t first = a.e[i].tile, numel = a.e[i].numel;
        const void* p = a.e[i].p;
        const int head = a.e[i].head, type = a.e[i].type;
        const int64_t stop = min(end, i + 1 < a.count ? (int64_t)a.e[i + 1].tile : a.tiles);
        const int64_t lo = tile - first, hi = stop - first;
        const double sum = type == ZERO_TYPE_BF16
                               ? sum_squares<ZERO_TYPE_BF16>(p, numel, head, lo, hi)
                           : type == ZERO_TYPE_FP16
                               ? sum_squares<ZERO_TYPE_FP16>(p, numel, head, lo, hi)
                               : sum_squares<ZERO_TYPE_FP32>(p, numel, head, lo, hi);
        if (threadIdx.x == 0) {
            for (; slot < (int)blockIdx.x + i; ++slot) a.parts[slot] = 0.0;
            a.parts[slot++] = sum;
        }
        tile = stop;
        while (i + 1 < a.count && a.e[i + 1].tile <= tile) ++i;
    }
}

// The root of a sum of squares, rounded to fp32.  A 64-bit root takes about 2 us here; the
// sum's fraction in [1, 4) rounded to fp32 is off by 2^-24 of itself, half of which is
// left in the root, beside the root's own rounding.
__device__ __forceinline__ float root(double s)
{
    if (!(s > 0.0) || s > 1.7e308) return (float)s;      // 0, Inf, NaN
    // (squares of fp32 values, the smallest 2^-298: no subnormal number)
    const int power = ((int)(__double2hiint(s) >> 20) - 1023) & ~1;
    const float f = (float)__hiloint2double(__double2hiint(s) - power * (1 << 20), __double2loint(s));
    return ldexpf(sqrtf(f), power / 2);
}

// The tensors' norms, a warp each, and by the last block that of all of them.
template <int N>
__global__ void __launch_bounds__(kJoinThreads) k_grad_norm_join(const __grid_constant__ ClipArgs<N> a)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x + 1 < gridDim.x) {
        const int i = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
        if (i >= a.count) return;
        const int from = a.e[i].tile, to = i + 1 < a.count ? a.e[i + 1].tile : (int)a.tiles;
        double s = 0.0;
        if (from < to) {
            const int first = from / a.per_block, last = (to - 1) / a.per_block;
#pragma unroll 4
            for (int b = first + lane; b <= last; b += 32) s += a.parts[b + i];
        }
        s = warp_sum64(s);
        if (lane == 0) a.norms[i] = root(s);
        return;
    }
    __shared__ double sums[kJoinThreads / 32];
    double s = 0.0;
#pragma unroll 4
    for (int k = threadIdx.x; k < a.slots; k += kJoinThreads) s += a.parts[k];
    s = warp_sum64(s);
    if (lane == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = a.first ? 0.0 : *a.total;
#pragma unroll
    for (int k = 0; k < kJoinThreads / 32; ++k) s += sums[k];
    if (!a.last) {
        *a.total = s;
        return;
    }
    const float norm = root(s);
    a.norm[0] = norm;
    if (a.status && !(norm <= 3.402823466e38f)) atomicOr(a.status, ZERO_DEV_NONFINITE);
}

// A tile of a tensor times coef.
template <int IN, int OUT>
__device__ __forceinline__ void clip_tile(const void* in, void* out, int64_t numel, int head,
                                          int64_t tile, float coef)
{
    using X = Elem<IN>;
    using Y = Elem<OUT>;
    const int tid = threadIdx.x;
    if (head == kNoVectors) {
        const auto* p = static_cast<const typename X::E*>(in);
        auto* o = static_cast<typename Y::E*>(out);
        const int64_t end = min((tile + 1) * kTile, numel);
        for (int64_t i = tile * kTile + tid; i < end; i += kThreads)
            Y::store1(o + i, X::load1(p + i) * coef);
        return;
    }
    const Place at = place_of(numel, head, tile);
    const auto* p0 = static_cast<const typename X::E*>(in);
    auto* o0 = static_cast<typename Y::E*>(out);
    const auto* p = p0 + at.start;
    auto* o = o0 + at.start;
    const int nv = at.n >> 3, rest = at.n & 7;
    typename X::Raw r[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        // (a register that only a predicated load sets stays taken through the loop over
        // the tiles, for every type's case at once)
        r[u] = {};
        if (tid + u * kThreads < nv) r[u] = X::load8(p + (tid + u * kThreads) * 8);
    }
    if (tid < rest) Y::store1(o + nv * 8 + tid, X::load1(p + nv * 8 + tid) * coef);
    if (tid < at.before) Y::store1(o0 + tid, X::load1(p0 + tid) * coef);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        if (tid + u * kThreads < nv) {
            float x[8];
            X::unpack(r[u], x);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] *= coef;
            Y::store8(o + (tid + u * kThreads) * 8, x);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) k_grad_clip(const __grid_constant__ ClipArgs<N> a)
{
    pdl_enter();
    // (one warp: the eight of a block take 64-bit operations in turn)
    __shared__ float the_coef;
    if (threadIdx.x < 32) {
        const double coef = (double)a.max_norm / ((double)*a.norm_in + 1e-6);
        the_coef = coef < 1.0 ? (float)coef : 1.0f;      // a norm that is NaN clips nothing
    }
    __syncthreads();
    const float coef = the_coef;
    if (coef == 1.0f && a.in_place) return;
    const int64_t begin = (int64_t)blockIdx.x * a.per_block;
    int64_t tile = min(begin + a.per_block, a.tiles) - 1;
    // backwards: the ends of the norm's blocks' runs are what it has read last
    int i = tensor_of(a, tile);
#pragma unroll 1
    for (; tile >= begin; --tile) {
        while (a.e[i].tile > tile) --i;
        const void* p = a.e[i].p;
        void* o = a.e[i].out;
        const int64_t numel = a.e[i].numel, t = tile - a.e[i].tile;
        const int head = a.e[i].head;
        switch (a.e[i].type * 4 + a.e[i].out_type) {
#define CLIP_CASE(in, out) \
    case in * 4 + out: clip_tile<in, out>(p, o, numel, head, t, coef); break
            CLIP_CASE(ZERO_TYPE_BF16, ZERO_TYPE_BF16);
            CLIP_CASE(ZERO_TYPE_FP16, ZERO_TYPE_FP16);
            CLIP_CASE(ZERO_TYPE_FP16, ZERO_TYPE_BF16);
            CLIP_CASE(ZERO_TYPE_FP32, ZERO_TYPE_FP32);
            CLIP_CASE(ZERO_TYPE_FP32, ZERO_TYPE_BF16);
#undef CLIP_CASE
        }
    }
}

int elem_bytes(int32_t type) { return type == ZERO_TYPE_FP32 ? 4 : 2; }

zero_status check_tensors(const zero_tensor* t, int32_t count)
{
    if (count < 0) return ZERO_ERR_INVALID_ARG;
    if (count > ZERO_MAX_TENSORS) return ZERO_ERR_SIZE;
    if (count == 0) return ZERO_OK;
    if (!t) return ZERO_ERR_NULL;
    int64_t total = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (t[i].numel < 0 || t[i].type < ZERO_TYPE_BF16 || t[i].type > ZERO_TYPE_FP32)
            return ZERO_ERR_INVALID_ARG;
        if (t[i].numel > kMaxNumel || (total += t[i].numel) > kMaxTotal) return ZERO_ERR_SIZE;
        if (t[i].numel > 0) LM_CHECK(check_ptr(t[i].data, (unsigned)elem_bytes(t[i].type)));
    }
    return ZERO_OK;
}

Span span_of(const zero_tensor& t, bool out)
{
    const uintptr_t lo = (uintptr_t)t.data;
    return Span{lo, lo + (uintptr_t)(t.numel * elem_bytes(t.type)), out};
}

// Whether a buffer overlaps one of the tensors.
bool meets(const zero_tensor* t, int32_t count, const void* p, int64_t bytes)
{
    const uintptr_t lo = (uintptr_t)p, hi = lo + (uintptr_t)bytes;
    for (int32_t i = 0; i < count; ++i) {
        const Span s = span_of(t[i], false);
        if (s.lo < s.hi && s.lo < hi && lo < s.hi) return true;
    }
    return false;
}

// Outputs may overlap nothing.  In ascending order, as views of flat buffers come, one
// look at each does; else they are sorted first.
zero_status check_overlaps(const zero_tensor* in, const zero_tensor* out, int32_t count)
{
    Span* s = new (std::nothrow) Span[2 * (size_t)count];
    if (!s) return ZERO_ERR_SIZE;
    int64_t n = 0;
    bool sorted = true;
    auto take = [&](const zero_tensor* t, bool is_out) {
        for (int32_t i = 0; i < count; ++i) {
            if (t[i].numel == 0) continue;
            s[n] = span_of(t[i], is_out);
            if (n && s[n].lo < s[n - 1].lo) sorted = false;
            ++n;
        }
    };
    if (out) take(in, false);
    take(out ? out : in, true);
    if (!sorted) std::sort(s, s + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t any = 0, outs = 0;                     // how far what came before reaches
    zero_status r = ZERO_OK;
    for (int64_t i = 0; i < n && r == ZERO_OK; ++i) {
        if (s[i].lo < (s[i].out ? any : outs)) r = ZERO_ERR_OVERLAP;
        any = std::max(any, s[i].hi);
        if (s[i].out) outs = std::max(outs, s[i].hi);
    }
    delete[] s;
    return r;
}

// The elements before the first place where both tensors have a 16-byte vector.
uint8_t head_of(const zero_tensor& t, const zero_tensor* out)
{
    for (int h = 0; h < 8; ++h) {
        if (!aligned(static_cast<const char*>(t.data) + h * elem_bytes(t.type), 16)) continue;
        if (!out || aligned(static_cast<const char*>(out->data) + h * elem_bytes(out->type), 16))
            return (uint8_t)h;
    }
    return kNoVectors;
}

int64_t slots(int64_t count)
{
    return count + ((count + kMany - 1) / kMany) * kNormBlocks;
}

// The launches of a call, each with at most N tensors in `most` blocks: f(args, blocks, first
// tensor).
template <int N, typename F>
cudaError_t for_launches(const zero_tensor* t, const zero_tensor* outs, int32_t count, int most,
                         F&& f)
{
    ClipArgs<N> a;
    for (int32_t at = 0; at < count; at += N) {
        a.count = std::min(count - at, N);
        a.tiles = 0;
        a.last_full = 0;
        for (int32_t i = 0; i < a.count; ++i) {
            const zero_tensor& x = t[at + i];
            Entry& e = a.e[i];
            e.p = x.data;
            e.out = outs ? outs[at + i].data : x.data;
            e.numel = x.numel;
            e.tile = (int32_t)a.tiles;
            e.type = (uint8_t)x.type;
            e.out_type = (uint8_t)(outs ? outs[at + i].type : x.type);
            e.head = x.numel ? head_of(x, outs ? &outs[at + i] : nullptr) : 0;
            e.pad = 0;
            const int64_t before = e.head == kNoVectors ? 0 : e.head;
            if (x.numel) a.last_full = i;
            if (x.numel) a.tiles += std::max<int64_t>(1, (x.numel - before + kTile - 1) / kTile);
        }
        a.per_block = (int32_t)std::max<int64_t>(1, (a.tiles + most - 1) / most);
        const unsigned blocks = (unsigned)((a.tiles + a.per_block - 1) / a.per_block);
        if (cudaError_t e = f(a, blocks, at)) return e;
    }
    return cudaSuccess;
}

template <int N>
cudaError_t norm_launches(const zero_tensor* t, int32_t count, float* norm, float* norms,
                          double* scratch, int32_t* status, cudaStream_t st)
{
    return for_launches<N>(t, nullptr, count, kNormBlocks, [&](ClipArgs<N>& a, unsigned blocks, int32_t at) {
        a.norm = norm;
        a.norms = norms ? norms + at : nullptr;
        a.total = scratch;
        a.parts = scratch + 2 + at + (int64_t)(at / N) * kNormBlocks;
        a.status = status;
        a.first = at == 0;
        a.last = at + N >= count;
        cudaError_t e = cudaSuccess;
        // (what ends with empty tensors leaves their slots to nobody: they are not summed)
        a.slots = blocks ? (int32_t)blocks + a.last_full : 0;
        const unsigned join = norms ? (unsigned)((a.count + kJoinThreads / 32 - 1) / (kJoinThreads / 32)) : 0;
        if (blocks) e = launch(k_grad_norm<N>, dim3(blocks), kThreads, 0, st, a);
        if (e == cudaSuccess)
            e = launch(k_grad_norm_join<N>, dim3(join + 1), kJoinThreads, 0, st, a);
        return e;
    });
}

template <int N>
cudaError_t clip_launches(const zero_tensor* t, const zero_tensor* outs, int32_t count,
                          const float* norm, float max_norm, cudaStream_t st)
{
    return for_launches<N>(t, outs, count, kClipBlocks, [&](ClipArgs<N>& a, unsigned blocks, int32_t) {
        a.norm_in = norm;
        a.max_norm = max_norm;
        a.in_place = outs == nullptr;
        return blocks ? launch(k_grad_clip<N>, dim3(blocks), kThreads, 0, st, a) : cudaSuccess;
    });
}

}  // namespace

extern "C" int64_t zero_grad_norm_scratch_bytes(int32_t count)
{
    if (count < 0 || count > ZERO_MAX_TENSORS) return -1;
    return up(8 * (2 + slots(count)), 256);
}

extern "C" zero_status zero_grad_norm(const zero_tensor* tensors, int32_t count, float* norm,
                                      float* norms, void* scratch, int64_t scratch_bytes,
                                      int32_t* dev_status, void* stream)
{
    LM_CHECK(check_tensors(tensors, count));
    LM_CHECK(check_status(dev_status));
    LM_CHECK(check_ptr(norm, 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (count == 0) return status_of(cudaMemsetAsync(norm, 0, 4, st));
    if (norms) LM_CHECK(check_ptr(norms, 4));
    LM_CHECK(check_ptr(scratch));
    const int64_t need = zero_grad_norm_scratch_bytes(count);
    if (scratch_bytes < need) return ZERO_ERR_SIZE;
    Spans sp;
    sp.add(norm, 4, true);
    sp.add(norms, 4 * (int64_t)count, true);
    sp.add(scratch, need, true);
    sp.add(dev_status, 4, true);
    LM_CHECK(sp.check());
    for (int i = 0; i < sp.n; ++i)
        if (meets(tensors, count, (const void*)sp.s[i].lo, (int64_t)(sp.s[i].hi - sp.s[i].lo)))
            return ZERO_ERR_OVERLAP;
    double* s = static_cast<double*>(scratch);
    return status_of(count <= kFew
                         ? norm_launches<kFew>(tensors, count, norm, norms, s, dev_status, st)
                     : count <= kSome
                         ? norm_launches<kSome>(tensors, count, norm, norms, s, dev_status, st)
                         : norm_launches<kMany>(tensors, count, norm, norms, s, dev_status, st));
}

extern "C" zero_status zero_grad_clip(const zero_tensor* tensors, const zero_tensor* outs,
                                      int32_t count, const float* norm, float max_norm,
                                      void* stream)
{
    LM_CHECK(check_tensors(tensors, count));
    if (outs) {
        LM_CHECK(check_tensors(outs, count));
        for (int32_t i = 0; i < count; ++i)
            if (outs[i].numel != tensors[i].numel ||
                (outs[i].type != tensors[i].type && outs[i].type != ZERO_TYPE_BF16))
                return ZERO_ERR_INVALID_ARG;
    }
    if (!(max_norm > 0.0f) || max_norm > 3.402823466e38f) return ZERO_ERR_INVALID_ARG;
    if (count == 0) return ZERO_OK;
    LM_CHECK(check_ptr(norm, 4));
    LM_CHECK(check_overlaps(tensors, outs, count));
    if (meets(outs ? outs : tensors, count, norm, 4)) return ZERO_ERR_OVERLAP;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return status_of(count <= kFew
                         ? clip_launches<kFew>(tensors, outs, count, norm, max_norm, st)
                     : count <= kSome
                         ? clip_launches<kSome>(tensors, outs, count, norm, max_norm, st)
                         : clip_launches<kMany>(tensors, outs, count, norm, max_norm, st));
}
