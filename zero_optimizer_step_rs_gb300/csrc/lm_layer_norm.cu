// lm_layer_norm.cu - layer norm of (activation + residual) and its gradients
// (declared in include/zero_step.h).
//
//   s = x + r (fp32; the new residual stream is bf16(s)),  mean = mean(s)
//   rstd = 1 / sqrt(mean((s - mean)^2) + eps),   y = bf16((s - mean) * rstd * w + b)
// and, with xhat = (s - mean) * rstd and u = dy * w:
//   dx = bf16(rstd * (u - mean(u) - xhat * mean(u * xhat)) + dsum)
//   dw = sum_t dy * xhat,  db = sum_t dy
//
// Bound by HBM traffic: forward 2+2 bytes an element read and 2+2 written, gradient
// 2+2+2 read and 2 written.  Measured, one GB300, 32768 x 2048: forward 79 us (6.8 TB/s, the
// rate of a copy), gradient 80 us (6.7 TB/s, 3 of them the join of dw and db).  333 x 768: 2.4 us
// and 4.2 us, one launch and two.
#include "lm_common.cuh"

namespace {

using namespace lm;

struct LayerNormArgs {
    const uint16_t* x;
    const uint16_t* res;             // may be null
    const uint16_t* w;               // may be null: ones
    const uint16_t* b;               // may be null: zeros
    uint16_t* y;
    uint16_t* sum;                   // may be null
    float* mean;
    float* rstd;
    int64_t T, x_ld, res_ld, y_ld, sum_ld;
    int32_t D;
    float eps;
};

constexpr uint32_t kOnes = 0x3F803F80u;              // two bf16 ones

// How a row's vectors of 8 elements are spread over threads, NV to each.  SUB = 8, 16 or
// 32: over so many lanes of a warp, and a block of 128 threads has 128 / SUB rows.  SUB = 0:
// over the whole block, whose size is the row's number of vectors / NV in whole warps, so that
// few threads have nothing: with sizes in powers of two rows of 2056 columns ran at 4.0 TB/s and
// rows of 64 at 2.0.
template <int SUB>
struct Spread {
    static constexpr int kRows = SUB ? 128 / SUB : 1;            // of a block
    static __device__ __forceinline__ int threads() { return SUB ? SUB : (int)blockDim.x; }
    static __device__ __forceinline__ int row() { return SUB ? (int)threadIdx.x / SUB : 0; }
    static __device__ __forceinline__ int lane()
    {
        return SUB ? (int)threadIdx.x % SUB : (int)threadIdx.x;
    }
};

// The sum over the lanes of a row that lie in one warp.
template <int SUB>
__device__ __forceinline__ float lane_sum(float x)
{
#pragma unroll
    for (int o = (SUB ? SUB : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// The row stays in registers.  The lanes of a warp take the mean of their own elements and
// their squared distances from it, and the warps' pairs are joined by
//   mean = sum of sums / D,  M2 = sum of (M2_w + n_w (mean_w - mean)^2),
// which cancels nothing and needs one barrier where two passes over the row would
// need two.
template <int SUB, int NV>
__global__ void __launch_bounds__(SUB ? 128 : 512)
    k_layer_norm(const __grid_constant__ LayerNormArgs a)
{
    using S = Spread<SUB>;
    pdl_enter();
    const int64_t t = (int64_t)blockIdx.x * S::kRows + S::row();
    const int lane = S::lane(), step = S::threads();
    const int nv = t < a.T ? a.D >> 3 : 0;                 // a row past the last has no vectors
    const uint16_t* x = a.x + t * a.x_ld;
    const uint16_t* r = a.res ? a.res + t * a.res_ld : nullptr;

    float f[NV][8];
    {
        uint4 v[NV], u[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = lane + k * step;
            v[k] = u[k] = make_uint4(0, 0, 0, 0);
            if (c < nv) {
                v[k] = ld16_stream(x + c * 8);
                if (r) u[k] = ld16_stream(r + c * 8);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float g[8];
            bf_unpack8(v[k], f[k]);
            bf_unpack8(u[k], g);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[k][q] += g[q];
        }
    }
    // elements of the row that these lanes hold
    int held = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        held += min(max(nv - (SUB ? 0 : lane & ~31) - k * step, 0), SUB ? SUB : 32) * 8;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) s += f[k][q];
    s = lane_sum<SUB>(s);
    float mean = held ? s / (float)held : 0.0f, m2 = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * step < nv)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float d = f[k][q] - mean;
                m2 = fmaf(d, d, m2);
            }
    m2 = lane_sum<SUB>(m2);
    if constexpr (SUB == 0) {
        __shared__ float4 parts[16];
        const int warps = step >> 5;
        if ((threadIdx.x & 31) == 0)
            parts[threadIdx.x >> 5] = make_float4(s, mean, m2, (float)held);
        __syncthreads();
        float total = 0.0f;
        for (int k = 0; k < warps; ++k) total += parts[k].x;
        mean = total / (float)a.D;
        m2 = 0.0f;
        for (int k = 0; k < warps; ++k) {
            const float4 p = parts[k];
            const float d = p.y - mean;
            m2 += fmaf(p.w * d, d, p.z);
        }
    }
    const float rstd = 1.0f / sqrtf(m2 / (float)a.D + a.eps);
    if (lane == 0 && nv) {
        a.mean[t] = mean;
        a.rstd[t] = rstd;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = lane + k * step;
        if (c < nv) {
            if (a.sum) st16_stream(a.sum + t * a.sum_ld + c * 8, bf_pack8(f[k]));
            float w[8], b[8];
            bf_unpack8(a.w ? ld16(a.w + c * 8) : make_uint4(kOnes, kOnes, kOnes, kOnes), w);
            bf_unpack8(a.b ? ld16(a.b + c * 8) : make_uint4(0, 0, 0, 0), b);
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = fmaf((f[k][q] - mean) * rstd, w[q], b[q]);
            st16_stream(a.y + t * a.y_ld + c * 8, bf_pack8(w));
        }
    }
}

// -------------------------------------------------------------- gradient --

struct LayerNormGradArgs {
    const uint16_t* dy;
    const uint16_t* dsum;            // may be null
    const uint16_t* x;
    const float* mean;
    const float* rstd;
    const uint16_t* w;               // may be null: ones
    uint16_t* dx;
    uint16_t* dw;                    // may be null
    uint16_t* db;                    // may be null
    float* parts;                    // [blocks][2][D]; null: neither is wanted
    int64_t T, dy_ld, dsum_ld, x_ld, dx_ld;
    int32_t D, blocks;
    int32_t apart, groups;           // SUB = 0: threads of a row, rows of a block at a time,
    int32_t near;                    // and whether these lie one behind the other
};

// The sums of two values over the threads of a row: a warp's lanes or less, or the `warps` warps
// of a group, whose first is warp `base` of the block and which has a barrier of its own.  `slot`
// alternates from row to row, so that one barrier a row is enough.
template <int SUB>
__device__ __forceinline__ float2 row_sums(float x, float y, float2 (*slots)[32], int slot, int group,
                                           int base, int warps)
{
    x = lane_sum<SUB>(x);
    y = lane_sum<SUB>(y);
    if constexpr (SUB == 0) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) slots[slot][threadIdx.x >> 5] = make_float2(x, y);
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
        if (warps > 8) {
            const float2 p = lane < warps ? slots[slot][base + lane] : make_float2(0.0f, 0.0f);
            x = warp_sum(p.x);
            y = warp_sum(p.y);
        } else {
            x = y = 0.0f;
            for (int k = 0; k < warps; ++k) {
                const float2 p = slots[slot][base + k];
                x += p.x;
                y += p.y;
            }
        }
    }
    return make_float2(x, y);
}

// A copy of 16 bytes from global memory into the thread's own place in shared memory,
// which only that thread reads: no barrier, only its own wait.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Two fp32 values in one register pair, which add, multiply and fma take in one instruction
// (each value rounded by itself).  The gradient's rows filled 56 % of the issue slots without, and
// rows that leave lanes without a vector more: in blocks of one row 32768 x 2048 took 84 us with
// pairs and 89 without, 30000 x 2056 90 and 97.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float lo, float hi)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ Two both(float x) { return two(x, x); }
__device__ __forceinline__ float2 apart2(Two x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ Two add2(Two x, Two y)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ Two mul2(Two x, Two y)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ Two fma2(Two x, Two y, Two z)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ void bf_unpack_twos(const uint4& x, Two (&f)[4])
{
    f[0] = two(bf_lo(x.x), bf_hi(x.x));
    f[1] = two(bf_lo(x.y), bf_hi(x.y));
    f[2] = two(bf_lo(x.z), bf_hi(x.z));
    f[3] = two(bf_lo(x.w), bf_hi(x.w));
}

// Rows that a thread has asked for ahead of the one it works on, plus that one.
__host__ __device__ constexpr int grad_stages(int most) { return most <= 512 ? 3 : 2; }
constexpr int kMostSmem = 225 * 1024;                // of a block, beside its static part

// Blocks that an SM is to hold: they set the registers.  One vector a thread runs best with
// many warps, 2 in 128 registers and 3 or 4 in 168.
constexpr int grad_blocks_min(int sub, int nv, int most)
{
    if (sub) return nv == 1 ? 7 : nv == 2 ? 4 : 3;
    return 1;
}

// A row's threads walk over many rows and keep the sums of dw and db in
// registers; a block's row groups are added in order at its end.  The rows ahead wait in
// shared memory, where a thread finds its own vectors: with a barrier in the middle of each
// row a block would otherwise have nothing in flight for half of the time.
template <int SUB, int NV, int MOST>
__global__ void __launch_bounds__(SUB ? 128 : MOST, grad_blocks_min(SUB, NV, MOST))
    k_layer_norm_grad(const __grid_constant__ LayerNormGradArgs a)
{
    using W = Spread<SUB>;
    constexpr int S = grad_stages(MOST);
    constexpr bool KEEP = (NV == 2 || NV == 3) && MOST <= 512;
    const int threads = SUB ? 128 : (int)blockDim.x;
    const int N = NV * threads * 16, STAGE = 3 * N;          // a stage: dy, x, dsum
    pdl_enter();
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 slots[2][32];
    // `apart`: between a thread's vectors
    const int apart = SUB ? SUB : a.apart, groups = SUB ? W::kRows : a.groups;
    const int group = threadIdx.x / apart, lane = threadIdx.x % apart;
    const int nv = a.D >> 3;
    const int64_t step = (int64_t)gridDim.x * groups;
    const int64_t first = SUB || a.near ? (int64_t)blockIdx.x * groups + group
                                        : blockIdx.x + (int64_t)group * gridDim.x;
    const float inv = 1.0f / (float)a.D;

    // where the row to ask for next lies; a thread past the row's end asks for
    // nothing and keeps the zeros that its places start with
    const uint16_t* p_d = a.dy + first * a.dy_ld + lane * 8;
    const uint16_t* p_x = a.x + first * a.x_ld + lane * 8;
    const uint16_t* p_s = a.dsum ? a.dsum + first * a.dsum_ld + lane * 8 : nullptr;
    const int64_t d_step = step * a.dy_ld, x_step = step * a.x_ld, s_step = step * a.dsum_ld;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    auto ask = [&](bool in, uint32_t stage) {
        if (in) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (lane + k * apart >= nv) break;
                const uint32_t at = mine + stage + k * threads * 16;
                copy_async(at, p_d + k * apart * 8);
                copy_async(at + N, p_x + k * apart * 8);
                if (p_s) copy_async(at + 2 * N, p_s + k * apart * 8);
            }
        }
        p_d += d_step;
        p_x += x_step;
        if (p_s) p_s += s_step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * apart >= nv)
#pragma unroll
            for (int i = 0; i < 3 * S; ++i)
                st16(ring + i * N + (k * threads + threadIdx.x) * 16, make_uint4(0, 0, 0, 0));

    uint4 w4[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        w4[k] = make_uint4(kOnes, kOnes, kOnes, kOnes);
        if (a.w && lane + k * apart < nv) w4[k] = ld16(a.w + (lane + k * apart) * 8);
    }
    Two dw[NV][4] = {}, db[NV][4] = {};
    uint32_t stage = 0;                                   // offset of the row at hand
    int slot = 0;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) ask(first + s * step < a.T, s * STAGE);
    float mean_next = 0.0f, rstd_next = 0.0f;
    if (first < a.T) {
        mean_next = a.mean[first];
        rstd_next = a.rstd[first];
    }
    uint16_t* p_o = a.dx + first * a.dx_ld + lane * 8;
    // (the groups that share a warp go on while one of the block's has a row: the sums take whole
    // warps)
    int64_t t = first;
    for (int64_t top = SUB && SUB < 32 ? (int64_t)blockIdx.x * groups : first; top < a.T;
         top += step, t += step, p_o += step * a.dx_ld) {
        const bool in = !(SUB && SUB < 32) || t < a.T;
        const float mean = mean_next, rstd = rstd_next;
        if (t + step < a.T) {
            mean_next = a.mean[t + step];
            rstd_next = a.rstd[t + step];
        }
        ask(t + (S - 1) * step < a.T,
            stage == 0 ? (S - 1) * STAGE : stage - STAGE);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        // xhat and dy * w are kept for the row's second part where the registers allow it, else
        // made again from what shared memory holds (30000 x 2056: 84 us kept, 90 made again; 64 and
        // 1024 columns: 91 and 103 kept, 82 and 76 made again)
        const uint32_t here = mine + stage;
        const Two less = both(-mean), scale = both(rstd);
        Two s1 = 0, s2 = 0, kept_u[KEEP ? NV : 1][4], kept_x[KEEP ? NV : 1][4];
        if (in)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                Two w[4], x[4], d[4];
                // (past the row's end xhat is 0 too: -mean * rstd may be past fp32's range)
                const Two here_scale = lane + k * apart < nv ? scale : 0;
                bf_unpack_twos(w4[k], w);
                bf_unpack_twos(ld_shared(here + k * threads * 16), d);
                bf_unpack_twos(ld_shared(here + k * threads * 16 + N), x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const Two xh = mul2(add2(x[q], less), here_scale), u = mul2(d[q], w[q]);
                    if constexpr (KEEP) {
                        kept_u[k][q] = u;
                        kept_x[k][q] = xh;
                    }
                    db[k][q] = add2(db[k][q], d[q]);
                    dw[k][q] = fma2(d[q], xh, dw[k][q]);
                    s1 = add2(s1, u);
                    s2 = fma2(u, xh, s2);
                }
            }
        const float2 p1 = apart2(s1), p2 = apart2(s2);
        const float2 all = row_sums<SUB>(p1.x + p1.y, p2.x + p2.y, slots, slot, group,
                                        group * (apart >> 5), apart >> 5);
        slot ^= 1;
        const Two c1 = both(-all.x * inv), c2 = both(-all.y * inv);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!in || lane + k * apart >= nv) break;
            Two s[4] = {}, xh[4], v[4];                     // v: u - mean(u)
            if constexpr (KEEP) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    xh[q] = kept_x[k][q];
                    v[q] = add2(kept_u[k][q], c1);
                }
            } else {
                Two w[4], x[4], d[4];
                bf_unpack_twos(w4[k], w);
                bf_unpack_twos(ld_shared(here + k * threads * 16), d);
                bf_unpack_twos(ld_shared(here + k * threads * 16 + N), x);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    xh[q] = mul2(add2(x[q], less), scale);
                    v[q] = fma2(d[q], w[q], c1);
                }
            }
            if (p_s) bf_unpack_twos(ld_shared(here + k * threads * 16 + 2 * N), s);
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 r = apart2(fma2(scale, fma2(xh[q], c2, v[q]), s[q]));
                o[q] = bf_pack(r.x, r.y);
            }
            st16_stream(p_o + k * apart * 8, make_uint4(o[0], o[1], o[2], o[3]));
        }
        stage = stage == (S - 1) * STAGE ? 0 : stage + STAGE;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.parts) return;
    float* part = a.parts + (int64_t)blockIdx.x * 2 * a.D;
    // the groups' sums, in order (the ring is free once every thread's copies have landed)
    float* all = reinterpret_cast<float*>(ring);              // [groups][width]
    const int width = apart * NV * 8;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<float2*>(all + group * width + (lane + k * apart) * 8 + 2 * q) =
                    apart2(side ? db[k][q] : dw[k][q]);
        __syncthreads();
        for (int i = threadIdx.x * 4; i < a.D; i += threads * 4) {
            float4 sum = *reinterpret_cast<const float4*>(all + i);
            for (int g = 1; g < groups; ++g) {
                const float4 y = *reinterpret_cast<const float4*>(all + g * width + i);
                sum.x += y.x; sum.y += y.y; sum.z += y.z; sum.w += y.w;
            }
            *reinterpret_cast<float4*>(part + side * a.D + i) = sum;
        }
    }
}

// dw and db = the blocks' parts, added in an order that depends on their number only (so T, D and
// the GPU's number of SMs decide the order of all additions):
// 32 of the 2 D columns a block, 128 shares of the rows; four shares lie in a warp's
// lanes, the 32 warps' sums are added by the first one.
constexpr int kJoinThreads = 1024;
constexpr int kJoinCols = 32;
constexpr int kJoinShares = kJoinThreads / (kJoinCols / 4);

__device__ __forceinline__ float4 add4(const float4& p, const float4& q)
{
    return make_float4(p.x + q.x, p.y + q.y, p.z + q.z, p.w + q.w);
}
// Over the lanes that have the same columns.
__device__ __forceinline__ float4 share_sum(float4 s)
{
#pragma unroll
    for (int o = 8; o < 32; o <<= 1)
        s = add4(s, make_float4(__shfl_xor_sync(0xFFFFFFFFu, s.x, o),
                                __shfl_xor_sync(0xFFFFFFFFu, s.y, o),
                                __shfl_xor_sync(0xFFFFFFFFu, s.z, o),
                                __shfl_xor_sync(0xFFFFFFFFu, s.w, o)));
    return s;
}

__global__ void __launch_bounds__(kJoinThreads)
    k_layer_norm_join(const __grid_constant__ LayerNormGradArgs a)
{
    pdl_enter();
    __shared__ float4 sums[kJoinThreads / 32][kJoinCols / 4];
    const int cv = threadIdx.x % (kJoinCols / 4), sh = threadIdx.x / (kJoinCols / 4);
    const int col = blockIdx.x * kJoinCols + cv * 4;
    float4 s = make_float4(0, 0, 0, 0);
    if (col < 2 * a.D)
#pragma unroll 4
        for (int r = sh; r < a.blocks; r += kJoinShares)
            s = add4(s, __ldcs(reinterpret_cast<const float4*>(a.parts + (int64_t)r * 2 * a.D + col)));
    s = share_sum(s);
    if ((threadIdx.x & 31) < kJoinCols / 4) sums[threadIdx.x >> 5][cv] = s;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    s = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) s = add4(s, sums[sh * 8 + k][cv]);
    s = share_sum(s);
    if (sh == 0 && col < 2 * a.D) {
        uint16_t* to = col < a.D ? a.dw : a.db;            // 4 columns never straddle the two
        if (to)
            *reinterpret_cast<uint2*>(to + (col < a.D ? col : col - a.D)) =
                make_uint2(bf_pack(s.x, s.y), bf_pack(s.z, s.w));
    }
}

// Blocks of a form of k_layer_norm_grad that fit on an SM, by their number of warps and per
// device (0: not asked yet).
template <int SUB, int NV, int MOST>
std::atomic<int> grad_per_sm[64][33];

// The most blocks that k_layer_norm_grad takes.
int grad_blocks(int64_t T) { return (int)std::min<int64_t>(T, 1216); }

}  // namespace

// The warps that a row of D columns needs with NV vectors a thread.
static int warps_of(int32_t D, int nv) { return (D / 8 + 32 * nv - 1) / (32 * nv); }

extern "C" zero_status zero_layer_norm(const uint16_t* x, int64_t x_ld, const uint16_t* residual,
                                       int64_t residual_ld, const uint16_t* weight,
                                       const uint16_t* bias, int64_t T, int32_t D, float eps,
                                       uint16_t* y, int64_t y_ld, uint16_t* sum, int64_t sum_ld,
                                       float* mean, float* rstd, void* stream)
{
    LM_CHECK(check_sizes(T, 1, D, ZERO_NORM_MAX_WIDTH));
    LM_CHECK(check_ld(x_ld, D));
    LM_CHECK(check_ld(y_ld, D));
    if (residual) LM_CHECK(check_ld(residual_ld, D));
    if (sum) LM_CHECK(check_ld(sum_ld, D));
    if (!(eps >= 0.0f) || eps > 3.0e38f) return ZERO_ERR_INVALID_ARG;
    if (T == 0) return ZERO_OK;
    LM_CHECK(check_ptr(x));
    if (residual) LM_CHECK(check_ptr(residual));
    if (weight) LM_CHECK(check_ptr(weight));
    if (bias) LM_CHECK(check_ptr(bias));
    LM_CHECK(check_ptr(y));
    if (sum) LM_CHECK(check_ptr(sum));
    LM_CHECK(check_ptr(mean, 4));
    LM_CHECK(check_ptr(rstd, 4));
    Spans sp;
    sp.rows(x, T, x_ld, D, 2, false);
    if (residual) sp.rows(residual, T, residual_ld, D, 2, false);
    sp.add(weight, 2 * D, false);
    sp.add(bias, 2 * D, false);
    sp.rows(y, T, y_ld, D, 2, true);
    if (sum) sp.rows(sum, T, sum_ld, D, 2, true);
    sp.add(mean, 4 * T, true);
    sp.add(rstd, 4 * T, true);
    LM_CHECK(sp.check());

    LayerNormArgs a{};
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.sum = sum;
    a.mean = mean;
    a.rstd = rstd;
    a.T = T;
    a.x_ld = x_ld;
    a.res_ld = residual_ld;
    a.y_ld = y_ld;
    a.sum_ld = sum_ld;
    a.D = D;
    a.eps = eps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Up to 1024 columns a row is one warp's or less, with lanes that hold as many vectors as leave
    // few without one: 500000 x 128 takes 75 us in 8 lanes and 81 in 16, 200000 x 256 60 in 16 and 65
    // in 32, 80000 x 768 72 in a warp and 98 in four.  Wider rows get as many warps as their vectors
    // fill, with 3 or 4 vectors a thread: 8000 x 8192 77 us with 4, 83 with 3 and 98 with 2; 30000 x
    // 2056 74 with 3, 80 with 4 and 85 with 2.  Rows that do not fill the SMs take more threads each:
    // 333 x 768 2.4 us with a vector a thread, 2.7 in a warp.
#define LAYER_NORM_GO(sub, nv)                                                                  \
    status_of(launch(k_layer_norm<sub, nv>,                                                     \
                     dim3((unsigned)((T + Spread<sub>::kRows - 1) / Spread<sub>::kRows)),       \
                     sub ? 128 : 32 * warps_of(D, nv), 0, st, a))
    if (T <= 1216 && D > 256 && D <= 4096) return LAYER_NORM_GO(0, 1);
    if (D <= 64) return LAYER_NORM_GO(8, 1);
    if (D <= 128) return LAYER_NORM_GO(8, 2);
    if (D <= 192) return LAYER_NORM_GO(8, 3);
    if (D <= 256) return LAYER_NORM_GO(16, 2);
    if (D <= 384) return LAYER_NORM_GO(16, 3);
    if (D <= 512) return LAYER_NORM_GO(32, 2);
    if (D <= 768) return LAYER_NORM_GO(32, 3);
    if (D <= 1024) return LAYER_NORM_GO(32, 4);
    if (D <= 12288 && 3 * warps_of(D, 3) < 4 * warps_of(D, 4)) return LAYER_NORM_GO(0, 3);
    return LAYER_NORM_GO(0, 4);
#undef LAYER_NORM_GO
}

extern "C" int64_t zero_layer_norm_grad_scratch_bytes(int64_t T, int32_t D)
{
    if (check_sizes(T, 1, D, ZERO_NORM_MAX_WIDTH) != ZERO_OK) return -1;
    return up(8 * (int64_t)grad_blocks(T) * D, 256);
}

extern "C" zero_status zero_layer_norm_grad(const uint16_t* dy, int64_t dy_ld,
                                            const uint16_t* dsum, int64_t dsum_ld,
                                            const uint16_t* x, int64_t x_ld, const float* mean,
                                            const float* rstd, const uint16_t* weight, int64_t T,
                                            int32_t D, uint16_t* dx, int64_t dx_ld,
                                            uint16_t* dweight, uint16_t* dbias, void* scratch,
                                            int64_t scratch_bytes, void* stream)
{
    LM_CHECK(check_sizes(T, 1, D, ZERO_NORM_MAX_WIDTH));
    LM_CHECK(check_ld(dy_ld, D));
    LM_CHECK(check_ld(x_ld, D));
    LM_CHECK(check_ld(dx_ld, D));
    if (dsum) LM_CHECK(check_ld(dsum_ld, D));
    if (dweight) LM_CHECK(check_ptr(dweight));
    if (dbias) LM_CHECK(check_ptr(dbias));
    const bool wanted = dweight || dbias;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Spans sp;
    sp.add(dweight, 2 * D, true);
    sp.add(dbias, 2 * D, true);
    if (T == 0) {
        LM_CHECK(sp.check());
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)(2 * D), st);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)(2 * D), st);
        return status_of(e);
    }
    LM_CHECK(check_ptr(dy));
    if (dsum) LM_CHECK(check_ptr(dsum));
    LM_CHECK(check_ptr(x));
    LM_CHECK(check_ptr(mean, 4));
    LM_CHECK(check_ptr(rstd, 4));
    if (weight) LM_CHECK(check_ptr(weight));
    LM_CHECK(check_ptr(dx));
    if (wanted) {
        LM_CHECK(check_ptr(scratch));
        const int64_t need = zero_layer_norm_grad_scratch_bytes(T, D);
        if (scratch_bytes < need) return ZERO_ERR_SIZE;
        sp.add(scratch, need, true);
    }
    sp.rows(dy, T, dy_ld, D, 2, false);
    if (dsum) sp.rows(dsum, T, dsum_ld, D, 2, false);
    sp.rows(x, T, x_ld, D, 2, false);
    sp.add(mean, 4 * T, false);
    sp.add(rstd, 4 * T, false);
    sp.add(weight, 2 * D, false);
    sp.rows(dx, T, dx_ld, D, 2, true);
    LM_CHECK(sp.check());

    LayerNormGradArgs a{};
    a.dy = dy;
    a.dsum = dsum;
    a.x = x;
    a.mean = mean;
    a.rstd = rstd;
    a.w = weight;
    a.dx = dx;
    a.dw = dweight;
    a.db = dbias;
    a.parts = wanted ? static_cast<float*>(scratch) : nullptr;
    a.T = T;
    a.dy_ld = dy_ld;
    a.dsum_ld = dsum_ld;
    a.x_ld = x_ld;
    a.dx_ld = dx_ld;
    a.D = D;
    auto run = [&](void (*kernel)(LayerNormGradArgs), int sub, int nv, int most,
                   std::atomic<int> (*per_sm)[33]) {
        // up to 1024 columns blocks of 128 threads, several on an SM; else one block an SM, with as
        // many rows at a time as its registers allow: fewer parts to join than with a block for
        // each (2000 x 2048 in blocks of a row 13.2 us)
        a.apart = sub ? sub : 32 * warps_of(D, nv);
        a.groups = sub ? 128 / sub : std::max(1, most / a.apart);
        const int warps = a.apart * a.groups / 32, threads = 32 * warps;
        const int smem = grad_stages(most) * nv * threads * 48;
        // as many blocks as are resident at once: a second wave would be a short one.  Where a row
        // is a warp's or less at 4 rows a group at least, but one block an SM: 10000 x 256 takes
        // 8.0 us so and 10.1 with 16 rows, 333 x 768 4.3 us, in as many blocks as fit 5.5
        const int64_t few = std::max<int64_t>(device_sms(), T / (a.groups * 4));
        int dev = 0;
        cudaGetDevice(&dev);
        int fit = per_sm[dev & 63][warps].load(std::memory_order_relaxed);
        cudaError_t e = cudaSuccess;
        if (fit == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, smem);
            if (e == cudaSuccess && fit > 0)
                per_sm[dev & 63][warps].store(fit, std::memory_order_relaxed);
        }
        a.blocks = (int)std::min<int64_t>({sub ? (T + a.groups - 1) / a.groups : T, few,
                                           (int64_t)grad_blocks(T),
                                           (int64_t)std::max(1, fit) * device_sms()});
        // Rows of a block at a time: few are spread over all blocks; of many those that share the
        // cache line between them go to one block (30000 x 2056 90 us spread, 85 near;
        // 32768 x 2048 80 and 82).  By the width, not by the strides: which rows' sums are added first
        // would else depend on the rows' padding, and with it the last bits of dw and db.
        a.near = T > 4 * (int64_t)a.blocks * a.groups && D % 64 != 0;
        if (e == cudaSuccess) e = launch(kernel, dim3((unsigned)a.blocks), threads, smem, st, a);
        if (e == cudaSuccess && wanted)
            e = launch(k_layer_norm_join, dim3((unsigned)((2 * D + kJoinCols - 1) / kJoinCols)),
                       kJoinThreads, 0, st, a);
        return status_of(e);
    };
#define GRAD_GO(sub, nv, most) \
    run(k_layer_norm_grad<sub, nv, most>, sub, nv, most, grad_per_sm<sub, nv, most>)
    // Up to 1024 columns as in the forward pass: 500000 x 128 takes 77 us in 8 lanes and 82 in 16,
    // 200000 x 256 63 in 16 and 69 in 32, 80000 x 768 74 in a warp and 93 in four, 60000 x 1024 76
    // and 90.
    if (D <= 64) return GRAD_GO(8, 1, 128);
    if (D <= 128) return GRAD_GO(8, 2, 128);
    if (D <= 192) return GRAD_GO(8, 3, 128);
    if (D <= 256) return GRAD_GO(16, 2, 128);
    if (D <= 384) return GRAD_GO(16, 3, 128);
    if (D <= 512) return GRAD_GO(32, 2, 128);
    if (D <= 768) return GRAD_GO(32, 3, 128);
    if (D <= 1024) return GRAD_GO(32, 4, 128);
    // wider rows: 2 vectors a thread, 16 warps an SM; where that leaves one row an SM and 3
    // vectors in 12 warps two, those (12000 x 4104: 86 us with 2, 75 with 3; with more vectors
    // elsewhere, 2048 columns 83 with 2 and 91 with 4, 2056 columns 84 with 2 and 92 with 3)
    if (D <= 8192 && 16 / warps_of(D, 2) == 1 && 12 / warps_of(D, 3) > 1) return GRAD_GO(0, 3, 384);
    if (D <= 8192) return GRAD_GO(0, 2, 512);
    // Beyond, a row of 2 vectors a thread takes 1024 threads, which leave 64 registers: the sums of dw
    // and db alone are 32, and the loop spills (364 bytes a thread).  8000 x 8200 takes 225 us (2.3
    // TB/s; 8000 x 8192 81), 6000 x 12000 207, 4000 x 16384 174 (3.0 TB/s).
    return GRAD_GO(0, 2, 1024);
#undef GRAD_GO
}
