// lm_norm.cu - root-mean-square norm of (activation + residual) that keeps its
// input as an 8-bit checkpoint, the normalised activation rebuilt from the
// checkpoint, and the gradient computed from it (declared in
// include/zero_step.h).
//
//   s = x + r                      (fp32; the new residual stream is bf16(s))
//   rstd = 1 / sqrt(mean(s^2) + eps),   y = bf16(s * rstd * w)
//   checkpoint, per 128 elements of a row: amax = max |s|, scale = amax / 127,
//   code = rint(s * (127 / amax)) in [-127, 127]
// and, with xhat = code * scale * rstd and u = dy * w:
//   replay: y' = bf16(xhat * w)
//   dx = bf16(rstd * (u - xhat * mean(u * xhat)) + dsum),  dw = sum_t dy * xhat
//
// Backward needs neither s nor y in 16 bits: the checkpoint is 1 byte an
// element and 4 bytes per 128, and every value that the backward pass takes
// from it is made in registers.  All of it is bound by HBM traffic: forward
// 2+2 bytes an element read and 2+2+1 written, replay 1 and 2, gradient 2+2+1
// and 2.  Measured, one GB300, 32768 x 2048: forward and replay together 119.7 us
// (6.77 TB/s, the rate of a copy), gradient 77 us (6.1 TB/s; the rows' 25
// instructions an element fill 63 % of the issue slots).  333 x 768: 5.1 us for
// forward and replay, 5.7 us for the gradient, bound by their two launches each.
#include "lm_common.cuh"

namespace {

using namespace lm;

constexpr int kBlock = ZERO_NORM_BLOCK;          // elements that share a scale
constexpr int kLanesPerBlock = kBlock / 8;       // 16 lanes of 8 elements
constexpr float kTiny = 1e-30f;                  // 127 / amax stays finite from here up

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;             // may be null
    const uint16_t* w;
    uint16_t* y;
    uint16_t* sum;                   // may be null
    int8_t* codes;                   // may be null (with scales): no checkpoint
    float* scales;
    float* rstd;
    int64_t T, x_ld, res_ld, y_ld, sum_ld;
    int32_t D;
    float eps;
};

// The sum of one value over the TPR threads of a row: a warp by shuffles, more
// through shared memory.  `slot` alternates from row to row, so that one
// barrier a row is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float (*slots)[32], int slot)
{
    x = warp_sum(x);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) slots[slot][warp] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int k = 0; k < TPR / 32; ++k) x += slots[slot][k];
    }
    return x;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d)
{
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 |
           (uint32_t)(d & 255) << 24;
}

// Signed bytes as floats without the conversion unit, which has a quarter of
// the other units' rate: with its sign bit flipped a byte is code + 128, and as
// the low bits of 2^23 it is that much above 2^23.
__device__ __forceinline__ void unpack_codes(const uint2& q, float (&f)[8])
{
    const uint32_t x = q.x ^ 0x80808080u, y = q.y ^ 0x80808080u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[k] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7540 | k)) - 8388736.0f;
        f[4 + k] = __uint_as_float(__byte_perm(y, 0x4B000000u, 0x7540 | k)) - 8388736.0f;
    }
}

// TPR threads take a row, each NV vectors of 8 elements; blocks of at least
// 128 threads, so a block holds several rows where a row is one warp's.
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128) k_norm(const __grid_constant__ NormArgs a)
{
    constexpr int THREADS = TPR > 128 ? TPR : 128;
    pdl_enter();
    __shared__ float slots[2][32];
    const int64_t t = (int64_t)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
    if (t >= a.T) return;                                  // whole warps; whole blocks if TPR > 32
    const int lane = threadIdx.x % TPR;
    const int nv = a.D >> 3;
    const uint16_t* x = a.x + t * a.x_ld;
    const uint16_t* r = a.res ? a.res + t * a.res_ld : nullptr;

    float f[NV][8];
    {
        uint4 v[NV], u[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = lane + k * TPR;
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
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(f[k][q], f[k][q], ss);
    ss = row_sum<TPR>(ss, slots, 0);
    const float rstd = 1.0f / sqrtf(ss / (float)a.D + a.eps);
    if (lane == 0) a.rstd[t] = rstd;

    const int blocks = (a.D + kBlock - 1) / kBlock;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = lane + k * TPR;
        if (a.codes) {
            // 16 consecutive lanes hold a block; as integers, so that Inf and NaN win
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(f[k][q]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = kLanesPerBlock / 2; o > 0; o >>= 1)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float amax = __uint_as_float(m);
            float scale = 0.0f, inv = 0.0f;
            if (m >= 0x7F800000u) {
                scale = __uint_as_float(0x7FC00000u);      // the block stands for NaN
            } else if (amax >= kTiny) {
                scale = __fdiv_rn(amax, 127.0f);
                inv = __fdiv_rn(127.0f, amax);
            }
            if (c < nv) {
                int q8[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) q8[q] = __float2int_rn(__fmul_rn(f[k][q], inv));
                __stcs(reinterpret_cast<uint2*>(a.codes + t * a.D + c * 8),
                       make_uint2(pack4(q8[0], q8[1], q8[2], q8[3]),
                                  pack4(q8[4], q8[5], q8[6], q8[7])));
                if (c % kLanesPerBlock == 0) a.scales[t * blocks + c / kLanesPerBlock] = scale;
            }
        }
        if (c < nv) {
            if (a.sum) st16_stream(a.sum + t * a.sum_ld + c * 8, bf_pack8(f[k]));
            float w[8];
            bf_unpack8(ld16(a.w + c * 8), w);
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] *= f[k][q] * rstd;
            st16_stream(a.y + t * a.y_ld + c * 8, bf_pack8(w));
        }
    }
}

// ---------------------------------------------------------------- replay --

struct ReplayArgs {
    const int8_t* codes;
    const float* scales;
    const float* rstd;
    const uint16_t* w;
    uint16_t* y;
    int64_t T, y_ld;
    int32_t D;
};

constexpr int kReplayThreads = 256;
constexpr int kReplayVecs = 4;

// A warp takes a row, 4 vectors of each lane in flight.
__global__ void __launch_bounds__(kReplayThreads) k_replay(const __grid_constant__ ReplayArgs a)
{
    pdl_enter();
    const int64_t t = ((int64_t)blockIdx.x * kReplayThreads + threadIdx.x) >> 5;
    if (t >= a.T) return;
    const int lane = threadIdx.x & 31, nv = a.D >> 3;
    const float rstd = a.rstd[t];
    const float* scales = a.scales + t * ((a.D + kBlock - 1) / kBlock);
    const int8_t* codes = a.codes + t * a.D;
    uint16_t* y = a.y + t * a.y_ld;
    for (int base = lane; base < nv; base += 32 * kReplayVecs) {
        uint2 q[kReplayVecs];
        float s[kReplayVecs];
#pragma unroll
        for (int k = 0; k < kReplayVecs; ++k) {
            const int c = base + k * 32;
            if (c < nv) {
                q[k] = __ldcs(reinterpret_cast<const uint2*>(codes + c * 8));
                s[k] = scales[c / kLanesPerBlock];
            }
        }
#pragma unroll
        for (int k = 0; k < kReplayVecs; ++k) {
            const int c = base + k * 32;
            if (c >= nv) break;
            float f[8], w[8];
            unpack_codes(q[k], f);
            bf_unpack8(ld16(a.w + c * 8), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * s[k] * rstd * w[j];
            st16_stream(y + c * 8, bf_pack8(f));
        }
    }
}

// -------------------------------------------------------------- gradient --

struct NormGradArgs {
    const uint16_t* dy;
    const uint16_t* dsum;            // may be null
    const int8_t* codes;
    const float* scales;
    const float* rstd;
    const uint16_t* w;
    uint16_t* dx;
    uint16_t* dw;
    float* parts;                    // [blocks][D]
    int64_t T, dy_ld, dsum_ld, dx_ld;
    int32_t D, blocks;
};

// A copy of N bytes from global memory into the thread's own place in shared
// memory, which only that thread reads: no barrier, only its own wait.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
                     : "memory");
}

// Rows that a thread has asked for ahead of the one it works on, plus that one.
template <int TPR, int NV>
__host__ __device__ constexpr int grad_stages() { return TPR * NV <= 512 ? 3 : 2; }
template <int TPR, int NV>
__host__ __device__ constexpr int grad_smem()
{
    return grad_stages<TPR, NV>() * NV * (TPR > 128 ? TPR : 128) * (16 + 16 + 8 + 4);
}

// As k_norm, but a row's threads walk over many rows and keep the sums of dw
// in registers; a block's row groups are added in order at its end.  A row has
// one barrier in its middle, so without loads for later rows a block has
// nothing in flight for half of the time; registers for them cost the warps that
// hide the rest (spills, or 6 blocks of 128 threads an SM), so they wait in
// shared memory.  With that and pointers that only advance, the rows of 32768 x
// 2048 take 73 us instead of 91.
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128, TPR > 128 ? 1024 / TPR : 6)
    k_norm_grad(const __grid_constant__ NormGradArgs a)
{
    constexpr int THREADS = TPR > 128 ? TPR : 128;
    constexpr int GROUPS = THREADS / TPR;
    constexpr int S = grad_stages<TPR, NV>();
    pdl_enter();
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float slots[2][32];
    // a stage: [NV][THREADS] of dy, dsum (16 bytes), codes (8) and scales (4)
    constexpr int N = NV * THREADS, STAGE = N * 44;
    const uint8_t* mine = ring + threadIdx.x * 16;
    const int group = threadIdx.x / TPR, lane = threadIdx.x % TPR;
    const int nv = a.D >> 3;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    const int64_t first = (int64_t)blockIdx.x * GROUPS + group;

    // where the row to ask for next lies; a thread past the row's end asks for
    // nothing and keeps the zeros that its places start with
    const int nb = (a.D + kBlock - 1) / kBlock;
    const uint16_t* p_d = a.dy + first * a.dy_ld + lane * 8;
    const uint16_t* p_s = a.dsum ? a.dsum + first * a.dsum_ld + lane * 8 : nullptr;
    const int8_t* p_q = a.codes + first * a.D + lane * 8;
    const float* p_c = a.scales + first * nb + lane / kLanesPerBlock;
    const int64_t d_step = step * a.dy_ld, s_step = step * a.dsum_ld;
    const int64_t q_step = step * a.D, c_step = step * nb;
    const uint32_t at16 = (uint32_t)__cvta_generic_to_shared(mine);
    const uint32_t at8 = at16 + N * 32 - threadIdx.x * 8;
    const uint32_t at4 = at16 + N * 40 - threadIdx.x * 12;
    auto ask = [&](bool in, uint32_t stage) {
        if (in) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (lane + k * TPR >= nv) break;
                copy_async<16>(at16 + stage + k * THREADS * 16, p_d + k * TPR * 8);
                copy_async<8>(at8 + stage + k * THREADS * 8, p_q + k * TPR * 8);
                copy_async<4>(at4 + stage + k * THREADS * 4, p_c + k * (TPR / kLanesPerBlock));
                if (p_s) copy_async<16>(at16 + stage + N * 16 + k * THREADS * 16, p_s + k * TPR * 8);
            }
        }
        p_d += d_step;
        if (p_s) p_s += s_step;
        p_q += q_step;
        p_c += c_step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = threadIdx.x; i < S * STAGE / 4; i += THREADS)
        reinterpret_cast<uint32_t*>(ring)[i] = 0;
    __syncthreads();

    uint4 w4[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k)
        w4[k] = lane + k * TPR < nv ? ld16(a.w + (lane + k * TPR) * 8) : make_uint4(0, 0, 0, 0);
    float dw[NV][8] = {};
    uint32_t stage = 0;                                   // offset of the row at hand
    int slot = 0;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) ask(first + s * step < a.T, s * STAGE);
    float rstd_next = first < a.T ? a.rstd[first] : 0.0f;
    uint16_t* p_x = a.dx + first * a.dx_ld + lane * 8;
    const float inv = 1.0f / (float)a.D;
    // (barriers: where a row has more than a warp, the block has one row at a time)
    for (int64_t t = first; t < a.T; t += step, p_x += step * a.dx_ld) {
        const float rstd = rstd_next;
        rstd_next = t + step < a.T ? a.rstd[t + step] : 0.0f;
        ask(t + (S - 1) * step < a.T, stage == 0 ? (S - 1) * STAGE : stage - STAGE);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        // xhat and dy * w are made twice, from what shared memory holds:
        // keeping them would cost 16 registers a vector
        float inner = 0.0f;
        const uint8_t* here = mine + stage;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8], xh[8], d[8];
            bf_unpack8(w4[k], w);
            unpack_codes(*reinterpret_cast<const uint2*>(here + N * 32 - threadIdx.x * 8 +
                                                         k * THREADS * 8), xh);
            bf_unpack8(*reinterpret_cast<const uint4*>(here + k * THREADS * 16), d);
            const float sc = *reinterpret_cast<const float*>(here + N * 40 - threadIdx.x * 12 +
                                                             k * THREADS * 4) * rstd;
            float part = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float p = d[q] * xh[q];
                dw[k][q] = fmaf(p, sc, dw[k][q]);
                part = fmaf(p, w[q], part);
            }
            inner = fmaf(part, sc, inner);
        }
        inner = row_sum<TPR>(inner, slots, slot) * inv;
        slot ^= 1;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (lane + k * TPR >= nv) break;
            float s[8] = {}, w[8], xh[8], d[8];
            bf_unpack8(w4[k], w);
            unpack_codes(*reinterpret_cast<const uint2*>(here + N * 32 - threadIdx.x * 8 +
                                                         k * THREADS * 8), xh);
            bf_unpack8(*reinterpret_cast<const uint4*>(here + k * THREADS * 16), d);
            if (p_s) bf_unpack8(*reinterpret_cast<const uint4*>(here + N * 16 +
                                                                k * THREADS * 16), s);
            const float back =
                -*reinterpret_cast<const float*>(here + N * 40 - threadIdx.x * 12 +
                                                 k * THREADS * 4) * rstd * inner;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                s[q] = fmaf(rstd, fmaf(xh[q], back, d[q] * w[q]), s[q]);
            st16_stream(p_x + k * TPR * 8, bf_pack8(s));
        }
        stage = stage == (S - 1) * STAGE ? 0 : stage + STAGE;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float* part = a.parts + (int64_t)blockIdx.x * a.D;
    if constexpr (GROUPS == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = lane + k * TPR;
            if (c < nv)
#pragma unroll
                for (int q = 0; q < 8; ++q) part[c * 8 + q] = dw[k][q];
        }
    } else {
        __shared__ float all[GROUPS][TPR * NV * 8];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int q = 0; q < 8; ++q) all[group][(lane + k * TPR) * 8 + q] = dw[k][q];
        __syncthreads();
        for (int i = threadIdx.x; i < a.D; i += THREADS) {
            float s = all[0][i];
#pragma unroll
            for (int g = 1; g < GROUPS; ++g) s += all[g][i];
            part[i] = s;
        }
    }
}

// dw = the blocks' parts, added in an order that depends on their number only:
// 32 columns a block, 128 shares of the rows, then the shares in order.
constexpr int kJoinThreads = 1024;
constexpr int kJoinCols = 32;
constexpr int kJoinShares = kJoinThreads / (kJoinCols / 4);

__global__ void __launch_bounds__(kJoinThreads) k_norm_join(const __grid_constant__ NormGradArgs a)
{
    pdl_enter();
    __shared__ float4 share[kJoinShares][kJoinCols / 4];
    const int cv = threadIdx.x % (kJoinCols / 4), sh = threadIdx.x / (kJoinCols / 4);
    const int col = blockIdx.x * kJoinCols + cv * 4;
    float4 s = make_float4(0, 0, 0, 0);
    if (col < a.D)
#pragma unroll 4
        for (int r = sh; r < a.blocks; r += kJoinShares) {
            const float4 x =
                __ldcs(reinterpret_cast<const float4*>(a.parts + (int64_t)r * a.D + col));
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
    share[sh][cv] = s;
    __syncthreads();
#pragma unroll
    for (int o = kJoinShares / 2; o > 0; o >>= 1) {
        if (sh < o) {
            float4 p = share[sh][cv];
            const float4 q = share[sh + o][cv];
            p.x += q.x; p.y += q.y; p.z += q.z; p.w += q.w;
            share[sh][cv] = p;
        }
        __syncthreads();
    }
    if (sh == 0 && col < a.D) {
        const float4 p = share[0][cv];
        *reinterpret_cast<uint2*>(a.dw + col) = make_uint2(bf_pack(p.x, p.y), bf_pack(p.z, p.w));
    }
}

// Blocks of a form of k_norm_grad that fit on an SM, per device (0: not asked yet).
template <int TPR, int NV>
std::atomic<int> grad_per_sm[64];

// The most blocks that k_norm_grad takes: 8 for each of 152 SMs, so 8 fp32 rows
// of parts per SM.
int grad_blocks(int64_t T) { return (int)std::min<int64_t>(T, 1216); }

}  // namespace

// The widths each form takes: a row of up to 512 columns is one warp's, wider
// ones are shared by 128 to 1024 threads with one or two vectors each.
#define NORM_FORMS(F)                  \
    if (D <= 256) return F(32, 1);     \
    if (D <= 512) return F(32, 2);     \
    if (D <= 1024) return F(128, 1);   \
    if (D <= 2048) return F(128, 2);   \
    if (D <= 4096) return F(256, 2);   \
    if (D <= 8192) return F(512, 2);   \
    return F(1024, 2)

extern "C" zero_status zero_norm(const uint16_t* x, int64_t x_ld, const uint16_t* residual,
                                 int64_t residual_ld, const uint16_t* weight, int64_t T, int32_t D,
                                 float eps, uint16_t* y, int64_t y_ld, uint16_t* sum,
                                 int64_t sum_ld, int8_t* codes, float* scales, float* rstd,
                                 void* stream)
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
    LM_CHECK(check_ptr(weight));
    LM_CHECK(check_ptr(y));
    if (sum) LM_CHECK(check_ptr(sum));
    LM_CHECK(check_ptr(rstd));
    if (codes || scales) {
        LM_CHECK(check_ptr(codes));
        LM_CHECK(check_ptr(scales));
    }
    const int64_t nb = (D + kBlock - 1) / kBlock;
    Spans sp;
    sp.rows(x, T, x_ld, D, 2, false);
    if (residual) sp.rows(residual, T, residual_ld, D, 2, false);
    sp.add(weight, 2 * D, false);
    sp.rows(y, T, y_ld, D, 2, true);
    if (sum) sp.rows(sum, T, sum_ld, D, 2, true);
    if (codes) sp.add(codes, T * D, true);
    if (codes) sp.add(scales, 4 * T * nb, true);
    sp.add(rstd, 4 * T, true);
    LM_CHECK(sp.check());

    NormArgs a{};
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.y = y;
    a.sum = sum;
    a.codes = codes;
    a.scales = scales;
    a.rstd = rstd;
    a.T = T;
    a.x_ld = x_ld;
    a.res_ld = residual_ld;
    a.y_ld = y_ld;
    a.sum_ld = sum_ld;
    a.D = D;
    a.eps = eps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
#define NORM_GO(tpr, nv)                                                                       \
    status_of(launch(k_norm<tpr, nv>,                                                          \
                     dim3((unsigned)((T + (tpr > 128 ? 1 : 128 / tpr) - 1) /                   \
                                     (tpr > 128 ? 1 : 128 / tpr))),                            \
                     tpr > 128 ? tpr : 128, 0, st, a))
    NORM_FORMS(NORM_GO);
#undef NORM_GO
}

extern "C" zero_status zero_norm_replay(const int8_t* codes, const float* scales,
                                        const float* rstd, const uint16_t* weight, int64_t T,
                                        int32_t D, uint16_t* y, int64_t y_ld, void* stream)
{
    LM_CHECK(check_sizes(T, 1, D, ZERO_NORM_MAX_WIDTH));
    LM_CHECK(check_ld(y_ld, D));
    if (T == 0) return ZERO_OK;
    LM_CHECK(check_ptr(codes));
    LM_CHECK(check_ptr(scales));
    LM_CHECK(check_ptr(rstd));
    LM_CHECK(check_ptr(weight));
    LM_CHECK(check_ptr(y));
    Spans sp;
    sp.add(codes, T * D, false);
    sp.add(scales, 4 * T * ((D + kBlock - 1) / kBlock), false);
    sp.add(rstd, 4 * T, false);
    sp.add(weight, 2 * D, false);
    sp.rows(y, T, y_ld, D, 2, true);
    LM_CHECK(sp.check());
    const ReplayArgs a{codes, scales, rstd, weight, y, T, y_ld, D};
    const int per = kReplayThreads / 32;
    return status_of(launch(k_replay, dim3((unsigned)((T + per - 1) / per)), kReplayThreads, 0,
                            static_cast<cudaStream_t>(stream), a));
}

extern "C" int64_t zero_norm_grad_scratch_bytes(int64_t T, int32_t D)
{
    if (check_sizes(T, 1, D, ZERO_NORM_MAX_WIDTH) != ZERO_OK) return -1;
    return up(4 * (int64_t)grad_blocks(T) * D, 256);
}

extern "C" zero_status zero_norm_grad(const uint16_t* dy, int64_t dy_ld, const uint16_t* dsum,
                                      int64_t dsum_ld, const int8_t* codes, const float* scales,
                                      const float* rstd, const uint16_t* weight, int64_t T,
                                      int32_t D, uint16_t* dx, int64_t dx_ld, uint16_t* dweight,
                                      void* scratch, int64_t scratch_bytes, void* stream)
{
    LM_CHECK(check_sizes(T, 1, D, ZERO_NORM_MAX_WIDTH));
    LM_CHECK(check_ld(dy_ld, D));
    LM_CHECK(check_ld(dx_ld, D));
    if (dsum) LM_CHECK(check_ld(dsum_ld, D));
    LM_CHECK(check_ptr(dweight));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return status_of(cudaMemsetAsync(dweight, 0, (size_t)(2 * D), st));
    LM_CHECK(check_ptr(dy));
    if (dsum) LM_CHECK(check_ptr(dsum));
    LM_CHECK(check_ptr(codes));
    LM_CHECK(check_ptr(scales));
    LM_CHECK(check_ptr(rstd));
    LM_CHECK(check_ptr(weight));
    LM_CHECK(check_ptr(dx));
    LM_CHECK(check_ptr(scratch));
    const int64_t need = zero_norm_grad_scratch_bytes(T, D);
    if (scratch_bytes < need) return ZERO_ERR_SIZE;
    Spans sp;
    sp.rows(dy, T, dy_ld, D, 2, false);
    if (dsum) sp.rows(dsum, T, dsum_ld, D, 2, false);
    sp.add(codes, T * D, false);
    sp.add(scales, 4 * T * ((D + kBlock - 1) / kBlock), false);
    sp.add(rstd, 4 * T, false);
    sp.add(weight, 2 * D, false);
    sp.rows(dx, T, dx_ld, D, 2, true);
    sp.add(dweight, 2 * D, true);
    sp.add(scratch, need, true);
    LM_CHECK(sp.check());

    NormGradArgs a{};
    a.dy = dy;
    a.dsum = dsum;
    a.codes = codes;
    a.scales = scales;
    a.rstd = rstd;
    a.w = weight;
    a.dx = dx;
    a.dw = dweight;
    a.parts = static_cast<float*>(scratch);
    a.T = T;
    a.dy_ld = dy_ld;
    a.dsum_ld = dsum_ld;
    a.dx_ld = dx_ld;
    a.D = D;
    auto run = [&](void (*kernel)(NormGradArgs), int tpr, int smem, std::atomic<int>* per_sm) {
        const int threads = tpr > 128 ? tpr : 128, groups = threads / tpr;
        // as many blocks as are resident at once: a second wave would be a short one
        int dev = 0;
        cudaGetDevice(&dev);
        int fit = per_sm[dev & 63].load(std::memory_order_relaxed);
        cudaError_t e = cudaSuccess;
        if (fit == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, smem);
            if (e == cudaSuccess && fit > 0)
                per_sm[dev & 63].store(fit, std::memory_order_relaxed);
        }
        a.blocks = (int)std::min<int64_t>({(T + groups - 1) / groups, (int64_t)grad_blocks(T),
                                           (int64_t)std::max(1, fit) * device_sms()});
        if (e == cudaSuccess)
            e = launch(kernel, dim3((unsigned)a.blocks), threads, smem, st, a);
        if (e == cudaSuccess)
            e = launch(k_norm_join, dim3((unsigned)((D + kJoinCols - 1) / kJoinCols)),
                       kJoinThreads, 0, st, a);
        return status_of(e);
    };
#define GRAD_GO(tpr, nv) run(k_norm_grad<tpr, nv>, tpr, grad_smem<tpr, nv>(), grad_per_sm<tpr, nv>)
    NORM_FORMS(GRAD_GO);
#undef GRAD_GO
}
