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
// 2+2+2 read and 2 written.
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

// TPR threads take a row, each NV vectors of 8 elements; blocks of at least
// 128 threads, so a block holds several rows where a row is one warp's.
//
// The row stays in registers.  Each warp takes the mean of its own elements and
// their squared distances from it, and the warps' pairs are joined by
//   mean = sum of sums / D,  M2 = sum of (M2_w + n_w (mean_w - mean)^2),
// which cancels nothing and needs one barrier where two passes over the row would
// need two.
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128, 1)
    k_layer_norm(const __grid_constant__ LayerNormArgs a)
{
    constexpr int THREADS = TPR > 128 ? TPR : 128;
    pdl_enter();
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
    // elements of the row that this warp holds
    int held = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        held += min(max(nv - ((lane & ~31) + k * TPR), 0), 32) * 8;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) s += f[k][q];
    s = warp_sum(s);
    float mean = held ? s / (float)held : 0.0f, m2 = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * TPR < nv)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float d = f[k][q] - mean;
                m2 = fmaf(d, d, m2);
            }
    m2 = warp_sum(m2);
    if constexpr (TPR > 32) {
        __shared__ float4 parts[TPR / 32];
        if ((threadIdx.x & 31) == 0)
            parts[threadIdx.x >> 5] = make_float4(s, mean, m2, (float)held);
        __syncthreads();
        float total = 0.0f;
#pragma unroll 8
        for (int k = 0; k < TPR / 32; ++k) total += parts[k].x;
        mean = total / (float)a.D;
        m2 = 0.0f;
#pragma unroll 8
        for (int k = 0; k < TPR / 32; ++k) {
            const float4 p = parts[k];
            const float d = p.y - mean;
            m2 += fmaf(p.w * d, d, p.z);
        }
    }
    const float rstd = 1.0f / sqrtf(m2 / (float)a.D + a.eps);
    if (lane == 0) {
        a.mean[t] = mean;
        a.rstd[t] = rstd;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = lane + k * TPR;
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
};

// The sums of two values over the TPR threads of a row.  `slot` alternates from
// row to row, so that one barrier a row is enough.
template <int TPR>
__device__ __forceinline__ float2 row_sums(float x, float y, float2 (*slots)[32], int slot)
{
    x = warp_sum(x);
    y = warp_sum(y);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) slots[slot][warp] = make_float2(x, y);
        __syncthreads();
        if constexpr (TPR > 256) {
            const int lane = threadIdx.x & 31;
            const float2 p = lane < TPR / 32 ? slots[slot][lane] : make_float2(0.0f, 0.0f);
            x = warp_sum(p.x);
            y = warp_sum(p.y);
        } else {
            x = y = 0.0f;
#pragma unroll
            for (int k = 0; k < TPR / 32; ++k) {
                const float2 p = slots[slot][k];
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

// Rows that a thread has asked for ahead of the one it works on, plus that one.
template <int TPR, int NV>
__host__ __device__ constexpr int grad_stages() { return TPR * NV <= 512 ? 3 : 2; }
template <int TPR, int NV>
__host__ __device__ constexpr int grad_smem()
{
    return grad_stages<TPR, NV>() * NV * (TPR > 128 ? TPR : 128) * 48;
}

// A row's threads walk over many rows and keep the sums of dw and db in
// registers; a block's row groups are added in order at its end.  The rows ahead wait in
// shared memory, where a thread finds its own vectors: with a barrier in the middle of each
// row a block would otherwise have nothing in flight for half of the time.
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR > 128 ? TPR : 128, TPR > 512 ? 1 : TPR > 128 ? 512 / TPR : 4)
    k_layer_norm_grad(const __grid_constant__ LayerNormGradArgs a)
{
    constexpr int THREADS = TPR > 128 ? TPR : 128;
    constexpr int GROUPS = THREADS / TPR;
    constexpr int S = grad_stages<TPR, NV>();
    constexpr int N = NV * THREADS * 16, STAGE = 3 * N;      // a stage: dy, x, dsum
    pdl_enter();
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 slots[2][32];
    const int group = threadIdx.x / TPR, lane = threadIdx.x % TPR;
    const int nv = a.D >> 3;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    const int64_t first = (int64_t)blockIdx.x * GROUPS + group;
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
                if (lane + k * TPR >= nv) break;
                const uint32_t at = mine + stage + k * THREADS * 16;
                copy_async(at, p_d + k * TPR * 8);
                copy_async(at + N, p_x + k * TPR * 8);
                if (p_s) copy_async(at + 2 * N, p_s + k * TPR * 8);
            }
        }
        p_d += d_step;
        p_x += x_step;
        if (p_s) p_s += s_step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * TPR >= nv)
#pragma unroll
            for (int i = 0; i < 3 * S; ++i)
                st16(ring + i * N + (k * THREADS + threadIdx.x) * 16, make_uint4(0, 0, 0, 0));

    uint4 w4[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        w4[k] = make_uint4(kOnes, kOnes, kOnes, kOnes);
        if (a.w && lane + k * TPR < nv) w4[k] = ld16(a.w + (lane + k * TPR) * 8);
    }
    float dw[NV][8] = {}, db[NV][8] = {};
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
    // (barriers: where a row has more than a warp, the block has one row at a time)
    for (int64_t t = first; t < a.T; t += step, p_o += step * a.dx_ld) {
        const float mean = mean_next, rstd = rstd_next;
        if (t + step < a.T) {
            mean_next = a.mean[t + step];
            rstd_next = a.rstd[t + step];
        }
        ask(t + (S - 1) * step < a.T,
            stage == 0 ? (S - 1) * STAGE : stage - STAGE);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        // xhat and dy * w are made twice, from what shared memory holds: keeping them
        // would cost 16 registers a vector
        const uint32_t here = mine + stage;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8], x[8], d[8];
            bf_unpack8(w4[k], w);
            bf_unpack8(ld_shared(here + k * THREADS * 16), d);
            bf_unpack8(ld_shared(here + k * THREADS * 16 + N), x);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float xh = (x[q] - mean) * rstd, u = d[q] * w[q];
                db[k][q] += d[q];
                dw[k][q] = fmaf(d[q], xh, dw[k][q]);
                s1 += u;
                s2 = fmaf(u, xh, s2);
            }
        }
        const float2 all = row_sums<TPR>(s1, s2, slots, slot);
        slot ^= 1;
        const float c1 = all.x * inv, c2 = all.y * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (lane + k * TPR >= nv) break;
            float s[8] = {}, w[8], x[8], d[8];
            bf_unpack8(w4[k], w);
            bf_unpack8(ld_shared(here + k * THREADS * 16), d);
            bf_unpack8(ld_shared(here + k * THREADS * 16 + N), x);
            if (p_s) bf_unpack8(ld_shared(here + k * THREADS * 16 + 2 * N), s);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float xh = (x[q] - mean) * rstd;
                s[q] = fmaf(rstd, fmaf(-xh, c2, fmaf(d[q], w[q], -c1)), s[q]);
            }
            st16_stream(p_o + k * TPR * 8, bf_pack8(s));
        }
        stage = stage == (S - 1) * STAGE ? 0 : stage + STAGE;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.parts) return;
    float* part = a.parts + (int64_t)blockIdx.x * 2 * a.D;
    if constexpr (GROUPS == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = lane + k * TPR;
            if (c < nv)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    part[c * 8 + q] = dw[k][q];
                    part[a.D + c * 8 + q] = db[k][q];
                }
        }
    } else {
        __shared__ float all[GROUPS][TPR * NV * 8];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    all[group][(lane + k * TPR) * 8 + q] = side ? db[k][q] : dw[k][q];
            __syncthreads();
            for (int i = threadIdx.x; i < a.D; i += THREADS) {
                float s = all[0][i];
#pragma unroll
                for (int g = 1; g < GROUPS; ++g) s += all[g][i];
                part[side * a.D + i] = s;
            }
            __syncthreads();
        }
    }
}

// dw and db = the blocks' parts, added in an order that depends on their number only:
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

// Blocks of a form of k_layer_norm_grad that fit on an SM, per device (0: not asked yet).
template <int TPR, int NV>
std::atomic<int> grad_per_sm[64];

// The most blocks that k_layer_norm_grad takes.
int grad_blocks(int64_t T) { return (int)std::min<int64_t>(T, 1216); }

}  // namespace

// The widths each form takes: a row of up to 512 columns is one warp's, wider
// ones are shared by 128 to 1024 threads with one or two vectors each.
#define LAYER_NORM_FORMS(F)            \
    if (D <= 256) return F(32, 1);     \
    if (D <= 512) return F(32, 2);     \
    if (D <= 1024) return F(128, 1);   \
    if (D <= 2048) return F(128, 2);   \
    if (D <= 4096) return F(256, 2);   \
    if (D <= 8192) return F(512, 2);   \
    return F(1024, 2)

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
#define LAYER_NORM_GO(tpr, nv)                                                                 \
    status_of(launch(k_layer_norm<tpr, nv>,                                                    \
                     dim3((unsigned)((T + (tpr > 128 ? 1 : 128 / tpr) - 1) /                   \
                                     (tpr > 128 ? 1 : 128 / tpr))),                            \
                     tpr > 128 ? tpr : 128, 0, st, a))
    LAYER_NORM_FORMS(LAYER_NORM_GO);
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
    auto run = [&](void (*kernel)(LayerNormGradArgs), int tpr, int smem, std::atomic<int>* per_sm) {
        const int threads = tpr > 128 ? tpr : 128, groups = threads / tpr;
        // as many blocks as are resident at once: a second wave would be a short one.  With
        // few rows fewer, one an SM at least, so that there are fewer parts to join: at 16 rows
        // a group 2000 x 2048 takes 13.6 us and 1000 x 768 7.0, in as many blocks as fit 19.6
        // and 12.3; a row that is one warp's is short, and 10000 x 256 takes 10.1 us at 16, 8.0 at 4
        const int64_t few = std::max<int64_t>(device_sms(), T / (groups * (tpr == 32 ? 4 : 16)));
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
        a.blocks = (int)std::min<int64_t>({(T + groups - 1) / groups, few, (int64_t)grad_blocks(T),
                                           (int64_t)std::max(1, fit) * device_sms()});
        if (e == cudaSuccess) e = launch(kernel, dim3((unsigned)a.blocks), threads, smem, st, a);
        if (e == cudaSuccess && wanted)
            e = launch(k_layer_norm_join, dim3((unsigned)((2 * D + kJoinCols - 1) / kJoinCols)),
                       kJoinThreads, 0, st, a);
        return status_of(e);
    };
#define GRAD_GO(tpr, nv) \
    run(k_layer_norm_grad<tpr, nv>, tpr, grad_smem<tpr, nv>(), grad_per_sm<tpr, nv>)
    LAYER_NORM_FORMS(GRAD_GO);
#undef GRAD_GO
}
