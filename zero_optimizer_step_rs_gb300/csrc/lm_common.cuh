// lm_common.cuh - what the language-model operators (lm_embed.cu, lm_norm.cu,
// lm_xent.cu) share: bf16 vectors, launches, argument checks.
//
// Conventions of these three files: matrices are row-major with the columns
// contiguous and a row stride ("ld") in elements; widths and strides are
// multiples of 8 and pointers are 16-byte aligned, so that every row starts on
// a 16-byte vector of 8 bf16 values.  Row offsets are 64-bit.
#ifndef ZERO_LM_COMMON_CUH
#define ZERO_LM_COMMON_CUH

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "zero_step.h"

namespace lm {

// ------------------------------------------------------- device helpers --

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// round to nearest even; the hardware conversion gives every NaN as 0x7FFF
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void bf_unpack8(const uint4& x, float (&f)[8])
{
    f[0] = bf_lo(x.x); f[1] = bf_hi(x.x);
    f[2] = bf_lo(x.y); f[3] = bf_hi(x.y);
    f[4] = bf_lo(x.z); f[5] = bf_hi(x.z);
    f[6] = bf_lo(x.w); f[7] = bf_hi(x.w);
}

__device__ __forceinline__ uint4 bf_pack8(const float (&f)[8])
{
    return make_uint4(bf_pack(f[0], f[1]), bf_pack(f[2], f[3]), bf_pack(f[4], f[5]),
                      bf_pack(f[6], f[7]));
}

__device__ __forceinline__ uint4 ld16(const void* p)
{
    return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ uint4 ld16_stream(const void* p)
{
    return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void st16(void* p, const uint4& x) { *reinterpret_cast<uint4*>(p) = x; }
__device__ __forceinline__ void st16_stream(void* p, const uint4& x)
{
    __stcs(reinterpret_cast<uint4*>(p), x);
}

// Token ids come as 4- or 8-byte integers.
__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t i)
{
    return bytes == 8 ? static_cast<const long long*>(tokens)[i]
                      : (int64_t)static_cast<const int*>(tokens)[i];
}

// Programmatic dependent launch: wait for the grid before and its writes.
// Unlike the step kernels these do not let the next launch in early: blocks of
// 256 to 1024 threads that wait beside them took places from the next pass
// (gradient of the norm, 32768 x 2048: 89 us with, 77 without; 18000 x 3600: 165
// and 102), and the launches follow closely enough without.
__device__ __forceinline__ void pdl_enter()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// ------------------------------------------------------- launch helpers --

inline int device_sms()
{
    static std::atomic<int> cached[64];
    int dev = 0;
    cudaGetDevice(&dev);
    int n = cached[dev & 63].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (n < 1) n = 1;
        cached[dev & 63].store(n, std::memory_order_relaxed);
    }
    return n;
}

// One launch with programmatic stream serialization; the kernel begins with
// pdl_enter().
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t st,
                   Args&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// A launch of thread-block clusters, in plain stream order.  A cluster needs
// places on several SMs at once, and waiting blocks of programmatic dependents
// hold such places: when these kernels let the next launch in early and were
// launched early themselves, passes of the cross entropy queued one behind
// another stopped for good at 8192 x 128256, where a pass by itself never did.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, int threads, int smem,
                            int cluster, cudaStream_t st, Args&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Raise a kernel's dynamic shared memory limit once per device; `done` is
// one flag per device and kernel.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ------------------------------------------------------- argument checks --

constexpr int64_t kMaxRows = (1ll << 31) - 1024;     // tokens, vocabulary rows
constexpr int32_t kMaxWidth = 1 << 16;

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline zero_status check_ptr(const void* p, unsigned align = 16)
{
    if (!p) return ZERO_ERR_NULL;
    return aligned(p, align) ? ZERO_OK : ZERO_ERR_ALIGN;
}

struct Span {
    uintptr_t lo, hi;
    bool out;
};

// Collects the buffers of a call; outputs may overlap nothing, inputs may
// overlap inputs.  Buffers are kept as whole spans, rows' gaps included.
struct Spans {
    Span s[20];
    int n = 0;
    void add(const void* p, int64_t bytes, bool out)
    {
        if (p && bytes > 0) s[n++] = Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, out};
    }
    void rows(const void* p, int64_t rows, int64_t ld, int64_t width, int elem, bool out)
    {
        if (rows > 0) add(p, ((rows - 1) * ld + width) * elem, out);
    }
    zero_status check() const
    {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((s[i].out || s[j].out) && s[i].lo < s[j].hi && s[j].lo < s[i].hi)
                    return ZERO_ERR_OVERLAP;
        return ZERO_OK;
    }
};

// T tokens, V rows (or 1 where there is no table), D columns
inline zero_status check_sizes(int64_t T, int64_t V, int32_t D, int32_t max_width = kMaxWidth)
{
    if (T < 0 || V < 1 || D < 8 || D % 8 != 0) return ZERO_ERR_INVALID_ARG;
    if (T > kMaxRows || V > kMaxRows || D > max_width) return ZERO_ERR_SIZE;
    return ZERO_OK;
}

inline zero_status check_ld(int64_t ld, int32_t D)
{
    if (ld < D || ld % 8 != 0) return ZERO_ERR_INVALID_ARG;
    return ld <= (1ll << 31) ? ZERO_OK : ZERO_ERR_SIZE;
}

inline zero_status check_tokens(const void* tokens, int32_t bytes)
{
    if (bytes != 4 && bytes != 8) return ZERO_ERR_INVALID_ARG;
    return check_ptr(tokens, (unsigned)bytes);
}

inline zero_status check_status(const int32_t* p)
{
    return p && !aligned(p, 4) ? ZERO_ERR_ALIGN : ZERO_OK;
}

inline zero_status status_of(cudaError_t e)
{
    if (e != cudaSuccess) cudaGetLastError();        // not left for the next caller to find
    return e == cudaSuccess ? ZERO_OK : ZERO_ERR_CUDA;
}

inline int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

}  // namespace lm

#define LM_CHECK(expr) \
    if (zero_status e_ = (expr)) return e_

#endif
