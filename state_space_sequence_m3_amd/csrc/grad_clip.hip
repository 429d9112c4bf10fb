// grad_clip.hip -- the 2-norm over many tensors and the scaling that clips it.
//
// The tensors' table travels as a kernel argument, so a call needs no copy to the device and no
// launch per tensor.  Work is cut into units of kGradChunk elements of one tensor; a workgroup
// takes every gridDim-th unit, so which sums meet in which order is fixed.
//
// Squares and sums are in fp64, at its full rate here: a square of an fp32 value neither overflows nor loses
// digits.  Bound: memory.  The norm must be known before the first product, so elements are read twice and written
// once, and the second time from the last-level cache where it still holds them: 60 tensors, 482 MB, in 260 us,
// where two reads and a write at a copy's rate take 273 us.
#include "block_launch.h"
#include "m3_device.h"

namespace m3 {
namespace {

constexpr int kThreads = 256, kSmallThreads = 1024;

struct __attribute__((packed, aligned(2))) Bytes16 { uint32_t v[4]; };
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

// The tensor that holds unit u: the last one whose first unit is at or before it (tensors have at
// least one unit each).
__device__ __forceinline__ int tensor_of(const GradBatch& b, uint32_t u) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.first[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ bool is_bf16(const GradBatch& b, int i) { return (b.is_bf16[i >> 5] >> (i & 31)) & 1; }
__device__ __forceinline__ int unit_size(const GradBatch& b, int i, int64_t at) {
    const int64_t left = b.numel[i] - at;
    return (int)(left < b.chunk ? left : b.chunk);
}

// the sum over all NT threads, in every one of them
template <int NT>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[NT / 64];
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    for (int k = 0; k < NT / 64; ++k) t += s[k];
    __syncthreads();
    return t;
}

// Thread t of NT: its share of the unit at element `at` of tensor i.
template <int NT>
__device__ __forceinline__ void add_squares(const GradBatch& b, int i, int64_t at, int t, double (&acc)[2]) {
    const int n = unit_size(b, i, at);
    if (is_bf16(b, i)) {
        const uint16_t* p = (const uint16_t*)b.src[i] + at;
        int e = t * 8;
#pragma unroll 4
        for (; e + 8 <= n; e += NT * 8) {
            const Bytes16 v = *(const Bytes16*)(p + e);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const double lo = __uint_as_float(v.v[k] << 16), hi = __uint_as_float(v.v[k] & 0xffff0000u);
                acc[0] = fma(lo, lo, acc[0]);
                acc[1] = fma(hi, hi, acc[1]);
            }
        }
        for (; e < n; ++e) {
            const double g = __uint_as_float((uint32_t)p[e] << 16);
            acc[0] = fma(g, g, acc[0]);
        }
    } else {
        const float* p = (const float*)b.src[i] + at;
        int e = t * 4;
#pragma unroll 4
        for (; e + 4 <= n; e += NT * 4) {
            const Bytes16 v = *(const Bytes16*)(p + e);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const double g = __uint_as_float(v.v[k]);
                acc[k & 1] = fma(g, g, acc[k & 1]);
            }
        }
        for (; e < n; ++e) {
            const double g = p[e];
            acc[0] = fma(g, g, acc[0]);
        }
    }
}

// STREAM: non-temporal stores (a template argument, since the compiler makes one ordinary store of two that
// differ in nothing else)
template <int NT, bool STREAM>
__device__ __forceinline__ void scale_unit(const GradBatch& b, int i, int64_t at, int t, float coef) {
    if (coef == 1.f && b.src[i] == b.dst[i]) return;
    const int n = unit_size(b, i, at);
    auto put = [&](void* o, const u32x4& v) {
        if constexpr (STREAM) __builtin_nontemporal_store(v, (u32x4_at2*)o);
        else *(u32x4_at2*)o = v;
    };
    if (is_bf16(b, i)) {
        const uint16_t* p = (const uint16_t*)b.src[i] + at;
        uint16_t* o = (uint16_t*)b.dst[i] + at;
        int e = t * 8;
#pragma unroll 4
        for (; e + 8 <= n; e += NT * 8) {
            const Bytes16 v = *(const Bytes16*)(p + e);
            u32x4 w;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(coef * __uint_as_float(v.v[k] << 16), coef * __uint_as_float(v.v[k] & 0xffff0000u));
            put(o + e, w);
        }
        for (; e < n; ++e) o[e] = bf16_bits_rne(coef * __uint_as_float((uint32_t)p[e] << 16));
    } else {
        const float* p = (const float*)b.src[i] + at;
        float* o = (float*)b.dst[i] + at;
        int e = t * 4;
#pragma unroll 4
        for (; e + 4 <= n; e += NT * 4) {
            const Bytes16 v = *(const Bytes16*)(p + e);
            u32x4 w;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(coef * __uint_as_float(v.v[k]));
            put(o + e, w);
        }
        for (; e < n; ++e) o[e] = coef * p[e];
    }
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const GradBatch b, double* part) {
    double acc[2] = {0.0, 0.0};
    const uint32_t units = b.first[b.n];
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = tensor_of(b, u);
        add_squares<kThreads>(b, i, (int64_t)(u - b.first[i]) * kGradChunk, threadIdx.x, acc);
    }
    const double t = block_sum<kThreads>(acc[0] + acc[1]);
    if (threadIdx.x == 0) part[blockIdx.x] = t;
}

// the sum of n partial sums, the same in every workgroup
__device__ __forceinline__ double all_parts(const double* part, int64_t n) {
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) v += part[i];
    return block_sum<kThreads>(v);
}
__device__ __forceinline__ float2 norm_and_coef(double sum, float max_norm) {
    const double norm = sqrt(sum);
    const double c = (double)max_norm / (norm + 1e-6);
    return make_float2((float)norm, c > 1.0 ? 1.f : (float)c);   // a NaN stays one
}
__device__ __forceinline__ void write_stats(float* stats, float2 nc) {
    if (stats && blockIdx.x == 0 && threadIdx.x == 0) {
        stats[0] = nc.x;
        stats[1] = nc.y;
    }
}

__global__ __launch_bounds__(kThreads) void grad_stats_kernel(const double* part, int64_t n, float max_norm,
                                                              float* stats, double* sum) {
    const double t = all_parts(part, n);
    write_stats(stats, norm_and_coef(t, max_norm));
    if (sum && threadIdx.x == 0) *sum = t;
}

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradBatch b, const double* part, int n_part,
                                                              float max_norm, float* stats) {
    const float2 nc = norm_and_coef(all_parts(part, n_part), max_norm);
    write_stats(stats, nc);
    const uint32_t units = b.first[b.n];
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = tensor_of(b, u);
        // each tensor's units from its end, as the tensors are
        scale_unit<kThreads, STREAM>(b, i, (int64_t)(b.first[i + 1] - 1 - u) * kGradChunk, threadIdx.x, nc.y);
    }
}

// Few elements: sum and scaling in one launch by one workgroup, a unit to a wave at a time, which reads them
// again from its caches.
__global__ __launch_bounds__(kSmallThreads) void grad_small_kernel(const GradBatch b, int write, float max_norm,
                                                                   float* stats) {
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), units = b.first[b.n];
    double acc[2] = {0.0, 0.0};
    for (uint32_t u = wave; u < units; u += kSmallThreads / 64) {
        const int i = tensor_of(b, u);
        add_squares<64>(b, i, (int64_t)(u - b.first[i]) * kGradSmallChunk, lane, acc);
    }
    const float2 nc = norm_and_coef(block_sum<kSmallThreads>(acc[0] + acc[1]), max_norm);
    write_stats(stats, nc);
    if (!write) return;
    for (uint32_t u = wave; u < units; u += kSmallThreads / 64) {
        const int i = tensor_of(b, u);
        scale_unit<64, false>(b, i, (int64_t)(u - b.first[i]) * kGradSmallChunk, lane, nc.y);
    }
}

}  // namespace

hipError_t launch_grad_small(const GradBatch& b, bool write, float max_norm, float* stats, hipStream_t s) {
    hipLaunchKernelGGL(grad_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, b, write ? 1 : 0, max_norm, stats);
    return hipGetLastError();
}
hipError_t launch_grad_sumsq(const GradBatch& b, double* part, hipStream_t s) {
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(grad_blocks(b)), dim3(kThreads), 0, s, b, part);
    return hipGetLastError();
}
hipError_t launch_grad_stats(const double* part, int64_t n, float max_norm, float* stats, double* sum, hipStream_t s) {
    hipLaunchKernelGGL(grad_stats_kernel, dim3(1), dim3(kThreads), 0, s, part, n, max_norm, stats, sum);
    return hipGetLastError();
}
hipError_t launch_grad_scale(const GradBatch& b, const double* part, int n, float max_norm, float* stats,
                             hipStream_t s) {
    const dim3 grid(grad_blocks(b)), block(kThreads);
    if (b.stream) hipLaunchKernelGGL(grad_scale_kernel<true>, grid, block, 0, s, b, part, n, max_norm, stats);
    else hipLaunchKernelGGL(grad_scale_kernel<false>, grid, block, 0, s, b, part, n, max_norm, stats);
    return hipGetLastError();
}

}  // namespace m3
