// rmsnorm.hip -- residual addition, RMS norm and 8-bit rows in one pass, and the norm's backward
// pass.
//
// A row is held in registers by TPR threads, 8 elements (16 bytes of bf16) per thread and chunk: chunk c
// of thread t begins at element (c TPR + t) 8.  One read of the row serves the sum of squares, the
// outputs and the 8-bit scale.  Where 8 does not divide the width, the row's last chunk is moved back to
// end with the row: it reads and writes whole, and its first `skip` elements, which belong to the chunk
// before it as well, are left out of sums and scales (both chunks write the same values there).
//
// Bound: memory, each tensor travelling once.  16384 x 4096 bf16, x and residual in, r, y and q out: 604 MB in 119 us,
// 5.1 TB/s; backward with dr_out 537 MB in 103 us, 5.2 TB/s (a copy: 5.3 to 5.5).  Sums and statistics are in fp32.
#include "block_launch.h"
#include "m3_device.h"

#include <algorithm>

namespace m3 {
namespace {

// 8 consecutive elements; rows may start at any element (gfx950 takes wide global accesses at any
// byte address, at the cost of the extra line they touch).
struct __attribute__((packed, aligned(2))) Bf16x8 { uint32_t v[4]; };
struct __attribute__((packed, aligned(4))) F32x4 { float v[4]; };
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));

template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    Bf16x8 v;
    __device__ __forceinline__ void zero() { v.v[0] = v.v[1] = v.v[2] = v.v[3] = 0; }
    __device__ __forceinline__ void load(const char* p) { v = *(const Bf16x8*)p; }
    __device__ __forceinline__ void load_some(const char* p, int n) {
        zero();
        for (int k = 0; k < 8; ++k)
            if (k < n) v.v[k >> 1] |= (uint32_t)((const uint16_t*)p)[k] << (16 * (k & 1));
    }
    __device__ __forceinline__ float get(int k) const {
        return __uint_as_float(k & 1 ? v.v[k >> 1] & 0xffff0000u : v.v[k >> 1] << 16);
    }
};
template <> struct Raw8<float> {
    F32x4 a, b;
    __device__ __forceinline__ void zero() {
        for (int k = 0; k < 4; ++k) a.v[k] = b.v[k] = 0.f;
    }
    __device__ __forceinline__ void load(const char* p) {
        a = *(const F32x4*)p;
        b = *(const F32x4*)(p + 16);
    }
    __device__ __forceinline__ void load_some(const char* p, int n) {
        zero();
        for (int k = 0; k < 8; ++k)
            if (k < n) (k < 4 ? a.v[k] : b.v[k - 4]) = ((const float*)p)[k];
    }
    __device__ __forceinline__ float get(int k) const { return k < 4 ? a.v[k] : b.v[k - 4]; }
};
// A thread's chunk: its first element (-1: none), and how many of its elements are another chunk's.
struct Chunk {
    int at, skip;
};
__device__ __forceinline__ Chunk chunk_at(int e, int D) {
    if (e >= D) return {-1, 8};
    if (e + 8 <= D || D < 8) return {e, 0};
    return {D - 8, e + 8 - D};
}
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const char* row, Chunk c, int D) {
    const char* p = row + (int64_t)c.at * sizeof(T);
    if (c.at < 0) r.zero();
    else if (D >= 8) r.load(p);
    else r.load_some(p, D);
}
// STREAM: non-temporal.  A template argument, since the compiler makes one ordinary store of two that differ
// in nothing else.  (A macro: templates drop the alignment of a pointer's type.)
#define M3_PUT(TYPE, p, v)                                          \
    do {                                                            \
        if constexpr (STREAM) __builtin_nontemporal_store(v, (TYPE*)(p)); \
        else *(TYPE*)(p) = (v);                                     \
    } while (0)
template <bool STREAM>
__device__ __forceinline__ void store8(char* row, Chunk c, int D, const float (&f)[8], bf16) {
    if (c.at < 0) return;
    uint16_t* p = (uint16_t*)(row + (int64_t)c.at * 2);
    if (D >= 8) {
        u32x4 v;
        for (int k = 0; k < 4; ++k) v[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
        M3_PUT(u32x4_at2, p, v);
    } else {
        for (int k = 0; k < 8; ++k)
            if (k < D) p[k] = bf16_bits_rne(f[k]);
    }
}
template <bool STREAM>
__device__ __forceinline__ void store8(char* row, Chunk c, int D, const float (&f)[8], float) {
    if (c.at < 0) return;
    float* p = (float*)(row + (int64_t)c.at * 4);
    if (D >= 8) {
        u32x4 a, b;
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(f[k]);
            b[k] = __float_as_uint(f[k + 4]);
        }
        M3_PUT(u32x4_at4, p, a);
        M3_PUT(u32x4_at4, p + 4, b);
    } else {
        for (int k = 0; k < 8; ++k)
            if (k < D) p[k] = f[k];
    }
}
// The 8-bit elements that are the chunk's own (the others may have another scale).
template <bool STREAM>
__device__ __forceinline__ void store_q8(uint8_t* row, Chunk c, int D, const float (&f)[8]) {
    if (c.at < 0) return;
    u32x2 v;
    for (int k = 0; k < 2; ++k) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k], f[4 * k + 1], 0, false);
        v[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k + 2], f[4 * k + 3], u, true);
    }
    uint8_t* p = row + c.at + c.skip;
    const int n = D < 8 ? D : 8 - c.skip;
    if (n == 8) {
        M3_PUT(u32x2_at1, p, v);
    } else {
        uint64_t w = (((uint64_t)v[1] << 32) | v[0]) >> (8 * c.skip);
        for (int size = 4; size >= 1; size >>= 1)
            if (n & size) {
                for (int k = 0; k < size; ++k) p[k] = (uint8_t)(w >> (8 * k));
                p += size;
                w >>= 8 * size;
            }
    }
}

// The largest of the magnitudes' bit patterns over aligned groups of R lanes: as patterns, so that
// a NaN is larger than everything and comes through.
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL> __device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t group_umax(uint32_t v, int R) {
    if (R >= 2) v = umax(v, dpp_u<0xB1>(v));
    if (R >= 4) v = umax(v, dpp_u<0x4E>(v));
    if (R >= 8) v = umax(v, dpp_u<0x141>(v));
    if (R >= 16) v = umax(v, dpp_u<0x140>(v));
    if (R >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = umax(p[0], p[1]);
    }
    if (R >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = umax(p[0], p[1]);
    }
    return v;
}

// Rows on 16 lanes, on a wave, or (TPR = kBlock) on a workgroup of as many waves as the row needs.
constexpr int kBlock = 0;
template <int TPR> constexpr int max_threads() { return TPR == kBlock ? 1024 : 256; }
// Waves per SIMD that registers are left for, and with it the workgroups that are resident: the grid is
// that many, each takes every gridDim-th row.  Forward: 4 waves for all 8000 x 5120 bf16 57 -> 65 us (one
// workgroup of 10 waves per compute unit instead of two), 65536 x 300 33 -> 36 us; 8 waves 16384 x 4096
// 90 -> 92 us, 65536 x 128 14 -> 17 us (spills).  Backward: 4 waves for all 8000 x 5120 bf16 73 -> 78 us; 6
// waves 16384 x 4096 104 -> 113 us (spills).
template <typename T, int C> constexpr int kFwdOcc = C > 1 ? 4 : 6;
template <typename T, int C> constexpr int kBwdOcc = C > 1 || sizeof(T) == 4 ? 4 : 5;
// The backward grid of rows on a workgroup leaves out what is over 4 waves per SIMD: with three and more streams of
// rows to a workgroup, fewer of them run at a better rate (30000 x 1111 bf16 73 -> 68 us, 2048 wide 101 -> 98 us).
constexpr int kBwdWant = 4;

// Sums or maxima over a row: over the row's lanes, then, for a row on a workgroup, over its waves.
template <int TPR> __device__ __forceinline__ float row_sum(float v) { return group_sum(v, TPR == kBlock ? 64 : TPR); }

// ---------------------------------------------------------------------------------- forward
template <typename T, int TPR, int C, bool STREAM>
__global__ __launch_bounds__(max_threads<TPR>(), (kFwdOcc<T, C>)) void rmsnorm_kernel(const RmsNormArgs a) {
    __shared__ float s_sum[2][16];
    __shared__ uint32_t s_max[2][16];
    const int tpr = TPR == kBlock ? blockDim.x : TPR, rpw = TPR == kBlock ? 1 : 256 / TPR;
    const int waves = blockDim.x / 64;
    const int t = TPR == kBlock ? threadIdx.x : threadIdx.x % TPR;
    const int slot = TPR == kBlock ? 0 : threadIdx.x / TPR;
    const int D = a.D;
    Chunk ch[C];
    float wt[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        ch[c] = chunk_at((c * tpr + t) * 8, D);
#pragma unroll
        for (int k = 0; k < 8; ++k) wt[c][k] = a.weight && ch[c].at >= 0 && ch[c].at + k < D ? a.weight[ch[c].at + k] : 1.f;
    }
    const float inv_d = 1.f / (float)D;
    Raw8<T> rx[C], rr[C];
    auto load = [&](int64_t row) {             // a row past the end reads nothing
        const char* xp = (const char*)a.x + row * a.x_p;
        const char* pp = (const char*)a.residual + row * a.res_p;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const Chunk m = {row < a.rows ? ch[c].at : -1, 0};
            load8<T>(rx[c], xp, m, D);
            if (a.residual) load8<T>(rr[c], pp, m, D);
        }
    };
    int flip = 0;
    load((int64_t)blockIdx.x * rpw + slot);
    for (int64_t row0 = (int64_t)blockIdx.x * rpw; row0 < a.rows; row0 += (int64_t)gridDim.x * rpw) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;        // a row past the end writes nothing
        float r[C][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) r[c][k] = rx[c].get(k) + (a.residual ? rr[c].get(k) : 0.f);
        if (D % 8 == 0 || D < 8) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k) ss = fmaf(r[c][k], r[c][k], ss);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k) ss = k >= ch[c].skip ? fmaf(r[c][k], r[c][k], ss) : ss;
        }
        // the next row travels while this one is worked on
        if (row0 + (int64_t)gridDim.x * rpw < a.rows) load(row + (int64_t)gridDim.x * rpw);
        ss = row_sum<TPR>(ss);
        if constexpr (TPR == kBlock) {
            if ((threadIdx.x & 63) == 0) s_sum[flip][threadIdx.x >> 6] = ss;
            __syncthreads();                   // and every thread has read its part of the row: outputs may lie over it
            ss = 0.f;
            for (int k = 0; k < waves; ++k) ss += s_sum[flip][k];
        }
        if (a.r_out && live) {
            char* op = (char*)a.r_out + row * a.r_p;
#pragma unroll
            for (int c = 0; c < C; ++c) store8<STREAM>(op, ch[c], D, r[c], T{});
        }
        const float rs = 1.f / sqrtf(ss * inv_d + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) r[c][k] = r[c][k] * rs * wt[c][k];
        if (a.y && live) {
            char* op = (char*)a.y + row * a.y_p;
#pragma unroll
            for (int c = 0; c < C; ++c) store8<STREAM>(op, ch[c], D, r[c], T{});
        }
        if (a.q) {
            uint32_t top[C], all = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                top[c] = 0;
                const int end = D < 8 ? D : 8;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= ch[c].skip && k < end) top[c] = umax(top[c], __float_as_uint(r[c][k]) & 0x7fffffffu);
                all = umax(all, top[c]);
            }
            if (a.group == 0) {
                all = group_umax(all, TPR == kBlock ? 64 : TPR);
                if constexpr (TPR == kBlock) {
                    if ((threadIdx.x & 63) == 0) s_max[flip][threadIdx.x >> 6] = all;
                    __syncthreads();
                    for (int k = 0; k < waves; ++k) all = umax(all, s_max[flip][k]);
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float m = __uint_as_float(a.group == 0 ? all : group_umax(top[c], a.group >> 3));
                float scale = m == 0.f ? 1.f : m / 448.f;
                // a scale with few digits left (or none) is rounded up, since n over one rounded down exceeds 448
                if (scale < 1e-37f && scale * 448.f < m) scale = __uint_as_float(__float_as_uint(scale) + 1);
                float qv[8];
                // q is the fp32 quotient, rounded.  The product with 1 / scale alone lands on the other side of a border
                // between two 8-bit values for 10% of the quotients next to one; with its remainder added it is the
                // quotient.  Where 1 / scale or the remainder could leave fp32's range (a NaN scale is there, too): divided.
                // 16384 x 4096 bf16, x in and q out: the product alone 54 us, this 57, dividing always 75.
                if (scale > 1e-30f && scale < 1e30f) {
                    const float inv = 1.f / scale;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float q0 = r[c][k] * inv;
                        qv[k] = fmaf(fmaf(-q0, scale, r[c][k]), inv, q0);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) qv[k] = r[c][k] / scale;
                }
                const int e = (c * tpr + t) * 8;
                if (live && e < D) {
                    store_q8<STREAM>(a.q + row * (int64_t)D, ch[c], D, qv);
                    if (a.group == 0) {
                        if (e == 0) a.scale[row] = scale;
                    } else if (e % a.group == 0) {
                        a.scale[row * a.ngroups + e / a.group] = scale;
                    }
                }
            }
        }
        flip ^= 1;
    }
}

// --------------------------------------------------------------------------------- backward
// Each workgroup takes rows blockIdx, blockIdx + grid, ... and keeps its share of dweight in
// registers; the shares are added in a second launch.
template <typename T, int TPR, int C, bool STREAM>
__global__ __launch_bounds__(max_threads<TPR>(), (kBwdOcc<T, C>)) void rmsnorm_backward_kernel(const RmsNormArgs a) {
    constexpr int SLOTS = TPR == kBlock ? 1 : 256 / TPR;
    __shared__ float2 s_sum[2][16];
    __shared__ float s_dw[SLOTS > 1 ? SLOTS : 1][SLOTS > 1 ? TPR * C * 8 : 1];
    const int tpr = TPR == kBlock ? blockDim.x : TPR;
    const int waves = blockDim.x / 64;
    const int t = TPR == kBlock ? threadIdx.x : threadIdx.x % TPR;
    const int slot = TPR == kBlock ? 0 : threadIdx.x / TPR;
    const int D = a.D;
    Chunk ch[C];
    float wt[C][8], dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        ch[c] = chunk_at((c * tpr + t) * 8, D);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            wt[c][k] = a.weight && ch[c].at >= 0 && ch[c].at + k < D ? a.weight[ch[c].at + k] : 1.f;
            dw[c][k] = 0.f;
        }
    }
    const float inv_d = 1.f / (float)D;
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * SLOTS; row0 < a.rows; row0 += (int64_t)gridDim.x * SLOTS) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;
        Raw8<T> rr[C], ry[C], rd[C];
        const char* rp = (const char*)a.r + row * a.r_p;
        const char* yp = (const char*)a.dy + row * a.y_p;
        const char* dp = (const char*)a.dr_out + row * a.res_p;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const Chunk m = {live ? ch[c].at : -1, 0};
            load8<T>(rr[c], rp, m, D);
            load8<T>(ry[c], yp, m, D);
            if (a.dr_out) load8<T>(rd[c], dp, m, D);
        }
        float ss = 0.f, su = 0.f;
        if (D % 8 == 0 || D < 8) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float r = rr[c].get(k);
                    ss = fmaf(r, r, ss);
                    su = fmaf(r, ry[c].get(k) * wt[c][k], su);
                }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float r = rr[c].get(k);
                    ss = k >= ch[c].skip ? fmaf(r, r, ss) : ss;
                    su = k >= ch[c].skip ? fmaf(r, ry[c].get(k) * wt[c][k], su) : su;
                }
        }
        ss = row_sum<TPR>(ss);
        su = row_sum<TPR>(su);
        if constexpr (TPR == kBlock) {
            if ((threadIdx.x & 63) == 0) s_sum[flip][threadIdx.x >> 6] = make_float2(ss, su);
            __syncthreads();                   // and every thread has read its part of the row: dx may lie over it
            ss = su = 0.f;
            for (int k = 0; k < waves; ++k) {
                ss += s_sum[flip][k].x;
                su += s_sum[flip][k].y;
            }
        }
        const float rs = 1.f / sqrtf(ss * inv_d + a.eps);
        // r rs and not rs^3: the cube leaves fp32's range for rows of root mean squares beyond 1e13 or below 1e-13
        const float along = su * inv_d * rs;
        char* op = (char*)a.dx + row * a.dx_p;
        if (live) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float n = rr[c].get(k) * rs, dy = ry[c].get(k);
                    o[k] = rs * (dy * wt[c][k] - n * along);
                    if (a.dr_out) o[k] += rd[c].get(k);
                    dw[c][k] = fmaf(dy, n, dw[c][k]);
                }
                store8<STREAM>(op, ch[c], D, o, T{});
            }
        }
        flip ^= 1;
    }
    if (a.part == nullptr) return;
    float* out = a.part + (int64_t)blockIdx.x * D;
    if constexpr (SLOTS == 1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (ch[c].at >= 0 && ch[c].at + k < D) out[ch[c].at + k] = dw[c][k];   // twice the same in a moved chunk
    } else {                                   // the rows side by side, added in order
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (ch[c].at >= 0 && ch[c].at + k < D) s_dw[slot][ch[c].at + k] = dw[c][k];
        __syncthreads();
        for (int e = threadIdx.x; e < D; e += 256) {
            float v = s_dw[0][e];
            for (int k = 1; k < SLOTS; ++k) v += s_dw[k][e];
            out[e] = v;
        }
    }
}

// How rows of D elements are laid out: lanes per row (kBlock: a workgroup), chunks, threads per workgroup.  A row
// is on as few lanes as hold it in 8 (or 16) elements each, so that loads are 16 bytes and few lanes idle: 65536 x
// 64 on a wave each took 39 us backward, on 16 lanes 17; 30000 x 1111 on a workgroup of 4 waves 104 us, on the 3 it
// needs 61.  65536 x 768 on a wave with two chunks 71 us, on a workgroup of two waves 72 (fp32 129, 134); 8000 x
// 8192 fp32 with one chunk 163 us, with two 180.
struct Plan {
    int tpr, chunks, threads;
};
Plan plan_of(int64_t D) {
    if (D <= 128) return {16, 1, 256};
    if (D <= 512) return {64, 1, 256};
    if (D <= 1024) return {64, 2, 256};
    const int chunks = D <= 8192 ? 1 : 2;
    return {kBlock, chunks, (int)((D + 8 * chunks * 64 - 1) / (8 * chunks * 64) * 64)};
}
// f<TPR, C>() for the plan
template <typename F>
auto with_plan(const Plan& p, F&& f) {
    if (p.tpr == 16) return f.template operator()<16, 1>();
    if (p.tpr == 64 && p.chunks == 1) return f.template operator()<64, 1>();
    if (p.tpr == 64) return f.template operator()<64, 2>();
    if (p.chunks == 1) return f.template operator()<kBlock, 1>();
    return f.template operator()<kBlock, 2>();
}
// Workgroups: as many as fit with `occ` waves per SIMD; for rows on a workgroup, of those as many as come
// nearest to `want` waves per SIMD.
unsigned grid_of(int64_t rows, const Plan& p, int occ, int want, int cus) {
    const int per_wg = p.tpr == kBlock ? 1 : p.threads / p.tpr;
    int per_cu = occ * 256 / p.threads;
    if (p.tpr == kBlock) per_cu = std::min(per_cu, (want * 256 + p.threads / 2) / p.threads);
    const int64_t n = (rows + per_wg - 1) / per_wg, most = (int64_t)std::max(per_cu, 1) * cus;
    return (unsigned)std::min(n, most);
}
template <typename T>
struct Forward {
    const RmsNormArgs& a;
    Plan p;
    hipStream_t s;
    template <int TPR, int C>
    hipError_t operator()() {
        const dim3 grid(grid_of(a.rows, p, kFwdOcc<T, C>, kFwdOcc<T, C>, a.cus)), block(p.threads);
        if (a.stream) hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, C, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, C, false>), grid, block, 0, s, a);
        return hipGetLastError();
    }
};
template <typename T>
struct Backward {
    const RmsNormArgs& a;
    Plan p;
    hipStream_t s;
    bool launch;
    int64_t* parts;        // rows of dweight partial sums
    template <int TPR, int C>
    hipError_t operator()() {
        const dim3 grid(grid_of(a.rows, p, kBwdOcc<T, C>, kBwdWant, a.cus)), block(p.threads);
        *parts = (int64_t)grid.x;
        if (!launch) return hipSuccess;
        if (a.stream) hipLaunchKernelGGL((rmsnorm_backward_kernel<T, TPR, C, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((rmsnorm_backward_kernel<T, TPR, C, false>), grid, block, 0, s, a);
        return hipGetLastError();
    }
};
template <typename T>
hipError_t backward(const RmsNormArgs& a, bool launch, int64_t* parts, hipStream_t s) {
    const Plan p = plan_of(a.D);
    return with_plan(p, Backward<T>{a, p, s, launch, parts});
}

}  // namespace

int64_t rmsnorm_backward_parts(int64_t rows, int64_t D, bool bf16_io, int cus) {
    RmsNormArgs a{};
    a.rows = rows;
    a.D = (int)D;
    a.cus = cus;
    int64_t parts = 0;
    (void)(bf16_io ? backward<bf16>(a, false, &parts, nullptr) : backward<float>(a, false, &parts, nullptr));
    return parts;
}

hipError_t launch_rmsnorm(const RmsNormArgs& a, bool bf16_io, hipStream_t s) {
    const Plan p = plan_of(a.D);
    return bf16_io ? with_plan(p, Forward<bf16>{a, p, s}) : with_plan(p, Forward<float>{a, p, s});
}

hipError_t launch_rmsnorm_backward(const RmsNormArgs& a, bool bf16_io, hipStream_t s) {
    int64_t parts = 0;
    hipError_t e = bf16_io ? backward<bf16>(a, true, &parts, s) : backward<float>(a, true, &parts, s);
    if (e == hipSuccess && a.dweight) e = launch_column_sum(a.part, parts, a.D, a.dweight, s);
    return e;
}

}  // namespace m3
