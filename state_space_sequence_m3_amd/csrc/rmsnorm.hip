// rmsnorm.hip -- residual addition, RMS norm and 8-bit rows in one pass, and the norm's backward
// pass.
//
// A row is held in registers by TPR threads, 8 elements (16 bytes of bf16) per thread and chunk:
// element (c TPR + t) 8 + k is element k of chunk c of thread t.  One read of the row serves the
// sum of squares, the outputs and the 8-bit scale.
#include "block_launch.h"
#include "m3_device.h"

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
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const char* row, int e, int D) {
    const char* p = row + (int64_t)e * sizeof(T);
    if (e + 8 <= D) r.load(p);
    else if (e < D) r.load_some(p, D - e);
    else r.zero();
}
// STREAM: non-temporal.  A template argument, since the compiler makes one ordinary store of two that differ
// in nothing else.
template <bool STREAM, typename V, typename P>
__device__ __forceinline__ void put(P* p, V v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool STREAM>
__device__ __forceinline__ void store8(char* row, int e, int D, const float (&f)[8], bf16) {
    uint16_t* p = (uint16_t*)(row + (int64_t)e * 2);
    if (e + 8 <= D) {
        u32x4 v;
        for (int k = 0; k < 4; ++k) v[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
        put<STREAM>((u32x4_at2*)p, v);
    } else {
        for (int k = 0; k < 8; ++k)
            if (e + k < D) p[k] = bf16_bits_rne(f[k]);
    }
}
template <bool STREAM>
__device__ __forceinline__ void store8(char* row, int e, int D, const float (&f)[8], float) {
    float* p = (float*)(row + (int64_t)e * 4);
    if (e + 8 <= D) {
        u32x4 a, b;
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(f[k]);
            b[k] = __float_as_uint(f[k + 4]);
        }
        put<STREAM>((u32x4_at4*)p, a);
        put<STREAM>((u32x4_at4*)(p + 4), b);
    } else {
        for (int k = 0; k < 8; ++k)
            if (e + k < D) p[k] = f[k];
    }
}
template <bool STREAM>
__device__ __forceinline__ void store_q8(uint8_t* p, int e, int D, const float (&f)[8]) {
    u32x2 v;
    for (int k = 0; k < 2; ++k) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k], f[4 * k + 1], 0, false);
        v[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k + 2], f[4 * k + 3], u, true);
    }
    p += e;
    if (e + 8 <= D) {
        put<STREAM>((u32x2_at1*)p, v);
    } else {
        for (int k = 0; k < 8; ++k)
            if (e + k < D) p[k] = (uint8_t)(v[k >> 2] >> (8 * (k & 3)));
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

template <int TPR> constexpr int wg_threads() { return TPR < 256 ? 256 : TPR; }
// Waves per SIMD that registers are left for, and with it the workgroups that are resident: the grid is
// that many, each takes every gridDim-th row.
template <typename T, int TPR, int C> constexpr int kFwdOcc = C > 1 ? 4 : 6;
template <typename T, int TPR, int C> constexpr int kBwdOcc = C > 1 || sizeof(T) == 4 ? 4 : 5;
constexpr int resident(int occ, int threads) { return occ * 256 / threads > 0 ? occ * 256 / threads : 1; }

// ---------------------------------------------------------------------------------- forward
template <typename T, int TPR, int C, bool STREAM>
__global__ __launch_bounds__(wg_threads<TPR>(), (kFwdOcc<T, TPR, C>)) void rmsnorm_kernel(const RmsNormArgs a) {
    constexpr int NT = wg_threads<TPR>(), RPW = NT / TPR, WPR = TPR / 64;   // rows per workgroup, waves per row
    __shared__ float s_sum[2][WPR > 1 ? WPR : 1];
    __shared__ uint32_t s_max[2][WPR > 1 ? WPR : 1];
    const int t = threadIdx.x % TPR;
    const int slot = threadIdx.x / TPR;
    float wt[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int e = (c * TPR + t) * 8 + k;
            wt[c][k] = a.weight && e < a.D ? a.weight[e] : 1.f;
        }
    const float inv_d = 1.f / (float)a.D;
    Raw8<T> rx[C], rr[C];
    auto load = [&](int64_t row) {             // a row past the end reads nothing
        const int D = row < a.rows ? a.D : 0;
        const char* xp = (const char*)a.x + row * a.x_p;
        const char* pp = (const char*)a.residual + row * a.res_p;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            load8<T>(rx[c], xp, (c * TPR + t) * 8, D);
            if (a.residual) load8<T>(rr[c], pp, (c * TPR + t) * 8, D);
        }
    };
    int flip = 0;
    load((int64_t)blockIdx.x * RPW + slot);
    for (int64_t row0 = (int64_t)blockIdx.x * RPW; row0 < a.rows; row0 += (int64_t)gridDim.x * RPW) {
        const int64_t row = row0 + slot;
        const int D = row < a.rows ? a.D : 0;  // and writes nothing
        float r[C][8];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                r[c][k] = rx[c].get(k) + (a.residual ? rr[c].get(k) : 0.f);
                ss = fmaf(r[c][k], r[c][k], ss);
            }
        // the next row travels while this one is worked on; its places are read before they are written
        // (outputs may lie over inputs, row on row)
        if (row0 + (int64_t)gridDim.x * RPW < a.rows) load(row + (int64_t)gridDim.x * RPW);
        ss = group_sum(ss, TPR < 64 ? TPR : 64);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0) s_sum[flip][threadIdx.x >> 6] = ss;
            __syncthreads();
            ss = 0.f;
#pragma unroll
            for (int k = 0; k < WPR; ++k) ss += s_sum[flip][k];
        }
        if (a.r_out) {
            char* op = (char*)a.r_out + row * a.r_p;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if ((c * TPR + t) * 8 < D) store8<STREAM>(op, (c * TPR + t) * 8, D, r[c], T{});
        }
        const float rs = 1.f / sqrtf(ss * inv_d + a.eps);
        uint32_t top[C], all = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            top[c] = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                r[c][k] = r[c][k] * rs * wt[c][k];
                if ((c * TPR + t) * 8 + k < D) top[c] = umax(top[c], __float_as_uint(r[c][k]) & 0x7fffffffu);
            }
            all = umax(all, top[c]);
        }
        if (a.y) {
            char* op = (char*)a.y + row * a.y_p;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if ((c * TPR + t) * 8 < D) store8<STREAM>(op, (c * TPR + t) * 8, D, r[c], T{});
        }
        if (a.q) {
            if (a.group == 0) {
                all = group_umax(all, TPR < 64 ? TPR : 64);
                if constexpr (WPR > 1) {
                    if ((threadIdx.x & 63) == 0) s_max[flip][threadIdx.x >> 6] = all;
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < WPR; ++k) all = umax(all, s_max[flip][k]);
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = (c * TPR + t) * 8;
                const float m = __uint_as_float(a.group == 0 ? all : group_umax(top[c], a.group >> 3));
                const float scale = m == 0.f ? 1.f : m / 448.f;
                float qv[8];
                if (scale > 1e-37f) {
                    const float inv = 1.f / scale;
#pragma unroll
                    for (int k = 0; k < 8; ++k) qv[k] = r[c][k] * inv;
                } else {   // 1 / scale could overflow (a NaN scale comes here, too)
#pragma unroll
                    for (int k = 0; k < 8; ++k) qv[k] = r[c][k] / scale;
                }
                if (e < D) {
                    store_q8<STREAM>(a.q + row * (int64_t)a.D, e, D, qv);
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
__global__ __launch_bounds__(wg_threads<TPR>(), (kBwdOcc<T, TPR, C>)) void rmsnorm_backward_kernel(const RmsNormArgs a) {
    constexpr int NT = wg_threads<TPR>(), RPW = NT / TPR, WPR = TPR / 64;
    __shared__ float2 s_sum[2][WPR > 1 ? WPR : 1];
    const int t = threadIdx.x % TPR;
    const int slot = threadIdx.x / TPR;
    float wt[C][8], dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int e = (c * TPR + t) * 8 + k;
            wt[c][k] = a.weight && e < a.D ? a.weight[e] : 1.f;
            dw[c][k] = 0.f;
        }
    const float inv_d = 1.f / (float)a.D;
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPW; row0 < a.rows; row0 += (int64_t)gridDim.x * RPW) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;
        const int D = live ? a.D : 0;
        Raw8<T> rr[C], ry[C], rd[C];
        const char* rp = (const char*)a.r + row * a.r_p;
        const char* yp = (const char*)a.dy + row * a.y_p;
        const char* dp = (const char*)a.dr_out + row * a.res_p;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            load8<T>(rr[c], rp, (c * TPR + t) * 8, D);
            load8<T>(ry[c], yp, (c * TPR + t) * 8, D);
            if (a.dr_out) load8<T>(rd[c], dp, (c * TPR + t) * 8, D);
        }
        float ss = 0.f, su = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float r = rr[c].get(k);
                ss = fmaf(r, r, ss);
                su = fmaf(r, ry[c].get(k) * wt[c][k], su);
            }
        ss = group_sum(ss, TPR < 64 ? TPR : 64);
        su = group_sum(su, TPR < 64 ? TPR : 64);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & 63) == 0) s_sum[flip][threadIdx.x >> 6] = make_float2(ss, su);
            __syncthreads();
            ss = su = 0.f;
#pragma unroll
            for (int k = 0; k < WPR; ++k) {
                ss += s_sum[flip][k].x;
                su += s_sum[flip][k].y;
            }
        }
        const float rs = 1.f / sqrtf(ss * inv_d + a.eps);
        const float along = rs * rs * rs * (su * inv_d);
        char* op = (char*)a.dx + row * a.dx_p;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float r = rr[c].get(k), dy = ry[c].get(k);
                o[k] = rs * (dy * wt[c][k]) - r * along;
                if (a.dr_out) o[k] += rd[c].get(k);
                if (live) dw[c][k] = fmaf(dy, r * rs, dw[c][k]);
            }
            if ((c * TPR + t) * 8 < D) store8<STREAM>(op, (c * TPR + t) * 8, D, o, T{});
        }
        flip ^= 1;
    }
    if (a.part) {
        float* out = a.part + ((int64_t)blockIdx.x * RPW + slot) * a.D;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int e = (c * TPR + t) * 8 + k;
                if (e < a.D) out[e] = dw[c][k];
            }
    }
}

// Threads per row and chunks per thread for a row of D elements.
struct Plan {
    int tpr, chunks;
};
Plan plan_of(int64_t D) {
    if (D <= 128) return {16, 1};
    if (D <= 512) return {64, 1};
    if (D <= 1024) return {64, 2};
    if (D <= 2048) return {256, 1};
    if (D <= 4096) return {512, 1};
    if (D <= 8192) return {1024, 1};
    return {1024, 2};
}
constexpr int rows_per_wg(int tpr) { return tpr < 256 ? 256 / tpr : 1; }

// f<TPR, C>() for the plan
template <typename F>
auto with_plan(const Plan& p, F&& f) {
    if (p.tpr == 16) return f.template operator()<16, 1>();
    if (p.tpr == 64 && p.chunks == 1) return f.template operator()<64, 1>();
    if (p.tpr == 64) return f.template operator()<64, 2>();
    if (p.tpr == 256) return f.template operator()<256, 1>();
    if (p.tpr == 512) return f.template operator()<512, 1>();
    if (p.chunks == 1) return f.template operator()<1024, 1>();
    return f.template operator()<1024, 2>();
}
unsigned grid_of(int64_t rows, int tpr, int per_cu, int cus) {
    const int64_t n = (rows + rows_per_wg(tpr) - 1) / rows_per_wg(tpr), most = (int64_t)per_cu * cus;
    return (unsigned)(n < most ? n : most);
}
template <typename T>
struct Forward {
    const RmsNormArgs& a;
    hipStream_t s;
    template <int TPR, int C>
    hipError_t operator()() {
        constexpr int NT = wg_threads<TPR>();
        const dim3 grid(grid_of(a.rows, TPR, resident(kFwdOcc<T, TPR, C>, NT), a.cus));
        if (a.stream) hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, C, true>), grid, dim3(NT), 0, s, a);
        else hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, C, false>), grid, dim3(NT), 0, s, a);
        return hipGetLastError();
    }
};
template <typename T>
struct Backward {
    const RmsNormArgs& a;
    hipStream_t s;
    bool launch;
    int64_t* parts;        // rows of dweight partial sums
    template <int TPR, int C>
    hipError_t operator()() {
        constexpr int NT = wg_threads<TPR>();
        const dim3 grid(grid_of(a.rows, TPR, resident(kBwdOcc<T, TPR, C>, NT), a.cus));
        *parts = (int64_t)grid.x * rows_per_wg(TPR);
        if (!launch) return hipSuccess;
        if (a.stream) hipLaunchKernelGGL((rmsnorm_backward_kernel<T, TPR, C, true>), grid, dim3(NT), 0, s, a);
        else hipLaunchKernelGGL((rmsnorm_backward_kernel<T, TPR, C, false>), grid, dim3(NT), 0, s, a);
        return hipGetLastError();
    }
};

}  // namespace

int64_t rmsnorm_backward_parts(int64_t rows, int64_t D, bool bf16_io, int cus) {
    RmsNormArgs a{};
    a.rows = rows;
    a.cus = cus;
    int64_t parts = 0;
    if (bf16_io) with_plan(plan_of(D), Backward<bf16>{a, nullptr, false, &parts});
    else with_plan(plan_of(D), Backward<float>{a, nullptr, false, &parts});
    return parts;
}

hipError_t launch_rmsnorm(const RmsNormArgs& a, bool bf16_io, hipStream_t s) {
    return bf16_io ? with_plan(plan_of(a.D), Forward<bf16>{a, s}) : with_plan(plan_of(a.D), Forward<float>{a, s});
}

hipError_t launch_rmsnorm_backward(const RmsNormArgs& a, bool bf16_io, hipStream_t s) {
    int64_t parts = 0;
    hipError_t e = bf16_io ? with_plan(plan_of(a.D), Backward<bf16>{a, s, true, &parts})
                           : with_plan(plan_of(a.D), Backward<float>{a, s, true, &parts});
    if (e == hipSuccess && a.dweight) e = launch_column_sum(a.part, parts, a.D, a.dweight, s);
    return e;
}

}  // namespace m3
