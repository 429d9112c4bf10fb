// attention_backward.hip -- gradients of causal attention over whole prompts (m3_attention_backward).
//
// Two launches, so that every gradient is one workgroup's own sum, in a fixed order: one over query rows (dq, and
// delta = dout . o on the way), one over keys (dk and dv, over all query heads of the key head).  Both compute scores and
// probabilities again from q, k and the forward pass's lse, which costs 7 products where 5 would do, and saves
// the atomic or partial sums of dq.
#include "m3_attn_tile.h"

namespace m3 {
namespace {

// dq: as the forward pass, scores transposed, 128 query rows to a workgroup and 32 to a wave.
template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_dq(const AttnArgs a) {
    using X = HeadTile<T, DC>;
    __shared__ alignas(16) char lds[2][2 * X::BYTES];
    RowBlock w;
    if (!locate_rows<true>(a, a.heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kv_head = w.head / (a.heads / a.kv_heads), row_bytes = a.dim * X::ES;
    const RowSource ks = head_rows(a.k, w, kv_head, row_bytes), vs = head_rows(a.v, w, kv_head, row_bytes);
    const int64_t q0 = w.r0 + 32 * wave;
    const int half = lane >> 5, row = lane & 31;
    const bool active = q0 < w.len;

    uint4 qf[X::SG], df[X::SG];
    float delta = 0.f;
    {
        load_rows<X>(qf, head_rows(a.o, w, w.head, row_bytes), q0, w.len, lane);
        load_rows<X>(df, head_rows(a.dout, w, w.head, row_bytes), q0, w.len, lane);
#pragma unroll
        for (int g = 0; g < X::SG; ++g) delta += X::dot(qf[g], df[g]);
        delta = halves_sum(delta);
    }
    load_rows<X>(qf, head_rows(a.q, w, w.head, row_bytes), q0, w.len, lane);
    const int64_t at = token_row(a, w, w.head) + q0 + row;
    float lse = 1e30f;   // rows that are not there: probabilities of 0
    if (q0 + row < w.len) {
        lse = a.lse[at] * kLog2e;
        if (half == 0) a.delta[at] = delta;
    }
    const float c = a.scale * kLog2e;
    floatx16 dq[X::DB] = {};

    auto add = [&](const char* K, const char* V, int r0, bool diagonal) {
        floatx16 s = X::rows_by(K, r0, qf, lane);
        const floatx16 dp = X::rows_by(V, r0, df, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = fast_exp2(fmaf(s[i], c, -lse)) * (dp[i] - delta);
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = acc_row(i, half) > row ? 0.f : s[i];
        }
        X::columns_by(K, r0, s, dq, lane);
    };

    const int before = (int)(w.r0 / X::ROWS);
    const int64_t kend = w.len < w.r0 + kAttnRows ? w.len : w.r0 + kAttnRows;
    const int ntiles = (int)((kend + X::ROWS - 1) / X::ROWS);
    Staged<X> kt, vt;
    kt.load(ks, 0, w.len, tid);
    vt.load(vs, 0, w.len, tid);
    kt.store(lds[0], tid);
    vt.store(lds[0] + X::BYTES, tid);
    __syncthreads();
    int t = 0;
    for (; t < before; ++t) {
        const char* K = lds[t & 1];
        char* next = lds[(t + 1) & 1];
        kt.load(ks, (int64_t)(t + 1) * X::ROWS, w.len, tid);
        vt.load(vs, (int64_t)(t + 1) * X::ROWS, w.len, tid);
#pragma unroll
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) add(K, K + X::BYTES, r0, false);
        kt.store(next, tid);
        vt.store(next + X::BYTES, tid);
        __syncthreads();
    }
    for (; t < ntiles; ++t) {
        const char* K = lds[t & 1];
        char* next = lds[(t + 1) & 1];
        if (t + 1 < ntiles) {
            kt.load(ks, (int64_t)(t + 1) * X::ROWS, w.len, tid);
            vt.load(vs, (int64_t)(t + 1) * X::ROWS, w.len, tid);
        }
#pragma unroll 1
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) {
            const int64_t k0 = (int64_t)t * X::ROWS + r0;
            if (active && k0 <= q0) add(K, K + X::BYTES, r0, k0 == q0);
        }
        if (t + 1 < ntiles) {
            kt.store(next, tid);
            vt.store(next + X::BYTES, tid);
        }
        __syncthreads();
    }
    if (active) store_columns<T, X::DB>(dq, a.scale, head_rows(a.dq, w, w.head, row_bytes), q0, w.len, lane);
}

// dk and dv: 128 keys to a workgroup and 32 to a wave, the keys along the lanes; query rows and their gradients
// go by in tiles, head after head of the group.
template <typename T, int DC>
__global__ __launch_bounds__(256, 1) void attn_dkv(const AttnArgs a) {
    using X = HeadTile<T, DC>;
    __shared__ alignas(16) char lds[2][2 * X::BYTES];
    __shared__ alignas(16) float rows[2][2][X::ROWS];   // lse in log2 units, delta
    RowBlock w;
    if (!locate_rows<false>(a, a.kv_heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads, row_bytes = a.dim * X::ES;
    const int64_t k0 = w.r0 + 32 * wave;
    const int half = lane >> 5, col = lane & 31;
    const bool active = k0 < w.len;

    uint4 kf[X::SG], vf[X::SG];
    load_rows<X>(kf, head_rows(a.k, w, w.head, row_bytes), k0, w.len, lane);
    load_rows<X>(vf, head_rows(a.v, w, w.head, row_bytes), k0, w.len, lane);
    const float c = a.scale * kLog2e;
    floatx16 dk[X::DB] = {}, dv[X::DB] = {};

    auto add = [&](const char* Q, const char* D, const float* lse, const float* delta, int r0, bool diagonal) {
        floatx16 p = X::rows_by(Q, r0, kf, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const floatx4 e = *(const floatx4*)(lse + r0 + 8 * n + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * n + i] = fast_exp2(fmaf(p[4 * n + i], c, -e[i]));
        }
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = acc_row(i, half) < col ? 0.f : p[i];
        }
        X::columns_by(D, r0, p, dv, lane);
        const floatx16 dp = X::rows_by(D, r0, vf, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const floatx4 e = *(const floatx4*)(delta + r0 + 8 * n + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * n + i] *= dp[4 * n + i] - e[i];
        }
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = acc_row(i, half) < col ? 0.f : p[i];
        }
        X::columns_by(Q, r0, p, dk, lane);
    };

    const int first = (int)(w.r0 / X::ROWS), last = (int)((w.len + X::ROWS - 1) / X::ROWS);
    const int per = last - first, ntiles = per * group;
    Staged<X> qt, dt;
    float row_value = 0.f;
    auto load = [&](int n) {
        const int head = w.head * group + n / per, t = first + n % per;
        qt.load(head_rows(a.q, w, head, row_bytes), (int64_t)t * X::ROWS, w.len, tid);
        dt.load(head_rows(a.dout, w, head, row_bytes), (int64_t)t * X::ROWS, w.len, tid);
        if (tid < 2 * X::ROWS) {
            const int64_t r = (int64_t)t * X::ROWS + tid % X::ROWS, at = token_row(a, w, head) + r;
            const bool is_lse = tid < X::ROWS;
            row_value = is_lse ? 1e30f : 0.f;   // rows that are not there: probabilities of 0
            if (r < w.len) row_value = is_lse ? a.lse[at] * kLog2e : a.delta[at];
        }
    };
    auto store = [&](int buf) {
        qt.store(lds[buf], tid);
        dt.store(lds[buf] + X::BYTES, tid);
        if (tid < 2 * X::ROWS) rows[buf][tid / X::ROWS][tid % X::ROWS] = row_value;
    };
    load(0);
    store(0);
    __syncthreads();
#pragma unroll 1
    for (int n = 0; n < ntiles; ++n) {
        const char* Q = lds[n & 1];
        if (n + 1 < ntiles) load(n + 1);
#pragma unroll 1
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) {
            const int64_t q0 = (int64_t)(first + n % per) * X::ROWS + r0;
            if (active && q0 >= k0) add(Q, Q + X::BYTES, rows[n & 1][0], rows[n & 1][1], r0, q0 == k0);
        }
        if (n + 1 < ntiles) store((n + 1) & 1);
        __syncthreads();
    }
    if (!active) return;
    store_columns<T, X::DB>(dk, a.scale, head_rows(a.dk, w, w.head, row_bytes), k0, w.len, lane);
    store_columns<T, X::DB>(dv, 1.f, head_rows(a.dv, w, w.head, row_bytes), k0, w.len, lane);
}

template <typename T, int DC>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s) {
    const uint64_t blocks = a.blocks * (uint64_t)(a.cu ? 1 : a.b);
    attn_dq<T, DC><<<dim3((uint32_t)(blocks * a.heads)), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attn_dkv<T, DC><<<dim3((uint32_t)(blocks * a.kv_heads)), 256, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_type(const AttnArgs& a, hipStream_t s) {
    if (a.dim <= 32) return launch_dim<T, 32>(a, s);
    if (a.dim <= 64) return launch_dim<T, 64>(a, s);
    return a.dim <= 96 ? launch_dim<T, 96>(a, s) : launch_dim<T, 128>(a, s);
}

}  // namespace

hipError_t launch_attention_backward(const AttnArgs& a, bool bf16_io, hipStream_t s) {
    return bf16_io ? launch_type<bf16>(a, s) : launch_type<float>(a, s);
}

}  // namespace m3
