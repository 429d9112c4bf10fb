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
    __shared__ alignas(16) char k0[X::BYTES];
    __shared__ alignas(16) char k1[X::BYTES];
    __shared__ alignas(16) char v0[X::BYTES];
    __shared__ alignas(16) char v1[X::BYTES];
    RowBlock w;
    if (!locate_rows<true>(a, a.heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kv_head = w.head / (a.heads / a.kv_heads), row_bytes = a.dim * X::ES;
    const TileLoad<X> load_k(head_rows(a.k, w, kv_head, row_bytes), tid);
    const TileLoad<X> load_v(head_rows(a.v, w, kv_head, row_bytes), tid);
    const int before = (int)(w.r0 / X::ROWS);
    const int64_t kend = w.len < w.r0 + kAttnRows ? w.len : w.r0 + kAttnRows;
    const int ntiles = (int)((kend + X::ROWS - 1) / X::ROWS);
    load_k(k0, 0, w.len, wave);
    load_v(v0, 0, w.len, wave);
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

    auto add = [&](const char* K, const char* V, int r0, bool diagonal) __attribute__((always_inline)) {
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

    auto turn = [&](int t, const char* K, const char* V, char* next_k, char* next_v) __attribute__((always_inline)) {
        tiles_ready();
        load_k(next_k, (int64_t)(t + 1) * X::ROWS, w.len, wave);
        load_v(next_v, (int64_t)(t + 1) * X::ROWS, w.len, wave);
#pragma unroll
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) add(K, V, r0, false);
    };
    for (int t = 0; t < before; t += 2) {
        turn(t, k0, v0, k1, v1);
        turn(t + 1, k1, v1, k0, v0);
    }
    for (int t = before; t < ntiles; ++t) {
        const bool odd = t & 1;
        tiles_ready();
        if (t + 1 < ntiles) {
            load_k(odd ? k0 : k1, (int64_t)(t + 1) * X::ROWS, w.len, wave);
            load_v(odd ? v0 : v1, (int64_t)(t + 1) * X::ROWS, w.len, wave);
        }
#pragma unroll 1
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) {
            const int64_t at = (int64_t)t * X::ROWS + r0;
            if (active && at <= q0) add(odd ? k1 : k0, odd ? v1 : v0, r0, at == q0);
        }
    }
    if (active) store_columns<T, X::DB>(dq, a.scale, head_rows(a.dq, w, w.head, row_bytes), q0, w.len, lane);
}

// dk and dv: 128 keys to a workgroup and 32 to a wave, the keys along the lanes; query rows and their gradients
// go by in tiles of 32, head after head of the group.
//
// Registers bound it: keys, dk and dv of 32 x 128 elements are 160 of the 256 that two waves to a SIMD have, so bf16 heads
// over 64 elements keep their values in LDS, a right operand that is read again for every tile.
template <typename T, int DC>
struct Grads {
    static constexpr bool V_LDS = sizeof(T) == 2 && DC > 64;
    using X = HeadTile<T, DC, 32>;
    uint4 k[X::SG], v[V_LDS ? 1 : X::SG];
    floatx16 dk[X::DB] = {}, dv[X::DB] = {};

    // rows of one tile; OWN: they may be the keys' own tokens (`diagonal`)
    template <bool OWN>
    __device__ __forceinline__ void add(const char* Q, const char* D, const char* V, const float* lse, const float* delta,
                                        float c, bool diagonal, int wave, int lane) {
        // what follows from the lane is computed again for every tile: kept over the loop (with the values' rows, which
        // do not change either) it would not fit the registers
        asm volatile("" : "+v"(lane));
        const int half = lane >> 5, col = lane & 31;
        floatx16 p = X::rows_by(Q, 0, k, lane), dp;
        if constexpr (V_LDS) dp = X::rows_by_rows(D, 0, V, 32 * wave, lane);
        else dp = X::rows_by(D, 0, v, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const floatx4 e = *(const floatx4*)(lse + 8 * n + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = fast_exp2(fmaf(p[4 * n + i], c, -e[i]));
                p[4 * n + i] = OWN && diagonal && acc_row(4 * n + i, half) < col ? 0.f : x;
            }
        }
        X::columns_by(D, 0, p, dv, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const floatx4 e = *(const floatx4*)(delta + 8 * n + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = p[4 * n + i] * (dp[4 * n + i] - e[i]);
                p[4 * n + i] = OWN && diagonal && acc_row(4 * n + i, half) < col ? 0.f : x;
            }
        }
        X::columns_by(Q, 0, p, dk, lane);
    }
};

template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_dkv(const AttnArgs a) {
    using G = Grads<T, DC>;
    using X = typename G::X;
    using Y = HeadTile<T, DC, kAttnRows>;
    __shared__ alignas(16) char qa[X::BYTES];
    __shared__ alignas(16) char qb[X::BYTES];
    __shared__ alignas(16) char da[X::BYTES];
    __shared__ alignas(16) char db[X::BYTES];
    __shared__ alignas(16) char vs[G::V_LDS ? Y::BYTES : 16];
    __shared__ alignas(16) float ra[2][32];   // lse in log2 units, delta
    __shared__ alignas(16) float rb[2][32];
    RowBlock w;
    if (!locate_rows<false>(a, a.kv_heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = a.heads / a.kv_heads, row_bytes = a.dim * X::ES;
    const int64_t k0 = w.r0 + 32 * wave;
    const bool active = k0 < w.len;

    G grads;
    const TileLoad<X> load_q(head_rows(a.q, w, w.head * group, row_bytes), tid);
    const TileLoad<X> load_d(head_rows(a.dout, w, w.head * group, row_bytes), tid);
    // Lanes i and 32 + i of the first wave bring lse and delta of row i.  Without divergent branches, here and in all that
    // runs at the full number of registers: a compiler that has none to spare may put the copies that it splits
    // values with before the execution mask is whole again.
    auto load = [&](int h, int64_t r0, char* Q, char* D, float (&rows)[2][32]) __attribute__((always_inline)) {
        TileLoad<X> lq = load_q, ld = load_d;
        lq.src.p += h * a.q.head;
        ld.src.p += h * a.dout.head;
        lq(Q, r0, w.len, wave);
        ld(D, r0, w.len, wave);
        if (wave == 0) {
            const int64_t at = token_row(a, w, w.head * group + h) + r0;
            const int left = (int)(w.len - r0 < 32 ? w.len - r0 : 32), row = lane & 31;
            const float e = bits_to_f32(buffer_load_bits(make_rsrc(a.lse + at, left * 4), row * 4, 0.f)) * kLog2e;
            const float d = bits_to_f32(buffer_load_bits(make_rsrc(a.delta + at, left * 4), row * 4, 0.f));
            // rows that are not there: probabilities of 0
            rows[lane >> 5][row] = lane >= 32 ? d : row < left ? e : 1e30f;
        }
    };
    if constexpr (G::V_LDS) {
        const TileLoad<Y> load_v(head_rows(a.v, w, w.head, row_bytes), tid);
        load_v(vs, w.r0, w.len, wave);
    } else {
        load_rows<X>(grads.v, head_rows(a.v, w, w.head, row_bytes), k0, w.len, lane);
    }
    load_rows<X>(grads.k, head_rows(a.k, w, w.head, row_bytes), k0, w.len, lane);
    const float c = a.scale * kLog2e;

    // all heads' tiles from row `from` to `to`, the next one on its way while one is worked on
    auto run = [&](int64_t from, int64_t to, auto work) __attribute__((always_inline)) {
        if (from >= to) return;
        int h = 0;
        int64_t r0 = from;   // the tile at hand
        load(0, r0, qa, da, ra);
        auto turn = [&](const char* Q, const char* D, const float (&rows)[2][32], char* next_q, char* next_d,
                        float (&next_rows)[2][32]) __attribute__((always_inline)) {
            tiles_ready();
            const bool more = r0 + 32 < to;
            const int64_t at = r0;
            r0 = more ? r0 + 32 : from;
            h += more ? 0 : 1;
            if (h < group) load(h, r0, next_q, next_d, next_rows);
            work(at, Q, D, rows);
        };
        while (true) {
            turn(qa, da, ra, qb, db, rb);
            if (h >= group) break;
            turn(qb, db, rb, qa, da, ra);
            if (h >= group) break;
        }
        tiles_ready();
    };
    const int64_t own = w.len < w.r0 + kAttnRows ? w.len : w.r0 + kAttnRows;
    run(w.r0, own, [&](int64_t r0, const char* Q, const char* D, const float (&rows)[2][32]) __attribute__((always_inline)) {
        if (active && r0 >= k0) grads.template add<true>(Q, D, vs, rows[0], rows[1], c, r0 == k0, wave, lane);
    });
    run(own, w.len, [&](int64_t, const char* Q, const char* D, const float (&rows)[2][32]) __attribute__((always_inline)) {
        grads.template add<false>(Q, D, vs, rows[0], rows[1], c, false, wave, lane);
    });
    if (!active) return;
    store_columns<T, X::DB>(grads.dk, a.scale, head_rows(a.dk, w, w.head, row_bytes), k0, w.len, lane);
    store_columns<T, X::DB>(grads.dv, 1.f, head_rows(a.dv, w, w.head, row_bytes), k0, w.len, lane);
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
