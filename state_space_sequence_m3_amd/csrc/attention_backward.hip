// attention_backward.hip -- gradients of causal attention over whole prompts (m3_attention_backward).
//
// Two launches, so that every gradient is one workgroup's own sum, in a fixed order: one over query rows (dq, and
// delta = dout . o on the way), one over keys (dk and dv, over all query heads of the key head).  Both compute scores and
// probabilities again from q, k and the forward pass's lse, which costs 7 products where 5 would do, and saves
// the atomic or partial sums of dq.
#include "m3_attn_tile.h"

namespace m3 {
namespace {

// Adds up four waves' sums of the same columns, into the first's.
template <int DB>
__device__ __forceinline__ void join_sums(float* lds, int wave, int lane, floatx16 (&acc)[DB]) {
    join_waves<16 * DB>(lds, wave, lane,
        [&](float* at) __attribute__((always_inline)) {
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) at[(db * 16 + i) * 64] = acc[db][i];
        },
        [&](float* at) __attribute__((always_inline)) {
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[db][i] += at[(db * 16 + i) * 64];
        });
}

// One wave's 32 query rows for dq, along the lanes as in the forward pass.
template <typename T, int DC>
struct DqRows {
    using X = HeadTile<T, DC>;
    uint4 q[X::SG], dout[X::SG];
    floatx16 dq[X::DB] = {};
    float lse, delta;

    // reads the rows, and computes delta from o; `write`: keeps it for the second launch
    __device__ __forceinline__ DqRows(const AttnArgs& a, const RowBlock& w, int64_t q0, bool write, int lane) {
        const int row = lane & 31, row_bytes = a.dim * X::ES;
        load_rows<X>(q, head_rows(a.o, w, w.head, row_bytes), q0, w.len, lane);
        load_rows<X>(dout, head_rows(a.dout, w, w.head, row_bytes), q0, w.len, lane);
        float d = 0.f;
#pragma unroll
        for (int g = 0; g < X::SG; ++g) d += X::dot(q[g], dout[g]);
        delta = halves_sum(d);
        load_rows<X>(q, head_rows(a.q, w, w.head, row_bytes), q0, w.len, lane);
        const int64_t at = token_row(a, w, w.head) + q0 + row;
        lse = 1e30f;   // rows that are not there: probabilities of 0
        if (q0 + row < w.len) {
            lse = a.lse[at] * kLog2e;
            if (write && lane < 32) a.delta[at] = delta;
        }
    }
    // delta without o's rounding: this half's sums of p dp and of p over 32 keys, and what all sums make.  (p is off by as
    // much as lse is, the same for a whole row, which drops out of the quotient.)
    __device__ __forceinline__ void delta_parts(const floatx16& s, const floatx16& dp, float c, bool diagonal, int lane,
                                                float& top, float& bottom) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = fast_exp2(fmaf(s[i], c, -lse));
            const bool seen = !diagonal || acc_row(i, lane >> 5) <= (lane & 31);
            top += seen ? p * dp[i] : 0.f;
            bottom += seen ? p : 0.f;
        }
    }
    __device__ __forceinline__ void set_delta(const AttnArgs& a, const RowBlock& w, int64_t q0, float top, float bottom,
                                              bool write, int lane) {
        delta = bottom != 0.f ? top / bottom : 0.f;   // (rows that are not there)
        if (write && lane < 32 && q0 + lane < w.len) a.delta[token_row(a, w, w.head) + q0 + lane] = delta;
    }
    // scores and the products of dout with the values become ds
    __device__ __forceinline__ void turn(floatx16& s, const floatx16& dp, float c, bool diagonal, int lane) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = fast_exp2(fmaf(s[i], c, -lse)) * (dp[i] - delta);
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = acc_row(i, lane >> 5) > (lane & 31) ? 0.f : s[i];
        }
    }
    __device__ __forceinline__ void add(const char* K, const char* V, int r0, float c, bool diagonal, int lane) {
        floatx16 s = X::rows_by(K, r0, q, lane);
        const floatx16 dp = X::rows_by(V, r0, dout, lane);
        turn(s, dp, c, diagonal, lane);
        X::columns_by(K, r0, s, dq, lane);
    }
};

// A row that sees few keys has most of dp - delta cancel: delta from the rounded o would leave half a step of o whole, 2^-9 of
// dout and o where ds itself may be nothing (dq and dk of sequences of one token: 0.01 for 0).  Bf16 rows that see at most
// 128 keys, whose scores are at hand together, take delta as sum_j p_ij dp_ij / sum_j p_ij in fp32 instead.  o of later
// rows is smaller, as a mean of more values: with even weights its rounding counts for less than a tenth of theirs.  (dq and
// dk of 8 sequences of 16 tokens are 0.0023 off, as those of long ones are.  Backward of 32 x 128 tokens, 32/8 heads of
// 128: 118 -> 126 us, 64 x 40, 16 heads of 64 26.5 -> 29.1, 8 x 2048 unchanged.)
template <typename T>
__device__ __forceinline__ bool takes_sum(int64_t keys) { return sizeof(T) == 2 && keys <= kAttnRows; }

// dq: as the forward pass, scores transposed, 128 query rows to a workgroup and 32 to a wave.  3 products to the forward
// pass's 2 with the same softmax to hide: at b8 L2048, 32/8 heads of 128 bf16, 408 us, matrix units busy 55% of the time, LDS
// 27%; 9 packed sequences of up to 1100, 12/4 heads of 96 fp32, 197 us.
template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_dq(const AttnArgs a) {
    using X = HeadTile<T, DC>;
    __shared__ alignas(16) char k0[X::BYTES];
    __shared__ alignas(16) char k1[X::BYTES];
    __shared__ alignas(16) char v0[X::BYTES];
    __shared__ alignas(16) char v1[X::BYTES];
    RowBlock w;
    if (!locate_rows<kAttnRows, true>(a, a.heads, blockIdx.x, w)) return;
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
    const bool active = q0 < w.len;
    const bool sums = takes_sum<T>(kend);
    DqRows<T, DC> rows(a, w, q0, !sums, lane);
    const float c = a.scale * kLog2e;
    if constexpr (sizeof(T) == 2) {
        if (sums) {
            static_assert(kAttnRows == 2 * X::ROWS, "all keys of the first block are in the two buffers");
            if (ntiles > 1) {
                load_k(k1, X::ROWS, w.len, wave);
                load_v(v1, X::ROWS, w.len, wave);
            }
            tiles_ready();
            if (active) {
                float top = 0.f, bottom = 0.f;
#pragma unroll 1
                for (int r0 = 0; r0 <= q0; r0 += 32) {
                    const floatx16 s = X::rows_by(r0 < X::ROWS ? k0 : k1, r0 % X::ROWS, rows.q, lane);
                    const floatx16 dp = X::rows_by(r0 < X::ROWS ? v0 : v1, r0 % X::ROWS, rows.dout, lane);
                    rows.delta_parts(s, dp, c, r0 == q0, lane, top, bottom);
                }
                rows.set_delta(a, w, q0, halves_sum(top), halves_sum(bottom), true, lane);
            }
        }
    }

    auto turn = [&](int t, const char* K, const char* V, char* next_k, char* next_v) __attribute__((always_inline)) {
        tiles_ready();
        load_k(next_k, (int64_t)(t + 1) * X::ROWS, w.len, wave);
        load_v(next_v, (int64_t)(t + 1) * X::ROWS, w.len, wave);
#pragma unroll
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) rows.add(K, V, r0, c, false, lane);
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
            if (active && at <= q0) rows.add(odd ? k1 : k0, odd ? v1 : v0, r0, c, at == q0, lane);
        }
    }
    if (active) store_columns<T, X::DB>(rows.dq, a.scale, head_rows(a.dq, w, w.head, row_bytes), q0, w.len, lane);
}

// For few rows: 32 of them to a workgroup, and the four parts of 32 keys of each tile of 128 to its waves, whose sums
// are joined at the end.
template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_dq_few(const AttnArgs a) {
    using X = HeadTile<T, DC, 128>;
    using R = DqRows<T, DC>;
    __shared__ alignas(16) char ks[X::BYTES];
    __shared__ alignas(16) char vs[X::BYTES];
    __shared__ float parts[sizeof(T) == 2 ? 4 : 1][2][32];   // of delta, over the waves' keys
    RowBlock w;
    if (!locate_rows<kAttnFew, true>(a, a.heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kv_head = w.head / (a.heads / a.kv_heads), row_bytes = a.dim * X::ES;
    const TileLoad<X> load_k(head_rows(a.k, w, kv_head, row_bytes), tid);
    const TileLoad<X> load_v(head_rows(a.v, w, kv_head, row_bytes), tid);
    const int64_t q0 = w.r0, kend = w.len < q0 + kAttnFew ? w.len : q0 + kAttnFew;
    const bool sums = takes_sum<T>(kend);
    R rows(a, w, q0, wave == 0 && !sums, lane);
    const float c = a.scale * kLog2e;
    in_order();
    load_v(vs, 0, kend, wave);
    in_order();
    load_k(ks, 0, kend, wave);
    in_order();
    if constexpr (sizeof(T) == 2) {
        if (sums) {
            const bool mine = 32 * wave < kend, diagonal = 32 * wave == q0;
            floatx16 s, dp;
            float top = 0.f, bottom = 0.f;
            tiles_ready();
            if (mine) {
                s = X::rows_by(ks, 32 * wave, rows.q, lane);
                dp = X::rows_by(vs, 32 * wave, rows.dout, lane);
                rows.delta_parts(s, dp, c, diagonal, lane, top, bottom);
                top = halves_sum(top), bottom = halves_sum(bottom);
            }
            parts[wave][lane >> 5][lane & 31] = lane < 32 ? top : bottom;
            tiles_ready();
            const int row = lane & 31;
            top = bottom = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n) top += parts[n][0][row], bottom += parts[n][1][row];
            rows.set_delta(a, w, q0, top, bottom, wave == 0, lane);
            if (mine) {
                rows.turn(s, dp, c, diagonal, lane);
                X::columns_by(ks, 32 * wave, s, rows.dq, lane);
            }
        }
    }
    for (int64_t t = sums ? kend : 0; t < kend; t += 128) {
        const int64_t k0 = t + 32 * wave;
        const bool mine = k0 < kend, more = t + 128 < kend;
        floatx16 s, dp;
        tiles_ready_but<X::NLD>();
        if (mine) dp = X::rows_by(vs, 32 * wave, rows.dout, lane);
        tiles_ready();
        if (more) load_v(vs, t + 128, kend, wave);
        if (mine) {
            s = X::rows_by(ks, 32 * wave, rows.q, lane);
            rows.turn(s, dp, c, k0 == q0, lane);
            X::columns_by(ks, 32 * wave, s, rows.dq, lane);
        }
        __syncthreads();
        if (more) load_k(ks, t + 128, kend, wave);
    }
    join_sums<X::DB>((float*)ks, wave, lane, rows.dq);
    if (wave == 0) store_columns<T, X::DB>(rows.dq, a.scale, head_rows(a.dq, w, w.head, row_bytes), q0, w.len, lane);
}

// Scores of 32 query rows against the keys along the lanes become probabilities, and with the products of dout and
// the values ds.  lse (log2 units) and delta: of the rows; `diagonal`: the rows are the keys' own tokens.
__device__ __forceinline__ void soften(floatx16& s, const float* lse, float c, bool diagonal, int lane) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const floatx4 e = *(const floatx4*)(lse + 8 * n + 4 * (lane >> 5));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = fast_exp2(fmaf(s[4 * n + i], c, -e[i]));
            s[4 * n + i] = diagonal && acc_row(4 * n + i, lane >> 5) < (lane & 31) ? 0.f : x;
        }
    }
}
__device__ __forceinline__ void turn(floatx16& p, const floatx16& dp, const float* delta, bool diagonal, int lane) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const floatx4 e = *(const floatx4*)(delta + 8 * n + 4 * (lane >> 5));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = p[4 * n + i] * (dp[4 * n + i] - e[i]);
            p[4 * n + i] = diagonal && acc_row(4 * n + i, lane >> 5) < (lane & 31) ? 0.f : x;
        }
    }
}

// The first query head of part `split` of a key head's, and their number: parts differ by at most one head.
__device__ __forceinline__ int part_heads(const AttnArgs& a, int head, uint32_t split, int& number) {
    const uint32_t all = a.heads / a.kv_heads, from = split * all / a.splits, to = (split + 1) * all / a.splits;
    number = (int)(to - from);
    return head * (int)all + (int)from;
}

// 32 keys' dk and dv, as they are or as part `split` of what is added up by another launch.
template <typename T, int DB>
__device__ __forceinline__ void store_grads(const AttnArgs& a, const RowBlock& w, uint32_t split, const floatx16 (&dk)[DB],
                                            const floatx16 (&dv)[DB], int64_t k0, int lane) {
    const int row_bytes = a.dim * (int)sizeof(T);
    if (a.splits == 1) {
        store_columns<T, DB>(dk, a.scale, head_rows(a.dk, w, w.head, row_bytes), k0, w.len, lane);
        store_columns<T, DB>(dv, 1.f, head_rows(a.dv, w, w.head, row_bytes), k0, w.len, lane);
        return;
    }
    const int64_t tokens = a.cu ? a.L : a.b * a.L, first = a.cu ? w.start : w.seq * a.L;
    const uint32_t token = (uint32_t)a.kv_heads * a.dim * 4;
    char* p = (char*)a.part + (split * tokens + first) * token + w.head * a.dim * 4;
    const RowSource rk{p, token, a.dim * 4}, rv{p + a.splits * tokens * (int64_t)token, token, a.dim * 4};
    store_columns<float, DB>(dk, a.scale, rk, k0, w.len, lane);
    store_columns<float, DB>(dv, 1.f, rv, k0, w.len, lane);
}

// dk and dv: 32 keys to a wave and 128 (4 waves) or 256 (8) to a workgroup, the keys along the lanes; query rows and their
// gradients go by in tiles of 32 or 64, head after head of the group.
//
// Registers bound it: keys, dk and dv of 32 x 128 elements are 160 of the 256 that two waves to a SIMD have, so bf16 heads
// over 64 elements keep their values in LDS, a right operand that is read again for every tile.
template <typename T, int DC>
struct Grads {
    static constexpr bool V_LDS = sizeof(T) == 2 && DC > 64;
    using X = HeadTile<T, DC>;
    uint4 k[X::SG], v[V_LDS ? 1 : X::SG];
    floatx16 dk[X::DB] = {}, dv[X::DB] = {};

    // rows r0 .. r0 + 31 of a tile; OWN: they may be the keys' own tokens (`diagonal`)
    template <bool OWN>
    __device__ __forceinline__ void add(const char* Q, const char* D, const char* V, const float* lse, const float* delta,
                                        int r0, float c, bool diagonal, int wave, int lane) {
        // what follows from the lane is computed again for every tile: kept over the loop (with the values' rows, which
        // do not change either) it would not fit the registers
        asm volatile("" : "+v"(lane));
        floatx16 p = X::rows_by(Q, r0, k, lane), dp;
        if constexpr (V_LDS) dp = X::rows_by_rows(D, r0, V, 32 * wave, lane);
        else dp = X::rows_by(D, r0, v, lane);
        soften(p, lse + r0, c, OWN && diagonal, lane);
        X::columns_by(D, r0, p, dv, lane);
        turn(p, dp, delta + r0, OWN && diagonal, lane);
        X::columns_by(Q, r0, p, dk, lane);
    }
};

// dk, dv: 32 keys to a wave, whose two sums stay in registers over all rows and heads of the group; query and dout rows
// go by in LDS.  Bound by waiting: b8 L2048, 32/8 heads of 128 bf16, 8 waves, 670 us, matrix units busy 39% of the
// time, waves waiting 57% of theirs, without LDS conflicts; of 411 vector instructions to a tile of 64 rows 250 are
// addresses.
template <typename T, int DC, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 ? 2 : 1) void attn_dkv(const AttnArgs a) {
    using G = Grads<T, DC>;
    constexpr int KEYS = 32 * WAVES, ROWS = 8 * WAVES, N = 64 * WAVES;
    using X = HeadTile<T, DC, ROWS>;
    using Y = HeadTile<T, DC, KEYS>;
    __shared__ alignas(16) char qa[X::BYTES];
    __shared__ alignas(16) char qb[X::BYTES];
    __shared__ alignas(16) char da[X::BYTES];
    __shared__ alignas(16) char db[X::BYTES];
    __shared__ alignas(16) char vs[G::V_LDS ? Y::BYTES : 16];
    __shared__ alignas(16) float ra[2][ROWS];   // lse in log2 units, delta
    __shared__ alignas(16) float rb[2][ROWS];
    RowBlock w;
    const uint32_t split = blockIdx.x % a.splits;
    if (!locate_rows<KEYS, false>(a, a.kv_heads, blockIdx.x / a.splits, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int group;
    const int head0 = part_heads(a, w.head, split, group);
    const int row_bytes = a.dim * X::ES;
    const int64_t k0 = w.r0 + 32 * wave;
    const bool active = k0 < w.len;

    G grads;
    const TileLoad<X, N> load_q(head_rows(a.q, w, head0, row_bytes), tid);
    const TileLoad<X, N> load_d(head_rows(a.dout, w, head0, row_bytes), tid);
    // The first wave brings lse and delta of the tile's rows.  Without divergent branches, here and in all that
    // runs at the full number of registers: a compiler that has none to spare may put the copies that it splits
    // values with before the execution mask is whole again.
    auto load = [&](int h, int64_t r0, char* Q, char* D, float (&rows)[2][ROWS]) __attribute__((always_inline)) {
        TileLoad<X, N> lq = load_q, ld = load_d;
        lq.src.p += h * a.q.head;
        ld.src.p += h * a.dout.head;
        lq(Q, r0, w.len, wave);
        ld(D, r0, w.len, wave);
        if (wave == 0) {
            const int64_t at = token_row(a, w, head0 + h) + r0;
            const int left = (int)(w.len - r0 < ROWS ? w.len - r0 : ROWS), row = lane % ROWS;
            const float e = bits_to_f32(buffer_load_bits(make_rsrc(a.lse + at, left * 4), row * 4, 0.f)) * kLog2e;
            const float d = bits_to_f32(buffer_load_bits(make_rsrc(a.delta + at, left * 4), row * 4, 0.f));
            // rows that are not there: probabilities of 0
            if constexpr (ROWS == 32) {
                rows[lane >> 5][row] = lane >= 32 ? d : row < left ? e : 1e30f;
            } else {
                rows[0][row] = row < left ? e : 1e30f;
                rows[1][row] = d;
            }
        }
    };
    if constexpr (G::V_LDS) {
        const TileLoad<Y, N> load_v(head_rows(a.v, w, w.head, row_bytes), tid);
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
        auto turn = [&](const char* Q, const char* D, const float (&rows)[2][ROWS], char* next_q, char* next_d,
                        float (&next_rows)[2][ROWS]) __attribute__((always_inline)) {
            tiles_ready();
            const bool more = r0 + ROWS < to;
            const int64_t at = r0;
            r0 = more ? r0 + ROWS : from;
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
    const int64_t own = w.len < w.r0 + KEYS ? w.len : w.r0 + KEYS;
    run(w.r0, own, [&](int64_t r0, const char* Q, const char* D, const float (&rows)[2][ROWS]) __attribute__((always_inline)) {
#pragma unroll 1
        for (int n = 0; n < ROWS; n += 32)
            if (active && r0 + n >= k0) grads.template add<true>(Q, D, vs, rows[0], rows[1], n, c, r0 + n == k0, wave, lane);
    });
    run(own, w.len, [&](int64_t, const char* Q, const char* D, const float (&rows)[2][ROWS]) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < ROWS; n += 32) grads.template add<false>(Q, D, vs, rows[0], rows[1], n, c, false, wave, lane);
    });
    if (!active) return;
    store_grads<T>(a, w, split, grads.dk, grads.dv, k0, lane);
}

// For few keys: 32 of them to a workgroup, and the four parts of 32 rows of each tile of 128 to its waves, whose sums
// are joined at the end.  9 packed sequences of up to 1100, 12/4 heads of 96 fp32: 305 us.
template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 && DC <= 64 ? 2 : 1) void attn_dkv_few(const AttnArgs a) {
    using X = HeadTile<T, DC, 128>;
    __shared__ alignas(16) char qs[X::BYTES];
    __shared__ alignas(16) char ds[X::BYTES];
    __shared__ alignas(16) float rows[4][2][32];   // each wave's lse in log2 units, delta
    RowBlock w;
    const uint32_t split = blockIdx.x % a.splits;
    if (!locate_rows<kAttnFew, false>(a, a.kv_heads, blockIdx.x / a.splits, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    int group;
    const int head0 = part_heads(a, w.head, split, group);
    const int row_bytes = a.dim * X::ES;
    const int64_t k0 = w.r0;
    TileLoad<X> load_q(head_rows(a.q, w, head0, row_bytes), tid);
    TileLoad<X> load_d(head_rows(a.dout, w, head0, row_bytes), tid);
    const float c = a.scale * kLog2e;
    uint4 k[X::SG], v[X::SG];
    load_rows<X>(k, head_rows(a.k, w, w.head, row_bytes), k0, w.len, lane);
    load_rows<X>(v, head_rows(a.v, w, w.head, row_bytes), k0, w.len, lane);
    floatx16 dk[X::DB] = {}, dv[X::DB] = {};
    in_order();
    load_d(ds, k0, w.len, wave);
    in_order();
    load_q(qs, k0, w.len, wave);
    in_order();
    int64_t t = k0;
    for (int h = 0; h < group;) {
        const int64_t r0 = t + 32 * wave;
        const bool mine = r0 < w.len, last = t + 128 >= w.len, more = !last || h + 1 < group;
        const int head = head0 + h;
        t = last ? k0 : t + 128;
        if (last) {
            ++h;
            load_q.src.p += a.q.head;
            load_d.src.p += a.dout.head;
        }
        floatx16 p, dp;
        tiles_ready_but<X::NLD>();
        if (mine) dp = X::rows_by(ds, 32 * wave, v, lane);
        tiles_ready();
        if (mine) {
            p = X::rows_by(qs, 32 * wave, k, lane);
            const int64_t at = token_row(a, w, head) + r0;
            const int left = (int)(w.len - r0 < 32 ? w.len - r0 : 32);
            const float e = bits_to_f32(buffer_load_bits(make_rsrc(a.lse + at, left * 4), col * 4, 0.f)) * kLog2e;
            const float d = bits_to_f32(buffer_load_bits(make_rsrc(a.delta + at, left * 4), col * 4, 0.f));
            rows[wave][half][col] = half ? d : col < left ? e : 1e30f;
            __builtin_amdgcn_wave_barrier();
            soften(p, rows[wave][0], c, r0 == k0, lane);
            X::columns_by(ds, 32 * wave, p, dv, lane);
            turn(p, dp, rows[wave][1], r0 == k0, lane);
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();
        if (more) load_d(ds, t, w.len, wave);
        if (mine) X::columns_by(qs, 32 * wave, p, dk, lane);
        __syncthreads();
        if (more) load_q(qs, t, w.len, wave);
    }
    join_sums<X::DB>((float*)qs, wave, lane, dk);
    join_sums<X::DB>((float*)ds, wave, lane, dv);
    if (wave != 0) return;
    store_grads<T>(a, w, split, dk, dv, k0, lane);
}

// dk and dv out of the parts that the heads of a group were split into, 4 elements to a thread.
template <typename T>
__global__ __launch_bounds__(256) void attn_dkv_join(const AttnArgs a) {
    const int64_t tokens = a.cu ? a.L : a.b * a.L, quads = a.dim / 4, n = tokens * a.kv_heads * quads;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, i = e < n ? e : e - n;
    if (e >= 2 * n) return;
    const int d = (int)(i % quads) * 4, head = (int)(i / quads % a.kv_heads);
    const int64_t t = i / quads / a.kv_heads;
    if (a.cu && t >= packed_offset(a.cu, a.b, a.L)) return;
    const float* p = a.part + (e < n ? 0 : a.splits) * n * 4 + i * 4;
    floatx4 v = *(const floatx4*)p;
    for (int j = 1; j < a.splits; ++j) v += *(const floatx4*)(p + j * n * 4);
    const HeadRows& to = e < n ? a.dk : a.dv;
    char* at = to.p + head * to.head + d * (int)sizeof(T);
    at += a.cu ? t * to.token : t / a.L * to.batch + t % a.L * to.token;
    if constexpr (sizeof(T) == 2) *(uint2*)at = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else *(floatx4*)at = v;
}

template <typename T, int DC>
hipError_t launch_dim(AttnArgs a, hipStream_t s) {
    // bf16: two workgroups to a compute unit (4096 tokens, 16/8 heads of 128, backward 399 -> 393 us)
    a.paired = sizeof(T) == 2;
    const uint64_t b = a.cu ? 1 : a.b;
    const dim3 rows((uint32_t)(a.blocks * b * a.heads)), keys((uint32_t)(a.kblocks * b * a.kv_heads * a.splits));
    if (a.few) attn_dq_few<T, DC><<<rows, 256, 0, s>>>(a);
    else attn_dq<T, DC><<<rows, 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.paired = sizeof(T) == 2 && !a.kwide;
    if (a.kfew) attn_dkv_few<T, DC><<<keys, 256, 0, s>>>(a);
    else if (!a.kwide) attn_dkv<T, DC, 4><<<keys, 256, 0, s>>>(a);
    else if constexpr (Grads<T, DC>::V_LDS) attn_dkv<T, DC, 8><<<keys, 512, 0, s>>>(a);
    const hipError_t k = hipGetLastError();
    if (k != hipSuccess || a.splits == 1) return k;
    const int64_t quads = 2 * (a.cu ? a.L : a.b * a.L) * a.kv_heads * (a.dim / 4);
    attn_dkv_join<T><<<dim3((uint32_t)((quads + 255) / 256)), 256, 0, s>>>(a);
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
