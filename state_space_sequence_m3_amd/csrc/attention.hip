// attention.hip -- causal attention over whole prompts (m3_attention).
//
// A workgroup of 4 waves takes 128 query rows of one head, a wave 32 of them, and walks over the keys in tiles that
// all four share in LDS, with the running maximum and sum of a softmax.  Scores are computed transposed (keys
// down, query rows along the lanes): a row's maximum and sum then are a lane's own registers and one exchange
// between the wave's halves, the probabilities are the right operand of the product with the values as they lie in
// their registers, and rescaling a row is one factor per lane.
#include "m3_attn_tile.h"
#include "m3_softmax.h"

namespace m3 {
namespace {

// The running maximum is moved only when a score exceeds it by more (in log2 units): until then probabilities are up to
// 2^8 larger, which costs no digits.  Less than half a unit in the last place of a maximum of kFar, so that it is
// nothing there.
constexpr float kSlack = 7.9f;

// One wave's 32 query rows.
template <typename T, int DC>
struct Rows {
    using X = HeadTile<T, DC>;
    uint4 q[X::SG];
    floatx16 o[X::DB] = {};
    float top = kLowest, sum = 0.f;   // this half's part of the sum
    float by;                         // score_factor of top

    __device__ __forceinline__ explicit Rows(float c) : by(score_factor(kLowest, c)) {}

    // makes room for scores against 32 N keys: the running maximum is their bound within kSlack
    template <int N>
    __device__ __forceinline__ void raise(const floatx16 (&s)[N], float c, float slack) {
        float m = s[0][0];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, s[n][i]);
        m = halves_max(m);
        if (__ballot(m > top + slack)) {
            const float to = fmaxf(top, m), f = top_moved(top, to, c);
#pragma unroll
            for (int db = 0; db < X::DB; ++db) o[db] *= f;
            sum *= f;
            top = to;
            by = score_factor(to, c);
        }
    }
    // they become probabilities
    template <int N>
    __device__ __forceinline__ void soften(floatx16 (&s)[N]) {
        const float base = top * by;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[n][i] = fast_exp2(fmaf(s[n][i], by, -base));
                part += s[n][i];
            }
            sum += part;
        }
    }

    // 32 keys at tile row r0 that are the rows' own tokens (`diagonal`), or earlier ones
    __device__ __forceinline__ void add(const char* K, const char* V, int r0, float c, float slack, bool diagonal, int lane) {
        floatx16 s[1] = {X::rows_by(K, r0, q, lane)};
        add_scores(s, V, r0, c, slack, diagonal, lane);
    }
    __device__ __forceinline__ void add_scores(floatx16 (&s)[1], const char* V, int r0, float c, float slack, bool diagonal,
                                               int lane) {
        const int half = lane >> 5, row = lane & 31;
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[0][i] = acc_row(i, half) > row ? -INFINITY : s[0][i];
        }
        raise(s, c, slack);
        soften(s);
        if (diagonal && any_odd(V, r0, lane)) {
            // key by key, each for the rows that see it
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
                float p = s[0][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) p = i == 4 * (j >> 3) + (j & 3) ? s[0][i] : p;
                p = __shfl(p, row + 32 * ((j >> 2) & 1), 64);
                if (j <= row) {
#pragma unroll
                    for (int db = 0; db < X::DB; ++db)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[db][i] = fmaf(p, X::element(V, r0 + j, 32 * db + acc_row(i, half)), o[db][i]);
                }
            }
        } else {
            X::columns_by(V, r0, s[0], o, lane);
        }
    }

    __device__ __forceinline__ void finish(const AttnArgs& a, const RowBlock& w, int64_t q0, int row_bytes, float c, int lane) {
        const float all = halves_sum(sum);
        store_columns<T, X::DB>(o, 1.f / all, head_rows(a.o, w, w.head, row_bytes), q0, w.len, lane);
        if (a.lse && lane < 32 && q0 + lane < w.len)
            a.lse[token_row(a, w, w.head) + q0 + lane] = log_sum(top, all, c);
    }

    // A probability of 0 times an infinity or NaN in a later token's value would be NaN: the values of the one block
    // that holds later tokens are looked over.
    static __device__ __forceinline__ bool any_odd(const char* V, int r0, int lane) {
        constexpr int per = DC * X::ES / 16;
        bool odd = false;
#pragma unroll 1
        for (int e = lane; e < 32 * per; e += 64) {
            const uint4 u = X::row_chunk(V, r0 + e / per, e % per);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                odd |= (x[n] & 0x7f800000u) == 0x7f800000u;
                if constexpr (X::ES == 2) odd |= (x[n] & 0x7f80u) == 0x7f80u;
            }
        }
        return __ballot(odd) != 0;
    }
};

// Bound by how far two waves to a SIMD cover each other's softmax, LDS reads and barriers: at b8 L2048, 32/8 heads of 128
// bf16, 327 us (840 TFLOP/s of the causal half), the matrix units are busy 45% of the time, vector units 51%, LDS 23%, and
// waves wait 32% of theirs.  8192 tokens, 32/4 heads of 64: 309 us, vector units 84%, matrix units 51%.
template <typename T, int DC, int PER_CU>
__global__ __launch_bounds__(256, PER_CU) void attn_fwd(const AttnArgs a) {
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
    const int64_t q0 = w.r0 + 32 * wave;
    const bool active = q0 < w.len;

    // tiles that all rows see, and those that hold the rows' own tokens
    const int before = (int)(w.r0 / X::ROWS);
    const int64_t kend = w.len < w.r0 + kAttnRows ? w.len : w.r0 + kAttnRows;
    const int ntiles = (int)((kend + X::ROWS - 1) / X::ROWS);
    load_k(k0, 0, w.len, wave);
    load_v(v0, 0, w.len, wave);
    if (ntiles > 1) load_k(k1, X::ROWS, w.len, wave);

    const float c = a.scale * kLog2e, slack = kSlack / c;
    Rows<T, DC> rows(c);
    load_rows<X>(rows.q, head_rows(a.q, w, w.head, row_bytes), q0, w.len, lane);

    // Tile t's keys are in k0 (t even) or k1, its values in v0 or v1.  Scores of tile t + 1 are computed while tile
    // t's become probabilities, keys are loaded two tiles ahead and values one.
    floatx16 s[X::SUB], ahead[X::SUB];
    tiles_ready();
    if (before > 0) {
#pragma unroll
        for (int n = 0; n < X::SUB; ++n) s[n] = X::rows_by(k0, 32 * n, rows.q, lane);
    }
    auto turn = [&](int t, const char* K, char* old_k, const char* V, char* old_v) __attribute__((always_inline)) {
        tiles_ready();
        if (t + 2 < ntiles) load_k(old_k, (int64_t)(t + 2) * X::ROWS, w.len, wave);
        load_v(old_v, (int64_t)(t + 1) * X::ROWS, w.len, wave);
        rows.raise(s, c, slack);
        // a wave with products to issue goes first: 340 -> 334 us at b8 L2048, 32/8 heads of 128 bf16, 73 -> 69 for 2 x 2048,
        // 32/16 heads of 96; 16 x 512, 32/8 heads of 128 loses, 74 -> 78
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < X::SUB; ++n) ahead[n] = X::rows_by(K, 32 * n, rows.q, lane);
        rows.soften(s);
        // (no pragma: unrolled at once, this takes registers that are not there)
        for (int n = 0; n < X::SUB; ++n) X::columns_by(V, 32 * n, s[n], rows.o, lane);
        __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int n = 0; n < X::SUB; ++n) s[n] = ahead[n];
    };
    // before is even: 128 rows are an even number of tiles
    for (int t = 0; t < before; t += 2) {
        turn(t, k1, k0, v0, v1);
        turn(t + 1, k0, k1, v1, v0);
    }
    for (int t = before; t < ntiles; ++t) {
        const bool odd = t & 1;
        tiles_ready();
        if (t + 1 < ntiles) {
            if (t > before) load_k(odd ? k0 : k1, (int64_t)(t + 1) * X::ROWS, w.len, wave);
            load_v(odd ? v0 : v1, (int64_t)(t + 1) * X::ROWS, w.len, wave);
        }
#pragma unroll 1
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) {
            const int64_t at = (int64_t)t * X::ROWS + r0;
            if (active && at <= q0) rows.add(odd ? k1 : k0, odd ? v1 : v0, r0, c, slack, at == q0, lane);
        }
    }
    if (active) rows.finish(a, w, q0, row_bytes, c, lane);
}

// For few rows: a workgroup takes 32 query rows, and its waves the four parts of 32 keys of each tile of 128, with a
// softmax of their own each, which are joined at the end.  Keys are loaded while probabilities meet values, values
// while queries meet keys.  64 tokens, 32/8 heads of 128 bf16: 8.4 us, latency; 13 packed prompts of up to 701, 6/2 heads
// of 80 fp32: 83 us, matrix units 33% busy.
template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_fwd_few(const AttnArgs a) {
    using X = HeadTile<T, DC, 128>;
    using R = Rows<T, DC>;
    __shared__ alignas(16) char ks[X::BYTES];
    __shared__ alignas(16) char vs[X::BYTES];
    RowBlock w;
    if (!locate_rows<kAttnFew, true>(a, a.heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kv_head = w.head / (a.heads / a.kv_heads), row_bytes = a.dim * X::ES;
    const TileLoad<X> load_k(head_rows(a.k, w, kv_head, row_bytes), tid);
    const TileLoad<X> load_v(head_rows(a.v, w, kv_head, row_bytes), tid);
    const int64_t q0 = w.r0, kend = w.len < q0 + kAttnFew ? w.len : q0 + kAttnFew;
    const float c = a.scale * kLog2e, slack = kSlack / c;
    R rows(c);
    load_rows<typename R::X>(rows.q, head_rows(a.q, w, w.head, row_bytes), q0, w.len, lane);
    in_order();
    load_k(ks, 0, kend, wave);
    in_order();
    load_v(vs, 0, kend, wave);
    in_order();
    for (int64_t t = 0; t < kend; t += 128) {
        const int64_t k0 = t + 32 * wave;
        const bool mine = k0 < kend, more = t + 128 < kend;
        tiles_ready_but<X::NLD>();
        floatx16 s[1];
        if (mine) s[0] = R::X::rows_by(ks, 32 * wave, rows.q, lane);
        tiles_ready();
        if (more) load_k(ks, t + 128, kend, wave);
        if (mine) rows.add_scores(s, vs, 32 * wave, c, slack, k0 == q0, lane);
        __syncthreads();
        if (more) load_v(vs, t + 128, kend, wave);
    }
    static_assert(2 * 64 * 16 * X::DB * 4 <= X::BYTES, "two waves' values fit a tile");
    __shared__ float ends[2][2][64];
    float* const end = &ends[wave >> 1][0][lane];
    join_waves<16 * X::DB>((float*)ks, wave, lane,
        [&](float* at) __attribute__((always_inline)) {
            float* e = wave == 2 ? &ends[0][0][lane] : end;
            e[0] = rows.top, e[64] = rows.sum;
#pragma unroll
            for (int db = 0; db < X::DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) at[(db * 16 + i) * 64] = rows.o[db][i];
        },
        [&](float* at) __attribute__((always_inline)) {
            const float to = fmaxf(rows.top, end[0]), f = top_moved(rows.top, to, c), g = top_moved(end[0], to, c);
            rows.top = to;
            rows.sum = rows.sum * f + end[64] * g;
#pragma unroll
            for (int db = 0; db < X::DB; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) rows.o[db][i] = rows.o[db][i] * f + at[(db * 16 + i) * 64] * g;
        });
    if (wave == 0) rows.finish(a, w, q0, row_bytes, c, lane);
}

// Two workgroups to a compute unit, heavy with light ones (paired_item).  Fp32 heads of up to 96 elements fit too, but
// only dense batches have an order to pair by: 4096 tokens, 16 heads of 64 415 -> 313 us, 2 x 2048, 32 heads of 96 504 ->
// 437 us; 9 packed sequences, with backward, 662 -> 700 us.
template <typename T, int DC>
void launch_dim(AttnArgs a, hipStream_t s) {
    const dim3 grid((uint32_t)(a.blocks * (uint64_t)a.heads * (a.cu ? 1 : a.b)));
    constexpr int FIT = sizeof(T) == 2 || DC <= 96 ? 2 : 1;
    a.paired = FIT == 2 && (sizeof(T) == 2 || !a.cu);
    if (a.few) {
        a.paired = 0;
        attn_fwd_few<T, DC><<<grid, 256, 0, s>>>(a);
    } else if (a.paired) {
        attn_fwd<T, DC, FIT><<<grid, 256, 0, s>>>(a);
    } else if constexpr (sizeof(T) == 4) {
        attn_fwd<T, DC, 1><<<grid, 256, 0, s>>>(a);
    }
}
template <typename T>
hipError_t launch_type(const AttnArgs& a, hipStream_t s) {
    if (a.dim <= 32) launch_dim<T, 32>(a, s);
    else if (a.dim <= 64) launch_dim<T, 64>(a, s);
    else if (a.dim <= 96) launch_dim<T, 96>(a, s);
    else launch_dim<T, 128>(a, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, bool bf16_io, hipStream_t s) {
    return bf16_io ? launch_type<bf16>(a, s) : launch_type<float>(a, s);
}

}  // namespace m3
