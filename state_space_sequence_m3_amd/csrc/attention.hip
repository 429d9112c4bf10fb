// attention.hip -- causal attention over whole prompts (m3_attention).
//
// A workgroup of 4 waves takes 128 query rows of one head, a wave 32 of them, and walks over the keys in tiles that
// all four share in LDS, with the running maximum and sum of a softmax.  Scores are computed transposed (keys
// down, query rows along the lanes): a row's maximum and sum then are a lane's own registers and one exchange
// between the wave's halves, the probabilities are the right operand of the product with the values as they lie in
// their registers, and rescaling a row is one factor per lane.
#include "m3_attn_tile.h"

namespace m3 {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
// The running maximum (in log2 units) is moved only when a score exceeds it by more: until then
// probabilities are up to 2^8 larger, which costs no digits.
constexpr float kSlack = 8.f;

// One wave's 32 query rows.
template <typename T, int DC>
struct Rows {
    using X = HeadTile<T, DC>;
    uint4 q[X::SG];
    floatx16 o[X::DB] = {};
    float top = -1e37f, sum = 0.f;   // log2 units; this half's part of the sum

    // 32 keys at tile row r0; `diagonal`: they are the rows' own tokens
    __device__ __forceinline__ void add(const char* K, const char* V, int r0, float c, bool diagonal, int lane) {
        const int half = lane >> 5, row = lane & 31;
        floatx16 s = X::rows_by(K, r0, q, lane);
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = acc_row(i, half) > row ? -INFINITY : s[i];
        }
        float m = fmaxf(s[0], s[1]);
#pragma unroll
        for (int i = 2; i < 16; ++i) m = fmaxf(m, s[i]);
        m = fmaxf(m, other_half(m)) * c;
        if (__ballot(m > top + kSlack)) {
            const float to = fmaxf(top, m), f = fast_exp2(top - to);
#pragma unroll
            for (int db = 0; db < X::DB; ++db) o[db] *= f;
            sum *= f;
            top = to;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = fast_exp2(fmaf(s[i], c, -top));
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) part += s[i];
        sum += part;
        if (diagonal && any_odd(V, r0, lane)) {
            // key by key, each for the rows that see it
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
                float p = s[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) p = i == 4 * (j >> 3) + (j & 3) ? s[i] : p;
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
            X::columns_by(V, r0, s, o, lane);
        }
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

template <typename T, int DC>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void attn_fwd(const AttnArgs a) {
    using X = HeadTile<T, DC>;
    __shared__ alignas(16) char lds[2][2 * X::BYTES];
    RowBlock w;
    if (!locate_rows<true>(a, a.heads, blockIdx.x, w)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kv_head = w.head / (a.heads / a.kv_heads), row_bytes = a.dim * X::ES;
    const RowSource ks = head_rows(a.k, w, kv_head, row_bytes), vs = head_rows(a.v, w, kv_head, row_bytes);
    const int64_t q0 = w.r0 + 32 * wave;
    const bool active = q0 < w.len;

    Rows<T, DC> rows;
    load_rows<X>(rows.q, head_rows(a.q, w, w.head, row_bytes), q0, w.len, lane);
    const float c = a.scale * kLog2e;

    // tiles that all rows see, and those that hold the rows' own tokens
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
        for (int r0 = 0; r0 < X::ROWS; r0 += 32) rows.add(K, K + X::BYTES, r0, c, false, lane);
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
            if (active && k0 <= q0) rows.add(K, K + X::BYTES, r0, c, k0 == q0, lane);
        }
        if (t + 1 < ntiles) {
            kt.store(next, tid);
            vt.store(next + X::BYTES, tid);
        }
        __syncthreads();
    }
    if (!active) return;
    const float sum = rows.sum + other_half(rows.sum);
    store_columns<T, X::DB>(rows.o, 1.f / sum, head_rows(a.o, w, w.head, row_bytes), q0, w.len, lane);
    if (a.lse && lane < 32 && q0 + lane < w.len) {
        a.lse[token_row(a, w, w.head) + q0 + lane] = (rows.top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
}

template <typename T>
hipError_t launch_type(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)(a.blocks * (uint64_t)a.heads * (a.cu ? 1 : a.b)));
    if (a.dim <= 32) attn_fwd<T, 32><<<grid, 256, 0, s>>>(a);
    else if (a.dim <= 64) attn_fwd<T, 64><<<grid, 256, 0, s>>>(a);
    else if (a.dim <= 96) attn_fwd<T, 96><<<grid, 256, 0, s>>>(a);
    else attn_fwd<T, 128><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, bool bf16_io, hipStream_t s) {
    return bf16_io ? launch_type<bf16>(a, s) : launch_type<float>(a, s);
}

}  // namespace m3
