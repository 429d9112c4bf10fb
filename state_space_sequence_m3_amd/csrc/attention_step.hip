// attention_step.hip -- one token's attention per sequence over a paged cache (m3_attention_step).
//
// Memory-bound: each key and value is read once for the query heads that share it.  All sequences' keys, one after the
// other, are cut into equal pieces, so that the GPU is filled once whatever the lengths are; a piece is a
// workgroup's, whose 4 waves take the tiles of a sequence in turn, each with a running maximum and sum of its own, and what
// pieces hold of a sequence that is cut is joined by a second launch.
//
// Up to 16 query heads of a key head are the columns of 16x16 products.  Scores are computed transposed (keys down), with
// the keys in an order that makes a lane's probabilities those of 8 (fp32: 4) consecutive keys: the right operand of the
// product with the values, whose left operand is the values' rows as they are loaded, 16 lanes to a row, with (bf16) an
// 8 x 8 transpose inside each lane.  Nothing goes through LDS but the join of the waves.
//
// 32/8 heads of 128 bf16: 64 sequences of up to 8192 182 us and 6.6 for the join (5.4 TB/s over the call, 5.5 with pages of
// 16); one of 32768 26 and 4.7 us.  16 sequences of up to 8192, fp32: 106 us, 4.7 TB/s.
#include "m3_mma.h"
#include "m3_pages.h"
#include "m3_softmax.h"

namespace m3 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int64_t length_of(const StepArgs& a, int64_t s) {
    const int64_t n = a.lens[s], most = a.pages.table_w * (int64_t)a.pages.size;
    return n < 0 ? 0 : n > most ? most : n;
}
__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    return v;
}
// The keys of a piece.  first: the lane's of the first 64 rounded lengths.
__device__ __forceinline__ int64_t cut_batch(const StepArgs& a, int64_t& first) {
    const int64_t lane = threadIdx.x & 63;
    first = lane < a.b ? rounded_keys(length_of(a, lane)) : 0;
    int64_t all = first;
    for (int64_t s = lane + 64; s < a.b; s += 64) all += rounded_keys(length_of(a, s));
    return piece_keys(wave_sum(all), a.items);
}
// The sequence that key `at` of the batch belongs to (-1: there are fewer), and the keys before it.
__device__ __forceinline__ int64_t find_key(const StepArgs& a, int64_t first, int64_t at, int64_t& before) {
    const int lane = threadIdx.x & 63;
    before = 0;
    for (int64_t s0 = 0; s0 < a.b; s0 += 64) {
        const int64_t mine = s0 == 0 ? first : s0 + lane < a.b ? rounded_keys(length_of(a, s0 + lane)) : 0;
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t u = __shfl_up(upto, d, 64);
            if (lane >= d) upto += u;
        }
        const uint64_t past = __ballot(before + upto > at);
        if (past) {
            const int i = __ffsll((unsigned long long)past) - 1;
            before += __shfl(upto - mine, i, 64);
            return s0 + i;
        }
        before += __shfl(upto, 63, 64);
    }
    return -1;
}
// The keys before sequence s.
__device__ __forceinline__ int64_t keys_before(const StepArgs& a, int64_t first, int64_t s) {
    const int64_t lane = threadIdx.x & 63;
    int64_t n = lane < s ? first : 0;
    for (int64_t i = lane + 64; i < s; i += 64) n += rounded_keys(length_of(a, i));
    return wave_sum(n);
}

// DC: elements of a head that are worked on, 64 or 128.  TILED: a page holds whole tiles.
template <typename T, int DC, bool TILED>
struct Piece {
    static constexpr bool BF = sizeof(T) == 2;
    static constexpr int ES = sizeof(T);
    static constexpr int TILE = BF ? 32 : 16;        // keys
    static constexpr int BLK = TILE / 16;            // score blocks of 16 keys
    static constexpr int KS = DC * ES / 64;          // steps of 4 chunks along a row
    static constexpr int VE = DC / 16;               // a lane's elements of a value row
    static constexpr int VK = TILE / 4;              // a lane's value rows
    static constexpr int VW = VE * ES / 4;           // words of them

    uint4 k[BLK][KS];
    uint32_t v[VK][VW];
    uint32_t there;                                  // bits of the lane's score keys that exist

    // the key of score row r in block n
    static __device__ __forceinline__ int key_of(int r, int n) { return BF ? 8 * (r >> 2) + 4 * n + (r & 3) : r; }

    // Where a tile's keys are: the tile's page and place (TILED), or lane i's those of key i.
    struct Where {
        int id = -1, place = 0;
    };
    static __device__ __forceinline__ Where look(const StepArgs& a, const int32_t* table, int64_t k0, int64_t kend, int lane) {
        Where w;
        const int64_t k = TILED ? k0 : k0 + (lane & 31);
        if (k < kend && (TILED || (lane & 31) < TILE)) w.id = page_of(a.pages, table, (int32_t)k, w.place);
        return w;
    }

    __device__ __forceinline__ void load(const StepArgs& a, Where w, int kv_head, int64_t k0, int64_t kend, int lane) {
        const int r16 = lane & 15, g = lane >> 4, row_bytes = a.dim * ES;
        const Pages& p = a.pages;
        const int left = (int)(kend - k0 < TILE ? kend - k0 : TILE);
        const int vcol = r16 * VE * ES;
        if constexpr (TILED) {
            const int id = __builtin_amdgcn_readfirstlane(w.id), place = __builtin_amdgcn_readfirstlane(w.place);
            const int rows = id >= 0 ? left : 0;
            const int64_t at = id >= 0 ? id : 0;
            const rsrc_t kr = make_rsrc(p.k + at * p.k_page + kv_head * p.k_head + place * (int64_t)p.k_token,
                                        rows > 0 ? (uint32_t)(rows - 1) * p.k_token + row_bytes : 0u);
            const rsrc_t vr = make_rsrc(p.v + at * p.v_page + kv_head * p.v_head + place * (int64_t)p.v_token,
                                        rows > 0 ? (uint32_t)(rows - 1) * p.v_token + row_bytes : 0u);
#pragma unroll
            for (int n = 0; n < BLK; ++n)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int col = (4 * s + g) * 16;
                    k[n][s] = buffer_load16(kr, col < row_bytes ? (uint32_t)key_of(r16, n) * p.k_token + col : 0x80000000u);
                }
#pragma unroll
            for (int i = 0; i < VK; ++i) {
                const uint32_t off = vcol < row_bytes ? (uint32_t)(VK * g + i) * p.v_token + vcol : 0x80000000u;
                load_value(i, vr, off);
            }
            there = 0;
#pragma unroll
            for (int i = 0; i < 4 * BLK; ++i) there |= (VK * g + i < rows ? 1u : 0u) << i;
        } else {
            const int id = w.id, place = w.place;
#pragma unroll
            for (int n = 0; n < BLK; ++n) {
                const int key = key_of(r16, n), kid = __shfl(id, key, 64), kplace = __shfl(place, key, 64);
                const char* row = p.k + kid * p.k_page + kv_head * p.k_head + kplace * (int64_t)p.k_token;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int col = (4 * s + g) * 16;
                    k[n][s] = make_uint4(0, 0, 0, 0);
                    if (kid >= 0 && col < row_bytes) k[n][s] = *(const uint4*)(row + col);
                }
            }
            there = 0;
#pragma unroll
            for (int i = 0; i < VK; ++i) {
                const int key = VK * g + i, kid = __shfl(id, key, 64), kplace = __shfl(place, key, 64);
                const char* row = p.v + kid * p.v_page + kv_head * p.v_head + kplace * (int64_t)p.v_token + vcol;
                const bool ok = kid >= 0 && vcol < row_bytes;
#pragma unroll
                for (int w = 0; w < VW; w += (VW < 4 ? VW : 4)) {
                    if constexpr (VW == 2) {
                        const uint2 u = ok ? *(const uint2*)row : make_uint2(0, 0);
                        v[i][0] = u.x, v[i][1] = u.y;
                    } else {
                        const uint4 u = ok && vcol + 4 * w < row_bytes ? *(const uint4*)(row + 4 * w) : make_uint4(0, 0, 0, 0);
                        v[i][w] = u.x, v[i][w + 1] = u.y, v[i][w + 2] = u.z, v[i][w + 3] = u.w;
                    }
                }
                there |= (kid >= 0 ? 1u : 0u) << i;
            }
        }
    }
    __device__ __forceinline__ void load_value(int i, rsrc_t r, uint32_t off) {
        if constexpr (VW == 2) {
            const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
            v[i][0] = u[0], v[i][1] = u[1];
        } else {
#pragma unroll
            for (int w = 0; w < VW; w += 4) {
                const uint4 u = buffer_load16(r, off + 4 * w);
                v[i][w] = u.x, v[i][w + 1] = u.y, v[i][w + 2] = u.z, v[i][w + 3] = u.w;
            }
        }
    }

    // scores of the tile; key VK g + i in register i
    __device__ __forceinline__ void scores(const uint4 (&q)[KS], float (&s)[4 * BLK]) const {
#pragma unroll
        for (int n = 0; n < BLK; ++n) {
            floatx4 d = {};
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                if constexpr (BF) {
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[n][j]),
                                                                __builtin_bit_cast(bf16x8, q[j]), d, 0, 0, 0);
                } else {
                    d = Mma<float>::mma(__builtin_bit_cast(floatx4, k[n][j]), __builtin_bit_cast(floatx4, q[j]), d);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * n + i] = (there >> (4 * n + i)) & 1 ? d[i] : -INFINITY;
        }
    }
    // acc[j][m]: element (4 g + m) VE + j of the lane's query head
    __device__ __forceinline__ void values(const float (&p)[4 * BLK], floatx4 (&acc)[VE]) const {
        if constexpr (BF) {
            uint4 b;
            b.x = pack_bf16x2(p[0], p[1]);
            b.y = pack_bf16x2(p[2], p[3]);
            b.z = pack_bf16x2(p[4], p[5]);
            b.w = pack_bf16x2(p[6], p[7]);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
                uint4 t;
                t.x = __builtin_amdgcn_perm(v[1][j >> 1], v[0][j >> 1], sel);
                t.y = __builtin_amdgcn_perm(v[3][j >> 1], v[2][j >> 1], sel);
                t.z = __builtin_amdgcn_perm(v[5][j >> 1], v[4][j >> 1], sel);
                t.w = __builtin_amdgcn_perm(v[7][j >> 1], v[6][j >> 1], sel);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, t), __builtin_bit_cast(bf16x8, b),
                                                                 acc[j], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[m][j]), p[m], acc[j], 0, 0, 0);
        }
    }
};

// Partial results: of each part (piece + sequence) the heads one after another, {largest score, sum, D unscaled elements}
// each.  A largest score of -infinity: there is no position (where all score -infinity it is kLowest, and the sum 0).
__device__ __forceinline__ int64_t part_row(const StepArgs& a, int64_t part, int head) {
    return (part * a.heads + head) * (2 + a.dim);
}

template <typename T, int DC, bool TILED>
__global__ __launch_bounds__(256, 2) void attn_step(const StepArgs a) {
    using P = Piece<T, DC, TILED>;
    constexpr int VE = P::VE, STEP = 4 * P::TILE;
    __shared__ float tops[4][16], sums[4][16];
    __shared__ float outs[4][16][DC + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int hb = blockIdx.x % a.head_blocks, kv_head = blockIdx.x / a.head_blocks % a.kv_heads;
    const int64_t item = blockIdx.x / a.head_blocks / a.kv_heads;
    const int group = a.heads / a.kv_heads, in_group = hb * 16 + col;
    const int heads_here = group - hb * 16 < 16 ? group - hb * 16 : 16;
    const float c = a.scale * kLog2e;
    int64_t first, start;
    const int64_t keys = cut_batch(a, first), lo = item * keys;
    int64_t s = find_key(a, first, lo, start);
    if (s < 0) return;

    while (true) {
        // keys k0 .. kend - 1 of sequence s, which starts at `start`
        const int64_t len = length_of(a, s), stop = start + rounded_keys(len);
        const int64_t k0 = lo > start ? lo - start : 0;
        const int64_t kend = lo + keys < start + len ? lo + keys - start : len;
        const int32_t* table = a.pages.table + s * a.pages.table_w;
        const int head = kv_head * group + in_group;

        uint4 q[P::KS];
#pragma unroll
        for (int j = 0; j < P::KS; ++j) {
            const int at = (4 * j + g) * 16;
            q[j] = make_uint4(0, 0, 0, 0);
            if (in_group < group && at < a.dim * P::ES) q[j] = *(const uint4*)(a.q.p + s * a.q.batch + head * a.q.head + at);
        }
        floatx4 acc[VE] = {};
        float top = kLowest, sum = 0.f;
        bool some = false;   // a position, for all of the wave

        // keys and values are loaded a tile ahead, and looked up two
        P now, next;
        int64_t k = k0 + wave * P::TILE;
        typename P::Where ahead = P::look(a, table, k + STEP, kend, lane);
        if (k < kend) now.load(a, P::look(a, table, k, kend, lane), kv_head, k, kend, lane);
        for (; k < kend; k += STEP) {
            const typename P::Where far = P::look(a, table, k + 2 * STEP, kend, lane);
            if (k + STEP < kend) next.load(a, ahead, kv_head, k + STEP, kend, lane);
            ahead = far;
            float p[4 * P::BLK];
            now.scores(q, p);
            some |= __ballot(now.there) != 0;
            float m = p[0];
#pragma unroll
            for (int i = 1; i < 4 * P::BLK; ++i) m = fmaxf(m, p[i]);
            m = fmaxf(m, __shfl_xor(m, 16, 64));
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            if (__ballot(m > top)) {
                const float to = fmaxf(top, m), f = top_moved(top, to, c);
#pragma unroll
                for (int j = 0; j < VE; ++j) acc[j] *= f;
                sum *= f;
                top = to;
            }
            float by = c, base = top * c;
            if (__ballot(!(fabsf(base) < kFar))) {
                by = score_factor(top, c);
                base = top * by;
            }
#pragma unroll
            for (int i = 0; i < 4 * P::BLK; ++i) {
                p[i] = fast_exp2(fmaf(p[i], by, -base));
                sum += p[i];
            }
            now.values(p, acc);
            now = next;
        }
        sum += __shfl_xor(sum, 16, 64);
        sum += __shfl_xor(sum, 32, 64);

        // the four waves' results
        __syncthreads();
        if (g == 0) {
            tops[wave][col] = some ? top : -INFINITY;
            sums[wave][col] = sum;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < VE; ++j) outs[wave][col][(4 * g + m) * VE + j] = acc[j][m];
        __syncthreads();
        const bool whole = start >= lo && stop <= lo + keys;
        for (int e = threadIdx.x; e < heads_here * a.dim; e += 256) {
            const int h = e / a.dim, d = e % a.dim, at = kv_head * group + hb * 16 + h;
            const float t = fmaxf(fmaxf(tops[0][h], tops[1][h]), fmaxf(tops[2][h], tops[3][h]));
            float n = 0.f, o = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = top_moved(tops[w][h], t, c);
                n = fmaf(f, sums[w][h], n);
                o = fmaf(f, outs[w][h][d], o);
            }
            if (whole) {
                // nothing to attend to: zeros
                *(T*)(a.o.p + s * a.o.batch + at * a.o.head + d * P::ES) = from_f32<T>(t > -INFINITY ? o / n : 0.f);
                if (a.lse && d == 0) a.lse[s * a.heads + at] = log_sum(t, n, c);
            } else {
                float* part = a.part + part_row(a, item + s, at);
                part[2 + d] = o;
                if (d == 0) part[0] = t, part[1] = n;
            }
        }
        if (stop >= lo + keys || ++s >= a.b) return;
        start = stop;
    }
}

// Joins the parts of one head of one sequence: 16 groups of 16 lanes take a part each at a time, 8 elements to a lane.
template <typename T>
__global__ __launch_bounds__(256) void attn_step_join(const StepArgs a) {
    __shared__ float outs[16][128 + 8];
    __shared__ float tops[16], sums[16];
    const int64_t s = blockIdx.x / a.heads;
    const int head = (int)(blockIdx.x % a.heads);
    int64_t first;
    const int64_t keys = cut_batch(a, first), start = keys_before(a, first, s);
    const int64_t own = s < 64 ? __shfl(first, (int)s, 64) : rounded_keys(length_of(a, s));
    const int64_t item = start / keys, n = (start + own - 1) / keys - item + 1;
    if (n <= 1) return;
    const float* part = a.part + part_row(a, item + s, head);
    const int64_t next = (int64_t)a.heads * (2 + a.dim);   // from a part to the next one
    const int tid = threadIdx.x, group = tid >> 4, d0 = (tid & 15) * 8;
    const float c = a.scale * kLog2e;
    float o[8] = {}, top = -INFINITY, sum = 0.f;
    for (int64_t i = group; i < n; i += 16) {
        const float* p = part + i * next;
        const float t = p[0], w = p[1];
        float x[8] = {};
        if (d0 < a.dim) {   // rows of 2 + dim floats: pairs are aligned
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 u = *(const float2*)(p + 2 + d0 + j);
                x[j] = u.x, x[j + 1] = u.y;
            }
        }
        const float to = fmaxf(top, t), f = top_moved(top, to, c), g = top_moved(t, to, c);
        top = to;
        sum = sum * f + w * g;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = o[j] * f + x[j] * g;
    }
    if (d0 < a.dim) {
#pragma unroll
        for (int j = 0; j < 8; ++j) outs[group][d0 + j] = o[j];
    }
    if (d0 == 0) tops[group] = top, sums[group] = sum;
    __syncthreads();
    if (tid < a.dim) {
        float t = tops[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) t = fmaxf(t, tops[i]);
        float v = 0.f, w = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float f = top_moved(tops[i], t, c);
            w = fmaf(f, sums[i], w);
            v = fmaf(f, outs[i][tid], v);
        }
        // nothing to attend to: zeros
        *(T*)(a.o.p + s * a.o.batch + head * a.o.head + tid * (int)sizeof(T)) =
            from_f32<T>(t > -INFINITY ? v / w : 0.f);
        if (a.lse && tid == 0) a.lse[s * a.heads + head] = log_sum(t, w, c);
    }
}

template <typename T, int DC>
hipError_t launch_dim(const StepArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)(a.items * a.kv_heads * a.head_blocks));
    if (a.pages.size % Piece<T, DC, true>::TILE == 0) attn_step<T, DC, true><<<grid, 256, 0, s>>>(a);
    else attn_step<T, DC, false><<<grid, 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.joined) return e;
    attn_step_join<T><<<dim3((uint32_t)(a.b * a.heads)), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_step(const StepArgs& a, bool bf16_io, hipStream_t s) {
    if (bf16_io) return a.dim <= 64 ? launch_dim<bf16, 64>(a, s) : launch_dim<bf16, 128>(a, s);
    return a.dim <= 64 ? launch_dim<float, 64>(a, s) : launch_dim<float, 128>(a, s);
}

}  // namespace m3
