// m3_attn_tile.h -- tiles of head rows in LDS and the matrix products on them, shared by the attention kernels
// over whole prompts (forward and backward).
//
// All products are 32x32 result tiles.  Lane (c = lane % 32, h = lane / 32) holds of a result D, in
// register i = 0..15, row 8 (i / 4) + 4 h + i % 4 of column c.  An operand with its rows along the lanes takes 16
// bytes of row c at a time, the 16-byte chunk 2 g + h in step g (bf16: one product of depth 16; fp32: four of
// depth 2); which elements share a step does not matter as long as both operands agree.
//
// A result is used as the right operand of the next product without leaving its registers: of 32 rows of the
// result, lane half h holds those with (row / 4) % 2 == h, so the left operand's lanes of half h are given the
// tile rows of the same numbers (bf16: transposed reads of 4 rows; fp32: a row per step).
#pragma once

#include "attn_launch.h"
#include "m3_mma.h"
#include "m3_pages.h"

namespace m3 {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short shortx8 __attribute__((ext_vector_type(8)));

// row of result register i in lane half h
__device__ __forceinline__ constexpr int acc_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }
// over both halves of a column (v_permlane32_swap of a value with itself gives both halves')
__device__ __forceinline__ float halves_sum(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float halves_max(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// DC: elements of a head that are worked on (the head's own number rounded up to 32); T: io type; R: rows of a tile
template <typename T, int DC, int R = (sizeof(T) == 2 ? 64 : 32)>
struct HeadTile {
    static constexpr int ES = sizeof(T);
    static constexpr int PITCH = (DC <= 64 ? 64 : 128) * ES;   // bytes between rows
    static constexpr int CPR = PITCH / 16;                     // chunks per row
    static constexpr int ROWS = R;
    static constexpr int SUB = ROWS / 32;
    static constexpr int BYTES = ROWS * PITCH;
    static constexpr int SG = DC * ES / 32;                    // steps along a row
    static constexpr int DB = DC / 32;                         // result tiles across a row
    static constexpr int NLD = BYTES / 16 / 256;               // chunks each of 256 threads stages

    // Rows are a power of two apart, so the chunks of a row are exchanged by an exclusive or with the row's number:
    // 8 consecutive rows hold a chunk in 8 places (row reads), and the rows that transposed reads take together
    // lie in different quarters of the banks.
    static __device__ __forceinline__ int swz(int row) {
        if constexpr (ES == 4) return (((row >> 2) & 1) << 3) | ((row & 3) << 1);
        else if constexpr (CPR == 16) return ((row & 3) << 2) | ((row >> 2) & 3);
        else return (((row >> 1) & 1) << 2) | ((row >> 2) & 1) | (((row >> 3) & 1) << 1);
    }
    static __device__ __forceinline__ int at(int row, int chunk) { return row * PITCH + ((chunk ^ swz(row)) << 4); }

    // 16 bytes of a row
    static __device__ __forceinline__ uint4 row_chunk(const char* tile, int row, int chunk) {
        return *(const uint4*)(tile + at(row, chunk));
    }
    static __device__ __forceinline__ float element(const char* tile, int row, int d) {
        const char* p = tile + at(row, d * ES / 16) + (d * ES & 15);
        if constexpr (ES == 2) return to_f32(*(const bf16*)p);
        else return *(const float*)p;
    }

    static __device__ __forceinline__ floatx16 mma(uint4 a, uint4 b, floatx16 c) {
        if constexpr (ES == 2) {
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                           0, 0);
        } else {
            const floatx4 x = __builtin_bit_cast(floatx4, a), y = __builtin_bit_cast(floatx4, b);
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[0], y[0], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[1], y[1], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[2], y[2], c, 0, 0, 0);
            return __builtin_amdgcn_mfma_f32_32x32x2f32(x[3], y[3], c, 0, 0, 0);
        }
    }

    // the products of 16 bytes of two rows
    static __device__ __forceinline__ float dot(uint4 a, uint4 b) {
        float x[16 / ES], y[16 / ES], d = 0.f;
        unpack16(a, x, T{});
        unpack16(b, y, T{});
#pragma unroll
        for (int i = 0; i < 16 / ES; ++i) d = fmaf(x[i], y[i], d);
        return d;
    }

    // sum over a row's elements: result[tile row r0 + .., column c] of tile rows and the rows held in `b`
    static __device__ __forceinline__ floatx16 rows_by(const char* tile, int r0, const uint4 (&b)[SG], int lane) {
        floatx16 s = {};
#pragma unroll
        for (int g = 0; g < SG; ++g) s = mma(row_chunk(tile, r0 + (lane & 31), 2 * g + (lane >> 5)), b[g], s);
        return s;
    }

    // the same with the other rows in LDS too, from row b0 of tile `b` on
    static __device__ __forceinline__ floatx16 rows_by_rows(const char* tile, int r0, const char* b, int b0, int lane) {
        floatx16 s = {};
#pragma unroll
        for (int g = 0; g < SG; ++g)
            s = mma(row_chunk(tile, r0 + (lane & 31), 2 * g + (lane >> 5)),
                    row_chunk(b, b0 + (lane & 31), 2 * g + (lane >> 5)), s);
        return s;
    }

    // four elements of a column, tile rows r .. r + 3 with r = r0 + 4 h
    static __device__ __forceinline__ shortx4 column4(const char* tile, int r0, int db, int lane) {
        const int l16 = lane & 15, row = r0 + 4 * (lane >> 5) + (l16 >> 2);
        const int d = 32 * db + (lane & 16) + 4 * (l16 & 3);
        const char* p = tile + at(row, d >> 3) + (d & 4) * 2;
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4*)(lds_char*)p);
    }

    // acc[db][d, c] += sum over the 32 tile rows r of tile[r0 + r][32 db + d] * p[r, c]
    static __device__ __forceinline__ void columns_by(const char* tile, int r0, const floatx16& p, floatx16 (&acc)[DB],
                                                      int lane) {
        if constexpr (ES == 2) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint4 b;
                b.x = pack_bf16x2(p[8 * g], p[8 * g + 1]);
                b.y = pack_bf16x2(p[8 * g + 2], p[8 * g + 3]);
                b.z = pack_bf16x2(p[8 * g + 4], p[8 * g + 5]);
                b.w = pack_bf16x2(p[8 * g + 6], p[8 * g + 7]);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const shortx4 lo = column4(tile, r0 + 16 * g, db, lane), hi = column4(tile, r0 + 16 * g + 8, db, lane);
                    const shortx8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    acc[db] = mma(__builtin_bit_cast(uint4, a), b, acc[db]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const int row = r0 + acc_row(i, lane >> 5), d = 32 * db + (lane & 31);
                    const float a = *(const float*)(tile + at(row, d >> 2) + (d & 3) * 4);
                    acc[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p[i], acc[db], 0, 0, 0);
                }
        }
    }
};

// An offset that is past every descriptor's end (they cover less than 2^31 bytes).
constexpr uint32_t kOutside = 0x80000000u;

// Rows of one head: rows past `left` and chunks past the head's own are read as zero.
struct RowSource {
    const char* p;       // first row of the head
    uint32_t token;      // bytes between rows
    int row_bytes;
    // a descriptor that ends with row `len` - 1, from row r0 on, of at most `most` rows
    __device__ __forceinline__ rsrc_t rows(int64_t r0, int64_t len, int most) const {
        const int64_t left = len - r0 < most ? len - r0 : most;
        const uint32_t bytes = left > 0 ? (uint32_t)(left - 1) * token + (uint32_t)row_bytes : 0u;
        return make_rsrc(p + (left > 0 ? r0 : 0) * (int64_t)token, bytes);
    }
};

// What a workgroup works on: R rows of one head of one sequence.
struct RowBlock {
    int64_t seq, start, len;   // sequence; its first token on the packed axis (dense: 0); its tokens
    int head;
    int64_t r0;                // first row, in the sequence
};

// Of query rows (LAST_FIRST) or keys.  Dense batches: blocks of equal numbers run side by side over all heads, from the one with most work on (the last
// queries, the first keys), and an XCD's workgroups share the heads of a contiguous range, so that query heads of a key head meet in one L2.
// Packed ones: numbers that first_block's map leaves over have no rows.
template <int R, bool LAST_FIRST>
__device__ __forceinline__ bool locate_rows(const AttnArgs& a, int heads, uint32_t id, RowBlock& w) {
    const uint32_t blocks = LAST_FIRST ? a.blocks : a.kblocks;
    if (!a.cu) {
        const uint32_t pairs = (uint32_t)a.b * heads;
        if (a.paired) id = (uint32_t)paired_item(id, (int64_t)pairs * blocks);
        uint32_t pair, blk;
        if (pairs % kXcds == 0) {
            const uint32_t per = pairs / kXcds, r = id / kXcds;
            pair = (id % kXcds) * per + r % per;
            blk = r / per;
        } else {
            pair = id % pairs;
            blk = id / pairs;
        }
        if (LAST_FIRST) blk = blocks - 1 - blk;
        w.seq = pair / heads;
        w.head = (int)(pair % heads);
        w.start = 0;
        w.len = a.L;
        w.r0 = (int64_t)blk * R;
        return true;
    }
    w.head = (int)(id % heads);
    const uint32_t slot = LAST_FIRST ? blocks - 1 - id / heads : id / heads;
    // the last sequence whose first number is at most the slot
    const int64_t lo = last_at_most(a.b, slot, [&](int64_t s) { return first_block(packed_offset(a.cu, s, a.L), s, R); });
    w.seq = lo;
    w.start = packed_offset(a.cu, lo, a.L);
    w.len = packed_offset(a.cu, lo + 1, a.L) - w.start;
    w.r0 = ((int64_t)slot - first_block(w.start, lo, R)) * R;
    return w.r0 >= 0 && w.r0 < w.len;
}

__device__ __forceinline__ RowSource head_rows(const HeadRows& t, const RowBlock& w, int head, int row_bytes) {
    return {t.p + w.seq * t.batch + w.start * (int64_t)t.token + head * t.head, t.token, row_bytes};
}

// lse and delta have a row per head, over all tokens of the sequence or of the packed batch
__device__ __forceinline__ int64_t token_row(const AttnArgs& a, const RowBlock& w, int head) {
    return a.cu ? head * a.L + w.start : (w.seq * a.heads + head) * a.L;
}

// A tile from global memory straight into LDS, by N threads.  Lanes fill consecutive chunks of LDS, so each
// asks for the chunk that swz puts there; what the descriptor does not cover arrives as zero.  Buffers that are
// filled while others are read have to be arrays of their own: the compiler then knows that reads need not wait for
// the fill.  A wave knows of its own loads only: tiles_ready lets each wait for its own and then for the others.
typedef __attribute__((address_space(3))) void lds_void;
template <typename X, int N = 256>
struct TileLoad {
    static constexpr int STEP = N / X::CPR;   // rows that one load of all threads covers
    RowSource src;
    uint32_t off;
    __device__ __forceinline__ TileLoad(const RowSource& s, int tid) : src(s) {
        static_assert(STEP % 8 == 0, "swz has a period of 8 or 16 rows");
        const int row = tid / X::CPR, chunk = (tid % X::CPR) ^ X::swz(row);
        off = chunk * 16 < s.row_bytes ? (uint32_t)row * s.token + chunk * 16 : kOutside;
    }
    __device__ __forceinline__ void operator()(char* tile, int64_t r0, int64_t len, int wave) const {
        const rsrc_t r = src.rows(r0, len, X::ROWS);
#pragma unroll
        for (int i = 0; i < X::BYTES / 16 / N; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(tile + (i * (N / 64) + wave) * 1024), 16,
                                                     (int)(off + (uint32_t)(i * STEP) * src.token), 0, 0, 0);
    }
};

// All tiles asked for before are whole, and all reads of tiles before are done.
__device__ __forceinline__ void tiles_ready() {
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): loads into LDS count there
    __syncthreads();
}

// Loads asked for after it are issued after those before it, so that tiles_ready_but can tell them apart.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// tiles_ready for all but the last N loads of each wave.
template <int N>
__device__ __forceinline__ void tiles_ready_but() {
    static_assert(N < 64, "vmcnt has 6 bits");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4 << 14));
    __syncthreads();
}

// Adds up what the four waves of a workgroup hold for the same columns, into the first: `mine` is called with a place
// of N floats per lane to put its values to, `theirs` with one to take another wave's from.  The place is
// 2 * 64 * N floats of LDS that no tile needs any more.
template <int N, typename F, typename G>
__device__ __forceinline__ void join_waves(float* lds, int wave, int lane, F&& mine, G&& theirs) {
    float* at = lds + (wave >> 1) * 64 * N + lane;
    __syncthreads();
    if (wave & 1) mine(at);
    __syncthreads();
    if (!(wave & 1)) theirs(at);
    __syncthreads();
    if (wave == 2) mine(lds + lane);
    __syncthreads();
    if (wave == 0) theirs(lds + lane);
}

// The chunks 2 g + h of row (lane % 32), for use as a right operand.
template <typename X>
__device__ __forceinline__ void load_rows(uint4 (&f)[X::SG], const RowSource& s, int64_t r0, int64_t len, int lane) {
    const rsrc_t r = s.rows(r0, len, 32);
#pragma unroll
    for (int g = 0; g < X::SG; ++g) {
        const int chunk = 2 * g + (lane >> 5);
        f[g] = buffer_load16(r, chunk * 16 < s.row_bytes ? (uint32_t)(lane & 31) * s.token + chunk * 16 : kOutside);
    }
}

// Rows r0 .. r0 + 31 from a transposed result: column c (a row) has 4 consecutive elements in 4 registers.
template <typename T, int DB>
__device__ __forceinline__ void store_columns(const floatx16 (&acc)[DB], float factor, const RowSource& s, int64_t r0,
                                              int64_t len, int lane) {
    const rsrc_t r = s.rows(r0, len, 32);
    const uint32_t row = (uint32_t)(lane & 31) * s.token;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * db + 8 * i + 4 * (lane >> 5);
            const uint32_t off = d * (int)sizeof(T) < s.row_bytes ? row + d * (int)sizeof(T) : kOutside;
            const float a = acc[db][4 * i] * factor, b = acc[db][4 * i + 1] * factor;
            const float c = acc[db][4 * i + 2] * factor, e = acc[db][4 * i + 3] * factor;
            if constexpr (sizeof(T) == 2)
                buffer_store8(r, off, make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, e)));
            else
                buffer_store16(r, off, make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(e)));
        }
}

}  // namespace m3
