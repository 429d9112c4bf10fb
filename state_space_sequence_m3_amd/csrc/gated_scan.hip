// gated_scan.hip -- per-channel gated linear recurrence  h_t = (1 - z_t) h_{t-1} + z_t x_t,
// z_t = sigmoid(gate_t + bias), forward, backward and for single tokens.
//
// A run of steps is the affine map h -> A h + B with A the product of (1 - z_t) and B the run's
// end from a zero state, and maps compose: (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2).  A
// sequence's first token forgets what came before: its map is h -> B (A = 0), with B taking the
// carried h_in in.  Tiles of a sequence run at the same time and are joined by a single-pass scan with decoupled
// look-back (Merrill and Garland, 2016).
//
// Bound: memory.  A forward pass reads gate and x and writes y, a backward pass reads gate, x and dy and writes
// dgate and dx; the arithmetic (an exponential, a reciprocal and some fifteen more per element) hides behind that.  So
// every element travels once: a workgroup takes a tile of 128 tokens (backward 64) x 128 channels, each of its 8
// waves 16 (8) consecutive tokens, two channels to a lane, all in registers from the load to the store; the waves'
// maps are composed through shared memory, the tiles' through a chain of words in the workspace, and the tokens are
// then run once more from registers.  b8 L2048 D4096 bf16, calls with all their launches: 403 MB in 86 us, 4.7 TB/s,
// backward 671 MB in 155 us, 4.3 TB/s (a copy of that size: 5.3 to 5.5 TB/s); fp32 141 us, 5.7 TB/s, and 251 us, 5.3
// TB/s.  What is left: 5 us for the launch that resets the chain, 5 us for taking tiles in order, and waits for the
// chain: one sequence of 16384 tokens takes 93 us, where a copy of its bytes takes 76.
// Here and at the constants below, times of alternatives are from the build that each was compared in.
// Shapes, b8 L2048 D4096 fp32 unless said: 4 waves to a tile of 64 tokens 160 us, 16 waves to one of 256 170 us;
// fp32 in tiles of 64 tokens 111 us instead of 100 (13 packed sequences); a backward tile of 128 tokens spills
// (bf16 420 us); workgroups that stay and fetch the next tile ahead 110 us (bf16), backward 433 us; gates computed
// again for the second run instead of held 107 us (bf16).
#include "block_launch.h"
#include "m3_device.h"

namespace m3 {
namespace {

constexpr int kWaves = 8;          // waves per tile; each holds as many consecutive tokens in registers
constexpr int kFwdSteps = kScanTile / kWaves, kBwdSteps = kScanBwdTile / kWaves;
// Sequences whose tiles are taken in turns: b8 L2048 D4096 bf16 82 us, backward 144; 1: 88, 154, 2: 86, 148; 8: 82,
// 143, but 16 x 1024 fp32 backward 254 -> 272.
constexpr uint32_t kSideBySide = 4;
constexpr int kWavesPerSimd = 4;   // two workgroups on a compute unit: 128 registers.  3 waves: 126 us for 94, 5: 98
constexpr uint32_t kFar = 56;      // chain words looked at, at most: 1 KB of shared memory each

// z = sigmoid(u) and keep = 1 - z, u = gate + bias, both to a few units in their last place: with e = e^-|u| the larger
// of the two is 1 / (1 + e) and the smaller one e / (1 + e), never a difference from 1.  The rounding of u log2(e) is
// carried along.  For bf16 gates, too: their logits are added in fp32 like any other, since the sum is close to exact
// where gate and bias cancel (one fused product with log2(e) on top of a rounded bias log2(e) was up to 100 units off
// there, 140 elsewhere).
// The reciprocal takes a Newton step: the hardware's errs to one side, by up to a step, which adds up over
// a recurrence of many tokens (fp32 gradient of a bias over 12000 tokens 7e-7 off, with the step 3e-7, as the formula in
// torch's fp32; bf16 forward 84.7 -> 86 us at b8 L2048 D4096, 76 -> 81 at 16 x 1024 tokens with the carried
// rounding's share, fp32 and backward the same).
constexpr float kLog2eLo = 1.925963033500e-8f;   // log2(e) - kLog2e
__device__ __forceinline__ void gate_of(float g, float bias, float& z, float& keep) {
    const float u = g + bias, m = -fabsf(u), t = m * kLog2e;
    const float rest = fmaf(m, kLog2e, -t) + m * kLog2eLo;
    float e = fast_exp2(t);
    e = t < -126.f ? e : fmaf(e, rest * 0.6931471805599453f, e);
    const float d = 1.f + e;
    float big = __builtin_amdgcn_rcpf(d);
    big = fmaf(big, fmaf(-d, big, 1.f), big);
    const float small = e * big;
    const bool up = u >= 0.f;
    z = up ? big : small;
    keep = up ? small : big;
}
// Two channels of one token per lane.  VEC: neighbours 2 lane, 2 lane + 1 in one access; else lane and
// lane + 64, element by element.  Rows are addressed through a descriptor of the tile's first row, a
// lane's byte offset in the row and the row's scalar offset: no vector arithmetic, and a lane offset of
// kNowhere (beyond the descriptor's 2^31 bytes) reads zero and stores nothing.
constexpr uint32_t kNowhere = 0xfffffff0u;
// Inputs are read once: non-temporal, which leaves the caches to y's rows and the chain (b8 L2048 D4096 bf16:
// forward 94 -> 89 us, backward 170 -> 158 us; no difference seen on small batches).
constexpr int kStream = 2;
__device__ __forceinline__ rsrc_t rows_at(const void* base, int64_t bytes) {
    return make_rsrc((const char*)base + bytes, 0x80000000u);
}
template <typename T, bool VEC> struct Pair;
template <> struct Pair<float, true> {
    u32x2 v;
    __device__ __forceinline__ void zero() { v = (u32x2){0, 0}; }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v)); }
    __device__ __forceinline__ void load(rsrc_t r, uint32_t o0, uint32_t, int row) {
        v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)o0, row, kStream);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v.y : v.x); }
};
template <> struct Pair<bf16, true> {
    uint32_t v;
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v)); }
    __device__ __forceinline__ void load(rsrc_t r, uint32_t o0, uint32_t, int row) {
        v = __builtin_amdgcn_raw_buffer_load_b32(r, (int)o0, row, kStream);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
};
template <> struct Pair<float, false> {
    uint32_t v[2];
    __device__ __forceinline__ void zero() { v[0] = v[1] = 0; }
    __device__ __forceinline__ void hide() {
        asm volatile("" : "+v"(v[0]));
        asm volatile("" : "+v"(v[1]));
    }
    __device__ __forceinline__ void load(rsrc_t r, uint32_t o0, uint32_t o1, int row) {
        v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)o0, row, kStream);
        v[1] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)o1, row, kStream);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i]); }
};
template <> struct Pair<bf16, false> {
    uint16_t v[2];
    __device__ __forceinline__ void zero() { v[0] = v[1] = 0; }
    __device__ __forceinline__ void hide() {
        asm volatile("" : "+v"(v[0]));
        asm volatile("" : "+v"(v[1]));
    }
    __device__ __forceinline__ void load(rsrc_t r, uint32_t o0, uint32_t o1, int row) {
        v[0] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)o0, row, kStream);
        v[1] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)o1, row, kStream);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float((uint32_t)v[i] << 16); }
};

// Makes the compiler unpack rows again from here on, where it would carry the elements in registers.
template <int N, typename T, bool VEC>
__device__ __forceinline__ void forget(Pair<T, VEC> (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i].hide();
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_pair(rsrc_t r, uint32_t o0, uint32_t o1, int row, float v0, float v1) {
    if constexpr (VEC && sizeof(T) == 2) {
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(v0, v1), r, (int)o0, row, 0);
    } else if constexpr (VEC) {
        __builtin_amdgcn_raw_buffer_store_b64((u32x2){__float_as_uint(v0), __float_as_uint(v1)}, r, (int)o0, row, 0);
    } else if constexpr (sizeof(T) == 2) {
        __builtin_amdgcn_raw_buffer_store_b16(bf16_bits_rne(v0), r, (int)o0, row, 0);
        __builtin_amdgcn_raw_buffer_store_b16(bf16_bits_rne(v1), r, (int)o1, row, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v0), r, (int)o0, row, 0);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v1), r, (int)o1, row, 0);
    }
}

// Where a lane's two channels are.
template <typename T, bool VEC>
struct Cols {
    int d[2];           // channels, possibly past D
    bool ok[2];
    uint32_t off[2];    // byte offsets in a row, kNowhere past D
    __device__ __forceinline__ Cols(int col, int lane, int64_t D) {
        d[0] = col * kScanCols + (VEC ? 2 * lane : lane);
        d[1] = d[0] + (VEC ? 1 : 64);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            ok[v] = d[v] < D;
            off[v] = ok[v] ? (uint32_t)d[v] * (uint32_t)sizeof(T) : kNowhere;
        }
    }
};

// First token of sequence s (s = b: the end of the last one).  Packed offsets are clamped to
// [0, T], so that offsets that break the rules cannot lead out of the buffers.
__device__ __forceinline__ int64_t seq_start(const GatedScanArgs& a, int64_t s) {
    if (a.cu == nullptr) return s * a.L;
    const int64_t v = a.cu[s];
    return v < 0 ? 0 : (v > a.T ? a.T : v);
}
// Tokens that belong to sequences: those behind the last one, or without any, are left as they are.
__device__ __forceinline__ int64_t tokens_of(const GatedScanArgs& a) { return a.b > 0 ? seq_start(a, a.b) : 0; }
// The sequence that holds token t: the last one that starts at or before t (empty sequences at
// the same place come before it).
__device__ __forceinline__ int64_t seq_of(const GatedScanArgs& a, int64_t t) {
    if (a.cu == nullptr) return t / a.L;
    int64_t lo = 0, hi = a.b - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (seq_start(a, mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A tile's place: tokens [t0, t0 + nv) of sequence seq (FLAT: of any), its number, and the tiles of the
// same chain before and after it.
struct Tile {
    int64_t t0;
    uint32_t c, seq, before, after;
    int link;        // the number of the tile after it in its chain is c + link
    int nv;
};
__device__ __forceinline__ uint32_t uniform32(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

template <int TILE, bool FLAT, bool SERIAL>
__device__ __forceinline__ Tile tile_of(const GatedScanArgs& a, uint32_t c) {
    Tile t;
    t.c = c;
    int64_t left;
    if constexpr (!FLAT) {
        // Chained: kTogether sequences side by side, tile by tile, then the next ones: of the tiles that run at
        // the same time fewer belong to one chain.  Serial: sequence by sequence.
        constexpr uint32_t kTogether = SERIAL ? 1 : kSideBySide;
        const uint32_t n = a.seq_tiles, group = uniform32(c / (kTogether * n)), r = c - group * (kTogether * n);
        const uint32_t left_over = (uint32_t)a.b - group * kTogether, size = left_over < kTogether ? left_over : kTogether;
        const uint32_t j = uniform32(r / size);
        t.seq = group * kTogether + (r - j * size);
        t.link = (int)size;
        t.t0 = (int64_t)t.seq * a.L + (int64_t)j * TILE;
        left = a.L - (int64_t)j * TILE;
        t.before = j;
        t.after = a.seq_tiles - 1 - j;
    } else {
        t.seq = 0;
        t.link = 1;
        t.t0 = (int64_t)c * TILE;
        left = tokens_of(a) - t.t0;
        t.before = c;
        t.after = (uint32_t)a.ntiles - 1 - c;
    }
    t.nv = (int)(left < 0 ? 0 : (left < TILE ? left : TILE));
    return t;
}
// the row of `states` that token 0 of the tile starts from
template <int TILE, bool FLAT>
__device__ __forceinline__ uint32_t state_row(const GatedScanArgs& a, const Tile& t) {
    return (FLAT ? 0 : t.seq * a.seq_blocks) + t.before * (TILE / kScanBlock);
}

// FLAT: which tokens start or end a sequence.  Every token's sequence is searched once, by the launch that
// resets the chain; a lone tile's, which has no such launch, by the tile itself, one thread per token.
struct Place {
    int seq;
    bool start, end;
};
__device__ __forceinline__ Place place_of(const GatedScanArgs& a, int64_t t) {
    const int64_t s = seq_of(a, t);
    return {(int)s, seq_start(a, s) == t, seq_start(a, s + 1) == t + 1};
}
template <int TILE>
struct Marks {
    int seq[TILE];                                     // the sequence of each token
    uint64_t starts[(TILE + 63) / 64], ends[(TILE + 63) / 64];
};
template <int TILE>
__device__ __forceinline__ void find_marks(const GatedScanArgs& a, const Tile& tile, Marks<TILE>& m) {
    const int i = threadIdx.x;
    if (i < TILE) {
        Place p = {0, false, false};
        if (i < tile.nv) {
            p = place_of(a, tile.t0 + i);
            m.seq[i] = p.seq;
        }
        const uint64_t ms = __ballot(p.start), me = __ballot(p.end);
        if ((i & 63) == 0) {
            m.starts[i >> 6] = ms;
            m.ends[i >> 6] = me;
        }
    }
    __syncthreads();
}
// N of a mask's bits, from token i of the tile on
template <int N>
__device__ __forceinline__ uint32_t mark_bits(const uint64_t* m, int i) {
    return uniform32((uint32_t)(m[i / 64] >> (i % 64))) & ((1u << N) - 1);
}
// ------------------------------------------------------------------------------ chain words
// Tiles of one sequence are chained through 64-bit words, one per tile and channel, each written
// whole by one relaxed agent-scope store (so a word is its own flag and needs no fence): low half
// A, high half B of the tile's map.  A with its sign bit set (-0) marks a final word: B is the state
// after the tile, whatever came before it.  All ones: not written yet.
constexpr uint32_t kUnset = 0xffffffffu, kFinal = 0x80000000u;

__device__ __forceinline__ uint64_t map_word(float A, float B) {
    const uint32_t bits = A != A ? 0x7fc00000u : __float_as_uint(A);
    return ((uint64_t)__float_as_uint(B) << 32) | bits;
}
__device__ __forceinline__ uint64_t final_word(float B) { return ((uint64_t)__float_as_uint(B) << 32) | kFinal; }
__device__ __forceinline__ void put_word(uint64_t* p, uint64_t w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

constexpr int kMaxReads = 1 << 22;    // some seconds: a wait that long means a workspace in use twice

// The state that enters a tile whose neighbour in the chain is `first`, the one after that
// first + step, and so on for `links` tiles.  It starts from the nearest final word and applies
// the maps after it in order.  A tile's own final word is made by the same steps, so the value
// does not depend on which word was found final.  Words are read one by one, the next only while all
// so far are maps: reads beyond the final word cost more than they save where many channels keep it near
// (b8 L2048 D4096 bf16: one at a time 83 us, backward 143; four 88, 151), and where few channels
// leave many tiles of one chain running at once it is far (b1 L65536 D256 bf16: up to 4 words 147 us,
// backward 282; up to 16: 75, 131; up to 56: 57, 92).  Ends: workgroups take tiles from a counter in chain order, so
// every tile waited for here is held by a workgroup that runs (or is done) and itself waits for
// earlier ones only; the first tile of a chain waits for none.  A wait of kMaxReads words gives NaN.
template <uint32_t N>
struct FarWords {
    uint64_t w[N][2][64];
};
__device__ __forceinline__ void chain_wait(const uint64_t* words, int64_t stride, int64_t first, int64_t step,
                                           uint32_t links, const int (&d)[2], int lane, FarWords<kFar>& far,
                                           float (&carry)[2]) {
    auto apply = [](uint64_t w, float h) {
        const float B = __uint_as_float((uint32_t)(w >> 32));
        return (uint32_t)w == kFinal ? B : fmaf(__uint_as_float((uint32_t)w), h, B);
    };
    const uint32_t most = links < kFar ? links : kFar;
#pragma unroll 1
    for (int reads = 0; reads < kMaxReads; ++reads) {
        bool found[2] = {false, false}, maps[2] = {true, true};   // a final word; only maps so far
#pragma unroll 1
        for (uint32_t n = 0; n < most; ++n, ++reads) {
            const char* row = (const char*)(words + (first + (int64_t)n * step) * stride);
            uint64_t w[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) w[v] = get_word((const uint64_t*)(row + (uint32_t)d[v] * 8u));
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                found[v] = found[v] || (maps[v] && (uint32_t)w[v] == kFinal);
                maps[v] = maps[v] && (uint32_t)w[v] != kFinal && (uint32_t)w[v] != kUnset;
            }
            if (__all(found[0] && found[1])) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    float h = apply(w[v], 0.f);
#pragma unroll 4
                    for (int k = (int)n - 1; k >= 0; --k) h = apply(far.w[k][v][lane], h);
                    carry[v] = h;
                }
                return;
            }
            if (!__all((found[0] || maps[0]) && (found[1] || maps[1]))) break;
#pragma unroll
            for (int v = 0; v < 2; ++v) far.w[n][v][lane] = w[v];
        }
        __builtin_amdgcn_s_sleep(1);
    }
    carry[0] = carry[1] = __uint_as_float(0x7fc00000u);
}

// Before a chained launch: the words unset, the counter at 0, and (flat) the tokens' marks.
__global__ __launch_bounds__(256) void chain_reset_kernel(const GatedScanArgs a, int64_t n16) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += step)
        ((uint4*)a.words)[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    if (a.per_seq) return;
    const int64_t total = tokens_of(a);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (a.T + 63) / 64 * 64; i += step) {   // whole waves
        Place p = {0, false, false};
        if (i < total) {
            p = place_of(a, i);
            a.seqs[i] = p.seq;
        }
        const uint64_t ms = __ballot(p.start), me = __ballot(p.end);
        if ((i & 63) == 0) {
            a.starts[i >> 6] = ms;
            a.ends[i >> 6] = me;
        }
    }
}

// ---------------------------------------------------------------------------------- forward
// Chained tiles: a workgroup's tile and column come from a counter, so that tiles are begun in chain order
// whatever order workgroups start in.  The lowest tile that is not done is then always held by a
// workgroup that waits for nothing.
__device__ __forceinline__ bool take_item(const GatedScanArgs& a, unsigned& s_ticket, uint32_t& c, int& col) {
    if (threadIdx.x == 0) s_ticket = atomicAdd(a.ticket, 1u);
    __syncthreads();
    const uint32_t item = uniform32(s_ticket);
    if (item >= (uint32_t)a.ntiles * (uint32_t)a.ncols) return false;
    c = uniform32(item / (uint32_t)a.ncols);
    col = (int)(item - c * (uint32_t)a.ncols);
    return true;
}

// N rows of pitch `pitch`, of which nv exist: rows past the last one read the last one again.
template <int N, typename T, bool VEC>
__device__ __forceinline__ void load_rows(Pair<T, VEC> (&r)[N], rsrc_t base, int pitch, int nv,
                                          const Cols<T, VEC>& cols) {
    int row = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        r[i].load(base, cols.off[0], cols.off[1], row);
        row += i + 1 < nv ? pitch : 0;
    }
}
__device__ __forceinline__ int clamp_rows(int left, int n) { return left < 0 ? 0 : (left < n ? left : n); }

// the values of sequence seq in a [b, D] tensor, 0 without one
template <typename T, bool VEC>
__device__ __forceinline__ void from_seq(const float* p, int64_t seq, int64_t D, const Cols<T, VEC>& cols,
                                         float (&o)[2]) {
#pragma unroll
    for (int v = 0; v < 2; ++v) o[v] = p && cols.ok[v] ? p[seq * D + cols.d[v]] : 0.f;
}
template <typename T, bool VEC>
__device__ __forceinline__ void to_seq(float* p, int64_t seq, int64_t D, const Cols<T, VEC>& cols, const float (&o)[2]) {
#pragma unroll
    for (int v = 0; v < 2; ++v)
        if (cols.ok[v]) p[seq * D + cols.d[v]] = o[v];
}
// Empty sequences pass `from` (0 without one) through to `to`.  512 sequences to a tile at a time, every 8th of
// them to a wave, one to a lane to find the empty ones, which are then copied four at a time.
template <typename T, bool VEC>
__device__ __forceinline__ void pass_empty(const GatedScanArgs& a, uint32_t c, const Cols<T, VEC>& cols, int lane, int w,
                                           const float* from, float* to) {
    if (a.cu == nullptr && a.L != 0) return;
    for (int64_t s0 = (int64_t)c * (64 * kWaves); s0 < a.b; s0 += a.ntiles * (64 * kWaves)) {
        const int64_t mine = s0 + lane * kWaves + w;
        uint64_t empty = __ballot(mine < a.b && !(seq_start(a, mine + 1) > seq_start(a, mine)));
        while (empty != 0) {
            int64_t s[4];
            float v[4][2];
            int n = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[k] = s0 + (empty ? __builtin_ctzll(empty) : 0) * kWaves + w;
                n += empty != 0 ? 1 : 0;
                empty &= empty - 1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) from_seq(k < n ? from : nullptr, s[k], a.D, cols, v[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < n) to_seq(to, s[k], a.D, cols, v[k]);
        }
    }
}
// The sequences of a wave's N tokens, one to a lane (FLAT), so that they are read once and together.
template <int N, bool FLAT, bool SERIAL>
__device__ __forceinline__ int seqs_of(const GatedScanArgs& a, const int* marks, int64_t tw, int lane, int w, int nv) {
    const int i = min(lane & (N - 1), nv - 1);
    if constexpr (!FLAT) return 0;
    else if constexpr (SERIAL) return marks[w * N + i];
    else return a.seqs[tw + i];
}

template <typename T, bool FLAT, bool SERIAL>
struct FwdShared {
    float2 sA[kWaves][64], sB[kWaves][64], sCarry[64];
    int sHard[kWaves];   // bit 0: the wave's tokens hold a sequence start; bit 1: its first token is one
    Marks<FLAT && SERIAL ? kWaves * kFwdSteps : 1> marks;
    FarWords<SERIAL ? 1 : kFar> far;
    unsigned sTicket;
};

// One tile.  SERIAL: `state`, the last wave's, is the state before the tile, and then the one after it; else it
// comes from the chain.
template <typename T, bool VEC, bool FLAT, bool SERIAL>
__device__ __forceinline__ void forward_tile(const GatedScanArgs& a, FwdShared<T, FLAT, SERIAL>& sh, uint32_t c, int col,
                                             int lane, int w, float (&state)[2]) {
    constexpr int N = kFwdSteps, TILE = kWaves * N;
    const Tile tile = tile_of<TILE, FLAT, SERIAL>(a, c);
    const Cols<T, VEC> cols(col, lane, a.D);
    const int64_t tw = tile.t0 + w * N;
    const int nv = clamp_rows(tile.nv - w * N, N);
    float keep[N][2], add[N][2];               // h <- keep h + add
    float bias[2];
    from_seq(a.bias, 0, 0, cols, bias);
    uint32_t starts = 0, ends = 0;
    {
        Pair<T, VEC> g[N], x[N];
        if (nv > 0) {
            load_rows(g, rows_at(a.gate, tw * a.gate_p), (int)a.gate_p, nv, cols);
            load_rows(x, rows_at(a.x, tw * a.x_p), (int)a.x_p, nv, cols);
        }
        if constexpr (FLAT && SERIAL) {
            find_marks(a, tile, sh.marks);
            starts = mark_bits<N>(sh.marks.starts, w * N);
            ends = mark_bits<N>(sh.marks.ends, w * N);
        } else if constexpr (FLAT) {
            if (nv > 0) {
                starts = mark_bits<N>(a.starts + tile.t0 / 64, w * N);
                ends = mark_bits<N>(a.ends + tile.t0 / 64, w * N);
            }
        } else {                               // a sequence's first and last token
            if (w == 0 && tile.before == 0) starts = 1;
            if (tile.after == 0 && nv > 0 && w * N + nv == tile.nv) ends = 1u << (nv - 1);
        }
        if (nv > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    float z;
                    gate_of(g[i].get(v), bias[v], z, keep[i][v]);
                    add[i][v] = z * x[i].get(v);
                }
        }
    }
    if (nv < N) {                              // tokens that are not there: keep = 1, nothing added
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= nv) {
                keep[i][0] = keep[i][1] = 1.f;
                add[i][0] = add[i][1] = 0.f;
            }
    }
    const int ids = (starts | ends) != 0 ? seqs_of<N, FLAT, SERIAL>(a, sh.marks.seq, tw, lane, w, nv) : 0;
    auto seq_at = [&](int i) -> int64_t {
        if constexpr (FLAT) return __builtin_amdgcn_readlane(ids, i);
        else return tile.seq;
    };
    auto first = [&](int i) { return (FLAT || i == 0) && ((starts >> i) & 1) != 0; };
    if (starts != 0 && a.h_in) {               // the states that sequences start from are in their first tokens' `add`
        constexpr int K = FLAT ? 8 : 1;        // as many are read together
#pragma unroll
        for (int i = 0; i < (FLAT ? N : 1); i += K) {
            float h0[K][2];
#pragma unroll
            for (int k = 0; k < K; ++k) from_seq(a.h_in, seq_at(i + k), a.D, cols, h0[k]);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (first(i + k)) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) add[i + k][v] = fmaf(keep[i + k][v], h0[k][v], add[i + k][v]);
                }
        }
    }
    float A[2] = {1.f, 1.f}, B[2] = {0.f, 0.f};   // the wave's map
    auto step = [&](int i, float (&h)[2]) {
#pragma unroll
        for (int v = 0; v < 2; ++v) h[v] = first(i) ? add[i][v] : fmaf(keep[i][v], h[v], add[i][v]);
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int v = 0; v < 2; ++v) A[v] = first(i) ? 0.f : A[v] * keep[i][v];
        step(i, B);
    }
    sh.sA[w][lane] = make_float2(A[0], A[1]);
    sh.sB[w][lane] = make_float2(B[0], B[1]);
    if (lane == 0) sh.sHard[w] = (starts != 0 ? 1 : 0) | (starts & 1 ? 2 : 0);
    __syncthreads();
    // the map of the waves before this one
    float Ap[2] = {1.f, 1.f}, Bp[2] = {0.f, 0.f};
    bool hard = false;                         // a start among them: what came before does not matter
    auto compose = [&](int k) {
        const float2 A = sh.sA[k][lane], B = sh.sB[k][lane];
        if (uniform32(sh.sHard[k]) & 1) {
            hard = true;
            Ap[0] = Ap[1] = 0.f;
            Bp[0] = B.x;
            Bp[1] = B.y;
        } else {
            Ap[0] *= A.x;
            Ap[1] *= A.y;
            Bp[0] = fmaf(A.x, Bp[0], B.x);
            Bp[1] = fmaf(A.y, Bp[1], B.y);
        }
    };
    for (int k = 0; k < w; ++k) compose(k);
    if (w == kWaves - 1) {                     // the last one does the chaining
        const float A0[2] = {Ap[0], Ap[1]}, B0[2] = {Bp[0], Bp[1]};
        const bool hard0 = hard;
        float carry[2] = {0.f, 0.f};
        compose(w);
        if constexpr (SERIAL) {
            const bool starts_here = (uniform32(sh.sHard[0]) & 2) != 0;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                carry[v] = starts_here ? 0.f : state[v];
                state[v] = hard ? Bp[v] : fmaf(Ap[v], carry[v], Bp[v]);
            }
        } else {
            const int64_t stride = (int64_t)a.ncols * kScanCols;
            uint64_t* mine = a.words + c * stride;
#pragma unroll
            for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], hard ? final_word(Bp[v]) : map_word(Ap[v], Bp[v]));
            const bool starts_here = (uniform32(sh.sHard[0]) & 2) != 0;
            if (tile.before > 0 && tile.nv > 0 && !starts_here) {
                const int64_t step = -tile.link;
                chain_wait(a.words, stride, c + step, step, tile.before, cols.d, lane, sh.far, carry);
            }
            if (!hard) {
#pragma unroll
                for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], final_word(fmaf(Ap[v], carry[v], Bp[v])));
            }
        }
        sh.sCarry[lane] = make_float2(carry[0], carry[1]);
        Ap[0] = A0[0]; Ap[1] = A0[1];
        Bp[0] = B0[0]; Bp[1] = B0[1];
        hard = hard0;
    }
    __syncthreads();
    float h[2];
    {
        const float2 cy = sh.sCarry[lane];
        h[0] = hard ? Bp[0] : fmaf(Ap[0], cy.x, Bp[0]);
        h[1] = hard ? Bp[1] : fmaf(Ap[1], cy.y, Bp[1]);
    }
    if (a.states && nv > 0 && w * N % kScanBlock == 0)
        to_seq(a.states, (int64_t)state_row<TILE, FLAT>(a, tile) + w * N / kScanBlock, a.D, cols, h);
    const rsrc_t yr = rows_at(a.y, tw * a.y_p);
    int row = 0;
    if (nv == N && (starts | ends) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int v = 0; v < 2; ++v) h[v] = fmaf(keep[i][v], h[v], add[i][v]);
            store_pair<T, VEC>(yr, cols.off[0], cols.off[1], row, h[0], h[1]);
            row += (int)a.y_p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i < nv) {
                step(i, h);
                store_pair<T, VEC>(yr, cols.off[0], cols.off[1], row, h[0], h[1]);
                row += (int)a.y_p;
                if ((ends >> i) & 1) to_seq(a.h_out, seq_at(i), a.D, cols, h);
            }
        }
    }
    if (FLAT) pass_empty(a, c, cols, lane, w, a.h_in, a.h_out);
}

// SERIAL: a workgroup takes one sequence (FLAT: the whole batch) tile by tile: no chain to wait for, none to
// reset.  For chains so short, or sequences so many, that the tiles need not run at the same time.
template <typename T, bool VEC, bool FLAT, bool SERIAL>
__global__ __launch_bounds__(kWaves * 64, kWavesPerSimd) void gated_scan_kernel(const GatedScanArgs a) {
    __shared__ FwdShared<T, FLAT, SERIAL> sh;
    const int lane = threadIdx.x & 63;
    const int w = uniform32(threadIdx.x >> 6);
    float state[2] = {0.f, 0.f};
    if constexpr (SERIAL) {
        const uint32_t seq = uniform32(blockIdx.x / (uint32_t)a.ncols), n = FLAT ? (uint32_t)a.ntiles : a.seq_tiles;
        const int col = (int)(blockIdx.x - seq * (uint32_t)a.ncols);
        for (uint32_t j = 0; j < n; ++j) {
            if (j > 0) __syncthreads();        // the tile before is done with the shared memory
            forward_tile<T, VEC, FLAT, true>(a, sh, seq * n + j, col, lane, w, state);
        }
    } else {
        uint32_t c;
        int col;
        if (take_item(a, sh.sTicket, c, col)) forward_tile<T, VEC, FLAT, false>(a, sh, c, col, lane, w, state);
    }
}

// --------------------------------------------------------------------------------- backward
// With G_t = (1 - z_t) l_t, what flows from token t to h_{t-1}: l_t = dy_t + G_{t+1}, so backwards
// G_t = keep_t G_{t+1} + keep_t dy_t, an affine map again, and the same chain in the other
// direction.  A sequence's last token takes dh_out for G_{t+1}.
template <typename T, bool FLAT, bool SERIAL>
struct BwdShared {
    float2 sA[kWaves][64], sB[kWaves][64], sRA[kWaves][64], sRB[kWaves][64], sCarry[64];
    int sHard[kWaves];   // bit 0: holds a sequence start; 1: holds an end; 2: its last token is an end
    Marks<FLAT && SERIAL ? kWaves * kBwdSteps : 1> marks;
    FarWords<SERIAL ? 1 : kFar> far;
    unsigned sTicket;
};

// One tile.  SERIAL: `state`, the first wave's, is what flows in from behind the tile, and then what flows out
// of it; else it comes from the chain.  `sum`: the wave's share of dbias grows.
template <typename T, bool VEC, bool FLAT, bool SERIAL>
__device__ __forceinline__ void backward_tile(const GatedScanArgs& a, BwdShared<T, FLAT, SERIAL>& sh, uint32_t c, int col,
                                              int lane, int w, float (&state)[2], float (&sum)[2]) {
    constexpr int N = kBwdSteps, TILE = kWaves * N;
    const Tile tile = tile_of<TILE, FLAT, SERIAL>(a, c);
    const Cols<T, VEC> cols(col, lane, a.D);
    const int64_t tw = tile.t0 + w * N;
    const int nv = clamp_rows(tile.nv - w * N, N);
    Pair<T, VEC> x[N], dy[N];
    float z[N][2], keep[N][2];
    float bias[2], h[2];
    from_seq(a.bias, 0, 0, cols, bias);
    from_seq(a.states, state_row<TILE, FLAT>(a, tile), a.D, cols, h);
    uint32_t starts = 0, ends = 0;
    {
        Pair<T, VEC> g[N];
        if (nv > 0) {
            load_rows(g, rows_at(a.gate, tw * a.gate_p), (int)a.gate_p, nv, cols);
            load_rows(x, rows_at(a.x, tw * a.x_p), (int)a.x_p, nv, cols);
            load_rows(dy, rows_at(a.dy, tw * a.y_p), (int)a.y_p, nv, cols);
        }
        if constexpr (FLAT && SERIAL) {
            find_marks(a, tile, sh.marks);
            starts = mark_bits<N>(sh.marks.starts, w * N);
            ends = mark_bits<N>(sh.marks.ends, w * N);
        } else if constexpr (FLAT) {
            if (nv > 0) {
                starts = mark_bits<N>(a.starts + tile.t0 / 64, w * N);
                ends = mark_bits<N>(a.ends + tile.t0 / 64, w * N);
            }
        } else {                               // a sequence's first and last token
            if (w == 0 && tile.before == 0) starts = 1;
            if (tile.after == 0 && nv > 0 && w * N + nv == tile.nv) ends = 1u << (nv - 1);
        }
        if (nv > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) gate_of(g[i].get(v), bias[v], z[i][v], keep[i][v]);
        }
    }
    if (nv < N) {                              // tokens that are not there: keep = 1, nothing added
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= nv) {
                z[i][0] = z[i][1] = 0.f;
                keep[i][0] = keep[i][1] = 1.f;
                x[i].zero();
                dy[i].zero();
            }
    }
    const int ids = (starts | ends) != 0 ? seqs_of<N, FLAT, SERIAL>(a, sh.marks.seq, tw, lane, w, nv) : 0;
    auto seq_at = [&](int i) -> int64_t {
        if constexpr (FLAT) return __builtin_amdgcn_readlane(ids, i);
        else return tile.seq;
    };
    auto first = [&](int i) { return (FLAT || i == 0) && ((starts >> i) & 1) != 0; };
    auto last = [&](int i) { return ((ends >> i) & 1) != 0; };
    // the rows of p that belong to the tokens' sequences, read together
    auto at_marks = [&](const float* p, float (&o)[N][2]) {
        if constexpr (FLAT) {
#pragma unroll
            for (int i = 0; i < N; ++i) from_seq(p, seq_at(i), a.D, cols, o[i]);
        } else {
            from_seq(p, tile.seq, a.D, cols, o[0]);
#pragma unroll
            for (int i = 1; i < N; ++i) {
                o[i][0] = o[0][0];
                o[i][1] = o[0][1];
            }
        }
    };
    {   // the wave's maps, forwards and backwards
        float A[2] = {1.f, 1.f}, B[2] = {0.f, 0.f}, RA[2] = {1.f, 1.f}, RB[2] = {0.f, 0.f};
        if (starts == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    A[v] *= keep[i][v];
                    B[v] = fmaf(keep[i][v], B[v], z[i][v] * x[i].get(v));
                }
        } else {
            float h0[N][2];
            at_marks(a.h_in, h0);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    A[v] = first(i) ? 0.f : A[v] * keep[i][v];
                    B[v] = fmaf(keep[i][v], first(i) ? h0[i][v] : B[v], z[i][v] * x[i].get(v));
                }
        }
        forget(x);
        if (ends == 0) {
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    RA[v] *= keep[i][v];
                    RB[v] = keep[i][v] * (RB[v] + dy[i].get(v));
                }
        } else {
            float l0[N][2];
            at_marks(a.dh_out, l0);
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    RA[v] = last(i) ? 0.f : RA[v] * keep[i][v];
                    RB[v] = keep[i][v] * ((last(i) ? l0[i][v] : RB[v]) + dy[i].get(v));
                }
        }
        sh.sA[w][lane] = make_float2(A[0], A[1]);
        sh.sB[w][lane] = make_float2(B[0], B[1]);
        sh.sRA[w][lane] = make_float2(RA[0], RA[1]);
        sh.sRB[w][lane] = make_float2(RB[0], RB[1]);
        if (lane == 0)
            sh.sHard[w] = (starts != 0 ? 1 : 0) | (ends != 0 ? 2 : 0) | (nv > 0 && ((ends >> (nv - 1)) & 1) ? 4 : 0);
    }
    forget(x);
    forget(dy);
    __syncthreads();
    // map of the waves after this one, backwards
    float Ap[2] = {1.f, 1.f}, Bp[2] = {0.f, 0.f};
    bool hard = false;
    auto compose = [&](int k) {
        const float2 A = sh.sRA[k][lane], B = sh.sRB[k][lane];
        if (uniform32(sh.sHard[k]) & 2) {
            hard = true;
            Ap[0] = Ap[1] = 0.f;
            Bp[0] = B.x;
            Bp[1] = B.y;
        } else {
            Ap[0] *= A.x;
            Ap[1] *= A.y;
            Bp[0] = fmaf(A.x, Bp[0], B.x);
            Bp[1] = fmaf(A.y, Bp[1], B.y);
        }
    };
    for (int k = kWaves - 1; k > w; --k) compose(k);
    if (w == 0) {                              // the first one does the chaining
        const float A0[2] = {Ap[0], Ap[1]}, B0[2] = {Bp[0], Bp[1]};
        const bool hard0 = hard;
        float carry[2] = {0.f, 0.f};
        compose(0);
        // nothing enters from behind when the tile's last token ends a sequence, or tokens end here
        int last = 0;
        for (int k = 0; k < kWaves; ++k) last = tile.nv > k * N ? sh.sHard[k] : last;
        const bool ends_here = tile.nv == 0 || (uniform32(last) & 4) != 0;
        if constexpr (SERIAL) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                carry[v] = ends_here ? 0.f : state[v];
                state[v] = hard ? Bp[v] : fmaf(Ap[v], carry[v], Bp[v]);
            }
        } else {
            const int64_t stride = (int64_t)a.ncols * kScanCols;
            uint64_t* mine = a.words + c * stride;
#pragma unroll
            for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], hard ? final_word(Bp[v]) : map_word(Ap[v], Bp[v]));
            if (tile.after > 0 && !ends_here) {
                const int64_t step = tile.link;
                chain_wait(a.words, stride, c + step, step, tile.after, cols.d, lane, sh.far, carry);
            }
            if (!hard) {
#pragma unroll
                for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], final_word(fmaf(Ap[v], carry[v], Bp[v])));
            }
        }
        sh.sCarry[lane] = make_float2(carry[0], carry[1]);
        Ap[0] = A0[0]; Ap[1] = A0[1];
        Bp[0] = B0[0]; Bp[1] = B0[1];
        hard = hard0;
    }
    // state that enters this wave
    for (int k = 0; k < w; ++k) {
        const float2 A = sh.sA[k][lane], B = sh.sB[k][lane];
        const bool cut = uniform32(sh.sHard[k]) & 1;
        h[0] = cut ? B.x : fmaf(A.x, h[0], B.x);
        h[1] = cut ? B.y : fmaf(A.y, h[1], B.y);
    }
    // forwards: what dgate is of l_t
    float fac[N][2];
    auto factor = [&](int i) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float xv = x[i].get(v);
            fac[i][v] = z[i][v] * keep[i][v] * (xv - h[v]);
            h[v] = fmaf(keep[i][v], h[v], z[i][v] * xv);
        }
    };
    if (starts == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) factor(i);
    } else {
        float h0[N][2];
        at_marks(a.h_in, h0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int v = 0; v < 2; ++v) h[v] = first(i) ? h0[i][v] : h[v];
            factor(i);
        }
    }
    __syncthreads();
    float G[2];
    {
        const float2 cy = sh.sCarry[lane];
        G[0] = hard ? Bp[0] : fmaf(Ap[0], cy.x, Bp[0]);
        G[1] = hard ? Bp[1] : fmaf(Ap[1], cy.y, Bp[1]);
    }
    // backwards
    const rsrc_t gr = rows_at(a.dgate, tw * a.dgate_p), xr = rows_at(a.dx, tw * a.dx_p);
    int grow = (nv - 1) * (int)a.dgate_p, xrow = (nv - 1) * (int)a.dx_p;
    auto token = [&](int i) {
        float dg[2], dx[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float l = dy[i].get(v) + G[v];
            dx[v] = z[i][v] * l;
            dg[v] = fac[i][v] * l;
            sum[v] += dg[v];
            G[v] = keep[i][v] * l;
        }
        store_pair<T, VEC>(gr, cols.off[0], cols.off[1], grow, dg[0], dg[1]);
        store_pair<T, VEC>(xr, cols.off[0], cols.off[1], xrow, dx[0], dx[1]);
        grow -= (int)a.dgate_p;
        xrow -= (int)a.dx_p;
    };
    if (nv == N && (starts | ends) == 0) {
#pragma unroll
        for (int i = N - 1; i >= 0; --i) token(i);
    } else {
        float l0[N][2];
        if (ends != 0) at_marks(a.dh_out, l0);
#pragma unroll
        for (int i = N - 1; i >= 0; --i) {
            if (i < nv) {
#pragma unroll
                for (int v = 0; v < 2; ++v) G[v] = last(i) ? l0[i][v] : G[v];
                token(i);
                if (first(i) && a.dh_in) to_seq(a.dh_in, seq_at(i), a.D, cols, G);
            }
        }
    }
    if (FLAT && a.dh_in) pass_empty(a, c, cols, lane, w, a.dh_out, a.dh_in);
}

// the workgroup's share of dbias: its waves' added in order
template <typename T, bool VEC, bool FLAT, bool SERIAL>
__device__ __forceinline__ void add_dbias(const GatedScanArgs& a, BwdShared<T, FLAT, SERIAL>& sh, uint32_t row, int col,
                                          int lane, int w, const float (&sum)[2]) {
    if (a.dbias == nullptr) return;
    __syncthreads();
    sh.sA[w][lane] = make_float2(sum[0], sum[1]);
    __syncthreads();
    if (w != 0) return;
    float2 t = sh.sA[0][lane];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) {
        t.x += sh.sA[k][lane].x;
        t.y += sh.sA[k][lane].y;
    }
    const float o[2] = {t.x, t.y};
    to_seq(a.parts > 1 ? a.part : a.dbias, a.parts > 1 ? row : 0, a.D, Cols<T, VEC>(col, lane, a.D), o);
}

template <typename T, bool VEC, bool FLAT, bool SERIAL>
__global__ __launch_bounds__(kWaves * 64, kWavesPerSimd) void gated_scan_backward_kernel(const GatedScanArgs a) {
    __shared__ BwdShared<T, FLAT, SERIAL> sh;
    const int lane = threadIdx.x & 63;
    const int w = uniform32(threadIdx.x >> 6);
    float state[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f};
    if constexpr (SERIAL) {
        const uint32_t seq = uniform32(blockIdx.x / (uint32_t)a.ncols), n = FLAT ? (uint32_t)a.ntiles : a.seq_tiles;
        const int col = (int)(blockIdx.x - seq * (uint32_t)a.ncols);
        for (uint32_t j = n; j-- > 0;) {       // from the last tile to the first
            if (j + 1 < n) __syncthreads();
            backward_tile<T, VEC, FLAT, true>(a, sh, seq * n + j, col, lane, w, state, sum);
        }
        add_dbias<T, VEC>(a, sh, seq, col, lane, w, sum);
    } else {
        uint32_t c;
        int col;
        if (!take_item(a, sh.sTicket, c, col)) return;
        c = (uint32_t)a.ntiles - 1 - c;
        backward_tile<T, VEC, FLAT, false>(a, sh, c, col, lane, w, state, sum);
        add_dbias<T, VEC>(a, sh, c, col, lane, w, sum);
    }
}

// ------------------------------------------------------------------------------- one token
// One lane per run of W channels: W = 4 (16 bytes of state per access) where rows allow it, else 1.  Bound: memory, the
// state's 8 bytes per channel first of all: b4096 D4096 bf16 235 MB in 49 us, 4.8 TB/s, b16384 5.3 TB/s; b8 3.0 us,
// a launch.
template <typename T, int W>
__global__ __launch_bounds__(256) void gated_step_kernel(const GatedStepArgs a, int64_t per_row) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / per_row, d = (i - row * per_row) * W;
    if (row >= a.b) return;
    const T* gp = (const T*)((const char*)a.gate + row * a.gate_p) + d;
    const T* xp = (const T*)((const char*)a.x + row * a.x_p) + d;
    T* yp = (T*)((char*)a.y + row * a.y_p) + d;
    const float* hp = a.h + row * a.D + d;
    float* op = a.h_out + row * a.D + d;
    struct alignas(W * sizeof(T)) Io { T v[W]; };
    struct alignas(W * 4) Fl { float v[W]; };
    const Io g = *(const Io*)gp, x = *(const Io*)xp;
    const Fl h = *(const Fl*)hp;
    Fl o;
    Io y;
#pragma unroll
    for (int v = 0; v < W; ++v) {
        float z, keep;
        gate_of(to_f32(g.v[v]), a.bias ? a.bias[d + v] : 0.f, z, keep);
        o.v[v] = fmaf(keep, h.v[v], z * to_f32(x.v[v]));
        y.v[v] = from_f32<T>(o.v[v]);
    }
    *(Fl*)op = o;
    *(Io*)yp = y;
}

// out[d] = sum over rows of part[row, d]: 16 columns per workgroup, every 64th row per thread, the
// 64 partial sums added in order, so the sum's order is fixed.  256 rows of 4096: 4.8 us, a launch and one latency.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* part, int64_t n, int64_t D, float* out) {
    __shared__ float s[64][17];
    const int cx = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t d = (int64_t)blockIdx.x * 16 + cx;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (d < D) {
        int64_t i = g;
        for (; i + 192 < n; i += 256) {
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += part[(i + 64 * k) * D + d];
        }
        for (; i < n; i += 64) acc[0] += part[i * D + d];
    }
    s[g][cx] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    if (g < 4) {
        float t = 0.f;
        for (int k = 0; k < 16; ++k) t += s[g * 16 + k][cx];
        s[g * 16][cx] = t;
    }
    __syncthreads();
    if (g == 0 && d < D) out[d] = (s[0][cx] + s[16][cx]) + (s[32][cx] + s[48][cx]);
}

hipError_t reset_chain(const GatedScanArgs& a, hipStream_t s) {
    const int64_t n16 = a.ntiles * a.ncols * kScanCols / 2, most = a.per_seq || n16 > a.T ? n16 : a.T;
    const int64_t blocks = (most + 255) / 256;
    hipLaunchKernelGGL(chain_reset_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s, a, n16);
    return hipGetLastError();
}

}  // namespace

#define M3_SCAN(KERNEL, T, VEC)                                                                                  \
    do {                                                                                                          \
        if (a.serial && flat) hipLaunchKernelGGL((KERNEL<T, VEC, true, true>), grid, block, 0, s, a);             \
        else if (a.serial) hipLaunchKernelGGL((KERNEL<T, VEC, false, true>), grid, block, 0, s, a);               \
        else if (flat) hipLaunchKernelGGL((KERNEL<T, VEC, true, false>), grid, block, 0, s, a);                   \
        else hipLaunchKernelGGL((KERNEL<T, VEC, false, false>), grid, block, 0, s, a);                            \
    } while (0)
#define M3_SCAN_TYPES(KERNEL)                            \
    do {                                                 \
        if (bf16_io && vec) M3_SCAN(KERNEL, bf16, true); \
        else if (bf16_io) M3_SCAN(KERNEL, bf16, false);  \
        else if (vec) M3_SCAN(KERNEL, float, true);      \
        else M3_SCAN(KERNEL, float, false);              \
    } while (0)

namespace {
dim3 scan_grid(const GatedScanArgs& a) {
    return dim3((unsigned)((a.serial ? (a.per_seq ? a.b : 1) : a.ntiles) * a.ncols));
}
}  // namespace

hipError_t launch_gated_scan(const GatedScanArgs& a, bool bf16_io, bool vec, hipStream_t s) {
    if (!a.serial) {
        const hipError_t e = reset_chain(a, s);
        if (e != hipSuccess) return e;
    }
    const dim3 grid = scan_grid(a), block(kWaves * 64);
    const bool flat = !a.per_seq;
    M3_SCAN_TYPES(gated_scan_kernel);
    return hipGetLastError();
}

hipError_t launch_gated_scan_backward(const GatedScanArgs& a, bool bf16_io, bool vec, hipStream_t s) {
    if (!a.serial) {
        const hipError_t e = reset_chain(a, s);
        if (e != hipSuccess) return e;
    }
    const dim3 grid = scan_grid(a), block(kWaves * 64);
    const bool flat = !a.per_seq;
    M3_SCAN_TYPES(gated_scan_backward_kernel);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.dbias && a.parts > 1) e = launch_column_sum(a.part, a.parts, a.D, a.dbias, s);
    return e;
}

hipError_t launch_gated_step(const GatedStepArgs& a, bool bf16_io, bool vec, hipStream_t s) {
    const int64_t per_row = vec ? a.D / 4 : a.D;
    const dim3 grid((unsigned)((a.b * per_row + 255) / 256)), block(256);
    if (bf16_io && vec) hipLaunchKernelGGL((gated_step_kernel<bf16, 4>), grid, block, 0, s, a, per_row);
    else if (bf16_io) hipLaunchKernelGGL((gated_step_kernel<bf16, 1>), grid, block, 0, s, a, per_row);
    else if (vec) hipLaunchKernelGGL((gated_step_kernel<float, 4>), grid, block, 0, s, a, per_row);
    else hipLaunchKernelGGL((gated_step_kernel<float, 1>), grid, block, 0, s, a, per_row);
    return hipGetLastError();
}

hipError_t launch_column_sum(const float* part, int64_t n, int64_t D, float* out, hipStream_t s) {
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((D + 15) / 16)), dim3(1024), 0, s, part, n, D, out);
    return hipGetLastError();
}

}  // namespace m3
