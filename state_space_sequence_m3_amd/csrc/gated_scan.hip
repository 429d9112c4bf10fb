// gated_scan.hip -- per-channel gated linear recurrence  h_t = (1 - z_t) h_{t-1} + z_t x_t,
// z_t = sigmoid(gate_t + bias), forward, backward and for single tokens.
//
// A run of steps is the affine map h -> A h + B with A the product of (1 - z_t) and B the run's
// end from a zero state, and maps compose: (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2).  A
// sequence's first token forgets what came before: its map is h -> B (A = 0), with B taking the
// carried h_in in.
#include "block_launch.h"
#include "m3_device.h"

namespace m3 {
namespace {

constexpr int kWaves = 8;                        // waves per tile
constexpr int kSteps = kScanTile / kWaves;       // consecutive tokens of one wave
constexpr int kFwdWavesPerSimd = 4, kBwdWavesPerSimd = 2;

// z = sigmoid(u) and 1 - z, each to a few units in its last place: the smaller one is e^-|u| / (1 + e^-|u|),
// not a difference from 1.  fp32 io carries the rounding of u log2(e) along; with bf16 io the
// logit's own rounding is larger than that.
template <typename T>
__device__ __forceinline__ void gate_of(float u, float& z, float& keep) {
    const float m = -fabsf(u);
    const float t = m * kLog2e;
    float e = fast_exp2(t);
    if constexpr (sizeof(T) == 4) {
        const float lo = fmaf(m, kLog2e, -t) + m * 1.925963033500e-8f;   // log2(e) - kLog2e
        e = fmaf(e, lo * 0.6931471805599453f, e);
        e = t < -126.f ? fast_exp2(t) : e;
    }
    const float big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
    z = u >= 0.f ? big : small;
    keep = u >= 0.f ? small : big;
}

// Two channels of one token per lane.  VEC: neighbours 2 lane, 2 lane + 1 in one load; else
// lane and lane + 64, element by element.
template <typename T, bool VEC> struct Pair;
template <> struct Pair<float, true> {
    float2 v;
    __device__ __forceinline__ void load(const char* row, uint32_t o0, uint32_t) { v = *(const float2*)(row + o0); }
    __device__ __forceinline__ float get(int i) const { return i ? v.y : v.x; }
};
template <> struct Pair<bf16, true> {
    uint32_t v;
    __device__ __forceinline__ void load(const char* row, uint32_t o0, uint32_t) { v = *(const uint32_t*)(row + o0); }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
};
template <> struct Pair<float, false> {
    float v[2];
    __device__ __forceinline__ void load(const char* row, uint32_t o0, uint32_t o1) {
        v[0] = *(const float*)(row + o0);
        v[1] = *(const float*)(row + o1);
    }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <> struct Pair<bf16, false> {
    uint16_t v[2];
    __device__ __forceinline__ void load(const char* row, uint32_t o0, uint32_t o1) {
        v[0] = *(const uint16_t*)(row + o0);
        v[1] = *(const uint16_t*)(row + o1);
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float((uint32_t)v[i] << 16); }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_pair(char* row, uint32_t o0, uint32_t o1, bool ok0, bool ok1, float v0, float v1) {
    if constexpr (VEC) {
        if (ok0) {
            if constexpr (sizeof(T) == 4) *(float2*)(row + o0) = make_float2(v0, v1);
            else *(uint32_t*)(row + o0) = pack_bf16x2(v0, v1);
        }
    } else {
        if (ok0) *(T*)(row + o0) = from_f32<T>(v0);
        if (ok1) *(T*)(row + o1) = from_f32<T>(v1);
    }
}

// Where a lane's two channels are.
template <typename T, bool VEC>
struct Cols {
    int64_t d[2];       // channels, possibly past D
    bool ok[2];
    uint32_t off[2];    // byte offsets in a row, clamped into it (lanes past D read valid data)
    __device__ __forceinline__ Cols(int col, int lane, int64_t D) {
        d[0] = (int64_t)col * kScanCols + (VEC ? 2 * lane : lane);
        d[1] = d[0] + (VEC ? 1 : 64);
        for (int v = 0; v < 2; ++v) {
            ok[v] = d[v] < D;
            const int64_t last = VEC ? D - 2 + v : D - 1;
            off[v] = (uint32_t)((d[v] < last ? d[v] : last) * (int64_t)sizeof(T));
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

// A tile's place: tokens [t0, t0 + nv), its neighbours in the chain, and its row of `states`.
struct Tile {
    int64_t t0, prev, next, row;
    uint32_t links_before, links_after;   // tiles of the same chain
    int nv;
};
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ uint32_t uniform32(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ Tile tile_of(const GatedScanArgs& a, uint32_t c) {
    Tile t;
    if (a.per_seq) {
        // tiles in the order (place in the sequence, sequence): the tiles that run at the same time
        // belong to as many sequences as there are, and a chain link waits less
        const uint32_t b = (uint32_t)a.b, j = uniform32(c / b), s = c - j * b, n = (uint32_t)a.seq_chunks;
        t.t0 = (int64_t)s * a.L + (int64_t)j * kScanTile;
        const int64_t left = a.L - (int64_t)j * kScanTile;
        t.nv = (int)(left < kScanTile ? left : kScanTile);
        t.prev = j > 0 ? (int64_t)c - b : -1;
        t.next = j + 1 < n ? (int64_t)c + b : -1;
        t.links_before = j;
        t.links_after = n - 1 - j;
        t.row = (int64_t)s * n + j;
    } else {
        const int64_t total = a.cu ? seq_start(a, a.b) : a.T;
        t.t0 = (int64_t)c * kScanTile;
        const int64_t left = total - t.t0;
        t.nv = (int)(left < 0 ? 0 : (left < kScanTile ? left : kScanTile));
        t.prev = (int64_t)c - 1;
        t.next = (int64_t)c + 1 < a.nchunks ? (int64_t)c + 1 : -1;
        t.links_before = c;
        t.links_after = (uint32_t)a.nchunks - 1 - c;
        t.row = c;
    }
    return t;
}

// Which tokens of a tile start or end a sequence.  A tile of one long sequence (per_seq) knows by its
// place; else one thread per token looks its sequence up, and all threads must come here.
struct Marks {
    int seq[kScanTile];                          // the sequence of each token
    uint64_t starts[kScanTile / 64], ends[kScanTile / 64];
};
__device__ __forceinline__ void find_marks(const GatedScanArgs& a, const Tile& tile, Marks& m) {
    if (a.per_seq) return;
    const int i = threadIdx.x;
    if (i < kScanTile) {
        bool start = false, end = false;
        if (i < tile.nv) {
            const int64_t t = tile.t0 + i, s = seq_of(a, t);
            m.seq[i] = (int)s;
            start = seq_start(a, s) == t;
            end = seq_start(a, s + 1) == t + 1;
        }
        const uint64_t ms = __ballot(start), me = __ballot(end);
        if ((i & 63) == 0) {
            m.starts[i >> 6] = ms;
            m.ends[i >> 6] = me;
        }
    }
    __syncthreads();
}
// the kSteps tokens of wave w, as bits
__device__ __forceinline__ uint32_t wave_starts(const GatedScanArgs& a, const Tile& tile, const Marks& m, int w) {
    if (a.per_seq) return w == 0 && tile.prev < 0 ? 1u : 0u;
    return uniform32((uint32_t)(m.starts[w * kSteps / 64] >> (w * kSteps % 64))) & ((1u << kSteps) - 1);
}
__device__ __forceinline__ uint32_t wave_ends(const GatedScanArgs& a, const Tile& tile, const Marks& m, int w) {
    if (a.per_seq) {
        const int last = tile.nv - 1 - w * kSteps;
        return tile.next < 0 && last >= 0 && last < kSteps ? 1u << last : 0u;
    }
    return uniform32((uint32_t)(m.ends[w * kSteps / 64] >> (w * kSteps % 64))) & ((1u << kSteps) - 1);
}
// the sequence of token i of wave w (a start or an end)
__device__ __forceinline__ int64_t mark_seq(const GatedScanArgs& a, const Tile& tile, const Marks& m, int w, int i) {
    return a.per_seq ? tile.row / a.seq_chunks : (int64_t)uniform32((uint32_t)m.seq[w * kSteps + i]);
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

constexpr int kWindow = 4;            // words looked at together
constexpr int kMaxPolls = 1 << 22;    // some seconds: a wait that long means a workspace in use twice

// The state that enters a tile whose neighbour in the chain is `first`, the one after that
// first + step, and so on for `links` tiles.  It starts from the nearest final word and applies
// the maps after it in order.  A tile's own final word is made by the same steps, so the value
// does not depend on which word was found final.  Ends: workgroups take tiles from a counter in
// chain order, so every tile waited for here is held by a workgroup that runs (or is done) and
// itself waits for earlier ones only; the first tile of a chain waits for none.  A wait that
// outlasts kMaxPolls gives NaN.
__device__ __forceinline__ void chain_wait(const uint64_t* words, int64_t stride, int64_t first, int64_t step,
                                           uint32_t links, const int64_t (&d)[2], float (&carry)[2]) {
    for (int poll = 0; poll < kMaxPolls; ++poll) {
        uint64_t w[kWindow][2];
#pragma unroll
        for (int k = 0; k < kWindow; ++k) {
            if ((uint32_t)k < links) {
                const uint64_t* row = words + (first + k * step) * stride;
                w[k][0] = get_word(row + d[0]);
                w[k][1] = get_word(row + d[1]);
            } else {
                w[k][0] = w[k][1] = ~0ull;
            }
        }
        bool done = true;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            bool valid = false;
            float h = 0.f;
#pragma unroll
            for (int k = kWindow - 1; k >= 0; --k) {
                const uint32_t A = (uint32_t)w[k][v];
                const float B = __uint_as_float((uint32_t)(w[k][v] >> 32));
                const float next = A == kFinal ? B : fmaf(__uint_as_float(A), h, B);
                valid = A == kFinal || (valid && A != kUnset);
                h = next;
            }
            carry[v] = h;
            done = done && valid;
        }
        if (__all(done)) return;
        __builtin_amdgcn_s_sleep(1);
    }
    carry[0] = carry[1] = __uint_as_float(0x7fc00000u);
}

__global__ __launch_bounds__(256) void chain_reset_kernel(uint4* words, int64_t n16, unsigned* ticket) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n16) words[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
    if (i == 0) *ticket = 0;
}

// ---------------------------------------------------------------------------------- forward
// The tile a workgroup works on, and its columns: the workgroup's place in the grid, or, where tiles
// wait for each other, a number from a counter, so that tiles start in chain order.
__device__ __forceinline__ bool take_item(const GatedScanArgs& a, unsigned& s_ticket, uint32_t& c, int& col) {
    uint32_t item = blockIdx.x;
    if (a.nchunks > 1) {
        if (threadIdx.x == 0) s_ticket = atomicAdd(a.ticket, 1u);
        __syncthreads();
        item = uniform32(s_ticket);
        if (item >= (uint32_t)a.nchunks * (uint32_t)a.ncols) return false;
    }
    c = uniform32(item / (uint32_t)a.ncols);
    col = (int)(item - c * (uint32_t)a.ncols);
    return true;
}

template <typename T, bool VEC>
__global__ __launch_bounds__(kWaves * 64, kFwdWavesPerSimd) void gated_scan_kernel(const GatedScanArgs a) {
    __shared__ float2 sA[kWaves][64], sB[kWaves][64], sCarry[64];
    __shared__ int sHard[kWaves];   // bit 0: the wave's tokens hold a sequence start; bit 1: its first token is one
    __shared__ Marks sMarks;
    __shared__ unsigned sTicket;
    const int lane = threadIdx.x & 63;
    const int w = uniform32(threadIdx.x >> 6);
    uint32_t c;
    int col;
    if (!take_item(a, sTicket, c, col)) return;
    const Tile tile = tile_of(a, c);
    const Cols<T, VEC> cols(col, lane, a.D);
    const int64_t tw = tile.t0 + w * kSteps;
    const int left = tile.nv - w * kSteps;
    const int nv = left < 0 ? 0 : (left < kSteps ? left : kSteps);

    // rows past the last one are read as the last one again, and do nothing
    Pair<T, VEC> rg[kSteps], rx[kSteps];
    if (nv > 0) {
        const char* gp = (const char*)a.gate + tw * a.gate_p;
        const char* xp = (const char*)a.x + tw * a.x_p;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            rg[i].load(gp, cols.off[0], cols.off[1]);
            rx[i].load(xp, cols.off[0], cols.off[1]);
            gp += i + 1 < nv ? a.gate_p : 0;
            xp += i + 1 < nv ? a.x_p : 0;
        }
    }
    float bias[2] = {0.f, 0.f};
    if (a.bias) {
        bias[0] = a.bias[cols.off[0] / sizeof(T)];
        bias[1] = a.bias[cols.off[1] / sizeof(T)];
    }
    find_marks(a, tile, sMarks);
    const uint32_t starts = wave_starts(a, tile, sMarks, w);
    float keep[kSteps][2], add[kSteps][2];
    float A[2] = {1.f, 1.f}, B[2] = {0.f, 0.f};   // the wave's map
    if (nv > 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float z;
                gate_of<T>(rg[i].get(v) + bias[v], z, keep[i][v]);
                add[i][v] = z * rx[i].get(v);
            }
    }
    if (nv < kSteps) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (i >= nv) {
                keep[i][0] = keep[i][1] = 1.f;
                add[i][0] = add[i][1] = 0.f;
            }
    }
    if (starts == 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                A[v] *= keep[i][v];
                B[v] = fmaf(keep[i][v], B[v], add[i][v]);
            }
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if ((starts >> i) & 1) {
                if (a.h_in) {
                    const float* h = a.h_in + mark_seq(a, tile, sMarks, w, i) * a.D;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        if (cols.ok[v]) add[i][v] = fmaf(keep[i][v], h[cols.d[v]], add[i][v]);
                }
                A[0] = A[1] = 0.f;
                B[0] = add[i][0];
                B[1] = add[i][1];
            } else {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    A[v] *= keep[i][v];
                    B[v] = fmaf(keep[i][v], B[v], add[i][v]);
                }
            }
        }
    }
    sA[w][lane] = make_float2(A[0], A[1]);
    sB[w][lane] = make_float2(B[0], B[1]);
    if (lane == 0) sHard[w] = (starts != 0 ? 1 : 0) | (starts & 1 ? 2 : 0);
    __syncthreads();
    // the map of the waves before this one
    float Ap[2] = {1.f, 1.f}, Bp[2] = {0.f, 0.f};
    bool hard = false;
    auto compose = [&](int k) {
        const float2 A = sA[k][lane], B = sB[k][lane];
        if (uniform32(sHard[k]) & 1) {
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
    float carry[2] = {0.f, 0.f};
    if (w == kWaves - 1) {
        const float A0[2] = {Ap[0], Ap[1]}, B0[2] = {Bp[0], Bp[1]};
        const bool hard0 = hard;
        compose(w);
        if (a.nchunks > 1) {
            const int64_t stride = (int64_t)a.ncols * kScanCols;
            uint64_t* mine = a.words + c * stride;
#pragma unroll
            for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], hard ? final_word(Bp[v]) : map_word(Ap[v], Bp[v]));
            const bool starts_here = (uniform32(sHard[0]) & 2) != 0;
            if (tile.prev >= 0 && tile.nv > 0 && !starts_here)
                chain_wait(a.words, stride, tile.prev, a.per_seq ? -a.b : -1, tile.links_before, cols.d, carry);
            if (!hard) {
#pragma unroll
                for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], final_word(fmaf(Ap[v], carry[v], Bp[v])));
            }
        }
        sCarry[lane] = make_float2(carry[0], carry[1]);
        if (a.states) {
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (cols.ok[v]) a.states[tile.row * a.D + cols.d[v]] = carry[v];
        }
        Ap[0] = A0[0]; Ap[1] = A0[1];
        Bp[0] = B0[0]; Bp[1] = B0[1];
        hard = hard0;
    }
    __syncthreads();
    float h[2];
    {
        const float2 cy = sCarry[lane];
        h[0] = hard ? Bp[0] : fmaf(Ap[0], cy.x, Bp[0]);
        h[1] = hard ? Bp[1] : fmaf(Ap[1], cy.y, Bp[1]);
    }
    const uint32_t ends = wave_ends(a, tile, sMarks, w);
    char* yp = (char*)a.y + tw * a.y_p;
    if (nv == kSteps && (starts | ends) == 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
#pragma unroll
            for (int v = 0; v < 2; ++v) h[v] = fmaf(keep[i][v], h[v], add[i][v]);
            store_pair<T, VEC>(yp, cols.off[0], cols.off[1], cols.ok[0], cols.ok[1], h[0], h[1]);
            yp += a.y_p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i < nv) {
                if ((starts >> i) & 1) h[0] = h[1] = 0.f;   // and the carried state is in add
#pragma unroll
                for (int v = 0; v < 2; ++v) h[v] = fmaf(keep[i][v], h[v], add[i][v]);
                store_pair<T, VEC>(yp, cols.off[0], cols.off[1], cols.ok[0], cols.ok[1], h[0], h[1]);
                yp += a.y_p;
                if ((ends >> i) & 1) {
                    float* o = a.h_out + mark_seq(a, tile, sMarks, w, i) * a.D;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        if (cols.ok[v]) o[cols.d[v]] = h[v];
                }
            }
        }
    }
    // empty sequences: the carried state passes through
    if (w == 0 && (a.cu != nullptr || a.L == 0)) {
        for (int64_t s = c; s < a.b; s += a.nchunks) {
            if (seq_start(a, s + 1) > seq_start(a, s)) continue;
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (cols.ok[v]) a.h_out[s * a.D + cols.d[v]] = a.h_in ? a.h_in[s * a.D + cols.d[v]] : 0.f;
        }
    }
}

// --------------------------------------------------------------------------------- backward
// With G_t = (1 - z_t) l_t, what flows from token t to h_{t-1}: l_t = dy_t + G_{t+1}, so backwards
// G_t = keep_t G_{t+1} + keep_t dy_t, an affine map again, and the same chain in the other
// direction.  A sequence's last token takes dh_out for G_{t+1}.
template <typename T, bool VEC>
__global__ __launch_bounds__(kWaves * 64, kBwdWavesPerSimd) void gated_scan_backward_kernel(const GatedScanArgs a) {
    __shared__ float2 sA[kWaves][64], sB[kWaves][64], sRA[kWaves][64], sRB[kWaves][64], sCarry[64];
    __shared__ int sHard[kWaves];   // bit 0: holds a sequence start; 1: holds an end; 2: its last token is an end
    __shared__ Marks sMarks;
    __shared__ unsigned sTicket;
    const int lane = threadIdx.x & 63;
    const int w = uniform32(threadIdx.x >> 6);
    uint32_t c;
    int col;
    if (!take_item(a, sTicket, c, col)) return;
    c = (uint32_t)a.nchunks - 1 - c;   // from the last tile to the first
    const Tile tile = tile_of(a, c);
    const Cols<T, VEC> cols(col, lane, a.D);
    const int64_t tw = tile.t0 + w * kSteps;
    const int left = tile.nv - w * kSteps;
    const int nv = left < 0 ? 0 : (left < kSteps ? left : kSteps);

    Pair<T, VEC> rg[kSteps], rx[kSteps], rd[kSteps];
    if (nv > 0) {
        const char* gp = (const char*)a.gate + tw * a.gate_p;
        const char* xp = (const char*)a.x + tw * a.x_p;
        const char* dp = (const char*)a.dy + tw * a.y_p;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            rg[i].load(gp, cols.off[0], cols.off[1]);
            rx[i].load(xp, cols.off[0], cols.off[1]);
            rd[i].load(dp, cols.off[0], cols.off[1]);
            gp += i + 1 < nv ? a.gate_p : 0;
            xp += i + 1 < nv ? a.x_p : 0;
            dp += i + 1 < nv ? a.y_p : 0;
        }
    }
    float h[2], bias[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < 2; ++v) h[v] = cols.ok[v] ? a.states[tile.row * a.D + cols.d[v]] : 0.f;
    if (a.bias) {
        bias[0] = a.bias[cols.off[0] / sizeof(T)];
        bias[1] = a.bias[cols.off[1] / sizeof(T)];
    }
    find_marks(a, tile, sMarks);
    const uint32_t starts = wave_starts(a, tile, sMarks, w), ends = wave_ends(a, tile, sMarks, w);

    float z[kSteps][2], keep[kSteps][2], xs[kSteps][2], lam[kSteps][2];   // lam: dy
    if (nv > 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                gate_of<T>(rg[i].get(v) + bias[v], z[i][v], keep[i][v]);
                xs[i][v] = rx[i].get(v);
                lam[i][v] = rd[i].get(v);
            }
    }
    if (nv < kSteps) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (i >= nv) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    z[i][v] = 0.f;
                    keep[i][v] = 1.f;
                    xs[i][v] = 0.f;
                    lam[i][v] = 0.f;
                }
            }
    }
    const bool marked = (starts | ends) != 0;
    if (ends != 0 && a.dh_out) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if ((ends >> i) & 1) {
                const float* d = a.dh_out + mark_seq(a, tile, sMarks, w, i) * a.D;
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    if (cols.ok[v]) lam[i][v] += d[cols.d[v]];
            }
    }
    {   // the wave's maps, forwards and backwards
        float A[2] = {1.f, 1.f}, B[2] = {0.f, 0.f}, RA[2] = {1.f, 1.f}, RB[2] = {0.f, 0.f};
        if (!marked) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    A[v] *= keep[i][v];
                    B[v] = fmaf(keep[i][v], B[v], z[i][v] * xs[i][v]);
                }
            RA[0] = A[0];
            RA[1] = A[1];
#pragma unroll
            for (int i = kSteps - 1; i >= 0; --i)
#pragma unroll
                for (int v = 0; v < 2; ++v) RB[v] = keep[i][v] * (RB[v] + lam[i][v]);
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if ((starts >> i) & 1) {
                    A[0] = A[1] = B[0] = B[1] = 0.f;
                    if (a.h_in) {
                        const float* hi = a.h_in + mark_seq(a, tile, sMarks, w, i) * a.D;
#pragma unroll
                        for (int v = 0; v < 2; ++v) B[v] = cols.ok[v] ? hi[cols.d[v]] : 0.f;
                    }
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    A[v] *= keep[i][v];
                    B[v] = fmaf(keep[i][v], B[v], z[i][v] * xs[i][v]);
                }
            }
#pragma unroll
            for (int i = kSteps - 1; i >= 0; --i) {
                if ((ends >> i) & 1) RA[0] = RA[1] = RB[0] = RB[1] = 0.f;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    RA[v] *= keep[i][v];
                    RB[v] = keep[i][v] * (RB[v] + lam[i][v]);
                }
            }
        }
        sA[w][lane] = make_float2(A[0], A[1]);
        sB[w][lane] = make_float2(B[0], B[1]);
        sRA[w][lane] = make_float2(RA[0], RA[1]);
        sRB[w][lane] = make_float2(RB[0], RB[1]);
        if (lane == 0)
            sHard[w] = (starts != 0 ? 1 : 0) | (ends != 0 ? 2 : 0) | (nv > 0 && ((ends >> (nv - 1)) & 1) ? 4 : 0);
    }
    __syncthreads();
    // state that enters this wave
    for (int k = 0; k < w; ++k) {
        const float2 A = sA[k][lane], B = sB[k][lane];
        const bool cut = uniform32(sHard[k]) & 1;
        h[0] = cut ? B.x : fmaf(A.x, h[0], B.x);
        h[1] = cut ? B.y : fmaf(A.y, h[1], B.y);
    }
    // map of the waves after this one, backwards
    float Ap[2] = {1.f, 1.f}, Bp[2] = {0.f, 0.f};
    bool hard = false;
    auto compose = [&](int k) {
        const float2 A = sRA[k][lane], B = sRB[k][lane];
        if (uniform32(sHard[k]) & 2) {
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
    float carry[2] = {0.f, 0.f};
    if (w == 0) {
        const float A0[2] = {Ap[0], Ap[1]}, B0[2] = {Bp[0], Bp[1]};
        const bool hard0 = hard;
        compose(0);
        if (a.nchunks > 1) {
            const int64_t stride = (int64_t)a.ncols * kScanCols;
            uint64_t* mine = a.words + c * stride;
#pragma unroll
            for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], hard ? final_word(Bp[v]) : map_word(Ap[v], Bp[v]));
            // nothing enters from behind when the tile's last token ends a sequence, or tokens end here
            int last = 0;
            for (int k = 0; k < kWaves; ++k) last = tile.nv > k * kSteps ? sHard[k] : last;
            const bool ends_here = tile.nv == 0 || (uniform32(last) & 4) != 0;
            if (tile.next >= 0 && !ends_here)
                chain_wait(a.words, stride, tile.next, a.per_seq ? a.b : 1, tile.links_after, cols.d, carry);
            if (!hard) {
#pragma unroll
                for (int v = 0; v < 2; ++v) put_word(mine + cols.d[v], final_word(fmaf(Ap[v], carry[v], Bp[v])));
            }
        }
        sCarry[lane] = make_float2(carry[0], carry[1]);
        Ap[0] = A0[0]; Ap[1] = A0[1];
        Bp[0] = B0[0]; Bp[1] = B0[1];
        hard = hard0;
    }
    // forwards: what dgate is of l_t, in the place of x
    if (starts == 0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float x = xs[i][v];
                xs[i][v] = z[i][v] * keep[i][v] * (x - h[v]);
                h[v] = fmaf(keep[i][v], h[v], z[i][v] * x);
            }
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if ((starts >> i) & 1) {
                const float* hi = a.h_in ? a.h_in + mark_seq(a, tile, sMarks, w, i) * a.D : nullptr;
#pragma unroll
                for (int v = 0; v < 2; ++v) h[v] = hi && cols.ok[v] ? hi[cols.d[v]] : 0.f;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float x = xs[i][v];
                xs[i][v] = z[i][v] * keep[i][v] * (x - h[v]);
                h[v] = fmaf(keep[i][v], h[v], z[i][v] * x);
            }
        }
    }
    __syncthreads();
    float G[2];
    {
        const float2 cy = sCarry[lane];
        G[0] = hard ? Bp[0] : fmaf(Ap[0], cy.x, Bp[0]);
        G[1] = hard ? Bp[1] : fmaf(Ap[1], cy.y, Bp[1]);
    }
    // backwards
    float sum[2] = {0.f, 0.f};
    char* gp = (char*)a.dgate + (tw + nv - 1) * a.dgate_p;
    char* xp = (char*)a.dx + (tw + nv - 1) * a.dx_p;
    auto token = [&](int i) {
        float dg[2], dx[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float l = lam[i][v] + G[v];
            dx[v] = z[i][v] * l;
            dg[v] = xs[i][v] * l;
            sum[v] += dg[v];
            G[v] = keep[i][v] * l;
        }
        store_pair<T, VEC>(gp, cols.off[0], cols.off[1], cols.ok[0], cols.ok[1], dg[0], dg[1]);
        store_pair<T, VEC>(xp, cols.off[0], cols.off[1], cols.ok[0], cols.ok[1], dx[0], dx[1]);
        gp -= a.dgate_p;
        xp -= a.dx_p;
    };
    if (nv == kSteps && !marked) {
#pragma unroll
        for (int i = kSteps - 1; i >= 0; --i) token(i);
    } else {
#pragma unroll
        for (int i = kSteps - 1; i >= 0; --i) {
            if (i < nv) {
                if ((ends >> i) & 1) G[0] = G[1] = 0.f;
                token(i);
                if (((starts >> i) & 1) && a.dh_in) {
                    float* o = a.dh_in + mark_seq(a, tile, sMarks, w, i) * a.D;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        if (cols.ok[v]) o[cols.d[v]] = G[v];
                }
            }
        }
    }
    if (a.dbias) {   // the tile's share: waves summed in order
        sA[w][lane] = make_float2(sum[0], sum[1]);
        __syncthreads();
        if (w == 0) {
            float2 t = sA[0][lane];
#pragma unroll
            for (int k = 1; k < kWaves; ++k) {
                t.x += sA[k][lane].x;
                t.y += sA[k][lane].y;
            }
            float* out = a.nchunks > 1 ? a.part + (int64_t)c * a.D : a.dbias;
            if (cols.ok[0]) out[cols.d[0]] = t.x;
            if (cols.ok[1]) out[cols.d[1]] = t.y;
        }
    }
    // empty sequences: dh_out passes through
    if (w == 0 && a.dh_in && (a.cu != nullptr || a.L == 0)) {
        for (int64_t e = c; e < a.b; e += a.nchunks) {
            if (seq_start(a, e + 1) > seq_start(a, e)) continue;
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (cols.ok[v]) a.dh_in[e * a.D + cols.d[v]] = a.dh_out ? a.dh_out[e * a.D + cols.d[v]] : 0.f;
        }
    }
}

// ------------------------------------------------------------------------------- one token
// One lane per run of W channels: W = 4 (16 bytes of state per access) where rows allow it, else 1.
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
        gate_of<T>(to_f32(g.v[v]) + (a.bias ? a.bias[d + v] : 0.f), z, keep);
        o.v[v] = fmaf(keep, h.v[v], z * to_f32(x.v[v]));
        y.v[v] = from_f32<T>(o.v[v]);
    }
    *(Fl*)op = o;
    *(Io*)yp = y;
}

// out[d] = sum over rows of part[row, d]: 16 columns per workgroup, every 64th row per thread, the
// 64 partial sums added in order, so the sum's order is fixed.
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
    const int64_t n16 = a.nchunks * a.ncols * kScanCols / 2;
    hipLaunchKernelGGL(chain_reset_kernel, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, s, (uint4*)a.words, n16,
                       a.ticket);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_scan(const GatedScanArgs& a, bool bf16_io, bool vec, hipStream_t s) {
    if (a.nchunks > 1) {
        const hipError_t e = reset_chain(a, s);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)(a.nchunks * a.ncols)), block(kWaves * 64);
    if (bf16_io && vec) hipLaunchKernelGGL((gated_scan_kernel<bf16, true>), grid, block, 0, s, a);
    else if (bf16_io) hipLaunchKernelGGL((gated_scan_kernel<bf16, false>), grid, block, 0, s, a);
    else if (vec) hipLaunchKernelGGL((gated_scan_kernel<float, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((gated_scan_kernel<float, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gated_scan_backward(const GatedScanArgs& a, bool bf16_io, bool vec, hipStream_t s) {
    if (a.nchunks > 1) {
        const hipError_t e = reset_chain(a, s);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)(a.nchunks * a.ncols)), block(kWaves * 64);
    if (bf16_io && vec) hipLaunchKernelGGL((gated_scan_backward_kernel<bf16, true>), grid, block, 0, s, a);
    else if (bf16_io) hipLaunchKernelGGL((gated_scan_backward_kernel<bf16, false>), grid, block, 0, s, a);
    else if (vec) hipLaunchKernelGGL((gated_scan_backward_kernel<float, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((gated_scan_backward_kernel<float, false>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.dbias && a.nchunks > 1) e = launch_column_sum(a.part, a.nchunks, a.D, a.dbias, s);
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
