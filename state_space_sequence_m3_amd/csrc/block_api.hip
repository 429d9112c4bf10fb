// block_api.hip -- the C ABI of include/m3block.h: argument validation, workspace sizing and
// dispatch to the kernels of gated_scan.hip, rmsnorm.hip and grad_clip.hip.  Like api.hip it
// computes nothing: every call validates, then only enqueues kernels on the caller's stream.
#include "block_launch.h"
#include "m3_check.h"
#include "m3block.h"

#include <algorithm>
#include <exception>
#include <vector>

namespace {

using m3::aligned;
using m3::check_device;
using m3::fail;
using m3::launched;

constexpr int64_t kMaxCount = (int64_t)1 << 31;   // sequences, tokens, rows, pitches
constexpr int64_t kMaxWidth = (int64_t)1 << 24;
// Outputs of a call that together with its inputs is beyond the last-level cache are stored
// non-temporally: nothing of them would be found there anyway.  16384 rows of 4096 bf16: norm 124 -> 121 us,
// backward 109 -> 106 us; 60 gradients, 482 MB: 292 -> 280 us.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// `rows` rows of `width` bytes, `pitch` bytes apart.
struct Region {
    const void* p;
    int64_t rows, width, pitch;
    const char* name;
    int64_t span() const { return rows > 0 && width > 0 ? (rows - 1) * pitch + width : 0; }
};

// Some byte belongs to both.  Two regions of one pitch may lie in each other's gaps (slices of
// one buffer); regions of different pitches are taken to clash when their spans overlap.
bool clash(const Region& a, const Region& b) {
    if (!m3::overlap(a.p, (size_t)a.span(), b.p, (size_t)b.span())) return false;
    if (a.pitch != b.pitch || (a.rows == 1 && b.rows == 1)) return true;
    const int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p);
    const int64_t delta = ((d % a.pitch) + a.pitch) % a.pitch;
    return !(delta >= a.width && delta + b.width <= a.pitch);
}
bool same(const Region& a, const Region& b) { return a.p == b.p && (a.rows <= 1 || a.pitch == b.pitch); }

m3_status check_clash(const Region& out, const Region& other, bool may_be_same) {
    if (!clash(out, other) || (may_be_same && same(out, other))) return M3_OK;
    return fail(M3_E_ALIAS, "%s overlaps %s", out.name, other.name);
}
m3_status check_need(const Region& r) {
    return !r.p && r.span() > 0 ? fail(M3_E_NULL, "%s is NULL", r.name) : M3_OK;
}
m3_status check_aligned(const void* p, size_t a, const char* name) {
    return p && !aligned(p, a) ? fail(M3_E_ALIGN, "%s is not %zu-byte aligned", name, a) : M3_OK;
}
// pitch in bytes of `rows` rows of `width` elements (0: dense)
m3_status check_pitch(int64_t pitch, int64_t rows, int64_t width, int64_t es, const char* name, int64_t* bytes) {
    const int64_t p = pitch == 0 ? width : pitch;
    if (p < width || p >= kMaxCount)
        return fail(M3_E_DIMS, "%s = %lld must be 0 or from the width %lld to 2^31 - 1", name, (long long)pitch,
                    (long long)width);
    *bytes = p * es;
    int64_t all;
    if (__builtin_mul_overflow(rows, *bytes, &all) || all >= (int64_t)1 << 48)
        return fail(M3_E_DIMS, "%lld rows of %s = %lld: size out of range", (long long)rows, name, (long long)p);
    return M3_OK;
}
m3_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
    if (need == 0) return M3_OK;
    if (!ws || bytes < need)
        return fail(M3_E_WORKSPACE, "%s needs %zu workspace bytes, got %zu", fn, need, ws ? bytes : (size_t)0);
    if (!aligned(ws, 16)) return fail(M3_E_ALIGN, "workspace is not 16-byte aligned");
    return M3_OK;
}

#define M3_TRY(expr)                     \
    do {                                 \
        const m3_status st_ = (expr);    \
        if (st_ != M3_OK) return st_;    \
    } while (0)

// ------------------------------------------------------------------------------- gated scan
struct ScanPlan {
    int64_t T = 0, ntiles = 1, seq_tiles = 1, blocks = 1, seq_blocks = 1;
    int ncols = 0;
    bool per_seq = false, serial = false;
    int64_t parts = 1;
    size_t words_off = 256, marks_off = 0, seqs_off = 0, part_off = 0, bytes = 0;
};

m3_status check_scan_dims(const m3_scan_dims* d) {
    if (!d) return fail(M3_E_NULL, "dims is NULL");
    if (d->io != M3_F32 && d->io != M3_BF16) return fail(M3_E_DTYPE, "dims->io = %d is not M3_F32 or M3_BF16", d->io);
    if (d->flags != 0) return fail(M3_E_DIMS, "dims->flags must be 0");
    if (d->batch < 0 || d->seqlen < 0 || d->width < 0) return fail(M3_E_DIMS, "negative size");
    if (d->batch >= kMaxCount || d->seqlen >= kMaxCount || d->width > kMaxWidth)
        return fail(M3_E_DIMS, "size out of range");
    return M3_OK;
}

// When a workgroup works its sequence off tile by tile instead of chaining tiles that run at the same time (times of
// the builds that both forms were compared in).
// Bf16, D 4096, forward (backward): two tiles of few sequences 14.5 -> 12.9 us (4 x 256 tokens; four tiles lose: 23.1 ->
// 25.1 us); many sequences, which fill the GPU anyway, 88 -> 79 us (161 -> 140) at 64 x 256 tokens, 91 -> 83 us at
// 16 x 1024, but 162 -> 172 us at 8 x 2048 x 8192 channels, 16 tiles.  Packed batches never gain: their tiles wait
// for the search of their sequences, which then adds up.  The forward pass of fp32 holds twice the bytes and spills in
// that form: it gains where there is one tile to a sequence and few of those (4 x 128 tokens 13.6 -> 12.5 us), and
// loses beyond (147 -> 160 us at 64 x 256 tokens); its backward pass gains as bf16 does (260 -> 241 us at 128 x 128).
// Two workgroups on each of 256 compute units, not asked of the device: which batches are cut sequence by sequence decides
// the rows of `states`, which belong to sizes alone.
constexpr int64_t kMaxLoneTiles = 512;
constexpr int64_t kMaxSerialTiles = 2, kMaxFullSerialTiles = 8;
constexpr int64_t kMaxScanBlocks = (int64_t)1 << 23;
// Workgroups that keep the GPU full: no last round of two to a compute unit that is mostly empty.
bool fills_rounds(int64_t wgs) {
    const int64_t slots = 2 * (int64_t)m3::device_cus(), rounds = (wgs + slots - 1) / slots;
    return rounds > 0 && wgs * 100 >= rounds * slots * 85;
}

// The tiles of the forward or the backward pass, and the blocks that have a row of `states`.
m3_status plan_scan(const m3_scan_dims* d, bool packed, bool backward, ScanPlan* p) {
    M3_TRY(check_scan_dims(d));
    constexpr int64_t block = m3::kScanBlock;
    const int64_t tile = backward ? m3::kScanBwdTile : m3::kScanTile;
    p->T = packed ? d->seqlen : d->batch * d->seqlen;
    p->ncols = (int)((d->width + m3::kScanCols - 1) / m3::kScanCols);
    // Short sequences share tiles, unless they are so few that all can have a tile of their own at the same time
    // (then no tile waits for another, and a call is one launch).
    p->per_seq = !packed && d->batch > 0 && d->seqlen > 0 &&
                 (d->seqlen > block || d->batch * p->ncols <= kMaxLoneTiles);
    if (p->per_seq) {
        p->seq_tiles = (d->seqlen + tile - 1) / tile;
        p->seq_blocks = (d->seqlen + block - 1) / block;
        p->ntiles = d->batch * p->seq_tiles;
        p->blocks = d->batch * p->seq_blocks;
    } else {
        p->ntiles = std::max<int64_t>(1, (p->T + tile - 1) / tile);
        p->blocks = std::max<int64_t>(1, (p->T + block - 1) / block);
    }
    // a launch has fewer than 2^32 threads, and 512 of them to a tile
    if (p->blocks >= kMaxScanBlocks || p->blocks * p->ncols >= kMaxScanBlocks)
        return fail(M3_E_DIMS, "%lld tokens of %lld channels: the limit is 2^23 blocks of 64 tokens and 128 channels",
                    (long long)p->T, (long long)d->width);
    const int64_t wgs = p->per_seq ? d->batch * p->ncols : p->ncols;
    p->serial = !p->per_seq                        ? p->ntiles <= 1
                : d->io != M3_BF16 && !backward ? p->seq_tiles <= 1 && wgs <= kMaxLoneTiles
                                                : p->seq_tiles <= kMaxSerialTiles ||
                                                      (p->seq_tiles <= kMaxFullSerialTiles && fills_rounds(wgs));
    p->parts = p->serial ? (p->per_seq ? d->batch : 1) : p->ntiles;
    if (!p->serial) {
        p->marks_off = p->words_off + round256((size_t)p->ntiles * p->ncols * m3::kScanCols * 8);
        p->seqs_off = p->marks_off + (p->per_seq ? 0 : round256((size_t)p->blocks * 16));
        p->part_off = p->seqs_off + (p->per_seq ? 0 : round256((size_t)p->T * 4));
    }
    p->bytes = p->part_off + (backward && p->parts > 1 ? (size_t)p->parts * d->width * 4 : 0);
    return M3_OK;
}

void scan_args(const m3_scan_dims* d, const ScanPlan& p, const int32_t* cu, void* ws, m3::GatedScanArgs* a) {
    a->cu = cu;
    a->b = d->batch;
    a->L = d->seqlen;
    a->T = p.T;
    a->D = d->width;
    a->ntiles = p.ntiles;
    a->seq_tiles = (uint32_t)p.seq_tiles;
    a->seq_blocks = (uint32_t)p.seq_blocks;
    a->ncols = p.ncols;
    a->per_seq = p.per_seq ? 1 : 0;
    a->serial = p.serial ? 1 : 0;
    a->parts = p.parts;
    a->ticket = (unsigned*)ws;
    a->words = (uint64_t*)((char*)ws + p.words_off);
    a->starts = (uint64_t*)((char*)ws + p.marks_off);
    a->ends = a->starts + p.blocks;
    a->seqs = (int*)((char*)ws + p.seqs_off);
    a->part = (float*)((char*)ws + p.part_off);
}

// A tile's rows are addressed with 31-bit offsets from its first one.
constexpr int64_t kMaxScanPitch = ((int64_t)1 << 31) / m3::kScanTile;   // bytes
m3_status check_scan_pitch(int64_t pitch, int64_t rows, int64_t width, int64_t es, const char* name, int64_t* bytes) {
    M3_TRY(check_pitch(pitch, rows, width, es, name, bytes));
    if (*bytes >= kMaxScanPitch)
        return fail(M3_E_DIMS, "%s: rows are %lld bytes apart, the limit is 2^24", name, (long long)*bytes);
    return M3_OK;
}

// Two channels per access: an even width, and rows that start on whole pairs.
bool pairs_ok(int64_t D, int64_t es, const Region* r, int n) {
    if (D % 2 != 0) return false;
    for (int i = 0; i < n; ++i)
        if (!aligned(r[i].p, (size_t)(2 * es)) || r[i].pitch % (2 * es) != 0) return false;
    return true;
}

// ---------------------------------------------------------------------------------- RMS norm
m3_status check_norm_dims(const m3_norm_dims* d) {
    if (!d) return fail(M3_E_NULL, "dims is NULL");
    if (d->io != M3_F32 && d->io != M3_BF16) return fail(M3_E_DTYPE, "dims->io = %d is not M3_F32 or M3_BF16", d->io);
    if (d->flags != 0) return fail(M3_E_DIMS, "dims->flags must be 0");
    if (d->rows < 0 || d->width < 0) return fail(M3_E_DIMS, "negative size");
    if (d->rows >= kMaxCount) return fail(M3_E_DIMS, "size out of range");
    if (d->width > m3::kNormMaxWidth)
        return fail(M3_E_UNSUPPORTED, "width D = %lld is over %lld", (long long)d->width, (long long)m3::kNormMaxWidth);
    if (!(d->eps >= 0.f)) return fail(M3_E_DIMS, "eps must not be negative");
    return M3_OK;
}

// --------------------------------------------------------------------------- gradient tensors
m3_status check_grads(const m3_grad_tensor* t, int64_t n, bool write) {
    if (n < 0 || n >= kMaxCount) return fail(M3_E_DIMS, "count out of range");
    if (n > 0 && !t) return fail(M3_E_NULL, "tensors is NULL");
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].io != M3_F32 && t[i].io != M3_BF16)
            return fail(M3_E_DTYPE, "tensor %lld: io = %d is not M3_F32 or M3_BF16", (long long)i, t[i].io);
        if (t[i].numel < 0 || t[i].numel >= ((int64_t)1 << 40))
            return fail(M3_E_DIMS, "tensor %lld: numel out of range", (long long)i);
        if (t[i].numel == 0) continue;
        if (!t[i].src || (write && !t[i].dst))
            return fail(M3_E_NULL, "tensor %lld: %s is NULL", (long long)i, t[i].src ? "dst" : "src");
        const size_t es = t[i].io == M3_BF16 ? 2 : 4;
        if (!aligned(t[i].src, es) || (write && !aligned(t[i].dst, es)))
            return fail(M3_E_ALIGN, "tensor %lld is not aligned to its elements", (long long)i);
    }
    return M3_OK;
}

// No output may overlap another entry's input or output, nor its own input in part: over all
// extents sorted by address, an output is compared with what starts before its end.
struct Extent {
    uintptr_t lo, hi;
    int64_t i;      // entry
    bool out;
};
m3_status check_grad_overlap(const m3_grad_tensor* t, int64_t n, const Extent* more, int n_more) {
    std::vector<Extent> e;
    e.reserve((size_t)(2 * n + n_more));
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].numel == 0) continue;
        const uintptr_t bytes = (uintptr_t)t[i].numel * (t[i].io == M3_BF16 ? 2 : 4);
        e.push_back({(uintptr_t)t[i].dst, (uintptr_t)t[i].dst + bytes, i, true});
        if (t[i].src != t[i].dst) e.push_back({(uintptr_t)t[i].src, (uintptr_t)t[i].src + bytes, i, false});
    }
    for (int k = 0; k < n_more; ++k) e.push_back(more[k]);
    std::sort(e.begin(), e.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
    // furthest end so far of any extent, and of outputs: a new one must start behind the outputs',
    // a new output behind all of them
    uintptr_t any_hi = 0, out_hi = 0;
    for (const Extent& x : e) {
        if (x.lo < out_hi || (x.out && x.lo < any_hi)) {
            if (x.i >= 0)
                return fail(M3_E_ALIAS, "tensor %lld overlaps another tensor, stats or the workspace", (long long)x.i);
            return fail(M3_E_ALIAS, "stats or the workspace overlap a tensor");
        }
        any_hi = std::max(any_hi, x.hi);
        if (x.out) out_hi = std::max(out_hi, x.hi);
    }
    return M3_OK;
}

struct GradPlan {
    int64_t batches = 0, parts = 0, elements = 0, bytes = 0;
};
// Launch tables of the tensors with elements, kGradBatch to a launch (fewer where their units would
// not fit 32 bits), from the first tensor on or from the last; `each` is called with every table and
// the place of its partial sums.
template <typename F>
m3_status for_batches(const m3_grad_tensor* t, int64_t n, bool back, bool stream, int64_t chunk, F&& each) {
    m3::GradBatch b;
    b.chunk = (int)chunk;
    b.stream = stream ? 1 : 0;
    int64_t k = 0, parts = 0;
    auto at = [&](int64_t i) -> const m3_grad_tensor& { return t[back ? n - 1 - i : i]; };
    while (true) {
        while (k < n && at(k).numel == 0) ++k;
        if (k >= n) return M3_OK;
        b.n = 0;
        b.first[0] = 0;
        for (uint32_t& w : b.is_bf16) w = 0;
        for (; k < n && b.n < m3::kGradBatch; ++k) {
            const m3_grad_tensor& g = at(k);
            if (g.numel == 0) continue;
            const int64_t units = (g.numel + chunk - 1) / chunk;
            if (b.n > 0 && b.first[b.n] + units >= (int64_t)1 << 31) break;
            b.src[b.n] = g.src;
            b.dst[b.n] = g.dst;
            b.numel[b.n] = g.numel;
            if (g.io == M3_BF16) b.is_bf16[b.n >> 5] |= 1u << (b.n & 31);
            b.first[b.n + 1] = (uint32_t)(b.first[b.n] + units);
            ++b.n;
        }
        M3_TRY(each(b, parts));
        parts += m3::grad_blocks(b);
    }
}
GradPlan plan_grads(const m3_grad_tensor* t, int64_t n) {
    GradPlan p;
    for (int64_t i = 0; i < n; ++i) {
        p.elements += t[i].numel;
        p.bytes += t[i].numel * (t[i].io == M3_BF16 ? 2 : 4);
    }
    for_batches(t, n, false, false, m3::kGradChunk, [&](const m3::GradBatch& b, int64_t at) {
        p.batches++;
        p.parts = at + m3::grad_blocks(b);
        return M3_OK;
    });
    return p;
}
bool grad_small(const GradPlan& p) { return p.batches == 1 && p.elements <= m3::kGradSmall; }
// partial sums, and their sum
size_t grad_bytes(const GradPlan& p) { return p.parts == 0 || grad_small(p) ? 0 : (size_t)(p.parts + 1) * 8; }

// As many partial sums are added again by every workgroup of the scaling pass; more are added once, by a
// launch of their own.
constexpr int64_t kMaxSharedParts = 4096;

m3_status grads(const char* fn, bool write, const m3_grad_tensor* t, int64_t n, float max_norm, float* stats,
                void* ws, size_t ws_bytes, hipStream_t stream) {
    M3_TRY(check_grads(t, n, write));
    if (!(max_norm >= 0.f)) return fail(M3_E_DIMS, "max_norm must not be negative");
    if (!stats) return fail(M3_E_NULL, "stats is NULL");
    M3_TRY(check_aligned(stats, 4, "stats"));
    const GradPlan p = plan_grads(t, n);
    M3_TRY(check_workspace(fn, ws, ws_bytes, grad_bytes(p)));
    const Extent more[] = {{(uintptr_t)stats, (uintptr_t)stats + 8, -1, true},
                           {(uintptr_t)ws, (uintptr_t)ws + grad_bytes(p), -1, true}};
    if (write) {
        M3_TRY(check_grad_overlap(t, n, more, grad_bytes(p) ? 2 : 1));
    } else {
        for (int64_t i = 0; i < n; ++i)
            for (const Extent& x : more)
                if (m3::overlap((const void*)x.lo, x.hi - x.lo, t[i].src,
                                (size_t)t[i].numel * (t[i].io == M3_BF16 ? 2 : 4)))
                    return fail(M3_E_ALIAS, "stats or the workspace overlap tensor %lld", (long long)i);
        if (m3::overlap(stats, 8, ws, grad_bytes(p))) return fail(M3_E_ALIAS, "stats overlaps the workspace");
    }
    M3_TRY(check_device());
    double* part = (double*)ws;
    if (grad_small(p))
        return for_batches(t, n, false, false, m3::kGradSmallChunk, [&](const m3::GradBatch& b, int64_t) {
            return launched(m3::launch_grad_small(b, write, max_norm, stats, stream), fn);
        });
    M3_TRY(for_batches(t, n, false, false, m3::kGradChunk, [&](const m3::GradBatch& b, int64_t at) {
        return launched(m3::launch_grad_sumsq(b, part + at, stream), fn);
    }));
    const bool own_stats = !write || p.parts == 0 || p.parts > kMaxSharedParts;
    double* sum = part ? part + p.parts : nullptr;
    if (own_stats)
        M3_TRY(launched(m3::launch_grad_stats(part, p.parts, max_norm, stats, p.parts ? sum : nullptr, stream), fn));
    if (!write) return M3_OK;
    // backwards: what was read last for the sum is still in the last-level cache
    return for_batches(t, n, true, p.bytes * 2 > kCacheBytes, m3::kGradChunk, [&](const m3::GradBatch& b, int64_t at) {
        return launched(m3::launch_grad_scale(b, own_stats ? sum : part, own_stats ? 1 : (int)p.parts, max_norm,
                                              own_stats || at > 0 ? nullptr : stats, stream), fn);
    });
}

// The overlap check sorts a list of its own: running out of host memory there is an error like any other.
m3_status guarded_grads(const char* fn, bool write, const m3_grad_tensor* t, int64_t n, float max_norm, float* stats,
                        void* ws, size_t ws_bytes, hipStream_t stream) {
    try {
        return grads(fn, write, t, n, max_norm, stats, ws, ws_bytes, stream);
    } catch (const std::exception& e) {
        return fail(M3_E_LAUNCH, "%s: %s", fn, e.what());
    }
}

}  // namespace

extern "C" {

int64_t m3_gated_scan_chunks(const m3_scan_dims* d, int packed) {
    ScanPlan p;
    return plan_scan(d, packed != 0, true, &p) == M3_OK ? p.blocks : 0;
}

size_t m3_gated_scan_workspace_bytes(const m3_scan_dims* d, int packed) {
    ScanPlan p;
    return plan_scan(d, packed != 0, false, &p) == M3_OK ? p.bytes : 0;
}

size_t m3_gated_scan_backward_workspace_bytes(const m3_scan_dims* d, int packed) {
    ScanPlan p;
    return plan_scan(d, packed != 0, true, &p) == M3_OK ? p.bytes : 0;
}

m3_status m3_gated_scan(const m3_scan_dims* d, const int32_t* cu_seqlens, const void* gate, const void* x,
                        const float* bias, const float* h_in, void* y, float* h_out, float* states, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    ScanPlan p;
    const bool packed = cu_seqlens != nullptr;
    M3_TRY(plan_scan(d, packed, false, &p));
    const int64_t es = d->io == M3_BF16 ? 2 : 4, D = d->width, b = d->batch;
    int64_t gp, xp, yp;
    M3_TRY(check_scan_pitch(d->gate_pitch, p.T, D, es, "gate_pitch", &gp));
    M3_TRY(check_scan_pitch(d->x_pitch, p.T, D, es, "x_pitch", &xp));
    M3_TRY(check_scan_pitch(d->y_pitch, p.T, D, es, "y_pitch", &yp));
    const Region rg{gate, p.T, D * es, gp, "gate"}, rx{x, p.T, D * es, xp, "x"}, ry{y, p.T, D * es, yp, "y"};
    const Region rb{bias, 1, D * 4, D * 4, "bias"}, rhi{h_in, b, D * 4, D * 4, "h_in"};
    const Region rho{h_out, b, D * 4, D * 4, "h_out"}, rst{states, p.blocks, D * 4, D * 4, "states"};
    const Region rcu{cu_seqlens, packed ? b + 1 : 0, 4, 4, "cu_seqlens"};
    const Region rws{workspace, 1, (int64_t)p.bytes, (int64_t)p.bytes, "workspace"};
    for (const Region* r : {&rg, &rx, &ry, &rho}) M3_TRY(check_need(*r));
    for (const Region* r : {&rg, &rx, &ry}) M3_TRY(check_aligned(r->p, (size_t)es, r->name));
    for (const Region* r : {&rb, &rhi, &rho, &rst, &rcu}) M3_TRY(check_aligned(r->p, 4, r->name));
    M3_TRY(check_workspace("m3_gated_scan", workspace, workspace_bytes, p.bytes));
    const Region* outs[] = {&ry, &rho, &rst, &rws};
    for (int i = 0; i < 4; ++i) {
        for (const Region* in : {&rg, &rx, &rb, &rcu}) M3_TRY(check_clash(*outs[i], *in, false));
        M3_TRY(check_clash(*outs[i], rhi, outs[i] == &rho));
        for (int j = i + 1; j < 4; ++j) M3_TRY(check_clash(*outs[i], *outs[j], false));
    }
    M3_TRY(check_device());
    if (D == 0) return M3_OK;
    m3::GatedScanArgs a{};
    scan_args(d, p, cu_seqlens, workspace, &a);
    a.gate = gate; a.x = x; a.bias = bias; a.h_in = h_in; a.y = y; a.h_out = h_out; a.states = states;
    a.gate_p = gp; a.x_p = xp; a.y_p = yp;
    const Region io[] = {rg, rx, ry};
    return launched(m3::launch_gated_scan(a, es == 2, pairs_ok(D, es, io, 3), stream), "m3_gated_scan");
}

m3_status m3_gated_scan_step(const m3_scan_dims* d, const void* gate, const void* x, const float* bias,
                             const float* h, void* y, float* h_out, hipStream_t stream) {
    M3_TRY(check_scan_dims(d));
    if (d->seqlen != 1) return fail(M3_E_DIMS, "m3_gated_scan_step takes one token: seqlen = %lld", (long long)d->seqlen);
    const int64_t es = d->io == M3_BF16 ? 2 : 4, D = d->width, b = d->batch;
    if (b * D >= kMaxCount)
        return fail(M3_E_DIMS, "%lld rows of %lld channels: the limit is 2^31 elements", (long long)b, (long long)D);
    int64_t gp, xp, yp;
    M3_TRY(check_scan_pitch(d->gate_pitch, b, D, es, "gate_pitch", &gp));
    M3_TRY(check_scan_pitch(d->x_pitch, b, D, es, "x_pitch", &xp));
    M3_TRY(check_scan_pitch(d->y_pitch, b, D, es, "y_pitch", &yp));
    const Region rg{gate, b, D * es, gp, "gate"}, rx{x, b, D * es, xp, "x"}, ry{y, b, D * es, yp, "y"};
    const Region rb{bias, 1, D * 4, D * 4, "bias"}, rhi{h, b, D * 4, D * 4, "h"}, rho{h_out, b, D * 4, D * 4, "h_out"};
    for (const Region* r : {&rg, &rx, &ry, &rhi, &rho}) M3_TRY(check_need(*r));
    for (const Region* r : {&rg, &rx, &ry}) M3_TRY(check_aligned(r->p, (size_t)es, r->name));
    for (const Region* r : {&rb, &rhi, &rho}) M3_TRY(check_aligned(r->p, 4, r->name));
    M3_TRY(check_clash(ry, rg, true));
    M3_TRY(check_clash(ry, rx, true));
    M3_TRY(check_clash(rho, rhi, true));
    for (const Region* r : {&rb, &rhi, &rho}) M3_TRY(check_clash(ry, *r, false));
    for (const Region* r : {&rg, &rx, &rb}) M3_TRY(check_clash(rho, *r, false));
    M3_TRY(check_device());
    if (D == 0 || b == 0) return M3_OK;
    m3::GatedStepArgs a{gate, x, bias, h, y, h_out, b, D, gp, xp, yp};
    // four channels per lane: whole groups in every row
    bool vec = D % 4 == 0 && aligned(h, 16) && aligned(h_out, 16);
    for (const Region* r : {&rg, &rx, &ry}) vec = vec && aligned(r->p, (size_t)(4 * es)) && r->pitch % (4 * es) == 0;
    return launched(m3::launch_gated_step(a, es == 2, vec, stream), "m3_gated_scan_step");
}

m3_status m3_gated_scan_backward(const m3_scan_dims* d, const int32_t* cu_seqlens, const void* gate, const void* x,
                                 const float* bias, const float* h_in, const float* states, const void* dy,
                                 const float* dh_out, void* dgate, void* dx, float* dbias, float* dh_in,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
    ScanPlan p;
    const bool packed = cu_seqlens != nullptr;
    M3_TRY(plan_scan(d, packed, true, &p));
    const int64_t es = d->io == M3_BF16 ? 2 : 4, D = d->width, b = d->batch;
    int64_t gp, xp, yp, dgp, dxp;
    M3_TRY(check_scan_pitch(d->gate_pitch, p.T, D, es, "gate_pitch", &gp));
    M3_TRY(check_scan_pitch(d->x_pitch, p.T, D, es, "x_pitch", &xp));
    M3_TRY(check_scan_pitch(d->y_pitch, p.T, D, es, "y_pitch", &yp));
    M3_TRY(check_scan_pitch(d->dgate_pitch, p.T, D, es, "dgate_pitch", &dgp));
    M3_TRY(check_scan_pitch(d->dx_pitch, p.T, D, es, "dx_pitch", &dxp));
    const Region rg{gate, p.T, D * es, gp, "gate"}, rx{x, p.T, D * es, xp, "x"}, rdy{dy, p.T, D * es, yp, "dy"};
    const Region rdg{dgate, p.T, D * es, dgp, "dgate"}, rdx{dx, p.T, D * es, dxp, "dx"};
    const Region rb{bias, 1, D * 4, D * 4, "bias"}, rhi{h_in, b, D * 4, D * 4, "h_in"};
    const Region rst{states, p.blocks, D * 4, D * 4, "states"}, rdho{dh_out, b, D * 4, D * 4, "dh_out"};
    const Region rdb{dbias, 1, D * 4, D * 4, "dbias"}, rdhi{dh_in, b, D * 4, D * 4, "dh_in"};
    const Region rcu{cu_seqlens, packed ? b + 1 : 0, 4, 4, "cu_seqlens"};
    const Region rws{workspace, 1, (int64_t)p.bytes, (int64_t)p.bytes, "workspace"};
    for (const Region* r : {&rg, &rx, &rdy, &rdg, &rdx, &rst}) M3_TRY(check_need(*r));
    for (const Region* r : {&rg, &rx, &rdy, &rdg, &rdx}) M3_TRY(check_aligned(r->p, (size_t)es, r->name));
    for (const Region* r : {&rb, &rhi, &rst, &rdho, &rdb, &rdhi, &rcu}) M3_TRY(check_aligned(r->p, 4, r->name));
    M3_TRY(check_workspace("m3_gated_scan_backward", workspace, workspace_bytes, p.bytes));
    const Region* outs[] = {&rdg, &rdx, &rdb, &rdhi, &rws};
    for (int i = 0; i < 5; ++i) {
        for (const Region* in : {&rg, &rx, &rdy, &rb, &rhi, &rst, &rdho, &rcu}) M3_TRY(check_clash(*outs[i], *in, false));
        for (int j = i + 1; j < 5; ++j) M3_TRY(check_clash(*outs[i], *outs[j], false));
    }
    M3_TRY(check_device());
    if (D == 0) return M3_OK;
    m3::GatedScanArgs a{};
    scan_args(d, p, cu_seqlens, workspace, &a);
    a.gate = gate; a.x = x; a.bias = bias; a.h_in = h_in; a.states = const_cast<float*>(states);
    a.dy = dy; a.dh_out = dh_out; a.dgate = dgate; a.dx = dx; a.dbias = dbias; a.dh_in = dh_in;
    a.gate_p = gp; a.x_p = xp; a.y_p = yp; a.dgate_p = dgp; a.dx_p = dxp;
    const Region io[] = {rg, rx, rdy, rdg, rdx};
    return launched(m3::launch_gated_scan_backward(a, es == 2, pairs_ok(D, es, io, 5), stream),
                    "m3_gated_scan_backward");
}

m3_status m3_rmsnorm(const m3_norm_dims* d, const void* x, const void* residual, const float* weight, void* r_out,
                     void* y, void* q, float* scale, hipStream_t stream) {
    M3_TRY(check_norm_dims(d));
    if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128 && d->group != 256)
        return fail(M3_E_UNSUPPORTED, "group = %lld is not 0, 32, 64, 128 or 256", (long long)d->group);
    const int64_t es = d->io == M3_BF16 ? 2 : 4, D = d->width, n = d->rows;
    const int64_t ng = d->group == 0 ? (D > 0 ? 1 : 0) : (D + d->group - 1) / d->group;
    int64_t xp, pp, rp, yp;
    M3_TRY(check_pitch(d->x_pitch, n, D, es, "x_pitch", &xp));
    M3_TRY(check_pitch(d->res_pitch, n, D, es, "res_pitch", &pp));
    M3_TRY(check_pitch(d->r_pitch, n, D, es, "r_pitch", &rp));
    M3_TRY(check_pitch(d->y_pitch, n, D, es, "y_pitch", &yp));
    if (!y && !q && n > 0 && D > 0) return fail(M3_E_NULL, "y and q are NULL");
    if ((q == nullptr) != (scale == nullptr)) return fail(M3_E_NULL, "q and scale go together");
    const Region rx{x, n, D * es, xp, "x"}, rres{residual, n, D * es, pp, "residual"};
    const Region rr{r_out, n, D * es, rp, "r_out"}, ry{y, n, D * es, yp, "y"};
    const Region rw{weight, 1, D * 4, D * 4, "weight"};
    const Region rq{q, n, D, D, "q"}, rs{scale, n, ng * 4, ng * 4, "scale"};
    M3_TRY(check_need(rx));
    for (const Region* r : {&rx, &rres, &rr, &ry}) M3_TRY(check_aligned(r->p, (size_t)es, r->name));
    for (const Region* r : {&rw, &rs}) M3_TRY(check_aligned(r->p, 4, r->name));
    const Region* outs[] = {&rr, &ry, &rq, &rs};
    for (int i = 0; i < 4; ++i) {
        for (const Region* in : {&rx, &rres}) M3_TRY(check_clash(*outs[i], *in, i < 2));
        M3_TRY(check_clash(*outs[i], rw, false));
        for (int j = i + 1; j < 4; ++j) M3_TRY(check_clash(*outs[i], *outs[j], false));
    }
    M3_TRY(check_device());
    if (n == 0 || D == 0) return M3_OK;
    m3::RmsNormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.r_out = r_out; a.y = y;
    a.q = (uint8_t*)q; a.scale = scale;
    a.rows = n; a.D = (int)D; a.x_p = xp; a.res_p = pp; a.r_p = rp; a.y_p = yp;
    a.group = d->group >= D ? 0 : (int)d->group;   // one group: the row
    a.ngroups = (int)ng;
    a.eps = d->eps;
    a.cus = m3::device_cus();
    const int64_t moved = es * (1 + (residual != nullptr) + (r_out != nullptr) + (y != nullptr)) + (q != nullptr);
    a.stream = n * D * moved > kCacheBytes;
    return launched(m3::launch_rmsnorm(a, es == 2, stream), "m3_rmsnorm");
}

size_t m3_rmsnorm_backward_workspace_bytes(const m3_norm_dims* d) {
    if (check_norm_dims(d) != M3_OK || d->rows == 0 || d->width == 0) return 0;
    return (size_t)m3::rmsnorm_backward_parts(d->rows, d->width, d->io == M3_BF16, m3::device_cus()) * d->width * 4;
}

m3_status m3_rmsnorm_backward(const m3_norm_dims* d, const void* r, const float* weight, const void* dy,
                              const void* dr_out, void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    M3_TRY(check_norm_dims(d));
    const int64_t es = d->io == M3_BF16 ? 2 : 4, D = d->width, n = d->rows;
    int64_t rp, yp, pp, dxp;
    M3_TRY(check_pitch(d->r_pitch, n, D, es, "r_pitch", &rp));
    M3_TRY(check_pitch(d->y_pitch, n, D, es, "y_pitch", &yp));
    M3_TRY(check_pitch(d->res_pitch, n, D, es, "res_pitch", &pp));
    M3_TRY(check_pitch(d->dx_pitch, n, D, es, "dx_pitch", &dxp));
    const Region rr{r, n, D * es, rp, "r"}, rdy{dy, n, D * es, yp, "dy"}, rdr{dr_out, n, D * es, pp, "dr_out"};
    const Region rdx{dx, n, D * es, dxp, "dx"}, rw{weight, 1, D * 4, D * 4, "weight"};
    const Region rdw{dweight, 1, D * 4, D * 4, "dweight"};
    const int64_t need = dweight ? (int64_t)m3_rmsnorm_backward_workspace_bytes(d) : 0;
    const Region rws{workspace, 1, need, need, "workspace"};
    for (const Region* q : {&rr, &rdy, &rdx}) M3_TRY(check_need(*q));
    for (const Region* q : {&rr, &rdy, &rdr, &rdx}) M3_TRY(check_aligned(q->p, (size_t)es, q->name));
    for (const Region* q : {&rw, &rdw}) M3_TRY(check_aligned(q->p, 4, q->name));
    M3_TRY(check_workspace("m3_rmsnorm_backward", workspace, workspace_bytes, (size_t)need));
    const Region* outs[] = {&rdx, &rdw, &rws};
    for (int i = 0; i < 3; ++i) {
        for (const Region* in : {&rr, &rdy, &rdr, &rw})
            M3_TRY(check_clash(*outs[i], *in, i == 0 && (in == &rdy || in == &rdr)));
        for (int j = i + 1; j < 3; ++j) M3_TRY(check_clash(*outs[i], *outs[j], false));
    }
    M3_TRY(check_device());
    if (D == 0) return M3_OK;
    if (n == 0) return dweight ? launched(m3::launch_column_sum(nullptr, 0, D, dweight, stream), "m3_rmsnorm_backward")
                               : M3_OK;
    m3::RmsNormArgs a{};
    a.r = r; a.dy = dy; a.dr_out = dr_out; a.weight = weight; a.dx = dx; a.dweight = dweight;
    a.part = dweight ? (float*)workspace : nullptr;
    a.rows = n; a.D = (int)D; a.r_p = rp; a.y_p = yp; a.res_p = pp; a.dx_p = dxp;
    a.eps = d->eps;
    a.cus = m3::device_cus();
    a.stream = n * D * es * (3 + (dr_out != nullptr)) > kCacheBytes;
    return launched(m3::launch_rmsnorm_backward(a, es == 2, stream), "m3_rmsnorm_backward");
}

size_t m3_grad_workspace_bytes(const m3_grad_tensor* tensors, int64_t count) {
    if (count < 0 || count >= kMaxCount || (count > 0 && !tensors)) return 0;
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].numel < 0 || tensors[i].numel >= ((int64_t)1 << 40)) return 0;
    return grad_bytes(plan_grads(tensors, count));
}

m3_status m3_grad_norm(const m3_grad_tensor* tensors, int64_t count, float max_norm, float* stats, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    return guarded_grads("m3_grad_norm", false, tensors, count, max_norm, stats, workspace, workspace_bytes, stream);
}

m3_status m3_grad_clip(const m3_grad_tensor* tensors, int64_t count, float max_norm, float* stats, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    return guarded_grads("m3_grad_clip", true, tensors, count, max_norm, stats, workspace, workspace_bytes, stream);
}

}  // extern "C"
