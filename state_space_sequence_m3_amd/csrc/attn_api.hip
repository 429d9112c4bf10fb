// attn_api.hip -- the C ABI of include/m3attn.h: argument validation, workspace sizing and dispatch to the
// kernels of attention.hip, attention_backward.hip, cache_append.hip and attention_step.hip.  Like block_api.hip
// it computes nothing: every call validates, then only enqueues kernels on the caller's stream.
#include "attn_launch.h"
#include "m3_check.h"
#include "m3_page_map.h"
#include "m3attn.h"

#include <math.h>

#include <algorithm>

namespace {

using m3::aligned;
using m3::check_device;
using m3::fail;
using m3::launched;

constexpr int64_t kMaxCount = (int64_t)1 << 31;
constexpr int64_t kMaxSpan = (int64_t)1 << 48;       // bytes of a tensor, gaps included
constexpr int64_t kMaxTokenBytes = (int64_t)1 << 24; // 128 rows of a tile are addressed with 31 bits
constexpr int64_t kMaxGroups = (int64_t)1 << 24;     // a launch has fewer than 2^32 threads, 256 to a workgroup

#define M3_TRY(expr)                  \
    do {                              \
        const m3_status st_ = (expr); \
        if (st_ != M3_OK) return st_; \
    } while (0)

// Rows of `row` bytes in up to three dimensions: sizes n and strides s in bytes.
struct Area {
    const char* name = "";
    const void* p = nullptr;
    int64_t row = 0;
    int64_t n[3] = {1, 1, 1}, s[3] = {0, 0, 0};
    bool empty() const { return row <= 0 || n[0] <= 0 || n[1] <= 0 || n[2] <= 0; }
    int64_t span() const {
        return empty() ? 0 : row + (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + (n[2] - 1) * s[2];
    }
};
Area flat(const void* p, int64_t bytes, const char* name) {
    Area a;
    a.p = p, a.row = bytes, a.name = name;
    return a;
}

// The bytes from the area's start, modulo a period, that are within `extent`: false where there is no such bound.
bool folds(const Area& a, int64_t period, int64_t* extent) {
    int64_t e = a.row;
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] <= 1 || a.s[i] % period == 0) continue;
        e += (a.n[i] - 1) * a.s[i];
    }
    *extent = e;
    return e <= period;
}
// Some byte may belong to both: their spans overlap, and no stride that both have keeps them apart.
bool clash(const Area& a, const Area& b) {
    if (!m3::overlap(a.p, (size_t)a.span(), b.p, (size_t)b.span())) return false;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            const int64_t period = a.s[i];
            int64_t ea, eb;
            if (a.n[i] <= 1 || b.n[j] <= 1 || period <= 0 || b.s[j] != period) continue;
            if (!folds(a, period, &ea) || !folds(b, period, &eb)) continue;
            const int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p), delta = ((d % period) + period) % period;
            if (delta >= ea && delta + eb <= period) return false;
        }
    return true;
}
bool same(const Area& a, const Area& b) {
    if (a.p != b.p || a.row != b.row) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.s[i] != b.s[i])) return false;
    return true;
}
m3_status check_clash(const Area& out, const Area& other, bool may_be_same = false) {
    if (!clash(out, other) || (may_be_same && same(out, other))) return M3_OK;
    return fail(M3_E_ALIAS, "%s overlaps %s", out.name, other.name);
}
// No byte of an output is written twice: each stride is beyond all that smaller ones reach.
m3_status check_apart(const Area& a) {
    if (a.empty()) return M3_OK;
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int i, int j) { return a.s[i] < a.s[j]; });
    int64_t e = a.row;
    for (int i : order) {
        if (a.n[i] <= 1) continue;
        if (a.s[i] < e) return fail(M3_E_ALIAS, "%s overlaps itself (its strides)", a.name);
        e += (a.n[i] - 1) * a.s[i];
    }
    return M3_OK;
}
m3_status check_need(const Area& a) {
    return !a.p && a.span() > 0 ? fail(M3_E_NULL, "%s is NULL", a.name) : M3_OK;
}
m3_status check_aligned(const Area& a, size_t n) {
    return a.p && !aligned(a.p, n) ? fail(M3_E_ALIGN, "%s is not %zu-byte aligned", a.name, n) : M3_OK;
}
m3_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
    if (need == 0) return M3_OK;
    if (!ws || bytes < need)
        return fail(M3_E_WORKSPACE, "%s needs %zu workspace bytes, got %zu", fn, need, ws ? bytes : (size_t)0);
    if (!aligned(ws, 16)) return fail(M3_E_ALIGN, "workspace is not 16-byte aligned");
    return M3_OK;
}

// The area of heads with `n` and strides `s` in elements ({0, 0, 0}: dense in the order given), checked.  tokens: which
// of the three is the token's.
m3_status make_area(Area* a, const void* p, const char* name, const int64_t (&n)[3], const int64_t (&s)[3], int64_t dim,
                    int64_t es, int tokens) {
    a->p = p, a->name = name, a->row = dim * es;
    const bool dense = s[0] == 0 && s[1] == 0 && s[2] == 0;
    int64_t at = dim;
    for (int i = 2; i >= 0; --i) {
        int64_t st = dense ? at : s[i];
        if (dense && __builtin_mul_overflow(at, n[i] > 1 ? n[i] : 1, &at))
            return fail(M3_E_DIMS, "%s: size out of range", name);
        if (n[i] <= 1) st = i == tokens ? dim : 0;   // a second row would be past the end
        if (st < 0 || st >= kMaxSpan) return fail(M3_E_DIMS, "%s: stride %lld out of range", name, (long long)st);
        st *= es;
        if (st % 16 != 0) return fail(M3_E_ALIGN, "%s: strides must be multiples of 16 bytes", name);
        if (i == tokens && st >= kMaxTokenBytes)
            return fail(M3_E_DIMS, "%s: tokens are %lld bytes apart, the limit is 2^24", name, (long long)st);
        int64_t reach;
        if (n[i] > 1 && (__builtin_mul_overflow(n[i] - 1, st, &reach) || reach >= kMaxSpan))
            return fail(M3_E_DIMS, "%s: size out of range", name);
        a->n[i] = n[i], a->s[i] = st;
    }
    return check_aligned(*a, 16);
}
m3::HeadRows rows_of(const Area& a) { return {(char*)const_cast<void*>(a.p), a.s[0], a.s[2], (uint32_t)a.s[1]}; }

m3_status check_heads(int64_t heads, int64_t kv_heads, int64_t dim, int32_t io) {
    if (io != M3_F32 && io != M3_BF16) return fail(M3_E_DTYPE, "dims->io = %d is not M3_F32 or M3_BF16", io);
    if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || heads >= (1 << 20))
        return fail(M3_E_DIMS, "heads = %lld must be a multiple of kv_heads = %lld, both at least 1", (long long)heads,
                    (long long)kv_heads);
    if (dim < 8 || dim % 8 != 0) return fail(M3_E_DIMS, "head_dim D = %lld must be a multiple of 8", (long long)dim);
    if (dim > m3::kAttnMaxDim)
        return fail(M3_E_UNSUPPORTED, "head_dim D = %lld is over %lld", (long long)dim, (long long)m3::kAttnMaxDim);
    return M3_OK;
}
m3_status check_counts(int64_t batch, int64_t seqlen) {
    if (batch < 0 || seqlen < 0) return fail(M3_E_DIMS, "negative size");
    if (batch >= kMaxCount || seqlen >= kMaxCount) return fail(M3_E_DIMS, "size out of range");
    return M3_OK;
}
m3_status check_scale(float scale, int64_t dim, float* use) {
    if (!(scale >= 0.f) || scale > 2.3e38f)   // its product with log2 e is an fp32 number
        return fail(M3_E_DIMS, "scale must be positive and at most 2.3e38, or 0 for 1 / sqrt(D)");
    *use = scale > 0.f ? scale : (float)(1.0 / sqrt((double)dim));
    return M3_OK;
}
m3_status check_groups(int64_t a, int64_t b, int64_t c) {
    int64_t n;
    if (__builtin_mul_overflow(a, b, &n) || __builtin_mul_overflow(n, c, &n) || n >= kMaxGroups)
        return fail(M3_E_DIMS, "more work than one launch takes (2^24 workgroups)");
    return M3_OK;
}

// ------------------------------------------------------------------------- whole prompts
// Blocks of R rows of all sequences of a head (packed: as many as there can be).
int64_t row_blocks(const m3_attn_dims* d, bool packed, int64_t R) {
    return packed ? d->seqlen / R + d->batch : (d->seqlen + R - 1) / R * d->batch;
}
// Workgroups of 128 rows need to be many: where they are at most so many, blocks of 32 rows are taken, whose waves
// share the other axis.  Forward, at 256 of them: 4096 x 8 heads of 128 bf16 86 -> 73 us, 4 x 1024 29.5 -> 29.6, fp32
// 155 -> 129; at 320: 2560 x 16 bf16 54.6 -> 61.3, fp32 355 -> 335; at 384: 4 x 1024 x 12 bf16 30.1 -> 43.5, 3 x 1024 x 16
// fp32 155 -> 196; at 512: 2 x 2048 x 16 heads bf16 57 -> 80, fp32 321 -> 429.  dk and dv (with dq) in bf16: at 320 blocks of
// keys 2560 x 16 235 -> 230, at 384 4 x 1024 x 12 113 -> 149, at 512 2 x 2048 x 16 202 -> 287; in fp32 they gain at 512 (4 x
// 2048, 32/8 heads 5051 -> 4704, 4096, 32/16 heads 4897 -> 4468) and lose at 640 (4 x 1024 x 20 945 -> 976) and 1024 (1394
// -> 1498).
// (A packed batch's block numbers are taken to be half a sequence's too many each.)
constexpr int64_t kFewBlocks = 256, kFewKeyBlocks = 256, kFewKeyBlocks32 = 512;
// dk and dv: the heads of a group are summed by one workgroup, or split over as many as make this number of blocks,
// whose parts are added up by another launch.  Bf16, with dq, parts for 512, 1024 and 2048 blocks: 2 x 2048, 64/8 heads
// of 128 758, 577 and 638 us, 4 x 2048, 32/8 heads 733, 586 and 653 us, 16 x 512, 32/8 heads 240, 269 and 330 us.  Blocks of
// 32 keys, for 64, 128 and 256: 2048 x 8/2 heads 113, 93 and 92 us, fp32 482, 345 and 344.
// Parts are equal where a number of them that divides the group makes at most twice as many blocks (and 2^18 rows of parts,
// 268 MB at 128 elements), else uneven ones for one and a half times as many.  Parts, backward in us: 16384 tokens, 28/4
// heads of 128 2: 7558, 3: 7228, 4: 7543, 7: 6995 (but 470 MB of parts); 8192, 40/8 heads 2: 2643, 3: 2401, 5: 2418.
constexpr int64_t kSplitBlocks = 1024, kSplitFew = 128;
// dk and dv of long sequences in bf16, heads over 64 elements: 8 waves with 256 keys share tiles of 64 rows instead of 4
// waves with 128 tiles of 32, half as many barriers and loads (8 x 2048, 32/8 heads of 128, with dq: 1108 -> 1056 us, 8 x
// 1024 408 -> 383; but 16 x 768, 16 heads 245 -> 258, 32 x 300 282 -> 306, since a last block is half empty on average).
constexpr int64_t kWideLength = 1024;
struct KeyPlan {
    int splits = 1;
    bool few = false, wide = false;
};
int64_t full_blocks(const m3_attn_dims* d, bool packed) {
    return row_blocks(d, packed, m3::kAttnRows) - (packed ? d->batch / 2 : 0);
}
KeyPlan plan_keys(const m3_attn_dims* d, bool packed) {
    const int64_t n = full_blocks(d, packed) * d->kv_heads;
    auto split = [&](int64_t to) {
        const int64_t group = d->kv_heads * d->head_dim * 4 < kMaxTokenBytes ? d->heads / d->kv_heads : 1;
        if (n < 1 || n >= to) return 1;
        const int64_t least = std::min(group, (to + n - 1) / n);
        for (int64_t s = least; s <= group && n * s <= 2 * to; ++s)
            if (group % s == 0) return (int)s;
        return (int)std::max(least, 3 * to / 2 / n);
    };
    KeyPlan p;
    if (d->io == M3_BF16) {
        p.splits = split(kSplitBlocks);
        p.few = n * p.splits <= kFewKeyBlocks;
    } else {
        p.few = n <= kFewKeyBlocks32;
    }
    if (p.few) p.splits = split(kSplitFew);
    const int64_t length = packed ? d->seqlen / std::max<int64_t>(1, d->batch) : d->seqlen;
    p.wide = !p.few && d->io == M3_BF16 && d->head_dim > 64 && length >= kWideLength;
    return p;
}

struct Attn {
    int64_t b, L, rows;   // rows: tokens of all sequences
    float scale;
    Area q, k, v, o, lse, cu;
    m3::AttnArgs args;
};
m3_status heads_area(Area* a, const m3_attn_dims* d, bool packed, const void* p, const m3_head_strides& s, int64_t heads,
                     const char* name) {
    return make_area(a, p, name, {packed ? 1 : d->batch, d->seqlen, heads}, {s.batch, s.token, s.head}, d->head_dim,
                     d->io == M3_BF16 ? 2 : 4, 1);
}
m3_status check_attn(const m3_attn_dims* d, bool packed) {
    if (!d) return fail(M3_E_NULL, "dims is NULL");
    M3_TRY(check_heads(d->heads, d->kv_heads, d->head_dim, d->io));
    if (d->flags != 0) return fail(M3_E_DIMS, "dims->flags must be 0");
    M3_TRY(check_counts(d->batch, d->seqlen));
    return check_groups(row_blocks(d, packed, m3::kAttnRows), d->heads, 1);
}
uint32_t blocks_of(const m3_attn_dims* d, bool packed, int64_t R) {   // of the batch, dense: of a sequence
    const int64_t n = row_blocks(d, packed, R);
    return (uint32_t)(packed || d->batch == 0 ? n : n / d->batch);
}
m3_status plan_attn(Attn* p, const m3_attn_dims* d, const int32_t* cu, const void* q, const void* k, const void* v,
                    const void* o, const float* lse) {
    const bool packed = cu != nullptr;
    M3_TRY(check_attn(d, packed));
    M3_TRY(check_scale(d->scale, d->head_dim, &p->scale));
    p->b = d->batch, p->L = d->seqlen, p->rows = packed ? d->seqlen : d->batch * d->seqlen;
    M3_TRY(heads_area(&p->q, d, packed, q, d->q, d->heads, "q"));
    M3_TRY(heads_area(&p->k, d, packed, k, d->k, d->kv_heads, "k"));
    M3_TRY(heads_area(&p->v, d, packed, v, d->v, d->kv_heads, "v"));
    M3_TRY(heads_area(&p->o, d, packed, o, d->o, d->heads, "o"));
    p->lse = flat(lse, p->rows * d->heads * 4, "lse");
    p->cu = flat(cu, packed ? (d->batch + 1) * 4 : 0, "cu_seqlens");
    for (const Area* a : {&p->q, &p->k, &p->v, &p->o}) M3_TRY(check_need(*a));
    for (const Area* a : {&p->lse, &p->cu}) M3_TRY(check_aligned(*a, 4));
    m3::AttnArgs& a = p->args;
    a = m3::AttnArgs{};
    a.q = rows_of(p->q), a.k = rows_of(p->k), a.v = rows_of(p->v), a.o = rows_of(p->o);
    a.lse = const_cast<float*>(lse);
    a.cu = cu;
    a.b = d->batch, a.L = d->seqlen;
    a.heads = (int)d->heads, a.kv_heads = (int)d->kv_heads, a.dim = (int)d->head_dim;
    a.scale = p->scale;
    const KeyPlan keys = plan_keys(d, packed);
    a.few = full_blocks(d, packed) * d->heads <= kFewBlocks;
    a.kfew = keys.few;
    a.splits = keys.splits;
    // a tile of kAttnWide values is addressed with 31 bits
    a.kwide = keys.wide && p->v.s[1] < kMaxTokenBytes / 2;
    a.blocks = blocks_of(d, packed, a.few ? m3::kAttnFew : m3::kAttnRows);
    a.kblocks = blocks_of(d, packed, a.kfew ? m3::kAttnFew : a.kwide ? m3::kAttnWide : m3::kAttnRows);
    return M3_OK;
}
// delta, then the parts of dk and dv
size_t delta_bytes(const m3_attn_dims* d, bool packed) {
    return ((size_t)(packed ? d->seqlen : d->batch * d->seqlen) * (size_t)d->heads * 4 + 15) & ~(size_t)15;
}
size_t backward_bytes(const m3_attn_dims* d, bool packed) {
    const size_t rows = (size_t)(packed ? d->seqlen : d->batch * d->seqlen), splits = (size_t)plan_keys(d, packed).splits;
    return delta_bytes(d, packed) + (splits > 1 ? 2 * splits * rows * (size_t)(d->kv_heads * d->head_dim) * 4 : 0);
}

// --------------------------------------------------------------------------- paged cache
struct Cache {
    int64_t es;
    Area k, v, table, lens;
    m3::Pages pages;
};
m3_status check_cache_dims(const m3_cache_dims* d, uint32_t flags) {
    if (!d) return fail(M3_E_NULL, "dims is NULL");
    M3_TRY(check_heads(d->heads, d->kv_heads, d->head_dim, d->io));
    if (d->flags & ~flags) return fail(M3_E_DIMS, "dims->flags has unknown bits");
    M3_TRY(check_counts(d->batch, d->seqlen));
    if (d->num_pages < 0 || d->table_width < 0 || d->page_size < 1) return fail(M3_E_DIMS, "negative size, or page_size < 1");
    if (d->num_pages >= kMaxCount || d->table_width >= kMaxCount || d->page_size >= kMaxCount)
        return fail(M3_E_DIMS, "size out of range");
    return M3_OK;
}
m3_status plan_cache(Cache* c, const m3_cache_dims* d, const void* k, const void* v, const int32_t* table,
                     const int32_t* lens) {
    c->es = d->io == M3_BF16 ? 2 : 4;
    const int64_t n[3] = {d->num_pages, d->kv_heads, d->page_size};
    M3_TRY(make_area(&c->k, k, "k_cache", n, {d->k_cache.page, d->k_cache.head, d->k_cache.token}, d->head_dim, c->es, 2));
    M3_TRY(make_area(&c->v, v, "v_cache", n, {d->v_cache.page, d->v_cache.head, d->v_cache.token}, d->head_dim, c->es, 2));
    if (d->batch * d->table_width >= kMaxSpan) return fail(M3_E_DIMS, "page_table: size out of range");
    c->table = flat(table, d->batch * d->table_width * 4, "page_table");
    c->lens = flat(lens, d->batch * 4, "lens");
    for (const Area* a : {&c->table, &c->lens}) M3_TRY(check_aligned(*a, 4));
    m3::Pages& p = c->pages;
    p.k = (char*)const_cast<void*>(k), p.v = (char*)const_cast<void*>(v);
    p.k_page = c->k.s[0], p.k_head = c->k.s[1], p.k_token = (uint32_t)c->k.s[2];
    p.v_page = c->v.s[0], p.v_head = c->v.s[1], p.v_token = (uint32_t)c->v.s[2];
    p.table = table;
    p.table_w = d->table_width;
    p.n = (int32_t)d->num_pages, p.size = (int32_t)d->page_size;
    p.shift = -1;
    for (int i = 0; i < 31; ++i)
        if (d->page_size == (int64_t)1 << i) p.shift = i;
    return M3_OK;
}

// How a decoding batch is cut: into as many pieces per key head (and block of 16 query heads) as fill the GPU once,
// two workgroups to a compute unit, but none shorter than a round of a workgroup.  Sequences that cannot be longer than
// a round are a piece each.  (64 sequences of 2048, 32/8 heads of 128 bf16, with one, two and four times as many pieces: 103,
// 111 and 120 us.)
struct StepPlan {
    int64_t items = 1, head_blocks = 1;
    bool joined = true;
    size_t bytes = 0;
};
m3_status plan_step(const m3_cache_dims* d, StepPlan* p) {
    M3_TRY(check_cache_dims(d, 0));
    p->head_blocks = (d->heads / d->kv_heads + 15) / 16;
    const int64_t most = d->table_width * d->page_size;   // below 2^62
    p->joined = most <= m3::kRound || d->batch == 0;
    p->items = d->batch;
    if (!p->joined) {
        const int64_t want = 2 * (int64_t)m3::device_cus() / (d->kv_heads * p->head_blocks);
        const int64_t per = most / m3::kRound + 1, all = per > kMaxCount / d->batch ? kMaxCount : per * d->batch;
        p->items = std::max<int64_t>(1, std::min(want, all));
    }
    M3_TRY(check_groups(p->items, d->kv_heads, p->head_blocks));
    M3_TRY(check_groups(d->batch, d->heads, 1));
    if (!p->joined) p->bytes = (size_t)(p->items + d->batch) * (size_t)d->heads * (size_t)(2 + d->head_dim) * 4;
    return M3_OK;
}

}  // namespace

extern "C" {

m3_status m3_attention(const m3_attn_dims* d, const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                       void* o, float* lse, hipStream_t stream) {
    Attn p;
    M3_TRY(plan_attn(&p, d, cu_seqlens, q, k, v, o, lse));
    const Area* outs[] = {&p.o, &p.lse};
    M3_TRY(check_apart(p.o));
    for (const Area* out : outs)
        for (const Area* in : {&p.q, &p.k, &p.v, &p.cu}) M3_TRY(check_clash(*out, *in));
    M3_TRY(check_clash(p.o, p.lse));
    M3_TRY(check_device());
    if (p.rows == 0 || p.b == 0) return M3_OK;
    return launched(m3::launch_attention(p.args, d->io == M3_BF16, stream), "m3_attention");
}

size_t m3_attention_backward_workspace_bytes(const m3_attn_dims* d, int packed) {
    return check_attn(d, packed != 0) == M3_OK ? backward_bytes(d, packed != 0) : 0;
}

m3_status m3_attention_backward(const m3_attn_dims* d, const int32_t* cu_seqlens, const void* q, const void* k,
                                const void* v, const void* o, const float* lse, const void* dout, void* dq, void* dk,
                                void* dv, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    Attn p;
    M3_TRY(plan_attn(&p, d, cu_seqlens, q, k, v, o, lse));
    const bool packed = cu_seqlens != nullptr;
    Area ado, adq, adk, adv;
    M3_TRY(heads_area(&ado, d, packed, dout, d->dout, d->heads, "dout"));
    M3_TRY(heads_area(&adq, d, packed, dq, d->dq, d->heads, "dq"));
    M3_TRY(heads_area(&adk, d, packed, dk, d->dk, d->kv_heads, "dk"));
    M3_TRY(heads_area(&adv, d, packed, dv, d->dv, d->kv_heads, "dv"));
    for (const Area* a : {&p.lse, &ado, &adq, &adk, &adv}) M3_TRY(check_need(*a));
    const size_t need = backward_bytes(d, packed);
    M3_TRY(check_workspace("m3_attention_backward", workspace, workspace_bytes, need));
    const Area ws = flat(workspace, (int64_t)need, "workspace");
    const Area* outs[] = {&adq, &adk, &adv, &ws};
    for (int i = 0; i < 4; ++i) {
        M3_TRY(check_apart(*outs[i]));
        for (const Area* in : {&p.q, &p.k, &p.v, &p.o, &p.lse, &ado, &p.cu}) M3_TRY(check_clash(*outs[i], *in));
        for (int j = i + 1; j < 4; ++j) M3_TRY(check_clash(*outs[i], *outs[j]));
    }
    M3_TRY(check_device());
    if (p.rows == 0 || p.b == 0) return M3_OK;
    p.args.dout = rows_of(ado), p.args.dq = rows_of(adq), p.args.dk = rows_of(adk), p.args.dv = rows_of(adv);
    p.args.delta = (float*)workspace;
    p.args.part = (float*)((char*)workspace + delta_bytes(d, packed));
    return launched(m3::launch_attention_backward(p.args, d->io == M3_BF16, stream), "m3_attention_backward");
}

m3_status m3_cache_append(const m3_cache_dims* d, const int32_t* cu_seqlens, const int32_t* lens, const float* inv_freq,
                          const void* q, const void* k, const void* v, void* q_out, void* k_out, void* k_cache,
                          void* v_cache, const int32_t* page_table, hipStream_t stream) {
    M3_TRY(check_cache_dims(d, M3_ROTATE_HALVES));
    if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 8 != 0)
        return fail(M3_E_DIMS, "rotary_dim = %lld must be a multiple of 8 up to head_dim = %lld", (long long)d->rotary_dim,
                    (long long)d->head_dim);
    const bool packed = cu_seqlens != nullptr, cached = k_cache || v_cache || page_table;
    const int64_t tokens = packed ? d->seqlen : d->batch * d->seqlen;
    M3_TRY(check_groups(tokens, 1, 1));
    Cache c;
    M3_TRY(plan_cache(&c, d, k_cache, v_cache, page_table, lens));
    Area aq, ak, av, aqo, ako;
    const int64_t nq[3] = {packed ? 1 : d->batch, d->seqlen, d->heads}, nk[3] = {nq[0], nq[1], d->kv_heads};
    M3_TRY(make_area(&aq, q, "q", nq, {d->q.batch, d->q.token, d->q.head}, d->head_dim, c.es, 1));
    M3_TRY(make_area(&ak, k, "k", nk, {d->k.batch, d->k.token, d->k.head}, d->head_dim, c.es, 1));
    M3_TRY(make_area(&av, v, "v", nk, {d->v.batch, d->v.token, d->v.head}, d->head_dim, c.es, 1));
    M3_TRY(make_area(&aqo, q_out, "q_out", nq, {d->q_out.batch, d->q_out.token, d->q_out.head}, d->head_dim, c.es, 1));
    M3_TRY(make_area(&ako, k_out, "k_out", nk, {d->k_out.batch, d->k_out.token, d->k_out.head}, d->head_dim, c.es, 1));
    const Area freq = flat(inv_freq, d->rotary_dim / 2 * 4, "inv_freq");
    const Area cu = flat(cu_seqlens, packed ? (d->batch + 1) * 4 : 0, "cu_seqlens");
    for (const Area* a : {(const Area*)&ak, &freq}) M3_TRY(check_need(*a));
    if (q || q_out)
        for (const Area* a : {&aq, &aqo}) M3_TRY(check_need(*a));
    if (cached)
        for (const Area* a : {&av, &c.k, &c.v, &c.table}) M3_TRY(check_need(*a));
    for (const Area* a : {&freq, &cu}) M3_TRY(check_aligned(*a, 4));
    const Area none;
    const Area* outs[] = {&aqo, &ako, cached ? &c.k : &none, cached ? &c.v : &none};
    for (int i = 0; i < 4; ++i) {
        if (!outs[i]->p) continue;
        M3_TRY(check_apart(*outs[i]));
        M3_TRY(check_clash(*outs[i], aq, i == 0));
        M3_TRY(check_clash(*outs[i], ak, i == 1));
        for (const Area* in : {(const Area*)&av, &freq, &cu, (const Area*)&c.table, (const Area*)&c.lens}) M3_TRY(check_clash(*outs[i], *in));
        for (int j = i + 1; j < 4; ++j) M3_TRY(check_clash(*outs[i], *outs[j]));
    }
    M3_TRY(check_device());
    if (tokens == 0 || d->batch == 0) return M3_OK;
    m3::AppendArgs a{};
    a.q = rows_of(aq), a.k = rows_of(ak), a.v = rows_of(av), a.q_out = rows_of(aqo), a.k_out = rows_of(ako);
    a.pages = c.pages;
    // a cache of no pages has none to write to
    if (c.k.empty()) a.pages.k = nullptr;
    a.cu = cu_seqlens;
    a.lens = lens;
    a.inv_freq = inv_freq;
    a.b = d->batch, a.L = d->seqlen;
    a.heads = (int)d->heads, a.kv_heads = (int)d->kv_heads, a.dim = (int)d->head_dim, a.rot = (int)d->rotary_dim;
    a.halves = (d->flags & M3_ROTATE_HALVES) != 0;
    return launched(m3::launch_cache_append(a, d->io == M3_BF16, stream), "m3_cache_append");
}

size_t m3_attention_step_workspace_bytes(const m3_cache_dims* d) {
    StepPlan p;
    return plan_step(d, &p) == M3_OK ? p.bytes : 0;
}

m3_status m3_attention_step(const m3_cache_dims* d, const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* page_table, const int32_t* lens, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    StepPlan p;
    M3_TRY(plan_step(d, &p));
    if (d->seqlen != 1) return fail(M3_E_DIMS, "seqlen = %lld must be 1", (long long)d->seqlen);
    float scale;
    M3_TRY(check_scale(d->scale, d->head_dim, &scale));
    Cache c;
    M3_TRY(plan_cache(&c, d, k_cache, v_cache, page_table, lens));
    Area aq, ao;
    const int64_t n[3] = {d->batch, 1, d->heads};
    M3_TRY(make_area(&aq, q, "q", n, {d->q.batch, d->q.token, d->q.head}, d->head_dim, c.es, 1));
    M3_TRY(make_area(&ao, o, "o", n, {d->o.batch, d->o.token, d->o.head}, d->head_dim, c.es, 1));
    const Area al = flat(lse, d->batch * d->heads * 4, "lse"), ws = flat(workspace, (int64_t)p.bytes, "workspace");
    for (const Area* a : {&aq, &ao, &c.k, &c.v, &c.table, &c.lens}) M3_TRY(check_need(*a));
    M3_TRY(check_aligned(al, 4));
    M3_TRY(check_workspace("m3_attention_step", workspace, workspace_bytes, p.bytes));
    M3_TRY(check_apart(ao));
    const Area* outs[] = {&ao, &al, &ws};
    for (int i = 0; i < 3; ++i) {
        M3_TRY(check_clash(*outs[i], aq, i == 0));
        for (const Area* in : {&c.k, &c.v, &c.table, &c.lens}) M3_TRY(check_clash(*outs[i], *in));
        for (int j = i + 1; j < 3; ++j) M3_TRY(check_clash(*outs[i], *outs[j]));
    }
    M3_TRY(check_device());
    if (d->batch == 0) return M3_OK;
    m3::StepArgs a{};
    a.q = rows_of(aq), a.o = rows_of(ao);
    a.pages = c.pages;
    a.lens = lens;
    a.lse = lse;
    a.part = (float*)workspace;
    a.b = d->batch;
    a.heads = (int)d->heads, a.kv_heads = (int)d->kv_heads, a.dim = (int)d->head_dim;
    a.scale = scale;
    a.items = p.items;
    a.head_blocks = (int)p.head_blocks;
    a.joined = p.joined ? 1 : 0;
    return launched(m3::launch_attention_step(a, d->io == M3_BF16, stream), "m3_attention_step");
}

}  // extern "C"
