// attn_launch.h -- argument blocks and launchers of the operators of m3attn.h, shared between their C-ABI file
// (attn_api.hip) and the kernels.  Shapes, pointers and workspaces are validated by the C-ABI file before any
// launcher runs.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

// ------------------------------------------------------------------------- whole prompts
constexpr int kAttnRows = 128;        // query rows (backward: keys) of a workgroup, 32 to a wave
constexpr int kAttnWide = 256;        // keys of a workgroup of 8 waves
constexpr int kAttnFew = 32;          // the same where the other axis is split over the waves
constexpr int64_t kAttnMaxDim = 128;  // elements of a head

// rows of heads: bytes between consecutive sequences (dense batches), tokens and heads
struct HeadRows {
    char* p;
    int64_t batch, head;
    uint32_t token;
};

struct AttnArgs {
    HeadRows q, k, v, o;
    HeadRows dout, dq, dk, dv;   // backward
    float* lse;                  // [b, Hq, L], packed [Hq, T] (forward: out, nullable)
    float* delta;                // like lse (backward's workspace)
    const int32_t* cu;           // packed offsets, or nullptr: dense
    int64_t b, L;                // sequences; tokens of each (dense) or of all (packed)
    int heads, kv_heads, dim;
    float scale;
    uint32_t blocks, kblocks;    // blocks of query rows and of keys (packed: as many as there can be)
    int few, kfew, kwide;        // they are kAttnFew rows (kwide: kAttnWide), not kAttnRows
    int paired;                  // two workgroups to a compute unit: paired_item's order
    int splits;                  // backward: parts that the heads of a group are split into for dk and dv
    float* part;                 // splits > 1: dk, then dv, of each part, [2, splits, tokens, kv_heads, D]
};
hipError_t launch_attention(const AttnArgs& a, bool bf16_io, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs& a, bool bf16_io, hipStream_t s);

// ------------------------------------------------------------------------- paged cache
struct Pages {
    char* k;
    char* v;
    int64_t k_page, k_head, v_page, v_head;   // bytes
    uint32_t k_token, v_token;
    const int32_t* table;                     // [b, table_w]
    int64_t table_w;
    int32_t n, size;                          // pages, tokens of a page
    int shift;                                // log2 of size, -1: not a power of two
};

struct AppendArgs {
    HeadRows q, k, v, q_out, k_out;   // p null: not there
    Pages pages;
    const int32_t* cu;           // packed offsets, or nullptr: dense
    const int32_t* lens;         // [b] tokens in the cache, the new ones counted in
    const float* inv_freq;       // [rot / 2], nullptr: no rotation
    int64_t b, L;                // sequences; new tokens of each (dense) or of all (packed)
    int heads, kv_heads, dim, rot;
    int halves;
};
hipError_t launch_cache_append(const AppendArgs& a, bool bf16_io, hipStream_t s);

struct StepArgs {
    HeadRows q, o;               // batch and head strides; token unused
    Pages pages;
    const int32_t* lens;
    float* lse;                  // [b, Hq], nullable
    float* part;                 // partial results (workspace)
    int64_t b;
    int heads, kv_heads, dim;
    float scale;
    int64_t items;               // pieces of work per key head and block of query heads
    int head_blocks;             // blocks of 16 query heads of a key head
    int joined;                  // no sequence is cut: no second launch
};
hipError_t launch_attention_step(const StepArgs& a, bool bf16_io, hipStream_t s);

}  // namespace m3
