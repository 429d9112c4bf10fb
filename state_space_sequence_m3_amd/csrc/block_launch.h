// block_launch.h -- argument blocks and launchers of the operators of m3block.h, shared between
// their C-ABI file (block_api.hip) and the kernels.  Shapes, pointers and workspaces are validated
// by the C-ABI file before any launcher runs.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m3 {

// ---------------------------------------------------------------------------- gated scan
// A tile is kScanTile tokens (backward: kScanBwdTile) x kScanCols channels, worked on by one workgroup;
// `states` has a row per block of kScanBlock tokens in either pass.  Dense batches of sequences longer than a
// block are cut sequence by sequence (`per_seq`), and so are few shorter ones; many shorter ones and packed
// batches are cut along the flat token axis, so a tile can hold many sequences.
constexpr int kScanTile = 128, kScanBwdTile = 64, kScanBlock = 64;
constexpr int kScanCols = 128;

struct GatedScanArgs {
    const int32_t* cu;      // packed offsets, or nullptr: dense
    const void* gate;
    const void* x;
    const float* bias;
    const float* h_in;
    void* y;
    float* h_out;
    float* states;          // [blocks, D] state each block starts from (forward: out, nullable)
    // backward
    const void* dy;
    const float* dh_out;
    void* dgate;
    void* dx;
    float* dbias;
    float* dh_in;
    float* part;            // [parts, D] each workgroup's share of dbias (parts > 1)
    int64_t parts;
    int64_t b, L, T;        // sequences; tokens of each (dense); tokens of all
    int64_t D;
    int64_t gate_p, x_p, y_p, dgate_p, dx_p;   // pitches in bytes
    uint64_t* words;        // [ntiles, ncols * kScanCols] chain words (not serial)
    unsigned* ticket;
    // flat, chained: which tokens start and end a sequence (a bit each), and the sequence of each token
    uint64_t* starts;
    uint64_t* ends;
    int* seqs;
    int64_t ntiles;
    uint32_t seq_tiles;     // tiles, and blocks, per sequence (per_seq)
    uint32_t seq_blocks;
    int ncols;              // column blocks
    int per_seq;
    int serial;             // a workgroup takes a sequence (flat: the batch) tile by tile; else tiles are chained
};

hipError_t launch_gated_scan(const GatedScanArgs& a, bool bf16_io, bool vec, hipStream_t s);
hipError_t launch_gated_scan_backward(const GatedScanArgs& a, bool bf16_io, bool vec, hipStream_t s);

struct GatedStepArgs {
    const void* gate;
    const void* x;
    const float* bias;
    const float* h;
    void* y;
    float* h_out;
    int64_t b, D;
    int64_t gate_p, x_p, y_p;   // pitches in bytes
};
hipError_t launch_gated_step(const GatedStepArgs& a, bool bf16_io, bool vec, hipStream_t s);

// ------------------------------------------------------------------------------ RMS norm
constexpr int64_t kNormMaxWidth = 16384;

struct RmsNormArgs {
    const void* x;
    const void* residual;
    const float* weight;
    void* r_out;
    void* y;
    uint8_t* q;
    float* scale;
    // backward
    const void* r;
    const void* dy;
    const void* dr_out;
    void* dx;
    float* dweight;
    float* part;               // [blocks, D]
    int64_t rows;
    int D;
    int64_t x_p, res_p, r_p, y_p, dx_p;   // pitches in bytes
    int group;                 // 0: the row
    int ngroups;
    float eps;
    int cus;                   // compute units
    int stream;                // outputs go past the caches
};
hipError_t launch_rmsnorm(const RmsNormArgs& a, bool bf16_io, hipStream_t s);
hipError_t launch_rmsnorm_backward(const RmsNormArgs& a, bool bf16_io, hipStream_t s);
// rows of dweight partial sums
int64_t rmsnorm_backward_parts(int64_t rows, int64_t D, bool bf16_io, int cus);

// ----------------------------------------------------------------- column sums, gradient norm
// out[d] = sum over i < n of part[i * D + d], in a fixed order
hipError_t launch_column_sum(const float* part, int64_t n, int64_t D, float* out, hipStream_t s);

constexpr int kGradBatch = 96;           // tensors per launch (their table is a kernel argument)
// Elements per unit of work, and workgroups (and partial sums) per launch at most.  Where nothing is clipped: 60 x
// 3333333 fp32 148 us, with 1024 or 4096 workgroups 157 and 155; 40 x 500000 31 us, 39 with units of 8192; 20 x
// 50000 7.3 us, 9.4 with units of 32768.
constexpr int64_t kGradChunk = 16384;
constexpr int kGradBlocks = 2048;
// As many elements in one table are left to a single workgroup, a unit of kGradSmallChunk to a wave: one launch
// and no partial sums, so that the call costs the host a third less (8 x 5125 elements 22 -> 17 us); on the GPU
// alone it takes 4.6 us instead of 5.9 for 8 x 1000 elements, 9.3 instead of 8.4 for 8 x 5125 (which a replayed graph
// pays without the host's gain).
constexpr int64_t kGradSmall = 65536;
constexpr int64_t kGradSmallChunk = 2048;   // 1024: 10.6 us for 8 x 5125 elements, 4096: 9.7

struct GradBatch {
    const void* src[kGradBatch];
    void* dst[kGradBatch];
    int64_t numel[kGradBatch];
    uint32_t first[kGradBatch + 1];      // first unit of work of each tensor, and their number
    int chunk;                           // elements per unit
    uint32_t is_bf16[(kGradBatch + 31) / 32];
    int n;
    int stream;                          // outputs go past the caches
};
inline int grad_blocks(const GradBatch& b) {
    const uint32_t units = b.first[b.n];
    return units < (uint32_t)kGradBlocks ? (int)units : kGradBlocks;
}
// part[0 .. grad_blocks): sums of squares
hipError_t launch_grad_sumsq(const GradBatch& b, double* part, hipStream_t s);
// stats = {norm, coef} of n partial sums; with sum, also their sum there
hipError_t launch_grad_stats(const double* part, int64_t n, float max_norm, float* stats, double* sum, hipStream_t s);
// dst = coef src, coef from n partial sums; with stats, also {norm, coef} there
hipError_t launch_grad_scale(const GradBatch& b, const double* part, int n, float max_norm, float* stats,
                             hipStream_t s);
// all of it, by one workgroup
hipError_t launch_grad_small(const GradBatch& b, bool write, float max_norm, float* stats, hipStream_t s);

}  // namespace m3
