// m3_page_map.h -- index maps of the attention operators, shared by the kernels and host-side tests (no HIP types).
#pragma once

#include <stdint.h>

#include "m3_mapping.h"

namespace m3 {

// Position `pos` of a sequence whose row of the page table is `row`: its page, and its place there; -1 where the
// position is negative, past the table, or on a number that is no page.  shift: log2 of the page's
// size, or -1.
M3_HD int32_t page_place(const int32_t* row, int64_t width, int32_t pages, int32_t size, int shift, int32_t pos,
                         int32_t* place) {
    *place = 0;
    if (pos < 0) return -1;
    const int32_t n = shift >= 0 ? pos >> shift : pos / size;
    *place = pos - n * size;
    if (n >= width) return -1;
    const int32_t id = row[n];
    return id >= 0 && id < pages ? id : -1;
}

// Blocks of R rows of a packed batch: sequence s, which starts at token `start`, has the numbers from start / R + s on.
// The next sequence's first number leaves it at least as many as it has blocks, and all are below T / R + b.
M3_HD int64_t first_block(int64_t start, int64_t s, int64_t R) { return start / R + s; }

// Workgroups that are given out from the heaviest on meet two to a compute unit, 256 numbers apart: the second 256 (in
// steps of 8, so that each stays on its XCD) are taken from the other end, heavy ones with light ones.  A permutation of
// [0, n).
constexpr int64_t kUnits = 256;
M3_HD int64_t paired_item(int64_t i, int64_t n) {
    const int64_t end = (n < 2 * kUnits ? n : 2 * kUnits) / kXcds * kXcds;
    if (i < kUnits || i >= end) return i;
    const int64_t r = i / kXcds, first = kUnits / kXcds, last = end / kXcds - 1;
    return (first + last - r) * kXcds + i % kXcds;
}

// A decoding batch as one row of keys, sequence after sequence, each rounded up to whole rounds of a workgroup (an empty
// one to one round): piece i is keys i * n .. (i + 1) * n - 1 of it, whatever sequences they belong to.  Going along the
// row, the piece or the sequence or both go up at each border, so that i + s numbers the parts of sequences in
// pieces, below pieces + b.
constexpr int64_t kRound = 128;
M3_HD int64_t rounded_keys(int64_t len) { return len <= kRound ? kRound : (len + kRound - 1) / kRound * kRound; }
// The length of pieces that makes at most `items` of them out of `all` keys.
M3_HD int64_t piece_keys(int64_t all, int64_t items) {
    const int64_t even = (all + items - 1) / items;
    return rounded_keys(even);
}

}  // namespace m3
