// m3_pages.h -- device-side lookups shared by the kernels of the paged cache (append, one token's attention).
#pragma once

#include "attn_launch.h"
#include "m3_device.h"
#include "m3_page_map.h"

namespace m3 {

__device__ __forceinline__ int page_of(const Pages& p, const int32_t* row, int32_t pos, int& place) {
    return page_place(row, p.table_w, p.n, p.size, p.shift, pos, &place);
}

// The last i < n with first(i) <= t (0 where there is none); first must not decrease.  64 candidates at a time.
template <typename F>
__device__ __forceinline__ int64_t last_at_most(int64_t n, int64_t t, F&& first) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0;
    while (n > 1) {
        const int64_t step = (n + 63) / 64, i = lane * step;
        const bool le = i < n && first(lo + i) <= t;
        const int c = __popcll(__ballot(le));
        const int64_t skip = c > 0 ? (c - 1) * step : 0;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    return lo;
}

// An offset of a packed batch, kept within its tokens whatever it holds.
__device__ __forceinline__ int64_t packed_offset(const int32_t* cu, int64_t s, int64_t tokens) {
    const int64_t c = cu[s];
    return c < 0 ? 0 : c > tokens ? tokens : c;
}

}  // namespace m3
