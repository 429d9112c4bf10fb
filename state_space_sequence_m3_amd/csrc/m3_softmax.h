// m3_softmax.h -- the running maximum of a softmax whose scores may be any finite number, shared by the attention kernels.
//
// With c = scale log2 e, a score s counts as exp2(fma(s, by, -fl(top by))), top the row's largest score so far.  As a rule
// by is c.  fl(top c) is off by up to half a unit in its last place, the same for all scores of a row; but where top c is
// 2^31 or more that alone can be over 128, past what exp2 takes.  From kFar on, by is therefore a power of two, whose
// products are exact, such that neighbouring numbers at top are 2^16 apart: the largest score counts as 1 and any smaller one
// as 0, which it is within what fp32 scores of that size are off.
#pragma once

#include "m3_device.h"

namespace m3 {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;   // a running maximum's start: every finite score is at least that
// half a unit in the last place there is 8 to 16: far below what exp2 takes, and more than a running maximum lags behind
constexpr float kFar = 268435456.f;

// what scores of a row with maximum `top` are multiplied with
__device__ __forceinline__ float score_factor(float top, float c) {
    if (fabsf(top * c) < kFar) return c;
    const int e = 40 - __builtin_amdgcn_frexp_expf(top);
    return __builtin_amdgcn_ldexpf(1.f, e < 127 ? e : 127);
}
// By what sums relative to a maximum `from` are multiplied for the maximum `to`, at least as large.  (-infinity as `from`,
// of nothing at all, gives 0.)
__device__ __forceinline__ float top_moved(float from, float to, float c) {
#pragma clang fp contract(off)
    const float b = to * c;
    return fast_exp2(fmaxf(fabsf(b) < kFar ? from * c - b : (from - to) * c, -INFINITY));
}
// log sum exp of a row's scores, from its maximum and the sum relative to it
__device__ __forceinline__ float log_sum(float top, float sum, float c) {
#pragma clang fp contract(off)
    const float a = top * c, l = __builtin_amdgcn_logf(sum);
    return fabsf(a) < kFar ? (a + l) * kLn2 : top * (c * kLn2) + l * kLn2;
}

}  // namespace m3
