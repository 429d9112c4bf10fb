// cache_append.hip -- new keys and values into a paged cache, rotated on the way (m3_cache_append).
//
// Memory-bound: every row is read once and written once.  A workgroup takes a token; a thread keeps one place of
// a row (16 bytes, or the two places that a rotation of halves pairs), computes that place's angles once, in fp64
// (a far position times its frequency has more digits than fp32 holds), and goes through the heads with
// them.  8 x 2048 tokens, 32/8 heads of 128 bf16: 77 us, 5.2 TB/s, as a copy; 64 single tokens: 4.5 us, latency.
#include "m3_mma.h"
#include "m3_pages.h"

namespace m3 {
namespace {

// U elements of io type T as one load
template <typename T, int U> struct Unit;
template <> struct Unit<bf16, 8> { typedef uint4 type; };
template <> struct Unit<bf16, 4> { typedef uint2 type; };
template <> struct Unit<float, 4> { typedef uint4 type; };

template <typename T, int U>
__device__ __forceinline__ void unpack(typename Unit<T, U>::type u, float (&x)[U]) {
    if constexpr (U == 4 && sizeof(T) == 2) {
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        unpack16(u, x, T{});
    }
}
template <typename T, int U>
__device__ __forceinline__ typename Unit<T, U>::type pack(const float (&x)[U]) {
    if constexpr (U == 4 && sizeof(T) == 2) return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else return pack16(x, T{});
}

// HALVES: element k is paired with k + rot / 2, else 2 k with 2 k + 1.
template <typename T, int U, bool HALVES>
__global__ __launch_bounds__(256) void cache_append(const AppendArgs a) {
    typedef typename Unit<T, U>::type unit;
    constexpr int PAIRS = HALVES ? U : U / 2;
    const int64_t t = blockIdx.x;
    int64_t s, at, n;   // sequence, place among its new tokens, their number
    if (a.cu) {
        s = last_at_most(a.b, t, [&](int64_t i) { return packed_offset(a.cu, i, a.L); });
        const int64_t first = packed_offset(a.cu, s, a.L);
        n = packed_offset(a.cu, s + 1, a.L) - first;
        at = t - first;
        if (at < 0 || at >= n) return;
    } else {
        s = t / a.L;
        at = t - s * a.L;
        n = a.L;
    }
    const int64_t pos = (a.lens ? (int64_t)a.lens[s] : n) - n + at;   // below 2^31, but not always above -2^31
    int place = 0, page = -1;
    if (a.pages.k && pos >= 0) page = page_of(a.pages, a.pages.table + s * a.pages.table_w, (int32_t)pos, place);

    // places of a row: pairs of units (halves) or units that are rotated, then units that are copied
    const int turned = a.rot / (HALVES ? 2 * U : U), places = turned + (a.dim - a.rot) / U;
    const int rows = 256 / places;   // rows that go by at a time
    const int mine = threadIdx.x % places, row0 = threadIdx.x / places;
    if (row0 >= rows) return;
    const bool turn = mine < turned;
    const int d = turn ? mine * U : a.rot + (mine - turned) * U;
    float cs[PAIRS], sn[PAIRS];
    if (turn) {
        const int k = HALVES ? d : d / 2;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const double turns = (double)pos * (double)a.inv_freq[k + i] * 0.15915494309189533577;
            sincospif(2.f * (float)(turns - rint(turns)), &sn[i], &cs[i]);
        }
    }
    // one row: src (rotated or not) to any of two places
    auto move = [&](const char* src, char* to, char* to2, bool rotated) {
        constexpr int es = sizeof(T);
        unit u = *(const unit*)(src + d * es);
        if constexpr (HALVES) {
            if (turn) {
                const int far = a.rot / 2 * es;
                unit v = *(const unit*)(src + d * es + far);
                if (rotated) {
                    float x[U], y[U];
                    unpack<T, U>(u, x);
                    unpack<T, U>(v, y);
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const float p = x[i] * cs[i] - y[i] * sn[i];
                        y[i] = x[i] * sn[i] + y[i] * cs[i];
                        x[i] = p;
                    }
                    u = pack<T, U>(x);
                    v = pack<T, U>(y);
                }
                if (to) *(unit*)(to + d * es + far) = v;
                if (to2) *(unit*)(to2 + d * es + far) = v;
            }
        } else if (turn && rotated) {
            float x[U];
            unpack<T, U>(u, x);
#pragma unroll
            for (int i = 0; i < U / 2; ++i) {
                const float p = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                x[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                x[2 * i] = p;
            }
            u = pack<T, U>(x);
        }
        if (to) *(unit*)(to + d * es) = u;
        if (to2) *(unit*)(to2 + d * es) = u;
    };
    auto row = [&](const HeadRows& r, int head) {
        return r.p + (a.cu ? t * r.token : s * r.batch + at * r.token) + head * r.head;
    };
    const int nq = a.q.p ? a.heads : 0, nk = a.k.p ? a.kv_heads : 0, nv = a.v.p ? a.kv_heads : 0;
    for (int r = row0; r < nq + nk + nv; r += rows) {
        if (r < nq) {
            move(row(a.q, r), row(a.q_out, r), nullptr, true);
        } else if (r < nq + nk) {
            const int h = r - nq;
            char* to = page >= 0 ? a.pages.k + page * a.pages.k_page + h * a.pages.k_head +
                                       place * (int64_t)a.pages.k_token : nullptr;
            char* to2 = a.k_out.p ? row(a.k_out, h) : nullptr;
            if (to || to2) move(row(a.k, h), to, to2, true);
        } else if (page >= 0) {
            const int h = r - nq - nk;
            move(row(a.v, h), a.pages.v + page * a.pages.v_page + h * a.pages.v_head + place * (int64_t)a.pages.v_token,
                 nullptr, false);
        }
    }
}

template <typename T, int U>
hipError_t launch_unit(const AppendArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)(a.cu ? a.L : a.b * a.L));
    if (a.halves) cache_append<T, U, true><<<grid, 256, 0, s>>>(a);
    else cache_append<T, U, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, bool bf16_io, hipStream_t s) {
    if (!bf16_io) return launch_unit<float, 4>(a, s);
    // half of the rotated elements have to be whole units
    return a.halves && a.rot % 16 != 0 ? launch_unit<bf16, 4>(a, s) : launch_unit<bf16, 8>(a, s);
}

}  // namespace m3
