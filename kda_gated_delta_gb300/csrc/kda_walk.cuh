// kda_walk.cuh -- who owns which packed rows.  On the host as well as on the device: a test takes the walk over every
// small table of lengths, sound or not.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

// Rows [first, last) of request b, clamped to the packed tensor; a bad pair is reported by the return.
__host__ __device__ __forceinline__ bool layer_rows(const int32_t* cu, int32_t b, int64_t T, int64_t& first, int64_t& last)
{
    if (cu == nullptr) {
        first = b;
        last = b + 1;
        return true;
    }
    first = cu[b];
    last = cu[b + 1];
    if (first < 0 || last < first || last > T) {
        first = last = 0;
        return false;
    }
    return true;
}

// The request that owns row t: the last b with cu[b] <= t, or -1 (row before the first entry).  May be n
// (row from the last entry on).
__host__ __device__ __forceinline__ int32_t layer_owner(const int32_t* cu, int32_t n, int64_t t)
{
    int32_t lo = 0, hi = n + 1;                 // first entry > t lies in [lo, hi]
    while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

// Rows of no request in a table that does not decrease: [0, lo) and [hi, T), lo <= hi.  They lie before the first entry that is
// not negative and behind the last that is not above T: a request that reaches past either is taken by nobody.
__host__ __device__ __forceinline__ void unowned_rows(const int32_t* cu, int32_t n, int64_t T, int64_t& lo, int64_t& hi)
{
    const int32_t from = layer_owner(cu, n, -1) + 1, to = layer_owner(cu, n, T);
    lo = from <= n && cu[from] < T ? cu[from] : T;
    hi = to >= 0 && cu[to] > lo ? cu[to] : lo;
}

// Where the convolution's tile that would end before row e ends: a request's first W - 1 tokens, whose outputs depend on
// its old state, stay with the CTA that has its first token and replaces that state.
template <int W>
__host__ __device__ __forceinline__ int64_t conv_tile_edge(const int32_t* cu, int32_t n, int64_t T, int64_t e)
{
    if (e >= T) return T;
    int64_t first, last;
    const int32_t b = layer_owner(cu, n, e);
    if (b < 0 || b >= n || !layer_rows(cu, b, T, first, last)) return e;
    if (first >= e || e - first >= W - 1) return e;
    return first + (W - 1) < last ? first + (W - 1) : last;
}

// The stretch of the convolution's rows that begins at row t of a tile: rows up to `last`, of request b (`own`) or of none.
// `b` is the owner of an earlier row of the tile and moves on.  A window that is not the request's state is read from the
// rows before t, so these have to be the request's own.  In a sound table they are, by the tiles' edges; where a table
// decreases, a stretch can begin behind its request's first row, and is taken for no request's.
struct Stretch {
    int64_t first, last;
    bool own;
};
template <int W>
__host__ __device__ __forceinline__ Stretch conv_stretch(const int32_t* cu, int32_t n, int64_t T, int64_t t, int32_t& b)
{
    while (b < n && cu[b + 1] <= t) ++b;
    Stretch s = {t, t, false};
    if (b >= 0 && b < n && layer_rows(cu, b, T, s.first, s.last)) s.own = s.first == t || t - s.first >= W - 1;
    else s.last = b < 0 ? cu[0] : b < n ? t + 1 : T;
    if (s.last <= t) s.last = t + 1;
    return s;
}

}  // namespace kda
