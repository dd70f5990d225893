// kda_attn.cuh -- what the attention kernels share: which cache tokens a call visits and in which parts,
// and the form in which parts of one row are handed to the kernel that joins them.
#pragma once

#include "kda_kv.cuh"

namespace kda {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The tokens that any of positions [first, last] of a request may see, [0, sink_end) and [lo, hi), as a
// list of tiles of kTile tokens aligned in the sequence: `sink_tiles` tiles from 0, then tiles from
// `tile0` on.  A tile of the list holds at least one visible token.
struct Span {
    int32_t lo, hi, sink_end;
    int32_t sink_tiles, tile0, tiles;
};

template <int kTile>
__host__ __device__ __forceinline__ Span make_span(int64_t first, int64_t last, int64_t room, int32_t window, int32_t sinks)
{
    Span s;
    const int64_t hi = last + 1 < room ? last + 1 : room;
    int64_t lo = window ? first - window + 1 : 0;
    if (lo < 0) lo = 0;
    if (lo > hi) lo = hi;
    s.hi = hi > 0 ? (int32_t)hi : 0;
    s.lo = hi > 0 ? (int32_t)lo : 0;
    s.sink_end = sinks < s.lo ? sinks : s.lo;
    s.sink_tiles = (s.sink_end + kTile - 1) / kTile;
    s.tile0 = s.lo / kTile;
    if (s.tile0 < s.sink_tiles) s.tile0 = s.sink_tiles;
    const int32_t end = (s.hi + kTile - 1) / kTile;
    s.tiles = s.sink_tiles + (end > s.tile0 ? end - s.tile0 : 0);
    return s;
}

template <int kTile>
__device__ __forceinline__ int32_t tile_base(const Span& s, int32_t i)
{
    return (i < s.sink_tiles ? i : s.tile0 + i - s.sink_tiles) * kTile;
}

// Parts of a row that several CTAs worked on: [row][part][D] fp32 outputs, each normalised by its own
// sum, and their log2 of the sum of exponentials [row][part], -inf for an empty part.
struct Parts {
    float* o;
    float* lse2;
    int32_t max_parts;
    int32_t tiles_per_part;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace attn
}  // namespace kda
