// kda_attn.cu -- attention of new tokens over the paged cache (kda_paged_attention): the form for few
// query rows (decode and short verifies), the joining of parts, and the dispatch.
//
// Few rows.  A kv head serves R = new tokens * G query rows.  For R <= 16 the cache's bytes are all that
// counts (at 128 channels in bf16 a token's 512 bytes meet 4 * 128 * R flops), so the keys and values go
// from global memory straight into the registers in which mma.sync m16n8k16 wants them, read once, and
// nothing is staged in shared memory:
//
//   S^T = K Q^T     A = 16 tokens x 16 channels, B = Q^T with the query rows as the 8 columns
//   O^T = V^T P^T   A = 16 channels x 16 tokens
//
// With the queries as the N = 8 side a tile computes 8 rows, not 16 of which most are padding, and the
// accumulator of 128 channels takes 32 registers.  The order of the channels of a contraction and of the
// rows of an output tile is free, so each lane's fragment is made of whole 16-byte loads (4-bit caches: 16
// and 8) from the rows as they lie in the cache:
//   K: lane (r, c) = (lane / 4, lane % 4) holds tokens r and r + 8, the c-th 16 bytes of each 64;
//   V: it holds tokens 2c, 2c + 1, 2c + 8, 2c + 9, the r-th 16 bytes of each 128; two byte permutes make
//      a register of one channel's two tokens.
// 4-bit values go to bf16 instead, with the weights, which need its range: a weight far below the largest
// still counts in a channel where the heavy tokens hold zeros.
// P^T is made from S^T by movmatrix (a transposition of 8 x 8 across the warp).
//
// The softmax runs along the lanes' own tokens; a new maximum is taken over the warp only when some score
// exceeds the current one by 8 in log2 (one vote), so that the common tile has no shuffles and no
// rescaling.  The weights, at most 2^8 then, lose nothing by that in a floating-point format.
//
// The weights are rounded to bf16 for their product with the values, half a step or 2^-8 of a weight at most; their
// sum takes them unrounded.  mma.sync has no wider operand beside bf16 values, and two products (a weight as the sum
// of two bf16 numbers) would double the tensor work; the output, rounded to bf16 once more, is off by 2.1e-3 to
// 2.3e-3 of its size in the mean, where its own rounding alone gives 1.7e-3.
//
// Measured (8 kv and 32 query heads of 128): 64 requests of 512 to 8,192 tokens in 193 us, 6,350 GB/s of the 6,776
// that a copy reaches; 16 requests of 4,096 to 131,072 tokens in 4 bits in 373 us, bound by the conversions (some
// 500 instructions per 16 tokens).
//
// A warp takes every fourth tile of its CTA's part, with the next tile's keys requested as soon as the
// present ones are used and likewise the values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kda_attn.cuh"
#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

__device__ int32_t g_attn_error = 0;

using attn::Parts;
using attn::Span;

constexpr int kWarps = 4;
constexpr float kSlack = 8.0f;      // growth of a maximum, in log2, that is let pass

__device__ __forceinline__ uint4 ld16(const void* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld8(const void* p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld4(const void* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld2(const void* p)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld1(const void* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// D += A B, 16 x 8 x 16, fp32 accumulators; bf16 or fp16 operands.
template <bool FP16>
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (FP16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// One warp's keys or values of TB x 16 tokens, as loaded.  `lane_at` and `lane_scale` point at the lane's
// part of cache row 0; row: cache row of token 0 of the 16.
template <int D, bool FP4>
__device__ __forceinline__ const uint8_t* row_at(const uint8_t* lane_at, int32_t row) { return lane_at + (int64_t)row * (FP4 ? D / 2 : 2 * D); }
template <int D>
__device__ __forceinline__ const uint8_t* scale_at(const uint8_t* lane_scale, int32_t row) { return lane_scale + (int64_t)row * (D / 16); }

template <int D, bool FP4, int TB>
struct KeyTile {
    static constexpr int kWords = FP4 ? D / 32 : D / 8;     // of one token, per lane
    uint32_t w[TB][2][kWords];
    uint32_t s[TB][2];                                        // 4 bits: the lane's scales

    // the lane reads tokens r and r + 8, the c-th quarter (bf16: the c-th 16 bytes of each 64)
    static __device__ __forceinline__ int lane_offset(int r, int c) { return FP4 ? r * (D / 2) + c * (D / 8) : r * 2 * D + c * 16; }
    static __device__ __forceinline__ int scale_offset(int r, int c) { return r * (D / 16) + c * (D / 64); }
    __device__ __forceinline__ void load(int tb, const uint8_t* lane_at, const uint8_t* lane_scale, int32_t row)
    {
        const uint8_t* p = row_at<D, FP4>(lane_at, row);
        const uint8_t* q = scale_at<D>(lane_scale, row);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if constexpr (!FP4) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 x = ld16(p + e * 16 * D + 64 * i);
                    w[tb][e][4 * i] = x.x, w[tb][e][4 * i + 1] = x.y, w[tb][e][4 * i + 2] = x.z, w[tb][e][4 * i + 3] = x.w;
                }
            } else if constexpr (D == 128) {
                const uint4 x = ld16(p + e * 4 * D);
                w[tb][e][0] = x.x, w[tb][e][1] = x.y, w[tb][e][2] = x.z, w[tb][e][3] = x.w;
                s[tb][e] = ld2(q + e * (D / 2));
            } else {
                const uint2 x = ld8(p + e * 4 * D);
                w[tb][e][0] = x.x, w[tb][e][1] = x.y;
                s[tb][e] = ld1(q + e * (D / 2));
            }
        }
    }
};

template <int D, bool FP4, int TB>
struct ValueTile {
    static constexpr int kWords = FP4 ? D / 64 : D / 16;
    uint32_t w[TB][4][kWords];
    uint32_t s[TB][4];

    // the lane reads tokens 2c, 2c + 1, 2c + 8, 2c + 9, the r-th eighth (bf16: the r-th 16 bytes of each 128)
    static __device__ __forceinline__ int lane_offset(int r, int c) { return FP4 ? 2 * c * (D / 2) + r * (D / 16) : 2 * c * 2 * D + r * 16; }
    static __device__ __forceinline__ int scale_offset(int r, int c) { return 2 * c * (D / 16) + (D == 128 ? r : r / 2); }
    static __device__ __forceinline__ constexpr int token(int e) { return (e & 1) + 8 * (e >> 1); }
    __device__ __forceinline__ void load_token(int tb, int e, const uint8_t* p, const uint8_t* q)
    {
        if constexpr (!FP4) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 x = ld16(p + token(e) * 2 * D + 128 * i);
                w[tb][e][4 * i] = x.x, w[tb][e][4 * i + 1] = x.y, w[tb][e][4 * i + 2] = x.z, w[tb][e][4 * i + 3] = x.w;
            }
        } else if constexpr (D == 128) {
            const uint2 x = ld8(p + token(e) * (D / 2));
            w[tb][e][0] = x.x, w[tb][e][1] = x.y;
            s[tb][e] = ld1(q + token(e) * (D / 16));
        } else {
            w[tb][e][0] = ld4(p + token(e) * (D / 2));
            s[tb][e] = ld1(q + token(e) * (D / 16));
        }
    }
    // tokens that nobody may see (not in [lo, hi) or [0, sink_end), or of a bad page) become zeros
    __device__ __forceinline__ void load(int tb, const uint8_t* lane_at, const uint8_t* lane_scale, int32_t row, int base, const Span& sp, int c)
    {
        const uint8_t* p = row_at<D, FP4>(lane_at, row);
        const uint8_t* q = scale_at<D>(lane_scale, row);
        if (row >= 0 && base + 16 <= sp.hi && (base >= sp.lo || base + 16 <= sp.sink_end)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) load_token(tb, e, p, q);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = base + 2 * c + token(e);
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[tb][e][i] = 0;
                s[tb][e] = 0;
                if (row >= 0 && j < sp.hi && (j >= sp.lo || j < sp.sink_end)) load_token(tb, e, p, q);
            }
        }
    }
};

// First row of the page of a token's 16-token block, -1 where the table holds none (recorded)
// (cache rows are below 2^31).
__device__ __forceinline__ int32_t block_row(const AttnCall& a, int b, int base, int h)
{
    const int64_t slot = kv::token_slot(a.c, b, base);
    return slot < 0 ? -1 : (int32_t)(slot + ((int64_t)h << a.c.page_shift));
}

// CLUSTER: the parts' CTAs are one cluster and join among themselves (a variant of its own, for the registers).
template <int D, bool FP4, int NT, int TB, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32) few_rows_kernel(AttnCall a, Parts parts)
{
    a.c.err = &g_attn_error;
    constexpr int kTile = 16 * TB;
    constexpr int KS = D / 16;                                  // contraction steps over the channels
    constexpr int MT = D / 16;                                  // 16-channel output tiles
    const int h = blockIdx.x % a.c.Hkv, b = blockIdx.x / a.c.Hkv, part = blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
    const int G = a.c.G;

    if (!CLUSTER && parts.o) attn::let_next_launch();
    if (a.c.cu && b == a.c.n) {                                 // the CTA past the last request
        if (part == 0) attn::clear_unowned<D>(a);
        return;
    }
    int64_t t0, t1;
    kv::request_rows(a.c, b, t0, t1);
    const int len = a.c.lens[b];
    const int fresh = (int)(t1 - t0);
    const int rows = min(fresh * G, 8 * NT);                     // rows past the caller's bound are left out
    if (rows == 0) return;
    const int64_t room = a.max_len;
    if (threadIdx.x == 0 && part == 0 && h == 0 && (len > room || fresh > a.max_new)) kv::record(a.c, kv::kErrLength);
    const int first = len > 0 ? len - fresh : -1 - fresh;          // position of the first new token; a padding request has none
    const Span sp = attn::make_span<kTile>(max(first, 0), len > 0 ? len - 1 : -1, room, a.window, a.sinks);
    const int parts_here = parts.max_parts > 1 ? min(parts.max_parts, max(1, (sp.tiles + parts.tiles_per_part - 1) / parts.tiles_per_part)) : 1;
    if (part >= parts_here && !CLUSTER) return;              // a cluster's CTA stays, with nothing to see
    const int tile_lo = parts_here > 1 ? part * parts.tiles_per_part : 0;
    const int tile_hi = part >= parts_here ? tile_lo : parts_here > 1 ? min(sp.tiles, tile_lo + parts.tiles_per_part) : sp.tiles;

    // ---- queries: B fragments in the channel order of the key loads -------------------------------------
    uint32_t q[NT][KS][2];
    float unit[NT][2];                                              // scores to log2, per column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + r;
        uint32_t w[D / 8];                                        // the lane's D / 4 channels of its row
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = 0;
        if (row < rows) {
            const uint8_t* p = reinterpret_cast<const uint8_t*>(a.q) + ((t0 + row / G) * a.q_stride + (int64_t)(h * G + row % G) * D) * 2;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(p + (FP4 ? c * (D / 2) + 16 * i : c * 16 + 64 * i));
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        }
        unit[nt][0] = unit[nt][1] = a.scale * attn::kLog2e;
        if constexpr (FP4) {
            // 4-bit keys meet the queries in fp16, where they convert in one instruction a pair: a query row
            // is divided by a power of two near its largest magnitude, which keeps every element's bf16
            // bits down to 2^-14 of the largest; the power goes back into the scores
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const int e = min(max((int)(top >> 7), 1), 253);          // biased exponent
            const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 f = kv::bf16x2_to_f32(w[i]);
                w[i] = kv::f32_to_f16x2(f.x * down, f.y * down);
            }
            unit[nt][0] *= __shfl_sync(~0u, up, 8 * c);
            unit[nt][1] *= __shfl_sync(~0u, up, 8 * c + 4);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) q[nt][s][0] = w[2 * s], q[nt][s][1] = w[2 * s + 1];
    }
    int pos[NT][2];                                                 // positions of the lane's two columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) pos[nt][i] = first + (nt * 8 + 2 * c + i) / G;
    const int last = len - 1;

    float o[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
    }

    KeyTile<D, FP4, TB> kt;
    ValueTile<D, FP4, TB> vt;
    int32_t row_of[TB], next_row[TB], far_row[TB];                        // of tiles i, i + kWarps, i + 2 kWarps
    int i = tile_lo + warp;
    const auto rows_of = [&](int tile, int32_t* out) {
        const int base = attn::tile_base<kTile>(sp, tile);
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            const int j = base + 16 * tb;                             // only pages that hold a visible token are looked up
            const bool needed = j < sp.hi && (j + 16 > sp.lo || j < sp.sink_end);
            out[tb] = needed ? block_row(a, b, j, h) : -1;
        }
    };
    const uint8_t* const k_at = a.c.k + kt.lane_offset(r, c);
    const uint8_t* const v_at = a.c.v + vt.lane_offset(r, c);
    const uint8_t* const ks_at = a.c.ks + kt.scale_offset(r, c);
    const uint8_t* const vs_at = a.c.vs + vt.scale_offset(r, c);
    const auto load_keys = [&](const int32_t* at) {
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
            if (at[tb] >= 0) kt.load(tb, k_at, ks_at, at[tb]);
    };
    const auto load_values = [&](int tile, const int32_t* at) {
        const int base = attn::tile_base<kTile>(sp, tile);
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) vt.load(tb, v_at, vs_at, at[tb], base + 16 * tb, sp, c);
    };
    // 16 tokens' keys and values into L2
    const auto prefetch = [&](int64_t row) {
        if (row < 0) return;
        constexpr int64_t kRow = FP4 ? D / 2 : 2 * D;
        tc::bulk_prefetch_l2(a.c.k + row * kRow, 16 * kRow);
        tc::bulk_prefetch_l2(a.c.v + row * kRow, 16 * kRow);
        if constexpr (FP4) {
            tc::bulk_prefetch_l2(a.c.ks + row * (D / 16), D);
            tc::bulk_prefetch_l2(a.c.vs + row * (D / 16), D);
        }
    };
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            kt.s[tb][e] = 0;
#pragma unroll
            for (int x = 0; x < KeyTile<D, FP4, TB>::kWords; ++x) kt.w[tb][e][x] = 0;
        }
    if (i < tile_hi) {
        rows_of(i, row_of);
        load_keys(row_of);
        load_values(i, row_of);
        if (i + kWarps < tile_hi) rows_of(i + kWarps, next_row);
        if (i + 2 * kWarps < tile_hi) rows_of(i + 2 * kWarps, far_row);
    }
    for (; i < tile_hi; i += kWarps) {
        const int base = attn::tile_base<kTile>(sp, i);
        const bool more = i + kWarps < tile_hi;
        // ---- S^T ---------------------------------------------------------------------------------------
        float s[NT][TB][4];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][tb][0] = s[nt][tb][1] = s[nt][tb][2] = s[nt][tb][3] = 0.f;
            if constexpr (!FP4) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma<false>(s[nt][tb], kt.w[tb][0][2 * k], kt.w[tb][1][2 * k], kt.w[tb][0][2 * k + 1], kt.w[tb][1][2 * k + 1],
                                   q[nt][k][0], q[nt][k][1]);
            } else {
                const uint32_t s0 = kv::e4m3x2_to_f16x2(kt.s[tb][0]), s1 = kv::e4m3x2_to_f16x2(kt.s[tb][1]);
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint32_t pick = (D == 128 && j >= 2) ? 0x3232u : 0x1010u;
                    const uint32_t f0 = __byte_perm(s0, 0, pick), f1 = __byte_perm(s1, 0, pick);
                    uint32_t x[4], y[4];
                    kv::e2m1x8_to_f16(kt.w[tb][0][j], x);
                    kv::e2m1x8_to_f16(kt.w[tb][1][j], y);
#pragma unroll
                    for (int z = 0; z < 4; ++z) x[z] = kv::mul_f16x2(x[z], f0), y[z] = kv::mul_f16x2(y[z], f1);
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma<true>(s[nt][tb], x[2 * z], y[2 * z], x[2 * z + 1], y[2 * z + 1], q[nt][2 * j + z][0], q[nt][2 * j + z][1]);
                }
            }
        }
        bool whole = base + kTile - 1 <= first && (a.window == 0 || base > last - a.window || base + kTile <= a.sinks);
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) whole = whole && row_of[tb] >= 0;
        uint32_t dead = 0;                                           // blocks of bad pages
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) dead |= row_of[tb] < 0 ? 1u << tb : 0u;
        if (more) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) row_of[tb] = next_row[tb];
            load_keys(row_of);
            if (i + 2 * kWarps < tile_hi) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) next_row[tb] = far_row[tb];
                #pragma unroll
                for (int tb = 0; tb < TB; ++tb)
                    if (lane == tb) prefetch(far_row[tb]);
                if (i + 3 * kWarps < tile_hi) rows_of(i + 3 * kWarps, far_row);
            }
        }
        // ---- softmax -------------------------------------------------------------------------------------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][tb][e] *= unit[nt][e & 1];
        if (!whole) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = base + 16 * tb + r + 8 * (e >> 1), p = pos[nt][e & 1];
                        const bool on = j <= p && j < sp.hi && (a.window == 0 || j > p - a.window || j < a.sinks) && !(dead >> tb & 1u);
                        if (!on) s[nt][tb][e] = -INFINITY;
                    }
        }
        float top[NT][2];
        bool grown = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(s[nt][0][e], s[nt][0][e + 2]);
#pragma unroll
                for (int tb = 1; tb < TB; ++tb) x = fmaxf(x, fmaxf(s[nt][tb][e], s[nt][tb][e + 2]));
                top[nt][e] = x;
                grown = grown || x > m[nt][e] + kSlack;
            }
        if (__any_sync(~0u, grown)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(top[nt][e], m[nt][e]);
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                    const float f = m[nt][e] == -INFINITY ? 0.f : attn::ex2(m[nt][e] - x);
                    m[nt][e] = x;
                    l[nt][e] *= f;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) o[nt][mt][e] *= f, o[nt][mt][e + 2] *= f;
                }
        }
        // ---- P^T, O^T += V^T P^T -----------------------------------------------------------------------------
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            uint32_t p[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
                const float e0 = attn::ex2(s[nt][tb][0] - m0), e1 = attn::ex2(s[nt][tb][1] - m1);
                const float e2 = attn::ex2(s[nt][tb][2] - m0), e3 = attn::ex2(s[nt][tb][3] - m1);
                l[nt][0] += e0 + e2;
                l[nt][1] += e1 + e3;
                p[nt][0] = transpose8x8(kv::f32_to_bf16x2(e0, e1));
                p[nt][1] = transpose8x8(kv::f32_to_bf16x2(e2, e3));
            }
            if constexpr (!FP4) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t a0 = __byte_perm(vt.w[tb][0][mt], vt.w[tb][1][mt], 0x5410), a1 = __byte_perm(vt.w[tb][0][mt], vt.w[tb][1][mt], 0x7632);
                    const uint32_t a2 = __byte_perm(vt.w[tb][2][mt], vt.w[tb][3][mt], 0x5410), a3 = __byte_perm(vt.w[tb][2][mt], vt.w[tb][3][mt], 0x7632);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<false>(o[nt][mt], a0, a1, a2, a3, p[nt][0], p[nt][1]);
                }
            } else {
                // to fp16 with the scale, exactly, then through fp32 to the bf16 pairs of two tokens
                uint32_t sc[4];
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const uint32_t s2 = kv::e4m3x2_to_f16x2(vt.s[tb][e] | vt.s[tb][e + 1] << 8);
                    sc[e] = __byte_perm(s2, 0, 0x1010), sc[e + 1] = __byte_perm(s2, 0, 0x3232);
                }
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    uint32_t x[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        kv::e2m1x8_to_f16(vt.w[tb][e][j], x[e]);
#pragma unroll
                        for (int z = 0; z < 4; ++z) x[e][z] = kv::mul_f16x2(x[e][z], sc[e]);
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 f0 = kv::f16x2_to_f32(x[0][z]), f1 = kv::f16x2_to_f32(x[1][z]);
                        const float2 f2 = kv::f16x2_to_f32(x[2][z]), f3 = kv::f16x2_to_f32(x[3][z]);
                        const uint32_t a0 = kv::f32_to_bf16x2(f0.x, f1.x), a1 = kv::f32_to_bf16x2(f0.y, f1.y);
                        const uint32_t a2 = kv::f32_to_bf16x2(f2.x, f3.x), a3 = kv::f32_to_bf16x2(f2.y, f3.y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma<false>(o[nt][4 * j + z], a0, a1, a2, a3, p[nt][0], p[nt][1]);
                    }
                }
            }
        }
        if (more) load_values(i + kWarps, row_of);
    }

    // ---- join the four warps ------------------------------------------------------------------------------
    constexpr int N = 8 * NT, kPad = D + 4;
    __shared__ float sm_m[kWarps][N], sm_l[kWarps][N];
    extern __shared__ float sm_o[];                                   // [warps][rows][kPad]; cluster: then [rows][D], [rows]
    float* const mine = sm_o + kWarps * N * kPad;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = l[nt][e];
            x += __shfl_xor_sync(~0u, x, 4);
            x += __shfl_xor_sync(~0u, x, 8);
            x += __shfl_xor_sync(~0u, x, 16);
            const int row = nt * 8 + 2 * c + e;
            if (r == 0) sm_m[warp][row] = m[nt][e], sm_l[warp][row] = x;
            if (row < rows) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    // channel of (tile, half) in the order of the value loads
                    const int d = FP4 ? r * (D / 8) + 2 * mt : r * 8 + 64 * (mt / 4) + 2 * (mt % 4);
                    *reinterpret_cast<float2*>(&sm_o[(warp * N + row) * kPad + d]) = make_float2(o[nt][mt][e], o[nt][mt][e + 2]);
                }
            }
        }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (D / 4); x += kWarps * 32) {
        const int row = x / (D / 4), d = x % (D / 4) * 4;
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w][row]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w][row] == -INFINITY ? 0.f : attn::ex2(sm_m[w][row] - mx);
            sum += f * sm_l[w][row];
            const float4 y = *reinterpret_cast<const float4*>(&sm_o[(w * N + row) * kPad + d]);
            acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
        }
        // a warp that saw nothing, or nothing but NaN, has no maximum; NaN reaches the sum through l
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (sm_l[w][row] != sm_l[w][row]) sum = acc.x = acc.y = acc.z = acc.w = sm_l[w][row];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t out_row = (t0 + row / G) * a.c.Hq + h * G + row % G;
        const float lse2 = sum == 0.f ? -INFINITY : mx + attn::lg2(sum);
        if constexpr (CLUSTER) {
            *reinterpret_cast<float4*>(mine + row * D + d) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (d == 0) mine[N * D + row] = lse2;
        } else if (parts_here > 1) {
            const int64_t at = out_row * parts.max_parts + part;
            *reinterpret_cast<float4*>(parts.o + at * D + d) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (d == 0) parts.lse2[at] = lse2;
        } else {
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + out_row * D + d) =
                make_uint2(kv::f32_to_bf16x2(acc.x * inv, acc.y * inv), kv::f32_to_bf16x2(acc.z * inv, acc.w * inv));
            if (a.lse && d == 0) a.lse[out_row] = lse2 * attn::kLn2;
        }
    }
    if constexpr (!CLUSTER) return;

    // ---- join the cluster's parts: each CTA some of the rows ------------------------------------------------
    attn::cluster_barrier();
    const int P = gridDim.y;
    for (int x = threadIdx.x; part + x / (D / 4) * P < rows; x += kWarps * 32) {
        const int row = part + x / (D / 4) * P, d = x % (D / 4) * 4;
        float mx = -INFINITY, sum = 0.f;
        for (int w = 0; w < P; ++w) mx = fmaxf(mx, attn::ld_cluster(attn::cluster_addr(mine + N * D + row, w)));
        if (mx == -INFINITY) mx = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < P; ++w) {
            const float f = attn::ex2(attn::ld_cluster(attn::cluster_addr(mine + N * D + row, w)) - mx);
            const float4 y = attn::ld_cluster4(attn::cluster_addr(mine + row * D + d, w));
            sum += f;
            acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t out_row = (t0 + row / G) * a.c.Hq + h * G + row % G;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + out_row * D + d) =
            make_uint2(kv::f32_to_bf16x2(acc.x * inv, acc.y * inv), kv::f32_to_bf16x2(acc.z * inv, acc.w * inv));
        if (a.lse && d == 0) a.lse[out_row] = sum == 0.f ? -INFINITY : (mx + attn::lg2(sum)) * attn::kLn2;
    }
    attn::cluster_barrier();                                          // nobody leaves while its parts are read
}

// Joins the parts of each row that has several.
template <int D, int kTile>
__global__ void __launch_bounds__(128) join_kernel(AttnCall a, Parts parts, const int share)
{
    a.c.err = &g_attn_error;
    const int64_t rows = a.c.T * a.c.Hq, row = min(attn::join_row_index(share), rows - 1), t = row / a.c.Hq;
    int b, n = 1;
    int64_t pos;
    if (kv::token_place(a.c, t, b, pos)) {                            // padding: written by the first part
        int64_t t0, t1;
        kv::request_rows(a.c, b, t0, t1);
        const int len = a.c.lens[b];
        const int64_t first = len - (t1 - t0);
        const Span sp = attn::make_span<kTile>(first > 0 ? first : 0, len - 1, a.max_len, a.window, a.sinks);
        n = min(parts.max_parts, (sp.tiles + parts.tiles_per_part - 1) / parts.tiles_per_part);
    }
    attn::wait_for_last();
    attn::join_row<D>(a, parts, row, attn::join_row_index(share) < rows ? n : 0, share);
}

}  // namespace

namespace {

// Rows of a (request, kv head) up to which this form is taken: 64 requests of 16 rows take 136 us here and 148
// in the tcgen05 form; more rows would not fit the registers.
constexpr int64_t kFewRows = 16;
int64_t rows_of(const kda_kv_params& p, int32_t max_new) { return (int64_t)max_new * (p.num_q_heads / p.num_kv_heads); }

// How a call of the few-rows form is cut along the cache.  An uncut call has one CTA per (request, kv
// head).  The cut aims at kCtas CTAs for the longest histories the caller's bound allows, so that ragged
// histories spread evenly (16 histories of 4096 to 131072 tokens in 4 bits: 410 us with 2,048 CTAs, 380 with
// 8,192), in parts whose fp32 outputs, written and read once, are at most 1/32 of the part's bytes (64
// requests of 4 x 4 rows: 199 us in 16 parts of 256 tokens, 148 in 4 of 1,024).  That rule does not look at how many
// CTAs result: 16 rows of one request leave most SMs idle (4 drafts over 32,768 tokens: 35 us in bf16, 66 in 4 bits).
// Tokens of a tile; in 4 bits two blocks of 16, whose shared softmax steps save instructions (380 -> 372 us).
constexpr int kFewTile(bool fp4) { return fp4 ? 32 : 16; }
constexpr int64_t kCtas = 8192;
constexpr int64_t kMinPart = 256;
// Up to eight parts are the CTAs of a cluster, which join through each other's shared memory: no workspace and
// no second launch (one token over 4,096: 12.9 -> 11.5 us on the GPU; calls in a row 20 -> 16 us, an allocation
// among them).  Only while all CTAs run at once: a cluster keeps its SMs' places until its last part is done (64
// ragged requests in clusters: 266 us against 192).  More parts, worth it from kClusterPart tokens each on, go
// through the workspace.
constexpr int64_t kCluster = 8, kClusterPart = 1024, kClusterCtas = 304;

attn::Cut cut_few(const kda_kv_params& p, int32_t n, int32_t max_new, int32_t max_len)
{
    const int tile = kFewTile(p.cache_dtype == KDA_CACHE_FP4);
    const int64_t rows = rows_of(p, max_new), min_part = std::max(kMinPart, p.cache_dtype == KDA_CACHE_FP4 ? 228 * rows : 64 * rows);
    int64_t tokens = max_len;
    if (p.window) {
        const int64_t seen = (int64_t)p.window + max_new + p.num_sinks + 3 * tile;   // both runs, rounded out to tiles
        if (seen < tokens) tokens = seen;
    }
    const int64_t tiles = (tokens + tile - 1) / tile;
    const int64_t ctas = (int64_t)n * p.num_kv_heads;
    int64_t parts = (kCtas + ctas - 1) / ctas;
    const int64_t most = tokens / min_part;
    if (parts > most) parts = most;
    if (parts > kCluster && tokens <= kCluster * kClusterPart && ctas * kCluster <= kClusterCtas) parts = kCluster;
    if (parts > 256) parts = 256;
    if (parts < 1) parts = 1;
    attn::Cut c;
    c.tiles_per_part = (int32_t)((tiles + parts - 1) / parts);
    c.parts = (int32_t)((tiles + c.tiles_per_part - 1) / c.tiles_per_part);
    c.in_cluster = c.parts > 1 && c.parts <= kCluster && ctas * c.parts <= kClusterCtas;
    return c;
}

size_t parts_bytes(const kda_kv_params& p, int64_t T, int32_t parts)
{
    return (size_t)T * p.num_q_heads * parts * (p.head_dim + 1) * 4 + 256;
}

Parts make_parts(const kda_kv_params& p, int64_t T, const attn::Cut& c, void* workspace)
{
    Parts x;
    x.max_parts = c.parts;
    x.tiles_per_part = c.tiles_per_part;
    x.o = c.parts > 1 && !c.in_cluster ? (float*)workspace : nullptr;
    x.lse2 = c.parts > 1 && !c.in_cluster ? (float*)workspace + (size_t)T * p.num_q_heads * c.parts * p.head_dim : nullptr;
    return x;
}

template <int D, bool FP4, int NT>
cudaError_t launch_few(const kda_kv_params& p, const AttnCall& a, const attn::Cut& cut, void* workspace, cudaStream_t stream)
{
    constexpr int TB = kFewTile(FP4) / 16;
    const Parts parts = make_parts(p, a.c.T, cut, workspace);
    const size_t smem = (size_t)kWarps * 8 * NT * (D + 4) * 4;
    const dim3 grid((unsigned)(a.c.n * a.c.Hkv) + attn::extra_cta(a.c), (unsigned)cut.parts);
    if (cut.in_cluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(kWarps * 32);
        cfg.dynamicSmemBytes = smem + (size_t)8 * NT * (D + 1) * 4;
        cfg.stream = stream;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 1;
        at.val.clusterDim.y = (unsigned)cut.parts;
        at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, few_rows_kernel<D, FP4, NT, TB, true>, a, parts);
    }
    few_rows_kernel<D, FP4, NT, TB, false><<<grid, kWarps * 32, smem, stream>>>(a, parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || cut.parts == 1) return e;
    return attn::launch_behind(join_kernel<D, 16 * TB>, attn::join_blocks(parts, a.c.T * a.c.Hq), 128, stream, a, parts, attn::join_warps(parts));
}

template <int D, bool FP4>
cudaError_t launch_typed(const kda_kv_params& p, const AttnCall& a, void* workspace, cudaStream_t stream)
{
    const int64_t rows = rows_of(p, a.max_new);
    if (rows <= kFewRows) {
        const attn::Cut cut = cut_few(p, a.c.n, a.max_new, a.max_len);
        return rows <= 8 ? launch_few<D, FP4, 1>(p, a, cut, workspace, stream) : launch_few<D, FP4, 2>(p, a, cut, workspace, stream);
    }
    const attn::Cut cut = cut_many(p, a.c.n, a.c.T, a.max_new, a.max_len);
    return launch_many<D, FP4>(p, a, make_parts(p, a.c.T, cut, workspace), stream);
}

}  // namespace

size_t attention_workspace_bytes(const kda_kv_params& p, int32_t num_seqs, int64_t total_tokens, int32_t max_new,
                                 int32_t max_len)
{
    const attn::Cut cut = rows_of(p, max_new) <= kFewRows ? cut_few(p, num_seqs, max_new, max_len) : cut_many(p, num_seqs, total_tokens, max_new, max_len);
    return cut.parts > 1 && !cut.in_cluster ? parts_bytes(p, total_tokens, cut.parts) : 0;
}

cudaError_t launch_attention(const kda_kv_params& p, const AttnCall& a, void* workspace, cudaStream_t stream)
{
    const bool fp4 = p.cache_dtype == KDA_CACHE_FP4;
    if (p.head_dim == 128) return fp4 ? launch_typed<128, true>(p, a, workspace, stream) : launch_typed<128, false>(p, a, workspace, stream);
    return fp4 ? launch_typed<64, true>(p, a, workspace, stream) : launch_typed<64, false>(p, a, workspace, stream);
}

cudaError_t attn_read_and_clear_error(int32_t* code)
{
    int32_t many = 0;
    cudaError_t e = read_and_clear(g_attn_error, code);
    if (e == cudaSuccess) e = attn_tc_read_and_clear_error(&many);
    if (*code == 0) *code = many;
    return e;
}

}  // namespace kda
