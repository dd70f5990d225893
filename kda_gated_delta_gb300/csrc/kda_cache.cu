// kda_cache.cu -- the paged key/value cache: kda_kv_append (rotation, 4-bit quantisation and the write)
// and kda_kv_read (back to bf16).  Both are bound by bytes: a token's rows are read once and written once.
//
// A unit is 16 channels of one row (one head of one token): in the rotated part of half style the 8
// channels 8u .. 8u+7 and their partners rot/2 away, elsewhere 16 neighbours; either way two 16-byte
// loads.  D / 16 neighbouring threads hold a row, a thread takes up to kRows rows of one token with all
// loads in flight at once, and the rotation's cosines and sines are loaded once for them.
//
// Measured: 16,412 tokens of 32 query and 8 kv heads of 128, bf16, in 72 us, 6,500 GB/s of the 6,776 that a copy
// reaches; 16,411 tokens into a 4-bit cache in 64 us (5,600 GB/s; the quantiser's instructions), and back in 24.5;
// back from a bf16 cache in 27.5 (4,900 GB/s).
// Into the 4-bit cache 2 rows per thread take 84 us and 6 take 77; CTAs of 256 threads 67 and of 64 threads 66.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kda_internal.cuh"
#include "kda_kv.cuh"

namespace kda {
namespace {

__device__ int32_t g_cache_error = 0;

constexpr int kThreads = 128;
constexpr int kRows = 4;

struct AppendArgs {
    kv::Paged c;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride;
    const float* rope;
    int64_t rope_rows;
    const int32_t* positions;
    int32_t rot, interleaved;
    int32_t rows_per_token;    // Hkv keys, Hkv values, then Hq queries when q is given
    int32_t groups;            // thread groups per token: ceil(rows_per_token / kRows)
};

// One group of 16 channels (or two halves of two groups) quantised: returns 8 codes of 8 values.
__device__ __forceinline__ uint32_t quantise8(const float* x, float rcp)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w |= kv::f32x2_to_e2m1x2(kv::settle(x[2 * i] * rcp), kv::settle(x[2 * i + 1] * rcp)) << (8 * i);
    return w;
}

__device__ __forceinline__ float max8(const float* x)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = kv::max_nan(m, fabsf(x[i]));
    return m;
}

// e4m3 scale of a group whose largest magnitude is m.  A group that holds a NaN gets a NaN scale: like in a bf16
// cache it then shows to whoever reads it.
__device__ __forceinline__ uint32_t scale_of(float m)
{
    return m == m ? kv::f32_to_e4m3(kv::settle(m * (1.0f / 6.0f))) : kv::kNanScale;
}

template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a)
{
    a.c.err = &g_cache_error;
    constexpr int U = D / 16;                                    // threads of a row
    const int64_t gid = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / U;
    const int u = threadIdx.x % U;
    const int64_t t = gid / a.groups;
    const int rg = (int)(gid - t * a.groups);
    if (t >= a.c.T) return;                                      // whole rows leave together
    const int Hkv = a.c.Hkv;

    // the thread's two runs of 8 channels
    const bool half_style = !a.interleaved && 16 * u < a.rot;
    const int c0 = half_style ? 8 * u : 16 * u;
    const int c1 = half_style ? a.rot / 2 + 8 * u : 16 * u + 8;

    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = rg + i * a.groups;
        if (row >= a.rows_per_token) break;
        const uint16_t* src = row < Hkv       ? a.k + t * a.k_stride + (int64_t)row * D
                              : row < 2 * Hkv ? a.v + t * a.v_stride + (int64_t)(row - Hkv) * D
                                              : a.q + t * a.q_stride + (int64_t)(row - 2 * Hkv) * D;
        x0[i] = *reinterpret_cast<const uint4*>(src + c0);
        x1[i] = *reinterpret_cast<const uint4*>(src + c1);
    }

    int b;
    int64_t pos, slot = -1, turn = 0;
    bool live = kv::token_place(a.c, t, b, pos);
    if (live) {
        slot = kv::token_slot(a.c, b, pos);
        turn = a.positions ? (int64_t)a.positions[t] : pos;
        if (a.rot > 0 && (turn < 0 || turn >= a.rope_rows)) {
            kv::record(a.c, kv::kErrPosition);
            live = false;
            slot = -1;
        }
    }

    const bool turned = 16 * u < a.rot;
    float co[8], si[8];
    if (turned && live) {
        const float* r = a.rope + turn * a.rot + 8 * u;          // pair p of the row: 8u .. 8u + 7 in both styles
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(r) + i);
            const float4 g = __ldg(reinterpret_cast<const float4*>(r + a.rot / 2) + i);
            co[4 * i] = f.x, co[4 * i + 1] = f.y, co[4 * i + 2] = f.z, co[4 * i + 3] = f.w;
            si[4 * i] = g.x, si[4 * i + 1] = g.y, si[4 * i + 2] = g.z, si[4 * i + 3] = g.w;
        }
    }

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = rg + i * a.groups;
        if (row >= a.rows_per_token) break;
        const bool is_v = row >= Hkv && row < 2 * Hkv, is_q = row >= 2 * Hkv;
        uint32_t w0[4] = {x0[i].x, x0[i].y, x0[i].z, x0[i].w};
        uint32_t w1[4] = {x1[i].x, x1[i].y, x1[i].z, x1[i].w};
        if (turned && live && !is_v) {
            // Each product is rounded by itself: with 16-bit table entries it is exact, and with any
            // others the result does not depend on how the compiler would contract the sum.
            if (half_style) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = kv::bf16x2_to_f32(w0[j]), y = kv::bf16x2_to_f32(w1[j]);
                    const float c = co[2 * j], s = si[2 * j], c2 = co[2 * j + 1], s2 = si[2 * j + 1];
                    w0[j] = kv::f32_to_bf16x2(__fsub_rn(__fmul_rn(x.x, c), __fmul_rn(y.x, s)),
                                              __fsub_rn(__fmul_rn(x.y, c2), __fmul_rn(y.y, s2)));
                    w1[j] = kv::f32_to_bf16x2(__fadd_rn(__fmul_rn(y.x, c), __fmul_rn(x.x, s)),
                                              __fadd_rn(__fmul_rn(y.y, c2), __fmul_rn(x.y, s2)));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = kv::bf16x2_to_f32(w0[j]), y = kv::bf16x2_to_f32(w1[j]);
                    const float c = co[j], s = si[j], c2 = co[4 + j], s2 = si[4 + j];
                    w0[j] = kv::f32_to_bf16x2(__fsub_rn(__fmul_rn(x.x, c), __fmul_rn(x.y, s)),
                                              __fadd_rn(__fmul_rn(x.y, c), __fmul_rn(x.x, s)));
                    w1[j] = kv::f32_to_bf16x2(__fsub_rn(__fmul_rn(y.x, c2), __fmul_rn(y.y, s2)),
                                              __fadd_rn(__fmul_rn(y.y, c2), __fmul_rn(y.x, s2)));
                }
            }
        }
        if (is_q) {
            uint16_t* dst = a.q_out + (t * a.c.Hq + (row - 2 * Hkv)) * D;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dst + c0) = live ? make_uint4(w0[0], w0[1], w0[2], w0[3]) : zero;
            *reinterpret_cast<uint4*>(dst + c1) = live ? make_uint4(w1[0], w1[1], w1[2], w1[3]) : zero;
            continue;
        }
        const int h = is_v ? row - Hkv : row;
        const int64_t at = slot + ((int64_t)h << a.c.page_shift);    // row of the cache
        if constexpr (!FP4) {
            if (slot >= 0) {
                uint16_t* dst = reinterpret_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at * D;
                *reinterpret_cast<uint4*>(dst + c0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
                *reinterpret_cast<uint4*>(dst + c1) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
            }
        } else {
            float x[8], y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = kv::bf16x2_to_f32(w0[j]), g = kv::bf16x2_to_f32(w1[j]);
                x[2 * j] = f.x, x[2 * j + 1] = f.y, y[2 * j] = g.x, y[2 * j + 1] = g.y;
            }
            // in half style each run is half a group: threads 2i and 2i + 1 of the row share both groups
            const unsigned mask = 3u << (threadIdx.x & 30);
            float m0 = max8(x), m1 = max8(y);
            const float o0 = __shfl_xor_sync(mask, m0, 1), o1 = __shfl_xor_sync(mask, m1, 1);
            m0 = kv::max_nan(m0, half_style ? o0 : m1);
            m1 = half_style ? kv::max_nan(m1, o1) : m0;
            const uint32_t e0 = scale_of(m0), e1 = scale_of(m1);
            if (slot >= 0) {
                const float2 s = kv::f16x2_to_f32(kv::e4m3x2_to_f16x2(e0 | e1 << 8));
                const float s0 = s.x, s1 = s.y;
                // codes of a group without a finite scale above zero: zeros
                const uint32_t q0 = e0 - 1 < kv::kNanScale - 1 ? quantise8(x, 1.0f / s0) : 0u;
                const uint32_t q1 = e1 - 1 < kv::kNanScale - 1 ? quantise8(y, 1.0f / s1) : 0u;
                uint8_t* dst = (is_v ? a.c.v : a.c.k) + at * (D / 2);
                *reinterpret_cast<uint32_t*>(dst + c0 / 2) = q0;
                *reinterpret_cast<uint32_t*>(dst + c1 / 2) = q1;
                uint8_t* ds = (is_v ? a.c.vs : a.c.ks) + at * (D / 16);
                if (!half_style || !(u & 1)) ds[c0 / 16] = (uint8_t)e0;
                if (half_style && !(u & 1)) ds[c1 / 16] = (uint8_t)e1;
            }
        }
    }
}

struct ReadArgs {
    kv::Paged c;
    uint16_t* k_out;
    uint16_t* v_out;
};

// kda_kv_read: a thread moves 16 channels of kRows rows (keys, then values) of one token.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a, const int groups)
{
    a.c.err = &g_cache_error;
    constexpr int U = D / 16;
    const int64_t gid = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / U;
    const int u = threadIdx.x % U;
    const int64_t t = gid / groups;
    const int rg = (int)(gid - t * groups);
    if (t >= a.c.T) return;
    const int Hkv = a.c.Hkv;
    int b;
    int64_t pos, slot = -1;
    if (kv::token_place(a.c, t, b, pos)) slot = kv::token_slot(a.c, b, pos);
    uint4 x0[kRows], x1[kRows];
    uint32_t sc[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = rg + i * groups;
        x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
        sc[i] = 0;
        if (row >= 2 * Hkv || slot < 0) continue;
        const bool is_v = row >= Hkv;
        const int64_t at = slot + ((int64_t)(is_v ? row - Hkv : row) << a.c.page_shift);
        const uint8_t* src = is_v ? a.c.v : a.c.k;
        if constexpr (!FP4) {
            const uint4* s = reinterpret_cast<const uint4*>(src + (at * D + 16 * u) * 2);
            x0[i] = s[0];
            x1[i] = s[1];
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(src + at * (D / 2) + 8 * u);
            x0[i].x = w.x;
            x0[i].y = w.y;
            sc[i] = (is_v ? a.c.vs : a.c.ks)[at * (D / 16) + u];
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = rg + i * groups;
        if (row >= 2 * Hkv) break;
        const bool is_v = row >= Hkv;
        uint16_t* dst = (is_v ? a.v_out : a.k_out) + (t * Hkv + (is_v ? row - Hkv : row)) * D + 16 * u;
        if constexpr (FP4) {
            uint32_t o[8];
            const float s = kv::f16x2_to_f32(kv::e4m3x2_to_f16x2(sc[i])).x;
            const uint32_t w[2] = {x0[i].x, x0[i].y};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = kv::f16x2_to_f32(kv::e2m1x2_to_f16x2((w[j / 4] >> (8 * (j % 4))) & 0xffu));
                o[j] = kv::f32_to_bf16x2(f.x * s, f.y * s);        // at most 6 significant bits: exact
            }
            x0[i] = make_uint4(o[0], o[1], o[2], o[3]);
            x1[i] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        reinterpret_cast<uint4*>(dst)[0] = x0[i];
        reinterpret_cast<uint4*>(dst)[1] = x1[i];
    }
}

template <typename F>
cudaError_t dispatch(int D, bool fp4, F f)
{
    if (D == 128) return fp4 ? f(std::integral_constant<int, 128>(), std::true_type()) : f(std::integral_constant<int, 128>(), std::false_type());
    return fp4 ? f(std::integral_constant<int, 64>(), std::true_type()) : f(std::integral_constant<int, 64>(), std::false_type());
}

}  // namespace

cudaError_t launch_kv_append(const kda_kv_params& p, kv::Paged c, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride, const float* rope, int64_t rope_rows,
                             const int32_t* positions, void* q_out, cudaStream_t stream)
{
    AppendArgs a;
    a.c = c;
    a.q = (const uint16_t*)q; a.k = (const uint16_t*)k; a.v = (const uint16_t*)v; a.q_out = (uint16_t*)q_out;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.rope = rope; a.rope_rows = rope_rows; a.positions = positions;
    a.rot = p.rot_dim; a.interleaved = p.rope_interleaved;
    a.rows_per_token = 2 * c.Hkv + (q ? c.Hq : 0);
    a.groups = (a.rows_per_token + kRows - 1) / kRows;
    return dispatch(p.head_dim, p.cache_dtype == KDA_CACHE_FP4, [&](auto d, auto fp4) {
        constexpr int D = decltype(d)::value;
        const int64_t blocks = (c.T * a.groups * (D / 16) + kThreads - 1) / kThreads;
        append_kernel<D, decltype(fp4)::value><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_kv_read(const kda_kv_params& p, kv::Paged c, void* k_out, void* v_out, cudaStream_t stream)
{
    ReadArgs a;
    a.c = c;
    a.k_out = (uint16_t*)k_out; a.v_out = (uint16_t*)v_out;
    const int groups = (2 * c.Hkv + kRows - 1) / kRows;
    return dispatch(p.head_dim, p.cache_dtype == KDA_CACHE_FP4, [&](auto d, auto fp4) {
        constexpr int D = decltype(d)::value;
        const int64_t blocks = (c.T * groups * (D / 16) + kThreads - 1) / kThreads;
        read_kernel<D, decltype(fp4)::value><<<(unsigned)blocks, kThreads, 0, stream>>>(a, groups);
        return cudaGetLastError();
    });
}

cudaError_t cache_read_and_clear_error(int32_t* code) { return read_and_clear(g_cache_error, code); }

}  // namespace kda
