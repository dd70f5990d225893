// kda_kv.cuh -- what the paged-cache kernels share: the cache's geometry, the checked walk from a
// token to its slot, and the 4-bit number formats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace kv {

// Device errors of the paged cache, next to those of kda_internal.cuh (first code wins).
enum : int32_t { kErrSeqlens = 2, kErrPage = 6, kErrPosition = 7, kErrLength = 8 };

// One call's cache and batch, resolved on the host.
struct Paged {
    uint8_t* k;               // page, head, token, channel order; row_bytes per token
    uint8_t* v;
    uint8_t* ks;              // 4-bit caches: D / 16 scale bytes per token
    uint8_t* vs;
    const int32_t* cu;        // may be null: one token per request
    const int32_t* lens;
    const int32_t* table;
    int64_t num_pages;
    int64_t T;
    int32_t n;                // requests
    int32_t max_pages;
    int32_t page_shift;       // page_size = 1 << page_shift
    int32_t Hq, Hkv, G;       // G = Hq / Hkv
    int32_t* err;             // device error word; each kernel sets it to its translation unit's
};

__device__ __forceinline__ void record(const Paged& a, int32_t code) { atomicCAS(a.err, 0, code); }

// Rows [t0, t1) of request b, clamped to the packed tensor.
__device__ __forceinline__ void request_rows(const Paged& a, int b, int64_t& t0, int64_t& t1)
{
    if (a.cu == nullptr) {
        t0 = b;
        t1 = b + 1;
        return;
    }
    t0 = a.cu[b];
    t1 = a.cu[b + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.T) {
        record(a, kErrSeqlens);
        t0 = t1 = 0;
    }
}

// Request and position of token t; false for a token that no request owns or that is padding.
__device__ __forceinline__ bool token_place(const Paged& a, int64_t t, int& b, int64_t& pos)
{
    if (a.cu == nullptr) {
        b = (int)t;
        pos = (int64_t)a.lens[b] - 1;
        return pos >= 0;
    }
    int lo = 0, hi = a.n - 1;             // the last request whose first row is <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    b = lo;
    const int64_t begin = a.cu[b], end = a.cu[b + 1];
    if (begin < 0 || t < begin || t >= end || end > a.T) {
        record(a, kErrSeqlens);
        return false;
    }
    const int32_t len = a.lens[b];
    pos = (int64_t)len - end + t;
    return len > 0 && pos >= 0;
}

// Slot of a token: page * Hkv * page_size + offset, i.e. head h's row is slot + h * page_size; -1 when
// the tables hold no such slot (recorded).
__device__ __forceinline__ int64_t token_slot(const Paged& a, int b, int64_t pos)
{
    const int64_t idx = pos >> a.page_shift;
    if (idx >= a.max_pages) {
        record(a, kErrLength);
        return -1;
    }
    const int32_t page = a.table[(int64_t)b * a.max_pages + idx];
    if (page < 0 || page >= a.num_pages) {
        record(a, kErrPage);
        return -1;
    }
    return (((int64_t)page * a.Hkv) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// ---- 4-bit values -----------------------------------------------------------------------------------
// Two e2m1 codes (one byte, low half first) as an fp16 pair, two e4m3 scales likewise: both exact.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b, x, y, z;\n\tmov.b32 {b, x, y, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(byte));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// Eight codes (one word) as four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* o)
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair)
{
    uint32_t r;
    asm("{\n\t.reg .b16 p, x;\n\tmov.b32 {p, x}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, p;\n\t}" : "=r"(r) : "r"(pair));
    return r;
}
__device__ __forceinline__ uint32_t f32_to_e4m3(float x)   // nearest even, saturating at 448; low byte
{
    uint32_t r;
    asm("{\n\t.reg .b16 p;\n\tcvt.rn.satfinite.e4m3x2.f32 p, %1, %2;\n\tcvt.u32.u16 %0, p;\n\t}" : "=r"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi)   // nearest even, saturating at 6
{
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, b, b, b};\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r & 0xffu;
}
// The larger of two magnitudes, NaN where either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
constexpr uint32_t kNanScale = 0x7f;   // e4m3: a group with this scale is NaN whatever its codes are
// A quotient computed by a product with a reciprocal is off by some 2^-23; one whose exact value has at
// most 7 significant bits is made exact again by rounding to 12.  The operands here have 8 bits (bf16)
// and 4 (e4m3) or 2 (6): a quotient that is not a rounding border of e4m3 or e2m1 (5 and 3 bits; times
// the divisor at most 7) is at least 2^-8 from one, so ties, which do occur, go the way of exact division.
// Infinities stay what they are; a NaN must not come here (the sum would carry its bits into the sign).
__device__ __forceinline__ float settle(float x)
{
    return __uint_as_float((__float_as_uint(x) + 0x800u) & 0xfffff000u);
}

__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t p)
{
    return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t p)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&p));
}
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f32_to_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace kv

// ---- launchers (kda_cache.cu, kda_attn.cu) --------------------------------------------------------------
cudaError_t launch_kv_append(const kda_kv_params& p, kv::Paged c, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride, const float* rope, int64_t rope_rows,
                             const int32_t* positions, void* q_out, cudaStream_t stream);
cudaError_t launch_kv_read(const kda_kv_params& p, kv::Paged c, void* k_out, void* v_out, cudaStream_t stream);
cudaError_t cache_error_word(int32_t** word);

struct AttnCall {
    kv::Paged c;
    const void* q;
    int64_t q_stride;
    int32_t max_new, max_len;  // host bounds
    int32_t window, sinks;
    float scale;
    int32_t min_exp;           // least biased exponent e with scale * log2(e) * 2^(e - 127) >= 2^-126: 4-bit caches divide
                               // no query row by less, or its factor would be zero and NaN beside a masked score's -inf
    void* out;
    float* lse;
    uint64_t by_group;         // 2^36 / G rounded up: row / G for row < 2^22 G is (row * by_group) >> 36
    __device__ __forceinline__ int token_of(int row) const { return (int)(((uint64_t)(uint32_t)row * by_group) >> 36); }
};
size_t attention_workspace_bytes(const kda_kv_params& p, int32_t num_seqs, int64_t total_tokens, int32_t max_new,
                                 int32_t max_len);
cudaError_t launch_attention(const kda_kv_params& p, const AttnCall& a, void* workspace, cudaStream_t stream);
cudaError_t attn_error_word(int32_t** word);
cudaError_t attn_tc_error_word(int32_t** word);

}  // namespace kda
