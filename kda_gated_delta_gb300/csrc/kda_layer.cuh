// kda_layer.cuh -- what the operators around a recurrence share (short convolution, selective
// recurrence, group norm): their resolved arguments, the walk over packed requests, activations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda.h"
#include "kda_internal.cuh"
#include "kda_walk.cuh"

namespace kda {

constexpr int kMaxOuts = 4;

// One call of the convolution, resolved on the host.
struct ConvCall {
    const void* x;
    int64_t x_stride;
    const float* weight;      // [C][W]
    const float* bias;        // [C] or null
    const int32_t* cu;        // null: one token per request
    int32_t n;                // requests
    int64_t T;
    void* pool;               // [slots][W - 1][C]
    int64_t num_slots;
    const int32_t* idx;
    int32_t C;
    int32_t num_outs;
    void* out[kMaxOuts];
    int32_t out_first[kMaxOuts + 1];  // first channel of each output; the last entry is C
};

// One call of the selective recurrence.
struct SsmCall {
    const void* x;
    const void* dt;
    const void* B;
    const void* C;
    int64_t x_stride, dt_stride, b_stride, c_stride;
    const float* A_log;
    const float* dt_bias;     // or null
    const float* D;           // or null
    const int32_t* cu;        // null: one token per request
    int32_t n;
    int64_t T;
    float* pool;              // [slots][H][P][N]
    int64_t num_slots;
    const int32_t* idx;
    void* out;
    int32_t H, P, N, G;
    int32_t dt_bf16;
    float threshold;
    int32_t short_len;        // requests of up to this many tokens go token by token; 0: all in the form that is called
};

struct NormCall {
    const void* x;
    int64_t x_stride;
    const void* gate;         // or null
    int64_t gate_stride;
    const float* weight;      // or null
    const float* bias;        // or null
    int64_t tokens;
    void* out;
    int32_t G, size;
    int32_t act, gate_first, center;
    float eps;
};

cudaError_t launch_conv(const kda_conv_params& p, const ConvCall& a, cudaStream_t stream);
cudaError_t launch_norm(const kda_norm_params& p, const NormCall& a, cudaStream_t stream);
cudaError_t launch_ssm_decode(const kda_ssm_params& p, const SsmCall& a, cudaStream_t stream);
size_t ssm_workspace_bytes(const kda_ssm_params& p, int32_t num_seqs, int64_t total_tokens);
cudaError_t launch_ssm_prefill(const kda_ssm_params& p, const SsmCall& a, void* workspace, cudaStream_t stream);
cudaError_t layer_error_word(int32_t** word);

// The device error word of these operators is one translation unit's.
__device__ __forceinline__ void record_layer_error(int32_t code);

// ---- vectors of V elements as fp32 -----------------------------------------------------------------
template <typename T, int V> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> { using Raw = uint4; };
template <> struct Vec<__nv_bfloat16, 4> { using Raw = uint2; };
template <> struct Vec<__nv_bfloat16, 1> { using Raw = uint16_t; };
template <> struct Vec<float, 4> { using Raw = uint4; };
template <> struct Vec<float, 1> { using Raw = uint32_t; };

__device__ __forceinline__ void unpack_bf16(uint32_t w, float* f)
{
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void to_floats(const typename Vec<T, V>::Raw& r, float* f)
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
        f[0] = __uint_as_float((uint32_t)r << 16);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) unpack_bf16(w[i], f + 2 * i);
    }
}
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::Raw from_floats(const float* f)
{
    typename Vec<T, V>::Raw r;
    if constexpr (sizeof(T) == 4) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
        r = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::Raw load_raw(const T* p)
{
    return *reinterpret_cast<const typename Vec<T, V>::Raw*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_raw(T* p, const typename Vec<T, V>::Raw& r)
{
    *reinterpret_cast<typename Vec<T, V>::Raw*>(p) = r;
}

// V elements (8 of fp32: two 16-byte words) as fp32 values, and back.
template <typename T, int V>
__device__ __forceinline__ void load_floats(const T* p, float* f)
{
    if constexpr (sizeof(T) == 4 && V == 8) {
        load_floats<T, 4>(p, f);
        load_floats<T, 4>(p + 4, f + 4);
    } else {
        to_floats<T, V>(load_raw<T, V>(p), f);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_floats(T* p, const float* f)
{
    if constexpr (sizeof(T) == 4 && V == 8) {
        store_floats<T, 4>(p, f);
        store_floats<T, 4>(p + 4, f + 4);
    } else {
        store_raw<T, V>(p, from_floats<T, V>(f));
    }
}

// sigmoid with the special-function unit's exponential and reciprocal, each off by some 2^-22.  The exponent x log2 e is
// off by up to 2^-23.7 of itself before, so a negative x adds |x| 2^-23.7 of the result: 2^-19.7 at 16, 2^-17.3 at 85.  Both are
// below a bf16 result's 2^-9; in fp32 they are the larger part of the error.  e^{-x} past the largest float gives
// 1 / inf = 0, and so do results below the smallest normal float (x < -87).
// (With flushing of subnormals: the plain forms take three further instructions an element for them, and 1 + e is
// the same.)
__device__ __forceinline__ float fast_sigmoid(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// SMs of the current device, looked up once each; where that fails, a number that is not kept.
inline int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace kda
