// kda_norm.cuh -- group norm of each token's channels (channels last) with an activation or an activated
// gate:  norm(x) = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias.
//
// Bound by bytes: x and the gate are read once into registers, both statistics are taken from there (the
// mean first, then the squares of the centered values: no difference of large sums), the result is written
// once.  LANES threads share a group, 8 to 32 of a warp, or a whole CTA for long groups.
#pragma once

#include "kda_layer.cuh"

namespace kda {

template <int ACT>
__device__ __forceinline__ float activate(float x)
{
    if constexpr (ACT == KDA_ACT_NONE) return x;
    const float s = fast_sigmoid(x);
    return ACT == KDA_ACT_SILU ? x * s : s;
}

// Sum over the LANES threads of a group; more than a warp: through shared memory, the same order always.
template <int LANES>
__device__ __forceinline__ float group_sum(float v, float* scratch)
{
#pragma unroll
    for (int off = (LANES < 32 ? LANES : 32) / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (LANES > 32) {
        constexpr int W = LANES / 32;
        __syncthreads();                        // the scratch of the sum before
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = scratch[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v += scratch[i];
    }
    return v;
}

// V elements at a time, NV times per thread.
template <typename TIn, typename TOut, int V, int NV, int LANES, int ACT>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256) norm_kernel(const NormCall a)
{
    constexpr int THREADS = LANES > 256 ? LANES : 256;
    __shared__ float scratch[32];
    const int lane = threadIdx.x % LANES;
    const int64_t rows = a.tokens * a.G;
    int64_t row = (int64_t)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
    const bool live = row < rows;
    if (!live) row = rows - 1;                  // keeps its place in the shuffles
    const int64_t t = row / a.G;
    const int g = (int)(row - t * a.G);
    const int n = a.size;
    const TIn* x = reinterpret_cast<const TIn*>(a.x) + t * a.x_stride + (int64_t)g * n;
    const TOut* gate = a.gate ? reinterpret_cast<const TOut*>(a.gate) + t * a.gate_stride + (int64_t)g * n : nullptr;

    float v[NV][V], z[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LANES + lane) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = 0.f, z[j][i] = 0.f;
        if (c < n) {
            load_floats<TIn, V>(x + c, v[j]);
            if (gate) load_floats<TOut, V>(gate + c, z[j]);
        }
    }
    if (a.gate) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) z[j][i] = activate<ACT>(z[j][i]);
        if (a.gate_first) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if ((j * LANES + lane) * V < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i) v[j][i] *= z[j][i];
                }
        }
    }
    const float inv_n = 1.0f / (float)n;
    if (a.center) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) s += v[j][i];
        const float m = group_sum<LANES>(s, scratch) * inv_n;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((j * LANES + lane) * V < n) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i] -= m;
            }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(v[j][i], v[j][i], s);
    const float r = 1.0f / sqrtf(fmaf(group_sum<LANES>(s, scratch), inv_n, a.eps));
    if (!live) return;
    TOut* out = reinterpret_cast<TOut*>(a.out) + row * n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LANES + lane) * V;
        if (c >= n) continue;
        float y[V], w[V];
        if (a.weight) load_floats<float, V>(a.weight + (int64_t)g * n + c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = a.weight ? v[j][i] * r * w[i] : v[j][i] * r;
        if (a.bias) {
            load_floats<float, V>(a.bias + (int64_t)g * n + c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] += w[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = a.gate == nullptr ? activate<ACT>(y[i]) : a.gate_first ? y[i] : y[i] * z[j][i];
        store_floats<TOut, V>(out + c, y);
    }
}

namespace {

template <typename TIn, typename TOut, int V, int NV, int LANES>
cudaError_t norm_launch(const NormCall& a, cudaStream_t s)
{
    constexpr int THREADS = LANES > 256 ? LANES : 256;
    const int64_t rows = a.tokens * a.G;
    const unsigned blocks = (unsigned)((rows + THREADS / LANES - 1) / (THREADS / LANES));
    switch (a.act) {
    case KDA_ACT_NONE: norm_kernel<TIn, TOut, V, NV, LANES, KDA_ACT_NONE><<<blocks, THREADS, 0, s>>>(a); break;
    case KDA_ACT_SILU: norm_kernel<TIn, TOut, V, NV, LANES, KDA_ACT_SILU><<<blocks, THREADS, 0, s>>>(a); break;
    default: norm_kernel<TIn, TOut, V, NV, LANES, KDA_ACT_SIGMOID><<<blocks, THREADS, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

// Lanes by the group's length: the fewest that hold it with few vectors each.
template <typename TIn, typename TOut, int V>
cudaError_t norm_lanes(const NormCall& a, cudaStream_t s)
{
    const int64_t vecs = (a.size + V - 1) / V;
    if constexpr (V > 1) {
        if (vecs <= 8) return norm_launch<TIn, TOut, V, 1, 8>(a, s);
        if (vecs <= 16) return norm_launch<TIn, TOut, V, 1, 16>(a, s);
        if (vecs <= 32) return norm_launch<TIn, TOut, V, 1, 32>(a, s);
        if (vecs <= 64) return norm_launch<TIn, TOut, V, 2, 32>(a, s);
        if (vecs <= 512) return norm_launch<TIn, TOut, V, 2, 256>(a, s);
        return norm_launch<TIn, TOut, V, 2, 1024>(a, s);
    } else {
        if (vecs <= 32) return norm_launch<TIn, TOut, V, 4, 8>(a, s);
        if (vecs <= 512) return norm_launch<TIn, TOut, V, 16, 32>(a, s);
        if (vecs <= 4096) return norm_launch<TIn, TOut, V, 16, 256>(a, s);
        return norm_launch<TIn, TOut, V, 16, 1024>(a, s);
    }
}

bool norm_vectors(const NormCall& a)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gate) | reinterpret_cast<uintptr_t>(a.weight) |
                        reinterpret_cast<uintptr_t>(a.bias) | reinterpret_cast<uintptr_t>(a.out);
    return (p & 15u) == 0 && a.size % 8 == 0 && a.x_stride % 8 == 0 && (a.gate == nullptr || a.gate_stride % 8 == 0);
}

template <typename TIn, typename TOut>
cudaError_t norm_dispatch(const NormCall& a, cudaStream_t s)
{
    return norm_vectors(a) ? norm_lanes<TIn, TOut, 8>(a, s) : norm_lanes<TIn, TOut, 1>(a, s);
}

}  // namespace

cudaError_t launch_norm(const kda_norm_params& p, const NormCall& a, cudaStream_t s)
{
    if (p.io_dtype == KDA_BF16)
        return p.out_dtype == KDA_BF16 ? norm_dispatch<__nv_bfloat16, __nv_bfloat16>(a, s) : norm_dispatch<__nv_bfloat16, float>(a, s);
    return p.out_dtype == KDA_BF16 ? norm_dispatch<float, __nv_bfloat16>(a, s) : norm_dispatch<float, float>(a, s);
}

}  // namespace kda
