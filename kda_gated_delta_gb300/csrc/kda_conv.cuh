// kda_conv.cuh -- short causal convolution over packed prompts and over single tokens, with the pooled
// state of each request's last inputs.
//
//     y_t[c] = act(bias[c] + sum_{i < W} weight[c][i] x_{t-W+1+i}[c])
//
// Bound by bytes: an input is read once, an output written once.  A thread owns V neighbouring channels
// (16 bytes) of a tile of tokens and carries the last W - 1 inputs in registers, so that only the tile's
// first W - 1 rows are read twice (from L2, mostly).  The thread that meets a request's first token also
// writes the request's new state: it has read the old one by then, and nobody else touches these
// channels of the slot, so the update in place needs neither a second launch nor an order among CTAs.
#pragma once

#include "kda_layer.cuh"

namespace kda {

constexpr int kConvThreads = 128;
constexpr int kConvTile = 32;        // tokens of a thread

// The V channels from `c` on, their output and the parameters of their taps.
template <typename T, int V, int W>
struct ConvLane {
    float w[W][V], bias[V];
    T* out;
    int64_t out_stride;

    __device__ __forceinline__ ConvLane(const ConvCall& a, int c)
    {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i][v] = a.weight[(int64_t)(c + v) * W + i];
            bias[v] = a.bias ? a.bias[c + v] : 0.f;
        }
        void* base = a.out[0];
        int first = 0, next = a.out_first[1];
#pragma unroll
        for (int j = 1; j < kMaxOuts; ++j)
            if (j < a.num_outs && c >= a.out_first[j]) {
                base = a.out[j];
                first = a.out_first[j];
                next = a.out_first[j + 1];
            }
        out_stride = next - first;
        out = reinterpret_cast<T*>(base) + (c - first);
    }

    // window[0 .. W - 2] holds the inputs before this token, oldest first; x is its own
    template <bool SILU>
    __device__ __forceinline__ void step(float (&window)[W - 1][V], const float* x, int64_t t)
    {
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = fmaf(window[0][v], w[0][v], bias[v]);
#pragma unroll
            for (int i = 1; i < W - 1; ++i) s = fmaf(window[i][v], w[i][v], s);
            s = fmaf(x[v], w[W - 1][v], s);
            y[v] = SILU ? s * fast_sigmoid(s) : s;
#pragma unroll
            for (int i = 0; i < W - 2; ++i) window[i][v] = window[i + 1][v];
            window[W - 2][v] = x[v];
        }
        store_raw<T, V>(out + t * out_stride, from_floats<T, V>(y));
    }
    __device__ __forceinline__ void zero(int64_t t)
    {
        const float y[V] = {};
        store_raw<T, V>(out + t * out_stride, from_floats<T, V>(y));
    }
};

// One token per request: blockIdx.x the request, blockIdx.y the channels.
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_token_kernel(const ConvCall a)
{
    const int c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    const int64_t b = blockIdx.x;
    int64_t slot = a.idx[b];
    const auto raw = load_raw<T, V>(reinterpret_cast<const T*>(a.x) + b * a.x_stride + c);
    ConvLane<T, V, W> lane(a, c);
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) record_layer_error(kDevErrStateIndex);
        slot = -1;
    }
    if (slot < 0) {
        lane.zero(b);
        return;
    }
    T* state = reinterpret_cast<T*>(a.pool) + slot * (W - 1) * a.C + c;
    typename Vec<T, V>::Raw old[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) old[i] = load_raw<T, V>(state + (int64_t)i * a.C);
    float window[W - 1][V], x[V];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) to_floats<T, V>(old[i], window[i]);
    to_floats<T, V>(raw, x);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store_raw<T, V>(state + (int64_t)i * a.C, i < W - 2 ? old[i < W - 2 ? i + 1 : 0] : raw);
    lane.template step<SILU>(window, x, b);
}

// Where the tile that would end before row e ends: a request's first W - 1 tokens, whose outputs depend on
// its old state, stay with the CTA that has its first token and replaces that state.
template <int W>
__device__ __forceinline__ int64_t conv_tile_edge(const ConvCall& a, int64_t e)
{
    if (e >= a.T) return a.T;
    int64_t first, last;
    const int32_t b = layer_owner(a.cu, a.n, e);
    if (b < 0 || b >= a.n || !layer_rows(a.cu, b, a.T, first, last)) return e;
    if (first >= e || e - first >= W - 1) return e;
    return first + (W - 1) < last ? first + (W - 1) : last;
}

// Packed prompts: blockIdx.x the tile of kConvTile tokens, blockIdx.y the channels.
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_rows_kernel(const ConvCall a)
{
    const int c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    const int64_t t0 = conv_tile_edge<W>(a, (int64_t)blockIdx.x * kConvTile);
    const int64_t t1 = conv_tile_edge<W>(a, ((int64_t)blockIdx.x + 1) * kConvTile);
    if (t0 >= t1) return;
    const T* x = reinterpret_cast<const T*>(a.x) + c;
    ConvLane<T, V, W> lane(a, c);

    float window[W - 1][V];
    int32_t b = layer_owner(a.cu, a.n, t0);
    int64_t last = t0, slot = -1;                   // the stretch of rows that t is in ends at `last`; slot < 0: zeros
    constexpr int U = 4;                            // rows in flight
    for (int64_t t = t0; t < t1; t += U) {
        typename Vec<T, V>::Raw raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load_raw<T, V>(x + (t + u < t1 ? t + u : t1 - 1) * a.x_stride);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t now = t + u;
            if (now >= t1) break;
            if (now >= last) {                       // a stretch begins, or the tile begins inside one
                while (b < a.n && a.cu[b + 1] <= now) ++b;
                int64_t first = now;
                slot = -1;
                bool ok = b >= 0 && b < a.n && layer_rows(a.cu, b, a.T, first, last);
                if (ok) {
                    slot = a.idx[b];
                    if (slot >= a.num_slots) {
                        if (threadIdx.x == 0) record_layer_error(kDevErrStateIndex);
                        slot = -1;
                    }
                } else {                             // rows of no request
                    if (threadIdx.x == 0) record_layer_error(kDevErrSeqlens);
                    last = b < 0 ? a.cu[0] : b < a.n ? now + 1 : a.T;
                }
                if (last <= now) last = now + 1;
                if (slot >= 0) {
                    T* state = reinterpret_cast<T*>(a.pool) + slot * (W - 1) * a.C + c;
                    typename Vec<T, V>::Raw old[W - 1];
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) {
                        old[i] = load_raw<T, V>(now == first ? state + (int64_t)i * a.C : x + (now - (W - 1) + i) * a.x_stride);
                        to_floats<T, V>(old[i], window[i]);
                    }
                    if (now == first) {              // the new state: the last W - 1 inputs
#pragma unroll
                        for (int i = 0; i < W - 1; ++i) {
                            const int64_t row = last - (W - 1) + i;
                            typename Vec<T, V>::Raw r = old[i];
                            if (row >= first) {
                                r = load_raw<T, V>(x + row * a.x_stride);
                            } else {                 // fewer tokens than that: the old state moves up
#pragma unroll
                                for (int k = 1; k < W - 1; ++k)
                                    if (row - first + (W - 1) == k) r = old[k];
                            }
                            store_raw<T, V>(state + (int64_t)i * a.C, r);
                        }
                    }
                }
            }
            if (slot < 0) {
                lane.zero(now);
                continue;
            }
            float xv[V];
            to_floats<T, V>(raw[u], xv);
            lane.template step<SILU>(window, xv, now);
        }
    }
}

namespace {

bool conv_vectors(const ConvCall& a, int elem)
{
    const int V = 16 / elem;
    if ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.pool)) & 15u || a.x_stride % V || a.C % V) return false;
    for (int j = 0; j < a.num_outs; ++j)
        if ((reinterpret_cast<uintptr_t>(a.out[j]) & 15u) || (a.out_first[j + 1] - a.out_first[j]) % V) return false;
    return true;
}

template <typename T, int V, int W, bool SILU>
cudaError_t conv_launch(const ConvCall& a, cudaStream_t s)
{
    const unsigned slabs = (unsigned)((a.C / V + kConvThreads - 1) / kConvThreads);
    if (a.cu == nullptr) conv_token_kernel<T, V, W, SILU><<<dim3((unsigned)a.n, slabs), kConvThreads, 0, s>>>(a);
    else conv_rows_kernel<T, V, W, SILU><<<dim3((unsigned)((a.T + kConvTile - 1) / kConvTile), slabs), kConvThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t conv_dispatch(int width, bool silu, const ConvCall& a, cudaStream_t s)
{
    switch (width) {
    case 2: return silu ? conv_launch<T, V, 2, true>(a, s) : conv_launch<T, V, 2, false>(a, s);
    case 3: return silu ? conv_launch<T, V, 3, true>(a, s) : conv_launch<T, V, 3, false>(a, s);
    default: return silu ? conv_launch<T, V, 4, true>(a, s) : conv_launch<T, V, 4, false>(a, s);
    }
}

}  // namespace

cudaError_t launch_conv(const kda_conv_params& p, const ConvCall& a, cudaStream_t s)
{
    const bool silu = p.activation == KDA_ACT_SILU;
    if (p.io_dtype == KDA_BF16)
        return conv_vectors(a, 2) ? conv_dispatch<__nv_bfloat16, 8>(p.width, silu, a, s) : conv_dispatch<__nv_bfloat16, 1>(p.width, silu, a, s);
    return conv_vectors(a, 4) ? conv_dispatch<float, 4>(p.width, silu, a, s) : conv_dispatch<float, 1>(p.width, silu, a, s);
}

}  // namespace kda
