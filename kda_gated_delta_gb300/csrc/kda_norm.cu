// kda_norm.cu -- group norm of each token's channels (channels last) with an activation or an activated
// gate:  norm(x) = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias.
//
// Bound by bytes: x and the gate are read once into registers, both statistics are taken from there (the
// mean first, then the squares of the centered values: no difference of large sums), the result is written
// once.  LANES threads share a group, 8 to 32 of a warp, or a whole CTA for long groups.  16,411 x 32 groups of 128 with a
// gate, bf16: 67 us, 90% of the measured copy rate.
#include "kda_layer.cuh"

namespace kda {

// The activation of a vector, act other than none.
template <int V>
__device__ __forceinline__ void activate(float* x, int act)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = fast_sigmoid(x[i]);
        x[i] = act == KDA_ACT_SILU ? x[i] * s : s;
    }
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

// V elements as they lie, to be turned into floats when they are wanted.
template <typename T, int V>
struct Held {
    static constexpr int PARTS = sizeof(T) == 4 && V == 8 ? 2 : 1, E = V / PARTS;
    typename Vec<T, E>::Raw r[PARTS];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < PARTS; ++i) r[i] = load_raw<T, E>(p + i * E);
    }
    __device__ __forceinline__ void floats(float* f) const
    {
#pragma unroll
        for (int i = 0; i < PARTS; ++i) to_floats<T, E>(r[i], f + i * E);
    }
};

// Whether the next loads are in flight meanwhile: for long groups, and for single elements, it costs more warps than it gains
__host__ __device__ constexpr bool norm_ahead(int v, int lanes) { return v > 1 ? lanes <= 256 : false; }

// V elements at a time, NV times per thread.  As many CTAs as fit at once walk over the (token, group)s, the next one's
// loads in flight while one is worked on: a CTA for each 16 groups (16,411 x 32 groups of 128) took 99 us, whatever
// it did, by the starts and ends of 33,000 CTAs.
template <typename TIn, typename TOut, int V, int NV, int LANES>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256) norm_kernel(const NormCall a)
{
    constexpr int THREADS = LANES > 256 ? LANES : 256;
    constexpr uint32_t UNITS = THREADS / LANES;
    __shared__ float scratch[32];
    const int lane = threadIdx.x % LANES, n = a.size;
    const uint32_t mine = threadIdx.x / LANES, G = a.G, units = (uint32_t)(a.tokens * G), step = gridDim.x * UNITS;
    const uint32_t step_t = step / G, step_g = step - step_t * G;
    uint32_t unit = blockIdx.x * UNITS + mine, t = unit / G, g = unit - t * G;
    Held<TIn, V> x[NV] = {};
    Held<TOut, V> z[NV] = {};
    auto ask = [&]() {
        if (unit >= units) return;
        const TIn* xp = reinterpret_cast<const TIn*>(a.x) + t * a.x_stride + (int64_t)g * n;
        const TOut* zp = reinterpret_cast<const TOut*>(a.gate) + t * a.gate_stride + (int64_t)g * n;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((j * LANES + lane) * V < n) x[j].load(xp + (j * LANES + lane) * V);
        if (a.gate) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if ((j * LANES + lane) * V < n) z[j].load(zp + (j * LANES + lane) * V);
        }
    };
    constexpr bool AHEAD = norm_ahead(V, LANES);
    if (AHEAD) ask();
    const float inv_n = 1.0f / (float)n;
    for (uint32_t first = blockIdx.x * UNITS; first < units; first += step) {
        const bool live = unit < units;
        const uint32_t t_now = t, g_now = g;
        if (!AHEAD) ask();
        float v[NV][V];
        Held<TOut, V> zr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j].floats(v[j]);
            if (!live || (j * LANES + lane) * V >= n) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) zr[j] = z[j];
        unit += step;
        t += step_t;
        g += step_g;
        if (g >= G) g -= G, ++t;
        if (AHEAD) ask();
        if (a.gate && a.gate_first) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if ((j * LANES + lane) * V < n) {
                    float w[V];
                    zr[j].floats(w);
                    if (a.act != KDA_ACT_NONE) activate<V>(w, a.act);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[j][i] *= w[i];
                }
        }
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
        const float root = rsqrtf(fmaf(group_sum<LANES>(s, scratch), inv_n, a.eps));
        if (!live) continue;
        TOut* out = reinterpret_cast<TOut*>(a.out) + ((int64_t)t_now * G + g_now) * n;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LANES + lane) * V;
            if (c >= n) continue;
            float y[V], w[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = v[j][i] * root;
            if (a.weight) {
                load_floats<float, V>(a.weight + (int64_t)g_now * n + c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] *= w[i];
            }
            if (a.bias) {
                load_floats<float, V>(a.bias + (int64_t)g_now * n + c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] += w[i];
            }
            if (!a.gate) {                      // branches around the loops: selects inside would take both sides
                if (a.act != KDA_ACT_NONE) activate<V>(y, a.act);
            } else if (!a.gate_first) {
                zr[j].floats(w);
                if (a.act != KDA_ACT_NONE) activate<V>(w, a.act);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] *= w[i];
            }
            store_floats<TOut, V>(out + c, y);
        }
    }
}

namespace {

template <typename TIn, typename TOut, int V, int NV, int LANES>
cudaError_t norm_launch(const NormCall& a, cudaStream_t s)
{
    constexpr int THREADS = LANES > 256 ? LANES : 256;
    const auto kernel = norm_kernel<TIn, TOut, V, NV, LANES>;
    constexpr int64_t units = THREADS / LANES;
    int64_t blocks = (a.tokens * a.G + units - 1) / units;
    if constexpr (norm_ahead(V, LANES)) {
        static std::atomic<int> known;           // CTAs of this kernel that an SM holds
        int per_sm = known.load(std::memory_order_relaxed);
        if (per_sm == 0) {
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, THREADS, 0) != cudaSuccess || per_sm < 1) {
                cudaGetLastError();
                per_sm = 2;
            }
            known.store(per_sm, std::memory_order_relaxed);
        }
        if (blocks > (int64_t)sm_count() * per_sm) blocks = (int64_t)sm_count() * per_sm;
    }
    kernel<<<(unsigned)blocks, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

// Lanes by the group's length: the fewest that hold it with few vectors each.  bf16 with a gate before, 16,411 tokens: 8 groups
// of 512 60 us and one of 4,096 63, of 60 by their bytes; between them and above, 256 or 1,024 threads are more than the
// vectors (8 groups of 1,024 279 us and 4 of 2,048 170, of 120; 4,099 tokens of one of 16,384 107, of 60).
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
        if (vecs <= 128) return norm_launch<TIn, TOut, V, 4, 32>(a, s);
        if (vecs <= 256) return norm_launch<TIn, TOut, V, 8, 32>(a, s);
        if (vecs <= 384) return norm_launch<TIn, TOut, V, 12, 32>(a, s);
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
