// kda_attn.cu -- attention of new tokens over the paged cache (kda_paged_attention).
//
// One warp per (token, query head): the lanes share the channels, the visible tokens are taken one at
// a time with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.cuh"
#include "kda_kv.cuh"

namespace kda {
namespace {

__device__ int32_t g_attn_error = 0;

template <int D, bool FP4>
__device__ __forceinline__ void load_row(const uint8_t* base, const uint8_t* scales, int64_t row, int lane, float* x)
{
    constexpr int N = D / 32;
    if constexpr (!FP4) {
        const uint16_t* s = reinterpret_cast<const uint16_t*>(base) + row * D + lane * N;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 f = kv::bf16x2_to_f32(*reinterpret_cast<const uint32_t*>(s + i));
            x[i] = f.x, x[i + 1] = f.y;
        }
    } else {
        const float s = kv::f16x2_to_f32(kv::e4m3x2_to_f16x2(scales[row * (D / 16) + lane * N / 16])).x;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 f = kv::f16x2_to_f32(kv::e2m1x2_to_f16x2(base[row * (D / 2) + (lane * N + i) / 2]));
            x[i] = f.x * s, x[i + 1] = f.y * s;
        }
    }
}

template <int D, bool FP4>
__global__ void __launch_bounds__(128) attention_kernel(AttnCall a)
{
    a.c.err = &g_attn_error;
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    const int64_t t = id / a.c.Hq;
    const int hq = (int)(id - t * a.c.Hq), h = hq / a.c.G;
    if (t >= a.c.T) return;
    int b;
    int64_t pos;
    float o[N] = {}, q[N], m = -INFINITY, l = 0.f;
    if (kv::token_place(a.c, t, b, pos)) {
        const uint16_t* qs = reinterpret_cast<const uint16_t*>(a.q) + t * a.q_stride + (int64_t)hq * D + lane * N;
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = __uint_as_float((uint32_t)qs[i] << 16) * a.scale;
        int64_t len = pos + 1;
        const int64_t room = min((int64_t)a.max_len, (int64_t)a.c.max_pages << a.c.page_shift);
        if (a.c.lens[b] > room) kv::record(a.c, kv::kErrLength);
        if (len > room) len = room;
        for (int64_t j = 0; j < len; ++j) {
            if (a.window && j >= a.sinks && j <= pos - a.window) {
                j = pos - a.window;
                continue;
            }
            const int64_t slot = kv::token_slot(a.c, b, j);
            if (slot < 0) continue;
            const int64_t row = slot + ((int64_t)h << a.c.page_shift);
            float x[N], s = 0.f;
            load_row<D, FP4>(a.c.k, a.c.ks, row, lane, x);
#pragma unroll
            for (int i = 0; i < N; ++i) s += x[i] * q[i];
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
            load_row<D, FP4>(a.c.v, a.c.vs, row, lane, x);
            const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : __expf(m - mn), e = __expf(s - mn);
            l = l * f + e;
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = o[i] * f + e * x[i];
            m = mn;
        }
    }
    const float r = l > 0.f ? 1.f / l : 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + (t * a.c.Hq + hq) * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = kv::f32_to_bf16x2(o[i] * r, o[i + 1] * r);
    if (a.lse && lane == 0) a.lse[t * a.c.Hq + hq] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attention_workspace_bytes(const kda_kv_params&, int32_t, int64_t, int32_t, int32_t) { return 0; }

cudaError_t launch_attention(const kda_kv_params& p, const AttnCall& a, void*, cudaStream_t stream)
{
    const int64_t blocks = (a.c.T * a.c.Hq + 3) / 4;
    const bool fp4 = p.cache_dtype == KDA_CACHE_FP4;
    if (p.head_dim == 128) {
        if (fp4) attention_kernel<128, true><<<(unsigned)blocks, 128, 0, stream>>>(a);
        else attention_kernel<128, false><<<(unsigned)blocks, 128, 0, stream>>>(a);
    } else {
        if (fp4) attention_kernel<64, true><<<(unsigned)blocks, 128, 0, stream>>>(a);
        else attention_kernel<64, false><<<(unsigned)blocks, 128, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t attn_read_and_clear_error(int32_t* code)
{
    int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_error, sizeof(int32_t));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(int32_t));
}

}  // namespace kda
