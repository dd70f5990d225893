// kda_ssm.cuh -- the selective state space recurrence token by token:
//
//     S_t = a_t S_{t-1} + (dt_t x_t) B_t^T,   y_t = S_t C_t + D x_t,   a_t = exp(-dt_t exp(A_log))
//
// Rows of S (channels of x) are independent.  A row is split over LPR lanes with CPL states each (16-byte
// groups 4 * (li + LPR * j), so that a load instruction of a warp reads whole rows), held in registers
// across the tokens; y_t takes log2(LPR) shuffles a row.
//
//   ssm_token_kernel   one token per request: bound by the state's bytes, read and written once.
//   ssm_rows_kernel    packed prompts, tokens staged through shared memory: 3 fp32 operations a state and
//                      token, bound by the fp32 pipes; the path of fp32 inputs and of the shapes that the
//                      tensor-core form (kda_ssm_tc.cuh) does not take.
#pragma once

#include <type_traits>

#include "kda_layer.cuh"
#include "kda_tc.cuh"

namespace kda {

constexpr int kSsmThreads = 128;

namespace ssm {
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| <= 1, by the series of log(1 + e) = 2 artanh(e / (2 + e)), whose argument is at
// most 1 / 3: the first term left out is below 2^-25 of the sum.
__device__ __forceinline__ float softplus_series(float x, float threshold)
{
    const float e = exp2_fast(-fabsf(x) * kLog2e);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(2.0f + e));
    const float u = e * r, q = u * u;
    float p = fmaf(q, 1.f / 15, 1.f / 13);
    p = fmaf(q, p, 1.f / 11);
    p = fmaf(q, p, 1.f / 9);
    p = fmaf(q, p, 1.f / 7);
    p = fmaf(q, p, 1.f / 5);
    p = fmaf(q, p, 1.f / 3);
    p = fmaf(q, p, 1.f);
    return x > threshold ? x : fmaf(2.f * u, p, fmaxf(x, 0.f));
}
}  // namespace ssm

template <int N>
struct SsmShape {
    static constexpr int CPL = N <= 32 ? 4 : N == 64 ? 8 : 16;   // states of a lane
    static constexpr int LPR = N / CPL;                          // lanes of a row
    static constexpr int RPS = 32 / LPR;                         // rows of a warp at once
    static constexpr int ROWS = kSsmThreads / LPR;               // rows of a CTA at once
    static constexpr int NV4 = CPL / 4;
};

// dt of one head and token before softplus.
__device__ __forceinline__ float ssm_raw_step(const SsmCall& a, int64_t t, int h)
{
    const int64_t i = t * a.dt_stride + h;
    return a.dt_bf16 ? to_f32(reinterpret_cast<const __nv_bfloat16*>(a.dt)[i]) : reinterpret_cast<const float*>(a.dt)[i];
}

// One token per request.  A CTA has STEPS * ROWS rows of one (request, head).
template <int N, int STEPS, typename TIn, typename TOut>
__global__ void __launch_bounds__(kSsmThreads, STEPS >= 4 ? 4 : 8) ssm_token_kernel(const SsmCall a, int splits, int64_t ahead)
{
    using Sh = SsmShape<N>;
    constexpr int NV4 = Sh::NV4, LPR = Sh::LPR;
    const int64_t bh = blockIdx.x / splits;
    const int row0 = (int)(blockIdx.x - bh * splits) * Sh::ROWS * STEPS;
    const int64_t b = bh / a.H;
    const int h = (int)(bh - b * a.H);
    const int li = threadIdx.x % LPR, r0 = row0 + threadIdx.x / LPR;
    int64_t slot = a.idx[b];
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) record_layer_error(kDevErrStateIndex);
        slot = -1;
    }
    TOut* out = reinterpret_cast<TOut*>(a.out) + (b * a.H + h) * a.P;
    if (slot < 0) {
        for (int r = row0 + threadIdx.x; r < a.P && r < row0 + Sh::ROWS * STEPS; r += kSsmThreads) out[r] = from_f32<TOut>(0.f);
        return;
    }
    float* state = a.pool + ((slot * a.H + h) * a.P + r0) * N + 4 * li;
    float4 st[STEPS][NV4];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < NV4; ++j)
            st[s][j] = r0 + s * Sh::ROWS < a.P ? __ldcs(reinterpret_cast<const float4*>(state + (int64_t)s * Sh::ROWS * N + 4 * LPR * j))
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
    if (ahead > 0 && threadIdx.x == 0 && blockIdx.x + ahead < gridDim.x) {
        // the state of the CTA one wave of resident CTAs ahead: it is in L2 when that CTA starts
        const int64_t nb = blockIdx.x + ahead, nbh = nb / splits, q = nbh / a.H;
        const int64_t ns = a.idx[q];
        if (ns >= 0 && ns < a.num_slots) {
            const int nr = (int)(nb - nbh * splits) * Sh::ROWS * STEPS;
            const int rows = a.P - nr < Sh::ROWS * STEPS ? a.P - nr : Sh::ROWS * STEPS;
            tc::bulk_prefetch_l2(a.pool + ((ns * a.H + (nbh - q * a.H)) * a.P + nr) * N, (uint32_t)rows * N * 4);
        }
    }
    const int g = h / (a.H / a.G);
    const TIn* Bp = reinterpret_cast<const TIn*>(a.B) + b * a.b_stride + (int64_t)g * N + 4 * li;
    const TIn* Cp = reinterpret_cast<const TIn*>(a.C) + b * a.c_stride + (int64_t)g * N + 4 * li;
    const TIn* xp = reinterpret_cast<const TIn*>(a.x) + b * a.x_stride + (int64_t)h * a.P;
    float Bv[4 * NV4], Cv[4 * NV4], xv[STEPS];
#pragma unroll
    for (int j = 0; j < NV4; ++j) {
        load_floats<TIn, 4>(Bp + 4 * LPR * j, Bv + 4 * j);
        load_floats<TIn, 4>(Cp + 4 * LPR * j, Cv + 4 * j);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) xv[s] = r0 + s * Sh::ROWS < a.P ? to_f32(xp[r0 + s * Sh::ROWS]) : 0.f;
    const float dt = ssm::softplus_series(ssm_raw_step(a, b, h) + (a.dt_bias ? a.dt_bias[h] : 0.f), a.threshold);
    const float decay = expf(-dt * expf(a.A_log[h]));
    const float D = a.D ? a.D[h] : 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int r = r0 + s * Sh::ROWS;
        const float u = dt * xv[s];
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < NV4; ++j) {
            float* e = reinterpret_cast<float*>(&st[s][j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[k] = fmaf(u, Bv[4 * j + k], decay * e[k]);
                y = fmaf(e[k], Cv[4 * j + k], y);
            }
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (r < a.P) {
#pragma unroll
            for (int j = 0; j < NV4; ++j) __stcs(reinterpret_cast<float4*>(state + (int64_t)s * Sh::ROWS * N + 4 * LPR * j), st[s][j]);
            if (li == 0) out[r] = from_f32<TOut>(fmaf(D, xv[s], y));
        }
    }
}

__device__ __forceinline__ void ssm_cp_async16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

// Zeros for the rows before the first request and behind the last, by one CTA.
template <typename TOut>
__device__ __forceinline__ void ssm_clear_unowned(const SsmCall& a, int tid, int threads)
{
    TOut* out = reinterpret_cast<TOut*>(a.out);
    const int64_t width = (int64_t)a.H * a.P;
    int64_t lo = a.cu[0], hi = a.cu[a.n];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < 0 ? 0 : hi > a.T ? a.T : hi;
    if ((lo > 0 || hi < a.T) && tid == 0) record_layer_error(kDevErrSeqlens);
    for (int64_t i = tid; i < lo * width; i += threads) out[i] = from_f32<TOut>(0.f);
    for (int64_t i = hi * width + tid; i < a.T * width; i += threads) out[i] = from_f32<TOut>(0.f);
}


// Packed prompts.  blockIdx.x: (request, head, slab of STEPS * ROWS rows); one CTA more gives zeros to rows of
// no request.
template <int N, int STEPS, typename TIn, typename TOut>
__global__ void __launch_bounds__(kSsmThreads) ssm_rows_kernel(const SsmCall a, int splits)
{
    using Sh = SsmShape<N>;
    constexpr int NV4 = Sh::NV4, LPR = Sh::LPR, R = Sh::ROWS * STEPS, E = 16 / (int)sizeof(TIn);
    constexpr int XR = R < 16 ? 16 : R;
    constexpr int kSsmTile = N * sizeof(TIn) > 512 ? 8 : 16;       // tokens staged at once: at most 39 KB
    __shared__ __align__(16) TIn sB[2][kSsmTile][N], sC[2][kSsmTile][N], sx[2][kSsmTile][XR];
    __shared__ float sdt[2][kSsmTile], sa[2][kSsmTile];
    __shared__ __align__(16) TOut sy[kSsmTile][XR];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x / splits;
    const int64_t b = bh / a.H;
    TOut* out = reinterpret_cast<TOut*>(a.out);
    const int64_t width = (int64_t)a.H * a.P;
    if (b >= a.n) {
        ssm_clear_unowned<TOut>(a, tid, kSsmThreads);
        return;
    }
    const int h = (int)(bh - b * a.H);
    const int row0 = (int)(blockIdx.x - bh * splits) * R;
    const int rows = a.P - row0 < R ? a.P - row0 : R;    // a multiple of 16
    int64_t first, last;
    if (!layer_rows(a.cu, (int32_t)b, a.T, first, last) && tid == 0) record_layer_error(kDevErrSeqlens);
    if (first == last || (a.short_len > 0 && last - first > a.short_len)) return;
    int64_t slot = a.idx[b];
    if (slot >= a.num_slots) {
        if (tid == 0) record_layer_error(kDevErrStateIndex);
        slot = -1;
    }
    out += (int64_t)h * a.P + row0;
    if (slot < 0) {
        for (int64_t t = first; t < last; ++t)
            for (int r = tid; r < rows; r += kSsmThreads) out[t * width + r] = from_f32<TOut>(0.f);
        return;
    }
    const int g = h / (a.H / a.G);
    const TIn* Bp = reinterpret_cast<const TIn*>(a.B) + (int64_t)g * N;
    const TIn* Cp = reinterpret_cast<const TIn*>(a.C) + (int64_t)g * N;
    const TIn* xp = reinterpret_cast<const TIn*>(a.x) + (int64_t)h * a.P + row0;
    const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;

    float raw = tid < kSsmTile && first + tid < last ? ssm_raw_step(a, first + tid, h) : 0.f;
    auto stage = [&](int buf, int64_t t0) {
        const int count = last - t0 < kSsmTile ? (int)(last - t0) : kSsmTile;
        for (int i = tid; i < count * (N / E); i += kSsmThreads) {
            const int k = i / (N / E), c = i % (N / E) * E;
            ssm_cp_async16(&sB[buf][k][c], Bp + (t0 + k) * a.b_stride + c);
            ssm_cp_async16(&sC[buf][k][c], Cp + (t0 + k) * a.c_stride + c);
        }
        for (int i = tid; i < count * (rows / E); i += kSsmThreads) {
            const int k = i / (rows / E), c = i % (rows / E) * E;
            ssm_cp_async16(&sx[buf][k][c], xp + (t0 + k) * a.x_stride + c);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (tid < count) {
            const float dt = ssm::softplus_series(raw + bias, a.threshold);
            sdt[buf][tid] = dt;
            sa[buf][tid] = expf(-dt * rate);
        }
        // the next tile's, so that nobody waits for it there
        if (tid < kSsmTile && t0 + kSsmTile + tid < last) raw = ssm_raw_step(a, t0 + kSsmTile + tid, h);
    };

    const int li = tid % LPR, r0 = tid / LPR;
    float* state = a.pool + ((slot * a.H + h) * a.P + row0 + r0) * N + 4 * li;
    float st[STEPS][4 * NV4];
    stage(0, first);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < NV4; ++j) {
            const float4 v = r0 + s * Sh::ROWS < rows ? *reinterpret_cast<const float4*>(state + (int64_t)s * Sh::ROWS * N + 4 * LPR * j)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            st[s][4 * j] = v.x; st[s][4 * j + 1] = v.y; st[s][4 * j + 2] = v.z; st[s][4 * j + 3] = v.w;
        }
    int buf = 0;
    for (int64_t t0 = first; t0 < last; t0 += kSsmTile, buf ^= 1) {
        const int count = last - t0 < kSsmTile ? (int)(last - t0) : kSsmTile;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                 // this tile is in, the last one's outputs are out
        if (t0 + kSsmTile < last) stage(buf ^ 1, t0 + kSsmTile);
        // K tokens at a time: their row sums are independent and go through the shuffles together
        constexpr int K = 4;
        const auto tokens = [&](auto many, int k0) {
            constexpr int M = decltype(many)::value;
            float y[STEPS][M];
#pragma unroll
            for (int kk = 0; kk < M; ++kk) {
                const int k = k0 + kk;
                const float decay = sa[buf][k], dt = sdt[buf][k];
                float Bv[4 * NV4], Cv[4 * NV4];
#pragma unroll
                for (int j = 0; j < NV4; ++j) {
                    load_floats<TIn, 4>(&sB[buf][k][4 * (li + LPR * j)], Bv + 4 * j);
                    load_floats<TIn, 4>(&sC[buf][k][4 * (li + LPR * j)], Cv + 4 * j);
                }
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const float u = dt * to_f32(sx[buf][k][r0 + s * Sh::ROWS]);
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4 * NV4; ++i) {
                        st[s][i] = fmaf(u, Bv[i], decay * st[s][i]);
                        sum[i & 1] = fmaf(st[s][i], Cv[i], sum[i & 1]);
                    }
                    y[s][kk] = sum[0] + sum[1];
                }
            }
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int kk = 0; kk < M; ++kk) y[s][kk] += __shfl_xor_sync(0xffffffffu, y[s][kk], off);
            if (li == 0) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int kk = 0; kk < M; ++kk) {
                        const int r = r0 + s * Sh::ROWS;
                        sy[k0 + kk][r] = from_f32<TOut>(fmaf(D, to_f32(sx[buf][k0 + kk][r]), y[s][kk]));
                    }
            }
        };
        int k = 0;
#pragma unroll 1
        for (; k + K <= count; k += K) tokens(std::integral_constant<int, K>(), k);
#pragma unroll 1
        for (; k < count; ++k) tokens(std::integral_constant<int, 1>(), k);
        __syncthreads();
        constexpr int O = 16 / (int)sizeof(TOut);
        for (int i = tid; i < count * (rows / O); i += kSsmThreads) {
            const int k = i / (rows / O), c = i % (rows / O) * O;
            *reinterpret_cast<uint4*>(out + (t0 + k) * width + c) = *reinterpret_cast<const uint4*>(&sy[k][c]);
        }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < NV4; ++j)
            if (r0 + s * Sh::ROWS < rows)
                *reinterpret_cast<float4*>(state + (int64_t)s * Sh::ROWS * N + 4 * LPR * j) =
                    make_float4(st[s][4 * j], st[s][4 * j + 1], st[s][4 * j + 2], st[s][4 * j + 3]);
}

namespace {

template <int N, int STEPS, typename TIn, typename TOut>
cudaError_t ssm_token_launch(const SsmCall& a, cudaStream_t s)
{
    constexpr int R = SsmShape<N>::ROWS * STEPS;
    const int splits = (a.P + R - 1) / R;
    const int64_t blocks = (int64_t)a.n * a.H * splits;
    const int64_t resident = (int64_t)sm_count() * (STEPS >= 4 ? 4 : 8);
    ssm_token_kernel<N, STEPS, TIn, TOut><<<(unsigned)blocks, kSsmThreads, 0, s>>>(a, splits, blocks > resident ? resident : 0);
    return cudaGetLastError();
}

// Rows of a CTA: four steps keep 64 states a thread in flight; few requests take one step each, so that
// more SMs have work.
template <int N, typename TIn, typename TOut>
cudaError_t ssm_token_steps(const SsmCall& a, cudaStream_t s)
{
    constexpr int R = SsmShape<N>::ROWS;
    const int64_t rows = (int64_t)a.n * a.H * a.P;
    if (a.P >= 4 * R && rows >= (int64_t)sm_count() * 4 * 4 * R) return ssm_token_launch<N, 4, TIn, TOut>(a, s);
    if (a.P >= 2 * R && rows >= (int64_t)sm_count() * 4 * 2 * R) return ssm_token_launch<N, 2, TIn, TOut>(a, s);
    return ssm_token_launch<N, 1, TIn, TOut>(a, s);
}

template <int N, int STEPS, typename TIn, typename TOut>
cudaError_t ssm_rows_launch(const SsmCall& a, cudaStream_t s)
{
    constexpr int R = SsmShape<N>::ROWS * STEPS;
    const int splits = (a.P + R - 1) / R;
    const int64_t blocks = (int64_t)a.n * a.H * splits + 1;
    ssm_rows_kernel<N, STEPS, TIn, TOut><<<(unsigned)blocks, kSsmThreads, 0, s>>>(a, splits);
    return cudaGetLastError();
}

template <int N, typename TIn, typename TOut>
cudaError_t ssm_rows_steps(const SsmCall& a, cudaStream_t s)
{
    constexpr int R = SsmShape<N>::ROWS;
    if (a.P >= 2 * R && (int64_t)a.n * a.H * a.P >= (int64_t)sm_count() * 4 * R) return ssm_rows_launch<N, 2, TIn, TOut>(a, s);
    return ssm_rows_launch<N, 1, TIn, TOut>(a, s);
}

template <bool TOKEN, typename TIn, typename TOut>
cudaError_t ssm_states(const SsmCall& a, cudaStream_t s)
{
#define KDA_SSM_N(n) case n: return TOKEN ? ssm_token_steps<n, TIn, TOut>(a, s) : ssm_rows_steps<n, TIn, TOut>(a, s)
    switch (a.N) {
        KDA_SSM_N(16);
        KDA_SSM_N(32);
        KDA_SSM_N(64);
        KDA_SSM_N(128);
        KDA_SSM_N(256);
    default: return cudaErrorInvalidValue;
    }
#undef KDA_SSM_N
}

template <bool TOKEN>
cudaError_t ssm_dispatch(const kda_ssm_params& p, const SsmCall& a, cudaStream_t s)
{
    if (p.io_dtype == KDA_BF16)
        return p.out_dtype == KDA_BF16 ? ssm_states<TOKEN, __nv_bfloat16, __nv_bfloat16>(a, s) : ssm_states<TOKEN, __nv_bfloat16, float>(a, s);
    return p.out_dtype == KDA_BF16 ? ssm_states<TOKEN, float, __nv_bfloat16>(a, s) : ssm_states<TOKEN, float, float>(a, s);
}

}  // namespace

cudaError_t launch_ssm_decode(const kda_ssm_params& p, const SsmCall& a, cudaStream_t s) { return ssm_dispatch<true>(p, a, s); }

}  // namespace kda
