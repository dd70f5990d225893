// kda_ssm.cuh -- the selective state space recurrence token by token:
//
//     S_t = a_t S_{t-1} + (dt_t x_t) B_t^T,   y_t = S_t C_t + D x_t,   a_t = exp(-dt_t exp(A_log))
//
// Rows of S (channels of x) are independent.  A row is split over LPR lanes with CPL states each (16-byte
// groups 4 * (li + LPR * j), so that a load instruction of a warp reads whole rows), held in registers
// across the tokens; y_t takes log2(LPR) shuffles a row.
//
//   ssm_token_kernel   one token per request: bound by the state's bytes, read and written once.
//                      256 requests of 64 heads x 64 x 128 states: 155 us, the 157 us of the measured copy rate.
//   ssm_rows_kernel    packed prompts, tokens staged through shared memory: 3 fp32 operations a state and
//                      token; the path of fp32 inputs, of the shapes that the tensor-core form
//                      (kda_ssm_tc.cuh) does not take and of requests of few tokens.  Bound by the fp32 pipes when
//                      it fills the SMs, by the chain loads - sums - shuffles of a token (some 240 cycles with one warp a
//                      scheduler: 72 us for 5 requests of up to 583 tokens of 8 heads) when it does not; long
//                      requests are then cut into segments.
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

constexpr int kChunk = 128;                      // segments are whole chunks of the tensor-core form, but a request's last

// One segment of a request.
struct Segment {
    int32_t b, slot;                             // slot < 0: padding, zeros
    int32_t first, len;
    int32_t k, count;                            // segment k of count
    int32_t base;                                // count > 1: the request's first state in the workspace
    int32_t pad;
};

// The call's segments, the states between them and how the slices are paired.
struct Plan {
    Segment* segments;
    int32_t* found;                              // numbers of segments, of segments that another follows, of requests in several
    int32_t* followed;                           // places of segments that another follows
    int32_t* chains;                             // places of the first segments of requests in several
    float* states;                               // [..][H][P][N]: state before segment k of a request at base + k
    float* decays;                               // [..][H]: log2 of a segment's whole decay, at base + k + 1
    int32_t max_segments, max_cuts;              // max_cuts bounds both lists
    int32_t pairs_per_group, pairs;              // slice pairs
    int32_t want;                                // tokens of a segment that fill the SMs
};

// Lists the segments, the longest first (by 64 classes of length), so that no long one starts last.
__global__ void __launch_bounds__(1024) ssm_plan_kernel(const SsmCall a, const Plan plan)
{
    __shared__ int32_t bucket[65], longest, all, states[2], cuts[2];
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < 65) bucket[tid] = 0;
    if (tid < 2) states[tid] = 0, cuts[tid] = 0;
    if (tid == 0) longest = 1;
    struct Cut {
        int64_t first, len, size;                // rows; `size` tokens a segment but the last
        int32_t slot, n;                         // segments
    };
    auto cut = [&](int32_t b) -> Cut {
        Cut c;
        int64_t last;
        c.slot = a.idx[b];
        if (!layer_rows(a.cu, b, a.T, c.first, last)) record_layer_error(kDevErrSeqlens);
        c.len = last - c.first;
        if (c.slot >= a.num_slots) {
            record_layer_error(kDevErrStateIndex);
            c.slot = -1;
        }
        c.size = c.len;
        c.n = c.len > a.short_len;
        const int64_t n = c.slot < 0 || c.len < 2 * (int64_t)plan.want ? 1 : c.len / plan.want;
        if (c.n > 0 && n > 1) {
            c.size = ((c.len + n - 1) / n + kChunk - 1) / kChunk * kChunk;
            c.n = (int32_t)((c.len + c.size - 1) / c.size);                  // whole chunks may need fewer
        }
        return c;
    };
    Cut mine = {};
    if (tid < a.n) mine = cut(tid);
    auto of = [&](int32_t b) { return b == tid ? mine : cut(b); };           // looked up once for up to 1,024 requests
    __syncthreads();
    for (int32_t b = tid; b < a.n; b += 1024) {
        const Cut c = of(b);
        if (c.n > 0) atomicMax(&longest, (int32_t)c.size);
    }
    __syncthreads();
    const float scale = 63.f / (float)longest;
    for (int pass = 0; pass < 2; ++pass) {
        for (int32_t b = tid; b < a.n; b += 1024) {
            const Cut c = of(b);
            const int32_t base = c.n > 1 ? atomicAdd(&states[pass], c.n) : 0;
            for (int32_t k = 0; k < c.n; ++k) {
                const int64_t at = k * c.size, part = c.len - at < c.size ? c.len - at : c.size;
                const int key = max(0, 63 - (int)((float)part * scale));
                const int32_t place = atomicAdd(&bucket[pass == 0 ? key + 1 : key], 1);
                if (pass == 0) continue;
                Segment s;
                s.b = b; s.slot = c.slot; s.first = (int32_t)(c.first + at); s.len = (int32_t)part;
                s.k = k; s.count = c.n; s.base = base; s.pad = 0;
                plan.segments[place] = s;
                if (k + 1 < c.n) plan.followed[atomicAdd(&cuts[0], 1)] = place;
                if (k == 0 && c.n > 1) plan.chains[atomicAdd(&cuts[1], 1)] = place;
            }
        }
        __syncthreads();
        if (pass == 0 && tid < 32) {                                         // first place of each class
            const int32_t v0 = bucket[2 * tid + 1], v1 = bucket[2 * tid + 2];
            int32_t sum = v0 + v1;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t u = __shfl_up_sync(~0u, sum, off);
                if (tid >= off) sum += u;
            }
            bucket[2 * tid + 1] = sum - v1;
            bucket[2 * tid + 2] = sum;
            if (tid == 31) all = sum;
        }
        __syncthreads();
        // Requests of a sound table share no rows, and then the workspace holds their segments and states.  If it does
        // not, nothing is done: the bounds are those of every write here and in the kernels behind.
        if (pass == 0 && (all > plan.max_segments || states[0] > plan.max_cuts)) {
            if (tid < 3) plan.found[tid] = 0;
            if (tid == 0) record_layer_error(kDevErrSeqlens);
            return;
        }
    }
    if (tid == 0) plan.found[0] = all;
    if (tid < 2) plan.found[1 + tid] = cuts[tid];
}

// The state before each segment: of the first the pool's, then S = decay S + (the segment's own).
// blockIdx.x: (request in several segments, head, 1024 states).
__global__ void __launch_bounds__(256) ssm_chain_kernel(const SsmCall a, const Plan plan)
{
    const int per = (a.P * a.N + 1023) / 1024, place = (int)(blockIdx.x % per) * 1024 + threadIdx.x * 4;
    const int64_t bh = blockIdx.x / per;
    const int32_t i = (int32_t)(bh / a.H), h = (int32_t)(bh - (int64_t)i * a.H);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (i >= plan.found[2] || place >= a.P * a.N) return;
    const Segment seg = plan.segments[plan.chains[i]];
    const int64_t all = (int64_t)a.H * a.P * a.N, at = (int64_t)h * a.P * a.N + place;
    float4 v = *reinterpret_cast<const float4*>(a.pool + seg.slot * all + at);
    float* to = plan.states + seg.base * all + at;
    *reinterpret_cast<float4*>(to) = v;
    for (int k = 1; k < seg.count; ++k) {
        to += all;
        const float decay = exp2_fast(plan.decays[(int64_t)(seg.base + k) * a.H + h]);
        const float4 e = *reinterpret_cast<const float4*>(to);
        v = make_float4(fmaf(decay, v.x, e.x), fmaf(decay, v.y, e.y), fmaf(decay, v.z, e.z), fmaf(decay, v.w, e.w));
        *reinterpret_cast<float4*>(to) = v;
    }
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

// Zeros for the rows of no request, by one CTA.  (A call, so that it takes no part in the registers of the kernels around it.)
template <typename TOut>
__device__ __noinline__ void ssm_clear_unowned(const SsmCall& a, int tid, int threads)
{
    if (a.cu[0] == 0 && a.cu[a.n] == a.T) return;
    if (tid == 0) record_layer_error(kDevErrSeqlens);
    int64_t lo, hi;
    unowned_rows(a.cu, a.n, a.T, lo, hi);
    TOut* out = reinterpret_cast<TOut*>(a.out);
    const int64_t width = (int64_t)a.H * a.P;
    for (int64_t i = tid; i < lo * width; i += threads) out[i] = from_f32<TOut>(0.f);
    for (int64_t i = hi * width + tid; i < a.T * width; i += threads) out[i] = from_f32<TOut>(0.f);
}

// Packed prompts.  blockIdx.x: (request, or segment of the plan; head; slab of STEPS * ROWS rows); one CTA more gives
// zeros to rows of no request.  ENDS: only the state that a segment leaves when it starts from zero.
template <int N, int STEPS, bool ENDS, typename TIn, typename TOut>
__global__ void __launch_bounds__(kSsmThreads) ssm_rows_kernel(const SsmCall a, const ssm::Plan plan, int splits)
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
    int64_t b = bh / a.H;
    TOut* out = reinterpret_cast<TOut*>(a.out);
    const int64_t width = (int64_t)a.H * a.P;
    if (plan.segments) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (ENDS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    if (!ENDS && blockIdx.x == gridDim.x - 1) {
        ssm_clear_unowned<TOut>(a, tid, kSsmThreads);
        return;
    }
    const int h = (int)(bh - b * a.H);
    const int row0 = (int)(blockIdx.x - bh * splits) * R;
    const int rows = a.P - row0 < R ? a.P - row0 : R;    // a multiple of 8
    int64_t first, last, slot;
    ssm::Segment seg = {};
    if (plan.segments) {
        if (b >= plan.found[ENDS ? 1 : 0]) return;
        seg = plan.segments[ENDS ? plan.followed[b] : b];
        first = seg.first;
        last = first + seg.len;
        slot = seg.slot;
    } else {
        const bool ok = layer_rows(a.cu, (int32_t)b, a.T, first, last);
        slot = a.idx[b];
        if (tid == 0 && !ok) record_layer_error(kDevErrSeqlens);
        if (tid == 0 && slot >= a.num_slots) record_layer_error(kDevErrStateIndex);
        if (first == last || (a.short_len > 0 && last - first > a.short_len)) return;
        if (slot >= a.num_slots) slot = -1;
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
            if (!ENDS) ssm_cp_async16(&sC[buf][k][c], Cp + (t0 + k) * a.c_stride + c);
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
    // where the state comes from and goes to: the pool, or the states between segments
    const int64_t all = (int64_t)a.H * a.P * N, mine = ((int64_t)h * a.P + row0 + r0) * N + 4 * li;
    const float* state = (seg.count > 1 ? plan.states + (seg.base + seg.k) * all : a.pool + slot * all) + mine;
    float spent = 0.f;                                   // log2 of the decays so far
    float st[STEPS][4 * NV4];
    stage(0, first);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < NV4; ++j) {
            const float4 v = !ENDS && r0 + s * Sh::ROWS < rows ? *reinterpret_cast<const float4*>(state + (int64_t)s * Sh::ROWS * N + 4 * LPR * j)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            st[s][4 * j] = v.x; st[s][4 * j + 1] = v.y; st[s][4 * j + 2] = v.z; st[s][4 * j + 3] = v.w;
        }
    int buf = 0;
    for (int64_t t0 = first; t0 < last; t0 += kSsmTile, buf ^= 1) {
        const int count = last - t0 < kSsmTile ? (int)(last - t0) : kSsmTile;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                 // this tile is in, the last one's outputs are out
        if (t0 + kSsmTile < last) stage(buf ^ 1, t0 + kSsmTile);
        if (ENDS && tid == 0)
            for (int k = 0; k < count; ++k) spent -= sdt[buf][k] * rate * ssm::kLog2e;
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
                    if (!ENDS) load_floats<TIn, 4>(&sC[buf][k][4 * (li + LPR * j)], Cv + 4 * j);
                }
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const float u = dt * to_f32(sx[buf][k][r0 + s * Sh::ROWS]);
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4 * NV4; ++i) {
                        st[s][i] = fmaf(u, Bv[i], decay * st[s][i]);
                        if (!ENDS) sum[i & 1] = fmaf(st[s][i], Cv[i], sum[i & 1]);
                    }
                    y[s][kk] = sum[0] + sum[1];
                }
            }
            if constexpr (!ENDS) {
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
            }
        };
        int k = 0;
#pragma unroll 1
        for (; k + K <= count; k += K) tokens(std::integral_constant<int, K>(), k);
#pragma unroll 1
        for (; k < count; ++k) tokens(std::integral_constant<int, 1>(), k);
        __syncthreads();
        if constexpr (!ENDS) {
            constexpr int O = 16 / (int)sizeof(TOut);
            for (int i = tid; i < count * (rows / O); i += kSsmThreads) {
                const int k = i / (rows / O), c = i % (rows / O) * O;
                *reinterpret_cast<uint4*>(out + (t0 + k) * width + c) = *reinterpret_cast<const uint4*>(&sy[k][c]);
            }
        }
    }
    if (!ENDS && seg.k + 1 < seg.count) return;              // only a request's last segment has its final state
    float* to = (ENDS ? plan.states + (seg.base + seg.k + 1) * all : a.pool + slot * all) + mine;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < NV4; ++j)
            if (r0 + s * Sh::ROWS < rows)
                *reinterpret_cast<float4*>(to + (int64_t)s * Sh::ROWS * N + 4 * LPR * j) =
                    make_float4(st[s][4 * j], st[s][4 * j + 1], st[s][4 * j + 2], st[s][4 * j + 3]);
    if (ENDS && tid == 0 && row0 == 0) plan.decays[(int64_t)(seg.base + seg.k + 1) * a.H + h] = spent;
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

// Launched while the kernel before it in the stream runs; it waits for that one itself (griddepcontrol).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int64_t blocks, int threads, int smem, cudaStream_t stream, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool ssm_on_tensor_cores(const kda_ssm_params& p)
{
    return p.io_dtype == KDA_BF16 && (p.head_dim == 64 || p.head_dim == 128) && p.state_dim <= 128;
}

struct SsmLayout {
    ssm::Plan plan;
    bool cut;                        // some request may have several segments
    int32_t short_len;               // as in SsmCall
    size_t segments, followed, chains, states, decays, total;

    void place(void* workspace)
    {
        uint8_t* base = reinterpret_cast<uint8_t*>(workspace);
        plan.found = reinterpret_cast<int32_t*>(base);
        plan.segments = reinterpret_cast<ssm::Segment*>(base + segments);
        plan.followed = reinterpret_cast<int32_t*>(base + followed);
        plan.chains = reinterpret_cast<int32_t*>(base + chains);
        plan.states = reinterpret_cast<float*>(base + states);
        plan.decays = reinterpret_cast<float*>(base + decays);
    }
};

// Rows of S that a CTA has at once in the token-by-token form.
int ssm_rows_at_once(int N)
{
    return N <= 16 ? SsmShape<16>::ROWS : N <= 32 ? SsmShape<32>::ROWS : N <= 64 ? SsmShape<64>::ROWS : N <= 128 ? SsmShape<128>::ROWS : SsmShape<256>::ROWS;
}

SsmLayout ssm_layout(const kda_ssm_params& p, int32_t n, int64_t T)
{
    SsmLayout w = {};
    const bool tensor = ssm_on_tensor_cores(p);
    // segments so long that all of them, times the CTAs of each, just fill the SMs: one CTA an SM on the tensor cores, four
    // token by token; at least eight chunks (shorter ones cost more in launches: 5 requests of up to 583 tokens 76 -> 88 us)
    int64_t ctas = (int64_t)p.num_heads * ((p.head_dim + ssm_rows_at_once(p.state_dim) - 1) / ssm_rows_at_once(p.state_dim)), room = 4 * (int64_t)sm_count();
    if (tensor) {
        w.plan.pairs_per_group = (p.num_heads / p.num_groups * (p.head_dim / 64) + 1) / 2;
        ctas = w.plan.pairs = w.plan.pairs_per_group * p.num_groups;
        room = sm_count();
    }
    int64_t want = (T * ctas + room - 1) / room;
    if (want < 8 * ssm::kChunk) want = 8 * ssm::kChunk;
    w.cut = T >= 2 * want;
    w.plan.want = (int32_t)(want < (int64_t)1 << 30 ? want : (int64_t)1 << 30);
    const int64_t more = T / w.plan.want;                          // a request of k > 1 segments has k * want tokens or more
    // A chunk costs the same for 1 token as for 128, so requests of few tokens are done sooner token by token.  16 and 64
    // requests, us token by token and in chunks: 64 heads, 4 tokens 23 and 64 against 60 and 199, 24 tokens 50 and 168 against
    // 58 and 192, 32 tokens 61 and 214 against 55 and 186; 8 heads, 4 tokens 8 and 15 against 16 and 32, 24 tokens 15 and 30
    // against 16 and 31, 32 tokens 17 and 37 against 15 and 32.  Where the mean says that there may be such requests, they are
    // taken out; which they are, the kernels see.
    w.short_len = tensor && T < 64 * (int64_t)n ? 24 : 0;
    int64_t requests = w.short_len && T / (w.short_len + 1) < n ? T / (w.short_len + 1) : n;
    if (!tensor && !w.cut) requests = 0;                            // each request whole, without a plan
    w.plan.max_segments = requests ? (int32_t)(requests + more) : 0;
    w.plan.max_cuts = w.cut ? (int32_t)more : 0;
    auto round = [](size_t x) { return (x + 255) / 256 * 256; };
    w.segments = 256;
    w.followed = w.segments + round(sizeof(ssm::Segment) * (size_t)w.plan.max_segments);
    w.chains = w.followed + round(4 * (size_t)w.plan.max_cuts);
    w.states = w.chains + round(4 * (size_t)w.plan.max_cuts);
    w.decays = w.states + round((size_t)w.plan.max_cuts * 4 * p.num_heads * p.head_dim * p.state_dim);
    w.total = w.plan.max_segments ? w.decays + round((size_t)w.plan.max_cuts * 4 * p.num_heads) : 0;
    return w;
}

template <int N, int STEPS, typename TIn, typename TOut>
cudaError_t ssm_rows_launch(const SsmCall& a, const ssm::Plan* plan, cudaStream_t s)
{
    constexpr int R = SsmShape<N>::ROWS * STEPS;
    const int splits = (a.P + R - 1) / R;
    if constexpr (STEPS == 1) {                  // calls in segments: as many CTAs as the plan counts on
        if (plan) {
            cudaError_t e = launch_after(ssm_rows_kernel<N, 1, true, TIn, TOut>, (int64_t)plan->max_cuts * a.H * splits, kSsmThreads, 0, s, a, *plan, splits);
            if (e == cudaSuccess) e = launch_after(ssm::ssm_chain_kernel, (int64_t)(plan->max_cuts / 2 + 1) * a.H * ((a.P * N + 1023) / 1024), 256, 0, s, a, *plan);
            if (e != cudaSuccess) return e;
            return launch_after(ssm_rows_kernel<N, 1, false, TIn, TOut>, (int64_t)plan->max_segments * a.H * splits + 1, kSsmThreads, 0, s, a, *plan, splits);
        }
    }
    ssm_rows_kernel<N, STEPS, false, TIn, TOut><<<(unsigned)((int64_t)a.n * a.H * splits + 1), kSsmThreads, 0, s>>>(a, ssm::Plan{}, splits);
    return cudaGetLastError();
}

template <int N, typename TIn, typename TOut>
cudaError_t ssm_rows_steps(const SsmCall& a, const ssm::Plan* plan, cudaStream_t s)
{
    constexpr int R = SsmShape<N>::ROWS;
    if (!plan && a.P >= 2 * R && (int64_t)a.n * a.H * a.P >= (int64_t)sm_count() * 4 * R) return ssm_rows_launch<N, 2, TIn, TOut>(a, plan, s);
    return ssm_rows_launch<N, 1, TIn, TOut>(a, plan, s);
}

template <bool TOKEN, typename TIn, typename TOut>
cudaError_t ssm_states(const SsmCall& a, const ssm::Plan* plan, cudaStream_t s)
{
#define KDA_SSM_N(n) case n: return TOKEN ? ssm_token_steps<n, TIn, TOut>(a, s) : ssm_rows_steps<n, TIn, TOut>(a, plan, s)
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
cudaError_t ssm_dispatch(const kda_ssm_params& p, const SsmCall& a, const ssm::Plan* plan, cudaStream_t s)
{
    if (p.io_dtype == KDA_BF16)
        return p.out_dtype == KDA_BF16 ? ssm_states<TOKEN, __nv_bfloat16, __nv_bfloat16>(a, plan, s) : ssm_states<TOKEN, __nv_bfloat16, float>(a, plan, s);
    return p.out_dtype == KDA_BF16 ? ssm_states<TOKEN, float, __nv_bfloat16>(a, plan, s) : ssm_states<TOKEN, float, float>(a, plan, s);
}

}  // namespace

cudaError_t launch_ssm_decode(const kda_ssm_params& p, const SsmCall& a, cudaStream_t s) { return ssm_dispatch<true>(p, a, nullptr, s); }

}  // namespace kda
