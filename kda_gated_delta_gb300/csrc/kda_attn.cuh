// kda_attn.cuh -- what the attention kernels share: which cache tokens a call visits and in which parts,
// and the form in which parts of one row are handed to the kernel that joins them.
#pragma once

#include "kda_kv.cuh"

namespace kda {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The tokens that any of positions [first, last] of a request may see, [0, sink_end) and [lo, hi), as a
// list of tiles of kTile tokens aligned in the sequence: `sink_tiles` tiles from 0, then tiles from
// `tile0` on.  A tile of the list holds at least one visible token.
struct Span {
    int32_t lo, hi, sink_end;
    int32_t sink_tiles, tile0, tiles;
};

template <int kTile>
__host__ __device__ __forceinline__ Span make_span(int64_t first, int64_t last, int64_t room, int32_t window, int32_t sinks)
{
    Span s;
    const int64_t hi = last + 1 < room ? last + 1 : room;
    int64_t lo = window ? first - window + 1 : 0;
    if (lo < 0) lo = 0;
    if (lo > hi) lo = hi;
    s.hi = hi > 0 ? (int32_t)hi : 0;
    s.lo = hi > 0 ? (int32_t)lo : 0;
    s.sink_end = sinks < s.lo ? sinks : s.lo;
    s.sink_tiles = (s.sink_end + kTile - 1) / kTile;
    s.tile0 = s.lo / kTile;
    if (s.tile0 < s.sink_tiles) s.tile0 = s.sink_tiles;
    const int32_t end = (s.hi + kTile - 1) / kTile;
    s.tiles = s.sink_tiles + (end > s.tile0 ? end - s.tile0 : 0);
    return s;
}

template <int kTile>
__device__ __forceinline__ int32_t tile_base(const Span& s, int32_t i)
{
    return (i < s.sink_tiles ? i : s.tile0 + i - s.sink_tiles) * kTile;
}

// Rows before the first request's and after the last one's belong to nobody; there are none with a good
// cu_seqlens.  The grid of a call with one has a CTA more than its work, which looks, and gives such rows what a
// query that sees nothing gets.  Others meet one comparison more for it at most: what every CTA runs once costs it
// some 200 cycles per eight instructions, and a look at the kernels' start took 1 to 2% of a call.  Still the 4-bit kernels'
// code came out 1% slower beside it (373 -> 376, 364 -> 370 us), with few query rows in bf16 1% faster.
inline unsigned extra_cta(const kv::Paged& c) { return c.cu ? 1 : 0; }
template <int D>
__device__ __forceinline__ void clear_unowned(const int32_t* cu, int32_t n, int32_t T, int32_t Hq, uint4* out, float* lse, int32_t* err)
{
    const int32_t first = cu[0], end = cu[n];
    if (first == 0 && end == T) return;
    atomicCAS(err, 0, kv::kErrSeqlens);
    const int64_t lo = min(max(first, 0), T), hi = min(max((int64_t)end, lo), (int64_t)T);
    for (int64_t x = threadIdx.x; x < (lo + T - hi) * Hq; x += blockDim.x) {
        const int64_t row = x < lo * Hq ? x : x + (hi - lo) * Hq;
        for (int i = 0; i < D / 8; ++i) out[row * (D / 8) + i] = make_uint4(0, 0, 0, 0);
        if (lse) lse[row] = -INFINITY;
    }
}
template <int D>
__device__ __forceinline__ void clear_unowned(const AttnCall& a)
{
    clear_unowned<D>(a.c.cu, a.c.n, (int32_t)a.c.T, a.c.Hq, reinterpret_cast<uint4*>(a.out), a.lse, a.c.err);
}
// The same as a call of plain values, for the tcgen05 kernels (4-bit prompts: written out 373 us, called 370).
template <int D>
__device__ __noinline__ void clear_unowned_call(const int32_t* cu, int32_t n, int32_t T, int32_t Hq, uint4* out, float* lse, int32_t* err)
{
    clear_unowned<D>(cu, n, T, Hq, out, lse, err);
}

// Parts of a row that several CTAs worked on: [row][part][D] fp32 outputs, each normalised by its own
// sum, and their log2 of the sum of exponentials [row][part], -inf for an empty part.
struct Parts {
    float* o;                  // null where the parts' CTAs join in a cluster, and where there is one part
    float* lse2;
    int32_t max_parts;
    int32_t tiles_per_part;
};

// How the host cuts a call along the cache; parts = 1: not at all.
struct Cut {
    int32_t parts, tiles_per_part;
    bool in_cluster = false;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Shared memory of the cluster's CTA `rank` at this CTA's address p.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
// All threads of all CTAs of the cluster, what they wrote to shared memory before included.
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The joining kernel may be launched as soon as every CTA of the parts' kernel has begun, and waits there for
// its end (programmatic dependent launch): its launch and its loads of the tables overlap the last CTAs.  Every CTA waits, also one with nothing to join, so
// that whatever follows in the stream follows both kernels.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), int64_t blocks, int threads, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// How many of a joining CTA's four warps share a row: one while there are few parts (a verify of 8,192 rows in
// 4 parts takes 140 us with a warp a row, 146 with a CTA a row), all four when a row's parts are a long chain
// of loads (a step of 512 rows in 64 parts: 380 us against 399).
inline int join_warps(const Parts& p) { return p.max_parts > 8 ? 4 : 1; }
inline int64_t join_blocks(const Parts& p, int64_t rows) { return p.max_parts > 8 ? rows : (rows + 3) / 4; }
__device__ __forceinline__ int64_t join_row_index(int share) { return ((int64_t)blockIdx.x * 4 + threadIdx.x / 32) / share; }

// One row's parts joined by `share` warps: each takes every share-th part, its lanes D / 32 channels each, and
// the first puts their sums together.  n <= 1: nothing to join.  All warps of the CTA come here.
template <int D>
__device__ __forceinline__ void join_row(const AttnCall& a, const Parts& parts, int64_t row, int n, int share)
{
    constexpr int N = D / 32;
    __shared__ float sm_o[4][D], sm_sum[4];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, first = warp % share;
    const float* lse = parts.lse2 + row * parts.max_parts;
    const float* src = parts.o + row * parts.max_parts * D + lane * N;
    float mx = -INFINITY, sum = 0.f, o[N] = {};
    if (n > 1) {
        for (int i = lane; i < n; i += 32) mx = fmaxf(mx, lse[i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
        if (mx == -INFINITY) mx = 0.f;                                // nothing seen, or NaN (which the weights carry on)
#pragma unroll 4
        for (int i = first; i < n; i += share) {
            const float w = ex2(lse[i] - mx);
            sum += w;
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] += w * src[(int64_t)i * D + j];
        }
    }
    if (share > 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) sm_o[warp][lane * N + j] = o[j];
        if (lane == 0) sm_sum[warp] = sum;
        __syncthreads();
        sum = (sm_sum[0] + sm_sum[1]) + (sm_sum[2] + sm_sum[3]);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = lane * N + j;
            o[j] = (sm_o[0][c] + sm_o[1][c]) + (sm_o[2][c] + sm_o[3][c]);
        }
    }
    if (n <= 1 || first != 0) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + row * D + lane * N;
#pragma unroll
    for (int j = 0; j < N; j += 2) *reinterpret_cast<uint32_t*>(dst + j) = kv::f32_to_bf16x2(o[j] * inv, o[j + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (mx + lg2(sum)) * kLn2;
}

}  // namespace attn

// kda_attn_tc.cu: the form for many query rows
attn::Cut cut_many(const kda_kv_params& p, int32_t n, int64_t T, int32_t max_new, int32_t max_len);
template <int D, bool FP4>
cudaError_t launch_many(const kda_kv_params& p, const AttnCall& a, const attn::Parts& parts, cudaStream_t stream);
cudaError_t attn_tc_read_and_clear_error(int32_t* code);

}  // namespace kda
