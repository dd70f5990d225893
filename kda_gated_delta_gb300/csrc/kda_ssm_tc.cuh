// kda_ssm_tc.cuh -- the selective state space recurrence over packed prompts on the tensor cores (bf16
// inputs, head_dim 64 or 128, up to 128 states; fewer than 64 are filled up with zeros by the copies).
//
// Unrolled over a chunk of 128 tokens that a state S [N][P] enters, with l_t = log2 a_t and G_r = sum_{i<=r} l_i:
//
//     y_r  = 2^{G_r} S^T C_r + sum_{j<=r} 2^{G_r - G_j} dt_j (C_r . B_j) x_j + D x_r
//     S'   = 2^{G_L} S + sum_j 2^{G_L - G_j} dt_j B_j x_j^T
//
// so a chunk is four products of matrices, and the state runs through elementwise operations only:
//
//     Gram = C B^T            M 128 (r) x N 128 (j) x K states, shared by the heads of a group
//     Y    = C S, scaled by 2^{G_r} and D x added in tensor memory, then += M X with
//            M_rj = Gram_rj 2^{G_r - G_j} dt_j (j <= r), from tensor memory
//     dS   = B^T X',  X'_j = 2^{G_L - G_j} dt_j x_j
//
// No exponent is positive, so nothing overflows, and none is a difference of long sums, which would lose the small
// steps behind large ones: G_L - G_j is a sum of its own from the chunk's end, G_r - G_j for rows of different
// warps is (j to the end of its block of 32) + (blocks between) + (start of its block to r).  Only inside a block
// it is a difference of sums over at most 32 steps.
// Roundings: M and S (for C S) to bf16 once, 2^-8 of a factor at most, for one operand type with x, B and C, which
// are exact.  X' is kept as the sum of two bf16 numbers, 2^-16, because its errors stay in the state: with one
// the states would be off by 2e-3 of their size, with two they are by 0.7e-6 to 1.8e-6, with three by 0.2e-6 (the third
// in S's tile, once C S has read it), but then the packed prompts below take 198 us; the fp32 recurrences of this
// library are held to 1e-5.  S itself stays in fp32 registers from a segment's first chunk to its last.
//
// A CTA takes the tokens of one request (or a segment of them) for two slices of 64 channels of x that share B
// and C: two heads of 64 channels or the halves of one of 128.  A slice has two warpgroups, one for its results (M, Y)
// and one for its state (X', S), thread = token row, and for S thread = state index.  All 512 tensor-memory columns:
// Gram 128, and per slice M 64, Y 64, dS 64.  Warp 16 issues the products, warp 17 the tensor-map copies.
//
// Long requests are cut into segments when there are fewer (request, slice pair) than SMs: a first pass
// computes each segment's own state from zero (dS only), a small kernel chains them, and every segment then
// starts from its true state.
//
// Measured (64 heads x 64 x 128 states, 8 groups, 8 prompts of 18,646 tokens): 153 us, 41% of the measured copy rate;
// one prompt of 16,411 tokens (32 heads x 128 x 128, one group) 191 us.  Bound by shared memory: a chunk of a pair moves
// 628 KB through it (products' operands 288, copies in 96, X' 96, S, X again and Y 128, the rest), 4,900 of some 6,600
// cycles, of which the products take 2,400.  A third pair of warpgroups only contended for it (180 us).
#pragma once

#include <atomic>
#include <cstddef>

#include "kda_layer.cuh"
#include "kda_ssm.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace ssm {

constexpr int kSlice = 64;                       // channels of a slice
// tensor-memory columns; Y and dS of the two slices side by side, so that one product makes both
constexpr uint32_t kGramCol = 0, kMCol = 128, kYCol = 256, kDsCol = 384;
constexpr int kTcThreads = 640;                  // state, results of two slices: 4 warps each; products, copies, two idle
// Registers of a thread at launch, and then of the state's groups (64 of them S), of the results' and of the last one.  A
// group that asks for more than the others have left waits forever, so the sum is checked here, and the launch's share
// before the launch.
constexpr int kLaunchRegs = 96, kStateRegs = 128, kResultRegs = 88, kOtherRegs = 48;
static_assert(256 * kStateRegs + 256 * kResultRegs + 128 * kOtherRegs <= kTcThreads * kLaunchRegs, "register shares");
template <int R> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
constexpr uint32_t kPolls = 1u << 24;
constexpr float kFarStep = -128.f;               // log2 of a step's decay, bounded: 2^-128 leaves nothing either way
__device__ __forceinline__ float bounded_step(float step)                                            // a NaN stays one
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(step), "f"(kFarStep));
    return r;
}

// ---- the chunk kernel ------------------------------------------------------------------------------
template <int N>
struct TcCfg {
    static constexpr int kPanel = kChunk * 128;                 // 64 columns of 128 rows
    static constexpr int kSteps = N / 16;                       // products along the states
    static constexpr int kC = 0, kB = 2 * kPanel, kX = 4 * kPanel;       // X: [slice][buffer]
    static constexpr int kXs = 8 * kPanel;                      // X': [high, low][slice]
    static constexpr int kS = 12 * kPanel;                      // S: [slice]
    static constexpr int kEnd = 14 * kPanel;
    static constexpr int kSmem = kEnd + 3072;
};

struct __align__(16) TcBars {
    uint64_t full_c, full_b[2], full_x[2];
    uint64_t gram, y_first, ds[2], y_full[2];                   // products done
    uint64_t drain;
    // what each warp of the group concerned (M and Y: of both groups) arrives at, for all slices:
    uint64_t next_s, next_y, xs, ready;                         // S written, Y read, X' written, M and Y written
    uint64_t x_free[2];                                         // an X tile is no longer needed
    uint32_t tmem;
    float total[2][2][4], tail[2][2][4];                        // [parity][slice][warp]: sums of the blocks' steps
    __align__(16) float col[2][kChunk];                         // [slice]: dt_j times the decay from j to its block's end
    __align__(16) float diag[2][kChunk];                        // [slice]: dt_j against the steps of its block up to j, or their log2
    int32_t odd_from[2][kSlice];                                // [slice][channel]: the segment's first token whose x is not finite
    int32_t odd[2];                                             // whether there is one
};
static_assert(sizeof(TcBars) <= 3072 && offsetof(TcBars, col) % 16 == 0 && offsetof(TcBars, diag) % 16 == 0, "barrier block; columns are read by 16 bytes");

__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
// Barriers of a warpgroup; the second also tells all whether any of them gave a true flag.
__device__ __forceinline__ void slice_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool slice_any(int id, bool flag)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %1, 0;\n\t"
        "bar.red.or.pred po, %2, 128, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)flag), "r"(id)
        : "memory");
    return r != 0;
}

__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (n >> 3) << 17 | (128u >> 4) << 24;
}

struct TcWork {
    Segment seg;
    int chunks, slices;
    int g;
    int first, halves;                                            // first slice of the pair; 1: two slices make a head
    int head0;                                                    // of the group
    __device__ __forceinline__ int head(int s) const { return head0 + ((first + s) >> halves); }
    __device__ __forceinline__ int channel(int s) const { return ((first + s) & halves) * kSlice; }
};

// One warp issues the products of all chunks, in the order of their operands.  It runs as one, with uniform bounds and
// addresses, so that the descriptors are uniform registers; only the products themselves are one lane's.  (One lane
// alone takes 100 to 170 cycles a product, most of them for its addresses.)
template <int N, bool ENDS, int SLICES>
__device__ bool tc_issue(const int chunks_, uint32_t smem_, TcBars* bars, uint32_t tmem_, const bool leader)
{
    using K = TcCfg<N>;
    constexpr uint32_t id_gram = idesc_bf16(128, false, false), id_y = idesc_bf16(64 * SLICES, false, true);
    constexpr uint32_t id_ds = idesc_bf16(64 * SLICES, true, true), id_mx = idesc_bf16(64, false, true);
    constexpr uint32_t kTile = K::kPanel >> 4;                       // descriptors count in units of 16 bytes
    const int chunks = (int)__reduce_max_sync(~0u, (unsigned)chunks_);
    const uint32_t tmem = __reduce_max_sync(~0u, tmem_), smem = __reduce_max_sync(~0u, smem_);
    const uint64_t c_k = tc::desc_sw128(smem + K::kC, 16, 1024), b_k = tc::desc_sw128(smem + K::kB, 16, 1024);
    const uint64_t b_mn = tc::desc_sw128(smem + K::kB, K::kPanel, 1024), other_mn = tc::desc_sw128(smem + K::kC, K::kPanel, 1024);
    const uint64_t s_mn = tc::desc_sw128(smem + K::kS, K::kPanel, 1024);
    const uint64_t xs_mn = tc::desc_sw128(smem + K::kXs, K::kPanel, 1024), x_mn = tc::desc_sw128(smem + K::kX, K::kPanel, 1024);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const uint32_t par = c & 1;
        if constexpr (!ENDS) {
            if (!tc::mbar_wait(&bars->full_c, par, kPolls)) return false;
        }
        if (!tc::mbar_wait(&bars->full_b[par], (c >> 1) & 1, kPolls)) return false;
        tc::tc_fence_after();
        if constexpr (!ENDS) {
            if (leader) {
#pragma unroll
                for (int k = 0; k < K::kSteps; ++k) {
                    const uint32_t off = (k / 4) * kTile + (k % 4) * 2;
                    tc::mma_f16_ss(tmem + kGramCol, c_k + off, b_k + off, id_gram, k > 0);
                }
                tc::mma_commit(&bars->gram);
            }
            if (!tc::mbar_wait(&bars->next_s, par, kPolls)) return false;
            if (c > 0 && !tc::mbar_wait(&bars->next_y, par ^ 1, kPolls)) return false;
            tc::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int k = 0; k < K::kSteps; ++k)
                    tc::mma_f16_ss(tmem + kYCol, c_k + ((k / 4) * kTile + (k % 4) * 2), s_mn + k * 128, id_y, k > 0);
                tc::mma_commit(&bars->y_first);
            }
        }
        if (!tc::mbar_wait(&bars->xs, par, kPolls)) return false;
        if (ENDS && c > 0 && !tc::mbar_wait(&bars->next_y, par ^ 1, kPolls)) return false;
        tc::tc_fence_after();
        if (leader) {
#pragma unroll
            for (int k = 0; k < 16; ++k)                              // eight steps with the high parts, eight with the low
                tc::mma_f16_ss(tmem + kDsCol, (ENDS && par ? other_mn : b_mn) + (k % 8) * 128, xs_mn + (k / 8) * 2 * kTile + (k % 8) * 128, id_ds, k > 0);
            tc::mma_commit(&bars->ds[par]);
        }
        if constexpr (!ENDS) {
            if (!tc::mbar_wait(&bars->ready, par, kPolls)) return false;
            tc::tc_fence_after();
            if (leader) {
                const uint64_t x = x_mn + par * kTile;
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int s = 0; s < SLICES; ++s)                  // the two slices' sums in turn
                        tc::mma_f16_ts(tmem + kYCol + 64 * s, tmem + kMCol + 64 * s + 8 * k, x + 2 * s * kTile + k * 128, id_mx, 1);
                tc::mma_commit(&bars->y_full[par]);
            }
        }
    }
    return true;
}

// One lane copies the chunks' tiles.  What a barrier is waited for here completes again only after the copy that
// follows, so no phase can be missed.
template <int N, bool ENDS>
__device__ bool tc_load(const SsmCall& a, const TcWork& w, uint8_t* smem, TcBars* bars, const CUtensorMap* xm, const CUtensorMap* bm,
                        const CUtensorMap* cm)
{
    using K = TcCfg<N>;
    for (int c = 0; c < w.chunks; ++c) {
        const int32_t t = w.seg.first + c * kChunk;
        const uint32_t par = c & 1;
        auto load_x = [&]() {
            tc::mbar_arrive_expect_tx(&bars->full_x[par], K::kPanel * w.slices);
            for (int s = 0; s < w.slices; ++s)
                tc::tma_load_2d(smem + K::kX + (2 * s + par) * K::kPanel, xm, w.head(s) * a.P + w.channel(s), t, &bars->full_x[par]);
        };
        auto load_tile = [&](uint64_t* bar, int at, const CUtensorMap* m) {
            tc::mbar_arrive_expect_tx(bar, K::kPanel * (N / 64));
#pragma unroll
            for (int p = 0; p < N / 64; ++p) tc::tma_load_3d(smem + at + p * K::kPanel, m, 64 * p, w.g, t, bar);
        };
        if constexpr (ENDS) {                                     // B in two buffers, one of them C's
            if (c > 1 && !tc::mbar_wait(&bars->ds[par], ((c >> 1) - 1) & 1, kPolls)) return false;
            load_x();
            load_tile(&bars->full_b[par], par ? K::kC : K::kB, bm);
        } else {
            if (c > 1 && !tc::mbar_wait(&bars->x_free[par], ((c >> 1) - 1) & 1, kPolls)) return false;
            load_x();
            if (c > 0 && !tc::mbar_wait(&bars->y_first, par ^ 1, kPolls)) return false;
            load_tile(&bars->full_c, K::kC, cm);
            if (c > 0 && !tc::mbar_wait(&bars->ds[par ^ 1], ((c - 1) >> 1) & 1, kPolls)) return false;
            load_tile(&bars->full_b[par], K::kB, bm);
        }
    }
    return true;
}

// What the two warpgroups of a slice share: thread r is token row r of a chunk and state r.
struct TcThread {
    TcBars* bars;
    int s, r, warp, lane, id;                                     // slice, row, its block of 32, barrier of the group
    int h, channel;
    uint32_t tmem;                                                // this warp's lanes
    float rate, bias;
    bool bad = false;                                             // a wait gave up

    __device__ __forceinline__ TcThread(const SsmCall& a, const TcWork& w, TcBars* bars_, uint32_t tmem_base, int s_, int r_, int id_)
        : bars(bars_), s(s_), r(r_), warp(r_ >> 5), lane(r_ & 31), id(id_), h(w.head(s_)), channel(w.channel(s_)),
          tmem(tmem_base + ((uint32_t)(r_ & 96) << 16)), rate(expf(a.A_log[h]) * kLog2e), bias(a.dt_bias ? a.dt_bias[h] : 0.f)
    {
    }
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity)
    {
        if (!bad) bad = !tc::mbar_wait(bar, parity, kPolls);
        __syncwarp();
    }
    __device__ __forceinline__ void arrive(uint64_t* bar) const
    {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    }
    // dt of this row in chunk c, before softplus
    __device__ __forceinline__ float raw_step(const SsmCall& a, const TcWork& w, int c) const
    {
        if (c * kChunk + r >= w.seg.len) return 0.f;
        const int64_t i = ((int64_t)w.seg.first + c * kChunk + r) * a.dt_stride + h;
        return a.dt_bf16 ? to_f32(reinterpret_cast<const __nv_bfloat16*>(a.dt)[i]) : reinterpret_cast<const float*>(a.dt)[i];
    }
};

// Zeros in M do not keep an x that is not finite from the rows before its token.  It is set to zero in the tile, and the
// rows from its token on get a NaN in its channel as they leave; the states have it from X'.  Looking for one costs an
// instruction a pair of channels (eight prompts 152.0 -> 153.6 us).
__device__ __noinline__ void tc_set_aside(TcBars* bars, int s, uint8_t* x_row, int r, int token)
{
    for (int i = 0; i < kSlice; ++i) {
        uint16_t* x = reinterpret_cast<uint16_t*>(x_row + (((i / 8) ^ (r & 7)) << 4)) + i % 8;
        if ((*x & 0x7f80u) == 0x7f80u) {
            atomicMin(&bars->odd_from[s][i], token);
            *x = 0;
            bars->odd[s] = 1;
        }
    }
}

// Who makes X' and who S: one warpgroup both; or, where no results are wanted, one each, so that the next chunk's X' is
// made while this one's S is updated (one prompt of 16,411 tokens: the first pass 75 us with one).
enum { kBoth = 0, kIncrements = 1, kStates = 2 };

// The warpgroup of a slice's state: X' and S.  A wait that gave up leaves the loop at the next barrier of the group, for
// all its threads at once.
template <int N, bool ENDS, int PART>
__device__ bool tc_state(const SsmCall& a, const Plan& plan, const TcWork& w, uint8_t* smem, TcThread t)
{
    using K = TcCfg<N>;
    TcBars* bars = t.bars;
    const int s = t.s, r = t.r, warp = t.warp, lane = t.lane;
    const uint32_t t_ds = t.tmem + kDsCol + 64 * s, t_y = t.tmem + kYCol + 64 * s;
    const float D = a.D ? a.D[t.h] : 0.f;
    uint8_t* xs_row = smem + K::kXs + s * K::kPanel + r * 128;
    uint8_t* s_row = smem + K::kS + s * K::kPanel + r * 128;

    // this thread has S[r][0 .. 63] of the slice
    float S[kSlice];
    const int64_t tile = ((int64_t)t.h * a.P + t.channel) * a.N + r, all = (int64_t)a.H * a.P * a.N;
    const bool own = r < a.N;
    if (ENDS) {
#pragma unroll
        for (int i = 0; i < kSlice; ++i) S[i] = 0.f;
    } else {
        const float* from = (w.seg.count > 1 ? plan.states + (w.seg.base + w.seg.k) * all : a.pool + w.seg.slot * all) + tile;
#pragma unroll
        for (int i = 0; i < kSlice; ++i) S[i] = own ? from[(int64_t)i * a.N] : 0.f;
    }
    auto store_s = [&]() {                                        // S in bf16, as the product with C takes it
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(s_row + ((c ^ (r & 7)) << 4)) =
                make_uint4(pack_bf16(S[8 * c], S[8 * c + 1]), pack_bf16(S[8 * c + 2], S[8 * c + 3]), pack_bf16(S[8 * c + 4], S[8 * c + 5]),
                           pack_bf16(S[8 * c + 6], S[8 * c + 7]));
        tc::fence_proxy_async();
    };
    if constexpr (!ENDS) {
        store_s();
        t.arrive(&bars->next_s);
    }
    float all_steps = 0.f;
    float weight = 0.f, gamma = 0.f, grow = 0.f;                  // of this row's X', of the state, of this row's C S
    // the steps from each token of a chunk to its end; false: a wait gave up
    auto steps = [&](int c, float raw) -> bool {
        const bool live = c * kChunk + r < w.seg.len;
        const float dt = live ? softplus_series(raw + t.bias, a.threshold) : 0.f;
        float head = live ? bounded_step(-dt * t.rate) : 0.f, tail = head;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float u = ENDS ? 0.f : __shfl_up_sync(~0u, head, off), v = __shfl_down_sync(~0u, tail, off);
            if (lane >= off) head += u;
            if (lane + off < 32) tail += v;
        }
        float (&sums)[4] = PART == kIncrements ? bars->total[c & 1][s] : bars->tail[c & 1][s];
        if (lane == 0) sums[warp] = tail;
        tail = __shfl_down_sync(~0u, tail, 1);
        if (lane == 31) tail = 0.f;
        if (slice_any(t.id, t.bad)) return false;
        float whole = 0.f;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const float f = sums[i];
            if (i > warp) tail += f;
            if (i < warp) head += f;
            whole += f;
        }
        weight = live ? dt * exp2_fast(tail) : 0.f;
        gamma = exp2_fast(whole);
        grow = exp2_fast(head);
        all_steps += whole;
        return true;
    };
    if (!steps(0, t.raw_step(a, w, 0))) return false;
    for (int c = 0; c < w.chunks; ++c) {
        const uint32_t par = c & 1;
        const int len = w.seg.len - c * kChunk < kChunk ? w.seg.len - c * kChunk : kChunk;
        const bool live = r < len;
        uint8_t* x_row = smem + K::kX + (2 * s + par) * K::kPanel + r * 128;
        if constexpr (PART != kStates) {
            // ---- X' = weight x, in two parts
            if (PART == kIncrements && c > 0) t.wait(&bars->ds[par ^ 1], ((c - 1) >> 1) & 1);      // the last X' has been read
            t.wait(&bars->full_x[par], (c >> 1) & 1);
            if (len < kChunk) t.wait(&bars->full_b[par], (c >> 1) & 1);
            if (live) {
                const uint64_t ww = pack2(weight, weight), minus = pack2(-1.f, -1.f);
                uint64_t nothing = 0;                              // two zeros, until a part of X' is not finite
#pragma unroll 4
                for (int q = 0; q < 8; ++q) {
                    const int at = (q ^ (r & 7)) << 4;
                    const uint4 raw_x = *reinterpret_cast<const uint4*>(x_row + at);
                    const uint32_t xw[4] = {raw_x.x, raw_x.y, raw_x.z, raw_x.w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        float f[2];
                        unpack_bf16(xw[z], f);
                        const uint64_t v = mul2(pack2(f[0], f[1]), ww);
                        const float2 vf = unpack2(v);
                        hi[z] = pack_bf16(vf.x, vf.y);
                        unpack_bf16(hi[z], f);
                        const uint64_t small = fma2(pack2(f[0], f[1]), minus, v);
                        const float2 rest = unpack2(small);
                        lo[z] = pack_bf16(rest.x, rest.y);
                        if (!ENDS) nothing = fma2(small, 0, nothing);
                    }
                    *reinterpret_cast<uint4*>(xs_row + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(xs_row + 2 * K::kPanel + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                const float2 flag = unpack2(nothing);
                if (!ENDS && !(flag.x + flag.y == 0.f)) tc_set_aside(bars, s, x_row, r, c * kChunk + r);
            } else {
                // rows behind the request's last: another's, or nobody's; zeros, for a weight of zero does not stop a NaN
                const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int q = 0; q < 128; q += 16) {
                    *reinterpret_cast<uint4*>(x_row + q) = none;
                    *reinterpret_cast<uint4*>(xs_row + q) = none;
                    *reinterpret_cast<uint4*>(xs_row + 2 * K::kPanel + q) = none;
#pragma unroll
                    for (int p = 0; p < N / 64; ++p) *reinterpret_cast<uint4*>(smem + K::kB + p * K::kPanel + r * 128 + q) = none;
                }
            }
            tc::fence_proxy_async();
            t.arrive(&bars->xs);
        }
        const float raw = t.raw_step(a, w, c + 1);                 // wanted further down
        // ---- Y = 2^G C S + D x; the product M X is added to it
        if constexpr (!ENDS) {
            t.wait(&bars->y_first, par);
            tc::tc_fence_after();
            const uint64_t gg = pack2(grow, grow), dd = pack2(D, D);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                uint32_t y[32];
                tc::tmem_ld32(t_y + 32 * half, y);
                tc::tmem_wait_ld();
                tc::pin32(y);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 raw_x = *reinterpret_cast<const uint4*>(x_row + (((4 * half + q) ^ (r & 7)) << 4));
                    const uint32_t xw[4] = {raw_x.x, raw_x.y, raw_x.z, raw_x.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        float f[2];
                        unpack_bf16(xw[z], f);
                        uint32_t* e = y + 8 * q + 2 * z;
                        const float2 v = unpack2(fma2(pack2(__uint_as_float(e[0]), __uint_as_float(e[1])), gg, mul2(pack2(f[0], f[1]), dd)));
                        e[0] = __float_as_uint(v.x);
                        e[1] = __float_as_uint(v.y);
                    }
                }
                tc::tmem_st32(t_y + 32 * half, y);
            }
            tc::tmem_wait_st();
            t.arrive(&bars->ready);
        }
        // ---- S = gamma S + dS
        const uint64_t gg = pack2(gamma, gamma);
        if (c + 1 < w.chunks && !steps(c + 1, raw)) return false;      // while the product runs
        if (PART == kIncrements) continue;
        t.wait(&bars->ds[par], (c >> 1) & 1);
        tc::tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t d[32];
            tc::tmem_ld32(t_ds + 32 * half, d);
            tc::tmem_wait_ld();
            tc::pin32(d);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float* e = &S[32 * half + i];
                const float2 v = unpack2(fma2(pack2(e[0], e[1]), gg, pack2(__uint_as_float(d[i]), __uint_as_float(d[i + 1]))));
                e[0] = v.x;
                e[1] = v.y;
            }
        }
        if (PART == kStates) t.arrive(&bars->next_y);              // dS has been read
        if constexpr (!ENDS) {
            store_s();                                             // (the product with the last S is done)
            t.arrive(&bars->next_s);
        }
    }
    if (ENDS && PART != kIncrements) {
        if (own) {
            float* to = plan.states + (w.seg.base + w.seg.k + 1) * all + tile;
#pragma unroll
            for (int i = 0; i < kSlice; ++i) to[(int64_t)i * a.N] = S[i];
        }
        if (r == 0 && t.channel == 0) plan.decays[(int64_t)(w.seg.base + w.seg.k + 1) * a.H + t.h] = all_steps;
    } else if (!ENDS && w.seg.k == w.seg.count - 1 && own) {
        float* to = a.pool + w.seg.slot * all + tile;
#pragma unroll
        for (int i = 0; i < kSlice; ++i) to[(int64_t)i * a.N] = S[i];
    }
    return !t.bad;
}

// The warpgroup of a slice's results: M and Y.
template <int N, typename TOut>
__device__ bool tc_results(const SsmCall& a, const TcWork& w, uint8_t* smem, TcThread t, const CUtensorMap* om)
{
    using K = TcCfg<N>;
    TcBars* bars = t.bars;
    const int s = t.s, r = t.r, warp = t.warp, lane = t.lane;
    const uint32_t t_gram = t.tmem + kGramCol, t_m = t.tmem + kMCol + 64 * s, t_y = t.tmem + kYCol + 64 * s;
    const uint32_t zero[16] = {};
    for (int b = warp + 1; b < 4; ++b) tc::tmem_st16u_nowait(t_m + 16 * b, zero);              // M above the diagonal stays zero
    tc::tmem_wait_st();

    float head = 0.f;                                              // steps of the block up to this row
    bool mild = false;                                             // the block's whole steps are no more than 60
    // prefix sums of a chunk's steps, and its columns' factors; false: a wait gave up
    auto steps = [&](int c, float raw) -> bool {
        const bool live = c * kChunk + r < w.seg.len;
        const float dt = live ? softplus_series(raw + t.bias, a.threshold) : 0.f;
        float tail = head = live ? bounded_step(-dt * t.rate) : 0.f;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float u = __shfl_up_sync(~0u, head, off), v = __shfl_down_sync(~0u, tail, off);
            if (lane >= off) head += u;
            if (lane + off < 32) tail += v;
        }
        if (lane == 31) bars->total[c & 1][s][warp] = head;
        tail = __shfl_down_sync(~0u, tail, 1);
        if (lane == 31) tail = 0.f;
        if (slice_any(t.id, t.bad)) return false;                  // all warps are through with the last chunk's M
        bars->col[s][r] = dt * exp2_fast(tail);
        // inside a block: with few steps two factors again, 2^head and dt_j 2^-head_j, neither past 2^64
        mild = __shfl_sync(~0u, head, 31) > -60.f;
        bars->diag[s][r] = mild ? dt * exp2_fast(-head) : __log2f(dt) - head;
        return true;
    };
    if (!steps(0, t.raw_step(a, w, 0))) return false;
    for (int c = 0; c < w.chunks; ++c) {
        const uint32_t par = c & 1;
        const int len = w.seg.len - c * kChunk < kChunk ? w.seg.len - c * kChunk : kChunk;
        uint8_t* x_row = smem + K::kX + (2 * s + par) * K::kPanel + r * 128;
        const float raw = t.raw_step(a, w, c + 1);                 // wanted behind M
        slice_sync(t.id);                                          // the columns' factors
        // ---- M
        t.wait(&bars->gram, par);
        tc::tc_fence_after();
        if (c > 0) {                                               // the last chunk's results are out of their X tile
            if (lane == 0) tc::bulk_wait_read();
            t.arrive(&bars->x_free[par ^ 1]);
        }
        uint32_t g[32], m[16];
        tc::tmem_ld32(t_gram + 32 * warp, g);
        tc::tmem_wait_ld();
        tc::pin32(g);
        const float* own = bars->diag[s] + 32 * warp;              // the diagonal block
        const float first = mild ? exp2_fast(head) : head;
        if (mild) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 e = *reinterpret_cast<const float4*>(own + i);
                m[i / 2] = pack_bf16(i > lane ? 0.f : e.x * first * __uint_as_float(g[i]), i + 1 > lane ? 0.f : e.y * first * __uint_as_float(g[i + 1]));
                m[i / 2 + 1] = pack_bf16(i + 2 > lane ? 0.f : e.z * first * __uint_as_float(g[i + 2]), i + 3 > lane ? 0.f : e.w * first * __uint_as_float(g[i + 3]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 e = *reinterpret_cast<const float4*>(own + i);
                m[i / 2] = pack_bf16(i > lane ? 0.f : exp2_fast(first + e.x) * __uint_as_float(g[i]), i + 1 > lane ? 0.f : exp2_fast(first + e.y) * __uint_as_float(g[i + 1]));
                m[i / 2 + 1] = pack_bf16(i + 2 > lane ? 0.f : exp2_fast(first + e.z) * __uint_as_float(g[i + 2]), i + 3 > lane ? 0.f : exp2_fast(first + e.w) * __uint_as_float(g[i + 3]));
            }
        }
        if (warp > 0) tc::tmem_ld32(t_gram + 32 * (warp - 1), g);
        tc::tmem_st16u_nowait(t_m + 16 * warp, m);
        float base = head;                                         // steps from the end of block b to this row
#pragma unroll 1
        for (int b = warp - 1; b >= 0; --b) {                      // the blocks before it: two factors, neither above dt
            if (b < warp - 1) base += bars->total[par][s][b + 1];
            const float row = exp2_fast(base);
            const uint64_t rr = pack2(row, row);
            const float* col = bars->col[s] + 32 * b;
            tc::tmem_wait_ld();
            tc::pin32(g);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(col + i);
                const float2 u = unpack2(mul2(mul2(e.x, rr), pack2(__uint_as_float(g[i]), __uint_as_float(g[i + 1]))));
                const float2 v = unpack2(mul2(mul2(e.y, rr), pack2(__uint_as_float(g[i + 2]), __uint_as_float(g[i + 3]))));
                m[i / 2] = pack_bf16(u.x, u.y);
                m[i / 2 + 1] = pack_bf16(v.x, v.y);
            }
            if (b > 0) tc::tmem_ld32(t_gram + 32 * (b - 1), g);
            tc::tmem_st16u_nowait(t_m + 16 * b, m);
        }
        tc::tmem_wait_st();
        t.arrive(&bars->ready);
        if (c + 1 < w.chunks && !steps(c + 1, raw)) return false;       // while the product runs
        // ---- results
        t.wait(&bars->y_full[par], (c >> 1) & 1);
        tc::tc_fence_after();
        // through the X tile's rows, which nobody needs any more, so that a warp writes whole lines
        constexpr int E = 16 / (int)sizeof(TOut);
        TOut* out = reinterpret_cast<TOut*>(a.out) + ((int64_t)(w.seg.first + c * kChunk + (r & 96)) * a.H + t.h) * a.P + t.channel + lane % 8 * E;
        const uint8_t* warp_rows = x_row - lane * 128;
        const int left = len - (r & 96);                           // rows of this warp that are the request's
        const bool whole = sizeof(TOut) == 2 && left >= 32;        // all rows of the warp: one tensor-map copy
        const bool odd = *(volatile int32_t*)&bars->odd[s] != 0;
#pragma unroll 1
        for (int part = 0; part < kSlice; part += 8 * E) {
            if (part) __syncwarp();
#pragma unroll
            for (int x = 0; x < 8 * E; x += 32) {
                uint32_t y[32];
                tc::tmem_ld32(t_y + part + x, y);
                tc::tmem_wait_ld();
                tc::pin32(y);
                if (odd) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (*(volatile int32_t*)&bars->odd_from[s][part + x + i] <= c * kChunk + r) y[i] = 0x7fc00000u;
                }
#pragma unroll
                for (int q = 0; q < 32 / E; ++q) {
                    float f[E];
#pragma unroll
                    for (int z = 0; z < E; ++z) f[z] = __uint_as_float(y[E * q + z]);
                    *reinterpret_cast<typename Vec<TOut, E>::Raw*>(x_row + (((x / E + q) ^ (r & 7)) << 4)) = from_floats<TOut, E>(f);
                }
            }
            if (whole) tc::fence_proxy_async();
            if (part + 8 * E >= kSlice) t.arrive(&bars->next_y);
            __syncwarp();
            if (whole) {
                if (lane == 0) {
                    tc::tma_store_2d(om, t.h * a.P + t.channel, w.seg.first + c * kChunk + (r & 96), warp_rows);
                    tc::bulk_commit();
                }
                continue;
            }
#pragma unroll 2
            for (int i = 0; i < 32; i += 4) {
                const int row = i + lane / 8;
                if (row < left)
                    *reinterpret_cast<uint4*>(out + (int64_t)row * a.H * a.P + part) =
                        *reinterpret_cast<const uint4*>(warp_rows + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            }
        }
        if (!whole) tc::fence_proxy_async();
    }
    if (lane == 0) tc::bulk_wait_read();                           // before the tile's memory goes
    return !t.bad;
}

// blockIdx.x: (segment, slice pair); one CTA more gives zeros to rows of no request.
template <int N, bool ENDS, typename TOut>
__global__ void __launch_bounds__(kTcThreads, 1)
    ssm_chunk_kernel(const SsmCall a, const Plan plan, const __grid_constant__ CUtensorMap xm, const __grid_constant__ CUtensorMap bm,
                     const __grid_constant__ CUtensorMap cm, const __grid_constant__ CUtensorMap om)
{
    using K = TcCfg<N>;
    extern __shared__ __align__(1024) uint8_t smem[];
    TcBars* bars = reinterpret_cast<TcBars*>(smem + K::kEnd);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t place = blockIdx.x / plan.pairs;
    const int32_t pair = blockIdx.x % plan.pairs;
    TOut* out = reinterpret_cast<TOut*>(a.out);
    // launched while the kernel before it runs; all wait for it, so that who waits for this one waits for that one too
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (ENDS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!ENDS && blockIdx.x == gridDim.x - 1) {
        if (a.short_len == 0) ssm_clear_unowned<TOut>(a, tid, kTcThreads);
        return;
    }
    if (place >= plan.found[ENDS ? 1 : 0]) return;
    if (ENDS) place = plan.followed[place];
    TcWork w;
    w.seg = plan.segments[place];
    const int per_head = a.P / kSlice, hpg = a.H / a.G;
    w.g = pair / plan.pairs_per_group;
    w.first = (pair % plan.pairs_per_group) * 2;
    w.halves = per_head - 1;
    w.head0 = w.g * hpg;
    w.slices = hpg * per_head - w.first < 2 ? 1 : 2;
    w.chunks = (w.seg.len + kChunk - 1) / kChunk;
    if (w.seg.slot < 0) {                                         // padding
        for (int s = 0; s < w.slices; ++s)
            for (int64_t i = tid; i < (int64_t)w.seg.len * kSlice; i += kTcThreads)
                out[((w.seg.first + i / kSlice) * a.H + w.head(s)) * a.P + w.channel(s) + i % kSlice] = from_f32<TOut>(0.f);
        return;
    }
    if (tc::smem_u32(smem) & 1023u) {                             // the swizzled tiles want whole kilobytes
        if (tid == 0) record_layer_error(kDevErrTimeout);
        return;
    }
    if (warp == 0) {
        if (lane == 0) {
            for (uint64_t* bar = &bars->full_c; bar <= &bars->drain; ++bar) tc::mbar_init(bar, 1);
            for (uint64_t* bar = &bars->next_s; bar <= &bars->x_free[1]; ++bar) tc::mbar_init(bar, (bar == &bars->ready ? 8 : 4) * w.slices);
            tc::fence_mbar_init();
        }
    } else if (warp == 1) {
        for (int i = lane; i < 2 * kSlice; i += 32) bars->odd_from[0][i] = 0x7fffffff;
        if (lane < 2) bars->odd[lane] = 0;
    } else if (warp == 16) {
        tc::tmem_alloc(&bars->tmem, 512);
        tc::tmem_relinquish();
    }
    if constexpr (N < 128) {                                      // the states that are not there: zero rows of dS
        for (int i = tid; i < K::kPanel / 16; i += kTcThreads) {
            reinterpret_cast<uint4*>(smem + K::kB + K::kPanel)[i] = make_uint4(0, 0, 0, 0);
            if (ENDS) reinterpret_cast<uint4*>(smem + K::kC + K::kPanel)[i] = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bars->tmem;
    bool ok = true;
    if (warp < 8) {
        fewer_registers<kResultRegs>();
        const int s = warp / 4;
        if (s < w.slices) {
            const TcThread t(a, w, bars, tmem, s, tid & 127, 1 + s);
            if constexpr (ENDS) ok = tc_state<N, true, kIncrements>(a, plan, w, smem, t);
            else ok = tc_results<N, TOut>(a, w, smem, t, &om);
        }
    } else if (warp < 16) {
        more_registers<kStateRegs>();
        const int s = warp / 4 - 2;
        if (s < w.slices) ok = tc_state<N, ENDS, ENDS ? kStates : kBoth>(a, plan, w, smem, TcThread(a, w, bars, tmem, s, tid & 127, 3 + s));
    } else {
        fewer_registers<kOtherRegs>();
        if (warp == 16) {
            uint32_t leader = 0;
            asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
            ok = w.slices == 2 ? tc_issue<N, ENDS, 2>(w.chunks, tc::smem_u32(smem), bars, tmem, leader) : tc_issue<N, ENDS, 1>(w.chunks, tc::smem_u32(smem), bars, tmem, leader);
            if (leader) tc::mma_commit(&bars->drain);             // everything issued ends before the exit
            __syncwarp();
            ok = tc::mbar_wait(&bars->drain, 0, kPolls) && ok;
        } else if (lane == 0 && warp == 17) {
            ok = tc_load<N, ENDS>(a, w, smem, bars, &xm, &bm, &cm);
            if (!ok) {                                             // and the copies in flight land
                for (uint32_t p = 0; p < 2; ++p) {
                    tc::mbar_wait(&bars->full_c, p, 1u << 16);
                    tc::mbar_wait(&bars->full_b[0], p, 1u << 16);
                    tc::mbar_wait(&bars->full_b[1], p, 1u << 16);
                    tc::mbar_wait(&bars->full_x[0], p, 1u << 16);
                    tc::mbar_wait(&bars->full_x[1], p, 1u << 16);
                }
            }
        }
    }
    if (!ok) record_layer_error(kDevErrTimeout);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    __syncwarp();
    if (warp == 16) tc::tmem_dealloc(tmem, 512);
}

}  // namespace ssm

namespace {

cudaError_t ssm_map(CUtensorMap* m, const void* base, int64_t rows, int64_t width, int64_t stride, int box_rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tc::tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// B or C as [tokens][groups][states], in boxes of 64 states of a group; states that are not there read as zeros.
cudaError_t ssm_group_map(CUtensorMap* m, const void* base, int64_t rows, int64_t groups, int64_t states, int64_t stride)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tc::tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)states, (cuuint64_t)groups, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)states * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)ssm::kChunk};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The kernel with its shared memory, if it was built with the registers that its groups share out.
template <int N, bool ENDS, typename TOut>
cudaError_t ssm_chunk_ready()
{
    const auto kernel = ssm::ssm_chunk_kernel<N, ENDS, TOut>;
    static std::atomic<int> registers;
    if (registers.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
        if (e != cudaSuccess) return e;
        registers.store(f.numRegs, std::memory_order_relaxed);
    }
    if (registers.load(std::memory_order_relaxed) != ssm::kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ssm::TcCfg<N>::kSmem);
}

template <int N, typename TOut>
cudaError_t ssm_tc_launch(const kda_ssm_params& p, SsmCall a, void* workspace, cudaStream_t s)
{
    SsmLayout w = ssm_layout(p, a.n, a.T);
    a.short_len = w.short_len;
    w.place(workspace);
    cudaError_t e = cudaSuccess;
    if (w.short_len) e = ssm_dispatch<false>(p, a, nullptr, s);
    if (e != cudaSuccess || w.plan.max_segments == 0) return e;
    CUtensorMap xm, bm, cm, om = {};
    e = ssm_map(&xm, a.x, a.T, (int64_t)a.H * a.P, a.x_stride, ssm::kChunk);
    if (e == cudaSuccess) e = ssm_group_map(&bm, a.B, a.T, a.G, a.N, a.b_stride);
    if (e == cudaSuccess) e = ssm_group_map(&cm, a.C, a.T, a.G, a.N, a.c_stride);
    if (e == cudaSuccess && sizeof(TOut) == 2) e = ssm_map(&om, a.out, a.T, (int64_t)a.H * a.P, (int64_t)a.H * a.P, 32);
    if (e != cudaSuccess) return e;
    constexpr int smem = ssm::TcCfg<N>::kSmem;
    ssm::ssm_plan_kernel<<<1, 1024, 0, s>>>(a, w.plan);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;                                // without its plan a workspace holds anything
    if (w.cut) {
        e = ssm_chunk_ready<N, true, TOut>();
        if (e == cudaSuccess) e = launch_after(ssm::ssm_chunk_kernel<N, true, TOut>, (int64_t)w.plan.max_cuts * w.plan.pairs, ssm::kTcThreads, smem, s, a, w.plan, xm, bm, cm, om);
        // a request in several segments has two at least
        if (e == cudaSuccess) e = launch_after(ssm::ssm_chain_kernel, (int64_t)(w.plan.max_cuts / 2 + 1) * a.H * ((a.P * a.N + 1023) / 1024), 256, 0, s, a, w.plan);
    }
    if (e == cudaSuccess) e = ssm_chunk_ready<N, false, TOut>();
    if (e != cudaSuccess) return e;
    return launch_after(ssm::ssm_chunk_kernel<N, false, TOut>, (int64_t)w.plan.max_segments * w.plan.pairs + 1, ssm::kTcThreads, smem, s, a, w.plan, xm, bm, cm, om);
}

}  // namespace

size_t ssm_workspace_bytes(const kda_ssm_params& p, int32_t num_seqs, int64_t total_tokens) { return ssm_layout(p, num_seqs, total_tokens).total; }

cudaError_t launch_ssm_prefill(const kda_ssm_params& p, const SsmCall& a, void* workspace, cudaStream_t s)
{
    if (!ssm_on_tensor_cores(p)) {
        SsmLayout w = ssm_layout(p, a.n, a.T);
        if (!w.cut) return ssm_dispatch<false>(p, a, nullptr, s);
        w.place(workspace);
        ssm::ssm_plan_kernel<<<1, 1024, 0, s>>>(a, w.plan);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess ? e : ssm_dispatch<false>(p, a, &w.plan, s);
    }
    if (p.state_dim <= 64)
        return p.out_dtype == KDA_BF16 ? ssm_tc_launch<64, __nv_bfloat16>(p, a, workspace, s) : ssm_tc_launch<64, float>(p, a, workspace, s);
    return p.out_dtype == KDA_BF16 ? ssm_tc_launch<128, __nv_bfloat16>(p, a, workspace, s) : ssm_tc_launch<128, float>(p, a, workspace, s);
}

}  // namespace kda
