// kda_attn_tc.cu -- attention of new tokens over the paged cache for many query rows (prompts, wide
// verifies): tcgen05 matrix products with the scores, the weights and the outputs in tensor memory.
//
// A kv head serves R = new tokens * G query rows, row = token * G + head of the group, so that the heads of
// a group share every key and value tile.  A CTA takes 256 rows as two tiles of 128 and walks the cache
// tokens that any of them may see in tiles of 128:
//
//   S_i = Q_i K_j^T      M 128 (rows) x N 128 (tokens) x K D, both operands K-major in shared memory
//   P_i = exp2(S_i - m)  one thread per row: no shuffles; packed in bf16 over half of S_i's own columns (half a
//                        step, 2^-8 of a weight at most, for one operand type with the values; the sum of the
//                        weights takes them unrounded)
//   O_i += P_i V_j       A from tensor memory, V_j as it lies in the cache (MN-major)
//
// Tensor memory, all 512 columns: S_0, S_1 (128 each; P_i takes the last 64 of S_i's) and O_0, O_1 (D each).
// Roles: warps 0-3 and 4-7 are the softmax of row tile 0 and 1, warp 8 issues the products,
// the warps after it fill a ring of key and value tiles (128 tokens x D, 128-byte swizzle).  The products go
// PV_0(j), S_0(j+1), PV_1(j), S_1(j+1), so that each softmax works while the other tile's products run.
//   bf16 cache: one warp, a lane per page, two tensor-map copies (64 channels each) per page and tile;
//   4-bit cache: seven warps convert on the way into shared memory, exactly: keys to fp16 (one instruction a
//   pair; the queries are fp16 then, each row divided by a power of two), values to bf16, whose range the
//   weights need.
// A rescaling of O happens only when a row's maximum grows by more than 2^8 since the last one; the S_i(j)
// barrier implies that PV_i(j-1) is complete, so the softmax warps do it themselves.
//
// Value rows of tokens that no row of the CTA may see (the ends of the cache and of a window) are zeroed in
// shared memory before their product, by a warp of its own: what lies there may be NaN, which a weight of
// zero does not stop.
//
// Measured (8 kv and 32 query heads of 128): 4,096 tokens over 32,768 in 1.52 ms, 1,360 TFLOP/s, bound by the
// chain scores - softmax - products of a tile, some 3,000 cycles where the products alone take 2,080; eight
// prompts of 512 to 4,096 tokens through a window of 1,024 in 0.34 ms, a third of it a CTA's start and end;
// 4 x 500..1,030 tokens over a 4-bit past of 2,000..9,000 in 0.37 ms, bound by the conversion.  Shared memory is
// the busiest unit beside the tensor cores: a product of 128 x 128 x 16 reads 8 KB of it in 64 cycles.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "kda_attn.cuh"
#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

__device__ int32_t g_attn_tc_error = 0;

using attn::Parts;
using attn::Span;

constexpr int kRows = 256;            // query rows of a CTA
constexpr int kTile = 128;            // cache tokens of a tile
constexpr uint32_t kPolls = 1u << 24;
constexpr float kSlack = 8.0f;        // growth of a maximum, in log2, that is let pass

template <int D, bool FP4>
struct Cfg {
    static constexpr int kFillThreads = FP4 ? 224 : 32;
    static constexpr int kThreads = FP4 ? 512 : 384;
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr int kPanel = kTile * 128;               // 64 channels of 128 rows
    static constexpr int kSmem = 2 * kTileBytes + kSlots * kTileBytes + 1024 /* alignment */ + 320 /* barriers */;
};

// A row tile: its request, that request's rows and length, and the tile's first row.
struct Tile {
    int32_t found, b, row0, len;
    int64_t t0, t1;
};

struct __align__(8) Bars {
    uint64_t full[8], empty[8];
    uint64_t q_full[2], s_full[2], p_ready[2][2], o_full[2];
    uint64_t drain;
    uint64_t patch[4];                // arrival of the value tiles that are mended before use
    uint32_t tmem;
    Tile tile;                        // the CTA's
};
static_assert(sizeof(Bars) <= 320, "barrier block");

// Matrix descriptor of a 128-byte-swizzled operand: 8 rows of 128 bytes make an atom, `sbo` the distance of
// atoms along the strided dimension, `lbo` (MN-major only) that of 64-element panels.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
template <bool FP16>
__host__ __device__ constexpr uint32_t idesc(uint32_t N, bool b_mn)
{
    return (1u << 4) | (FP16 ? 0u : 1u << 7 | 1u << 10) | (b_mn ? 1u << 16 : 0u) | (N >> 3) << 17 | (128u >> 4) << 24;
}

#define KDA_X8(p, i) p(r[i]), p(r[i + 1]), p(r[i + 2]), p(r[i + 3]), p(r[i + 4]), p(r[i + 5]), p(r[i + 6]), p(r[i + 7])
#define KDA_OUT(x) "=r"(x)
#define KDA_IN(x) "r"(x)
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : KDA_X8(KDA_OUT, 0), KDA_X8(KDA_OUT, 8), KDA_X8(KDA_OUT, 16), KDA_X8(KDA_OUT, 24)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        KDA_X8(KDA_IN, 0), KDA_X8(KDA_IN, 8), KDA_X8(KDA_IN, 16), KDA_X8(KDA_IN, 24)
        : "memory");
}
// Waits for the loads; the empty statements keep every use of their registers after the wait.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
#define KDA_BOTH(x) "+r"(x)
__device__ __forceinline__ void pin32(uint32_t* r)
{
    asm volatile("" : KDA_X8(KDA_BOTH, 0), KDA_X8(KDA_BOTH, 8), KDA_X8(KDA_BOTH, 16), KDA_X8(KDA_BOTH, 24)::"memory");
}
#undef KDA_X8
#undef KDA_OUT
#undef KDA_IN
#undef KDA_BOTH
// Whether the phase with the given parity is complete, without waiting (try_wait may suspend the thread).
__device__ __forceinline__ bool bar_test(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A warp's wait with one lane polling: 32 lanes on one barrier are 32 accesses, and they slow every other
// barrier operation of the SM down.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int lane)
{
    bool ok = true;
    if (lane == 0) ok = tc::mbar_wait(bar, parity, kPolls);
    return __all_sync(~0u, ok);
}

// Row tile x among all row tiles of the batch (found = 0 past the last one), by one warp: a lane per request.
// The grid holds the tiles of `max_new` tokens a request: one that brings more has its further tiles left out, so
// that the other requests keep theirs.
__device__ __forceinline__ Tile find_rows(const kv::Paged& c, int64_t x, int32_t max_new, int lane)
{
    for (int base = 0; base < c.n; base += 32) {
        int64_t t0 = 0, t1 = 0;
        int len = 0;
        if (base + lane < c.n) {
            len = c.lens[base + lane];
            kv::request_rows(c, base + lane, t0, t1);
        }
        const int64_t tiles = (min(t1 - t0, (int64_t)max_new) * c.G + kRows - 1) / kRows;
        int64_t sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, sum, d);
            if (lane >= d) sum += y;
        }
        const unsigned hit = __ballot_sync(~0u, x < sum);
        if (hit) {
            const int who = __ffs(hit) - 1;
            const int64_t before = __shfl_sync(~0u, sum - tiles, who), mine = __shfl_sync(~0u, tiles, who);
            Tile r;
            r.found = 1;
            r.b = base + who;
            r.row0 = (int32_t)((mine - 1 - (x - before)) * kRows);   // a request's last rows, which see most, first
            r.len = __shfl_sync(~0u, len, who);
            r.t0 = __shfl_sync(~0u, t0, who);
            r.t1 = __shfl_sync(~0u, t1, who);
            return r;
        }
        x -= __shfl_sync(~0u, sum, 31);
    }
    Tile none = {};
    return none;
}

struct Work {
    int b, h, nq, tile_lo, tile_hi;
    int64_t t0;
    int32_t R, row0;               // rows of (request, head), first row of this CTA
    int first;                     // position of the request's first new token
    Span sp;
};

// ---- filling the ring --------------------------------------------------------------------------------
__device__ __forceinline__ bool seen_by_any(const Span& sp, int j) { return j < sp.hi && (j >= sp.lo || j < sp.sink_end); }
__device__ __forceinline__ bool page_needed(const Span& sp, int j, int page) { return j < sp.hi && (j + page > sp.lo || j < sp.sink_end); }

// A value tile with rows that nobody may see: what lies there is not known, and a weight of zero does not
// stop a NaN.  Such tiles are at the end of the sinks, the start of the window and the end of the cache.
__device__ __forceinline__ bool needs_mending(const Span& sp, int base)
{
    return base + kTile > sp.hi || (base < sp.lo && base + kTile > sp.sink_end);
}

template <int D>
__device__ bool fill_bf16(const AttnCall& a, const Work& w, const CUtensorMap* km, const CUtensorMap* vm, uint8_t* ring, Bars* bars, int lane)
{
    using C = Cfg<D, false>;
    const int shift = a.c.page_shift, page = 1 << shift, per_tile = kTile >> shift;
    int idx = 0, mended = 0;
    for (int i = w.tile_lo; i < w.tile_hi; ++i) {
        const int base = attn::tile_base<kTile>(w.sp, i), j = base + lane * page;
        int64_t row = -1;
        if (lane < per_tile && page_needed(w.sp, j, page)) {
            row = kv::token_slot(a.c, w.b, j);
            if (row >= 0) row += (int64_t)w.h << shift;
        }
        const uint32_t bytes = __popc(__ballot_sync(~0u, row >= 0)) * (uint32_t)(page * D * 2);
#pragma unroll
        for (int which = 0; which < 2; ++which, ++idx) {
            const int slot = idx % C::kSlots;
            uint8_t* dst = ring + slot * C::kTileBytes + lane * page * 128;
            if (!warp_wait(&bars->empty[slot], ((idx / C::kSlots) & 1) ^ 1, lane)) return false;
            uint64_t* bar = which && needs_mending(w.sp, base) ? &bars->patch[mended++] : &bars->full[slot];
            if (lane == 0) tc::mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (row >= 0) {
#pragma unroll
                for (int p = 0; p < D / 64; ++p)
                    tc::tma_load_2d(dst + p * C::kPanel, which ? vm : km, p * 64, (int32_t)row, bar);
            }
        }
    }
    return true;
}

// One warp beside fill_bf16: value tiles that need it get zeros in their unseen rows before they count as full.
template <int D>
__device__ bool mend_bf16(const Work& w, uint8_t* ring, Bars* bars, int lane)
{
    using C = Cfg<D, false>;
    int mended = 0;
    for (int i = w.tile_lo; i < w.tile_hi; ++i) {
        const int base = attn::tile_base<kTile>(w.sp, i), slot = (2 * (i - w.tile_lo) + 1) % C::kSlots;
        if (!needs_mending(w.sp, base)) continue;
        if (!warp_wait(&bars->patch[mended++], 0, lane)) return false;
        uint8_t* vt = ring + slot * C::kTileBytes;
        for (int r = lane; r < kTile; r += 32) {
            if (seen_by_any(w.sp, base + r)) continue;
#pragma unroll
            for (int p = 0; p < D / 64; ++p)
#pragma unroll
                for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(vt + p * C::kPanel + r * 128 + x * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->full[slot]);
    }
    return true;
}

// 4-bit pages: the loads of the next tile are in flight while one is converted.
template <int D>
__device__ bool fill_fp4(const AttnCall& a, const Work& w, uint8_t* ring, Bars* bars, int tid)
{
    using C = Cfg<D, true>;
    constexpr int kUnits = D / 32, kAll = kTile * kUnits;                  // 32-channel units of a row, of a tile
    constexpr int kPer = (kAll + C::kFillThreads - 1) / C::kFillThreads;
    const int shift = a.c.page_shift, page = 1 << shift, total = 2 * (w.tile_hi - w.tile_lo), lane = tid & 31;
    uint4 x[kPer], nx[kPer];
    uint32_t s[kPer], ns[kPer];
    // a lane's page of a tile: the cache row it starts at (rows are below 2^31), -1 where nobody looks
    const auto page_of = [&](int i) {
        const int j = attn::tile_base<kTile>(w.sp, i) + lane * page;
        if (lane >= kTile >> shift || !page_needed(w.sp, j, page)) return -1;
        const int64_t row = kv::token_slot(a.c, w.b, j);
        return row < 0 ? -1 : (int32_t)(row + ((int64_t)w.h << shift));
    };
    int32_t here = page_of(w.tile_lo), ahead = -1;
    const auto load = [&](int idx, int32_t pages, uint4* data, uint32_t* scale) {
        const int base = attn::tile_base<kTile>(w.sp, w.tile_lo + (idx >> 1));
        const uint8_t* src = idx & 1 ? a.c.v : a.c.k;
        const uint8_t* scl = idx & 1 ? a.c.vs : a.c.ks;
#pragma unroll
        for (int n = 0; n < kPer; ++n) {
            const int at = tid + C::kFillThreads * n, r = at / kUnits, u = at % kUnits;
            const int32_t row = __shfl_sync(~0u, pages, (r & (kTile - 1)) >> shift);
            data[n] = make_uint4(0, 0, 0, 0);                               // zeros where nobody looks
            scale[n] = 0;
            if (at < kAll && row >= 0 && seen_by_any(w.sp, base + r)) {
                const int64_t t = row + (r & (page - 1));
                data[n] = __ldg(reinterpret_cast<const uint4*>(src + t * (D / 2) + u * 16));
                scale[n] = __ldg(reinterpret_cast<const uint16_t*>(scl + t * (D / 16) + u * 2));
            }
        }
    };
    load(0, here, x, s);
    int slot = 0;
    uint32_t parity = 1;
    for (int idx = 0; idx < total; ++idx) {
        if (!(idx & 1)) {
            load(idx + 1, here, nx, ns);                                    // the tile's values; its successor's pages
            if (idx + 2 < total) ahead = page_of(w.tile_lo + (idx >> 1) + 1);
        } else if (idx + 1 < total) {
            here = ahead;
            load(idx + 1, here, nx, ns);
        }
        uint8_t* dst = ring + slot * C::kTileBytes;
        if (!warp_wait(&bars->empty[slot], parity, lane)) return false;
#pragma unroll
        for (int n = 0; n < kPer; ++n) {
            const int at = tid + C::kFillThreads * n, r = at / kUnits, u = at % kUnits;
            if (at >= kAll) break;
            const uint32_t f = kv::e4m3x2_to_f16x2(s[n]);
            const uint32_t f0 = __byte_perm(f, 0, 0x1010), f1 = __byte_perm(f, 0, 0x3232);
            const uint32_t wd[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t y[4];
                kv::e2m1x8_to_f16(wd[q], y);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    y[z] = kv::mul_f16x2(y[z], q < 2 ? f0 : f1);
                    if (idx & 1) {                                          // at most 6 significant bits: exact in bf16 too
                        const float2 g = kv::f16x2_to_f32(y[z]);
                        y[z] = kv::f32_to_bf16x2(g.x, g.y);
                    }
                }
                const int chunk = (u * 4 + q) & 7, panel = (u * 4 + q) >> 3;
                *reinterpret_cast<uint4*>(dst + panel * C::kPanel + r * 128 + ((chunk ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->full[slot]);
        if (++slot == C::kSlots) slot = 0, parity ^= 1;
#pragma unroll
        for (int n = 0; n < kPer; ++n) x[n] = nx[n], s[n] = ns[n];
    }
    return true;
}

// ---- issuing the products ------------------------------------------------------------------------------------
// The tensor cores' queue is a few products deep, a wait costs its warp some 190 cycles even when there is
// nothing to wait for, and a commit 110.  So each barrier is first looked at (Peek) while products are still
// being issued and waited for only if it was not complete then, and the only commits are those of the scores:
// that a tile's scores are complete tells its softmax that the keys and the last values are free, and it says
// so.  The warp runs as one with bounds made uniform and both row tiles written out, so that the descriptors
// are uniform registers; only the products themselves are one lane's.  (A warp per row tile hides the same
// waits, but the tiles fall into step and the tensor cores idle while both softmaxes run: 2,178 us for the
// 4,096-token call.)
struct Peek {
    uint64_t* bar;
    uint32_t parity;
    bool done;
    __device__ __forceinline__ void look(uint64_t* b, uint32_t p) { bar = b, parity = p, done = bar_test(b, p); }
    __device__ __forceinline__ bool wait() const { return __all_sync(~0u, done) || __all_sync(~0u, tc::mbar_wait(bar, parity, kPolls)); }
};

template <int D, bool FP4, int NQ>
__device__ bool issue(const int n_, const uint8_t* q, uint8_t* ring, Bars* bars, const uint32_t tmem_, const bool leader)
{
    const int n = (int)__reduce_max_sync(~0u, (unsigned)n_);
    const uint32_t tmem = __reduce_max_sync(~0u, tmem_);
    using C = Cfg<D, FP4>;
    constexpr uint32_t id_s = idesc<FP4>(kTile, false), id_o = idesc<false>(D, true);
    constexpr uint32_t kStep = C::kTileBytes >> 4;                          // descriptors count in units of 16 bytes
    const uint64_t dq = desc_sw128(tc::smem_u32(q), 16, 1024);
    const uint64_t dk = desc_sw128(tc::smem_u32(ring), 16, 1024), dv = desc_sw128(tc::smem_u32(ring), C::kPanel, 1024);
    Peek vals, keys, part;
    int ks = 0, vs = 1;                                                     // slots of the keys and the values, and
    uint32_t kp = 0, vp = 0;                                                // the parities of their filling
    const auto next = [](int& slot, uint32_t& parity) {
        slot += 2;
        if (slot >= C::kSlots) slot -= C::kSlots, parity ^= 1;
    };
    // S_i from the keys in slot ks; the next weights to come are looked at before its end
    const auto scores = [&](const int i, const int next_i, uint32_t next_parity) {
        const uint64_t b = dk + (uint32_t)ks * kStep;
        if (leader) {
#pragma unroll
            for (int s = 0; s < D / 16 - 2; ++s) {
                const uint32_t off = ((s / 4) * C::kPanel + (s % 4) * 32) >> 4;
                tc::mma_f16_ss(tmem + 128 * i, dq + (i * kStep + off), b + off, id_s, s > 0);
            }
        }
        part.look(&bars->p_ready[next_i][1], next_parity);
        if (leader) {
#pragma unroll
            for (int s = D / 16 - 2; s < D / 16; ++s) {
                const uint32_t off = ((s / 4) * C::kPanel + (s % 4) * 32) >> 4;
                tc::mma_f16_ss(tmem + 128 * i, dq + (i * kStep + off), b + off, id_s, s > 0);
            }
            tc::mma_commit(&bars->s_full[i]);
        }
    };
    if (!tc::mbar_wait(&bars->full[0], 0, kPolls)) return false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        if (!tc::mbar_wait(&bars->q_full[i], 0, kPolls)) return false;
        scores(i, 0, 0);
    }
    next(ks, kp);
    vals.look(&bars->full[vs], vp);
    if (n > 1) keys.look(&bars->full[ks], kp);
    for (int j = 0; j < n; ++j) {
        const bool more = j + 1 < n;
        const uint64_t b = dv + (uint32_t)vs * kStep;
        if (!vals.wait()) return false;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            constexpr int kLast = NQ - 1;
#pragma unroll
            for (int half = 1; half >= 0; --half) {                        // the softmax hands over the high half first
                if (!part.wait()) return false;
                tc::tc_fence_after();
                if (half == 1) part.look(&bars->p_ready[i][0], j & 1);
                else if (i < kLast && !more) part.look(&bars->p_ready[kLast][1], j & 1);
                if (leader) {
#pragma unroll
                for (int s = 4 * half; s < 4 * half + 4; ++s)
                    tc::mma_f16_ts(tmem + 256 + D * i, tmem + 128 * i + 64 + 8 * s, b + (s * 2048 >> 4), id_o, s != 4 ? 1u : (uint32_t)j);
                }
            }
            if (more) {
                if (i == 0 && !keys.wait()) return false;
                if (i == kLast) {
                    next(vs, vp);
                    vals.look(&bars->full[vs], vp);
                }
                scores(i, i == kLast ? 0 : kLast, (i == kLast ? j + 1 : j) & 1);
                if (i == kLast) {
                    next(ks, kp);
                    if (j + 2 < n) keys.look(&bars->full[ks], kp);
                }
            } else if (leader) {
                tc::mma_commit(&bars->o_full[i]);
            }
        }
    }
    return true;
}

// ---- one thread per query row ------------------------------------------------------------------------------
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
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// A warp loads its 32 query rows of tile i into their swizzled places, D / 8 lanes to a row; returns the
// factor from scores to log2 of the lane's own row.  `own_at`: where the lane's own row starts, in elements,
// -1 past the last row; the lanes of a warp tell each other theirs.
template <int D, bool FP4>
__device__ __forceinline__ float load_queries(const AttnCall& a, uint8_t* q, int i, int tid, int64_t own_at)
{
    using C = Cfg<D, FP4>;
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;                    // lanes of a row, rows of a load
    const int lane = tid & 31, chunk = lane % kLanes;
    float unit = a.scale * attn::kLog2e;
    uint8_t* tile = q + i * C::kTileBytes + (tid & 96) * 128 + (chunk >> 3) * C::kPanel;
    const uint16_t* base = reinterpret_cast<const uint16_t*>(a.q) + 8 * chunk;
    if constexpr (!FP4) {
#pragma unroll 2
        for (int x = 0; x < 32; x += kAtOnce) {
            const int r = x + lane / kLanes;
            const int64_t at = __shfl_sync(~0u, own_at, r);
            // 16 bytes, or zeros for a row past the last
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(tile + r * 128 + (((chunk & 7) ^ (r & 7)) << 4))),
                         "l"(base + (at < 0 ? 0 : at)), "r"(at < 0 ? 0 : 16)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        return unit;
    }
    constexpr int kBatch = 8;
#pragma unroll 1
    for (int x0 = 0; x0 < 32 / kAtOnce; x0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t at = __shfl_sync(~0u, own_at, (x0 + b) * kAtOnce + lane / kLanes);
            v[b] = make_uint4(0, 0, 0, 0);
            if (at >= 0) v[b] = *reinterpret_cast<const uint4*>(base + at);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = (x0 + b) * kAtOnce + lane / kLanes;
            if constexpr (FP4) {
                // fp16 operands: the row is divided by a power of two near its largest magnitude (see the few-rows form)
                uint32_t y[4] = {v[b].x, v[b].y, v[b].z, v[b].w}, top = 0;
#pragma unroll
                for (int z = 0; z < 4; ++z) top = max(top, max(y[z] & 0x7fffu, (y[z] >> 16) & 0x7fffu));
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
                const int e = min(max((int)(top >> 7), a.min_exp), 253);
                const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float2 f = kv::bf16x2_to_f32(y[z]);
                    y[z] = kv::f32_to_f16x2(f.x * down, f.y * down);
                }
                v[b] = make_uint4(y[0], y[1], y[2], y[3]);
                // the lane whose row this is takes the factor
                const float mine = __shfl_sync(~0u, up, lane % kAtOnce * kLanes);
                if (lane / kAtOnce == x0 + b) unit *= mine;
            }
            *reinterpret_cast<uint4*>(tile + r * 128 + (((chunk & 7) ^ (r & 7)) << 4)) = v[b];
        }
    }
    return unit;
}

template <int D, bool FP4>
__device__ bool softmax(const AttnCall& a, const Parts& parts, const Work& w, int parts_here, int part, uint8_t* q, Bars* bars, uint32_t tmem,
                        int i, int tid)
{
    using C = Cfg<D, FP4>;
    const int row = w.row0 + 128 * i + tid, lane = tid & 31;
    const bool live = row < w.R;
    const int token = a.token_of(row), head = w.h * a.c.G + row - token * a.c.G;
    const float unit = load_queries<D, FP4>(a, q, i, tid, live ? (w.t0 + token) * a.q_stride + (int64_t)head * D : -1);
    tc::fence_proxy_async();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bars->q_full[i]);

    const uint32_t lanes = (uint32_t)(tid & 96) << 16;                  // the warp's 32 tensor-memory lanes
    const uint32_t ts = tmem + 128 * i + lanes, to = tmem + 256 + D * i + lanes;
    const int p = w.first + token;
    const int p_lo = w.first + a.token_of(w.row0 + 128 * i);                // of the tile's first and last row
    const int p_hi = w.first + a.token_of(min(w.R - 1, w.row0 + 128 * i + 127));
    const int n = w.tile_hi - w.tile_lo;
    float m = -INFINITY;
    uint64_t l2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
    int key_slot = 0;
    for (int j = 0; j < n; ++j) {
        const int base = attn::tile_base<kTile>(w.sp, w.tile_lo + j);
        if (!warp_wait(&bars->s_full[i], j & 1, lane)) return false;
        tc::tc_fence_after();
        const bool whole = base + kTile <= w.sp.hi && base + kTile - 1 <= p_lo && (a.window == 0 || base > p_hi - a.window || base + kTile <= a.sinks);
        // A tile that some row sees only in part is masked where it lies, in a short loop, and then goes the way of
        // all others: code that runs once or twice in a work is fetched anew each time, at some 200 cycles for
        // eight instructions, and a masking copy of what follows took 5,000 cycles.
        if (!whole) {
#pragma unroll 1
            for (int x = 0; x < 128; x += 32) {
                uint32_t s[32];
                tmem_ld32(ts + x, s);
                tmem_wait_ld();
                pin32(s);
                // visible columns: those below `end` that are from `from` on or below `sink`
                const int c = base + x;
                const uint32_t on = low_bits(min(p + 1, w.sp.hi) - c) & ((a.window ? ~low_bits(p - a.window + 1 - c) : ~0u) | low_bits(a.sinks - c));
#pragma unroll
                for (int z = 0; z < 32; ++z)
                    if (!(on & (1u << z))) s[z] = 0xff800000u;
                tmem_st32(ts + x, s);
            }
            tc::tmem_wait_st();
        }
        // Half a row of scores at a time: the low half for its maximum, then the high half, whose weights are
        // taken and handed over first, then the low half again: 64 scores and 32 packed weights at a time.  28 to 88
        // bytes a thread still spill (by the variant); with 128 scores at a time the calls were slower.
        float top = -INFINITY;
#pragma unroll
        for (int step = 0; step < 3; ++step) {
            const int half = step & 1;
            uint32_t s[64];
            tmem_ld32(ts + 64 * half, s);
            tmem_ld32(ts + 64 * half + 32, s + 32);
            tmem_wait_ld();
            pin32(s);
            pin32(s + 32);
            if (step < 2) {
                float t4[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) t4[z] = fmaxf(__uint_as_float(s[2 * z]), __uint_as_float(s[2 * z + 1]));
#pragma unroll
                for (int x = 8; x < 64; x += 8)
#pragma unroll
                    for (int z = 0; z < 4; ++z) t4[z] = max3(t4[z], __uint_as_float(s[x + 2 * z]), __uint_as_float(s[x + 2 * z + 1]));
                top = max3(top, fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                if (step == 0) continue;
                top *= unit;
                if (__any_sync(~0u, top > m + kSlack)) {
                    const float mn = fmaxf(m, top), f = m == -INFINITY ? 0.f : attn::ex2(m - mn);
                    m = mn;
                    const uint64_t f2 = pack2(f, f);
                    l2[0] = fma2(l2[0], f2, pack2(0.f, 0.f));
                    l2[1] = fma2(l2[1], f2, pack2(0.f, 0.f));
                    if (j > 0) {
#pragma unroll 1
                        for (int x = 0; x < D; x += 16) {
                            float o[16];
                            tc::tmem_ld16(to + x, o);
#pragma unroll
                            for (int z = 0; z < 16; ++z) o[z] *= f;
                            tc::tmem_st16_nowait(to + x, o);
                        }
                    }
                }
            }
            const float mu = m == -INFINITY ? 0.f : m;
            const uint64_t u2 = pack2(unit, unit), m2 = pack2(-mu, -mu);
            uint32_t pk[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const float2 y = unpack2(fma2(pack2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])), u2, m2));
                const float e0 = attn::ex2(y.x), e1 = attn::ex2(y.y);
                l2[x & 1] = add2(l2[x & 1], pack2(e0, e1));
                pk[x] = kv::f32_to_bf16x2(e0, e1);
            }
            tmem_st32(ts + 64 + 32 * half, pk);
            tc::tmem_wait_st();                                        // half of the product can start
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->p_ready[i][half]);
        }
        // these scores were complete, so the products before them are: their keys and the last values are free
        // (a CTA of one row tile counts for both)
        if (tid == 0) {
            for (int x = w.nq; x < 3; ++x) {
                tc::mbar_arrive(&bars->empty[key_slot]);
                if (j > 0) tc::mbar_arrive(&bars->empty[key_slot == 0 ? C::kSlots - 1 : key_slot - 1]);
            }
            key_slot = key_slot + 2 < C::kSlots ? key_slot + 2 : key_slot + 2 - C::kSlots;
        }
    }

    // ---- the row's output --------------------------------------------------------------------------------
    const float2 lp = unpack2(add2(l2[0], l2[1]));
    const float l = lp.x + lp.y;
    if (n > 0) {
        if (!warp_wait(&bars->o_full[i], 0, lane)) return false;
        tc::tc_fence_after();
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse2 = l == 0.f ? -INFINITY : m + attn::lg2(l);
    // the lane's own row of the output (or of its part), -1 past the last; the lanes tell each other theirs
    const bool in_parts = parts_here > 1;
    const int64_t out_row = (w.t0 + token) * a.c.Hq + head, own_at = !live ? -1 : in_parts ? out_row * parts.max_parts + part : out_row;
    // 32 channels at a time through the warp's place among the queries, which no product reads any more, so
    // that neighbouring lanes write a row.
    uint8_t* stage = q + i * C::kTileBytes + (tid & 96) * 128;
#pragma unroll 1
    for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        if (n > 0) {
            tmem_ld32(to + x, o);
            tmem_wait_ld();
        }
        pin32(o);
#pragma unroll
        for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * inv);
        if (__any_sync(~0u, l == 0.f)) {
            // a row whose weights are all zero may stand beside non-finite products: its output is zero
#pragma unroll
            for (int z = 0; z < 32; ++z) o[z] = l == 0.f ? 0u : o[z];
        }
        if (in_parts) {                                                // 128 bytes of fp32 a row
#pragma unroll
            for (int z = 0; z < 8; ++z)
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((z ^ (lane & 7)) << 4)) = make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
            __syncwarp();
#pragma unroll 2
            for (int z = 0; z < 32; z += 4) {
                const int r = z + lane / 8;
                const int64_t at = __shfl_sync(~0u, own_at, r);
                const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((lane % 8 ^ (r & 7)) << 4));
                if (at >= 0) *reinterpret_cast<uint4*>(parts.o + at * D + x + 4 * (lane % 8)) = v;
            }
        } else {                                                       // 64 bytes of bf16 a row, two rows to 128 bytes
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                uint32_t y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = kv::f32_to_bf16x2(__uint_as_float(o[8 * z + 2 * k]), __uint_as_float(o[8 * z + 2 * k + 1]));
                *reinterpret_cast<uint4*>(stage + (lane >> 1) * 128 + (((lane & 1) * 4 + z ^ (lane >> 1 & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            __syncwarp();
#pragma unroll 2
            for (int z = 0; z < 32; z += 8) {
                const int r = z + lane / 4;
                const int64_t at = __shfl_sync(~0u, own_at, r);
                const uint4 v = *reinterpret_cast<const uint4*>(stage + (r >> 1) * 128 + (((r & 1) * 4 + lane % 4 ^ (r >> 1 & 7)) << 4));
                if (at >= 0) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at * D + x + 8 * (lane % 4)) = v;
            }
        }
        __syncwarp();
    }
    if (live) {
        if (in_parts) parts.lse2[own_at] = lse2;
        else if (a.lse) a.lse[own_at] = lse2 * attn::kLn2;
    }
    return true;
}

template <int D, bool FP4>
__global__ void __launch_bounds__(Cfg<D, FP4>::kThreads, 1)
    many_rows_kernel(AttnCall a, Parts parts, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm)
{
    a.c.err = &g_attn_tc_error;
    using C = Cfg<D, FP4>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    uint8_t* q = smem;
    uint8_t* ring = smem + 2 * C::kTileBytes;
    Bars* bars = reinterpret_cast<Bars*>(ring + C::kSlots * C::kTileBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == 0) {
        const Tile tile = find_rows(a.c, blockIdx.x / a.c.Hkv, a.max_new, lane);
        if (lane == 0) bars->tile = tile;
    } else if (warp == 1) {
        // a lane per barrier
        if (lane < C::kSlots) {
            tc::mbar_init(&bars->full[lane], FP4 ? C::kFillThreads / 32 : 1);
            tc::mbar_init(&bars->empty[lane], 2);
        } else if (lane >= 8 && lane < 10) {
            const int i = lane - 8;
            tc::mbar_init(&bars->q_full[i], 4);
            tc::mbar_init(&bars->s_full[i], 1);
            tc::mbar_init(&bars->p_ready[i][0], 4);
            tc::mbar_init(&bars->p_ready[i][1], 4);
            tc::mbar_init(&bars->o_full[i], 1);
        } else if (lane >= 10 && lane < 14) {
            tc::mbar_init(&bars->patch[lane - 10], 1);
        } else if (lane == 14) {
            tc::mbar_init(&bars->drain, 1);
        }
        tc::fence_mbar_init();
    } else if (warp == 8) {
        tc::tmem_alloc(&bars->tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bars->tmem;
    attn::let_next_launch();

    Work w;
    const Tile tile = bars->tile;
    bool live = tile.found != 0;
    int parts_here = 1;
    const int part = blockIdx.y;
    if (live) {
        w.b = tile.b;
        w.h = blockIdx.x % a.c.Hkv;
        w.row0 = tile.row0;
        w.t0 = tile.t0;
        const int fresh = (int)(tile.t1 - tile.t0), len = tile.len;
        w.R = fresh * a.c.G;
        if (threadIdx.x == 0 && part == 0 && w.h == 0 && (len > a.max_len || fresh > a.max_new)) kv::record(a.c, kv::kErrLength);
        w.first = len > 0 ? len - fresh : -1 - fresh;
        const int lo = w.first + a.token_of(w.row0), hi = w.first + a.token_of(min(w.R - 1, w.row0 + kRows - 1));
        w.sp = attn::make_span<kTile>(max(lo, 0), len > 0 ? hi : -1, a.max_len, a.window, a.sinks);
        w.nq = w.R - w.row0 > 128 ? 2 : 1;
        if (parts.o) parts_here = min(parts.max_parts, max(1, (w.sp.tiles + parts.tiles_per_part - 1) / parts.tiles_per_part));
        w.tile_lo = parts_here > 1 ? part * parts.tiles_per_part : 0;
        w.tile_hi = parts_here > 1 ? min(w.sp.tiles, w.tile_lo + parts.tiles_per_part) : w.sp.tiles;
        live = part < parts_here;
    } else if (a.c.cu && part == 0 && blockIdx.x == gridDim.x - 1) {
        attn::clear_unowned_call<D>(a.c.cu, a.c.n, (int32_t)a.c.T, a.c.Hq, reinterpret_cast<uint4*>(a.out), a.lse, a.c.err);
    }
    bool ok = true;
    if (warp < 8) {
        if (live && warp / 4 < w.nq) ok = softmax<D, FP4>(a, parts, w, parts_here, part, q, bars, tmem, warp / 4, threadIdx.x % 128);
    } else {
        if (live && w.tile_hi > w.tile_lo) {
            if (warp == 8) {
                const int n = w.tile_hi - w.tile_lo;
                uint32_t leader = 0;
                asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
                ok = w.nq == 2 ? issue<D, FP4, 2>(n, q, ring, bars, tmem, leader) : issue<D, FP4, 1>(n, q, ring, bars, tmem, leader);
                if (leader) tc::mma_commit(&bars->drain);              // everything issued ends before the exit
                __syncwarp();
                ok = tc::mbar_wait(&bars->drain, 0, kPolls) && ok;
            } else if constexpr (FP4) {
                ok = fill_fp4<D>(a, w, ring, bars, threadIdx.x - 288);
            } else if (warp == 9) {
                ok = fill_bf16<D>(a, w, &km, &vm, ring, bars, lane);
                if (!ok)                                               // and the copies in flight land
                    for (int i = 0; i < C::kSlots; ++i) {
                        tc::mbar_wait(&bars->full[i], 0, 1u << 16);
                        tc::mbar_wait(&bars->full[i], 1, 1u << 16);
                        if (i < 4) tc::mbar_wait(&bars->patch[i], 0, 1u << 16);
                    }
            } else if (warp == 10) {
                ok = mend_bf16<D>(w, ring, bars, lane);
            }
        }
    }
    if (!ok) kv::record(a.c, kDevErrTimeout);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// Joins the parts of each row that has several.
template <int D>
__global__ void __launch_bounds__(128) join_rows_kernel(AttnCall a, Parts parts, const int share)
{
    a.c.err = &g_attn_tc_error;
    const int64_t rows = a.c.T * a.c.Hq, row = min(attn::join_row_index(share), rows - 1), t = row / a.c.Hq;
    int b = 0, n = 1;
    int64_t pos, t0, t1;
    const bool sees = kv::token_place(a.c, t, b, pos);
    kv::request_rows(a.c, b, t0, t1);
    const int len = a.c.lens[b];
    if ((sees || (t >= t0 && t < t1)) && len > 0) {
        const int fresh = (int)(t1 - t0), G = a.c.G, first = len - fresh;
        const int64_t row0 = ((t - t0) * G + row % a.c.Hq % G) / kRows * kRows;
        const int64_t last = min((int64_t)fresh * G - 1, row0 + kRows - 1);
        const Span sp = attn::make_span<kTile>(max(first + row0 / G, (int64_t)0), first + last / G, a.max_len, a.window, a.sinks);
        n = min(parts.max_parts, (sp.tiles + parts.tiles_per_part - 1) / parts.tiles_per_part);
    }
    attn::wait_for_last();
    attn::join_row<D>(a, parts, row, attn::join_row_index(share) < rows ? n : 0, share);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess || r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// The cache as rows of D channels, read in boxes of one page x 64 channels, 128-byte swizzle.
cudaError_t encode_pages(CUtensorMap* m, const void* base, int64_t rows, int D, int page)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)page};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int64_t row_tiles(const kda_kv_params& p, int32_t n, int64_t T, int32_t max_new)
{
    const int G = p.num_q_heads / p.num_kv_heads;
    const int64_t by_sum = T * G / kRows + n, by_most = (int64_t)n * (((int64_t)max_new * G + kRows - 1) / kRows);
    return by_sum < by_most ? by_sum : by_most;
}

}  // namespace

// How a call is cut along the cache when its row tiles do not fill the SMs: parts of at least kMinTiles
// tiles, kWaves parts per SM (64 requests of 16 rows, 512 CTAs uncut: 148 us, cut for eight parts per SM 177).
attn::Cut cut_many(const kda_kv_params& p, int32_t n, int64_t T, int32_t max_new, int32_t max_len)
{
    constexpr int64_t kSms = 152, kWaves = 2, kMinTiles = 4;
    const int G = p.num_q_heads / p.num_kv_heads;
    int64_t tokens = max_len;
    if (p.window) {
        const int64_t seen = (int64_t)p.window + kRows / G + 1 + p.num_sinks + 3 * kTile;
        if (seen < tokens) tokens = seen;
    }
    const int64_t tiles = (tokens + kTile - 1) / kTile, ctas = row_tiles(p, n, T, max_new) * p.num_kv_heads;
    int64_t parts = kSms * kWaves / ctas;
    if (parts > tiles / kMinTiles) parts = tiles / kMinTiles;
    if (parts > 256) parts = 256;
    if (parts < 1) parts = 1;
    attn::Cut c;
    c.tiles_per_part = (int32_t)((tiles + parts - 1) / parts);
    c.parts = (int32_t)((tiles + c.tiles_per_part - 1) / c.tiles_per_part);
    return c;
}

template <int D, bool FP4>
cudaError_t launch_many(const kda_kv_params& p, const AttnCall& a, const Parts& parts, cudaStream_t stream)
{
    using C = Cfg<D, FP4>;
    CUtensorMap km = {}, vm = {};
    if (!FP4) {
        const int64_t rows = a.c.num_pages * a.c.Hkv << a.c.page_shift;
        if (rows > 0) {
            cudaError_t e = encode_pages(&km, a.c.k, rows, D, p.page_size);
            if (e == cudaSuccess) e = encode_pages(&vm, a.c.v, rows, D, p.page_size);
            if (e != cudaSuccess) return e;
        }
    }
    cudaError_t e = cudaFuncSetAttribute(many_rows_kernel<D, FP4>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = row_tiles(p, a.c.n, a.c.T, a.max_new);
    many_rows_kernel<D, FP4><<<dim3((unsigned)(tiles * a.c.Hkv) + attn::extra_cta(a.c), (unsigned)parts.max_parts), C::kThreads, C::kSmem, stream>>>(a, parts, km, vm);
    e = cudaGetLastError();
    if (e != cudaSuccess || parts.max_parts == 1) return e;
    return attn::launch_behind(join_rows_kernel<D>, attn::join_blocks(parts, a.c.T * a.c.Hq), 128, stream, a, parts, attn::join_warps(parts));
}

template cudaError_t launch_many<64, false>(const kda_kv_params&, const AttnCall&, const Parts&, cudaStream_t);
template cudaError_t launch_many<64, true>(const kda_kv_params&, const AttnCall&, const Parts&, cudaStream_t);
template cudaError_t launch_many<128, false>(const kda_kv_params&, const AttnCall&, const Parts&, cudaStream_t);
template cudaError_t launch_many<128, true>(const kda_kv_params&, const AttnCall&, const Parts&, cudaStream_t);

cudaError_t attn_tc_read_and_clear_error(int32_t* code) { return read_and_clear(g_attn_tc_error, code); }

}  // namespace kda
