// kda_kv_api.cu -- the extern "C" entry points of the paged cache and its attention (include/kda.h):
// host-side argument checks, then the launch.  Nothing here allocates, synchronises or keeps state.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_internal.cuh"
#include "kda_kv.cuh"

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int32_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

int32_t check_params(const kda_kv_params* p)
{
    if (!p || p->num_q_heads <= 0 || p->num_kv_heads <= 0 || p->num_q_heads % p->num_kv_heads != 0 || p->window < 0 ||
        p->num_sinks < 0 || !(p->softmax_scale == p->softmax_scale) || p->rot_dim < 0)
        return KDA_ERR_INVALID_ARG;
    const int32_t s = p->page_size;
    if ((p->head_dim != 64 && p->head_dim != 128) || (s != 16 && s != 32 && s != 64 && s != 128) ||
        (p->cache_dtype != KDA_CACHE_BF16 && p->cache_dtype != KDA_CACHE_FP4) || p->rot_dim > p->head_dim ||
        p->rot_dim % 32 != 0 || p->num_q_heads / p->num_kv_heads > 128 || p->num_q_heads > 1024)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Checks of the cache and the batch; *noop is set for a valid call without work.
int32_t check_batch(const kda_kv_params* p, const void* kc, const void* vc, const void* ks, const void* vs,
                    int64_t num_pages, const int32_t* cu, const int32_t* lens, const int32_t* table, int32_t num_seqs,
                    int32_t max_pages, int64_t T, bool* noop)
{
    *noop = false;
    const int32_t rc = check_params(p);
    if (rc != KDA_OK) return rc;
    if (num_seqs < 0 || max_pages < 0 || T < 0 || num_pages < 0) return KDA_ERR_INVALID_ARG;
    if (!cu && T != num_seqs) return KDA_ERR_INVALID_ARG;
    if (T == 0 || num_seqs == 0) {
        *noop = true;
        return KDA_OK;
    }
    if (!kc || !vc || !lens || !table || max_pages == 0) return KDA_ERR_INVALID_ARG;
    if (p->cache_dtype == KDA_CACHE_FP4 && (!ks || !vs)) return KDA_ERR_INVALID_ARG;
    if (misaligned(kc) || misaligned(vc)) return KDA_ERR_MISALIGNED;
    if (p->cache_dtype == KDA_CACHE_FP4 && (misaligned(ks) || misaligned(vs))) return KDA_ERR_MISALIGNED;
    // counts that the kernels' 32-bit grids and tensor-map coordinates can hold
    if ((int64_t)num_seqs * p->num_kv_heads >= ((int64_t)1 << 30) || T >= ((int64_t)1 << 31) / 512 || (int64_t)max_pages * p->page_size >= ((int64_t)1 << 31) - 256 ||
        num_pages >= ((int64_t)1 << 31) || num_pages * p->num_kv_heads * p->page_size >= ((int64_t)1 << 31))   // no product past 2^48
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda::kv::Paged paged(const kda_kv_params* p, const void* kc, const void* vc, const void* ks, const void* vs,
                     int64_t num_pages, const int32_t* cu, const int32_t* lens, const int32_t* table, int32_t num_seqs,
                     int32_t max_pages, int64_t T)
{
    kda::kv::Paged c;
    c.k = (uint8_t*)kc; c.v = (uint8_t*)vc; c.ks = (uint8_t*)ks; c.vs = (uint8_t*)vs;
    c.cu = cu; c.lens = lens; c.table = table;
    c.num_pages = num_pages; c.T = T; c.n = num_seqs; c.max_pages = max_pages;
    c.page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
    c.Hq = p->num_q_heads; c.Hkv = p->num_kv_heads; c.G = p->num_q_heads / p->num_kv_heads;
    c.err = nullptr;
    return c;
}

// The bound on a request's new tokens that every size and form goes by, in the workspace query and in the call
// alike: a caller without one may pass any large number, and no request has more than all tokens.
int32_t new_tokens_bound(int32_t max_new_tokens, int64_t total_tokens)
{
    return total_tokens < max_new_tokens ? (int32_t)total_tokens : max_new_tokens;
}

bool bad_stride(int64_t stride, int heads, int D) { return stride < (int64_t)heads * D || stride % 8 != 0; }

}  // namespace

extern "C" {

void kda_kv_params_init(kda_kv_params* p, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t page_size)
{
    if (!p) return;
    p->num_q_heads = num_q_heads;
    p->num_kv_heads = num_kv_heads;
    p->head_dim = head_dim;
    p->page_size = page_size;
    p->cache_dtype = KDA_CACHE_BF16;
    p->rot_dim = head_dim;
    p->rope_interleaved = 0;
    p->window = 0;
    p->num_sinks = 0;
    p->softmax_scale = 0.0f;
}

int32_t kda_kv_append(const kda_kv_params* p, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const float* rope, int64_t rope_rows, const int32_t* positions,
                      const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table, int32_t num_seqs,
                      int32_t max_pages, int64_t total_tokens, void* k_cache, void* v_cache, uint8_t* k_scale,
                      uint8_t* v_scale, int64_t num_pages, void* q_out, kda_stream_t stream)
{
    bool noop;
    const int32_t rc = check_batch(p, k_cache, v_cache, k_scale, v_scale, num_pages, cu_seqlens, kv_lens, block_table,
                                   num_seqs, max_pages, total_tokens, &noop);
    if (rc != KDA_OK || noop) return rc;
    if (!k || !v || (q == nullptr) != (q_out == nullptr)) return KDA_ERR_INVALID_ARG;
    if (p->rot_dim > 0 && (!rope || rope_rows < 0)) return KDA_ERR_INVALID_ARG;
    if (bad_stride(k_stride, p->num_kv_heads, p->head_dim) || bad_stride(v_stride, p->num_kv_heads, p->head_dim) ||
        (q && bad_stride(q_stride, p->num_q_heads, p->head_dim)) ||
        (q && q == q_out && q_stride != (int64_t)p->num_q_heads * p->head_dim))
        return KDA_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(q_out) || misaligned(rope)) return KDA_ERR_MISALIGNED;
    return from_cuda(kda::launch_kv_append(*p, paged(p, k_cache, v_cache, k_scale, v_scale, num_pages, cu_seqlens,
                                                     kv_lens, block_table, num_seqs, max_pages, total_tokens),
                                           q, q_stride, k, k_stride, v, v_stride, rope, rope_rows, positions, q_out,
                                           (cudaStream_t)stream));
}

int32_t kda_kv_read(const kda_kv_params* p, const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                    const uint8_t* v_scale, int64_t num_pages, const int32_t* cu_seqlens, const int32_t* kv_lens,
                    const int32_t* block_table, int32_t num_seqs, int32_t max_pages, int64_t total_tokens,
                    void* k_out, void* v_out, kda_stream_t stream)
{
    bool noop;
    const int32_t rc = check_batch(p, k_cache, v_cache, k_scale, v_scale, num_pages, cu_seqlens, kv_lens, block_table,
                                   num_seqs, max_pages, total_tokens, &noop);
    if (rc != KDA_OK || noop) return rc;
    if (!k_out || !v_out) return KDA_ERR_INVALID_ARG;
    if (misaligned(k_out) || misaligned(v_out)) return KDA_ERR_MISALIGNED;
    return from_cuda(kda::launch_kv_read(*p, paged(p, k_cache, v_cache, k_scale, v_scale, num_pages, cu_seqlens,
                                                   kv_lens, block_table, num_seqs, max_pages, total_tokens),
                                         k_out, v_out, (cudaStream_t)stream));
}

size_t kda_paged_attention_workspace_size(const kda_kv_params* p, int32_t num_seqs, int64_t total_tokens,
                                          int32_t max_new_tokens, int32_t max_kv_len)
{
    if (check_params(p) != KDA_OK || num_seqs <= 0 || total_tokens <= 0 || max_new_tokens <= 0 || max_kv_len <= 0) return 0;
    return kda::attention_workspace_bytes(*p, num_seqs, total_tokens, new_tokens_bound(max_new_tokens, total_tokens), max_kv_len);
}

int32_t kda_paged_attention(const kda_kv_params* p, const void* q, int64_t q_stride, const void* k_cache,
                            const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale, int64_t num_pages,
                            const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* block_table,
                            int32_t num_seqs, int32_t max_pages, int64_t total_tokens, int32_t max_new_tokens,
                            int32_t max_kv_len, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            kda_stream_t stream)
{
    bool noop;
    const int32_t rc = check_batch(p, k_cache, v_cache, k_scale, v_scale, num_pages, cu_seqlens, kv_lens, block_table,
                                   num_seqs, max_pages, total_tokens, &noop);
    if (rc != KDA_OK || noop) return rc;
    if (!q || !out) return KDA_ERR_INVALID_ARG;
    if (max_new_tokens < 1 || (!cu_seqlens && max_new_tokens != 1) || max_kv_len < 1 ||
        (int64_t)max_kv_len > (int64_t)max_pages * p->page_size)
        return KDA_ERR_INVALID_ARG;
    if (bad_stride(q_stride, p->num_q_heads, p->head_dim)) return KDA_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(out)) return KDA_ERR_MISALIGNED;
    max_new_tokens = new_tokens_bound(max_new_tokens, total_tokens);
    const size_t need = kda::attention_workspace_bytes(*p, num_seqs, total_tokens, max_new_tokens, max_kv_len);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return KDA_ERR_WORKSPACE;
    kda::AttnCall a;
    a.c = paged(p, k_cache, v_cache, k_scale, v_scale, num_pages, cu_seqlens, kv_lens, block_table, num_seqs, max_pages,
                total_tokens);
    a.q = q;
    a.q_stride = q_stride;
    a.max_new = max_new_tokens;
    a.max_len = max_kv_len;
    a.window = p->window;
    a.sinks = p->num_sinks;
    a.scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / sqrtf((float)p->head_dim);
    int exponent = 0;
    if (isfinite(a.scale)) frexp(a.scale * 1.4426950408889634, &exponent);   // a product of at least 2^(exponent - 1)
    a.min_exp = 2 - exponent > 1 ? 2 - exponent : 1;
    a.out = out;
    a.lse = lse;
    a.by_group = (((uint64_t)1 << 36) + a.c.G - 1) / a.c.G;
    return from_cuda(kda::launch_attention(*p, a, workspace, (cudaStream_t)stream));
}

}  // extern "C"
