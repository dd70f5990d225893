// kda_layer_api.cu -- the extern "C" entry points of the operators around a recurrence (include/kda.h):
// host-side argument checks, then the launch.  Nothing here allocates, synchronises or keeps state.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "kda_layer.cuh"

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool odd(const void* p, uintptr_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; }
bool bad_dtype(int32_t d) { return d != KDA_F32 && d != KDA_BF16; }
uintptr_t size_of(int32_t d) { return d == KDA_F32 ? 4 : 2; }

int32_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 64;
constexpr int64_t kMaxStride = (int64_t)1 << 31;        // a row's offset then stays below 2^62

int32_t check_ssm_params(const kda_ssm_params* p)
{
    if (!p || p->num_heads <= 0 || p->num_groups <= 0 || p->num_heads % p->num_groups != 0 ||
        !(p->softplus_threshold >= 0.f))
        return KDA_ERR_INVALID_ARG;
    const int32_t P = p->head_dim, N = p->state_dim;
    if ((P != 16 && P != 32 && P != 64 && P != 128) || (N != 16 && N != 32 && N != 64 && N != 128 && N != 256) ||
        bad_dtype(p->io_dtype) || bad_dtype(p->dt_dtype) || bad_dtype(p->out_dtype) || p->num_heads > 4096)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Checks shared by the two entry points; `a` is filled, *noop set for a valid call without work.
int32_t check_ssm(const kda_ssm_params* p, const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const void* B,
                  int64_t b_stride, const void* C, int64_t c_stride, const float* A_log, const float* dt_bias, const float* D,
                  int32_t num_seqs, int64_t T, float* pool, int64_t num_slots, const int32_t* idx, void* out, kda::SsmCall* a,
                  bool* noop)
{
    *noop = false;
    const int32_t rc = check_ssm_params(p);
    if (rc != KDA_OK) return rc;
    if (num_seqs < 0 || T < 0 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (T == 0 || num_seqs == 0) {
        *noop = true;
        return KDA_OK;
    }
    if (!x || !dt || !B || !C || !A_log || !pool || !idx || !out) return KDA_ERR_INVALID_ARG;
    const int64_t xw = (int64_t)p->num_heads * p->head_dim, bw = (int64_t)p->num_groups * p->state_dim;
    if (x_stride < xw || b_stride < bw || c_stride < bw || dt_stride < p->num_heads || x_stride % 8 != 0 || b_stride % 8 != 0 ||
        c_stride % 8 != 0)
        return KDA_ERR_INVALID_ARG;
    if (x_stride >= kMaxStride || b_stride >= kMaxStride || c_stride >= kMaxStride || dt_stride >= kMaxStride) return KDA_ERR_UNSUPPORTED;
    if (misaligned(x) || misaligned(B) || misaligned(C) || misaligned(pool) || misaligned(out) || odd(dt, size_of(p->dt_dtype)) ||
        odd(A_log, 4) || odd(dt_bias, 4) || odd(D, 4) || odd(idx, 4))
        return KDA_ERR_MISALIGNED;
    if (T >= kMaxTokens || (int64_t)num_seqs * p->num_heads >= ((int64_t)1 << 29) / (p->head_dim / 16))
        return KDA_ERR_UNSUPPORTED;
    a->x = x; a->dt = dt; a->B = B; a->C = C;
    a->x_stride = x_stride; a->dt_stride = dt_stride; a->b_stride = b_stride; a->c_stride = c_stride;
    a->A_log = A_log; a->dt_bias = dt_bias; a->D = D;
    a->cu = nullptr; a->n = num_seqs; a->T = T;
    a->pool = pool; a->num_slots = num_slots; a->idx = idx; a->out = out;
    a->H = p->num_heads; a->P = p->head_dim; a->N = p->state_dim; a->G = p->num_groups;
    a->dt_bf16 = p->dt_dtype == KDA_BF16;
    a->threshold = p->softplus_threshold;
    a->short_len = 0;
    return KDA_OK;
}

}  // namespace

extern "C" {

int32_t kda_causal_conv(const kda_conv_params* p, const void* x, int64_t x_stride, const float* weight, const float* bias,
                        const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, void* state_pool, int64_t num_slots,
                        const int32_t* state_idx, void* const* outs, const int32_t* out_channels, int32_t num_outs,
                        kda_stream_t stream)
{
    if (!p || p->num_channels <= 0 || num_seqs < 0 || total_tokens < 0 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (p->width < 2 || p->width > 4 || bad_dtype(p->io_dtype) || (p->activation != KDA_ACT_NONE && p->activation != KDA_ACT_SILU) ||
        p->num_channels > (1 << 20))
        return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens && total_tokens != num_seqs) return KDA_ERR_INVALID_ARG;
    if (num_outs < 1 || num_outs > kda::kMaxOuts || !outs || !out_channels) return KDA_ERR_INVALID_ARG;
    kda::ConvCall a;
    int64_t sum = 0;
    for (int j = 0; j < num_outs; ++j) {
        if (out_channels[j] <= 0) return KDA_ERR_INVALID_ARG;
        a.out_first[j] = (int32_t)sum;
        a.out[j] = outs[j];
        sum += out_channels[j];
    }
    if (sum != p->num_channels) return KDA_ERR_INVALID_ARG;
    for (int j = num_outs; j <= kda::kMaxOuts; ++j) a.out_first[j] = (int32_t)sum;
    for (int j = num_outs; j < kda::kMaxOuts; ++j) a.out[j] = nullptr;
    if (total_tokens == 0 || num_seqs == 0) return KDA_OK;
    if (!x || !weight || !state_pool || !state_idx || x_stride < p->num_channels) return KDA_ERR_INVALID_ARG;
    const uintptr_t size = size_of(p->io_dtype);
    if (odd(x, size) || odd(state_pool, size) || odd(weight, 4) || odd(bias, 4) || odd(cu_seqlens, 4) || odd(state_idx, 4))
        return KDA_ERR_MISALIGNED;
    for (int j = 0; j < num_outs; ++j) {
        if (!outs[j]) return KDA_ERR_INVALID_ARG;
        if (odd(outs[j], size)) return KDA_ERR_MISALIGNED;
    }
    if (total_tokens >= kMaxTokens || num_seqs >= (1 << 30) || x_stride >= kMaxStride) return KDA_ERR_UNSUPPORTED;
    a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias;
    a.cu = cu_seqlens; a.n = num_seqs; a.T = total_tokens;
    a.pool = state_pool; a.num_slots = num_slots; a.idx = state_idx;
    a.C = p->num_channels; a.num_outs = num_outs;
    return from_cuda(kda::launch_conv(*p, a, (cudaStream_t)stream));
}

void kda_ssm_params_init(kda_ssm_params* p, int32_t num_heads, int32_t head_dim, int32_t state_dim, int32_t num_groups)
{
    if (!p) return;
    p->num_heads = num_heads;
    p->head_dim = head_dim;
    p->state_dim = state_dim;
    p->num_groups = num_groups;
    p->io_dtype = KDA_BF16;
    p->dt_dtype = KDA_F32;
    p->out_dtype = KDA_BF16;
    p->softplus_threshold = 20.0f;
}

size_t kda_ssm_prefill_workspace_size(const kda_ssm_params* p, int32_t num_seqs, int64_t total_tokens)
{
    if (check_ssm_params(p) != KDA_OK || num_seqs <= 0 || total_tokens <= 0 || total_tokens >= kMaxTokens) return 0;
    return kda::ssm_workspace_bytes(*p, num_seqs, total_tokens);
}

int32_t kda_ssm_prefill(const kda_ssm_params* p, const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const void* B,
                        int64_t b_stride, const void* C, int64_t c_stride, const float* A_log, const float* dt_bias, const float* D,
                        const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, float* state_pool, int64_t num_slots,
                        const int32_t* state_idx, void* out, void* workspace, size_t workspace_bytes, kda_stream_t stream)
{
    kda::SsmCall a;
    bool noop;
    const int32_t rc = check_ssm(p, x, x_stride, dt, dt_stride, B, b_stride, C, c_stride, A_log, dt_bias, D, num_seqs, total_tokens,
                                 state_pool, num_slots, state_idx, out, &a, &noop);
    if (rc != KDA_OK || noop) return rc;
    if (!cu_seqlens) return KDA_ERR_INVALID_ARG;
    if (odd(cu_seqlens, 4)) return KDA_ERR_MISALIGNED;
    const size_t need = kda::ssm_workspace_bytes(*p, num_seqs, total_tokens);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return KDA_ERR_WORKSPACE;
    a.cu = cu_seqlens;
    return from_cuda(kda::launch_ssm_prefill(*p, a, workspace, (cudaStream_t)stream));
}

int32_t kda_ssm_decode(const kda_ssm_params* p, const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const void* B,
                       int64_t b_stride, const void* C, int64_t c_stride, const float* A_log, const float* dt_bias, const float* D,
                       int32_t batch, float* state_pool, int64_t num_slots, const int32_t* state_idx, void* out, kda_stream_t stream)
{
    kda::SsmCall a;
    bool noop;
    const int32_t rc = check_ssm(p, x, x_stride, dt, dt_stride, B, b_stride, C, c_stride, A_log, dt_bias, D, batch, batch, state_pool,
                                 num_slots, state_idx, out, &a, &noop);
    if (rc != KDA_OK || noop) return rc;
    return from_cuda(kda::launch_ssm_decode(*p, a, (cudaStream_t)stream));
}

int32_t kda_group_norm(const kda_norm_params* p, const void* x, int64_t x_stride, const void* gate, int64_t gate_stride,
                       const float* weight, const float* bias, int64_t tokens, void* out, kda_stream_t stream)
{
    if (!p || p->num_groups <= 0 || p->group_size <= 0 || tokens < 0 || !(p->eps >= 0.f) || (p->gate_first && !gate && tokens > 0))
        return KDA_ERR_INVALID_ARG;
    if (bad_dtype(p->io_dtype) || bad_dtype(p->out_dtype) || p->activation < KDA_ACT_NONE || p->activation > KDA_ACT_SIGMOID ||
        p->group_size > 16384)
        return KDA_ERR_UNSUPPORTED;
    if (tokens == 0) return KDA_OK;
    const int64_t width = (int64_t)p->num_groups * p->group_size;
    if (!x || !out || x_stride < width || (gate && gate_stride < width)) return KDA_ERR_INVALID_ARG;
    if (odd(x, size_of(p->io_dtype)) || odd(out, size_of(p->out_dtype)) || odd(gate, size_of(p->out_dtype)) || odd(weight, 4) || odd(bias, 4))
        return KDA_ERR_MISALIGNED;
    if (tokens >= ((int64_t)1 << 31) || tokens * p->num_groups >= ((int64_t)1 << 31) || x_stride >= kMaxStride ||
        (gate && gate_stride >= kMaxStride))
        return KDA_ERR_UNSUPPORTED;
    kda::NormCall a;
    a.x = x; a.x_stride = x_stride; a.gate = gate; a.gate_stride = gate_stride;
    a.weight = weight; a.bias = bias; a.tokens = tokens; a.out = out;
    a.G = p->num_groups; a.size = p->group_size;
    a.act = p->activation; a.gate_first = p->gate_first != 0; a.center = p->center != 0;
    a.eps = p->eps;
    return from_cuda(kda::launch_norm(*p, a, (cudaStream_t)stream));
}

}  // extern "C"
