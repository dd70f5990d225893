// kda_layer.cu -- the operators around a recurrence, in one translation unit so that they share one device
// error word: the short convolution, the selective recurrence and the group norm.
#include "kda_layer.cuh"

namespace kda {
namespace {
__device__ int32_t g_layer_error = 0;
}
__device__ __forceinline__ void record_layer_error(int32_t code) { atomicCAS(&g_layer_error, 0, code); }
cudaError_t layer_read_and_clear_error(int32_t* code) { return read_and_clear(g_layer_error, code); }
}  // namespace kda

#include "kda_conv.cuh"
#include "kda_norm.cuh"
#include "kda_ssm.cuh"

namespace kda {

size_t ssm_workspace_bytes(const kda_ssm_params&, int32_t, int64_t) { return 0; }
cudaError_t launch_ssm_prefill(const kda_ssm_params& p, const SsmCall& a, void*, cudaStream_t s) { return ssm_dispatch<false>(p, a, s); }

}  // namespace kda
