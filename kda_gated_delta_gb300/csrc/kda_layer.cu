// kda_layer.cu -- the operators around a recurrence that record errors, in one translation unit so that they share one device
// error word: the short convolution and the selective recurrence.
#include "kda_layer.cuh"

namespace kda {
namespace {
__device__ int32_t g_layer_error = 0;
}
__device__ __forceinline__ void record_layer_error(int32_t code) { atomicCAS(&g_layer_error, 0, code); }
cudaError_t layer_error_word(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_layer_error); }
}  // namespace kda

#include "kda_conv.cuh"
#include "kda_ssm.cuh"
#include "kda_ssm_tc.cuh"
