// adapters_bf16.cu -- adapters with bf16 weights and inputs (adapters.cuh).
#include "adapters.cuh"

namespace lmh {

cudaError_t adapters_setup_bf16() { return adapters_setup_one<__nv_bfloat16>(); }
cudaError_t launch_down_bf16(const AdapterArgs& a, int grid, cudaStream_t stream) { return launch_down<__nv_bfloat16>(a, grid, stream); }
cudaError_t launch_up_bf16(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_tiles, int num_sms,
                        cudaStream_t stream) {
  return launch_up<__nv_bfloat16>(a, out_dtype, vec, max_tiles, num_sms, stream);
}

}  // namespace lmh
