// adapters_f16.cu -- adapters with f16 weights and inputs (adapters.cuh).
#include "adapters.cuh"

namespace lmh {

cudaError_t adapters_setup_f16() { return adapters_setup_one<__half>(); }
cudaError_t launch_down_f16(const AdapterArgs& a, int grid, cudaStream_t stream) { return launch_down<__half>(a, grid, stream); }
cudaError_t launch_up_f16(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_tiles, int num_sms,
                        cudaStream_t stream) {
  return launch_up<__half>(a, out_dtype, vec, max_tiles, num_sms, stream);
}

}  // namespace lmh
