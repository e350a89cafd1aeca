// q4_project_f16.cu -- lmh_project_q4 for f16 hidden rows.
#include "q4_project.cuh"

namespace lmh {

cudaError_t q4_setup_f16() { return q4_attr_type<__half>(); }

cudaError_t q4_launch_f16(const Q4ProjectArgs& a, int group, int num_sms, cudaStream_t stream) {
  return q4_launch<__half>(a, group, num_sms, stream);
}

}  // namespace lmh
