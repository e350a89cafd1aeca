// q4_project_bf16.cu -- lmh_project_q4 for bf16 hidden rows, and the choice of type.
#include "q4_project.cuh"

namespace lmh {

cudaError_t q4_setup_bf16() { return q4_attr_type<__nv_bfloat16>(); }

cudaError_t q4_launch_bf16(const Q4ProjectArgs& a, int group, int num_sms, cudaStream_t stream) {
  return q4_launch<__nv_bfloat16>(a, group, num_sms, stream);
}

cudaError_t q4_project_setup() {
  const cudaError_t e = q4_setup_bf16();
  return e == cudaSuccess ? q4_setup_f16() : e;
}

cudaError_t launch_project_q4(const void* hidden, lmh_dtype hidden_dtype, int64_t hidden_stride, int num_tokens,
                              const int32_t* row_idx, int rows, const lmh_q4_table& t, float logit_scale, void* out,
                              lmh_dtype out_dtype, int64_t out_stride, uint32_t* dev_status, int num_sms,
                              cudaStream_t stream) {
  Q4ProjectArgs a{};
  a.hidden = hidden;
  a.hidden_stride = hidden_stride;
  a.num_tokens = num_tokens;
  a.row_idx = row_idx;
  a.rows = rows;
  a.vec = reinterpret_cast<uintptr_t>(hidden) % 16 == 0 && hidden_stride % 8 == 0;
  a.t = q4_view(t);
  a.logit_scale = logit_scale;
  a.out = out;
  a.out_f32 = out_dtype == LMH_F32;
  a.out_stride = out_stride;
  a.dev_status = dev_status;
  a.wait_ns = wait_limit_ns();
  return hidden_dtype == LMH_BF16 ? q4_launch_bf16(a, t.group, num_sms, stream)
                                  : q4_launch_f16(a, t.group, num_sms, stream);
}

}  // namespace lmh
