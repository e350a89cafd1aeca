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
  a.vec = reinterpret_cast<uintptr_t>(hidden) % 16 == 0 && hidden_stride % 8 == 0;
  a.t = q4_view(t);
  a.logit_scale = logit_scale;
  a.out_f32 = out_dtype == LMH_F32;
  a.out_stride = out_stride;
  a.dev_status = dev_status;
  a.wait_ns = wait_limit_ns();
  // The passes are the grid's second dimension: 65535 at most, of at least 8 rows each.
  constexpr int kRowsPerLaunch = 65504 * 8;  // (whole passes of 8, 16 and 32)
  for (int first = 0; first < rows; first += a.rows) {
    a.rows = rows - first < kRowsPerLaunch ? rows - first : kRowsPerLaunch;
    a.row_idx = row_idx ? row_idx + first : nullptr;
    if (!row_idx) {
      a.hidden = static_cast<const char*>(hidden) + static_cast<int64_t>(first) * hidden_stride * 2;
      a.num_tokens = num_tokens - first;
    }
    a.out = static_cast<char*>(out) + static_cast<int64_t>(first) * out_stride * (a.out_f32 ? 4 : 2);
    const cudaError_t e = hidden_dtype == LMH_BF16 ? q4_launch_bf16(a, t.group, num_sms, stream)
                                                   : q4_launch_f16(a, t.group, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lmh
