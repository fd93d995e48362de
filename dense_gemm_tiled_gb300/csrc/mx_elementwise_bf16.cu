// The elementwise kernels (mx_elementwise.cuh) for bfloat16.
#include "mx_elementwise.cuh"

namespace gb300 {

cudaError_t mx_quantize_bf16(const MxQuantArgs& a, LaunchCtx& ctx) {
  return quantize_of<__nv_bfloat16>(a, ctx);
}
cudaError_t mx_dequantize_bf16(const MxDequantArgs& a, LaunchCtx& ctx) {
  return dequantize_of<__nv_bfloat16>(a, ctx);
}
cudaError_t mx_act_backward_bf16(const MxActBwdArgs& a, LaunchCtx& ctx) {
  return act_backward_t<__nv_bfloat16>(a, ctx);
}

}  // namespace gb300
