// The elementwise kernels (mx_elementwise.cuh) for fp16.
#include "mx_elementwise.cuh"

namespace gb300 {

cudaError_t mx_quantize_f16(const MxQuantArgs& a, LaunchCtx& ctx) {
  return quantize_of<__half>(a, ctx);
}
cudaError_t mx_dequantize_f16(const MxDequantArgs& a, LaunchCtx& ctx) {
  return dequantize_of<__half>(a, ctx);
}
cudaError_t mx_act_backward_f16(const MxActBwdArgs& a, LaunchCtx& ctx) {
  return act_backward_t<__half>(a, ctx);
}

}  // namespace gb300
