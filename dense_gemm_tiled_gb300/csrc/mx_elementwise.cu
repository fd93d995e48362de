// The elementwise kernels (mx_elementwise.cuh) for fp32, and the dispatch over
// element types.
#include "mx_elementwise.cuh"

namespace gb300 {

cudaError_t launch_mx_quantize(const MxQuantArgs& a, LaunchCtx& ctx) {
  return a.out == 0   ? quantize_of<float>(a, ctx)
         : a.out == 1 ? mx_quantize_f16(a, ctx)
                      : mx_quantize_bf16(a, ctx);
}
cudaError_t launch_mx_dequantize(const MxDequantArgs& a, LaunchCtx& ctx) {
  return a.out == 0   ? dequantize_of<float>(a, ctx)
         : a.out == 1 ? mx_dequantize_f16(a, ctx)
                      : mx_dequantize_bf16(a, ctx);
}
size_t mx_act_backward_scratch(int rows, int cols, int num_sms) {
  const dim3 grid = strip_grid(cols, act_tiles(rows), num_sms, BLOCKS_PER_SM - 1);
  return act_joined(grid) ? 0 : (size_t)grid.y * cols * sizeof(float);
}
cudaError_t launch_mx_act_backward(const MxActBwdArgs& a, LaunchCtx& ctx) {
  return a.out == 0   ? act_backward_t<float>(a, ctx)
         : a.out == 1 ? mx_act_backward_f16(a, ctx)
                      : mx_act_backward_bf16(a, ctx);
}

}  // namespace gb300
