// The converted product (mx_mixed.cuh) for bfloat16.
#include "mx_mixed.cuh"

namespace gb300 {

cudaError_t launch_mx_mixed_bf16(const MxStreamArgs& a, LaunchCtx& ctx) {
  return launch_mixed_t<__nv_bfloat16>(a, ctx);
}

}  // namespace gb300
