// bf16 instantiation of the fused and grouped products (fused_tcgen05.cuh).
#include "fused_tcgen05.cuh"

namespace gb300 {

cudaError_t launch_fused_bf16(const FusedArgs& a, LaunchCtx& ctx) {
  return launch_fused_t<__nv_bfloat16>(a, ctx);
}

}  // namespace gb300
