// fp16 instantiation of the fused and grouped products (fused_tcgen05.cuh).
#include "fused_tcgen05.cuh"

namespace gb300 {

cudaError_t launch_fused(const FusedArgs& a, LaunchCtx& ctx) {
  return a.dtype == 2 ? launch_fused_bf16(a, ctx) : launch_fused_t<__half>(a, ctx);
}

}  // namespace gb300
