// K3 for head dim 64 (fwd_kernel.cuh), in a translation unit of its own.
#include "fwd_kernel.cuh"

namespace bd {

cudaError_t launch_fwd64(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const int32_t* seg,
                         const Geom& g, __nv_bfloat16* out, float* lse, int32_t* status, int merge, cudaStream_t st) {
  return g.G % 2 == 0 ? launch_one<64, 2, 3>(mq, mk, mv, seg, g, out, lse, status, merge, st)
                      : launch_one<64, 1, 3>(mq, mk, mv, seg, g, out, lse, status, merge, st);
}

}  // namespace bd
