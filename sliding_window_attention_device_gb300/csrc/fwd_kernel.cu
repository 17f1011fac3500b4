// K3's entry: the forward kernel for head dim 128 (fwd_kernel.cuh), and the
// choice among the head dims' kernels.
#include "fwd_kernel.cuh"

namespace bd {

cudaError_t launch_fwd64(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const int32_t* seg,
                         const Geom& g, __nv_bfloat16* out, float* lse, int32_t* status, int merge, cudaStream_t st);
cudaError_t launch_fwd256(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const int32_t* seg,
                          const Geom& g, void* out, float* lse, int32_t* status, int merge, cudaStream_t st);

// Two query heads of one GQA group per CTA when the group size is even and
// D <= 128 (tensor memory: 2 x (128 + D) columns); one otherwise. D = 256 has
// its own kernel with K / V streamed in halves (fwd256_kernel.cu).
cudaError_t launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const int32_t* seg,
                       const Geom& g, void* out, float* lse, int32_t* status, int merge, cudaStream_t st) {
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  const bool pairs = (g.G % 2) == 0;
  switch (g.D) {
    case 64:
      return launch_fwd64(mq, mk, mv, seg, g, o, lse, status, merge, st);
    case 128:
      return pairs ? launch_one<128, 2, 2>(mq, mk, mv, seg, g, o, lse, status, merge, st)
                   : launch_one<128, 1, 2>(mq, mk, mv, seg, g, o, lse, status, merge, st);
    case 256:
      return launch_fwd256(mq, mk, mv, seg, g, out, lse, status, merge, st);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace bd
