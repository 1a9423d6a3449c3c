// Attention with windows and trees over the 4-bit cache for rows of few new tokens: the kernel of
// kv_decode.cuh.
#include "kv_decode.cuh"

namespace moe {
namespace kv {

cudaError_t launch_decode_view(const AttnArgs& a, cudaStream_t st) {
  const int D = a.kv.head_dim;
  return D == 256 ? launch<256, true>(a, st)
                  : D == 128 ? launch<128, true>(a, st) : launch<64, true>(a, st);
}

}  // namespace kv
}  // namespace moe
