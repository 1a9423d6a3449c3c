// Causal attention over the 4-bit cache for rows of few new tokens: the kernel of
// kv_decode.cuh.
#include "kv_decode.cuh"

namespace moe {
namespace kv {

size_t decode_workspace_bytes(int D) {
  return D == 256 ? bytes_for<256>() : D == 128 ? bytes_for<128>() : bytes_for<64>();
}

cudaError_t launch_decode(const AttnArgs& a, cudaStream_t st) {
  const int D = a.kv.head_dim;
  return D == 256 ? launch<256, false>(a, st)
                  : D == 128 ? launch<128, false>(a, st) : launch<64, false>(a, st);
}

cudaError_t launch_decode_join(const AttnArgs& a, cudaStream_t st) {
  const int D = a.kv.head_dim;
  return D == 256 ? launch_join<256>(a, st) : D == 128 ? launch_join<128>(a, st) : launch_join<64>(a, st);
}

}  // namespace kv
}  // namespace moe
