// Attention over the 4-bit key/value cache: which kernel takes which rows.
//
// Rows of up to decode_cols queries per kv head go through the decode kernel
// (kv_decode.cu), longer ones through the prompt kernel (kv_prompt.cu).  The
// rows' lengths are on the device, so both look at every row and leave the
// other's alone; the prompt kernel is launched only where max_new allows a long
// row.
#include "kv_common.cuh"

namespace moe {
namespace kv {

static bool may_have_prompts(const moe_kv& kv, int heads, int max_new) {
  return (int64_t)max_new * (heads / kv.kv_heads) > decode_cols(kv.head_dim);
}

size_t attn_workspace_bytes(const moe_kv& kv, int, int, int heads, int max_new) {
  return decode_workspace_bytes(kv.head_dim) +
         (may_have_prompts(kv, heads, max_new) ? prompt_workspace_bytes(kv.head_dim) : 0);
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_decode(a, st);
  if (e != cudaSuccess || !may_have_prompts(a.kv, a.heads, a.max_new)) return e;
  AttnArgs p = a;
  p.ws = static_cast<char*>(a.ws) + decode_workspace_bytes(a.kv.head_dim);
  return launch_prompt(p, st);
}

}  // namespace kv
}  // namespace moe
