// Attention over the 4-bit key/value cache: which kernel takes which rows.
//
// Rows of few queries per kv head (causal: up to decode_cols; with windows and
// trees: by the batch's work) go through the decode kernel (kv_decode.cuh), the others
// through the prompt kernel (kv_prompt.cuh).  The rows' lengths are on the device, so both look at every row and leave the
// other's alone; the prompt kernel is launched only where max_new allows a long
// row.  Both exist twice: for causal attention, and with windows and trees (View).
#include "kv_common.cuh"

namespace moe {
namespace kv {

static bool may_have_prompts(const moe_kv& kv, int heads, int max_new, bool view) {
  return (int64_t)max_new * (heads / kv.kv_heads) > (view ? view_cols(kv.head_dim) : decode_cols(kv.head_dim));
}

size_t attn_workspace_bytes(const moe_kv& kv, int heads, int max_new, bool view) {
  return decode_workspace_bytes(kv.head_dim) +
         (may_have_prompts(kv, heads, max_new, view) ? prompt_workspace_bytes(kv.head_dim) : 0);
}

cudaError_t launch_attention(const AttnArgs& args, cudaStream_t st) {
  AttnArgs a = args;
  a.mode = static_cast<int*>(a.ws) + kModeWord;
  const bool view = a.window > 0 || a.tree;
  bool prompts = may_have_prompts(a.kv, a.heads, a.max_new, view);
  if (view && prompts) {
    // where rows as long as there can be are little work, all rows are the decode kernel's
    int64_t tiles = (int64_t)a.kv.max_blocks * (a.kv.block_tokens / kTile);
    if (a.window > 0) tiles = min(tiles, ((int64_t)a.window + a.max_new + a.sinks) / kTile + 3);
    const int64_t r = a.heads / a.kv.kv_heads;
    const int64_t units = min(a.rows * ((a.max_new * r + 7) / 8), (a.T * r + a.rows * (int64_t)7) / 8);
    prompts = decode_cost(a.kv.head_dim, a.kv.kv_heads, units, tiles) > kDecodeAlone;
  }
  a.prompts = prompts;
  AttnArgs p = a;
  p.ws = static_cast<char*>(a.ws) + decode_workspace_bytes(a.kv.head_dim);
  cudaError_t e = view ? launch_decode_view(a, st) : launch_decode(a, st);
  if (e == cudaSuccess && prompts) e = view ? launch_prompt_view(p, st) : launch_prompt(p, st);
  if (e == cudaSuccess) e = launch_decode_join(a, st);
  if (e == cudaSuccess && prompts) e = launch_prompt_join(p, st);
  return e;
}

}  // namespace kv
}  // namespace moe
