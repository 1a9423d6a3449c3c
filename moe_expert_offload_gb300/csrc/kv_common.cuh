// The 4-bit key/value cache: its byte layout and the launchers of its kernels
// (entry points in kv_abi.cu, declared and documented in include/moe.h).
//
// A block holds block_tokens tokens of every kv head, head by head, each head's
// share as tiles of 16 tokens.  A tile of head_dim D (G = D / 64 groups) is
// 18 D contiguous bytes,
//   K codes [16][D/2] | V codes [16][D/2] |
//   K scale [16][G] | K bias [16][G] | V scale [G][16] | V bias [G][16]  (fp16)
// so that one bulk copy brings everything that 16 keys of one head need.  The
// 16-byte chunk j of code row r lies at chunk j ^ swizzle(r): eight rows read
// at one chunk (an ldmatrix) then touch every shared-memory bank once.
// K's scales go by key, V's by group: the order in which the two products read
// them (K as rows of the contraction's result, V along the contraction).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {
namespace kv {

constexpr int kTile = 16;  // tokens of a tile
constexpr int kGrid = 152; // CTAs of the attention kernels: one per SM
// Rows of up to this many queries per kv head (new tokens x query heads on it)
// go through the decode kernel, longer ones through the prompt kernel
// (microseconds, decode | prompt, 8 query heads on a kv head; 1 and 16 rows of
// 2000 to 4000 keys, 4 of 30000 to 60000):
//   head_dim 256, 32 queries  13 | 24   32 | 33    84 |  76
//                 48          14 | 26   43 | 35   120 |  80
//   head_dim 128, 64          14 | 25   54 | 47   155 | 100
//                 96          16 | 26   80 | 48   242 | 106
//   head_dim 64,  64          13 | 22   36 | 38    99 |  86
//                 96          13 | 22   48 | 37   152 |  91
// A compromise: a lone short row is faster in the decode kernel at every number
// of columns (its units are smaller), many or long ones in the prompt kernel
// from about these numbers on; the rule does not look at the lengths.
__host__ __device__ constexpr int decode_cols(int D) { return D == 256 ? 32 : 64; }

__host__ __device__ constexpr int tile_bytes(int D) { return 18 * D; }

template <int D>
__device__ __forceinline__ int swizzle(int r) {
  return D == 256 ? (r & 7) : D == 128 ? ((r >> 1) & 3) : ((r >> 2) & 1);
}

// scale * unit * 2^e, kept between 1e-37 and 2^88: a hidden key's -inf stays one (times 0 it would
// be NaN), and no score overflows (raw ones are below 2^39).  It changes no weight: distances of
// raw scores are 0 or between 2^-80 and 2^40, which times either end is nothing or past 2^7.
__device__ __forceinline__ float score_factor(float scale, float unit, int e) {
  const float f = scale * __int_as_float((e + 127) << 23) * unit;
  return fminf(fmaxf(f, 1e-37f), 0x1p88f);
}

// fp16 index (from the tile's 16 D bytes of codes on) of each scale and bias
template <int D>
struct Meta {
  static constexpr int G = D / 64;
  __device__ static int k_scale(int key, int g) { return key * G + g; }
  __device__ static int k_bias(int key, int g) { return 16 * G + key * G + g; }
  __device__ static int v_scale(int key, int g) { return 32 * G + g * 16 + key; }
  __device__ static int v_bias(int key, int g) { return 48 * G + g * 16 + key; }
};

struct PlanArgs {
  moe_kv kv;
  moe_kv_batch batch;
  const int32_t* new_len;
  int rows;
};
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st);
cudaError_t launch_reset(const moe_kv& kv, cudaStream_t st);

struct StoreArgs {
  moe_kv kv;
  moe_qkv proj;
  moe_rope rope;  // rotary_dim 0: no rotation
  const int32_t* slot;
  const int32_t* positions;
  int32_t* err;
  uint16_t* q_out;
  int T;
};
cudaError_t launch_store(const StoreArgs& a, cudaStream_t st);

struct LoadArgs {
  moe_kv kv;
  const int32_t* slot;
  uint16_t *k, *v;
  int32_t* err;
  int T;
};
cudaError_t launch_load(const LoadArgs& a, cudaStream_t st);

struct AttnArgs {
  moe_kv kv;
  moe_kv_batch batch;
  const uint16_t* q;
  uint16_t* out;
  void* ws;
  int rows, T, heads, max_new;
  float scale;
};
size_t attn_workspace_bytes(const moe_kv& kv, int rows, int T, int heads, int max_new);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st);
size_t decode_workspace_bytes(int D);
cudaError_t launch_decode(const AttnArgs& a, cudaStream_t st);
size_t prompt_workspace_bytes(int D);
cudaError_t launch_prompt(const AttnArgs& a, cudaStream_t st);

}  // namespace kv
}  // namespace moe
