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
// Causal rows of up to this many queries per kv head (new tokens x query heads on
// it) go through the decode kernel, longer ones through the prompt kernel
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
  // what a token sees (the kernels with View): the last `window` positions (0: all) and those
  // below `sinks`; the visibility of trees of up to tree_max tokens, `words` of a token
  int window, sinks, tree_max, words;
  const uint32_t* tree;
  // View: 0 if all rows are the decode kernel's; which kernel takes which rows (RowsMode), which the
  // decode kernel finds and the prompt kernel reads
  int prompts;
  int* mode;
};

// What a row's new tokens see of its keys, in whole tiles: the first sink_tiles tiles, then those
// from the first position of the window on.  The kernels walk a row without the gap between
// them: tile t of the walk is the row's tile t, or t + gap behind the sinks.
struct Sight {
  int sink_tiles, gap;
  __device__ __forceinline__ int tile(int t) const { return t < sink_tiles ? t : t + gap; }
};
// first: the first position that the window leaves to any of the tokens (below 0: all of them)
__device__ __forceinline__ Sight sight_of(const AttnArgs& a, int first) {
  Sight s;
  s.sink_tiles = a.sinks / kTile + (a.sinks % kTile != 0);
  s.gap = max(0, max(first, 0) / kTile - s.sink_tiles);
  return s;
}
__host__ __device__ constexpr int decode_warps(int D) { return D == 256 ? 8 : 16; }
__host__ __device__ constexpr int decode_unit_cost(int D) { return D == 64 ? 8 : 4; }

constexpr int kModeWord = 5;  // of the workspace: in the padding of the decode kernel's first Cut

// A row's new tokens and keys, if its bounds are consistent.
struct RowBounds {
  int start, n, len;
  bool ok;
};
__device__ __forceinline__ RowBounds row_bounds(const AttnArgs& a, int b) {
  RowBounds i;
  i.start = a.batch.q_start[b];
  i.n = a.batch.q_start[b + 1] - i.start;
  i.len = a.batch.kv_len[b];
  i.ok = i.start >= 0 && i.n > 0 && i.n <= a.max_new && i.n <= i.len &&
         (long long)i.len <= (long long)a.kv.max_blocks * a.kv.block_tokens &&
         (long long)i.start + i.n <= a.T;
  return i;
}

// With windows and trees, which kernel takes which rows goes by the whole batch: all rows through
// the decode kernel, all through the prompt kernel, or those of up to view_cols columns and the
// others, by what takes least time.  Times are modelled (10 ps a key tile of a unit, a fixed part),
// with numbers fitted to measured shapes (microseconds, decode | prompt; trees without a window, rows
// x keys; over 215 shapes the choice is 1% above the faster kernel on average).  It loses most where both
// take about as long and the other kernel's idle launch (6 us) comes on top: 34% with one row of 30000 keys and
// 64 columns (head_dim 256, 8 heads on one of 2: 50, 37 through the decode kernel alone), 30% with 64 rows of 1000
// keys and 24 columns (the same heads: 47, 36 through the prompt kernel), 25% with 16 rows of 1000 keys and 32
// columns (head_dim 128, 4 heads on one of 8: 40, 32 through the prompt kernel):
//   head_dim 256, 8 heads on one of 2    16 columns   24        64        256
//     1 x 2000                          14 | 22   14 | 22    15 | 25   21 | 27
//     16 x 1000                         17 | 24   19 | 25    33 | 27  101 | 32
//     64 x 4000                         64 | 82   90 | 82   200 | 84  727 | 148
//   head_dim 128, 8 on one of 4
//     1 x 2000                          17 | 20   17 | 20    17 | 22   24 | 29
//     16 x 1000                         20 | 26   21 | 27    34 | 28   88 | 38
//     64 x 4000                         71 | 102  98 | 100  224 | 103 791 | 138
//   head_dim 64, 8 on one of 8
//     1 x 2000                          14 | 21   15 | 21    15 | 21   24 | 28
//     16 x 1000                         19 | 28   22 | 28    39 | 29  105 | 38
//     64 x 4000                         78 | 140 106 | 140  243 | 142 860 | 210
__host__ __device__ constexpr int view_cols(int D) { return D == 256 ? 16 : D == 128 ? 24 : 32; }
__host__ __device__ constexpr long long decode_tile_cost(int D) { return D == 256 ? 55 : D == 128 ? 35 : 30; }
constexpr long long kPromptTileCost = 90;
__host__ __device__ constexpr int prompt_unit_tiles(int D) { return D == 128 ? 48 : 32; }
constexpr long long kDecodeFixed = 1950000;
// The host, which knows the rows' number and bounds but not their lengths, leaves the prompt kernel
// out where the decode kernel's part of such rows is at most this: an idle launch of the prompt
// kernel costs 6 to 8 us (12 with cold caches), rows that it would have taken sooner at most about 3.
// Without a window rows are as long as the block table is wide (a tree of 16 tokens on 1000 keys, 16 heads on 2 of
// 256: 14 us with a table of up to 10800 tokens, 20.6 with a wider one).
constexpr long long kDecodeAlone = 1200000;
constexpr long long kPromptFixed = 2200000, kBothFixed = 900000;
enum RowsMode { kByColumns, kAllDecode, kAllPrompt };

__host__ __device__ inline long long decode_cost(int D, int kv_heads, long long units, long long tiles) {
  return decode_tile_cost(D) * kv_heads * units * (tiles + decode_unit_cost(D));
}

struct BatchCost {
  long long decode, columns, prompt;  // all rows through one kernel, by columns, through the other
  bool few, many;                     // rows of up to view_cols columns, of more
};
__device__ __forceinline__ void add_row(const AttnArgs& a, const RowBounds& i, int r, BatchCost& c) {
  if (!i.ok) return;
  const int D = a.kv.head_dim, K = a.kv.kv_heads;
  const int gap = a.window > 0 ? sight_of(a, i.len - i.n - a.window + 1).gap : 0;
  const long long tiles = (i.len + kTile - 1) / kTile - gap, cols = (long long)i.n * r;
  const int per_tile = 128 / r, tok = D == 256 || a.max_new * (long long)r <= 128 ? per_tile : 2 * per_tile;
  const long long d = decode_cost(D, K, (cols + 7) / 8, tiles);
  const long long p = kPromptTileCost * K * ((i.n + tok - 1) / tok) * (tiles + prompt_unit_tiles(D));
  const bool few = cols <= view_cols(D);
  c.decode += d;
  c.prompt += p;
  c.columns += few ? d : p;
  c.few |= few;
  c.many |= !few;
}
__device__ __forceinline__ int mode_of(const BatchCost& c) {
  if (!c.many) return kAllDecode;
  const long long d = kDecodeFixed + c.decode, p = kPromptFixed + c.prompt;
  const long long m = kPromptFixed + (c.few ? kBothFixed : 0) + c.columns;
  return d <= p && d <= m ? kAllDecode : m <= p ? kByColumns : kAllPrompt;
}
// over a warp's rows, one a lane
__device__ __forceinline__ BatchCost warp_sum(BatchCost c) {
  c.many = __any_sync(~0u, c.many);
  if (!c.many) return c;
  c.few = __any_sync(~0u, c.few);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    c.decode += __shfl_xor_sync(~0u, c.decode, o);
    c.columns += __shfl_xor_sync(~0u, c.columns, o);
    c.prompt += __shfl_xor_sync(~0u, c.prompt, o);
  }
  return c;
}
// of up to 32 rows, for a warp (i: its lane's row); of more, for a CTA
__device__ __forceinline__ int warp_mode(const AttnArgs& a, const RowBounds& i, int r) {
  if (!a.prompts) return kAllDecode;
  BatchCost c = {};
  add_row(a, i, r, c);
  return mode_of(warp_sum(c));
}
__device__ __forceinline__ int block_mode(const AttnArgs& a, int r) {
  __shared__ unsigned long long s_cost[3];
  if (!a.prompts) return kAllDecode;
  BatchCost c = {};
  for (int b = threadIdx.x; b < a.rows; b += blockDim.x) add_row(a, row_bounds(a, b), r, c);
  if (threadIdx.x < 3) s_cost[threadIdx.x] = 0;
  c.many = __syncthreads_or(c.many) != 0;
  if (!c.many) return kAllDecode;
  c.few = __syncthreads_or(c.few) != 0;
  c = warp_sum(c);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&s_cost[0], (unsigned long long)c.decode);
    atomicAdd(&s_cost[1], (unsigned long long)c.columns);
    atomicAdd(&s_cost[2], (unsigned long long)c.prompt);
  }
  __syncthreads();
  c.decode = (long long)s_cost[0];
  c.columns = (long long)s_cost[1];
  c.prompt = (long long)s_cost[2];
  return mode_of(c);
}

// Whether a row of n new tokens is the decode kernel's.
template <bool View>
__device__ __forceinline__ bool takes_decode(const AttnArgs& a, int n, int r, int mode) {
  if constexpr (View)
    return mode == kAllDecode || (mode == kByColumns && (long long)n * r <= view_cols(a.kv.head_dim));
  return (long long)n * r <= decode_cols(a.kv.head_dim);
}

// of 16 keys, those below the x-th
__device__ __forceinline__ uint32_t below16(int x) {
  return x >= 16 ? 0xFFFFu : x <= 0 ? 0u : (1u << x) - 1u;
}
// for either kind of call, or (view false) for causal ones
size_t attn_workspace_bytes(const moe_kv& kv, int heads, int max_new, bool view);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st);
size_t decode_workspace_bytes(int D);
cudaError_t launch_decode(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_decode_view(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_decode_join(const AttnArgs& a, cudaStream_t st);  // of units cut between CTAs
size_t prompt_workspace_bytes(int D);
cudaError_t launch_prompt(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_prompt_view(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_prompt_join(const AttnArgs& a, cudaStream_t st);

struct TreePlanArgs {
  moe_kv_batch batch;
  const int32_t* parent;
  uint32_t* seen;
  int rows, T, max_new, words, window, sinks;
};
cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t st);

struct TreeAcceptArgs {
  moe_kv_batch batch;
  const int32_t *parent, *token, *next;
  int32_t *path, *kept, *drop, *last;
  int rows, T, max_new;
};
cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t st);

constexpr int kKeepLayers = 128;  // layers of one launch: their pools go by value
struct TreeKeepArgs {
  moe_kv_batch batch;
  const int32_t *path, *kept;
  int rows, T, num_blocks, block_tokens, kv_heads, layers;
  uint8_t* pool[kKeepLayers];
};
cudaError_t launch_tree_keep(const TreeKeepArgs& a, int head_dim, cudaStream_t st);

}  // namespace kv
}  // namespace moe
