// Trees of drafted tokens over the 4-bit cache: what each token sees, the path that a check keeps,
// and its keys and values moved into place.
//
// A row's n new tokens have parents of lower index, so with par(i) the parent of token i
//   depth(i) = 0 for a parent below 0, else depth(par(i)) + 1
//   seen(i) = {i} u seen(par(i))           as bits, one for each new token of the row
// Both by doubling: in round k every token knows its ancestors up to 2^k steps away and its 2^k-th
// one, takes over what that one knows and then stands 2^(k+1) steps from the next (8 rounds for 256
// tokens in a line; a round ends the loop when nobody has an ancestor that far).  A window takes
// out of seen(i) the ancestors `window` or more steps away, which are seen(the one that far), found
// on the way by jumping along the window's binary digits; but positions below `sinks` stay.
//
// The kept path starts at token 0 and goes on to the first child whose token the model chose.
// Children find their parents side by side (a minimum in shared memory), the path is then a walk
// of a few steps.
//
// All three are bound by latency: a CTA per row (and layer), a chain of dependent loads.  Measured:
// the plan of 4 trees of 16 tokens 1.6 us, of 256 trees of up to 256 through a window 4.2 us (33
// thousand tokens: eight rounds over their bits in shared memory); a path chosen and moved in 8 layers
// 3.9 us, 64 paths in 40 layers 5.7 us (two kernels each).
#include <climits>

#include "kv_common.cuh"

namespace moe {
namespace kv {
namespace {

struct TreeRow {
  int start, n, base;
  bool ok;
};
__device__ __forceinline__ TreeRow tree_row(const moe_kv_batch& batch, int T, int b) {
  TreeRow r;
  r.start = batch.q_start[b];
  r.n = batch.q_start[b + 1] - r.start;
  const int len = batch.kv_len[b];
  r.base = len - r.n;
  r.ok = r.n >= 0 && r.start >= 0 && r.n <= len && (long long)r.start + r.n <= T;
  return r;
}

// One CTA per row, a thread per token; W: words of bits.
template <int W>
__global__ void __launch_bounds__(MOE_KV_MAX_TREE) tree_plan_kernel(TreePlanArgs a) {
  constexpr int N = W * 32;
  __shared__ uint32_t s_bits[2][W][N];
  __shared__ short s_up[2][N], s_depth[2][N];
  griddep_wait();
  const int i = threadIdx.x;
  const TreeRow r = tree_row(a.batch, a.T, blockIdx.x);
  if (r.n == 0) return;
  if (!r.ok) {
    if (i == 0) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    return;
  }
  const int32_t* parent = a.parent + r.start;
  const int first = parent[0], n = r.n;
  if (n > a.max_new) {  // a chain of any length: its positions are the plan's
    if (i == 0 && first != MOE_KV_CHAIN) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    return;
  }
  int up = -1, depth = 0;
  uint32_t bits[W] = {};
  if (i < n) {
    up = first == MOE_KV_CHAIN ? i - 1 : parent[i];
    if (up < -1 || up >= i) {  // follows the cached tokens, then
      atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
      up = -1;
    }
    depth = up >= 0;
#pragma unroll
    for (int w = 0; w < W; ++w) bits[w] = w == i >> 5 ? 1u << (i & 31) : 0u;
  }
  int far = i < n && a.window > 0 ? i : -1, left = a.window, buf = 0;
  while (true) {
    s_up[buf][i] = (short)up;
    s_depth[buf][i] = (short)depth;
#pragma unroll
    for (int w = 0; w < W; ++w) s_bits[buf][w][i] = bits[w];
    if (!__syncthreads_or(up >= 0)) break;
    if ((left & 1) && far >= 0) far = s_up[buf][far];
    left >>= 1;
    if (up >= 0) {
      depth += s_depth[buf][up];
#pragma unroll
      for (int w = 0; w < W; ++w) bits[w] |= s_bits[buf][w][up];
      up = s_up[buf][up];
    }
    buf ^= 1;
  }
  if (left) far = -1;  // further than anybody's first ancestor
  if (far >= 0) {
    // of the tokens out of the window, those at positions below the sinks' end stay
    const int stay = a.sinks - r.base;  // by their depth
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint32_t out = s_bits[buf][w][far];
      if (stay > 0)
        for (uint32_t x = out; x; x &= x - 1) {
          const int bit = __ffs(x) - 1;
          if (s_depth[buf][w * 32 + bit] < stay) out &= ~(1u << bit);
        }
      bits[w] &= ~out;
    }
  }
  if (i < n) a.batch.pos[r.start + i] = r.base + depth;
  const int words = a.words;
  if constexpr (W <= 2) {
    if (i >= n) return;
    uint32_t* to = a.seen + (size_t)(r.start + i) * words;
    to[0] = (uint32_t)depth;
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (w + 1 < words) to[w + 1] = bits[w];
  } else {
    // many words go out in order, a warp's 32 tokens at a time, by way of the other buffer (whose
    // bits nobody reads any more): 256 trees of up to 256 tokens 4.2 us, 4.6 a token per thread
    const int lane = i & 31, first_token = i & ~31;
    uint32_t* out = &s_bits[buf ^ 1][0][0] + first_token * W;
#pragma unroll
    for (int w = 0; w < W; ++w) out[lane * W + (w + lane) % W] = bits[w];
    __syncwarp();
    uint32_t* to = a.seen + (size_t)(r.start + first_token) * words;
    const int inv = (65536 + words - 1) / words;  // x * inv >> 16 = x / words for x < 288
    for (int k = lane; k < min(32, n - first_token) * words; k += 32) {
      const int j = k * inv >> 16, w = k - j * words;
      to[k] = w ? out[j * W + (w - 1 + j) % W] : (uint32_t)s_depth[buf][first_token + j];
    }
  }
}

// One CTA per row.
__global__ void __launch_bounds__(MOE_KV_MAX_TREE) tree_accept_kernel(TreeAcceptArgs a) {
  __shared__ int s_child[MOE_KV_MAX_TREE], s_path[MOE_KV_MAX_TREE], s_kept;
  griddep_wait();
  const int i = threadIdx.x, b = blockIdx.x;
  const TreeRow r = tree_row(a.batch, a.T, b);
  const int n = r.n;
  if (n == 0 || !r.ok) {
    if (i == 0) {
      if (n) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
      a.kept[b] = a.drop[b] = 0;
      a.last[b] = -1;
    }
    return;
  }
  const int32_t *parent = a.parent + r.start, *next = a.next + r.start;
  const int first = parent[0];
  if (first == MOE_KV_CHAIN || n > a.max_new) {  // kept whole
    for (int k = i; k < n; k += blockDim.x) a.path[r.start + k] = k;
    if (i == 0) {
      if (first != MOE_KV_CHAIN) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
      a.kept[b] = n;
      a.drop[b] = 0;
      a.last[b] = next[n - 1];
    }
    return;
  }
  s_child[i] = INT_MAX;
  __syncthreads();
  if (i < n) {
    const int up = parent[i];
    if (up < -1 || up >= i)
      atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    else if (up >= 0 && a.token[r.start + i] == next[up])
      atomicMin(&s_child[up], i);
  }
  __syncthreads();
  if (i == 0) {  // (children have higher indexes: the walk ends)
    int kept = 0, at = 0;
    while (at != INT_MAX) {
      s_path[kept++] = at;
      at = s_child[at];
    }
    s_kept = kept;
    a.kept[b] = kept;
    a.drop[b] = kept - n;
    a.last[b] = next[s_path[kept - 1]];
  }
  __syncthreads();
  if (i < n) a.path[r.start + i] = i < s_kept ? s_path[i] : -1;
}

// A warp per row, layer and kv head: 8 tokens at a time, all of their bytes read before any is
// written.  Sources lie behind their places and both ascend, so what is written is never read again.
constexpr int kKeepWarps = 4;

template <int D>
__global__ void __launch_bounds__(kKeepWarps * 32) tree_keep_kernel(TreeKeepArgs a) {
  constexpr int G = D / 64, kChunks = D / 16;  // 16-byte chunks of a token's codes, K's and V's
  griddep_wait();
  const int lane = threadIdx.x & 31, b = blockIdx.x;
  const int head = blockIdx.z * kKeepWarps + (threadIdx.x >> 5);
  if (head >= a.kv_heads) return;
  const TreeRow r = tree_row(a.batch, a.T, b);
  const int kept = a.kept[b];
  if (kept == r.n && (r.ok || kept == 0)) return;  // all of them, where they are
  const bool flag = blockIdx.y == 0 && head == 0 && lane == 0;
  if (!r.ok || kept < 0 || kept > r.n) {
    if (flag) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    return;
  }
  const int32_t *path = a.path + r.start, *slot = a.batch.slot + r.start;
  // the path ascends within the row, or nothing moves
  bool bad = false, moves = false;
  for (int k = lane; k < kept; k += 32) {
    const int p = path[k], before = k ? path[k - 1] : -1;
    bad |= p <= before || p >= r.n;
    moves |= p != k;
  }
  if (__any_sync(~0u, bad)) {
    if (flag) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    return;
  }
  if (!__any_sync(~0u, moves)) return;
  const int P = a.block_tokens, p_shift = 31 - __clz(P);
  uint8_t* pool = a.pool[blockIdx.y];
  for (int k0 = 0; k0 < kept; k0 += 8) {
    // lanes 0-7: the tokens' sources, 8-15: their places
    int from = -1;
    bool live = false;
    if (lane < 16 && k0 + (lane & 7) < kept) {
      const int k = k0 + (lane & 7), p = path[k];
      live = p != k;
      from = slot[lane < 8 ? p : k];
    }
    // (slots below 2^31)
    const bool inside = from >= 0 && (from >> p_shift) < a.num_blocks;
    uint32_t there = __ballot_sync(~0u, live && inside);
    if (__any_sync(~0u, live && !inside) && flag) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    there &= there >> 8;  // both ends
    auto tile_of = [&](int s) {
      return (((int64_t)(s >> p_shift) * a.kv_heads + head) * (P / kTile) + (s & (P - 1)) / kTile) *
             tile_bytes(D);
    };
    auto chunk_at = [&](int s, int c) {  // K's chunks, then V's
      const int key = s & 15, v = c >= kChunks / 2, j = c - v * (kChunks / 2);
      return tile_of(s) + v * 8 * D + key * (D / 2) + ((j ^ swizzle<D>(key)) << 4);
    };
    auto meta_at = [&](int s, int e) {  // scale and bias of K by group, then V's
      const int key = s & 15, g = e % G, part = e / G;
      return tile_of(s) + 16 * D +
             2 * (part < 2 ? part * 16 * G + key * G + g : part * 16 * G + g * 16 + key);
    };
    uint4 code[kChunks / 4];
    uint16_t meta[G];
#pragma unroll
    for (int i = 0; i < kChunks / 4; ++i) {
      const int at = i * 32 + lane, k = at / kChunks;
      const int s = __shfl_sync(~0u, from, k);
      if ((there >> k) & 1u) code[i] = *reinterpret_cast<const uint4*>(pool + chunk_at(s, at % kChunks));
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int at = i * 32 + lane, k = at / (4 * G);
      const int s = __shfl_sync(~0u, from, k);
      if ((there >> k) & 1u) meta[i] = *reinterpret_cast<const uint16_t*>(pool + meta_at(s, at % (4 * G)));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunks / 4; ++i) {
      const int at = i * 32 + lane, k = at / kChunks;
      const int s = __shfl_sync(~0u, from, k + 8);
      if ((there >> k) & 1u) *reinterpret_cast<uint4*>(pool + chunk_at(s, at % kChunks)) = code[i];
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int at = i * 32 + lane, k = at / (4 * G);
      const int s = __shfl_sync(~0u, from, k + 8);
      if ((there >> k) & 1u) *reinterpret_cast<uint16_t*>(pool + meta_at(s, at % (4 * G))) = meta[i];
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t st) {
  const int w = (a.max_new + 31) / 32;
  auto go = [&](auto kernel, int words) {
    return launch_pdl(kernel, dim3(a.rows), dim3(words * 32), 0, st, a);
  };
  return w <= 1 ? go(tree_plan_kernel<1>, 1)
                : w <= 2 ? go(tree_plan_kernel<2>, 2)
                         : w <= 4 ? go(tree_plan_kernel<4>, 4) : go(tree_plan_kernel<8>, 8);
}

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t st) {
  const int threads = (a.max_new + 31) / 32 * 32;
  return launch_pdl(tree_accept_kernel, dim3(a.rows), dim3(threads), 0, st, a);
}

cudaError_t launch_tree_keep(const TreeKeepArgs& a, int D, cudaStream_t st) {
  const dim3 grid(a.rows, a.layers, (a.kv_heads + kKeepWarps - 1) / kKeepWarps);
  const dim3 block(kKeepWarps * 32);
  return D == 256 ? launch_pdl(tree_keep_kernel<256>, grid, block, 0, st, a)
                  : D == 128 ? launch_pdl(tree_keep_kernel<128>, grid, block, 0, st, a)
                             : launch_pdl(tree_keep_kernel<64>, grid, block, 0, st, a);
}

}  // namespace kv
}  // namespace moe
