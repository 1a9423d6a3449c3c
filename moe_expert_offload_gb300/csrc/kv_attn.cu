// Attention over the 4-bit key/value cache.
//
// Token i of row b's n new tokens (n = q_start[b+1] - q_start[b]) sits at
// position p = kv_len[b] - n + i and sees the keys 0 .. p of its row:
//   o = sum_j softmax_j(scale q . k_j) v_j,  k, v = scale * code + bias
// One warp per (token, query head) walks the keys once with a running maximum
// and sum; each lane owns D / 32 columns.
#include "kv_common.cuh"

namespace moe {
namespace kv {
namespace {

template <int D>
__global__ void __launch_bounds__(256) attn_simple_kernel(AttnArgs a) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int t = (int)(id / a.heads), h = (int)(id % a.heads);
  if (t >= a.T || t >= a.batch.q_start[a.rows]) return;
  int lo = 0, hi = a.rows;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.batch.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int P = a.kv.block_tokens, K = a.kv.kv_heads, kh = h / (a.heads / K);
  const int n = a.batch.q_start[lo + 1] - a.batch.q_start[lo];
  const int len = a.batch.kv_len[lo];
  if (n < 0 || n > a.max_new || n > len || len > (int64_t)a.kv.max_blocks * P ||
      a.batch.q_start[lo] < 0 || a.batch.q_start[lo] + (int64_t)n > a.T) {
    if (lane == 0) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    return;
  }
  if (n * (a.heads / K) <= kDecodeCols) return;
  const int last = len - n + (t - a.batch.q_start[lo]);
  const int64_t at = ((int64_t)t * a.heads + h) * D + lane * N;
  float q[N], o[N] = {}, m = -INFINITY, l = 0.0f;
  for (int i = 0; i < N; ++i) q[i] = __uint_as_float((uint32_t)a.q[at + i] << 16) * a.scale;
  for (int j = 0; j <= last; ++j) {
    const int block = a.kv.block_table[(int64_t)lo * a.kv.max_blocks + j / P];
    if (block < 0 || block >= a.kv.num_blocks) {
      if (lane == 0) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
      continue;
    }
    const uint8_t* tile = static_cast<const uint8_t*>(a.kv.pool) +
                          (((int64_t)block * K + kh) * (P / kTile) + j % P / kTile) * tile_bytes(D);
    const __half* meta = reinterpret_cast<const __half*>(tile + 16 * D);
    const int key = j % kTile, c0 = lane * N, g = c0 / 64;
    const int chunk = (c0 / 32) ^ swizzle<D>(key);
    const uint8_t* kc = tile + key * (D / 2) + chunk * 16 + c0 % 32 / 2;
    const float ks = __half2float(meta[Meta<D>::k_scale(key, g)]);
    const float kb = __half2float(meta[Meta<D>::k_bias(key, g)]);
    const float vs = __half2float(meta[Meta<D>::v_scale(key, g)]);
    const float vb = __half2float(meta[Meta<D>::v_bias(key, g)]);
    float x = 0.0f;
    for (int i = 0; i < N; ++i) x = fmaf(q[i], fmaf(ks, (float)((kc[i / 2] >> (4 * (i & 1))) & 15), kb), x);
    for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
    const float mm = fmaxf(m, x), f = __expf(m - mm), p = __expf(x - mm);
    m = mm;
    l = l * f + p;
    for (int i = 0; i < N; ++i)
      o[i] = o[i] * f + p * fmaf(vs, (float)((kc[8 * D + i / 2] >> (4 * (i & 1))) & 15), vb);
  }
  for (int i = 0; i < N; ++i)
    a.out[at + i] = __bfloat16_as_ushort(__float2bfloat16_rn(l > 0.0f ? o[i] / l : 0.0f));
}

}  // namespace

size_t attn_workspace_bytes(const moe_kv& kv, int, int, int, int) {
  return decode_workspace_bytes(kv.head_dim);
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t st) {
  cudaError_t e = launch_decode(a, st);
  if (e != cudaSuccess || (int64_t)a.max_new * (a.heads / a.kv.kv_heads) <= kDecodeCols) return e;
  const unsigned grid = (unsigned)(((int64_t)a.T * a.heads + 7) / 8);
  if (a.kv.head_dim == 256) attn_simple_kernel<256><<<grid, 256, 0, st>>>(a);
  else if (a.kv.head_dim == 128) attn_simple_kernel<128><<<grid, 256, 0, st>>>(a);
  else attn_simple_kernel<64><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace moe
