// Block tables and slot maps of the 4-bit key/value cache, from request
// lengths on the device: no length, block id or slot ever visits the host, so
// a decode loop over a growing cache can be one captured graph.
//
// Per row b with len = seq_len[b], n = new_len[b], P tokens a block:
//   kept = max(0, len + min(n, 0)), grown = kept + max(n, 0)
//   blocks ceil(kept / P) .. ceil(len / P) - 1 go back to the free list,
//   blocks ceil(kept / P) .. ceil(grown / P) - 1 are taken from its end,
// both ranked over all rows in (row, block) order: rank k goes to (comes from)
// place count - 1 - k, so blocks given back come out again in the same order.
// Exclusive scans over the rows give the ranks and q_start; token t of row b
// sits at position kept + (t - q_start[b]).  Block ids are moved as they are; one
// outside the pool (no plan writes such a table) is flagged when it is moved or
// mapped, and its tokens get a slot that every reader of slots flags and skips.
//
// Bound by latency: one CTA scans the rows (1024 at a time: up to that many are
// read once and kept in registers) and moves the blocks, a thread per block
// wherever its row is (binary search in the shared ranks).  The slot map of up
// to kInline tokens follows in the same kernel, a longer one in a second kernel
// over all SMs, whose CTAs search q_start in shared memory, four tokens a thread.
// Measured: 64 rows, one token each, taken and dropped again (two calls) 7.3 us;
// 256 rows with 90000 new tokens in 5600 blocks, and dropped again, 18.0 us.
#include <climits>

#include "kv_common.cuh"

namespace moe {
namespace kv {
namespace {

constexpr int kThreads = 1024;
// Tokens that the first kernel maps itself (two calls, in it | in a second kernel: 2700 tokens
// 8.9 | 9.5 us, 5300 tokens 10.2 | 9.3, 22000 tokens 20.2 | 9.3).
constexpr int kInline = 4096;
constexpr int kMapRows = 8192;   // rows whose q_start fits the map kernel's shared memory

struct Row {
  int h0, h1, h2;  // blocks held before, kept, held after
  int kept, add;   // tokens kept, tokens added
  bool bad;        // does not fit the block table
};

__device__ __forceinline__ Row row_of(const PlanArgs& a, int b) {
  Row r = {};
  if (b >= a.rows) return r;
  const int P = a.kv.block_tokens, p_shift = 31 - __clz(P);
  const long long cap = (long long)a.kv.max_blocks * P;  // < 2^31
  const int len = max(0, min(a.kv.seq_len[b], (int)cap));
  const int n = a.new_len[b];
  r.kept = n < 0 ? (int)max(0ll, (long long)len + n) : len;
  r.add = max(n, 0);
  r.bad = (long long)r.kept + r.add > cap;
  if (r.bad) r.add = 0;
  auto blocks = [&](int x) { return (int)(((long long)x + P - 1) >> p_shift); };
  r.h0 = blocks(len);
  r.h1 = blocks(r.kept);
  r.h2 = blocks(r.kept + r.add);
  return r;
}

// Three inclusive scans of one value per thread over the CTA; s: [3][32], whose last entries are
// the totals afterwards.
struct Three {
  long long v[3];
};
__device__ __forceinline__ Three block_scan(Three x, long long (*s)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long u = __shfl_up_sync(~0u, x.v[i], o);
      if (lane >= o) x.v[i] += u;
    }
  __syncthreads();  // the last call's totals have been read
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i][w] = x.v[i];
  __syncthreads();
  if (w < 3) {
    long long t = s[w][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, t, o);
      if (lane >= o) t += u;
    }
    s[w][lane] = t;
  }
  __syncthreads();
  if (w)
#pragma unroll
    for (int i = 0; i < 3; ++i) x.v[i] += s[i][w - 1];
  return x;
}

// The last of n ascending values that is <= k (the first one is).
__device__ __forceinline__ int last_below(const int* v, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void map_token(const PlanArgs& a, int t, int row, int start, int end,
                                          int len, int& slot, int& pos) {
  const int P = a.kv.block_tokens, p_shift = 31 - __clz(P);
  pos = len - (end - start) + (t - start);
  const int block = a.kv.block_table[(int64_t)row * a.kv.max_blocks + (pos >> p_shift)];
  slot = (block << p_shift) + (pos & (P - 1));
  if ((unsigned)block >= (unsigned)a.kv.num_blocks) {
    slot = INT_MIN;
    atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
  }
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a) {
  __shared__ long long s_scan[3][32];
  __shared__ int s_back[kThreads], s_need[kThreads], s_first[kThreads], s_start[kThreads + 1];
  __shared__ int s_len[kThreads];
  __shared__ int s_bad;
  const int tid = threadIdx.x, B = a.rows, W = a.kv.max_blocks;
  const bool one = B <= kThreads;
  if (tid == 0) s_bad = 0;
  griddep_wait();
  const int free_count = *a.kv.free_count;
  Row r = row_of(a, tid);
  __syncthreads();
  // totals decide whether the step fits; a step that does not adds nothing
  long long back = 0, need = 0, tokens = 0;
  for (int b = tid; b < B; b += kThreads) {
    const Row x = one ? r : row_of(a, b);
    back += x.h0 - x.h1;
    need += x.h2 - x.h1;
    tokens += x.add;
    if (x.bad) s_bad = 1;
  }
  const Three all = block_scan({{back, need, tokens}}, s_scan);
  const long long total_back = s_scan[0][31], total_need = s_scan[1][31],
                  total_tokens = s_scan[2][31];
  const int had = min(max(free_count, 0), a.kv.num_blocks);
  // tables that hold more blocks than the pool has are not the library's own
  const bool broken = had + total_back > a.kv.num_blocks;
  const bool refused = s_bad || broken || total_need > had + total_back ||
                       total_tokens > a.batch.max_tokens;
  const int count1 = broken ? had : had + (int)total_back;
  if (tid == 0) {
    if (refused) atomicOr(a.batch.err, MOE_DERR_KV_FULL | (broken ? MOE_DERR_KV_INDEX : 0));
    if (!broken) *a.kv.free_count = count1 - (refused ? 0 : (int)total_need);
    a.batch.q_start[0] = 0;
  }
  // Blocks given back, a chunk of rows at a time (all of it before any is taken), then blocks
  // taken, lengths and q_start.
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 0 && (broken || total_back == 0)) continue;
    long long carry[3] = {0, 0, 0};
    for (int b0 = 0; b0 < B; b0 += kThreads) {
      const int b = b0 + tid;
      Three inc = all;
      if (!one) {
        r = row_of(a, b);
        inc = block_scan({{r.h0 - r.h1, r.h2 - r.h1, r.add}}, s_scan);
      }
      const int add = refused ? 0 : r.add;
      __syncthreads();
      s_back[tid] = (int)(carry[0] + inc.v[0]) - (r.h0 - r.h1);
      s_need[tid] = (int)(carry[1] + inc.v[1]) - (r.h2 - r.h1);
      s_first[tid] = r.h1;
      if (pass == 1) {
        const int end = refused ? 0 : (int)(carry[2] + inc.v[2]);
        s_start[tid] = end - add;
        s_len[tid] = r.kept + add;
        if (b < B) {
          a.batch.q_start[b + 1] = end;
          a.batch.kv_len[b] = r.kept + add;
          if (!broken) a.kv.seq_len[b] = r.kept + add;
        }
      }
      __syncthreads();
      const int* rank = pass == 0 ? s_back : s_need;
      const long long from = carry[pass], to = carry[pass] + s_scan[pass][31];
      if (!(pass == 1 && refused)) {
        // four blocks of a thread on their way at a time
        bool outside = false;
        for (int k0 = (int)from + tid; k0 < (int)to; k0 += 4 * kThreads) {
          int32_t *src[4], *dst[4], v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = k0 + j * kThreads;
            if (k < (int)to) {
              const int i = last_below(rank, kThreads, k);
              int32_t* entry = a.kv.block_table + (int64_t)(b0 + i) * W + s_first[i] + (k - rank[i]);
              int32_t* place = a.kv.free_list + (count1 - 1 - k);
              src[j] = pass == 0 ? entry : place;
              dst[j] = pass == 0 ? place : entry;
              v[j] = *src[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k0 + j * kThreads < (int)to) {
              *dst[j] = v[j];
              if (pass == 0) *src[j] = -1;
              outside |= (unsigned)v[j] >= (unsigned)a.kv.num_blocks;
            }
        }
        if (outside) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
      }
      for (int i = 0; i < 3; ++i) carry[i] += s_scan[i][31];
    }
    __syncthreads();
  }
  if (a.batch.max_tokens > kInline) {
    griddep_launch();
    return;
  }
  const int T = refused ? 0 : (int)total_tokens;
  for (int t = tid; t < a.batch.max_tokens; t += kThreads) {
    int slot = -1, pos = 0;
    if (t < T) {
      if (one) {
        const int i = last_below(s_start, B, t);
        map_token(a, t, i, s_start[i], i + 1 < B ? s_start[i + 1] : T, s_len[i], slot, pos);
      } else {
        const int i = last_below(a.batch.q_start, B, t);
        map_token(a, t, i, a.batch.q_start[i], a.batch.q_start[i + 1], a.batch.kv_len[i], slot, pos);
      }
    }
    a.batch.slot[t] = slot;
    a.batch.pos[t] = pos;
  }
}

// The slot map of many tokens; `wide`: slot and pos take four entries at a time.
__global__ void __launch_bounds__(512) map_kernel(PlanArgs a, int wide) {
  extern __shared__ int s_start[];  // [rows + 1], for up to kMapRows rows
  const int B = a.rows;
  griddep_wait();
  const int* start = a.batch.q_start;
  if (B <= kMapRows) {
    for (int i = threadIdx.x; i <= B; i += blockDim.x) s_start[i] = a.batch.q_start[i];
    __syncthreads();
    start = s_start;
  }
  const int T = start[B], all = a.batch.max_tokens;
  const int step = gridDim.x * blockDim.x * 4;
  // (64 bits: the last step of a thread may pass 2^31)
  for (int64_t at = (blockIdx.x * blockDim.x + threadIdx.x) * 4; at < all; at += step) {
    const int t0 = (int)at;
    int slot[4], pos[4], row = t0 < T ? last_below(start, B, t0) : B;
    int len = row < B ? a.batch.kv_len[row] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      slot[i] = -1;
      pos[i] = 0;
      if (i < T - t0) {
        while (start[row + 1] <= t0 + i) len = a.batch.kv_len[++row];
        map_token(a, t0 + i, row, start[row], start[row + 1], len, slot[i], pos[i]);
      }
    }
    if (wide && all - t0 >= 4) {
      *reinterpret_cast<int4*>(a.batch.slot + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.batch.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int i = 0; i < 4 && i < all - t0; ++i) {
        a.batch.slot[t0 + i] = slot[i];
        a.batch.pos[t0 + i] = pos[i];
      }
    }
  }
}

__global__ void reset_kernel(moe_kv kv) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t k = i; k < (int64_t)kv.max_rows * kv.max_blocks; k += step) kv.block_table[k] = -1;
  for (int64_t k = i; k < kv.num_blocks; k += step) kv.free_list[k] = kv.num_blocks - 1 - (int)k;
  for (int64_t k = i; k < kv.max_rows; k += step) kv.seq_len[k] = 0;
  if (i == 0) *kv.free_count = kv.num_blocks;
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_pdl(plan_kernel, dim3(1), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess || a.batch.max_tokens <= kInline) return e;
  const int wide = ((reinterpret_cast<uintptr_t>(a.batch.slot) |
                     reinterpret_cast<uintptr_t>(a.batch.pos)) & 15) == 0;
  const int ctas = (int)min((int64_t)2 * kGrid, ((int64_t)a.batch.max_tokens + 2047) / 2048);
  const size_t smem = a.rows <= kMapRows ? sizeof(int) * (a.rows + 1) : 0;
  return launch_pdl(map_kernel, dim3(ctas), dim3(512), smem, st, a, wide);
}

cudaError_t launch_reset(const moe_kv& kv, cudaStream_t st) {
  reset_kernel<<<152, 256, 0, st>>>(kv);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace moe
