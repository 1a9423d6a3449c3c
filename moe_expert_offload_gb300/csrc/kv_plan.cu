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
// sits at position kept + (t - q_start[b]).
//
// Bound by latency: a few dependent passes over the rows by one CTA.
#include "kv_common.cuh"

namespace moe {
namespace kv {
namespace {

constexpr int kThreads = 1024;

struct Row {
  int h0, h1, h2;  // blocks held before, kept, held after
  int kept, add;   // tokens kept, tokens added
  bool bad;        // does not fit the block table
};

__device__ __forceinline__ Row row_of(const PlanArgs& a, int b) {
  Row r;
  const int P = a.kv.block_tokens;
  const long long cap = (long long)a.kv.max_blocks * P;
  const int len = max(0, min(a.kv.seq_len[b], (int)min(cap, 0x7fffffffll)));
  const int n = a.new_len[b];
  r.kept = n < 0 ? (int)max(0ll, (long long)len + n) : len;
  r.add = max(n, 0);
  r.bad = (long long)r.kept + r.add > cap;
  if (r.bad) r.add = 0;
  r.h0 = (int)(((long long)len + P - 1) / P);
  r.h1 = (int)(((long long)r.kept + P - 1) / P);
  r.h2 = (int)(((long long)r.kept + r.add + P - 1) / P);
  return r;
}

// Inclusive scan of one value per thread over the CTA; s: 32 words.
__device__ __forceinline__ long long block_scan(long long v, long long* s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s[w] = v;
  __syncthreads();
  if (w == 0) {
    long long t = s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, t, o);
      if (lane >= o) t += u;
    }
    s[lane] = t;
  }
  __syncthreads();
  if (w) v += s[w - 1];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a) {
  __shared__ long long s_scan[32];
  __shared__ int s_rank[kThreads + 1];  // ranks of the chunk's rows, then their sum
  __shared__ int s_first[kThreads];     // first block index of each row's run
  __shared__ int s_bad;
  const int tid = threadIdx.x, B = a.rows, W = a.kv.max_blocks;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // totals decide whether the step fits; a step that does not adds nothing
  long long back = 0, need = 0, tokens = 0;
  for (int b = tid; b < B; b += kThreads) {
    const Row r = row_of(a, b);
    back += r.h0 - r.h1;
    need += r.h2 - r.h1;
    tokens += r.add;
    if (r.bad) s_bad = 1;
  }
  const int had = min(max(*a.kv.free_count, 0), a.kv.num_blocks);
  block_scan(back, s_scan);
  const long long total_back = s_scan[31];
  __syncthreads();
  block_scan(need, s_scan);
  const long long total_need = s_scan[31];
  __syncthreads();
  block_scan(tokens, s_scan);
  const long long total_tokens = s_scan[31];
  __syncthreads();
  // tables that hold more blocks than the pool has are not the library's own
  const bool broken = had + total_back > a.kv.num_blocks;
  const bool refused = s_bad || broken || total_need > had + total_back ||
                       total_tokens > a.batch.max_tokens;
  const int count1 = broken ? had : had + (int)total_back;
  if (tid == 0) {
    if (broken) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    if (refused) atomicOr(a.batch.err, MOE_DERR_KV_FULL);
  }
  // give back, then take; each pass ranks a chunk of rows at a time
  for (int pass = broken ? 2 : 0; pass < 2; ++pass) {
    if (pass == 1 && refused) break;
    if ((pass == 0 ? total_back : total_need) == 0) continue;
    int carry = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
      const int b = b0 + tid;
      int n = 0, first = 0;
      if (b < B) {
        const Row r = row_of(a, b);
        first = r.h1;
        n = pass == 0 ? r.h0 - r.h1 : r.h2 - r.h1;
      }
      const int inc = (int)block_scan(n, s_scan);
      s_rank[tid] = inc - n;
      s_first[tid] = first;
      if (tid == kThreads - 1) s_rank[kThreads] = inc;
      __syncthreads();
      const int total = s_rank[kThreads];
      for (int k = tid; k < total; k += kThreads) {
        int lo = 0, hi = kThreads;  // the last row whose rank is <= k
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_rank[mid] <= k) lo = mid;
          else hi = mid;
        }
        int32_t* entry = a.kv.block_table + (int64_t)(b0 + lo) * W + s_first[lo] + (k - s_rank[lo]);
        int32_t* place = a.kv.free_list + (count1 - 1 - carry - k);
        if (pass == 0) {
          *place = *entry;
          *entry = -1;
        } else {
          *entry = *place;
        }
      }
      carry += total;
      __syncthreads();
    }
  }
  // lengths and q_start
  long long carry = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    Row r;
    r.add = 0;
    if (b < B) {
      r = row_of(a, b);
      if (refused) r.add = 0;
    }
    const long long inc = block_scan(r.add, s_scan) + carry;
    carry += s_scan[31];
    __syncthreads();
    if (b < B) {
      if (b == 0) a.batch.q_start[0] = 0;
      a.batch.q_start[b + 1] = (int)inc;
      a.batch.kv_len[b] = r.kept + r.add;
      if (!broken) a.kv.seq_len[b] = r.kept + r.add;
    }
  }
  if (tid == 0 && !broken) *a.kv.free_count = count1 - (refused ? 0 : (int)total_need);
  __syncthreads();
  const int T = refused ? 0 : (int)total_tokens, P = a.kv.block_tokens;
  for (int t = tid; t < a.batch.max_tokens; t += kThreads) {
    int slot = -1, at = 0;
    if (t < T) {
      int lo = 0, hi = B;  // the last row whose q_start is <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.batch.q_start[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int n = a.batch.q_start[lo + 1] - a.batch.q_start[lo];
      at = a.batch.kv_len[lo] - n + (t - a.batch.q_start[lo]);
      slot = a.kv.block_table[(int64_t)lo * W + at / P] * P + at % P;
    }
    a.batch.slot[t] = slot;
    a.batch.pos[t] = at;
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
  plan_kernel<<<1, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_reset(const moe_kv& kv, cudaStream_t st) {
  reset_kernel<<<152, 256, 0, st>>>(kv);
  return cudaGetLastError();
}

}  // namespace kv
}  // namespace moe
