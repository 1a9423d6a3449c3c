// Attention over the 4-bit cache for rows of few new tokens (decode, drafts).
//
// The cache is read once and little is computed on it per byte, so the work is
// a stream: every warp of the grid takes an equal, contiguous share of
// all (row, kv head, column tile) units' key tiles, however ragged the rows are.
// A warp walks its share and keeps a private ring of bulk copies full, starting
// the next stage's the moment it has read one out, and never waits for another
// warp.  Where a unit is cut between warps or CTAs, its
// running maximum, sum and accumulator are merged afterwards, in a fixed order.
//
// A unit's queries are 8 columns, column c = (token c / r, head c % r) of the r
// query heads that share the kv head; more columns are more units, each with a
// walk of its own over the keys.  (16 columns a unit, one walk instead of two,
// took 1.3 to 2 times as long at head_dim 256, whose registers it spilled, and
// was no faster at 64; at 128, 32 columns over 60000 keys took 77 instead of 88
// us, but over 100 rows of up to 1000 keys 62 instead of 52.)  Both
// products take the codes as the A operand, 16 keys x 16 columns (or their
// transpose, by ldmatrix.trans) at a time:
//   S^T[key][col] = sum_g scale_K[key][g] (codes . q_g) + sum_g bias_K[key][g] sum(q_g)
//   O^T[dim][col] = codes^T . (p scale_V[key][g]) + sum_key p bias_V[key][g]
// Codes need no conversion: a nibble masked out in place is an fp16 subnormal,
// code * 2^-24 (low nibble of a byte) or code * 2^-20 (high nibble), which the
// tensor cores multiply exactly; the powers of two are taken back in the
// queries' fragments and in the epilogue.  The two bias sums are one MMA each
// per 16 keys (the groups' biases as A; for O together with a row of ones that
// sums p).  Queries are scaled by a power of two per column into fp16's range
// (exact but for columns 2^-29 below the largest).  p is rounded to fp16 with
// its largest value between 2^7 and 2^15, and its product with the values' scale (after a
// power of two that brings the largest scale to between 2^-3 and 1) once more: 2^-11 each
// against the output's 2^-8; products below 2^-18 of the largest weight and scale lose
// that precision to fp16's subnormals.  The maximum that p refers to, a raw score, follows
// the scores only when they pass it by 2^8, so it rarely moves.  Codes are positive and the bias takes
// their mean back, so the accumulators would grow far past the result and lose
// it to the MMA's truncating sums (measured at 128k keys: 2.1e-3 from fp64
// against 1.6e-3 for bf16 rounding alone): every 16 tiles each group's mean is
// moved from them into a rounded fp32 sum of its own.
//
// Measured: 64 rows of 150 to 8191 keys, 32 query heads on 8 of 128 (330 MB): 76.8 us,
// 4.3 TB/s; 8 rows of 130000 keys, 16 heads on 2 of 256 (598 MB): 111.5 us, 5.4 TB/s.
// The stream alone takes 54.7 and 88 us.  A tile takes 321 and 409 instructions: 80
// and 160 unpack codes (four masks per product of them, and shifts), 18 and 34 are
// MMAs, the rest is what a stage and a tile cost besides (the copies' bookkeeping,
// the scan over the values' scales, the growth test, scales and biases).  Neither
// the issue slots (57 and 43%) nor the ALU pipe (53 and 46%) are full: every warp is
// one serial chain, and 16 (8) of them on an SM do not cover it.  Spilled: 20, 44 and
// 56 bytes a thread at head_dim 64, 128 and 256.  Few keys are latency: 1000 keys of
// one row 11.6 us, about 2 of them the scan over the rows and 2.5 the combine kernel.
#include <type_traits>

#include "kv_common.cuh"
#include "stream_common.cuh"

namespace moe {
namespace kv {
namespace {

using sc::bar_expect;
using sc::bar_init;
using sc::bulk_g2s;
using sc::su32;
using sc::warp_wait;

// Warps: as many as the registers allow, which are shared out by SM quarters: 16 warps of 128
// registers or 8 of 255, by what accumulators and query fragments take (48 registers at
// head_dim 128, 96 at 256).
template <int D>
struct Cfg {
  static constexpr int kWarps = D == 256 ? 8 : 16;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTiles = D == 64 ? 4 : 2;  // key tiles of a stage
  static constexpr int kStageBytes = kTiles * tile_bytes(D);
  static constexpr int kStages = 3;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kCols = 8;
  static constexpr int kPartial = kCols * (D + 3);  // floats: o [col][D], m, l, fac [col]
  // a unit's fixed cost, in key tiles (100 rows of up to 1000 keys, us at half of it, at it and at
  // twice: head_dim 64 16.9, 16.5, 16.5; 128 30.8, 29.0, 29.0; 256 25.2, 22.3, 22.9)
  static constexpr int kUnitCost = D == 64 ? 8 : 4;
  static constexpr int kCentre = 16 / kTiles;       // stages between two moves of the mean
  static constexpr size_t kSmem = (size_t)kWarps * kWarpBytes + 128;
  static_assert(kPartial * 4 <= kStages * kStageBytes, "a partial fits its warp's ring");
};
constexpr float kNone = -1e30f;  // a maximum before the first key: finite, so that it subtracts,
                                 // and below every raw score (2^15 at most)

// workspace: cuts [kGrid] | CTA parts [kGrid][2] | warp parts [kGrid * warps]
// The unit that a CTA began and did not end: the last CTA with a part of it
// (-1: there is none).
struct Cut {
  int last, unit, start, n, ntb, pad[3];
};
constexpr size_t kCutBytes = (kGrid * sizeof(Cut) + 255) / 256 * 256;
__host__ __device__ inline float* cta_parts(void* ws) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + kCutBytes);
}

struct RowInfo {
  int start, n, len, tiles, ntb;  // ntb 0: nothing here
};

// Row b's bounds, checked; flag: report what does not fit.
__device__ __forceinline__ RowInfo row_info(const AttnArgs& a, int b, int r, int cols, bool flag) {
  RowInfo i;
  i.start = a.batch.q_start[b];
  i.n = a.batch.q_start[b + 1] - i.start;
  i.len = a.batch.kv_len[b];
  i.tiles = (i.len + kTile - 1) / kTile;
  i.ntb = 0;
  if (i.n == 0) return i;
  if (i.start < 0 || i.n < 0 || i.n > a.max_new || i.n > i.len ||
      (long long)i.len > (long long)a.kv.max_blocks * a.kv.block_tokens ||
      (long long)i.start + i.n > a.T) {
    if (flag) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
    return i;
  }
  if (i.n * r <= decode_cols(a.kv.head_dim)) i.ntb = (i.n * r + cols - 1) / cols;
  return i;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void lds64(uint32_t& x, uint32_t& y, uint32_t addr) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 h2f(uint32_t v) {
  const __half2 h = *reinterpret_cast<const __half2*>(&v);
  return __half22float2(h);
}
// four fp32 times inv as bf16
__device__ __forceinline__ void store_bf16(uint16_t* dst, float4 y, float inv) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * inv, y.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(y.z * inv, y.w * inv);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                              *reinterpret_cast<const uint32_t*>(&hi));
}
// a warp's row of D, lane by lane two columns of every 64, divided by l
template <int D>
__device__ __forceinline__ void store_row(uint16_t* dst, const float (&y)[D / 32], float l,
                                          int lane) {
  const float inv = l > 0.0f ? 1.0f / l : l;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * i] * inv, y[2 * i + 1] * inv);
    *reinterpret_cast<uint32_t*>(dst + lane * 2 + i * 64) = *reinterpret_cast<const uint32_t*>(&v);
  }
}
// 2^8 above the reference, rounded down: no weight passes 2^15 before it follows
__device__ __forceinline__ float reach(float m, float fac) { return __fadd_rd(m, __fdividef(8.0f, fac)); }
__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}

struct Part {
  int unit, start, n, ntb;  // unit -1: none
  int first;                // holds the unit's first tile
  int left;                 // key tiles of the unit behind the part
};

// What is kept of a stage between the start of its copies and its use.
struct Stage {
  int tile;
  uint32_t what;  // tiles | begin << 8 | end << 9 | last << 10 | tiles present << 16
  int unit, ntb;
  int start, n, len, pad;
};
constexpr int kLeast = -14;  // a unit's first sigma: scales are below 2^sigma
constexpr uint32_t kBegin = 1u << 8, kEnd = 1u << 9, kLast = 1u << 10;

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) decode_kernel(AttnArgs a) {
  using C = Cfg<D>;
  constexpr int G = D / 64, W = C::kWarps, TS = C::kTiles, S = C::kStages;
  constexpr int C0 = C::kUnitCost;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[W][S];
  __shared__ __align__(16) Stage s_stage[W][S];
  __shared__ int s_rows[3][C::kThreads];  // start, new tokens, length of the rows, if they fit
  __shared__ long long s_scan[W];
  __shared__ long long s_x[W];  // each warp's start: offset in the row
  __shared__ int s_row[W];      // and the row; -1: no work
  // the parts of units left by each warp, the head one (it ends a unit that an
  // earlier warp began) and the last one (it does not end its unit)
  __shared__ Part s_part[W][2];
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring0 = (su32(smem_raw) + 127u) & ~127u;
  unsigned char* rings = smem_raw + (ring0 - su32(smem_raw));
  long long* s_pre = reinterpret_cast<long long*>(rings);  // before the rings are filled
  const int K = a.kv.kv_heads, r = a.heads / K, P = a.kv.block_tokens;
  float* cta_part = cta_parts(a.ws);
  float* warp_part = cta_part + (size_t)kGrid * 2 * C::kPartial;
  if (tid < W * S) bar_init(su32(&full[0][0] + tid), 1);
  if (lane == 0) {
    s_row[wid] = -1;
    s_part[wid][0].unit = s_part[wid][1].unit = -1;
  }
  __syncwarp();
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  griddep_wait();

  // ------------------------------------------------------------- the shares
  // cost of the rows before each row
  long long total = 0, share = 0;
  const int chunks = (a.rows + C::kThreads - 1) / C::kThreads;
  auto share_of = [&] {
    return max((total + (long long)kGrid * W - 1) / ((long long)kGrid * W), (long long)TS);
  };
  if (a.rows <= 32) {
    // up to 32 rows: every warp for itself, a lane per row (1000 keys of one row: 11.4 us, 11.8
    // the other way)
    RowInfo i = {};
    if (lane < a.rows) i = row_info(a, lane, r, C::kCols, blockIdx.x == 0 && wid == 0);
    const long long cost = (long long)K * i.ntb * (i.tiles + C0);
    if (wid == 0) {
      s_rows[0][lane] = i.start;
      s_rows[1][lane] = i.ntb ? i.n : 0;
      s_rows[2][lane] = i.len;
    }
    long long v = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += u;
    }
    total = __shfl_sync(~0u, v, 31);
    share = share_of();
    const long long x0 = ((long long)blockIdx.x * W + wid) * share;
    if (x0 < v && x0 >= v - cost) {
      s_row[wid] = lane;
      s_x[wid] = x0 - (v - cost);
    }
    __syncthreads();
  }
  // more: chunks of kThreads rows, twice over when there is more than one (the total comes first)
  for (int pass = a.rows <= 32 ? 2 : chunks > 1 ? 0 : 1; pass < 2; ++pass) {
    long long carry = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c * C::kThreads + tid;
      long long cost = 0;
      if (b < a.rows) {
        const RowInfo i = row_info(a, b, r, C::kCols, pass == 1 && blockIdx.x == 0);
        cost = (long long)K * i.ntb * (i.tiles + C0);
        if (chunks == 1) {
          s_rows[0][tid] = i.start;
          s_rows[1][tid] = i.ntb ? i.n : 0;
          s_rows[2][tid] = i.len;
        }
      }
      long long v = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) s_scan[wid] = v;
      __syncthreads();
      long long before = carry, sum = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i < wid) before += s_scan[i];
        sum += s_scan[i];
      }
      if (pass == 0 || chunks == 1) total = carry + sum;
      if (pass == 1) {
        if (c == 0) share = share_of();
        const long long pre = before + v - cost;
        s_pre[tid] = pre;
        __syncthreads();
        // the row that holds each warp's first cost unit
        const long long x0 = ((long long)blockIdx.x * W + tid) * share;
        if (tid < W && x0 < total && x0 >= carry && x0 < carry + sum) {
          int lo = 0, hi = C::kThreads;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] <= x0) lo = mid;
            else hi = mid;
          }
          s_row[tid] = c * C::kThreads + lo;
          s_x[tid] = x0 - s_pre[lo];
        }
      }
      carry += sum;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }
  }

  bool failed = false;
  if (s_row[wid] >= 0) {
    constexpr int NK = D / 16;  // MMAs along a head
    const uint32_t ring = ring0 + wid * C::kWarpBytes;
    // ---- the walk: units in order, each unit's tiles in stages that end at multiples of the stage
    auto row_of = [&](int b) {
      RowInfo i;
      if (chunks > 1) return row_info(a, b, r, C::kCols, false);
      i.start = s_rows[0][b];
      i.n = s_rows[1][b];
      i.len = s_rows[2][b];
      i.tiles = (i.len + kTile - 1) / kTile;
      i.ntb = (i.n * r + C::kCols - 1) / C::kCols;
      return i;
    };
    const int p_shift = 31 - __clz(P / kTile);
    int f_row = s_row[wid], f_unit, f_tile, f_end, f_kvh;
    RowInfo f = row_of(f_row);
    long long left = min(share, total - ((long long)blockIdx.x * W + wid) * share);
    bool f_begin;
    int id_at = -64, id = -1;  // 32 entries of the row's block table, from id_at on
    auto enter = [&](long long within) {  // the unit, from a cost offset in it
      const long long skip = within < C0 ? C0 - within : 0;
      f_tile = within > C0 ? (int)(within - C0) : 0;
      left -= skip;
      const int cnt = (int)min((long long)(f.tiles - f_tile), max(left, 0ll));
      f_end = f_tile + cnt;
      left -= cnt;
      f_begin = true;
      f_kvh = f_unit / f.ntb;
    };
    {
      const unsigned per = (unsigned)(f.tiles + C0);
      const long long x = s_x[wid];
      f_unit = (x >> 32) == 0 ? (int)((unsigned)x / per) : (int)(x / per);
      enter(x - (long long)f_unit * per);
    }
    // start the copies of the next stage into slot s, each lane its own tile's; false: no more
    auto issue = [&](int s) {
      while (f_tile >= f_end) {
        if (left <= 0) return false;
        if (++f_unit >= K * f.ntb) {
          do {
            if (++f_row >= a.rows) return false;
            f = row_of(f_row);
          } while (f.ntb == 0);
          f_unit = 0;
          id_at = -64;
        }
        enter(0);
      }
      const int cnt = min(TS - f_tile % TS, f_end - f_tile), at = f_tile + min(lane, cnt - 1);
      if ((f_tile >> p_shift) < id_at || ((f_tile + cnt - 1) >> p_shift) >= id_at + 32) {
        id_at = f_tile >> p_shift;
        id = ((id_at + lane) << p_shift) < f.tiles
                 ? a.kv.block_table[(int64_t)f_row * a.kv.max_blocks + id_at + lane] : -1;
      }
      const int block = __shfl_sync(~0u, id, (at >> p_shift) - id_at);
      const bool ok = (unsigned)block < (unsigned)a.kv.num_blocks;
      const uint32_t present = __ballot_sync(~0u, ok && lane < cnt), bar = su32(&full[wid][s]);
      if (lane == 0) {
        Stage& d = s_stage[wid][s];
        d.tile = f_tile;
        d.what = (uint32_t)cnt | (f_begin ? kBegin : 0u) | (f_tile + cnt == f_end ? kEnd : 0u) |
                 (f_tile + cnt == f.tiles ? kLast : 0u) | present << 16;
        if (f_begin || f_tile + cnt == f_end) {
          d.unit = f_unit;
          d.ntb = f.ntb;
          d.start = f.start;
          d.n = f.n;
          d.len = f.len;
        }
        if (present != (1u << cnt) - 1u) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
        bar_expect(bar, (uint32_t)__popc(present) * tile_bytes(D));
      }
      __syncwarp();
      if (ok && lane < cnt) {
        const int64_t tile = (((int64_t)block * K + f_kvh) << p_shift) + (at & ((1 << p_shift) - 1));
        bulk_g2s(ring + s * C::kStageBytes + lane * tile_bytes(D),
                 static_cast<const uint8_t*>(a.kv.pool) + tile * tile_bytes(D), tile_bytes(D), bar);
      }
      f_tile += cnt;
      f_begin = false;
      return true;
    };
    int issued = 0;
    while (issued < S && issue(issued)) ++issued;
    bool fill = issued == S;

    uint32_t qf[NK][2], qs[2];
    // per column: the factor of its scores (to log2), the reference (a raw score), the raw score
    // from which on the reference follows
    float fac[2], m[2], high[2], o[NK][4], off[G][2], ob[4];
    int sigma = kLeast, lim[2], open = 0, len = 0, age = 0, c_base = 0, cols = 0;
    bool first = false;
    const int key_l = ((lane >> 3) & 1) * 8 + (lane & 7), c0 = (lane >> 4) ^ swizzle<D>(key_l);
    const uint32_t row_off = key_l * (D / 2), c_off = c0 << 4;

    // one stage; Edge: some key of it is hidden from some column, or missing
    auto stage = [&](auto edge_tag, uint32_t st, int key0, int cnt, uint32_t present) {
      constexpr bool Edge = decltype(edge_tag)::value;
      auto has = [&](int tt) { return !Edge || tt < cnt; };  // (a stage without an edge is full)
      // ---- scores
      float x[TS][4];
#pragma unroll
      for (int tt = 0; tt < TS; ++tt) {
        if (has(tt)) {
          const uint32_t base = st + tt * tile_bytes(D), meta = base + 16 * D;
          // biases: groups along k, the upper eight k slots again for the sums' low parts
          uint32_t b0 = 0, b1 = 0;
          float sk[2][G];
          if constexpr (G == 1) {
            if (t == 0) {
              b0 = lds16(meta + 32 + g * 2);
              b1 = lds16(meta + 32 + g * 2 + 16);
            }
            sk[0][0] = h2f(lds16(meta + g * 2)).x;
            sk[1][0] = h2f(lds16(meta + g * 2 + 16)).x;
          } else {
            if (2 * t < G) {
              b0 = lds32(meta + 32 * G + (g * G + 2 * t) * 2);
              b1 = lds32(meta + 32 * G + ((g + 8) * G + 2 * t) * 2);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[2];
              if constexpr (G == 4)
                lds64(v[0], v[1], meta + (g + 8 * h) * 8);
              else
                v[0] = lds32(meta + (g + 8 * h) * 4);
#pragma unroll
              for (int i = 0; i < G / 2; ++i) {
                const float2 f = h2f(v[i]);
                sk[h][2 * i] = f.x;
                sk[h][2 * i + 1] = f.y;
              }
            }
          }
          float sum[4] = {};
          mma_f16(sum, b0, b1, b0, b1, qs[0], qs[1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[tt][j] = sum[j] * 1.52587890625e-05f;  // 2^-16
          // the groups' chains side by side
          uint32_t w[G][4];
          float d[G][4] = {};
#pragma unroll
          for (int grp = 0; grp < G; ++grp) ldsm4(w[grp], base + row_off + (c_off ^ (grp << 5)));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int grp = 0; grp < G; ++grp) {
              const uint32_t u0 = w[grp][(i >> 1) * 2] >> (8 * (i & 1));
              const uint32_t u1 = w[grp][(i >> 1) * 2 + 1] >> (8 * (i & 1));
              mma_f16(d[grp], u0 & 0x000F000Fu, u1 & 0x000F000Fu, u0 & 0x00F000F0u,
                      u1 & 0x00F000F0u, qf[4 * grp + i][0], qf[4 * grp + i][1]);
            }
#pragma unroll
          for (int grp = 0; grp < G; ++grp)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[tt][j] = fmaf(sk[j >> 1][grp], d[grp][j], x[tt][j]);
          if constexpr (Edge) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + tt * kTile + g + 8 * (j >> 1);
              if (key > lim[j & 1] || !((present >> tt) & 1)) x[tt][j] = -INFINITY;
            }
          }
        }
      }
      // ---- exponents relative to the reference, 7 above it; the largest value scale
      // (two keys of one group per word)
      bool grow = false;
#pragma unroll
      for (int tt = 0; tt < TS; ++tt)
        if (has(tt)) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            grow |= x[tt][j] > high[j & 1];
        }
      uint32_t big = 0;
      auto scales = [&](auto&& f) {  // f(address, tile, word in it): the stage's value scales
#pragma unroll
        for (int i = 0; i < TS * G * 8; i += 32) {
          const int word = i + lane, tt = word / (G * 8), in = word % (G * 8);
          if (tt < TS && has(tt)) f(st + tt * tile_bytes(D) + 16 * D + 64 * G + in * 4, tt, in);
        }
      };
      scales([&](uint32_t at, int tt, int in) {
        uint32_t v = lds32(at) & 0x7FFF7FFFu;
        if constexpr (Edge) {
          const int key = key0 + tt * kTile + (in & 7) * 2;
          const bool in_tile = (present >> tt) & 1;
          if (!in_tile || key >= len) v &= 0xFFFF0000u;
          if (!in_tile || key + 1 >= len) v &= 0x0000FFFFu;
        }
        big = __vmaxu2(big, v);
      });
      big = max(big & 0xFFFFu, big >> 16);
      // largest < 2^sigma, or the accumulators' scale moves
      const bool more_scale = (int)(big >> 10) - 14 > sigma;
      if (__any_sync(~0u, grow || more_scale)) {
        big = __reduce_max_sync(~0u, big);
        // (below 1 a bit to spare, so that sigma moves less often)
        int to = big >= 0x7C00u ? 16 : (int)(big >> 10) - 14;
        to = max(sigma, to < 0 ? to + 1 : to);
        if (to == -1) to = 0;
        const float turn = pow2(sigma - to);
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = m[i];
#pragma unroll
          for (int tt = 0; tt < TS; ++tt)
            if (has(tt))
              top = fmaxf(top, fmaxf(x[tt][i], x[tt][2 + i]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, sh));
          f[i] = exp2_fast((m[i] - top) * fac[i]);
          m[i] = top;
          high[i] = reach(m[i], fac[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ob[j] *= f[j & 1];
#pragma unroll
          for (int i = 0; i < NK; ++i) o[i][j] *= f[j & 1] * turn;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int grp = 0; grp < G; ++grp) off[grp][i] *= f[i] * turn;
        sigma = to;
      }
      // p * scale stays in range: large scales take p down (the scale itself could become
      // subnormal), small ones are moved up where they lie, exactly
      if (sigma < 0) {
        const uint32_t up = pack_h2(pow2(-sigma), pow2(-sigma));
        scales([&](uint32_t at, int, int) { sts32(at, hmul2(lds32(at), up)); });
        __syncwarp();
      }
      const float down = pow2(-max(sigma, 0));
      const uint32_t s_one = pack_h2(down, down);
      // ---- weights and the second product
      float bsum[4] = {};
#pragma unroll
      for (int tt = 0; tt < TS; ++tt) {
        if (has(tt)) {
          const uint32_t base = st + tt * tile_bytes(D), meta = base + 16 * D;
          // (The reference is taken off before the scaling: the largest weight is 2^7 however
          // large the scores are.  Of scaled scores past 2^27 the roundings alone could take it out
          // of fp16's range.)
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            p[j] = exp2_fast(fmaf(x[tt][j] - m[j & 1], fac[j & 1], 7.0f));
          const uint32_t p0 = transpose8(pack_h2(p[0], p[1])), p1 = transpose8(pack_h2(p[2], p[3]));
          const uint32_t ps0 = hmul2(p0, s_one), ps1 = hmul2(p1, s_one);
          uint32_t live0 = ~0u, live1 = ~0u;
          if constexpr (Edge) {  // this lane's keys: 2t, 2t + 1, 2t + 8, 2t + 9
            const int n = (present >> tt) & 1 ? len - (key0 + tt * kTile + 2 * t) : 0;
            live0 = (n > 0 ? 0xFFFFu : 0u) | (n > 1 ? 0xFFFF0000u : 0u);
            live1 = (n > 8 ? 0xFFFFu : 0u) | (n > 9 ? 0xFFFF0000u : 0u);
          }
          // rows 0 .. G-1: the groups' biases; row 7: ones, which sum the weights
          uint32_t a0 = g == 7 ? 0x3C003C00u : 0u, a2 = a0;
          if (g < G) {
            a0 = lds32(meta + 96 * G + (g * 16 + 2 * t) * 2) & live0;
            a2 = lds32(meta + 96 * G + (g * 16 + 2 * t + 8) * 2) & live1;
          }
          mma_f16(bsum, a0, 0, a2, 0, p0, p1);
#pragma unroll
          for (int grp = 0; grp < G; ++grp) {
            const uint32_t v0 = lds32(meta + 64 * G + (grp * 16 + 2 * t) * 2) & live0;
            const uint32_t v1 = lds32(meta + 64 * G + (grp * 16 + 2 * t + 8) * 2) & live1;
            uint32_t w[4];
            ldsm4t(w, base + 8 * D + row_off + (c_off ^ (grp << 5)));
            const uint32_t f0 = hmul2(ps0, v0), f1 = hmul2(ps1, v1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u0 = w[(i >> 1) * 2] >> (8 * (i & 1));
              const uint32_t u1 = w[(i >> 1) * 2 + 1] >> (8 * (i & 1));
              mma_f16(o[4 * grp + i], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu,
                      u1 & 0x00F000F0u, f0, f1);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) ob[j] += bsum[j];
      if (++age % C::kCentre == 0) {
#pragma unroll
        for (int grp = 0; grp < G; ++grp)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float d = 0.5f * fmaf(o[4 * grp][2 + i], 0.0625f, o[4 * grp][i]);
            off[grp][i] += d;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[4 * grp + k][i] -= d;
              o[4 * grp + k][2 + i] -= 16.0f * d;
            }
          }
      }
    };

    for (int used = 0; used < issued; ++used) {
      const int s = used % S;
      const Stage& d = s_stage[wid][s];
      const uint32_t what = d.what;
      const int cnt = (int)(what & 255u);
      const int key0 = d.tile * kTile;
      if (what & kBegin) {
        // a new unit (or this warp's part of one): queries and empty sums
        const int start = d.start, n = d.n, kvh = d.unit / d.ntb;
        len = d.len;
        c_base = (d.unit % d.ntb) * C::kCols;
        cols = n * r;
        first = d.tile == 0;
        open = len - n + 1;  // keys below are seen by every column
        sigma = kLeast;
        age = 0;
        const int c = c_base + g;
        const uint16_t* src = a.q + ((int64_t)(start + c / r) * a.heads + kvh * r + c % r) * D;
        uint4 raw[2 * G];
        float big = 0.0f;
#pragma unroll
        for (int ch = 0; ch < 2 * G; ++ch) {
          raw[ch] = c < cols ? *reinterpret_cast<const uint4*>(src + ch * 32 + t * 8)
                             : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[ch].x, raw[ch].y, raw[ch].z, raw[ch].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            big = fmaxf(big, fabsf(__uint_as_float(w[i] << 16)));
            big = fmaxf(big, fabsf(__uint_as_float(w[i] & 0xFFFF0000u)));
          }
        }
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
        int e = (int)((__float_as_uint(big) >> 23) & 255u) - 127;  // 2^e <= big < 2^(e+1)
        e = max(e, -100);
        const float up = pow2(14 - e);
        float sum[4] = {};
#pragma unroll
        for (int ch = 0; ch < 2 * G; ++ch) {
          const uint32_t w[4] = {raw[ch].x, raw[ch].y, raw[ch].z, raw[ch].w};
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16) * up;
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * up;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            qf[2 * ch + i][0] = pack_h2(v[2 * i], v[2 * i + 4]);
            qf[2 * ch + i][1] = pack_h2(v[2 * i + 1] * 0.0625f, v[2 * i + 5] * 0.0625f);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[ch / 2] += v[i];
        }
        float hi[4] = {}, lo[4] = {};
#pragma unroll
        for (int i = 0; i < G; ++i) {
          sum[i] += __shfl_xor_sync(~0u, sum[i], 1);
          sum[i] += __shfl_xor_sync(~0u, sum[i], 2);
          const float v = sum[i] * 0.00390625f;  // 2^-8: into fp16's range
          hi[i] = __half2float(__float2half_rn(v));
          lo[i] = v - hi[i];
        }
        qs[0] = t == 0 ? pack_h2(hi[0], hi[1]) : t == 1 ? pack_h2(hi[2], hi[3]) : 0u;
        qs[1] = t == 0 ? pack_h2(lo[0], lo[1]) : t == 1 ? pack_h2(lo[2], lo[3]) : 0u;
        // score = fac * accumulated, in units of log2; per C-fragment column 2t, 2t+1
        const float f = score_factor(a.scale, 1477.3197218702985f, e);  // log2(e) 2^24 2^(e-14)
        fac[0] = __shfl_sync(~0u, f, 8 * t);
        fac[1] = __shfl_sync(~0u, f, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int cc = c_base + 2 * t + i;
          // the last key that the column's token sees
          lim[i] = len - n + min(cc, cols - 1) / r;
          m[i] = kNone;
          high[i] = reach(m[i], fac[i]);
#pragma unroll
          for (int grp = 0; grp < G; ++grp) off[grp][i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ob[j] = 0.0f;
#pragma unroll
          for (int i = 0; i < NK; ++i) o[i][j] = 0.0f;
        }
      }
      if (!warp_wait(su32(&full[wid][s]), (uint32_t)(used / S) & 1u)) {
        failed = true;
        break;
      }
      const uint32_t present = what >> 16, st = ring + s * C::kStageBytes;
      if (key0 + cnt * kTile > open || present != (1u << TS) - 1u)
        stage(std::true_type{}, st, key0, cnt, present);
      else
        stage(std::false_type{}, st, key0, cnt, present);
      const int unit = d.unit, ntb = d.ntb, start = d.start, n_new = d.n;
      if (sigma < 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // scales moved
      __syncwarp();  // every lane has read the stage: its buffer may be filled again
      if (fill) {
        fill = issue(s);
        if (fill) ++issued;
      }
      if (!(what & kEnd)) continue;

      // ---- the unit's end (here): a result, or a part of one.  A part that does not end
      // its unit is the warp's last work, and its ring is idle
      const bool last = what & kLast;
      float* part = nullptr;
      if (!(first && last))
        part = last ? warp_part + ((size_t)blockIdx.x * W + wid) * C::kPartial
                    : reinterpret_cast<float*>(rings + wid * C::kWarpBytes);
      if (lane == 0 && part)
        s_part[wid][last ? 0 : 1] =
            Part{unit, start, n_new, ntb, first, (len + kTile - 1) / kTile - key0 / kTile - cnt};
      const int kvh = unit / ntb;
      const float even = pow2(24 + sigma), odd = pow2(20 + sigma);
      float l[2], inv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] = __shfl_sync(~0u, ob[i], 28 + t);
        inv[i] = l[i] > 0.0f ? 1.0f / l[i] : l[i];  // no key: 0; NaN stays
      }
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        float bias[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          bias[i] = fmaf(off[grp][i], even, __shfl_sync(~0u, ob[i], 4 * grp + t));
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const int d0 = grp * 64 + ch * 32 + 4 * g;
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // columns 2t, 2t + 1
            const int cc = 2 * t + i;
            const float(&u)[4] = o[4 * grp + 2 * ch], (&v)[4] = o[4 * grp + 2 * ch + 1];
            const float4 y = make_float4(fmaf(u[i], even, bias[i]), fmaf(u[2 + i], odd, bias[i]),
                                         fmaf(v[i], even, bias[i]), fmaf(v[2 + i], odd, bias[i]));
            if (part) {
              *reinterpret_cast<float4*>(part + cc * D + d0) = y;
            } else if (c_base + cc < cols) {
              const int c = c_base + cc;
              store_bf16(a.out + ((int64_t)(start + c / r) * a.heads + kvh * r + c % r) * D + d0,
                         y, inv[i]);
            }
          }
        }
      }
      if (part && g == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          part[C::kCols * D + 2 * t + i] = m[i];
          part[C::kCols * (D + 1) + 2 * t + i] = l[i];
          part[C::kCols * (D + 2) + 2 * t + i] = fac[i];
        }
      }
    }
    if (failed) {
      if (lane == 0) atomicOr(a.batch.err, MOE_DERR_WAIT);
      // the copies in flight land (or time out) before the ring is given up
      for (int i = max(issued - S, 0); i < issued; ++i)
        warp_wait(su32(&full[wid][i % S]), (uint32_t)(i / S) & 1u);
    }
  }
  const int any_failed = __syncthreads_or(failed);
  griddep_launch();
  if (any_failed) {
    if (tid == 0) static_cast<Cut*>(a.ws)[blockIdx.x].last = -1;
    return;
  }

  // ------------------------------------------------ parts merged over the CTA
  // In order: each warp's head part (it ends a unit) and its last part (it does
  // not).  A run of parts of one unit is closed by a head or by the CTA's end;
  // it takes the last parts of the warps from the previous head's on and then
  // the next head.  One warp per column of a run.
  const uint32_t heads = __ballot_sync(~0u, lane < W && s_part[lane < W ? lane : 0][0].unit >= 0);
  const uint32_t lasts = __ballot_sync(~0u, lane < W && s_part[lane < W ? lane : 0][1].unit >= 0);
  int from = 0, task = wid;
  for (uint32_t left = heads;; left &= left - 1) {
    const bool closed = left != 0;
    const int to = closed ? __ffs(left) - 1 : W;  // members: lasts of [from, to), head of `to`
    const uint32_t mine = lasts & (uint32_t)((1ull << to) - 1ull) & ~((1u << from) - 1u);
    if (!closed && mine == 0) {
      if (tid == 0) static_cast<Cut*>(a.ws)[blockIdx.x].last = -1;
      break;
    }
    const int w0 = mine ? __ffs(mine) - 1 : to, w1 = closed ? to : 31 - __clz(mine);
    const Part pt = closed ? s_part[to][0] : s_part[w1][1];
    const bool begun = mine != 0 && s_part[w0][1].first;
    const float* head_part = warp_part + ((size_t)blockIdx.x * W + to) * C::kPartial;
    float* dst = cta_part + ((size_t)blockIdx.x * 2 + (closed || !begun ? 0 : 1)) * C::kPartial;
    for (; task < C::kCols; task += W) {
      const int cc = task;
      // lane w: warp w's maximum, sum and (one of the column's) factor
      float mk = kNone, lk = 0.0f, fac = 0.0f;
      if (lane >= w0 && lane <= w1) {
        const float* src = closed && lane == to
                               ? head_part
                               : reinterpret_cast<const float*>(rings + lane * C::kWarpBytes);
        mk = src[C::kCols * D + cc];
        lk = src[C::kCols * (D + 1) + cc];
        fac = src[C::kCols * (D + 2) + cc];
      }
      float mm = mk;
#pragma unroll
      for (int o = 8; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
      const float fk = exp2_fast((mk - mm) * fac);
      lk *= fk;
#pragma unroll
      for (int o = 8; o; o >>= 1) lk += __shfl_xor_sync(~0u, lk, o);
      mm = __shfl_sync(~0u, mm, 0);
      lk = __shfl_sync(~0u, lk, 0);
      fac = __shfl_sync(~0u, fac, w1);
      float y[D / 32] = {};
      auto add = [&](const float* src, float f) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float2 v = *reinterpret_cast<const float2*>(src + cc * D + lane * 2 + i * 64);
          y[2 * i] = fmaf(f, v.x, y[2 * i]);
          y[2 * i + 1] = fmaf(f, v.y, y[2 * i + 1]);
        }
      };
#pragma unroll 4
      for (int w = w0; w < w1 + (closed ? 0 : 1); ++w)
        add(reinterpret_cast<const float*>(rings + w * C::kWarpBytes), __shfl_sync(~0u, fk, w));
      if (closed) add(head_part, __shfl_sync(~0u, fk, to));
      if (closed && begun) {
        const int c = (pt.unit % pt.ntb) * C::kCols + cc;
        if (c < pt.n * r)
          store_row<D>(a.out + ((int64_t)(pt.start + c / r) * a.heads + pt.unit / pt.ntb * r + c % r) * D,
                       y, lk, lane);
      } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          *reinterpret_cast<float2*>(dst + cc * D + lane * 2 + i * 64) =
              make_float2(y[2 * i], y[2 * i + 1]);
        if (lane == 0) {
          dst[C::kCols * D + cc] = mm;
          dst[C::kCols * (D + 1) + cc] = lk;
          dst[C::kCols * (D + 2) + cc] = fac;
        }
      }
    }
    task -= C::kCols;
    if (!closed) {
      // a unit begun here that goes on behind this CTA: its tiles go on from the share's end
      const long long per = share * W;
      if (tid == 0)
        static_cast<Cut*>(a.ws)[blockIdx.x] =
            Cut{begun ? (int)(blockIdx.x + (pt.left + per - 1) / per) : -1, pt.unit, pt.start, pt.n,
                pt.ntb, {}};
      break;
    }
    from = to;
  }
}

// Units that were cut between CTAs, each found at the CTA that began it: their
// parts in order, a few warps per column.
template <int D>
__global__ void __launch_bounds__(1024) combine_kernel(AttnArgs a) {
  using C = Cfg<D>;
  constexpr int kSplit = 32 / C::kCols;  // warps side by side on a column's parts
  __shared__ float s_y[kSplit - 1][C::kCols][D], s_m[kSplit][C::kCols], s_l[kSplit][C::kCols];
  griddep_wait();
  const int first = blockIdx.x, lane = threadIdx.x & 31;
  const int cc = (threadIdx.x >> 5) % C::kCols, split = (threadIdx.x >> 5) / C::kCols;
  const Cut cut = static_cast<const Cut*>(a.ws)[first];
  if (cut.last <= first) return;
  const float* cta_part = cta_parts(a.ws);
  const float fac = cta_part[((size_t)first * 2 + 1) * C::kPartial + C::kCols * (D + 2) + cc];
  float m = kNone, l = 0.0f, y[D / 32] = {};
  for (int k0 = first + split; k0 <= cut.last; k0 += kSplit * 32) {
    // lane i: part k0 + i * kSplit
    const int mine = k0 + lane * kSplit;
    float mk = kNone, lk = 0.0f;
    if (mine <= cut.last) {
      const float* src = cta_part + ((size_t)mine * 2 + (mine == first)) * C::kPartial;
      mk = src[C::kCols * D + cc];
      lk = src[C::kCols * (D + 1) + cc];
    }
    float mm = fmaxf(mk, m);
#pragma unroll
    for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
    const float fk = exp2_fast((mk - mm) * fac), f0 = exp2_fast((m - mm) * fac);
    lk *= fk;
#pragma unroll
    for (int o = 16; o; o >>= 1) lk += __shfl_xor_sync(~0u, lk, o);
    l = fmaf(l, f0, lk);
    m = mm;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) y[i] *= f0;
    const int n = min(32, (cut.last - k0) / kSplit + 1);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const int k = k0 + i * kSplit;
      const float f = __shfl_sync(~0u, fk, i);
      const float* src = cta_part + ((size_t)k * 2 + (k == first)) * C::kPartial + cc * D + lane * 2;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const float2 v = *reinterpret_cast<const float2*>(src + j * 64);
        y[2 * j] = fmaf(f, v.x, y[2 * j]);
        y[2 * j + 1] = fmaf(f, v.y, y[2 * j + 1]);
      }
    }
  }
  if (lane == 0) {
    s_m[split][cc] = m;
    s_l[split][cc] = l;
  }
  if (split) {
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
      *reinterpret_cast<float2*>(&s_y[split - 1][cc][lane * 2 + j * 64]) = make_float2(y[2 * j], y[2 * j + 1]);
  }
  __syncthreads();
  if (split) return;
  float mm = kNone;
#pragma unroll
  for (int k = 0; k < kSplit; ++k) mm = fmaxf(mm, s_m[k][cc]);
  const float f0 = exp2f((m - mm) * fac);
  l *= f0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) y[i] *= f0;
#pragma unroll
  for (int k = 1; k < kSplit; ++k) {
    const float f = exp2f((s_m[k][cc] - mm) * fac);
    l = fmaf(f, s_l[k][cc], l);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const float2 v = *reinterpret_cast<const float2*>(&s_y[k - 1][cc][lane * 2 + j * 64]);
      y[2 * j] = fmaf(f, v.x, y[2 * j]);
      y[2 * j + 1] = fmaf(f, v.y, y[2 * j + 1]);
    }
  }
  const int r = a.heads / a.kv.kv_heads, c = (cut.unit % cut.ntb) * C::kCols + cc;
  if (c < cut.n * r)
    store_row<D>(a.out + ((int64_t)(cut.start + c / r) * a.heads + cut.unit / cut.ntb * r + c % r) * D,
                 y, l, lane);
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e == cudaSuccess)
    e = launch_pdl(decode_kernel<D>, dim3(kGrid), dim3(C::kThreads), C::kSmem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine_kernel<D>, dim3(kGrid), dim3(1024), 0, st, a);
}

template <int D>
constexpr size_t bytes_for() {
  return (kCutBytes + kGrid * 4 * (2 + Cfg<D>::kWarps) * (size_t)Cfg<D>::kPartial + 255) /
         256 * 256;
}
}  // namespace

size_t decode_workspace_bytes(int D) {
  return D == 256 ? bytes_for<256>() : D == 128 ? bytes_for<128>() : bytes_for<64>();
}

cudaError_t launch_decode(const AttnArgs& a, cudaStream_t st) {
  const int D = a.kv.head_dim;
  return D == 256 ? launch<256>(a, st) : D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace kv
}  // namespace moe
