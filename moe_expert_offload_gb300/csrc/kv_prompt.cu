// Attention over the 4-bit cache for rows of many new tokens (prompt chunks),
// on the 5th-generation tensor cores.
//
// A unit is a tile of 128 (head_dim 256) or 2 x 128 queries of one row and kv
// head: tok tokens x the r query heads that share the head, row i * r + h.  It
// walks the keys that its last token sees in blocks of 128.  The blocks of all
// units form one line of work that is cut into equal shares, one per CTA, so a
// long row, a causal triangle and ragged batches keep all SMs equally busy;
// units cut by a share's end are merged afterwards in a fixed order.
//
// One CTA per SM, warp-specialised, blocks handed over with mbarriers:
//   warps 0-7   softmax: thread = query row.  Scores come from TMEM, weights go
//               back to TMEM in fp16 over the scores they came from, as the A
//               operand of the second product.  head_dim 256: the two warp
//               groups share a row's columns and swap maxima through shared
//               memory; else each has its own tile of 128 queries.
//   warps 8-15  dequantise keys to fp16, scale * code + bias, rounded once;
//   warps 16-23 values alike.  Codes come by 16-byte loads one block ahead, one
//               LOP3 per pair (1024 + c or 64 + c), the offset taken off exactly,
//               one fma.  Both land in the 128-byte swizzled layout, the keys read
//               K-major and the values MN-major by the MMAs.
//   warp 24     issues the MMAs (M = 128, fp32 accumulators in TMEM): the next
//               block's scores run while the softmax works on this one's.
// Registers move from the dequantising warps and the MMA warp's group to the
// softmax (the CTA starts with 72 a thread; what they add up to is checked below).
// The columns of a head run in the order 0,4,1,5,2,6,3,7 within every 8 (the
// order in which one LOP3 yields pairs): the queries are laid out alike, and the
// result is put in order when it is stored.
// fp16 roundings: keys and values 2^-11 once, weights 2^-11 once (2^7 for the
// maximum that they refer to, so that small ones keep their bits; at head_dim 64
// and 128 twice more for the first half of a block whose second half moves that
// maximum, by the factor's rounding and the product's); queries are scaled by a
// power of two per row.  That maximum follows the scores only when weights may pass
// fp16's range (a score 2^3 to 2^9 above it), so the accumulator in TMEM is rarely
// rescaled.
//
// Measured: 8192 tokens, 16 query heads on 2 of 256: 499 us, 1102 TFLOP/s (57% of a
// large bf16 matrix product); 2048 tokens on 30000, 32 heads on 4 of 128: 787 us,
// 1321 TFLOP/s (68%).  The compiler spills 400 to 430 bytes a thread
// (stack 72 to 120).  Bound by the chain of a block: at head_dim 64 and 128 scores,
// TMEM load, exponentials, TMEM store, product; at 256, whose one block of values
// takes all the shared memory there is, values freed, dequantised (1400 cycles),
// fenced (570), seen by the issuer (350) and multiplied (1500).  The tensor pipe is
// busy 57% (128) and 49% (256) of the time, the issue slots 57 and 59%.  Measured and
// dropped: two tiles with the next scores in halves of 64 keys, the first before
// the product (975 us then against 876), a warp of its own that issues for each
// tile (1046); one tile with keys and values handed over by halves of the columns
// (575 against 516), with a second issuing warp for the products (556).
#include <type_traits>

#include "kv_common.cuh"
#include "stream_common.cuh"

namespace moe {
namespace kv {
namespace {

using sc::bar_init;
using sc::bar_wait;
using sc::su32;

constexpr int kKeys = 128;  // keys of a block
constexpr int kSoftWarps = 8, kSideWarps = 8, kMmaWarp = 24;
constexpr int kThreads = 28 * 32;  // seven warp groups; three warps of the last one idle
constexpr int kStartRegs = 72;
constexpr float kNone = -1e30f;  // below every raw score (q and k in fp16's range: 2^38 at most)
// Scores this far from zero (in log2) have their reference taken off before they are scaled: the
// offset of the fused form is rounded by up to 2^-24 of itself, 2^-11 here.
constexpr float kFar = 8192.0f;
constexpr float kMost = 65504.0f;  // fp16's largest

template <int D>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;   // query tiles of a unit
  static constexpr int kStages = D == 256 ? 1 : 2;  // key and value blocks held
  static constexpr int kRows = 128 * kTiles;
  // a unit's fixed cost, in keys: queries in, results out (two rows of 1700 to 5000 new tokens,
  // us at 384, 512, 768 and 1024: head_dim 64 155, 148, 151, 153; 128 317, 293, 272, 280;
  // 256, 16 heads on 2, from 512 on 278, 285, 296)
  static constexpr int kUnitKeys = D == 128 ? 768 : 512;
  static constexpr int kBlockBytes = kKeys * D * 2;  // one block of keys (or values, or queries)
  // results on their way out: each softmax warp's 32 rows of 64 bytes, 80 apart
  static constexpr int kOutBytes = kSoftWarps * 32 * 80;
  static constexpr size_t kSmem = 1024 + (size_t)(kTiles + 2 * kStages) * kBlockBytes + kOutBytes;
  static constexpr int kPartial = kRows * (D + 3);  // floats: o [row][D], top, l, fac [row]
  static constexpr uint32_t kIdescS = (1u << 4) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                      ((128u >> 4) << 24);  // bit 16: B is MN-major
  static constexpr int kO = D == 256 ? 256 : 128;   // TMEM columns between the tiles' results
  static constexpr int kS = 256;                    // scores: two slots of 128 columns
  static constexpr int kSoftRegs = D == 256 ? 112 : 136, kSideRegs = D == 256 ? 56 : 48;
  static constexpr int kMmaRegs = D == 256 ? 48 : 40;
  static_assert(kSoftRegs * 256 + kSideRegs * 512 + kMmaRegs * 128 <= kStartRegs * kThreads,
                "the registers given out are there");
};

// The unit that a CTA began and did not end: the last CTA with a part of it (-1: there is none).
struct Cut {
  int last, start, n, tok0, kvh, pad[3];
};
constexpr size_t kCutBytes = (kGrid * sizeof(Cut) + 255) / 256 * 256;

struct Row {
  int start, n, len, tiles;  // tiles 0: nothing here
};

__device__ __forceinline__ Row row_info(const AttnArgs& a, int b, int r, int tok) {
  Row i;
  i.start = a.batch.q_start[b];
  i.n = a.batch.q_start[b + 1] - i.start;
  i.len = a.batch.kv_len[b];
  i.tiles = 0;
  // (the decode kernel, which sees every row, reports what does not fit)
  if (i.n <= 0 || i.start < 0 || i.n > a.max_new || i.n > i.len ||
      (long long)i.len > (long long)a.kv.max_blocks * a.kv.block_tokens ||
      (long long)i.start + i.n > a.T || (long long)i.n * r <= decode_cols(a.kv.head_dim))
    return i;
  i.tiles = (i.n + tok - 1) / tok;
  return i;
}

// Cost of the first j units of a head of the row: each its keys (taking every
// tile for a full one) and a fixed part.
template <int D>
__device__ __forceinline__ long long cost_before(const Row& i, int tok, long long j) {
  return j * (i.len - i.n + Cfg<D>::kUnitKeys) + (long long)tok * (j * (j + 1) / 2);
}

struct Unit {
  int kvh, tok0;     // kv head, first token
  int blk0, blk1;    // key blocks of this share
  int blocks;        // key blocks of the unit
  long long rest;    // cost behind this share's end that still holds blocks
};

// The walk over a CTA's share; every role runs it for itself.
struct Walk {
  int b, kvh, j;
  long long at, left;  // offset in unit (kvh, j) where the share goes on; what is left of it
  Row row;
};

template <int D>
__device__ __forceinline__ bool next_unit(Walk& w, const AttnArgs& a, int r, int tok, Unit& u) {
  constexpr int kUnitKeys = Cfg<D>::kUnitKeys;
  while (w.left > 0) {
    if (w.row.tiles == 0 || w.kvh >= a.kv.kv_heads) {
      do {
        if (++w.b >= a.rows) return false;
        w.row = row_info(a, w.b, r, tok);
      } while (w.row.tiles == 0);
      w.kvh = w.j = 0;
      w.at = 0;
    }
    const int seen = w.row.len - w.row.n + min(w.row.n, (w.j + 1) * tok);
    const long long cost = w.row.len - w.row.n + kUnitKeys + (long long)(w.j + 1) * tok;
    u.kvh = w.kvh;
    u.tok0 = w.j * tok;
    u.blocks = (seen + kKeys - 1) / kKeys;
    // both ends of a share fall on the same block for the CTAs on either side
    auto block_at = [&](long long x) {
      const long long k = (x - kUnitKeys + kKeys / 2) / kKeys;
      return x <= kUnitKeys ? 0 : (int)min(k, (long long)u.blocks);
    };
    u.blk0 = block_at(w.at);
    const bool whole = w.left >= cost - w.at;
    u.blk1 = whole ? u.blocks : block_at(w.at + w.left);
    u.rest = min(cost, kUnitKeys + (long long)u.blocks * kKeys - kKeys / 2) - (w.at + w.left);
    if (whole) {
      w.left -= cost - w.at;
      w.at = 0;
      if (++w.j >= w.row.tiles) {
        w.j = 0;
        ++w.kvh;
      }
    } else {
      w.left = 0;
    }
    if (u.blk0 < u.blk1) return true;
  }
  return false;
}

// ------------------------------------------------------------- PTX wrappers
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// 128-byte swizzled operand, groups of 8 rows 1024 bytes apart; lead: bytes from one
// 64-column stripe to the next (read MN-major only)
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// 32 lanes x 32 columns of 32 bits; the values are there after tm_wait_ld
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// The loads issued so far are over; their registers pass through, so that nothing reads them
// before.
template <int N>
__device__ __forceinline__ void tm_wait_regs(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// whether any thread of the softmax warps says so
__device__ __forceinline__ bool any_of_256(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}
// {x, y} * f + g, and a + b, two at a time
__device__ __forceinline__ float2 fma2(float x, float y, float f, float g) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n"
      " mov.b64 c, {%5, %5};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x), "f"(y), "f"(f), "f"(g));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// All lanes of a warp wait, bounded as every wait is (stream_common.cuh).  A wait that runs out
// sets `stop`, and from then on nothing waits: every role runs through (or leaves) its loop and
// the CTA ends.
__device__ __forceinline__ void wait_all(uint64_t* bar, uint32_t parity, volatile int& stop) {
  long long t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(su32(bar)), "r"(parity & 1u)
        : "memory");
    if (done) break;
    if ((i & 15u) == 15u) {
      if (stop) break;
      const long long t = clock64();
      if (t0 == 0) t0 = t;
      else if (t - t0 > sc::kWaitCycles || i > sc::kSpin) {
        stop = 1;
        break;
      }
    }
  }
  __syncwarp();
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
  return p != 0;
}

// eight codes as fp16 pairs (0,4) (1,5) (2,6) (3,7), scaled
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t s, uint32_t b) {
  const uint32_t v = w >> 8;
  uint4 r;
  r.x = hfma2(hadd2((w & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s, b);  // 1024 + c, - 1024
  r.y = hfma2(hadd2((w & 0x00F000F0u) | 0x54005400u, 0xD400D400u), s, b);  // 64 + c, - 64
  r.z = hfma2(hadd2((v & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s, b);
  r.w = hfma2(hadd2((v & 0x00F000F0u) | 0x54005400u, 0xD400D400u), s, b);
  return r;
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(AttnArgs a) {
  using C = Cfg<D>;
  constexpr int NT = C::kTiles, S = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  // A block of keys or values is there; a tile's scores, weights, product are.  The last two by
  // the block's parity: a buffer's next block waits for the scores (products) of the block that
  // it replaces, which are never more than one phase of that barrier ago.
  __shared__ __align__(8) uint64_t k_full[S], v_full[S], p_full[NT][2];
  __shared__ __align__(8) uint64_t s_full[NT][2], o_done[NT][2], q_full, drained;
  __shared__ uint32_t tmem_slot;
  __shared__ long long s_scan[kThreads / 32], s_at, s_share;
  __shared__ int s_row;
  __shared__ volatile int s_stop;  // a wait ran out
  __shared__ float s_fac[C::kRows], s_max[2][128], s_sum[2][128];
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int K = a.kv.kv_heads, r = a.heads / K, P = a.kv.block_tokens;
  const int p_shift = 31 - __clz(P);
  const int per_tile = 128 / r, tok = per_tile * NT;  // tokens of a tile, of a unit
  const uint32_t r_inv = (65536 + r - 1) / r;         // x * r_inv >> 16 = x / r for x < 128
  const uint32_t base = (su32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, k_at = q_at + NT * C::kBlockBytes, v_at = k_at + S * C::kBlockBytes;
  const uint32_t out_at = v_at + S * C::kBlockBytes;

  if (wid == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      bar_init(su32(&k_full[i]), kSideWarps);
      bar_init(su32(&v_full[i]), kSideWarps);
    }
    for (int i = 0; i < 2 * NT; ++i) {
      bar_init(su32(&s_full[0][0] + i), 1);
      bar_init(su32(&o_done[0][0] + i), 1);
      bar_init(su32(&p_full[0][0] + i), kSoftWarps / NT);
    }
    bar_init(su32(&q_full), kSoftWarps);
    bar_init(su32(&drained), 1);
    s_row = -1;
    s_stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  griddep_wait();

  // ------------------------------------------------------- this CTA's share
  long long total = 0;
  auto share_of = [&] { return max((total + kGrid - 1) / kGrid, 2ll * kKeys); };
  if (a.rows <= 32) {
    // every warp for itself, a lane per row (7 short prompts: 48.8 us, 52.0 the other way)
    long long cost = 0;
    if (lane < a.rows) {
      const Row i = row_info(a, lane, r, tok);
      if (i.tiles) cost = K * cost_before<D>(i, tok, i.tiles);
    }
    long long v = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += u;
    }
    total = __shfl_sync(~0u, v, 31);
    const long long share = share_of(), x0 = blockIdx.x * share;
    if (wid == 0 && x0 < v && x0 >= v - cost) {
      s_row = lane;
      s_at = x0 - (v - cost);
    }
    if (tid == 0) s_share = share;
  }
  const int chunks = (a.rows + kThreads - 1) / kThreads;
  // more: chunks of kThreads rows, twice over when there is more than one (the total comes first)
  for (int pass = a.rows <= 32 ? 2 : chunks > 1 ? 0 : 1; pass < 2; ++pass) {
    long long carry = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c * kThreads + tid;
      long long cost = 0;
      if (b < a.rows) {
        const Row i = row_info(a, b, r, tok);
        if (i.tiles) cost = K * cost_before<D>(i, tok, i.tiles);
      }
      long long v = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
      }
      __syncthreads();
      if (lane == 31) s_scan[wid] = v;
      __syncthreads();
      long long before = carry, sum = 0;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < wid) before += s_scan[i];
        sum += s_scan[i];
      }
      if (pass == 0 || chunks == 1) total = carry + sum;
      if (pass == 1) {
        const long long share = share_of();
        const long long pre = before + v - cost, x0 = blockIdx.x * share;
        if (x0 < total && x0 >= pre && x0 < pre + cost) {
          s_row = b;
          s_at = x0 - pre;
        }
        if (tid == 0) s_share = share;
      }
      carry += sum;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  Cut* cuts = static_cast<Cut*>(a.ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kCutBytes);
  if (tid == 0) cuts[blockIdx.x].last = -1;

  Walk walk;
  walk.left = 0;
  if (s_row >= 0) {
    walk.b = s_row;
    walk.row = row_info(a, walk.b, r, tok);
    walk.left = min(s_share, total - blockIdx.x * s_share);
    const long long per_head = cost_before<D>(walk.row, tok, walk.row.tiles);
    long long x = s_at;
    walk.kvh = (int)(x / per_head);
    x -= walk.kvh * per_head;
    int lo = 0, hi = walk.row.tiles;  // the last unit whose cost_before is <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cost_before<D>(walk.row, tok, mid) <= x) lo = mid;
      else hi = mid;
    }
    walk.j = lo;
    walk.at = x - cost_before<D>(walk.row, tok, lo);
  }
  Unit u;

  if (wid < kSoftWarps) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int wg = wid >> 2, row = (wid & 3) * 32 + lane;  // TMEM lane
    const int tile = NT == 1 ? 0 : wg;
    const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lanes + tile * C::kO;
    uint32_t n = 0;  // blocks seen
    // A unit's queries: a warp's rows, 8 columns a lane, all loads under way at once.  The
    // buffer is free once the last block's scores of the unit before are there.
    auto load_queries = [&](const Row& w_row, const Unit& u) {
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kRounds = C::kRows / kSoftWarps / kAtOnce;
      constexpr uint32_t kGroup = kLanes == 32 ? ~0u : (1u << kLanes) - 1u;
      const uint32_t group = kGroup << (lane / kLanes * kLanes);
      uint4 raw[kRounds];
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int qr = (wid * kRounds + i) * kAtOnce + lane / kLanes, in = qr & 127;
        const int i_tok = (int)(in * r_inv >> 16), t = u.tok0 + (qr >> 7) * per_tile + i_tok;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (in < per_tile * r && t < w_row.n)
          raw[i] = *reinterpret_cast<const uint4*>(
              a.q + ((int64_t)(w_row.start + t) * a.heads + u.kvh * r + in - i_tok * r) * D +
              lane % kLanes * 8);
      }
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int qr = (wid * kRounds + i) * kAtOnce + lane / kLanes, in = qr & 127;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) big = __vmaxu2(big, w[k] & 0x7FFF7FFFu);
        big = __reduce_max_sync(group, max(big & 0xFFFFu, big >> 16));
        const int e = max((int)(big >> 7) - 127, -100);  // 2^e <= largest < 2^(e+1)
        const float up = pow2(14 - e);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[2 * k] = __uint_as_float(w[k] << 16) * up;
          x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * up;
        }
        const int col8 = lane % kLanes;
        sts128(q_at + (qr >> 7) * C::kBlockBytes + (col8 >> 3) * (kKeys * 128) + in * 128 +
                   (((col8 & 7) ^ (in & 7)) << 4),
               make_uint4(pack_h2(x[0], x[4]), pack_h2(x[1], x[5]), pack_h2(x[2], x[6]),
                          pack_h2(x[3], x[7])));
        // score = fac * accumulated, in units of log2
        if (col8 == 0) s_fac[qr] = score_factor(a.scale, 8.8054160e-05f, e);  // log2(e) 2^-14 2^e
      }
      fence_async();
      __syncwarp();
      if (lane == 0) sc::bar_arrive(su32(&q_full));
    };
    bool have = next_unit<D>(walk, a, r, tok, u);
    if (have) load_queries(walk.row, u);
    while (have) {
      const Row ri = walk.row;
      const int b = walk.b;
      asm volatile("bar.sync 1, 256;" ::: "memory");  // s_fac of all rows
      const float fac = s_fac[tile * 128 + row];
      {
        // the next unit's queries come to L2 meanwhile: a row of queries a thread
        Walk ahead = walk;
        Unit un;
        if (next_unit<D>(ahead, a, r, tok, un) && tid < C::kRows) {
          const int in = tid & 127, i_tok = (int)(in * r_inv >> 16);
          const int t = un.tok0 + (tid >> 7) * per_tile + i_tok;
          if (in < per_tile * r && t < ahead.row.n) {
            const uint16_t* src =
                a.q + ((int64_t)(ahead.row.start + t) * a.heads + un.kvh * r + in - i_tok * r) * D;
#pragma unroll
            for (int k = 0; k < D; k += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + k));
          }
        }
      }
      const int row_tok = (int)(row * r_inv >> 16), row_h = row - row_tok * r;
      const int t = u.tok0 + tile * per_tile + row_tok;
      const bool live = row < per_tile * r && t < ri.n;
      const int lim = ri.len - ri.n + min(t, ri.n - 1);             // last key that the row sees
      const int open = ri.len - ri.n + u.tok0 + tile * per_tile;   // all rows see the keys up to it
      // The row's reference, a raw score; a score x weighs 2^(x fac + off), off = 7 - top fac.
      // Where that is far from zero every visible score shall weigh too much (an infinite query's
      // row is lost anyway, and the others' references shall not follow for it).
      float top = kNone, off, l = 0.0f;
      auto set_off = [&] {
        off = fmaf(-top, fac, 7.0f);
        if (fabsf(off) > kFar && top < -kNone) off = 3e38f;
      };
      set_off();
      // the tiles of a block that are missing (a block id outside the pool), looked up a block ahead
      auto block_of = [&](int i) {
        const int at = i * (kKeys / kTile) + lane;
        return lane < kKeys / kTile && at * kTile < ri.len
                   ? a.kv.block_table[(int64_t)b * a.kv.max_blocks + ((at * kTile) >> p_shift)] : 0;
      };
      int block = block_of(u.blk0);
      for (int i = u.blk0; i < u.blk1; ++i) {
        const int slot = NT == 1 ? (int)(n & 1u) : tile;
        const uint32_t miss = __ballot_sync(~0u, (unsigned)block >= (unsigned)a.kv.num_blocks);
        block = block_of(i + 1);
        wait_all(&s_full[tile][n & 1u], n >> 1, s_stop);
        tc_after();
        const uint32_t s_tm = tmem + lanes + C::kS + slot * 128;
        const int key0 = i * kKeys;
        const bool edge = key0 + kKeys > open + 1 || miss != 0;
        // 16 columns (a key tile) from column c * 16 on: what the row does not see
        auto hide = [&](uint32_t* v, int c) {
          if (edge) {
            const int last = (miss >> c) & 1u ? -1 : lim - key0 - c * 16;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k > last) v[k] = 0xFF800000u;
          }
        };
        // The weights relative to the maximum so far, 2^7 above it.  While a part's sum is below
        // 2^16 each of them fits fp16; where it is not, some weight of the 64 passes the maximum's
        // by 2^3 or more: the maximum follows, what there is is scaled and the weights are formed
        // again, now from each score's distance to the maximum: of any finite scores none weighs
        // more than 2^7 then.  (x fac + off of the maximum itself is as far from 7 as the two
        // roundings of top fac: for top fac past 2^27 that may pass fp16's range, or lose all.)
        float2 sum;
        auto weights = [&](auto apart_tag, const uint32_t* v, uint32_t* p) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float2 x = make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
            if constexpr (decltype(apart_tag)::value) {
              x = add2(x, make_float2(-top, -top));
              x = fma2(x.x, x.y, fac, 7.0f);
            } else {
              x = fma2(x.x, x.y, fac, off);
            }
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum = add2(sum, x);
            p[k] = pack_h2(x.x, x.y);
          }
        };
        using Fused = std::false_type;
        using Apart = std::true_type;
        auto refer = [&](float seen) {  // the largest score there is here
          const float to = fmaxf(top, seen), f = ex2((top - to) * fac);
          top = to;
          set_off();
          l *= f;
          if (i > u.blk0 && __any_sync(~0u, f != 1.0f)) {
            wait_all(&o_done[tile][(n - 1) & 1u], (n - 1) >> 1, s_stop);
            tc_after();
            constexpr int kCols = NT == 1 ? D / 2 : D;
#pragma unroll 1
            for (int c = 0; c < kCols; c += 16) {
              uint32_t v[16];
              const uint32_t at = o_tm + (NT == 1 ? wg * (D / 2) : 0) + c;
              tm_ld16(at, v);
              tm_wait_regs(v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
              tm_st16(at, v);
            }
            tm_wait_st();
          }
        };
        if constexpr (NT == 1) {
          uint32_t p[32];
          auto attempt = [&](auto apart_tag) {
            uint32_t v[64];
            tm_ld32(s_tm + wg * 64, v);
            tm_ld32(s_tm + wg * 64 + 32, v + 32);
            tm_wait_regs(v);
#pragma unroll
            for (int c = 0; c < 4; ++c) hide(v + 16 * c, wg * 4 + c);
            if constexpr (decltype(apart_tag)::value) {
              float seen = kNone;
#pragma unroll
              for (int k = 0; k < 64; ++k) seen = fmaxf(seen, __uint_as_float(v[k]));
              s_max[wg][row] = seen;
              asm volatile("bar.sync 1, 256;" ::: "memory");
              refer(fmaxf(seen, s_max[wg ^ 1][row]));
            }
            sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < 4; ++c) weights(apart_tag, v + 16 * c, p + 8 * c);
          };
          // Both halves of the rows agree on whether the reference follows, which it does once at
          // most.  Every score has been read by the barrier on the way: the weights may go over
          // the scores.
          bool follow = i == u.blk0;
          if (!follow) {
            attempt(Fused{});
            follow = any_of_256(sum.x + sum.y > kMost);
          }
          if (follow) attempt(Apart{});
          l += sum.x + sum.y;
          tm_st16(s_tm + wg * 32, p);
          tm_st16(s_tm + wg * 32 + 16, p + 16);
        } else {
          // 64 columns at a time (2048 tokens on 30000 of head_dim 128, at the time: 790 us, 863 with 32 at a
          // time, 926 with loads under way one part ahead, whose registers spill)
#pragma unroll(D == 128 ? 2 : 1)
          for (int c = 0; c < 2; ++c) {
            uint32_t x[64], p[32];
            tm_ld32(s_tm + c * 64, x);
            tm_ld32(s_tm + c * 64 + 32, x + 32);
            tm_wait_regs(x);
#pragma unroll
            for (int q = 0; q < 4; ++q) hide(x + 16 * q, 4 * c + q);
            sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < 4; ++q) weights(Fused{}, x + 16 * q, p + 8 * q);
            if (__any_sync(~0u, sum.x + sum.y > kMost)) {
              const float before = top;
              float seen = kNone;
#pragma unroll
              for (int k = 0; k < 64; ++k) seen = fmaxf(seen, __uint_as_float(x[k]));
              refer(seen);
              const float f = ex2((before - top) * fac);
              const uint32_t ff = pack_h2(f, f);
              for (int k = 0; k < 2 * c; ++k) {
                uint32_t old[16];
                tm_wait_st();
                tm_ld16(s_tm + k * 16, old);
                tm_wait_regs(old);
#pragma unroll
                for (int q = 0; q < 16; ++q) old[q] = hfma2(old[q], ff, 0u);
                tm_st16(s_tm + k * 16, old);
              }
              sum = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int q = 0; q < 4; ++q) weights(Apart{}, x + 16 * q, p + 8 * q);
            }
            l += sum.x + sum.y;
            tm_st16(s_tm + c * 32, p);
            tm_st16(s_tm + c * 32 + 16, p + 16);
          }
        }
        tm_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) sc::bar_arrive(su32(&p_full[tile][n & 1u]));
        ++n;
      }
      // the next unit's queries come while the last product runs
      const Unit done = u;
      have = next_unit<D>(walk, a, r, tok, u);
      if (have) load_queries(walk.row, u);
      // ---- the unit's end (here): a result, or a part of one
      wait_all(&o_done[tile][(n - 1) & 1u], (n - 1) >> 1, s_stop);
      tc_after();
      if constexpr (NT == 1) {
        s_sum[wg][row] = l;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        l += s_sum[wg ^ 1][row];
      }
      const bool whole = done.blk0 == 0 && done.blk1 == done.blocks;
      const float inv = l > 0.0f ? 1.0f / l : l;
      // A lane holds a row's columns; through shared memory four lanes get 64 bytes of a row each
      // time, so that stores fill sectors (a row per lane: 2.5 times as long).
      const long long out_row =
          live ? (long long)(ri.start + t) * a.heads + done.kvh * r + row_h : -1ll;
      float* part = parts + ((size_t)blockIdx.x * 2 + (done.blk0 == 0 ? 1 : 0)) * C::kPartial;
      const int pr = tile * 128 + row;
      constexpr int kCols = NT == 1 ? D / 2 : D;
      const int c_at = NT == 1 ? wg * (D / 2) : 0;
      const uint32_t stage = out_at + wid * (32 * 80), mine = stage + lane * 80;
      auto flush = [&](auto&& store) {  // store(row of the warp, its output row, 16-byte piece, data)
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2);
          const long long to = __shfl_sync(~0u, out_row, rr);
          uint4 d;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w)
                       : "r"(stage + rr * 80 + (lane & 3) * 16)
                       : "memory");
          if (to >= 0) store(rr, to, lane & 3, d);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        uint32_t v[32];
        tm_ld32(o_tm + c_at + c, v);
        tm_wait_regs(v);
        // columns in order: 0,4,1,5,2,6,3,7 -> 0..7
        auto y = [&](int k) { return __uint_as_float(v[(k & ~7) + (k & 3) * 2 + ((k >> 2) & 1)]); };
        if (whole) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __nv_bfloat162 x =
                  __floats2bfloat162_rn(y(k + 2 * q) * inv, y(k + 2 * q + 1) * inv);
              h[q] = *reinterpret_cast<const uint32_t*>(&x);
            }
            sts128(mine + k * 2, make_uint4(h[0], h[1], h[2], h[3]));
          }
          flush([&](int, long long to, int piece, uint4 d) {
            *reinterpret_cast<uint4*>(a.out + to * D + c_at + c + piece * 8) = d;
          });
        } else {
#pragma unroll
          for (int half = 0; half < 32; half += 16) {
#pragma unroll
            for (int k = half; k < half + 16; k += 4)
              sts128(mine + (k - half) * 4,
                     make_uint4(__float_as_uint(y(k)), __float_as_uint(y(k + 1)),
                                __float_as_uint(y(k + 2)), __float_as_uint(y(k + 3))));
            flush([&](int rr, long long, int piece, uint4 d) {
              *reinterpret_cast<uint4*>(part + (size_t)(pr - lane + rr) * D + c_at + c + half +
                                        piece * 4) = d;
            });
          }
        }
      }
      if (!whole && (NT == 2 || wg == 0)) {
        part[(size_t)C::kRows * D + pr] = top;
        part[(size_t)C::kRows * (D + 1) + pr] = l;
        part[(size_t)C::kRows * (D + 2) + pr] = fac;
      }
      if (done.blk0 == 0 && !whole && tid == 0)  // begun here; it goes on at the next share's start
        cuts[blockIdx.x] = Cut{(int)(blockIdx.x + (done.rest + s_share - 1) / s_share), ri.start, ri.n,
                               done.tok0, done.kvh, {}};
      tc_before();
      __syncwarp();
    }
  } else if (wid < kMmaWarp) {
    // ------------- keys (warps 8-15) and values (16-23): a thread per key and half of the columns
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kSideRegs));
    auto side = [&](auto value_tag, uint32_t room, uint64_t* full, uint64_t* freed) {
      constexpr bool kValues = decltype(value_tag)::value;
      constexpr int KC = D / 64, KG = D == 256 ? 2 : 1;  // 16-byte chunks, quantisation groups
      const int st = (tid - kSoftWarps * 32) & 255, key = st & 127, half = st >> 7;
      const int in_tile = key & 15, sw = swizzle<D>(in_tile), g0 = half * KC / 2;
      const int codes = (kValues ? 8 * D : 0) + in_tile * (D / 2);
      const int scales =
          16 * D + 2 * (kValues ? Meta<D>::v_scale(in_tile, g0) : Meta<D>::k_scale(in_tile, g0));
      constexpr int kBias = 32 * (D / 64), kGroup = kValues ? 32 : 2;  // bytes from a scale on
      uint4 code[KC];
      uint32_t meta[KG];  // scale | bias << 16
      uint32_t n = 0;     // blocks written
      while (next_unit<D>(walk, a, r, tok, u)) {
        const int len = walk.row.len;
        const int32_t* table = a.kv.block_table + (int64_t)walk.b * a.kv.max_blocks;
        const uint8_t* pool = static_cast<const uint8_t*>(a.kv.pool) +
                              (int64_t)u.kvh * (P / kTile) * tile_bytes(D);
        const int64_t stride = (int64_t)K * (P / kTile) * tile_bytes(D);
        auto tile_at = [&](int i) -> const uint8_t* {  // the key's tile; null: it is not there
          const int j = i * kKeys + key;
          if (i >= u.blk1 || j >= len) return nullptr;
          const int block = table[j >> p_shift];
          if ((unsigned)block >= (unsigned)a.kv.num_blocks) {
            if (!kValues) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
            return nullptr;
          }
          return pool + block * stride + (j & (P - 1)) / kTile * tile_bytes(D);
        };
        auto load = [&](const uint8_t* tile) {  // zeros for a key that is not there
#pragma unroll
          for (int c = 0; c < KC; ++c) code[c] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < KG; ++c) meta[c] = 0;
          if (tile) {
#pragma unroll
            for (int c = 0; c < KC; ++c)
              code[c] = *reinterpret_cast<const uint4*>(tile + codes + (((half * KC + c) ^ sw) << 4));
#pragma unroll
            for (int c = 0; c < KG; ++c) {
              const uint16_t* x = reinterpret_cast<const uint16_t*>(tile + scales + c * kGroup);
              meta[c] = x[0] | (uint32_t)x[kBias / 2] << 16;
            }
          }
        };
        load(tile_at(u.blk0));
        const uint8_t* next = tile_at(u.blk0 + 1);
        for (int i = u.blk0; i < u.blk1; ++i) {
          if (n >= S) wait_all(&freed[(n - S) & 1u], (n - S) >> 1, s_stop);
          const uint32_t to = room + n % S * C::kBlockBytes + key * 128;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const int chunk = half * KC + c, g = D == 256 ? c / 2 : 0;
            const uint32_t w[4] = {code[c].x, code[c].y, code[c].z, code[c].w};
            const uint32_t sc = __byte_perm(meta[g], 0, 0x1010);
            const uint32_t bi = __byte_perm(meta[g], 0, 0x3232);
            const uint32_t at = to + (chunk >> 1) * (kKeys * 128);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts128(at + ((((chunk & 1) * 4 + k) ^ (key & 7)) << 4), dequant8(w[k], sc, bi));
          }
          fence_async();
          __syncwarp();
          if (lane == 0) sc::bar_arrive(su32(&full[n % S]));
          ++n;
          // (not before the fence, which would wait for them)
          load(next);
          next = tile_at(i + 2);
        }
      }
    };
    // a buffer is free when the scores (the product) of its block are over
    if (wid < kSoftWarps + kSideWarps)
      side(std::false_type{}, k_at, k_full, s_full[NT - 1]);
    else
      side(std::true_type{}, v_at, v_full, o_done[NT - 1]);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMmaRegs));
    if (wid == kMmaWarp) {
      // -------------------------------------------------------------------- MMAs
      uint32_t n_u = 0, n_k = 0, n_p = 0;  // units; blocks scored, and multiplied
      const bool leader = elect_one();
      // descriptors: a byte offset moves them by a sixteenth
      const uint64_t dq = smem_desc(q_at, 16), dk = smem_desc(k_at, 16);
      const uint64_t dv = smem_desc(v_at, kKeys * 128);
      // A tile's scores of block n_k go where the weights of the block before (two blocks before,
      // with one tile) were: their product has to be over, as MMAs of other accumulators are not
      // ordered by themselves.
      auto scores = [&](int tile) {
        const int slot = NT == 1 ? (int)(n_k & 1u) : tile, st = n_k % S;
        const uint64_t da = dq + tile * (C::kBlockBytes / 16), db = dk + st * (C::kBlockBytes / 16);
        // (the wait that is over first comes first: it is not on the way then)
        if (tile == 0) wait_all(&k_full[st], n_k / S, s_stop);
        if (n_p > 0) wait_all(&o_done[tile][(n_p - 1) & 1u], (n_p - 1) >> 1, s_stop);
        tc_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int off = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) / 16;
            mma_ss(tmem + C::kS + slot * 128, da + off, db + off, C::kIdescS, k > 0);
          }
          commit(su32(&s_full[tile][n_k & 1u]));
        }
        __syncwarp();
      };
      auto product = [&](int tile, uint32_t n, bool more) {
        const int slot = NT == 1 ? (int)(n & 1u) : tile, st = n % S;
        const uint64_t db = dv + st * (C::kBlockBytes / 16);
        if (tile == 0) wait_all(&v_full[st], n / S, s_stop);
        wait_all(&p_full[tile][n & 1u], n >> 1, s_stop);
        tc_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(tmem + tile * C::kO, tmem + C::kS + slot * 128 + k * 8, db + k * (2048 / 16),
                   C::kIdescO, more || k > 0);
          commit(su32(&o_done[tile][n & 1u]));
        }
        __syncwarp();
      };
      auto stopped = [&] { return __any_sync(~0u, s_stop) != 0; };
      while (next_unit<D>(walk, a, r, tok, u)) {
        wait_all(&q_full, n_u++, s_stop);
        const int nb = u.blk1 - u.blk0;
        if constexpr (NT == 1) {
          for (int i = 0; i <= nb && !stopped(); ++i) {
            if (i < nb) {
              scores(0);
              ++n_k;
            }
            if (i > 0) product(0, n_p++, i > 1);
          }
        } else {
          scores(0);
          scores(1);
          ++n_k;
          for (int i = 0; i < nb && !stopped(); ++i) {
            product(0, n_p, i > 0);
            ++n_p;
            if (i + 1 < nb) scores(0);
            product(1, n_p - 1, i > 0);
            if (i + 1 < nb) {
              scores(1);
              ++n_k;
            }
          }
        }
        if (stopped()) break;
      }
      if (leader) commit(su32(&drained));  // nothing is under way when TMEM goes back
      __syncwarp();
      if (!__all_sync(~0u, bar_wait(su32(&drained), 0))) s_stop = 1;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  griddep_launch();
  if (tid == 0 && s_stop) {
    atomicOr(a.batch.err, MOE_DERR_WAIT);
    cuts[blockIdx.x].last = -1;
  }
  if (wid == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// Units that were cut between CTAs, each found at the CTA that began it: a
// thread per query row and four columns, its parts in order.
template <int D>
__global__ void __launch_bounds__(512) combine_kernel(AttnArgs a) {
  using C = Cfg<D>;
  griddep_wait();
  const int first = blockIdx.x, at = blockIdx.y * 512 + threadIdx.x;
  const int row = at / (D / 4), c = at % (D / 4) * 4;
  const Cut cut = static_cast<const Cut*>(a.ws)[first];
  if (cut.last <= first) return;
  const int r = a.heads / a.kv.kv_heads, per_tile = 128 / r, in = row & 127;
  const int t = cut.tok0 + (row >> 7) * per_tile + in / r;
  if (in >= per_tile * r || t >= cut.n) return;
  const float* parts = reinterpret_cast<const float*>(static_cast<const char*>(a.ws) + kCutBytes);
  float m = kNone, l = 0.0f;  // (raw scores, as the parts have them)
  const float fac = parts[((size_t)first * 2 + 1) * C::kPartial + (size_t)C::kRows * (D + 2) + row];
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = first; k <= cut.last; ++k) {
    const float* src = parts + ((size_t)k * 2 + (k == first)) * C::kPartial;
    const float mk = src[(size_t)C::kRows * D + row], lk = src[(size_t)C::kRows * (D + 1) + row];
    const float4 v = *reinterpret_cast<const float4*>(src + (size_t)row * D + c);
    const float mm = fmaxf(m, mk), f = ex2((m - mm) * fac), h = ex2((mk - mm) * fac);
    m = mm;
    l = l * f + lk * h;
    y.x = y.x * f + v.x * h;
    y.y = y.y * f + v.y * h;
    y.z = y.z * f + v.z * h;
    y.w = y.w * f + v.w * h;
  }
  const float inv = l > 0.0f ? 1.0f / l : l;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * inv, y.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(y.z * inv, y.w * inv);
  *reinterpret_cast<uint2*>(a.out + ((int64_t)(cut.start + t) * a.heads + cut.kvh * r + in % r) * D +
                            c) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e == cudaSuccess)
    e = launch_pdl(prompt_kernel<D>, dim3(kGrid), dim3(kThreads), C::kSmem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine_kernel<D>, dim3(kGrid, C::kRows * D / 2048), dim3(512), 0, st, a);
}

template <int D>
size_t bytes_for() {
  return kCutBytes + (size_t)kGrid * 2 * Cfg<D>::kPartial * 4;
}

}  // namespace

size_t prompt_workspace_bytes(int D) {
  return D == 256 ? bytes_for<256>() : D == 128 ? bytes_for<128>() : bytes_for<64>();
}

cudaError_t launch_prompt(const AttnArgs& a, cudaStream_t st) {
  const int D = a.kv.head_dim;
  return D == 256 ? launch<256>(a, st) : D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace kv
}  // namespace moe
