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
// View: windows and trees.  A unit's blocks are the key tiles of the sinks and of the window of
// its tokens, without the gap between them; what a token does not see of a block at either end
// is taken out of its scores, by bounds or by a tree's bits.  Split (View, head_dim 64 and 128):
// where no row has more queries than one tile, the two tiles take a unit's key blocks in turn,
// with the same queries, and join their results in the end (32 trees of 32 tokens, 4 heads on one
// of 8: 106 us, 164 with the second tile empty).
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
//               K-major and the values MN-major by the MMAs.  The values' warps
//               also bring the next unit's queries, while the softmax is still at
//               this one's last block and results.
//   warp 24     issues the MMAs (M = 128, fp32 accumulators in TMEM): the next
//               block's scores run while the softmax works on this one's.
//   warp 25     walks over the share and hands out its units, up to four ahead (each
//               role walking for itself, its code cold: 8192 tokens through a window of
//               1024 took 235 us, with everything around it, now 196).
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
// Measured: 8192 tokens, 16 query heads on 2 of 256: 487 us, 1129 TFLOP/s (58% of a
// large bf16 matrix product), through a window of 1024 195 to 202 us; 2048 tokens on 30000, 32
// heads on 4 of 128: 780 us, 1333 TFLOP/s (68%), through a window of 4096 145 us, 950
// TFLOP/s; 32 trees of up to 64 tokens on 150 to 8191 keys, 32 heads on 8 of 128: 165 us.
// The compiler spills 72 and 120 bytes a thread at head_dim 64 and 128, none at 256 (View: 168,
// 172 and 20; its split form 136 and 136).  Bound by the
// chain of a block: at head_dim 64 and 128 scores,
// TMEM load, exponentials, TMEM store, product; at 256, whose one block of values
// takes all the shared memory there is, values freed, dequantised (1400 cycles),
// fenced (570), seen by the issuer (350) and multiplied (1500).  The tensor pipe is
// busy 57% (128) and 49% (256) of the time, the issue slots 57 and 59%; through windows
// 44 and 32%, 51 and 49%: a unit's ends (queries in 4000 cycles where they are not hidden, results
// out 4500, a share's first unit 14000, blocks with hidden keys 3000 more than others)
// weigh on the 9 (33) blocks that it has there, its code for them not in the SM's
// instruction cache.  Measured and
// dropped: two tiles with the next scores in halves of 64 keys, the first before
// the product (975 us then against 876), a warp of its own that issues for each
// tile (1046); one tile with keys and values handed over by halves of the columns
// (575 against 516), with a second issuing warp for the products (556); split units among
// others in one kernel (the flags alone: 861 us for 2048 tokens on 30000 instead of 786);
// queries by two warps of their own (260 us for the window of 1024), by both dequantising
// groups (228 instead of 225), with a block's tiles brought to L2 ahead (225 instead of 221 us for
// 32 trees); warps without a query that leave their rows out (167 instead of 165 us for 32 trees, 150
// instead of 146 through the window of 4096); split units for rows of up to two tiles (186 instead of
// 165 us for 32 trees of up to 64 tokens).
#pragma once
#include <climits>
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
constexpr int kThreads = 28 * 32;  // seven warp groups; two warps of the last one idle
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
  static constexpr size_t kSmem = 1024 + (size_t)(kTiles + 2 * kStages) * kBlockBytes;
  static constexpr int kPartial = kRows * (D + 3);  // floats: o [row][D], top, l, fac [row]
  static constexpr uint32_t kIdescS = (1u << 4) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                      ((128u >> 4) << 24);  // bit 16: B is MN-major
  static constexpr int kO = D == 256 ? 256 : 128;   // TMEM columns between the tiles' results
  static constexpr int kS = 256;                    // scores: two slots of 128 columns
  // (8192 tokens, head_dim 256, through a window of 1024 and causal, us: 96, 64, 48 registers 196 and
  // 487; 112, 56, 48 200 and 496; 80, 72, 48 201 and 478.  2048 on 30000, 128, through 4096 and
  // causal: 136, 48, 40 147 and 772; 120, 56, 40 148 and 773; 112, 56, 56 160 and 792)
  static constexpr int kSoftRegs = D == 256 ? 96 : 136, kSideRegs = D == 256 ? 64 : 48;
  static constexpr int kMmaRegs = D == 256 ? 48 : 40;
  static_assert(kSoftRegs * 256 + kSideRegs * 512 + kMmaRegs * 128 <= kStartRegs * kThreads,
                "the registers given out are there");
};

// The unit that a CTA began and did not end: the last CTA with a part of it (-1: there is none).
struct Cut {
  int last, start, end, tok0, kvh, pad[3];  // tokens tok0 .. end - 1
};
constexpr size_t kCutBytes = (kGrid * sizeof(Cut) + 255) / 256 * 256;

struct Row {
  int start, n, len, tiles;  // tiles 0: nothing here
};

// Whether the row's tokens see each other by a tree's bits (longer rows are chains).
template <bool View>
__device__ __forceinline__ bool by_tree(const AttnArgs& a, const Row& i) {
  return View && a.tree && i.n <= a.tree_max;
}
// The first position that the window leaves to any token from tok0 on (a tree's tokens have
// depths in any order).
template <bool View>
__device__ __forceinline__ int first_seen(const AttnArgs& a, const Row& i, int tok0) {
  if (!View || a.window <= 0) return 0;
  return i.len - i.n + (by_tree<View>(a, i) ? 0 : tok0) - a.window + 1;
}
// Keys that a unit walks over at most, by its window (the sinks' tiles and one cut by the window's
// begin among them); no limit without one.
template <bool View>
__device__ __forceinline__ long long most_keys(const AttnArgs& a, const Row& i, int tok) {
  if (!View || a.window <= 0) return LLONG_MAX / 4;
  return (long long)a.window + a.sinks + (by_tree<View>(a, i) ? i.n : tok) + 2 * kTile;
}

// (the decode kernel, which sees every row, reports what does not fit)
template <bool View>
__device__ __forceinline__ Row row_info(const AttnArgs& a, const RowBounds& w, int r, int tok, int mode) {
  Row i = {w.start, w.n, w.len, 0};
  if (w.ok && !takes_decode<View>(a, w.n, r, mode)) i.tiles = (i.n + tok - 1) / tok;
  return i;
}

// Costs of a row's units: each its keys (taking every tile for a full one; with a window `most` at
// most, which the units from `full` on have) and a fixed part.
struct Costs {
  long long base, most;
  int tok, full;
};
template <bool View>
__device__ __forceinline__ Costs costs_of(const AttnArgs& a, const Row& i, int tok) {
  Costs c = {i.len - i.n, 0, tok, INT_MAX};
  if constexpr (View) {
    c.most = most_keys<View>(a, i, tok);
    if (a.window > 0) {
      const long long more = c.most - c.base;
      c.full = more < 0 ? 0 : more > INT_MAX ? INT_MAX : (int)more / tok;
    }
  }
  return c;
}
template <int D, bool View>
__device__ __forceinline__ long long cost_of(const Costs& c, int j) {
  const long long keys = c.base + (long long)(j + 1) * c.tok;
  return (View && j >= c.full ? c.most : keys) + Cfg<D>::kUnitKeys;
}
// of the first j of them
template <int D, bool View>
__device__ __forceinline__ long long cost_before(const Costs& c, int j) {
  const long long k = View ? min(j, c.full) : j;
  long long x = (long long)j * Cfg<D>::kUnitKeys + k * c.base + (long long)c.tok * (k * (k + 1) / 2);
  if constexpr (View)
    if (k < j) x += (j - k) * c.most;
  return x;
}

// A unit, or a CTA's share of one, as it is handed to the roles.
struct __align__(16) Job {
  int more;                // 0: there are no more units
  int b, start, n, len;    // its row
  int kvh, tok0;           // kv head, first token
  int blk0, blk1, blocks;  // key blocks of this share, and of the unit
  int low, gap;            // View: the first position that the window leaves to any of its tokens,
                           // and the tiles between the sinks' and that one's
  int last;                // the last CTA with a part of a unit that is begun here and not ended
};
constexpr int kJobs = 4;
constexpr int kTakers = kSoftWarps + 2 * kSideWarps + 1;  // warps that take jobs

// The walk over a CTA's share.
struct Walk {
  int b, kvh, j;
  long long at, left, share;  // offset in unit (kvh, j) where the share goes on; what is left of it
  int mode;
  Row row;
  Costs costs;
};

template <int D, bool View>
__device__ __forceinline__ bool next_unit(Walk& w, const AttnArgs& a, int r, int tok, Job& u) {
  constexpr int kUnitKeys = Cfg<D>::kUnitKeys;
  while (w.left > 0) {
    if (w.kvh >= a.kv.kv_heads) {
      do {
        if (++w.b >= a.rows) return false;
        w.row = row_info<View>(a, row_bounds(a, w.b), r, tok, w.mode);
      } while (w.row.tiles == 0);
      w.costs = costs_of<View>(a, w.row, tok);
      w.kvh = w.j = 0;
      w.at = 0;
    }
    const int seen = w.row.len - w.row.n + min(w.row.n, (w.j + 1) * tok);
    const long long cost = cost_of<D, View>(w.costs, w.j);
    u.b = w.b;
    u.start = w.row.start;
    u.n = w.row.n;
    u.len = w.row.len;
    u.kvh = w.kvh;
    u.tok0 = w.j * tok;
    u.blocks = (seen - 1) / kKeys + 1;  // (seen + kKeys may pass 2^31 - 1)
    u.low = u.gap = 0;
    if constexpr (View) {
      u.low = first_seen<View>(a, w.row, u.tok0);
      u.gap = sight_of(a, u.low).gap;
      u.blocks = (seen - u.gap * kTile - 1) / kKeys + 1;
    }
    // both ends of a share fall on the same block for the CTAs on either side
    auto block_at = [&](long long x) {
      const long long k = (x - kUnitKeys + kKeys / 2) / kKeys;
      return x <= kUnitKeys ? 0 : (int)min(k, (long long)u.blocks);
    };
    u.blk0 = block_at(w.at);
    const bool whole = w.left >= cost - w.at;
    u.blk1 = whole ? u.blocks : block_at(w.at + w.left);
    u.last = -1;
    if (u.blk0 == 0 && u.blk1 < u.blocks) {
      // it goes on at the next share's start: what of its cost behind there still holds blocks
      const long long rest =
          min(cost, kUnitKeys + (long long)u.blocks * kKeys - kKeys / 2) - (w.at + w.left);
      u.last = (int)(blockIdx.x + (rest + w.share - 1) / w.share);
    }
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

// 32 bytes, a whole sector
__device__ __forceinline__ void stg256(void* to, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Split: a unit is one tile of queries, whose key blocks two tiles take in turn.
template <int D, bool View, bool Split>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(AttnArgs a) {
  using C = Cfg<D>;
  constexpr int NT = C::kTiles, S = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  // A block of keys or values is there; a tile's scores, weights, product are.  The last two by
  // the block's parity: a buffer's next block waits for the scores (products) of the block that
  // it replaces, which are never more than one phase of that barrier ago.
  __shared__ __align__(8) uint64_t k_full[S], v_full[S], p_full[NT][2];
  __shared__ __align__(8) uint64_t s_full[NT][2], o_done[NT][2], drained;
  // a unit's queries are there; by the job's place, as the factors: those of the next units may come
  // before a softmax warp has looked for these (of a split unit of one block the second tile's
  // warps hold nobody up), and a place is filled again only after every warp has given its job back
  __shared__ __align__(8) uint64_t q_full[kJobs];
  __shared__ __align__(8) uint64_t k_free[S], v_free[S], q_free;  // nothing reads the buffer any more
  __shared__ __align__(8) uint64_t job_full[kJobs], job_free[kJobs];
  __shared__ Job s_job[kJobs];
  __shared__ uint32_t tmem_slot;
  __shared__ long long s_scan[kThreads / 32], s_at;
  __shared__ int s_row;
  __shared__ volatile int s_stop;  // a wait ran out
  // factors of the rows' scores, by the job's place
  __shared__ float s_fac[kJobs][C::kRows], s_max[2][128], s_sum[2][128];
  // key tiles of a block that are missing (a block id outside the pool): two bits of each byte, of
  // the last four blocks (the softmax reads a block's before the keys' side writes the fourth
  // behind it, which waits for scores that come after this block's weights)
  __shared__ uint32_t s_miss[4];
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int K = a.kv.kv_heads, r = a.heads / K, P = a.kv.block_tokens;
  const int p_shift = 31 - __clz(P);
  static_assert(NT == 2 || !Split, "two tiles");
  constexpr int kUnitTiles = Split ? 1 : NT;
  const int per_tile = 128 / r, tok = per_tile * kUnitTiles;  // tokens of a tile, of a unit
  const uint32_t r_inv = (65536 + r - 1) / r;         // x * r_inv >> 16 = x / r for x < 128
  const uint32_t base = (su32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, k_at = q_at + NT * C::kBlockBytes, v_at = k_at + S * C::kBlockBytes;

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
      bar_init(su32(&k_free[i]), 1);
      bar_init(su32(&v_free[i]), 1);
    }
    for (int i = 0; i < 2 * NT; ++i) {
      bar_init(su32(&s_full[0][0] + i), 1);
      bar_init(su32(&o_done[0][0] + i), 1);
      bar_init(su32(&p_full[0][0] + i), kSoftWarps / NT);
    }
    for (int i = 0; i < kJobs; ++i) {
      bar_init(su32(&q_full[i]), kSoftWarps);
      bar_init(su32(&job_full[i]), 1);
      bar_init(su32(&job_free[i]), kTakers);
    }
    bar_init(su32(&q_free), 1);
    bar_init(su32(&drained), 1);
    s_row = -1;
    s_stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  griddep_wait();
  Cut* cuts = static_cast<Cut*>(a.ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kCutBytes);
  if (tid == 0) cuts[blockIdx.x].last = -1;

  // ------------------------------------------------------- this CTA's share
  long long total = 0;
  auto share_of = [&] { return max((total + kGrid - 1) / kGrid, 2ll * kKeys); };
  auto row_cost = [&](const Row& i) {
    return i.tiles ? K * cost_before<D, View>(costs_of<View>(a, i, tok), i.tiles) : 0ll;
  };
  const int chunks = (a.rows + kThreads - 1) / kThreads;
  const int mode = View ? *a.mode : kByColumns;
  // Up to 32 rows are the walking warp's own business, a lane per row (below).  More: chunks of
  // kThreads rows, twice over when there is more than one (the total comes first)
  for (int pass = a.rows <= 32 || mode == kAllDecode ? 2 : chunks > 1 ? 0 : 1; pass < 2; ++pass) {
    long long carry = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c * kThreads + tid;
      long long cost = 0;
      if (b < a.rows) cost = row_cost(row_info<View>(a, row_bounds(a, b), r, tok, mode));
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
        const long long pre = before + v - cost, x0 = blockIdx.x * share_of();
        if (x0 < total && x0 >= pre && x0 < pre + cost) {
          s_row = b;
          s_at = x0 - pre;
        }
      }
      carry += sum;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  auto stopped = [&] { return __any_sync(~0u, s_stop) != 0; };
  // job k of this CTA: whether there is one; it stays in its place until the warp has given it back
  auto take = [&](uint32_t k) {
    wait_all(&job_full[k % kJobs], k / kJobs, s_stop);
    return !stopped() && s_job[k % kJobs].more != 0;
  };
  auto give = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) sc::bar_arrive(su32(&job_free[k % kJobs]));
  };
  // the row's tile that a unit's walk has as its tile t
  auto tile_of = [&](const Job& u, int t) {
    return View && u.gap && t >= sight_of(a, 0).sink_tiles ? t + u.gap : t;
  };
  // A unit's queries by eight warps, of which this is one: a warp's rows, 8 columns a lane, some
  // loads under way at a time.
  auto load_queries = [&](auto deep_tag, int warp, uint32_t n_u) {
    constexpr int kWarps = kSoftWarps;
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kRounds = 128 * kUnitTiles / kWarps / kAtOnce;
    constexpr int kMost = decltype(deep_tag)::value, kDeep = kRounds < kMost ? kRounds : kMost;
    static_assert(kRounds % kDeep == 0, "whole batches");
    const Job& u = s_job[n_u % kJobs];
    const int col8 = lane % kLanes;
    const int n = u.n, tok0 = u.tok0;
    const uint16_t* src = a.q + ((int64_t)(u.start + tok0) * a.heads + u.kvh * r) * D + col8 * 8;
    for (int i0 = 0; i0 < kRounds; i0 += kDeep) {
      uint4 raw[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int qr = (warp * kRounds + i0 + i) * kAtOnce + lane / kLanes, in = qr & 127;
        const int i_tok = (int)(in * r_inv >> 16), t = (qr >> 7) * per_tile + i_tok;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (in < per_tile * r && tok0 + t < n)
          raw[i] = *reinterpret_cast<const uint4*>(src + ((int64_t)t * a.heads + in - i_tok * r) * D);
      }
      // (the buffer is free once the last scores of the unit before are there)
      if (i0 == 0 && n_u > 0) wait_all(&q_free, n_u - 1, s_stop);
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int qr = (warp * kRounds + i0 + i) * kAtOnce + lane / kLanes, in = qr & 127;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) big = __vmaxu2(big, w[k] & 0x7FFF7FFFu);
        big = max(big & 0xFFFFu, big >> 16);
        if constexpr (kLanes == 32) {
          big = __reduce_max_sync(~0u, big);
        } else {
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) big = max(big, __shfl_xor_sync(~0u, big, o));
        }
        const int e = max((int)(big >> 7) - 127, -100);  // 2^e <= largest < 2^(e+1)
        const float up = pow2(14 - e);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[2 * k] = __uint_as_float(w[k] << 16) * up;
          x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * up;
        }
        sts128(q_at + (qr >> 7) * C::kBlockBytes + (col8 >> 3) * (kKeys * 128) + in * 128 +
                   (((col8 & 7) ^ (in & 7)) << 4),
               make_uint4(pack_h2(x[0], x[4]), pack_h2(x[1], x[5]), pack_h2(x[2], x[6]),
                          pack_h2(x[3], x[7])));
        // score = fac * accumulated, in units of log2
        if (col8 == 0)
          s_fac[n_u % kJobs][qr] = score_factor(a.scale, 8.8054160e-05f, e);  // log2(e) 2^-14 2^e
      }
    }
    fence_async();
    __syncwarp();
    if (lane == 0) sc::bar_arrive(su32(&q_full[n_u % kJobs]));
  };

  if (wid < kSoftWarps) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int wg = wid >> 2, row = (wid & 3) * 32 + lane;  // TMEM lane
    const int tile = NT == 1 ? 0 : wg;
    const uint32_t lanes = (uint32_t)((wid & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lanes + tile * C::kO;
    uint32_t n = 0;  // blocks seen
    auto is_tree = [&](const Job& u) { return View && a.tree && u.n <= a.tree_max; };
    // View: where the window of the unit's last token begins
    auto last_low = [&](const Job& u) {
      if (!View || a.window <= 0) return 0;
      return u.len - u.n + (is_tree(u) ? u.n : min(u.n, u.tok0 + tok)) - a.window;
    };
    // the token of this thread's row
    auto token_of = [&](const Job& u, int q_tile) {
      return u.tok0 + q_tile * per_tile + (int)(row * r_inv >> 16);
    };
    uint32_t n_u = 0;
    [[maybe_unused]] uint32_t n_blocks = 0;  // of the units before
    bool have = take(0);
    // (idle as yet, these warps bring the first unit's queries)
    if (have) load_queries(std::integral_constant<int, 8>{}, wid, 0);
    // (every softmax warp leaves at the same unit: they meet at barriers on the way)
    for (; !any_of_256(!have); ++n_u) {
      const Job& u = s_job[n_u % kJobs];
      const int q_tile = Split ? 0 : tile;  // the tile of the queries
      wait_all(&q_full[n_u % kJobs], n_u / kJobs, s_stop);
      const float fac = s_fac[n_u % kJobs][q_tile * 128 + row];
      // Blocks of which every row of the tile sees every key.  (A block's end, and that of a tile without
      // queries, may lie behind 2^31 - 1: unsigned.)
      const int base0 = u.len - u.n;
      const uint32_t open = is_tree(u) ? base0 : (uint32_t)base0 + u.tok0 + q_tile * per_tile + 1;
      int free0 = 0, free1 = (int)(open / kKeys);
      if constexpr (View) {
        constexpr int kTiles = kKeys / kTile;
        // (both ends lie behind the gap)
        free0 = (max(0, (max(last_low(u), 0) + kTile - 1) / kTile - u.gap) + kTiles - 1) / kTiles;
        free1 = ((int)(open / kTile) - u.gap) / kTiles;
      }
      // The row's reference, a raw score; a score x weighs 2^(x fac + off), off = 7 - top fac.
      // Where that is far from zero every visible score shall weigh too much (an infinite query's
      // row is lost anyway, and the others' references shall not follow for it).
      float top = kNone, off, l = 0.0f;
      auto set_off = [&] {
        off = fmaf(-top, fac, 7.0f);
        if (fabsf(off) > kFar && top < -kNone) off = 3e38f;
      };
      set_off();
      constexpr int by = Split ? 2 : 1;
      const int i0 = u.blk0 + (Split ? tile : 0), i1 = u.blk1;
      for (int i = i0; i < i1; i += by) {
        const int slot = NT == 1 ? (int)(n & 1u) : tile;
        wait_all(&s_full[tile][n & 1u], n >> 1, s_stop);
        tc_after();
        const uint32_t s_tm = tmem + lanes + C::kS + slot * 128;
        const uint32_t miss = s_miss[(Split ? n_blocks + i - u.blk0 : n) & 3u];
        const bool edge = (View && i < free0) || i >= free1 || miss != 0;
        // 64 columns (four key tiles) from column c * 16 on: what the row does not see is taken out.
        // (All of it is found again from the job: kept, it would take registers from the others.)
        auto is_missing = [&](int c) { return (miss >> (c / 2 * 8 + c % 2) & 1u) != 0; };
        auto hide = [&](uint32_t* v, int c0) {
          const int t = min(token_of(u, q_tile), u.n - 1), base = u.len - u.n;
          if constexpr (View) {
            const bool tree = is_tree(u);
            const int tree0 = tree ? base : INT_MAX, lim = tree ? u.len - 1 : base + t;
            const uint32_t open = tree ? base : (uint32_t)base + u.tok0 + q_tile * per_tile + 1;
            const int shut = last_low(u);
            const uint32_t* bits = a.tree + (size_t)(u.start + t) * a.words + 1;
            // (not below 0: with a key taken off it stays within 32 bits, however large the window)
            const int low = a.window > 0 ? max(base + (tree ? (int)bits[-1] : t) - a.window + 1, 0) : 0;
            uint32_t see[2] = {~0u, ~0u};
#pragma unroll(D == 64 ? 4 : 1)
            for (int q = 0; q < 4; ++q) {
              // (tiles behind the last position that there can be count as that one's, which no token sees)
              const int key = min(tile_of(u, i * (kKeys / kTile) + c0 + q), INT_MAX / kTile) * kTile;
              if ((uint32_t)key + kTile <= open && !is_missing(c0 + q) &&
                  (key >= shut || key <= a.sinks - kTile))
                continue;
              uint32_t x = below16(lim - key + 1);
              if (tree && key > tree0 - kTile) {
                const int at = key - tree0;  // -15 and on: the first -at keys are cached ones
                const int w = max(at, 0) >> 5, words = a.words - 1;
                const uint32_t lo = w < words ? bits[w] : 0u, hi = w + 1 < words ? bits[w + 1] : 0u;
                x &= at < 0 ? lo << -at | ((1u << -at) - 1u) : __funnelshift_r(lo, hi, at & 31);
              }
              // (a tree's key lies at its depth, not at its place: its bits know of the window)
              x &= ~(below16(min(low, tree0) - key) & ~below16(a.sinks - key));
              if (is_missing(c0 + q)) x = 0u;
              const uint32_t gone = ~x & 0xFFFFu;
              if (q & 2) see[1] &= ~(gone << (q * 16 & 31));
              else see[0] &= ~(gone << (q * 16 & 31));
            }
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (!((see[k >> 5] >> (k & 31)) & 1u)) v[k] = 0xFF800000u;
          } else {
            const int lim = base + t - i * kKeys;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int last = is_missing(c0 + q) ? -1 : lim - (c0 + q) * 16;
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (k > last) v[16 * q + k] = 0xFF800000u;
            }
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
          if (i > i0 && __any_sync(~0u, f != 1.0f)) {
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
            if (edge) hide(v, wg * 4);
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
          bool follow = i == i0;
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
            if (edge) hide(x, 4 * c);
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
      // ---- the unit's end (here): a result, or a part of one
      if (i0 < i1) wait_all(&o_done[tile][(n - 1) & 1u], (n - 1) >> 1, s_stop);
      tc_after();
      float f_mine = 1.0f, f_other = 0.0f;
      if (NT == 1 || Split) {
        const int other = wg ^ 1;
        s_sum[wg][row] = l;
        if (NT == 2) s_max[wg][row] = top;
        tc_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_after();
        if constexpr (NT == 1) {
          l += s_sum[other][row];
        } else {
          // both tiles' results of the same queries
          const float top_o = s_max[other][row], both = fmaxf(top, top_o);
          f_mine = ex2((top - both) * fac);
          f_other = ex2((top_o - both) * fac);
          l = l * f_mine + s_sum[other][row] * f_other;
          top = both;
        }
      }
      // (a tile that had no block of it has no result either)
      const bool mine = i0 < i1, others = u.blk0 + (tile ^ 1) < i1;
      const bool whole = u.blk0 == 0 && u.blk1 == u.blocks;
      const float inv = whole ? (l > 0.0f ? 1.0f / l : l) : 1.0f;
      f_mine *= inv;
      f_other *= inv;
      const int t = token_of(u, q_tile);
      const bool live = row < per_tile * r && t < u.n;
      uint16_t* dst = a.out + ((int64_t)(u.start + t) * a.heads + u.kvh * r + row - (int)(row * r_inv >> 16) * r) * D;
      float* part = parts + ((size_t)blockIdx.x * 2 + (u.blk0 == 0 ? 1 : 0)) * C::kPartial;
      const int pr = q_tile * 128 + row;
      have = take(n_u + 1);
      // A lane holds a row's columns: 32 at a time, in whole sectors.  (Where `out` is not aligned
      // to them, half sectors.)
      constexpr bool halves = NT == 1 || Split;  // of the columns, one for either tile (warp group)
      const int c_at = halves ? wg * (D / 2) : 0, c_end = halves ? c_at + D / 2 : D;
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll 1
      for (int c = c_at; c < c_end; c += 32) {
        uint32_t v[32];
        if constexpr (Split) {
          uint32_t w[32];
          tm_ld32(tmem + lanes + wg * C::kO + c, v);
          tm_ld32(tmem + lanes + (wg ^ 1) * C::kO + c, w);
          tm_wait_regs(v);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            asm volatile("" : "+r"(w[k]));
            const float x = mine ? __uint_as_float(v[k]) * f_mine : 0.0f;
            v[k] = __float_as_uint(others ? fmaf(__uint_as_float(w[k]), f_other, x) : x);
          }
        } else {
          tm_ld32(o_tm + c, v);
          tm_wait_regs(v);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f_mine);
        }
        // columns in order: 0,4,1,5,2,6,3,7 -> 0..7
        auto y = [&](int k) { return v[(k & ~7) + (k & 3) * 2 + ((k >> 2) & 1)]; };
        if (whole) {
          uint32_t h[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(y(2 * k)),
                                                           __uint_as_float(y(2 * k + 1)));
            h[k] = *reinterpret_cast<const uint32_t*>(&x);
          }
          if (live) {
            if (wide) {
              stg256(dst + c, h);
              stg256(dst + c + 16, h + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                *reinterpret_cast<uint4*>(dst + c + 2 * k) =
                    make_uint4(h[k], h[k + 1], h[k + 2], h[k + 3]);
            }
          }
        } else if (live) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const uint32_t h[8] = {y(k), y(k + 1), y(k + 2), y(k + 3), y(k + 4), y(k + 5), y(k + 6), y(k + 7)};
            stg256(part + (size_t)pr * D + c + k, h);
          }
        }
      }
      if (!whole && (halves ? wg == 0 : true)) {
        part[(size_t)C::kRows * D + pr] = top;
        part[(size_t)C::kRows * (D + 1) + pr] = l;
        part[(size_t)C::kRows * (D + 2) + pr] = fac;
      }
      n_blocks += u.blk1 - u.blk0;
      if (u.last >= 0 && tid == 0)
        cuts[blockIdx.x] = Cut{u.last, u.start, min(u.n, u.tok0 + tok), u.tok0, u.kvh, {}};
      tc_before();
      give(n_u);
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
      for (uint32_t n_u = 0; take(n_u); ++n_u) {
        const Job& u = s_job[n_u % kJobs];
        const int len = u.len, blk0 = u.blk0, blk1 = u.blk1, low = u.low;
        [[maybe_unused]] uint32_t sink_keys = 0, gap_keys = 0;
        if constexpr (View) {
          sink_keys = u.gap ? sight_of(a, 0).sink_tiles * kTile : 0;
          gap_keys = u.gap * kTile;
        }
        const int32_t* table = a.kv.block_table + (int64_t)u.b * a.kv.max_blocks;
        const uint8_t* pool = static_cast<const uint8_t*>(a.kv.pool) +
                              (int64_t)u.kvh * (P / kTile) * tile_bytes(D);
        const int64_t stride = (int64_t)K * (P / kTile) * tile_bytes(D);
        bool lost = false;  // what tile_at found last: the tile's block id lies outside the pool
        auto tile_at = [&](int i) -> const uint8_t* {  // the key's tile; null: it is not there
          lost = false;
          uint32_t j = (uint32_t)i * kKeys + key;  // (may pass 2^31 - 1 behind the row's end)
          if constexpr (View)
            if (j >= sink_keys) j += gap_keys;
          if (i >= blk1 || j >= (uint32_t)len) return nullptr;
          // (the window's begin within a tile, and behind the sinks: nothing is read there)
          if (View && (int)j < low && (int)j >= a.sinks) return nullptr;
          const int block = table[j >> p_shift];
          if ((unsigned)block >= (unsigned)a.kv.num_blocks) {
            if (!kValues) atomicOr(a.batch.err, MOE_DERR_KV_INDEX);
            lost = true;
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
        // (the values' side, which is the last to be needed, brings the queries of the units
        // behind the first one)
        // (eight loads under way spill what its loop over the blocks needs: 853 us instead of 779 for
        // 2048 tokens on 30000 of head_dim 128; split units, 32 trees of 32 tokens: 123 us with four)
        if (kValues && n_u > 0)
          load_queries(std::integral_constant<int, Split ? 2 : 4>{}, wid - kSoftWarps - kSideWarps, n_u);
        load(tile_at(blk0));
        bool lost_now = lost;
        const uint8_t* next = tile_at(blk0 + 1);
        for (int i = blk0; i < blk1; ++i) {
          const int st = n % S;
          if (n >= S) wait_all(&freed[st], n / S - 1, s_stop);
          const uint32_t to = room + st * C::kBlockBytes + key * 128;
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
          if (!kValues && half == 0) {
            const uint32_t gone = __ballot_sync(~0u, lost_now);
            if (lane == 0)
              reinterpret_cast<uint8_t*>(&s_miss[n & 3u])[key >> 5] = (uint8_t)((gone & 0xFFFFu ? 1 : 0) | (gone >> 16 ? 2 : 0));
          }
          fence_async();
          __syncwarp();
          if (lane == 0) sc::bar_arrive(su32(&full[st]));
          ++n;
          lost_now = lost;
          // (not before the fence, which would wait for them)
          load(next);
          next = tile_at(i + 2);
        }
        give(n_u);
      }
    };
    // (a buffer is free when the scores, or the products, of its block are over)
    if (wid < kSoftWarps + kSideWarps)
      side(std::false_type{}, k_at, k_full, k_free);
    else
      side(std::true_type{}, v_at, v_full, v_free);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMmaRegs));
    if (wid == kMmaWarp) {
      // -------------------------------------------------------------------- MMAs
      uint32_t n_k = 0, n_v = 0;                  // blocks of keys and values used
      uint32_t n_s[NT] = {}, n_p[NT] = {};        // each tile's scores and products
      const bool leader = elect_one();
      // descriptors: a byte offset moves them by a sixteenth
      const uint64_t dq = smem_desc(q_at, 16), dk = smem_desc(k_at, 16);
      const uint64_t dv = smem_desc(v_at, kKeys * 128);
      // A tile's scores go where the weights of its block before (two blocks before, with one
      // tile) were: their product has to be over, as MMAs of other accumulators are not ordered by
      // themselves.
      // (first, last: of the tiles that use the block; end: of the unit's scores)
      auto scores = [&](auto tile_tag, int q_tile, bool first, bool last, bool end) {
        constexpr int tile = decltype(tile_tag)::value;
        const int slot = NT == 1 ? (int)(n_s[tile] & 1u) : tile, st = n_k % S;
        const uint64_t da = dq + q_tile * (C::kBlockBytes / 16), db = dk + st * (C::kBlockBytes / 16);
        // (the wait that is over first comes first: it is not on the way then)
        if (first) wait_all(&k_full[st], n_k / S, s_stop);
        if (n_p[tile] > 0) wait_all(&o_done[tile][(n_p[tile] - 1) & 1u], (n_p[tile] - 1) >> 1, s_stop);
        tc_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int off = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) / 16;
            mma_ss(tmem + C::kS + slot * 128, da + off, db + off, C::kIdescS, k > 0);
          }
          commit(su32(&s_full[tile][n_s[tile] & 1u]));
          if (last) commit(su32(&k_free[st]));
          if (end) commit(su32(&q_free));
        }
        __syncwarp();
        ++n_s[tile];
        n_k += last;
      };
      auto product = [&](auto tile_tag, bool first, bool last, bool more) {
        constexpr int tile = decltype(tile_tag)::value;
        const uint32_t n = n_p[tile];
        const int slot = NT == 1 ? (int)(n & 1u) : tile, st = n_v % S;
        const uint64_t db = dv + st * (C::kBlockBytes / 16);
        if (first) wait_all(&v_full[st], n_v / S, s_stop);
        wait_all(&p_full[tile][n & 1u], n >> 1, s_stop);
        tc_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ts(tmem + tile * C::kO, tmem + C::kS + slot * 128 + k * 8, db + k * (2048 / 16),
                   C::kIdescO, more || k > 0);
          commit(su32(&o_done[tile][n & 1u]));
          if (last) commit(su32(&v_free[st]));
        }
        __syncwarp();
        ++n_p[tile];
        n_v += last;
      };
      using T0 = std::integral_constant<int, 0>;
      using T1 = std::integral_constant<int, NT - 1>;
      for (uint32_t n_u = 0; take(n_u); ++n_u) {
        const Job& u = s_job[n_u % kJobs];
        const int nb = u.blk1 - u.blk0;
        wait_all(&q_full[n_u % kJobs], n_u / kJobs, s_stop);
        if constexpr (NT == 1) {
          for (int i = 0; i <= nb && !stopped(); ++i) {
            if (i < nb) scores(T0{}, 0, true, true, i + 1 == nb);
            if (i > 0) product(T0{}, true, true, i > 1);
          }
        } else {
          // the tiles in turn, each its scores two steps ahead of the other's product
          const int steps = Split ? nb : 2 * nb;
          scores(T0{}, 0, true, Split, steps == 1);
          if (steps > 1) scores(T1{}, Split ? 0 : 1, Split, true, steps == 2);
          for (int i = 0; i < steps && !stopped(); i += 2) {
            product(T0{}, true, Split, i > 0);
            if (i + 2 < steps) scores(T0{}, 0, true, Split, i + 3 == steps);
            if (i + 1 < steps) product(T1{}, Split, true, i > 0);
            if (i + 3 < steps) scores(T1{}, Split ? 0 : 1, Split, true, i + 4 == steps);
          }
        }
        give(n_u);
      }
      if (leader) commit(su32(&drained));  // nothing is under way when TMEM goes back
      __syncwarp();
      if (!__all_sync(~0u, bar_wait(su32(&drained), 0))) s_stop = 1;
    } else if (wid == kMmaWarp + 1) {
      // ----------------------------------------------------- the walk, a job ahead of the others
      Walk w;
      w.left = 0;
      long long x = 0, per_head = 0;  // where the share begins, as a cost within its row; one head's cost
      w.b = -1;
      if (mode == kAllDecode) {  // nothing to do
      } else if (a.rows <= 32) {  // a lane per row
        RowBounds bounds = {};
        if (lane < a.rows) bounds = row_bounds(a, lane);
        const Row i = row_info<View>(a, bounds, r, tok, mode);
        const Costs costs = costs_of<View>(a, i, tok);
        const long long head = i.tiles ? cost_before<D, View>(costs, i.tiles) : 0, cost = K * head;
        long long v = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(~0u, v, o);
          if (lane >= o) v += y;
        }
        total = __shfl_sync(~0u, v, 31);
        const long long x0 = blockIdx.x * share_of();
        const uint32_t here = __ballot_sync(~0u, x0 < v && x0 >= v - cost);
        if (here) {
          w.b = __ffs(here) - 1;
          x = __shfl_sync(~0u, x0 - (v - cost), w.b);
          w.row.start = __shfl_sync(~0u, i.start, w.b);
          w.row.n = __shfl_sync(~0u, i.n, w.b);
          w.row.len = __shfl_sync(~0u, i.len, w.b);
          w.row.tiles = __shfl_sync(~0u, i.tiles, w.b);
          per_head = __shfl_sync(~0u, head, w.b);
          w.costs = {w.row.len - w.row.n, __shfl_sync(~0u, costs.most, w.b), tok,
                     __shfl_sync(~0u, costs.full, w.b)};
        }
      } else if (s_row >= 0) {
        w.b = s_row;
        x = s_at;
        w.row = row_info<View>(a, row_bounds(a, w.b), r, tok, mode);
        w.costs = costs_of<View>(a, w.row, tok);
        per_head = cost_before<D, View>(w.costs, w.row.tiles);
      }
      w.mode = mode;
      if (w.b >= 0) {
        w.share = share_of();
        w.left = min(w.share, total - blockIdx.x * w.share);
        // the kv head and the unit that hold it, a lane per candidate
        w.kvh = 0;
        for (int h = 1; h < K; h += 32) w.kvh += __popc(__ballot_sync(~0u, h + lane < K && (h + lane) * per_head <= x));
        x -= w.kvh * per_head;
        long long before = 0;
        int lo = 0, count = w.row.tiles;
        while (count > 1) {
          const int step = (count + 31) / 32, j = lo + lane * step;
          const long long c = cost_before<D, View>(w.costs, j);
          const int k = 31 - __clz(__ballot_sync(~0u, lane * step < count && c <= x));
          before = __shfl_sync(~0u, c, k);
          lo += k * step;
          count = min(step, count - k * step);
        }
        w.j = lo;
        w.at = x - before;
      }
      const int lines = r * D / 64;  // 128 bytes each, of a token's queries
      for (uint32_t k = 0;; ++k) {
        Job u = {};
        u.more = next_unit<D, View>(w, a, r, tok, u) ? 1 : 0;
        if (k >= kJobs) wait_all(&job_free[k % kJobs], k / kJobs - 1, s_stop);
        if (lane == 0) {
          s_job[k % kJobs] = u;
          sc::bar_arrive(su32(&job_full[k % kJobs]));
        }
        __syncwarp();
        if (!u.more || stopped()) break;
        if (k == 0) continue;  // (the first one's are on their way)
        // its queries come to L2
        const int tokens = min(tok, u.n - u.tok0);
        int t = lane / lines, c = lane - t * lines;
        const int dt = 32 / lines, dc = 32 - dt * lines;
        const uint16_t* src = a.q + ((int64_t)(u.start + u.tok0) * a.heads + u.kvh * r) * D;
        while (t < tokens) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src + (int64_t)t * a.heads * D + c * 64));
          t += dt;
          c += dc;
          if (c >= lines) {
            c -= lines;
            ++t;
          }
        }
      }
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
// thread per query row and 16 columns (four at a time, a quarter of the head apart), its parts in
// order.
template <int D>
__global__ void __launch_bounds__(512) combine_kernel(AttnArgs a) {
  using C = Cfg<D>;
  griddep_wait();
  const int first = blockIdx.x, at = blockIdx.y * 512 + threadIdx.x;
  const int row = at / (D / 16), c = at % (D / 16) * 4;
  const Cut cut = static_cast<const Cut*>(a.ws)[first];
  if (cut.last <= first) return;
  const int r = a.heads / a.kv.kv_heads, per_tile = 128 / r, in = row & 127;
  const int t = cut.tok0 + (row >> 7) * per_tile + in / r;
  if (in >= per_tile * r || t >= cut.end) return;
  const float* parts = reinterpret_cast<const float*>(static_cast<const char*>(a.ws) + kCutBytes);
  float m = kNone, l = 0.0f;  // (raw scores, as the parts have them)
  const float fac = parts[((size_t)first * 2 + 1) * C::kPartial + (size_t)C::kRows * (D + 2) + row];
  float4 y[4] = {};
#pragma unroll 2
  for (int k = first; k <= cut.last; ++k) {
    const float* src = parts + ((size_t)k * 2 + (k == first)) * C::kPartial;
    const float mk = src[(size_t)C::kRows * D + row], lk = src[(size_t)C::kRows * (D + 1) + row];
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const float4*>(src + (size_t)row * D + c + i * (D / 4));
    const float mm = fmaxf(m, mk), f = ex2((m - mm) * fac), h = ex2((mk - mm) * fac);
    m = mm;
    l = l * f + lk * h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i].x = y[i].x * f + v[i].x * h;
      y[i].y = y[i].y * f + v[i].y * h;
      y[i].z = y[i].z * f + v[i].z * h;
      y[i].w = y[i].w * f + v[i].w * h;
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : l;
  uint16_t* dst = a.out + ((int64_t)(cut.start + t) * a.heads + cut.kvh * r + in % r) * D + c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y[i].x * inv, y[i].y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(y[i].z * inv, y[i].w * inv);
    *reinterpret_cast<uint2*>(dst + i * (D / 4)) = make_uint2(
        *reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

template <int D, bool View, bool Split>
cudaError_t launch_kernel(const AttnArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D, View, Split>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e == cudaSuccess)
    e = launch_pdl(prompt_kernel<D, View, Split>, dim3(kGrid), dim3(kThreads), C::kSmem, st, a);
  return e;
}

template <int D>
cudaError_t launch_join(const AttnArgs& a, cudaStream_t st) {
  return launch_pdl(combine_kernel<D>, dim3(kGrid, Cfg<D>::kRows * D / (16 * 512)), dim3(512), 0, st, a);
}

template <int D, bool View>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  if constexpr (View && Cfg<D>::kTiles == 2)
    if ((int64_t)a.max_new * (a.heads / a.kv.kv_heads) <= 128) return launch_kernel<D, View, true>(a, st);
  return launch_kernel<D, View, false>(a, st);
}

template <int D>
size_t bytes_for() {
  return kCutBytes + (size_t)kGrid * 2 * Cfg<D>::kPartial * 4;
}

}  // namespace
}  // namespace kv
}  // namespace moe
