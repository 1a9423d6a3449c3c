// Query/key norms, rotation and the 4-bit store in one pass over the
// projections' output; and its reverse, reading slots back as bf16.
//
// Per token and head: y = x * rsqrt(mean(x^2) + eps) * w (q and k), then every
// rotated pair (a, b) -> (a cos - b sin, b cos + a sin) at the pair's own axis'
// position, all in fp32.  q goes out in bf16.  k and v are quantised straight
// from fp32, per 64 columns: scale = fp16((max - min) / 15), bias = fp16(min),
// code = round((y - bias) / scale) clamped to 0..15.
//
// A row of D columns is held by D / 8 lanes, 8 columns each (one 16-byte
// load); 8 lanes are one quantisation group, whose minimum and maximum take
// three shuffles, and a lane's eight codes are one 32-bit word.  One warp per
// token and part of its heads (few tokens: one part per row, so that a decode
// step's rows run side by side; many: one part, so that cosines, sines and norm
// weights are read once per token): it keeps four rows' loads under way.
// Measured with the read-back: 8192 tokens of 16 query and 2 + 2 key and value
// heads of 256, 47 us (179 MB: 3.8 TB/s); 1237 tokens of 32 and 8 + 8 heads of 128
// with three axes 16 us; 8 tokens 4.6 us.  Large calls are bound by instruction
// issue and latency together: 168 instructions a row at 55% of the issue slots,
// 17 warps per SM (96 registers), waiting on loads and shuffles in equal parts;
// a persistent loop over tokens took 63 us.
#include <type_traits>

#include "kv_common.cuh"

namespace moe {
namespace kv {
namespace {

constexpr float kMaxValue = 32768.0f;  // what an fp16 scale and bias can hold with room to spare

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf2(x[0], x[1]), bf2(x[2], x[3]), bf2(x[4], x[5]), bf2(x[6], x[7]));
}

// {a, b} * {c, d} + s, two at a time
__device__ __forceinline__ float2 fma2(float a, float b, float c, float d, float2 s) {
  float2 r;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(c), "f"(d), "f"(s.x), "f"(s.y));
  return r;
}

// The tile of (block, head, token) and the token's row in it.
template <int D>
__device__ __forceinline__ uint8_t* tile_of(const moe_kv& kv, int slot, int head, int& key) {
  const int p_shift = 31 - __clz(kv.block_tokens), at = slot & (kv.block_tokens - 1);
  key = at % kTile;
  const int64_t tile =
      (((int64_t)(slot >> p_shift) * kv.kv_heads + head) << (p_shift - 4)) + at / kTile;
  return static_cast<uint8_t*>(kv.pool) + tile * tile_bytes(D);
}

// One row's 8 columns of this lane into the cache (which: 0 = K, 1 = V).  The
// whole warp calls it (shuffles); lanes with `store` unset write nothing.
template <int D>
__device__ __forceinline__ void quantise_store(const float (&x)[8], uint8_t* tile, int key,
                                               int which, int sub, bool store) {
  float lo = kMaxValue, hi = -kMaxValue, v[8];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    nan |= x[i] != x[i];
    v[i] = fminf(fmaxf(x[i], -kMaxValue), kMaxValue);
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
  }
  const unsigned nans = __ballot_sync(~0u, nan);
  if (!store) return;
  __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.0f)), bh = __float2half_rn(lo);
  const float s = __half2float(sh), b = __half2float(bh);
  // (y - bias) / scale by the reciprocal, 4e-6 off at most; where that comes near a border the
  // quotient itself decides, so that a code is always the definition's
  const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
  uint32_t word = 0;
  bool near = false;
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = (v[i] - b) * inv;
    c[i] = rintf(q);
    near |= fabsf(fabsf(q - c[i]) - 0.5f) < 1e-5f;
  }
  if (near && s > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = rintf(__fdiv_rn(v[i] - b, s));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)  // (the sum's low bits are the code)
    word |= (__float_as_uint(fminf(fmaxf(c[i], 0.0f), 15.0f) + 8388608.0f) & 15u) << (4 * i);
  // a NaN makes its whole group NaN
  if (nans & (0xFFu << (threadIdx.x & 24))) sh = bh = __ushort_as_half(0x7FFFu);
  const int chunk = (sub >> 2) ^ swizzle<D>(key);
  *reinterpret_cast<uint32_t*>(tile + which * 8 * D + key * (D / 2) + chunk * 16 + (sub & 3) * 4) =
      word;
  if ((sub & 7) == 0) {
    __half* meta = reinterpret_cast<__half*>(tile + 16 * D);
    const int g = sub >> 3;
    meta[which ? Meta<D>::v_scale(key, g) : Meta<D>::k_scale(key, g)] = sh;
    meta[which ? Meta<D>::v_bias(key, g) : Meta<D>::k_bias(key, g)] = bh;
  }
}

template <int D>
__global__ void __launch_bounds__(128) store_kernel(StoreArgs a, int parts) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAtOnce = 4;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, mine = lane / kLanes;
  const int64_t id = blockIdx.x * 4ll + (threadIdx.x >> 5);
  const int t = (int)(id / parts), part = (int)(id % parts);
  griddep_wait();
  if (t >= a.T) return;
  const int slot = a.slot[t];
  if (slot == -1) return;  // padding
  if ((unsigned)slot >= (unsigned)(a.kv.num_blocks * a.kv.block_tokens)) {
    if (lane == 0) atomicOr(a.err, MOE_DERR_KV_INDEX);
    return;
  }
  const int H = a.proj.q_heads, K = a.kv.kv_heads, rot = a.rope.rotary_dim, half = rot / 2;
  const int rq = (H + kRows - 1) / kRows, rk = (K + kRows - 1) / kRows, rounds = rq + 2 * rk;
  const int r0 = (int)((int64_t)rounds * part / parts), r1 = (int)((int64_t)rounds * (part + 1) / parts);
  // one region after the other: rounds of kRows query heads, of key heads, of value heads
  const int64_t lane_at = sub * 8;
  auto pointer = [&](int which) {
    const int64_t at = which == 0 ? t * a.proj.q_token_stride
                                  : which == 1 ? t * a.proj.k_token_stride : t * a.proj.v_token_stride;
    return static_cast<const uint16_t*>(which == 0 ? a.proj.q : which == 1 ? a.proj.k : a.proj.v) +
           at + lane_at;
  };
  const uint16_t* const base[3] = {pointer(0), pointer(1), pointer(2)};
  const int64_t stride[3] = {a.proj.q_head_stride, a.proj.k_head_stride, a.proj.v_head_stride};
  const int heads[3] = {H, K, K};
  const int begin[4] = {0, rq, rq + rk, rounds};
  auto load = [&](int which, int round) {
    const int h = (round - begin[which]) * kRows + mine;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (h < heads[which])
      u = __ldcs(reinterpret_cast<const uint4*>(base[which] + h * stride[which]));
    return u;
  };
  // this lane's cosines and (signed) sines; the partner of column c is c + half
  // (halves) or c ^ 1 (adjacent)
  float cs[8], sn[8];
  const bool turns = sub * 8 < rot;
  bool bad = false;
  if (turns) {
    const int first = a.rope.adjacent ? sub * 4 : sub * 8 < half ? sub * 8 : sub * 8 - half;
    if (a.rope.axes == 1) {
      // one position: the pairs lie side by side in the table
      const int p = a.positions[t];
      bad = p < 0 || p >= a.rope.max_pos;
      if (!bad) {
        const float* e = a.rope.table + (int64_t)p * rot + first;
        const float4 c0 = *reinterpret_cast<const float4*>(e);
        const float4 n0 = *reinterpret_cast<const float4*>(e + half);
        if (a.rope.adjacent) {
          const float c[4] = {c0.x, c0.y, c0.z, c0.w}, n[4] = {n0.x, n0.y, n0.z, n0.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            cs[i] = c[i / 2];
            sn[i] = i & 1 ? n[i / 2] : -n[i / 2];
          }
        } else {
          const float4 c1 = *reinterpret_cast<const float4*>(e + 4);
          const float4 n1 = *reinterpret_cast<const float4*>(e + half + 4);
          const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          const float n[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            cs[i] = c[i];
            sn[i] = sub * 8 >= half ? n[i] : -n[i];
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pair = a.rope.adjacent ? first + i / 2 : first + i;
        const int p = a.positions[(int64_t)a.rope.pair_axis[pair] * a.T + t];
        cs[i] = sn[i] = 0.0f;
        if (p < 0 || p >= a.rope.max_pos) {
          bad = true;
        } else {
          const float* e = a.rope.table + (int64_t)p * rot + pair;
          const bool second = a.rope.adjacent ? (i & 1) : sub * 8 >= half;
          cs[i] = e[0];
          sn[i] = second ? e[half] : -e[half];
        }
      }
    }
  }
  if (__any_sync(~0u, bad)) {  // a position outside the table: the token is skipped
    if (lane == 0) atomicOr(a.err, MOE_DERR_KV_INDEX);
    return;
  }
  const int partner = (lane - sub + (sub * 8 < half ? sub + half / 8 : sub - half / 8)) & 31;
  // norm weights of queries and keys
  float wq[8], wk[8];
  auto weights = [&](const float* w, float (&x)[8]) {
    if (w == nullptr) return;
    const float4 lo = *reinterpret_cast<const float4*>(w + sub * 8);
    const float4 hi = *reinterpret_cast<const float4*>(w + sub * 8 + 4);
    x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w;
    x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
  };
  weights(a.proj.q_norm, wq);
  weights(a.proj.k_norm, wk);
  auto region = [&](auto which_tag) {
    constexpr int kWhich = decltype(which_tag)::value;
    const int from = max(r0, begin[kWhich]), to = min(r1, begin[kWhich + 1]);
    const bool normed = kWhich == 0 ? a.proj.q_norm != nullptr
                                    : kWhich == 1 && a.proj.k_norm != nullptr;
    if (from >= to) return;
    uint4 raw[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      raw[i] = from + i < to ? load(kWhich, from + i) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int i0 = from; i0 < to; i0 += kAtOnce) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i0 + i >= to) break;
        const int h = (i0 + i - begin[kWhich]) * kRows + mine;
        float x[8];
        unpack8(raw[i], x);
        if (i0 + i + kAtOnce < to) raw[i] = load(kWhich, i0 + i + kAtOnce);
        if (normed) {
          float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int j = 0; j < 8; j += 2) ss = fma2(x[j], x[j + 1], x[j], x[j + 1], ss);
          float sum = ss.x + ss.y;
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
          const float r = rsqrtf(fmaf(sum, 1.0f / D, a.proj.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = x[j] * r * (kWhich == 0 ? wq[j] : wk[j]);
        }
        if (kWhich < 2 && rot) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float u = x[j + 1], v = x[j];
            if (!a.rope.adjacent) {
              u = __shfl_sync(~0u, x[j], partner);
              v = __shfl_sync(~0u, x[j + 1], partner);
            }
            if (turns) {
              x[j] = fmaf(u, sn[j], x[j] * cs[j]);
              x[j + 1] = fmaf(v, sn[j + 1], x[j + 1] * cs[j + 1]);
            }
          }
        }
        if constexpr (kWhich == 0) {
          if (h < H)
            __stcs(reinterpret_cast<uint4*>(a.q_out + ((int64_t)t * H + h) * D + lane_at), pack8(x));
        } else {
          int key;
          uint8_t* tile = tile_of<D>(a.kv, slot, h < K ? h : 0, key);
          quantise_store<D>(x, tile, key, kWhich == 2, sub, h < K);
        }
      }
    }
  };
  region(std::integral_constant<int, 0>{});
  region(std::integral_constant<int, 1>{});
  region(std::integral_constant<int, 2>{});
}

// Slots read back: scale * code + bias in fp32, rounded once to bf16.
template <int D>
__global__ void __launch_bounds__(256) load_kernel(LoadArgs a) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes;
  const int K = a.kv.kv_heads, sub = threadIdx.x % kLanes;
  griddep_wait();
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;  // [T][K]
  if (row >= (int64_t)a.T * K) return;
  const int t = (int)(row / K), h = (int)(row - (int64_t)t * K);
  const int slot = a.slot[t];
  if (slot == -1) return;
  if ((unsigned)slot >= (unsigned)(a.kv.num_blocks * a.kv.block_tokens)) {
    if (sub == 0 && a.err) atomicOr(a.err, MOE_DERR_KV_INDEX);
    return;
  }
  int key;
  const uint8_t* tile = tile_of<D>(a.kv, slot, h, key);
  const __half* meta = reinterpret_cast<const __half*>(tile + 16 * D);
  const int g = sub >> 3, chunk = (sub >> 2) ^ swizzle<D>(key);
  const uint8_t* codes = tile + key * (D / 2) + chunk * 16 + (sub & 3) * 4;
  const uint32_t wk = *reinterpret_cast<const uint32_t*>(codes);
  const uint32_t wv = *reinterpret_cast<const uint32_t*>(codes + 8 * D);
  const float ks = __half2float(meta[Meta<D>::k_scale(key, g)]);
  const float kb = __half2float(meta[Meta<D>::k_bias(key, g)]);
  const float vs = __half2float(meta[Meta<D>::v_scale(key, g)]);
  const float vb = __half2float(meta[Meta<D>::v_bias(key, g)]);
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = fmaf(ks, (float)((wk >> (4 * i)) & 15u), kb);
    y[i] = fmaf(vs, (float)((wv >> (4 * i)) & 15u), vb);
  }
  const int64_t at = row * D + sub * 8;
  *reinterpret_cast<uint4*>(a.k + at) = pack8(x);
  *reinterpret_cast<uint4*>(a.v + at) = pack8(y);
}

template <int D>
cudaError_t store_d(const StoreArgs& a, cudaStream_t st) {
  // As many parts as run at once: 20 warps per SM have registers (16-byte loads of
  // 16 query and 2 + 2 key and value heads of 256, read back, us: 8 tokens 10.8 in
  // one part and 4.5 in six; 1024 tokens 12.4 in one, 10.1 in two, 13.8 in three, whose
  // last warps come in a second wave)
  const int per = 32 / (D / 8);
  const int rounds = (a.proj.q_heads + per - 1) / per + 2 * ((a.kv.kv_heads + per - 1) / per);
  const int64_t want = (int64_t)kGrid * 20 / a.T;
  const int parts = (int)(want < 1 ? 1 : want < rounds ? want : rounds);
  const int64_t warps = (int64_t)a.T * parts;
  return launch_pdl(store_kernel<D>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, a, parts);
}

template <int D>
cudaError_t load_d(const LoadArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.T * a.kv.kv_heads, per = 256 / (D / 8);
  return launch_pdl(load_kernel<D>, dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_store(const StoreArgs& a, cudaStream_t st) {
  return a.kv.head_dim == 256 ? store_d<256>(a, st)
         : a.kv.head_dim == 128 ? store_d<128>(a, st) : store_d<64>(a, st);
}

cudaError_t launch_load(const LoadArgs& a, cudaStream_t st) {
  return a.kv.head_dim == 256 ? load_d<256>(a, st)
         : a.kv.head_dim == 128 ? load_d<128>(a, st) : load_d<64>(a, st);
}

}  // namespace kv
}  // namespace moe
