// Device code of the prologue over the 4-bit cache (int4.cuh): RoPE -> per-head
// RMSNorm -> bf16 q, and K and V quantised into their record.
//
// One block of 8 warps per token; warp w takes query heads 8w .. 8w+7 and KV
// head w.  Half a warp holds a row: lane l of 16 has elements 4l .. 4l+3 and
// 64 + 4l .. +3, so RoPE pairs (i, i + 64) live in one lane, every load and
// store is 8 bytes a lane, a row's sum takes four shuffles for two rows at
// once, and the table's sines and cosines are read once for a token's nine
// rows of a warp.  K and V of the KV head are the two halves of one pass.
// Memory (38.5 KB a token, 16 of q in and 16 out) and issue slots (750 instructions
// a warp) come close to each other: 8191 tokens take 64 us, 5.0 TB/s, 0.74 of a
// copy's rate, at six blocks an SM (40 registers; five blocks took 3 % more, four
// 12 %); the other caches' prologue, a warp per row with a quarter of the bytes in
// flight, 98 us.
//
// The codes are those of the exact k'.  In fp32 a value is known to
// kI4RelErr: where scale or code could come out otherwise within that, about
// one row in 300, the row is done again in pairs of floats (48 bits; that a
// code still comes out wrong has odds of one in 10^10 a row), which takes a
// fifth of the time of this part's 64-bit arithmetic.  So are groups with a scale
// below 2^-100, times a power of two.
#pragma once

#include "int4.cuh"

namespace hpc {
namespace {

// Relative error of k' in fp32, in the order below: each rotated element
// 3 u (u = 2^-24; the difference of products with its error added back), the
// sum of squares 2 * 3 + 1 + 8 u (seven additions and the first rounding), its
// root half of that, + 1 (eps) + 4 (rsqrtf, two ulps), the products 2 u:
// 3 + 7.5 + 5 + 2 = 17.5 u.
constexpr float kI4RelErr = 0x1.2p-20f;   // 18 u

// a * c - b * s with an error of at most 3 u of the result: the second
// product's rounding error is added back.
__device__ __forceinline__ float i4_diff_of_products(float a, float c, float b, float s) {
  const float w = b * s;
  const float e = fmaf(-b, s, w);
  return fmaf(a, c, -w) + e;
}

// ---- pairs of floats (value = h + l, |l| at most half an ulp of h)
struct F2 {
  float h, l;
};
__device__ __forceinline__ F2 f2_sum(float a, float b) {   // exact
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ F2 f2_norm(float h, float l) {   // |l| < |h|
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  const F2 s = f2_sum(a.h, b.h);
  return f2_norm(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  const float p = __fmul_rn(a.h, b.h);
  const float e = fmaf(a.h, b.h, -p);
  return f2_norm(p, fmaf(a.h, b.l, fmaf(a.l, b.h, e)));
}
// 1 / sqrt(x), one step from the fp32 value: x0 + x0 / 2 * (1 - x x0^2)
__device__ __forceinline__ F2 f2_rsqrt(F2 x) {
  const float x0 = 1.0f / sqrtf(x.h);
  const float q = __fmul_rn(x0, x0);
  const F2 q2 = {q, fmaf(x0, x0, -q)};
  const F2 t = f2_mul(x, q2);
  const float r = __fsub_rn(__fsub_rn(1.0f, t.h), t.l);
  return f2_norm(x0, __fmul_rn(0.5f * x0, r));
}

// The largest of the 8 lanes that hold a group (bits of magnitudes, so that a
// NaN is the largest).
__device__ __forceinline__ uint32_t i4_max8(uint32_t x) {
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ float i4_round_bf16(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// Groups of scales below kI4Tiny are worked on times kI4Up, a power of two, so
// that no reciprocal overflows and no product or rounding error underflows
// (scales go down to bf16's smallest value, 2^-133).
constexpr float kI4Tiny = 0x1p-100f, kI4Up = 0x1p100f;
constexpr uint32_t kI4TinyBits = (127 - 97) << 23;   // of 8 kI4Tiny: no larger group has such a scale

// Code + 8 of x (+ l), x = h (+ l), for a group of scale s > 0: the half-way
// point below or above the approximate quotient decides by the sign of an
// exactly rounded difference, ties to the even code.
__device__ __forceinline__ uint32_t i4_code_of(float h, float l, float s) {
  const float k = fminf(fmaxf(floorf(h * (1.0f / s)), -7.f), 6.f);
  const float d = fmaf(-(k + 0.5f), s, h) + l;
  const int ki = static_cast<int>(k);
  const int up = d > 0.f || (d == 0.f && (ki & 1)) ? 1 : 0;
  return static_cast<uint32_t>(ki + up + 8);
}

// Query heads it, it + its, .. of the warp's four pairs, and (kv) its KV head.
// One block of 256 threads.
__device__ __forceinline__ void prologue_i4(
    int b, int it0, int its, bool kv, const uint16_t* q, const uint16_t* __restrict__ k,
    const uint16_t* __restrict__ v, const int32_t* __restrict__ positions,
    const float* __restrict__ cos_sin, int32_t max_pos, const uint16_t* __restrict__ q_w,
    const uint16_t* __restrict__ k_w, float eps, uint8_t* __restrict__ kv_cache, int32_t num_blocks,
    const int64_t* __restrict__ slot_mapping, uint16_t* q_out, int32_t* __restrict__ status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 15, row = lane >> 4;   // lane of the row, row of the pair
  const int d0 = 4 * l;
  const int32_t pos = positions[b];
  // the rows' loads go out before the position is known to be good
  uint2 xa[4], xb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i % its != it0) continue;
    const uint16_t* src = q + (static_cast<int64_t>(b) * kHq + 8 * warp + 2 * i + row) * kD;
    xa[i] = *reinterpret_cast<const uint2*>(src + d0);
    xb[i] = *reinterpret_cast<const uint2*>(src + kD / 2 + d0);
  }
  uint2 ka = make_uint2(0u, 0u), kb = ka;
  int64_t slot = -1;
  if (kv) {
    const uint16_t* src = (row == 0 ? k : v) + (static_cast<int64_t>(b) * kHkv + warp) * kD;
    ka = *reinterpret_cast<const uint2*>(src + d0);
    kb = *reinterpret_cast<const uint2*>(src + kD / 2 + d0);
    slot = slot_mapping[b];
  }
  if (pos < 0 || pos >= max_pos) {
    if (threadIdx.x == 0 && kv) atomicOr(status, HPC_STATUS_BAD_POSITION);
    return;
  }
  const float4 c4 = *reinterpret_cast<const float4*>(cos_sin + static_cast<int64_t>(pos) * kD + d0);
  const float4 s4 = *reinterpret_cast<const float4*>(cos_sin + static_cast<int64_t>(pos) * kD + kD / 2 + d0);
  const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
  auto unpack = [](uint2 x, float (&f)[4]) {
    f[0] = bf16_lo(x.x), f[1] = bf16_hi(x.x), f[2] = bf16_lo(x.y), f[3] = bf16_hi(x.y);
  };
  {
    // two elements at a time
    auto pair = [](uint32_t x) { return f32x2(bf16_lo(x), bf16_hi(x)); };
    const uint2 wa = *reinterpret_cast<const uint2*>(q_w + d0), wb = *reinterpret_cast<const uint2*>(q_w + kD / 2 + d0);
    const uint64_t w2[4] = {pair(wa.x), pair(wa.y), pair(wb.x), pair(wb.y)};
    const uint64_t cs2[2] = {f32x2(cs[0], cs[1]), f32x2(cs[2], cs[3])};
    const uint64_t sn2[2] = {f32x2(sn[0], sn[1]), f32x2(sn[2], sn[3])};
    const uint64_t ng2[2] = {f32x2(-sn[0], -sn[1]), f32x2(-sn[2], -sn[3])};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i % its != it0) continue;
      const uint64_t a[2] = {pair(xa[i].x), pair(xa[i].y)}, c[2] = {pair(xb[i].x), pair(xb[i].y)};
      uint64_t y[4];   // d0 .. d0 + 3, then 64 on
      uint64_t ss2 = 0ull;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        y[e] = fma_f32x2(a[e], cs2[e], mul_f32x2(c[e], ng2[e]));
        y[2 + e] = fma_f32x2(c[e], cs2[e], mul_f32x2(a[e], sn2[e]));
        ss2 = fma_f32x2(y[e], y[e], ss2);
        ss2 = fma_f32x2(y[2 + e], y[2 + e], ss2);
      }
      float ss, ss_hi;
      f32x2_split(ss2, ss, ss_hi);
      ss += ss_hi;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float inv = rsqrtf(ss * (1.0f / kD) + eps);
      const uint64_t inv2 = f32x2(inv, inv);
      uint32_t out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo, hi;
        f32x2_split(mul_f32x2(mul_f32x2(y[e], inv2), w2[e]), lo, hi);
        out[e] = pack_bf16(lo, hi);
      }
      uint16_t* dst = q_out + (static_cast<int64_t>(b) * kHq + 8 * warp + 2 * i + row) * kD;
      *reinterpret_cast<uint2*>(dst + d0) = make_uint2(out[0], out[1]);
      *reinterpret_cast<uint2*>(dst + kD / 2 + d0) = make_uint2(out[2], out[3]);
    }
  }
  if (!kv || slot < 0) return;                            // (negative: padding entry)
  if (slot >= static_cast<int64_t>(num_blocks) * kPage) {
    if (lane == 0) atomicOr(status, HPC_STATUS_BAD_SLOT);
    return;
  }
  // K in the first half of the warp, V in the second, which only skips the
  // rotation and the norm
  float x[8], y[8], w[8];
  {
    float t[4];
    unpack(ka, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = t[e];
    unpack(kb, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 + e] = t[e];
    unpack(*reinterpret_cast<const uint2*>(k_w + d0), t);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = t[e];
    unpack(*reinterpret_cast<const uint2*>(k_w + kD / 2 + d0), t);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[4 + e] = t[e];
  }
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = i4_diff_of_products(x[e], cs[e], x[4 + e], sn[e]);
    y[4 + e] = i4_diff_of_products(x[4 + e], cs[e], -x[e], sn[e]);
    ss += y[e] * y[e] + y[4 + e] * y[4 + e];
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float inv = rsqrtf(ss * (1.0f / kD) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = row == 0 ? y[e] * inv * w[e] : x[e];
  float s[2];
  uint32_t u[2] = {0x8888u, 0x8888u};   // four stored codes of each half (zeros)
  bool near = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t am = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) am = max(am, abs_bits(y[4 * h + e]));
    am = i4_max8(am);
    const float a7 = __uint_as_float(am) * (1.0f / kI4Levels);
    s[h] = am >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : i4_round_bf16(a7);
    // V: a seventh of an 8-bit value is never this near to a tie
    near = near || (row == 0 && am < 0x7f800000u &&
                    i4_round_bf16(a7 * (1.f + 1.25f * kI4RelErr)) != i4_round_bf16(a7 * (1.f - 1.25f * kI4RelErr)));
    near = near || am - 1u < kI4TinyBits;   // (tiny groups, K's and V's)
    if (s[h] > 0.f) {
      // the code nearest to x / s, and how far x is from it: near a tie (for K
      // within 7 s of the error of a value) it is looked at again below.
      // Elsewhere |x / s| < 7.1.
      const float si = rcp_approx(s[h]), lim = s[h] * (0.5f - 8.f * 1.25f * kI4RelErr);
      u[h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = fmaf(y[4 * h + e], si, 0x1.8p23f + 8.f);   // the code + 8 in its low bits
        u[h] |= (__float_as_uint(m) & 15u) << (4 * e);
        near = near || fabsf(fmaf(m - (0x1.8p23f + 8.f), -s[h], y[4 * h + e])) > lim;
      }
    }
  }
  const unsigned again = __ballot_sync(0xffffffffu, near);
  if ((again >> 16) != 0u && row == 1) {
    // V (its scales are sure): ties and all by exact differences
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!(s[h] > 0.f)) continue;
      const float t = s[h] < kI4Tiny ? kI4Up : 1.f;
      u[h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[h] |= i4_code_of(y[4 * h + e] * t, 0.f, s[h] * t) << (4 * e);
    }
  }
  if ((again & 0xffffu) != 0u) {
    // K again in pairs of floats (both halves of the warp go along; V's keeps
    // what it has), pairs of tiny elements rotated times kI4Up
    F2 z[8];
    unsigned raised = 0;   // bit e: elements e and 4 + e
    F2 sum = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool tiny = fmaxf(fabsf(x[e]), fabsf(x[4 + e])) < 0x1p-60f;
      raised |= tiny ? 1u << e : 0u;
      const float f = tiny ? kI4Up : 1.f;
      const F2 c = {cs[e], 0.f}, t = {sn[e], 0.f}, a = {x[e] * f, 0.f}, bb = {x[4 + e] * f, 0.f};
      const F2 at = f2_mul(a, t), bt = f2_mul(bb, t);
      z[e] = f2_add(f2_mul(a, c), F2{-bt.h, -bt.l});
      z[4 + e] = f2_add(f2_mul(bb, c), at);
      F2 sq = f2_add(f2_mul(z[e], z[e]), f2_mul(z[4 + e], z[4 + e]));
      if (tiny) sq = {sq.h / kI4Up / kI4Up, sq.l / kI4Up / kI4Up};
      sum = f2_add(sum, sq);
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
      sum = f2_add(sum, F2{__shfl_xor_sync(0xffffffffu, sum.h, off), __shfl_xor_sync(0xffffffffu, sum.l, off)});
    const F2 r = f2_rsqrt(f2_add(F2{sum.h * (1.0f / kD), sum.l * (1.0f / kD)}, F2{eps, 0.f}));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // k', of a tiny group times kI4Up, half of it in each factor (so neither
      // overflows), less what its rotation was raised by
      const bool lift = s[h] < kI4Tiny;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool was = raised >> e & 1u;
        const float f = lift == was ? 1.f : lift ? 0x1p50f : 0x1p-50f;
        const F2 zr = f2_mul(z[4 * h + e], r);
        z[4 * h + e] = f2_mul(F2{zr.h * f, zr.l * f}, F2{w[4 * h + e] * f, 0.f});
      }
      // the largest magnitude of the group as a pair: sign of h on both parts
      F2 m = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        F2 v = z[4 * h + e];
        if (v.h < 0.f) v = {-v.h, -v.l};
        if (v.h > m.h || (v.h == m.h && v.l > m.l)) m = v;
      }
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) {
        const F2 v = {__shfl_xor_sync(0xffffffffu, m.h, off), __shfl_xor_sync(0xffffffffu, m.l, off)};
        if (v.h > m.h || (v.h == m.h && v.l > m.l)) m = v;
      }
      // (a row with infinities or NaN never gets here for its own sake: its
      // half of the group keeps the NaN scale)
      if (row != 0 || !(s[h] >= 0.f)) continue;
      // a seventh rounded to bf16: the candidate below, and the half-way point
      // above it against the pair (7 times it is exact in fp32).  Steps below
      // 2^-126 are 2^-133.
      const float m7 = m.h * (1.0f / kI4Levels) * (1.f - 0x1p-20f);
      const bool coarse = lift && m7 < 0x1p-126f * kI4Up;
      const float unit = 0x1p-133f * kI4Up;
      const float c0 = coarse ? floorf(m7 * (1.f / unit)) * unit : __uint_as_float(__float_as_uint(m7) & 0xffff0000u);
      const float step = coarse ? unit : __uint_as_float(__float_as_uint(c0) & 0x7f800000u) * 0x1p-7f;
      const bool odd = coarse ? static_cast<int>(c0 * (1.f / unit)) & 1 : __float_as_uint(c0) >> 16 & 1u;
      const float d = __fadd_rn(__fsub_rn(m.h, 7.f * (c0 + 0.5f * step)), m.l);
      const float sc = d > 0.f || (d == 0.f && odd) ? c0 + step : c0;
      s[h] = lift ? sc * (1.f / kI4Up) : sc;
      u[h] = 0x8888u;
      if (sc > 0.f) {
        u[h] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[h] |= i4_code_of(z[4 * h + e].h, z[4 * h + e].l, sc) << (4 * e);
      }
    }
  }
  const int off = static_cast<int>(slot % kPage);
  uint8_t* rec = kv_cache + (slot / kPage * kHkv + warp) * kI4Record;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = d0 + 64 * h, g = d / kI4Group;
    *reinterpret_cast<uint16_t*>(rec + (row == 0 ? i4_k_byte(off, d) : i4_v_byte(off, d))) = static_cast<uint16_t>(u[h]);
    // (bf16 values already; the NaN is 0x7fc0)
    if ((l & 7) == 0)
      *reinterpret_cast<uint16_t*>(rec + (row == 0 ? i4_ks_byte(off, g) : i4_vs_byte(off, g))) =
          static_cast<uint16_t>(__float_as_uint(s[h]) >> 16);
  }
}

// Blocks per token: one once they fill the part (8 warps with all their rows'
// loads in flight); few tokens are spread wider, a quarter of the rows each
// (32 tokens: 4 us against 6 us).
inline int i4_prologue_rows(int32_t tokens) { return tokens <= 512 ? 4 : 1; }

// The buffers' alignment: rows are read and written 8 bytes a lane, the table 16.
inline bool i4_prologue_aligned(const void* q, const void* k, const void* v, const void* cos_sin,
                                const void* q_w, const void* k_w, const void* kv_cache, const void* q_out) {
  auto a = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  return ((a(q) | a(k) | a(v) | a(q_w) | a(k_w) | a(q_out)) & 7) == 0 && ((a(cos_sin) | a(kv_cache)) & 15) == 0;
}

}  // namespace
}  // namespace hpc
