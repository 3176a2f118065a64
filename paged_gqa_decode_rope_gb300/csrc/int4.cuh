// The 4-bit cache: number format and record layout, shared by the prologue
// that writes it and the kernels that read it.
//
// A group of 32 consecutive elements x of a head's K or V row is held as one
// bf16 scale s and 32 codes c in -7 .. 7, an element being c * s:
//   s = bf16(max|x| / 7),   c = clamp(round(x / s), -7, 7),   ties to even.
// A group of zeros, or one whose scale underflows to zero, has c = 0; a group
// with an infinity or a NaN has s = NaN, so it reads as NaN like a bf16 cache
// would.  Codes are stored as u = c + 8.  The group of 32 and the bf16 scale
// (4.5 bits an element with it) need no calibration and no per-tensor scale:
// bf16 has fp32's range.
//
// One record of kI4Record bytes per (block, KV head) holds the 64 tokens of
// the block, so a tile is one contiguous copy:
//   K codes   [64 tokens][4 quads c][4 groups g][8 nibbles]: d = 32g + 8c + i
//   V codes   [8 octets of tokens][8 rows r][4 pairs c][4 groups g][2 tokens]
//             [4 nibbles j]: token 8*octet + 2c + half, d = 32g + 4r + j
//   K scales  bf16 [64 tokens][4 groups]
//   V scales  bf16 [32 token pairs][4 groups][2 tokens]
// Both code orders are those in which a lane (r = lane / 4, c = lane % 4) of
// the m16n8 products holds its A fragments, 16 bytes at a time: K's with
// tokens on the rows, V's (transposed) with d on the rows and a token pair in
// the halves of each word.  So neither needs ldmatrix, a swizzle or a byte
// shuffle: a masked word is two F16 values, and a 16-bit half's nibble becomes
// a bf16 by a mask and one operation.
#pragma once

#include "common.cuh"

namespace hpc {

constexpr int kI4Group = HPC_INT4_GROUP;        // elements per scale
constexpr int kI4Groups = kD / kI4Group;        // 4 scales per row
constexpr int kI4Levels = 7;                    // codes -7 .. 7
constexpr int kI4Codes = kPage * kD / 2;        // 4096 bytes of codes of 64 rows
constexpr int kI4OffV = kI4Codes;
constexpr int kI4OffKs = 2 * kI4Codes;
constexpr int kI4OffVs = kI4OffKs + kPage * kI4Groups * 2;
constexpr int kI4Record = HPC_INT4_RECORD_BYTES;
static_assert(kI4OffVs + kPage * kI4Groups * 2 == kI4Record, "record size");
static_assert(kI4Record % 16 == 0, "records are copied 16 bytes at a time");

// Byte of the record that holds codes d, d + 1 (d even; the low nibble is d).
__host__ __device__ constexpr int i4_k_byte(int t, int d) {
  return t * 64 + ((d & 31) >> 3) * 16 + (d >> 5) * 4 + ((d & 7) >> 1);
}
__host__ __device__ constexpr int i4_v_byte(int t, int d) {
  return kI4OffV + ((t >> 3) * 32 + ((d & 31) >> 2) * 4 + ((t & 7) >> 1)) * 16 + (d >> 5) * 4 +
         (t & 1) * 2 + ((d & 3) >> 1);
}
// Byte of the scale of group g of token t.
__host__ __device__ constexpr int i4_ks_byte(int t, int g) { return kI4OffKs + (t * kI4Groups + g) * 2; }
__host__ __device__ constexpr int i4_vs_byte(int t, int g) {
  return kI4OffVs + ((t >> 1) * kI4Groups + g) * 4 + (t & 1) * 2;
}

// The low nibble of each half of w as a bf16 code: u in the low bits of the
// mantissa of 128, less 136.  Exact.
__device__ __forceinline__ uint32_t i4_code_lo(uint32_t w) {
  uint32_t y;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(y) : "r"(w));   // (w & mask) | 128.0
  asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0xc308c308u));
  return y;
}
// The second nibble of each half as a quarter of its code, without a shift:
// in place its four bits are the bf16 value 16 u 2^-133 (the subnormal steps
// go on through the first binade), times 2^127 less 2.  Exact.
__device__ __forceinline__ uint32_t i4_code_hi4(uint32_t w) {
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(w & 0x00f000f0u), "r"(0x7f007f00u), "r"(0xc000c000u));
  return y;
}
// Element i of 8 codes times their scale.
__device__ __forceinline__ float i4_value(uint32_t w, int i, float s) {
  return static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - 8) * s;
}
// Powers of two that a tile's K or V is staged by as F16 (prefill): bins of 16,
// 2^(9 - 16 k) for largest scales 2^(16 k - 12) up to 2^(16 k + 4), of the first
// `keep` tokens.  Code times scale is then below 57344, and an F16 value exactly
// for scales down to 2^-13 of the largest at least, 2^-29 at most.  k is 0 for
// scales of 2^-12 .. 2^4; not below kI4LowBin, where scales under 2^-106 are held
// less exactly.  x: the words of the lane's tokens 2 lane and 2 lane + 1.  *nan: of
// the first `keep` tokens, one has an infinity or a NaN.
constexpr int kI4LowBin = -5;
__device__ __forceinline__ int i4_bin_power(int bin) { return 9 - 16 * bin; }
template <bool kV>
__device__ __forceinline__ int i4_tile_bin(uint4 x, int lane, int keep, bool* nan) {
  const uint32_t w[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
  uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  *nan = false;
  if (keep < kPage || m >= 0x7f80u) {
    // without the tokens past the end, and without infinities and NaN (K's second
    // token has words 2 and 3, V's the high halves)
    m = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t half = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu;
      const bool live = 2 * lane + (kV ? i & 1 : i >> 2) < keep;
      if (live && half < 0x7f80u) m = max(m, half);
      bad = bad || (live && half >= 0x7f80u);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    *nan = __any_sync(0xffffffffu, bad);
  }
  return max((static_cast<int>(m >> 7) - 127 + 12) >> 4, kI4LowBin);
}
// 2^e, e in -126 .. 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}

}  // namespace hpc
