// Split-KV paged GQA decode attention over the 4-bit cache (int4.cuh), sm_103a:
// 1 to 4 new tokens per sequence, the plans, partials and results of
// hpc_decode_attn and its forms.
//
// With s_t = sm_scale q . K_t over the keys a query sees, out = sum_t p_t V_t,
// p = softmax(s): an item's partial is that over its tiles, with the
// log-sum-exp of its scores.
//
// What bounds it: a token's K and V of one head are 144 bytes (9 KB a tile of
// 64 tokens), a quarter to a half of the other caches', for the same products;
// so at HBM's rate an SM has about 400 cycles per tile, and the instructions
// that widen 16384 codes, not the copies, decide.  Hence:
//  * K codes enter the products as they lie, V codes with one mask and one
//    half-precision operation per pair (below); products are m16n8k16 with
//    tokens (K) and d (V) on the rows and the 8 query heads of the group on
//    the columns, without padding.
//  * One warp takes whole tiles by itself: maxima, rescaling and waits are
//    paid once per tile and not once per quarter of it, and no tile needs a
//    barrier.  A CTA's range of the plan is cut into as many equal runs of
//    tiles as it has warps; a warp keeps its state over its run and hands over
//    one state per work item.  States of an item that several warps share are
//    merged in shared memory when the range is done, in tile order: one
//    meeting of the warps per range, not per item.  (Queues of four warps that
//    met at every item's end spent 3 microseconds there on each.)
//  * A producer warp feeds them: lane w streams the run of warp w into two
//    stages, a tile's record by one bulk copy; descriptors and block ids are
//    loaded a tile ahead.  (Half tiles in a ring of three, for 15 warps, cost
//    four copies a tile: one warp could not issue them fast enough.)
//  * With more than one new token a warp serves all of them, so that every
//    code is widened once.
// Measured (attention alone, of a copy's 6.7 TB/s): 32 sequences of 4096 tokens
// 37 us, 0.61 (the tiles themselves 22; the rest is the first copies, the two
// merges and the launch); one of 131072 and 31 of 4096 59 us, 0.75; the heavy
// tail's 2.1 million tokens 420 us, 0.86; 1100 instructions a tile.  Two
// new tokens on 40 ragged sequences 106 us, 0.47; four on the long mix 175 us,
// 0.26: 1450 and 2400 instructions a tile, and with eight warps of that many
// registers two a scheduler, which hide little of the products' latency (1.5 of
// 4 issue slots, a third of the legacy tensor rate).  The same mix with four new
// tokens on the 5th-generation tensor cores took 164 us with the query rows on
// M = 128 (the 32 rows' padding; 106 without the widening), and 190 with 128
// tokens on M, codes widened straight into tensor memory (a dozen handshakes a
// step).  Issuing the copies from the consumer warps cost 10 to 20 %.
// Waits are bounded as in the other attention kernels (kWaitLimitNs).
#include "attn_kernel.cuh"
#include "int4.cuh"

namespace hpc {
namespace {

// kNq: queries a warp serves: 1, 2, or 4 (three and four new tokens).  A warp
// of one query makes do with 168 registers, which 12 warps leave; more queries
// want the 255 that 8 leave (10 warps of 168 took 7 us more on 40 sequences of
// 777 .. 30011 tokens with 2 queries; 4 queries as two pairs on 10 warps, each
// widening the codes, 11 us more on one of 131072 and 31 of 4096).
template <int kNq>
struct I4Cfg {
  static constexpr int kWarps = kNq == 1 ? 11 : 7;           // consumer warps
  static constexpr int kStages = kNq == 2 ? 3 : 2;          // tiles of a warp's ring
  static constexpr int kSlots = 4;                           // descriptions: tiles, piece openings, stop
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRing = kStages * kI4Record;
  static constexpr int kOStride = kD + 4;
  // A split item's state waits in tensor memory, two per warp (32 columns per
  // query), its maxima and sums in shared memory; for the merge up to two
  // queries' O at a time, [8 heads][kOStride], go to the ring.
  static constexpr int kRoundNq = kNq == 4 ? 2 : kNq;
  static constexpr int kState = kGroup * kOStride * 4 * kRoundNq;
  static constexpr int kTmemCols = kNq == 1 ? 256 : 512;     // 64 per query and warp of a lane quarter, rounded up
  static constexpr int kOffMeta = kWarps * kRing;            // int4 [warps][slots][2]
  static constexpr int kOffPieces = kOffMeta + kWarps * kSlots * 32;   // int4 [warps][2]
  static constexpr int kOffStats = kOffPieces + kWarps * 2 * 16;       // float [warps][2][queries][m, l][8]
  static constexpr int kOffBar = kOffStats + kWarps * 2 * kNq * 64;
  static constexpr int kBars = 2 * kSlots + kStages;         // per warp: full, empty, stage free
  static constexpr int kList = 64;                           // segments noted for the merge
  static constexpr int kOffList = (kOffBar + kWarps * kBars * 8 + 15) / 16 * 16;   // int4 [kList]: segment, items
  static constexpr int kOffCtl = kOffList + kList * 16;    // abort, range begin, end, list length
  static constexpr int kOffTmem = kOffCtl + 16;              // tensor memory's address
  // several queries: their operands and biases, per warp
  static constexpr int kOffQ = (kOffTmem + 16 + 127) / 128 * 128;
  static constexpr int kQBytes = kNq == 1 ? 0 : kNq / 2 * (8 * 512 + 512);
  static constexpr int kSmemBytes = kOffQ + kWarps * kQBytes + 128;   // slack for 128-byte alignment
  static_assert((kWarps + 3) / 4 * 64 * kNq <= kTmemCols, "two parked states per warp");
  static_assert(2 * kState <= kRing, "the states must fit in the ring");
  static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-CTA shared memory");
  static_assert(kState % 16 == 0, "16-byte rows");
};

// Flags of a ring slot's description.
enum : int {
  kI4Head = 0xff,        // KV head
  kI4Stop = 1 << 8,      // the run is over
  kI4Open = 1 << 9,      // no data: a piece of an item begins
  kI4Last = 1 << 10,     // the piece's last tile
  kI4Start = 1 << 11,    // the piece begins with the item's first tile
  kI4End = 1 << 12,      // the piece ends with the item's last tile
  kI4Ok = 1 << 13,       // the tile has data
  kI4Known = 1 << 14,    // sequence and head exist
};

// ---- What a warp keeps for its queries, and its work on a tile.
//
// A masked K word is two F16 values as it stands: u 2^-24 for the low nibble
// of each half, 16 u 2^-24 for the second (subnormal steps, which go on
// through the first binade), so K codes enter the products without a
// conversion: five integer operations for eight of them.  q is scaled per row
// by a power of two that puts its largest element in [16, 32) (divided by 16
// again where it meets second nibbles), exact for elements down to 2^-17 of
// the largest.  The codes' bias of 8 is taken off by starting the
// accumulators at -8 2^-24 times q's sum over the group; a magic number in the
// codes' place would cost its size in precision.  (E4M3 products of the
// codes' bytes would need fewer operations still, but mma.sync converts their
// operands to F16 first, at a quarter of the rate.)
//
// The softmax takes maxima of scores before their scale, which is therefore
// not negative (the calls refuse it); a scale of zero makes q zero.

// Scale of a row of q whose largest magnitude has these bits, and what takes
// scores of codes back to log2 units (NaN for a q with an infinity or a NaN).
__device__ __forceinline__ void i4_row_scale(uint32_t am, float scale_log2, float& sc, float& back) {
  const int e2 = static_cast<int>(am >> 23) - 127;
  const int se = 4 - max(e2, -100);   // in [-124, 104]
  sc = scale_log2 > 0.f ? __uint_as_float(static_cast<uint32_t>(127 + se) << 23) : 0.f;
  back = scale_log2 > 0.f ? __uint_as_float(static_cast<uint32_t>(127 - se) << 23) * scale_log2 * 0x1p24f : 1.f;
  if (am >= 0x7f800000u) back = __uint_as_float(0x7fc00000u);
}

// The lane's 8 elements of every group of one row of q, elements 32g + 8c ..
// +7, as products' operands: b[g][h] = {(2h, 2h + 4), (2h + 1, 2h + 5) / 16}.
// Returns the row's largest magnitude's bits over the lane's elements.
struct I4Row {
  uint4 w[kI4Groups];
  __device__ __forceinline__ void load(const uint16_t* row) {
#pragma unroll
    for (int g = 0; g < kI4Groups; ++g) w[g] = *reinterpret_cast<const uint4*>(row + 32 * g);
  }
  __device__ __forceinline__ uint32_t largest() const {   // of the row: over its four lanes
    uint32_t lo = 0, hi = 0;   // (a NaN's bits are the largest)
#pragma unroll
    for (int g = 0; g < kI4Groups; ++g) {
      const uint32_t x[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo = max(lo, x[e] << 16 & 0x7fff0000u);
        hi = max(hi, x[e] & 0x7fff0000u);
      }
    }
    lo = max(lo, hi);
    lo = max(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    return max(lo, __shfl_xor_sync(0xffffffffu, lo, 2));
  }
  __device__ __forceinline__ void operand(int g, int h, float sc, uint32_t& b0, uint32_t& b1) const {
    const uint32_t x = h == 0 ? w[g].x : w[g].y, y = h == 0 ? w[g].z : w[g].w;   // (0,1) (4,5) | (2,3) (6,7)
    b0 = pack_f16(bf16_lo(x) * sc, bf16_lo(y) * sc);
    b1 = pack_f16(bf16_hi(x) * (sc * 0.0625f), bf16_hi(y) * (sc * 0.0625f));
  }
};

// The scales of V rows that not every query of the warp sees, made harmless in
// the warp's own copy of the tile: past the last visible token (`most`) the
// cache may hold anything, NaN included, and 0 * NaN is NaN, so they become
// zero; of tokens `least` .. `most` - 1 (seen by the later queries only) NaN
// ones do, and bit 4j + g of the result says that query j sees a NaN in group
// g.  A partial tile then takes the same products as a full one.
template <int kNq>
__device__ __forceinline__ unsigned i4_hide_tokens(uint32_t st, int least, int most, int lane,
                                                   const int (&nv)[kNq]) {
  unsigned nan = 0;
#pragma unroll 1
  for (int t = lane; t < kPage; t += 32) {
    if (t < least) continue;
#pragma unroll 1
    for (int g = 0; g < kI4Groups; ++g) {
      const uint32_t at = st + i4_vs_byte(t, g);
      uint16_t s;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s) : "r"(at) : "memory");
      const bool bad = (s & 0x7f80u) == 0x7f80u;
      if (t >= most || bad) asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(0)) : "memory");
      if (bad) {
#pragma unroll
        for (int j = 0; j < kNq; ++j)
          if (t < nv[j]) nan |= 1u << (4 * j + g);
      }
    }
  }
  fence_proxy_async_smem();   // (the next copy into this stage comes after these stores)
  __syncwarp();
  return __reduce_or_sync(0xffffffffu, nan);
}

// A row's reference maximum moves only when its scores pass it by more than
// 2^8 (weights are then at most 2^8): with short runs of tiles and 8 or 16 rows
// a warp, some row's true maximum moves in most tiles (two of three on the
// ragged batch of two queries), and every move rescales all of O.
constexpr float kI4Grow = 8.f;

template <int kNq>
struct I4Warp;

// One query: tokens (K) and d (V) on the products' 16 rows, the 8 heads of the
// group on the columns; lane (r, c) = (lane / 4, lane % 4) has heads 2c and
// 2c+1.
template <>
struct I4Warp<1> {
  uint32_t b[kI4Groups][2][2];
  float bias[kI4Groups][4];        // heads 2c, 2c+1, twice: a product's C as it stands
  float c0, c1;                    // from scores to log2 units
  float m0, m1, l0, l1, o[8][4];

  __device__ __forceinline__ void open(const I4Row (&q)[1], float scale_log2, int lane) {
    float sc, back;
    i4_row_scale(q[0].largest(), scale_log2, sc, back);
    c0 = __shfl_sync(0xffffffffu, back, 8 * (lane & 3));       // lane of head 2c
    c1 = __shfl_sync(0xffffffffu, back, 8 * (lane & 3) + 4);
#pragma unroll
    for (int g = 0; g < kI4Groups; ++g) {
#pragma unroll
      for (int k = 0; k < 4; ++k) bias[g][k] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        q[0].operand(g, h, sc, b[g][h][0], b[g][h][1]);
        // -8 and -128 times 2^-24
        mma_f16(bias[g], 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, b[g][h][0], b[g][h][1]);
      }
    }
  }
  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int mi = 0; mi < 8; ++mi) o[mi][0] = o[mi][1] = o[mi][2] = o[mi][3] = 0.f;
  }

  // O^T += V^T P^T of 16 tokens: per group of 32 d the codes, widened exactly,
  // times P scaled by the tokens' scales: bf16, for its range, with one rounding
  // (2^-8), since P comes as the sum of two bf16, p and what it lacks (n).
  __device__ __forceinline__ void values(uint32_t st, int mb, int r, int c, uint32_t p0, uint32_t p1, uint32_t n0,
                                         uint32_t n1) {
    const uint4 v0 = lds128(st + kI4OffV + ((2 * mb) * 32 + r * 4 + c) * 16);
    const uint4 v1 = lds128(st + kI4OffV + ((2 * mb + 1) * 32 + r * 4 + c) * 16);
    const uint4 s0 = lds128(st + kI4OffVs + (8 * mb + c) * 16);
    const uint4 s1 = lds128(st + kI4OffVs + (8 * mb + 4 + c) * 16);
    const uint32_t va[4] = {v0.x, v0.y, v0.z, v0.w}, vb[4] = {v1.x, v1.y, v1.z, v1.w};
    const uint32_t sa[4] = {s0.x, s0.y, s0.z, s0.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int g = 0; g < kI4Groups; ++g) {
      const uint32_t q0 = fma_bf16x2(p0, sa[g], mul_bf16x2(n0, sa[g]));
      const uint32_t q1 = fma_bf16x2(p1, sb[g], mul_bf16x2(n1, sb[g]));
#pragma unroll
      for (int jp = 0; jp < 2; ++jp)
        // d = 32g + 4r + 2jp on rows r, a quarter of the next one on rows r + 8
        mma_bf16(o[2 * g + jp], i4_code_lo(va[g] >> (8 * jp)), i4_code_hi4(va[g] >> (8 * jp)),
                 i4_code_lo(vb[g] >> (8 * jp)), i4_code_hi4(vb[g] >> (8 * jp)), q0, q1);
    }
  }

  // A tile at shared address st; the query sees its first nv[0] tokens.
  __device__ __forceinline__ void tile(uint32_t st, const int (&nv)[1], int lane) {
    const int r = lane >> 2, c = lane & 3;
    // S^T = K Q^T: per group of 32 d two products on the codes, then the
    // tokens' scales in fp32; x[mb]: tokens 16 mb + r and + 8, unscaled
    float x[4][4];
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const int t0 = 16 * mb + r;
      const uint4 k0 = lds128(st + t0 * 64 + c * 16);
      const uint4 k1 = lds128(st + (t0 + 8) * 64 + c * 16);
      const uint2 s0 = lds64(st + kI4OffKs + t0 * 8);
      const uint2 s1 = lds64(st + kI4OffKs + (t0 + 8) * 8);
      const uint32_t ka[4] = {k0.x, k0.y, k0.z, k0.w}, kb[4] = {k1.x, k1.y, k1.z, k1.w};
      const float sa[4] = {bf16_lo(s0.x), bf16_hi(s0.x), bf16_lo(s0.y), bf16_hi(s0.y)};
      const float sb[4] = {bf16_lo(s1.x), bf16_hi(s1.x), bf16_lo(s1.y), bf16_hi(s1.y)};
#pragma unroll
      for (int g = 0; g < kI4Groups; ++g) {
        const uint32_t ka8 = ka[g] >> 8, kb8 = kb[g] >> 8;
        float acc[4];
        mma_f16_c(acc, ka[g] & 0x000f000fu, kb[g] & 0x000f000fu, ka[g] & 0x00f000f0u, kb[g] & 0x00f000f0u,
                  b[g][0][0], b[g][0][1], bias[g]);
        mma_f16(acc, ka8 & 0x000f000fu, kb8 & 0x000f000fu, ka8 & 0x00f000f0u, kb8 & 0x00f000f0u, b[g][1][0],
                b[g][1][1]);
        x[mb][0] = g == 0 ? sa[g] * acc[0] : fmaf(sa[g], acc[0], x[mb][0]);
        x[mb][1] = g == 0 ? sa[g] * acc[1] : fmaf(sa[g], acc[1], x[mb][1]);
        x[mb][2] = g == 0 ? sb[g] * acc[2] : fmaf(sb[g], acc[2], x[mb][2]);
        x[mb][3] = g == 0 ? sb[g] * acc[3] : fmaf(sb[g], acc[3], x[mb][3]);
      }
    }
    if (nv[0] < kPage) {   // tokens the query does not see
      i4_hide_tokens(st, nv[0], nv[0], lane, nv);
#pragma unroll
      for (int mb = 0; mb < 4; ++mb) {
        if (16 * mb + r >= nv[0]) x[mb][0] = x[mb][1] = -INFINITY;
        if (16 * mb + r + 8 >= nv[0]) x[mb][2] = x[mb][3] = -INFINITY;
      }
    }
    // the online softmax; P^T as B operands by 8x8 transposes
    float mt0 = -INFINITY, mt1 = -INFINITY;
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      mt0 = max3f(mt0, x[mb][0], x[mb][2]);
      mt1 = max3f(mt1, x[mb][1], x[mb][3]);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mt0 = fmaxf(mt0, __shfl_xor_sync(0xffffffffu, mt0, off));
      mt1 = fmaxf(mt1, __shfl_xor_sync(0xffffffffu, mt1, off));
    }
    mt0 *= c0;
    mt1 *= c1;
    const bool g0 = mt0 > m0 + kI4Grow, g1 = mt1 > m1 + kI4Grow;
    if (__any_sync(0xffffffffu, g0 || g1)) {
      const float al0 = g0 ? exp2_ftz(m0 - mt0) : 1.f, al1 = g1 ? exp2_ftz(m1 - mt1) : 1.f;
      if (g0) m0 = mt0;
      if (g1) m1 = mt1;
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int mi = 0; mi < 8; ++mi) {
        o[mi][0] *= al0;
        o[mi][1] *= al1;
        o[mi][2] *= al0;
        o[mi][3] *= al1;
      }
    }
    const float ms0 = m0 == -INFINITY ? 0.f : m0, ms1 = m1 == -INFINITY ? 0.f : m1;
    uint32_t pb[4][2], nb[4][2];
    auto transpose = [](float a, float b, uint32_t& p, uint32_t& n) {
      const uint32_t w = pack_bf16(a, b);
      p = movmatrix_t(w);
      n = movmatrix_t(pack_bf16(a - bf16_lo(w), b - bf16_hi(w)));
    };
    float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const float p0 = exp2_ftz(fmaf(x[mb][0], c0, -ms0)), p1 = exp2_ftz(fmaf(x[mb][1], c1, -ms1));
      const float p2 = exp2_ftz(fmaf(x[mb][2], c0, -ms0)), p3 = exp2_ftz(fmaf(x[mb][3], c1, -ms1));
      ps0 += p0 + p2;
      ps1 += p1 + p3;
      transpose(p0, p1, pb[mb][0], nb[mb][0]);
      transpose(p2, p3, pb[mb][1], nb[mb][1]);
    }
    l0 += ps0;
    l1 += ps1;
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) values(st, mb, r, c, pb[mb][0], pb[mb][1], nb[mb][0], nb[mb][1]);
  }

  // The state, once its tiles are done: sums over the lanes ..
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
  }
  // .. O as rows: f(query, head, d, elements d .. d+3, m, l) for what the lane
  // has; odd elements of V's code order are quarters (i4_code_hi4) ..
  template <int kFrom, int kTo, typename F>   // (queries kFrom .. kTo - 1)
  __device__ __forceinline__ void rows(int lane, F f) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int g = 0; g < kI4Groups; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f(0, 2 * c + h, 32 * g + 4 * r,
          make_float4(o[2 * g][h], 4.f * o[2 * g][2 + h], o[2 * g + 1][h], 4.f * o[2 * g + 1][2 + h]),
          h == 0 ? m0 : m1, h == 0 ? l0 : l1);
  }
  // .. and maxima and sums: f(query, head, m, l), each once per warp.
  template <typename F>
  __device__ __forceinline__ void stats(int lane, F f) const {
    if (lane < 4) {
      f(0, 2 * lane, m0, l0);
      f(0, 2 * lane + 1, m1, l1);
    }
  }
  // O to tensor memory and back (round: the queries of a round of the merge)
  __device__ __forceinline__ void park(uint32_t tm) const {
    uint32_t v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(o[k >> 2][k & 3]);
    tmem_st32(tm, v);
    tmem_wait_st();
  }
  __device__ __forceinline__ void unpark(uint32_t tm, int round) {
    (void)round;
    uint32_t v[32];
    tmem_ld32(tm, v);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k >> 2][k & 3] = __uint_as_float(v[k]);
  }
};

// Two or four queries: 8 heads of two on the 16 rows of a product (kM products
// side by side), tokens (K) and d (V) on the columns.  So every code is
// widened once for all of them, P passes from the scores' fragments to the
// next product's as it is, and a row's maximum takes two shuffles.  Lane
// (r, c) has head r of each query.  Half a tile at a time; the queries'
// operands and biases are read from shared memory, once for its 32 tokens.
template <int kM>
struct I4Rows {
  uint32_t qa;   // shared memory: [kM][4 groups][nibbles 0, 1 | 2, 3][lane] {query 2m, 2m + 1, 2m, 2m + 1},
                 // then biases [kM][4 groups][r] {query 2m twice, 2m + 1 twice}
  float cs[kM][2];                     // from scores to log2 units, per query
  float mx[kM][2], ls[kM][2], o[kM][16][4];   // o[m][4g + j]: query 2m (columns 2c, 2c+1), query 2m + 1

  __device__ __forceinline__ uint32_t operand_at(int m, int g, int h, int lane) const {
    return qa + ((m * kI4Groups + g) * 2 + h) * 512 + lane * 16;
  }
  __device__ __forceinline__ uint32_t bias_at(int m, int g, int r) const {
    return qa + kM * 4096 + (m * kI4Groups + g) * 128 + r * 16;
  }
  __device__ __forceinline__ void open(const I4Row (&q)[2 * kM], float scale_log2, int lane) {
    __syncwarp();   // the previous piece's biases are read
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      float s0, s1;
      i4_row_scale(q[2 * m].largest(), scale_log2, s0, cs[m][0]);
      i4_row_scale(q[2 * m + 1].largest(), scale_log2, s1, cs[m][1]);
#pragma unroll
      for (int g = 0; g < kI4Groups; ++g) {
        float b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[4];
          q[2 * m].operand(g, h, s0, a[0], a[2]);
          q[2 * m + 1].operand(g, h, s1, a[1], a[3]);
          sts128(operand_at(m, g, h, lane), a[0], a[1], a[2], a[3]);
          // -8 and -128 times 2^-24
          mma_f16(b, a[0], a[1], a[2], a[3], 0x80088008u, 0x80808080u);
        }
        if ((lane & 3) == 0)
          sts128(bias_at(m, g, lane >> 2), __float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]),
                 __float_as_uint(b[3]));
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      mx[m][0] = mx[m][1] = -INFINITY;
      ls[m][0] = ls[m][1] = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) o[m][k][0] = o[m][k][1] = o[m][k][2] = o[m][k][3] = 0.f;
    }
  }

  // O += P V of 16 tokens (see I4Warp<1>::values; here P x scale is rounded from
  // fp32): x[m][nt] = P of queries 2m (twice), 2m + 1 (twice) for tokens 2c, 2c+1,
  // x[m][nt + 1] for tokens 2c+8, 2c+9.
  __device__ __forceinline__ void values(uint32_t st, int mb, int r, int c, const float (&x)[kM][4][4], int nt) {
    const uint4 v0 = lds128(st + kI4OffV + ((2 * mb) * 32 + r * 4 + c) * 16);
    const uint4 v1 = lds128(st + kI4OffV + ((2 * mb + 1) * 32 + r * 4 + c) * 16);
    const uint4 s0 = lds128(st + kI4OffVs + (8 * mb + c) * 16);
    const uint4 s1 = lds128(st + kI4OffVs + (8 * mb + 4 + c) * 16);
    const uint32_t va[4] = {v0.x, v0.y, v0.z, v0.w}, vb[4] = {v1.x, v1.y, v1.z, v1.w};
    const uint32_t sa[4] = {s0.x, s0.y, s0.z, s0.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int g = 0; g < kI4Groups; ++g) {
      uint32_t p[kM][4];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const float a0 = bf16_lo(sa[g]), a1 = bf16_hi(sa[g]), b0 = bf16_lo(sb[g]), b1 = bf16_hi(sb[g]);
        const float(&u)[4] = x[m][nt], (&v)[4] = x[m][nt + 1];
        p[m][0] = pack_bf16(u[0] * a0, u[1] * a1), p[m][1] = pack_bf16(u[2] * a0, u[3] * a1);
        p[m][2] = pack_bf16(v[0] * b0, v[1] * b1), p[m][3] = pack_bf16(v[2] * b0, v[3] * b1);
      }
#pragma unroll
      for (int jp = 0; jp < 2; ++jp) {   // columns n: d = 32g + 4n + 2jp, then a quarter of the next
        const uint32_t l0 = i4_code_lo(va[g] >> (8 * jp)), l1 = i4_code_lo(vb[g] >> (8 * jp));
        const uint32_t h0 = i4_code_hi4(va[g] >> (8 * jp)), h1 = i4_code_hi4(vb[g] >> (8 * jp));
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          mma_bf16(o[m][4 * g + 2 * jp], p[m][0], p[m][1], p[m][2], p[m][3], l0, l1);
          mma_bf16(o[m][4 * g + 2 * jp + 1], p[m][0], p[m][1], p[m][2], p[m][3], h0, h1);
        }
      }
    }
  }

  // A tile at shared address st; query j sees its first nv[j] tokens.
  __device__ __forceinline__ void tile(uint32_t st, const int (&nv)[2 * kM], int lane) {
    const int r = lane >> 2, c = lane & 3;
    int most = 0, least = kPage;
#pragma unroll
    for (int j = 0; j < 2 * kM; ++j) {
      most = max(most, nv[j]);
      least = min(least, nv[j]);
    }
    if (least < kPage) hide(st, nv, max(least, 0), most, lane);
#pragma unroll 1
    for (int half = 0; half < 2 && 32 * half < most; ++half) {
      // x[m][nt]: tokens 32 half + 8 nt + 2c, + 1; queries 2m, 2m + 1, unscaled
      float x[kM][4][4];
      {
        uint32_t kw[4][4], sw[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t0 = 32 * half + 8 * e;
          const uint4 k0 = lds128(st + (t0 + r) * 64 + c * 16);
          const uint4 s0 = lds128(st + kI4OffKs + (t0 + 2 * c) * 8);   // token 2c: x, y; the next: z, w
          kw[e][0] = k0.x, kw[e][1] = k0.y, kw[e][2] = k0.z, kw[e][3] = k0.w;
          sw[e][0] = s0.x, sw[e][1] = s0.y, sw[e][2] = s0.z, sw[e][3] = s0.w;
        }
#pragma unroll
        for (int m = 0; m < kM; ++m) {
#pragma unroll
          for (int g = 0; g < kI4Groups; ++g) {
            const uint4 a = lds128(operand_at(m, g, 0, lane)), b = lds128(operand_at(m, g, 1, lane));
            const uint4 bb = lds128(bias_at(m, g, r));
            const float bias[4] = {__uint_as_float(bb.x), __uint_as_float(bb.y), __uint_as_float(bb.z),
                                   __uint_as_float(bb.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = kw[e][g], k8 = w >> 8;
              float acc[4];
              mma_f16_c(acc, a.x, a.y, a.z, a.w, w & 0x000f000fu, w & 0x00f000f0u, bias);
              mma_f16(acc, b.x, b.y, b.z, b.w, k8 & 0x000f000fu, k8 & 0x00f000f0u);
              const uint32_t u = sw[e][g >> 1], v = sw[e][2 + (g >> 1)];
              const float sa = (g & 1) ? bf16_hi(u) : bf16_lo(u), sb = (g & 1) ? bf16_hi(v) : bf16_lo(v);
              float(&y)[4] = x[m][e];
              y[0] = g == 0 ? sa * acc[0] : fmaf(sa, acc[0], y[0]);
              y[1] = g == 0 ? sb * acc[1] : fmaf(sb, acc[1], y[1]);
              y[2] = g == 0 ? sa * acc[2] : fmaf(sa, acc[2], y[2]);
              y[3] = g == 0 ? sb * acc[3] : fmaf(sb, acc[3], y[3]);
            }
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        if (least < kPage) {   // tokens a query does not see
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const int t = 32 * half + 8 * nt + 2 * c;
            if (t >= nv[2 * m]) x[m][nt][0] = -INFINITY;
            if (t + 1 >= nv[2 * m]) x[m][nt][1] = -INFINITY;
            if (t >= nv[2 * m + 1]) x[m][nt][2] = -INFINITY;
            if (t + 1 >= nv[2 * m + 1]) x[m][nt][3] = -INFINITY;
          }
        }
        float mt0 = -INFINITY, mt1 = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          mt0 = max3f(mt0, x[m][nt][0], x[m][nt][1]);
          mt1 = max3f(mt1, x[m][nt][2], x[m][nt][3]);
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
          mt0 = fmaxf(mt0, __shfl_xor_sync(0xffffffffu, mt0, off));
          mt1 = fmaxf(mt1, __shfl_xor_sync(0xffffffffu, mt1, off));
        }
        mt0 *= cs[m][0];
        mt1 *= cs[m][1];
        const bool g0 = mt0 > mx[m][0] + kI4Grow, g1 = mt1 > mx[m][1] + kI4Grow;
        if (__any_sync(0xffffffffu, g0 || g1)) {
          const float al0 = g0 ? exp2_ftz(mx[m][0] - mt0) : 1.f, al1 = g1 ? exp2_ftz(mx[m][1] - mt1) : 1.f;
          if (g0) mx[m][0] = mt0;
          if (g1) mx[m][1] = mt1;
          ls[m][0] *= al0;
          ls[m][1] *= al1;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            o[m][k][0] *= al0;
            o[m][k][1] *= al0;
            o[m][k][2] *= al1;
            o[m][k][3] *= al1;
          }
        }
        const float ms0 = mx[m][0] == -INFINITY ? 0.f : mx[m][0], ms1 = mx[m][1] == -INFINITY ? 0.f : mx[m][1];
        float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          x[m][nt][0] = exp2_ftz(fmaf(x[m][nt][0], cs[m][0], -ms0));
          x[m][nt][1] = exp2_ftz(fmaf(x[m][nt][1], cs[m][0], -ms0));
          x[m][nt][2] = exp2_ftz(fmaf(x[m][nt][2], cs[m][1], -ms1));
          x[m][nt][3] = exp2_ftz(fmaf(x[m][nt][3], cs[m][1], -ms1));
          ps0 += x[m][nt][0] + x[m][nt][1];
          ps1 += x[m][nt][2] + x[m][nt][3];
        }
        ls[m][0] += ps0;
        ls[m][1] += ps1;
      }
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) values(st, 2 * half + mb, r, c, x, 2 * mb);
    }
  }

  // A partial tile: V's scales behind the last visible token become zero; a
  // NaN scale that only the later queries see becomes zero as well, and their
  // outputs of that group NaN.
  __device__ __forceinline__ void hide(uint32_t st, const int (&nv)[2 * kM], int least, int most, int lane) {
    const unsigned nan = i4_hide_tokens(st, least, most, lane, nv);
    if (nan == 0u) return;
    // bit 4j + g: query j sees a NaN in group g
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float n = __uint_as_float(0x7fc00000u);
        if (nan >> (8 * m + (k >> 2)) & 1u) o[m][k][0] = o[m][k][1] = n;
        if (nan >> (8 * m + 4 + (k >> 2)) & 1u) o[m][k][2] = o[m][k][3] = n;
      }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) ls[m][q] += __shfl_xor_sync(0xffffffffu, ls[m][q], off);
  }
  template <int kFrom, int kTo, typename F>
  __device__ __forceinline__ void rows(int lane, F f) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int j = kFrom; j < kTo; ++j)
#pragma unroll
      for (int g = 0; g < kI4Groups; ++g)
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // column 2c + k
          const int e = 2 * (j & 1) + k;
          const float(&x)[16][4] = o[j >> 1];
          f(j, r, 32 * g + 8 * c + 4 * k,
            make_float4(x[4 * g][e], 4.f * x[4 * g + 1][e], x[4 * g + 2][e], 4.f * x[4 * g + 3][e]), mx[j >> 1][j & 1],
            ls[j >> 1][j & 1]);
        }
  }
  template <typename F>
  __device__ __forceinline__ void stats(int lane, F f) const {
    if ((lane & 3) == 0) {
#pragma unroll
      for (int j = 0; j < 2 * kM; ++j) f(j, lane >> 2, mx[j >> 1][j & 1], ls[j >> 1][j & 1]);
    }
  }
  __device__ __forceinline__ void park(uint32_t tm) const {
#pragma unroll
    for (int part = 0; part < 2 * kM; ++part) {
      uint32_t v[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(o[part >> 1][8 * (part & 1) + (k >> 2)][k & 3]);
      tmem_st32(tm + 32 * part, v);
    }
    tmem_wait_st();
  }
  // (a round's two queries, into o[0])
  __device__ __forceinline__ void unpark(uint32_t tm, int round) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      uint32_t v[32];
      tmem_ld32(tm + 64 * round + 32 * part, v);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) o[0][8 * part + (k >> 2)][k & 3] = __uint_as_float(v[k]);
    }
  }
};
template <>
struct I4Warp<2> : I4Rows<1> {};
template <>
struct I4Warp<4> : I4Rows<2> {};

// One row of a segment of several items, by one warp: the items' partials in
// item order (row p0, then per_seg rows on), with four elements a lane.  A NaN
// among the log-sum-exps makes the row NaN.
__device__ __forceinline__ void i4_merge_row(const float* partial_o, const float* partial_lse, int64_t p0, int cnt,
                                          int per_seg, void* out, int64_t orow, int out_dtype) {
  const int lane = threadIdx.x & 31;
  auto item_lse = [&](int k) { return __ldcg(partial_lse + p0 + static_cast<int64_t>(k) * per_seg); };
  auto o_of = [&](int k) {
    return __ldcg(reinterpret_cast<const float4*>(partial_o + (p0 + static_cast<int64_t>(k) * per_seg) * kD +
                                                  4 * lane));
  };
  // the first items' loads all go out at once (most segments have two)
  const float lse = lane < cnt ? item_lse(lane) : -INFINITY;
  float4 pre[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < cnt) pre[k] = o_of(k);
  float M = lse;
  for (int k = lane + 32; k < cnt; k += 32) M = max_nan(M, item_lse(k));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float wsum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, float4 v) {
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
    wsum += w;
  };
  for (int k0 = 0; k0 < cnt && M != -INFINITY; k0 += 32) {
    const int n = min(32, cnt - k0);
    const float w = lane < n ? __expf((k0 == 0 ? lse : item_lse(k0 + lane)) - M) : 0.f;
    if (k0 == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (k < cnt) add(wk, pre[k]);
      }
    }
#pragma unroll 8
    for (int k = k0 == 0 ? 2 : 0; k < n; ++k) add(__shfl_sync(0xffffffffu, w, k), o_of(k0 + k));
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  store_out4(out, orow * kD + 4 * lane, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv, out_dtype);
}

// Segments of several items, after a range: as in the other forms, the CTA that
// finishes a segment's last item merges its partials, in item order; one warp
// per (segment, query, head).  The whole CTA.  (Two items' loads ahead, not four,
// and inline: with four, or out of line, the tiles' loop of four queries spills
// more, 185 us against 177.)
template <int kList>
__device__ __forceinline__ void i4_merge_segments(int4* list, int* list_len, int i0, int i1, const int4* items4,
                                               const int32_t* seg_ptr, int32_t* seg_done, int batch, int q_len,
                                               int capacity, const float* partial_o, const float* partial_lse,
                                               void* out, int out_dtype) {
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int noted = *list_len;   // (complete since the barrier after the tiles)
  const bool many = noted > kList;   // more than the list holds: looked up again
  __syncthreads();               // the partials are written
  for (int b = 0; b < (many ? i1 - i0 : noted); b += kList) {
    const int k = b + static_cast<int>(threadIdx.x);
    int4 e = make_int4(-1, 0, 0, 0);   // segment, first item, items
    if (!many && threadIdx.x < kList && k < noted) e = list[k];
    if (many && threadIdx.x < kList && k < i1 - i0) {
      const int4 d = items4[i0 + k];
      if (d.x >= 0 && d.x < batch && d.y >= 0 && d.y < kHkv) {
        const int seg = d.x * kHkv + d.y, s0 = seg_ptr[seg], cnt = seg_ptr[seg + 1] - s0;
        if (cnt > 1 && s0 >= 0 && s0 <= capacity - cnt) e = make_int4(seg, s0, cnt, 0);
      }
    }
    if (e.x >= 0) {
      if (atomic_add_acq_rel_gpu(&seg_done[e.x], 1) == e.z - 1)
        seg_done[e.x] = 0;   // reset for the next run of this plan
      else
        e.x = -1;
    }
    if (threadIdx.x == 0) *list_len = 0;
    __syncthreads();
    if (e.x >= 0) list[atomicAdd(list_len, 1)] = e;
    __syncthreads();
    const int per_seg = q_len * kGroup, tasks = *list_len * per_seg;
    for (int task = warp; task < tasks; task += warps) {
      const int4 of = list[task / per_seg];
      const int row = task % per_seg;   // query, head
      const int seg = of.x, cnt = of.z;
      const int64_t p0 = static_cast<int64_t>(of.y) * per_seg + row;
      const int64_t orow = (static_cast<int64_t>(seg / kHkv) * q_len + row / kGroup) * kHq +
                           (seg % kHkv) * kGroup + row % kGroup;
      i4_merge_row(partial_o, partial_lse, p0, cnt, per_seg, out, orow, out_dtype);
    }
    __syncthreads();
  }
}

template <int kNq>
__global__ void __launch_bounds__(I4Cfg<kNq>::kThreads, 1) decode_attn_i4_kernel(
    // the plan arrays, q and the cache may be written by the kernel this one
    // is a programmatic dependent of: plain (coherent) loads, after the wait
    const uint8_t* kv_cache, const uint16_t* q, const int32_t* __restrict__ block_table,
    int32_t max_blocks, int32_t num_blocks, const int32_t* __restrict__ seq_lens, int32_t batch,
    int32_t q_len, const hpc_work_item* items, const int32_t* cta_ptr, const int32_t* home_end,
    int32_t* pool, int32_t capacity, float* __restrict__ partial_o, float* __restrict__ partial_lse,
    float sm_scale, int32_t* __restrict__ status, unsigned long long* __restrict__ cta_clock,
    const int32_t* seg_ptr, int32_t* seg_done, void* __restrict__ out, int32_t out_dtype) {
  using C = I4Cfg<kNq>;
  constexpr int W = C::kWarps, S = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 127u) & ~127u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (kept in registers: the compiler would read the thread's number anew several
  // times a tile; 0.8 % of the heavy tail, but 2 % the other way with more queries)
  if constexpr (kNq == 1) asm volatile("" : "+r"(warp), "+r"(lane));
  const bool fuse = out != nullptr;
  auto full_bar = [&](int w, int s) { return base + C::kOffBar + (w * C::kBars + s) * 8; };
  auto empty_bar = [&](int w, int s) { return base + C::kOffBar + (w * C::kBars + S + s) * 8; };
  auto free_bar = [&](int w, int st) { return base + C::kOffBar + (w * C::kBars + 2 * S + st) * 8; };
  auto meta_of = [&](int w, int s) {
    return reinterpret_cast<int4*>(smem + C::kOffMeta + (w * S + s) * 32);
  };
  int4* pieces = reinterpret_cast<int4*>(smem + C::kOffPieces);   // [W][2] {item, flags, seq, -}
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffCtl);
  volatile int* range = abort_flag + 1;
  int* list_len = reinterpret_cast<int*>(smem + C::kOffCtl) + 3;
  int4* list = reinterpret_cast<int4*>(smem + C::kOffList);
  const int4* items4 = reinterpret_cast<const int4*>(items);

  const unsigned long long t_start = cta_clock != nullptr ? globaltimer_ns() : 0ull;
  if (threadIdx.x < W * C::kBars) {
    mbar_init(base + C::kOffBar + 8 * threadIdx.x, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  // everything above is independent of the previous kernel on the stream
  pdl_wait();

  // The CTA's home range, then pooled items claimed one at a time; the last
  // CTA to find the pool empty resets its counters.
  const int vq = static_cast<int>(blockIdx.x);
  const int pool_len = pool[2];
  const int home_begin = cta_ptr[vq], home_stop = home_end[vq];
  auto finish_claims = [&]() {
    if (pool_len != 0 && atomicAdd(&pool[1], 1) == static_cast<int>(gridDim.x) - 1) {
      pool[0] = 0;
      pool[1] = 0;
    }
  };
  if (pool_len < 0 || pool_len > capacity || home_begin < 0 || home_stop < home_begin ||
      home_stop > capacity) {
    if (threadIdx.x == 0) {
      atomicOr(status, HPC_STATUS_BAD_PLAN);
      finish_claims();
      if (cta_clock != nullptr) record_cta_clock(cta_clock, t_start);
    }
    return;
  }

  if (warp == W) tmem_alloc(smem_u32(smem + C::kOffTmem), C::kTmemCols);
  tc_fence_before();   // (the first range's barrier)

  uint32_t n_slot = 0;   // slots issued (producer, per lane) or taken (consumer) so far
  uint32_t n_tile = 0;   // and tiles
  auto tmem_of = [&](int w) {
    return *reinterpret_cast<volatile uint32_t*>(smem + C::kOffTmem) + (static_cast<uint32_t>(32 * (w & 3)) << 16) +
           64u * kNq * (w >> 2);
  };
  auto stats_of = [&](int w, int k) {   // of state k of warp w: [queries][m, l][8]
    return reinterpret_cast<float*>(smem + C::kOffStats) + (w * 2 + k) * kNq * 2 * kGroup;
  };
  int next_begin = home_begin, next_end = home_stop;
  bool first_range = true;

  while (true) {
    // ------------------------------------------------------------ next range
    if (threadIdx.x == 0) {
      if (!first_range) {
        next_begin = next_end = 0;
        while (pool_len > 0 && !*abort_flag) {
          const int k = atomicAdd(&pool[0], 1);
          if (k >= pool_len) break;
          const int idx = pool[3 + k];
          if (idx >= 0 && idx < capacity) {
            next_begin = idx;
            next_end = idx + 1;
            break;
          }
          atomicOr(status, HPC_STATUS_BAD_PLAN);
        }
      }
      range[0] = next_begin;
      range[1] = next_end;
      *list_len = 0;
    }
    if (threadIdx.x < 2 * W) pieces[threadIdx.x] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    tc_fence_after();
    const int i0 = range[0], i1 = range[1];
    if (!first_range && i1 <= i0) break;

    if (warp == W) {
      // ---------------------------------------------------------- producer
      // An item's tiles, for the cut of the range (its length is looked up
      // later, together with the block ids).  An item out of any range counts
      // as one tile without data, so that it gets its (empty) partial.
      auto item_tiles = [&](int4 d) { return d.z >= 0 && d.z < d.w && d.w <= max_blocks ? d.w - d.z : 1; };
      // (ranges of up to 32 items, most of them, keep theirs in registers: lane j
      // item i0 + j)
      const bool few = i1 - i0 <= 32;
      int4 kd = make_int4(-1, -1, 0, 0);
      int kn = 0;
      int64_t total = 0;
      for (int b = i0; b < i1; b += 32) {
        kn = 0;
        if (b + lane < i1) {
          kd = items4[b + lane];
          kn = item_tiles(kd);
        }
        int n = kn;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        total += n;
      }
      // lane w: warp w's run [run0, run1) of the range's tiles
      // (a range holds fewer than 2^30 tiles)
      const int each = static_cast<int>(total) / W, more = static_cast<int>(total) - each * W;
      const int run0 = lane < W ? lane * each + min(lane, more) : 0;
      int rem = lane < W ? each + (lane < more ? 1 : 0) : 0;
      // its first item and the tile in it
      int idx = i0, off = 0;
      {
        int64_t seen = 0;
        for (int b = i0; b < i1 && seen < total; b += 32) {
          int n = kn;
          if (!few) {
            n = 0;
            if (b + lane < i1) n = item_tiles(items4[b + lane]);
          }
          int incl = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          const int excl = incl - n, chunk = __shfl_sync(0xffffffffu, incl, 31);
          const bool here = run0 >= seen && run0 < seen + chunk;
          const int v = here ? run0 - static_cast<int>(seen) : 0;
          int src = 0;   // the last item of the chunk that starts at or before v
#pragma unroll
          for (int step = 16; step > 0; step >>= 1)
            if (__shfl_sync(0xffffffffu, excl, (src + step) & 31) <= v && src + step < 32) src += step;
          const int e = __shfl_sync(0xffffffffu, excl, src);
          if (here) {
            idx = b + src;
            off = v - e;
          }
          seen += chunk;
        }
      }
      // cur: the tile being issued; nxt: the one after it, its loads in
      // flight; look: the descriptor of the item after nxt's
      struct Tile {
        int4 d;       // the item
        int idx, t, len, bid;
        bool begins;  // a piece begins with this tile
      };
      auto load_tile = [&](Tile& x, int4 d, int i, int t, bool begins) {
        x.d = d;
        x.idx = i;
        x.t = t;
        x.begins = begins;
        const int sq = d.x >= 0 && d.x < batch ? d.x : 0;
        x.len = batch > 0 ? __ldg(seq_lens + sq) : -1;
        x.bid = __ldg(block_table + static_cast<int64_t>(sq) * max_blocks + max(0, min(t, max_blocks - 1)));
      };
      auto item_of = [&](const Tile& x) {
        return make_item(x.d, x.d.x >= 0 && x.d.x < batch ? x.len : -1, batch, max_blocks);
      };
      Tile cur, nxt;
      int4 look = make_int4(-1, -1, 0, 0);
      auto advance = [&](int left) {   // nxt from the tile after it; left: tiles from nxt on
        cur = nxt;
        if (left <= 1) return;
        if (cur.t + 1 < cur.d.z + item_tiles(cur.d)) {
          load_tile(nxt, cur.d, cur.idx, cur.t + 1, false);
        } else {
          load_tile(nxt, look, cur.idx + 1, look.z, true);
          if (cur.idx + 2 < i1) look = items4[cur.idx + 2];
        }
      };
      int step = 0;   // 0: the opening of the tile's piece, 1: the tile, 2: stop
      {
        // the run's first item and the one after it
        int4 d;
        const int s0 = (idx - i0) & 31, s1 = (idx + 1 - i0) & 31;
        d.x = __shfl_sync(0xffffffffu, kd.x, s0), d.y = __shfl_sync(0xffffffffu, kd.y, s0);
        d.z = __shfl_sync(0xffffffffu, kd.z, s0), d.w = __shfl_sync(0xffffffffu, kd.w, s0);
        look.x = __shfl_sync(0xffffffffu, kd.x, s1), look.y = __shfl_sync(0xffffffffu, kd.y, s1);
        look.z = __shfl_sync(0xffffffffu, kd.z, s1), look.w = __shfl_sync(0xffffffffu, kd.w, s1);
        if (rem > 0) {
          if (!few) {
            d = items4[idx];
            if (idx + 1 < i1) look = items4[idx + 1];
          }
          load_tile(nxt, d, idx, d.z + off, true);
          advance(rem);
        } else {
          step = 2;
        }
      }
      bool done = lane >= W;
      const uint64_t policy = l2_evict_first_policy();
      unsigned long long idle_since = 0ull;
      while (true) {
        bool did = false;
        if (!done) {
          const int s = static_cast<int>(n_slot % S), sg = static_cast<int>(n_tile % C::kStages);
          const uint32_t use = n_slot / S, tuse = n_tile / C::kStages;
          if ((use == 0 || mbar_test_wait(empty_bar(lane, s), (use - 1) & 1)) &&
              (step != 1 || tuse == 0 || mbar_test_wait(free_bar(lane, sg), (tuse - 1) & 1))) {
            did = true;
            ++n_slot;
            int4* m = meta_of(lane, s);
            const uint32_t fb = full_bar(lane, s);
            if (step == 2) {
              m[0] = make_int4(0, kI4Stop, 0, 0);
              mbar_arrive(fb);
              done = true;
            } else {
              const Item it = item_of(cur);
              const bool known = cur.d.x >= 0 && cur.d.x < batch && cur.d.y >= 0 && cur.d.y < kHkv;
              if (step == 0) {
                // (run-begins inside an item do not start it)
                const int fl = (known ? kI4Known | cur.d.y : 0) | kI4Open |
                               (cur.t == cur.d.z ? kI4Start : 0);
                m[0] = make_int4(cur.idx, fl, cur.d.x, 0);
                mbar_arrive(fb);
                step = 1;
              } else {
                const bool data = it.ok && cur.bid >= 0 && cur.bid < num_blocks;
                const bool end = cur.t + 1 == cur.d.z + item_tiles(cur.d);
                m[0] = make_int4(cur.idx, (end || rem == 1 ? kI4Last : 0) | (end ? kI4End : 0) | (data ? kI4Ok : 0),
                                 0, it.len - cur.t * kPage);
                if (data) {
                  mbar_arrive_expect_tx(fb, kI4Record);
                  bulk_load(base + lane * C::kRing + sg * kI4Record,
                            kv_cache + (static_cast<int64_t>(cur.bid) * kHkv + it.h) * kI4Record, kI4Record, fb,
                            policy);
                } else {
                  atomicOr(status, it.ok ? HPC_STATUS_BAD_BLOCK : HPC_STATUS_BAD_PLAN);
                  mbar_arrive(fb);
                }
                ++n_tile;
                if (--rem > 0) {
                  advance(rem);
                  step = cur.begins ? 0 : 1;
                } else {
                  step = 2;
                }
              }
            }
          }
        }
        if (__all_sync(0xffffffffu, done)) break;
        if (__any_sync(0xffffffffu, did)) {
          idle_since = 0ull;
        } else {
          if (poll_give_up(idle_since, abort_flag, status, kWaitLimitNs)) break;
          __nanosleep(200);
        }
      }
      __syncwarp();
      if (*abort_flag && lane < W) {
        // copies still in flight land before anything else touches the ring
        for (uint32_t s = 0; s < static_cast<uint32_t>(S) && s < n_slot; ++s) {
          const uint32_t last = s + S * ((n_slot - 1 - s) / S);
          mbar_wait(full_bar(lane, s), (last / S) & 1, status);
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- consumer
      const float scale_log2 = sm_scale * 1.4426950408889634f;
      if (fuse) {
        // segments of several items whose items this range holds (at the
        // range's ends, as plans go): noted while the first tiles are on
        // their way, counted when they are done
        for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += 32 * W) {
          const int4 d = items4[i];
          if (d.x >= 0 && d.x < batch && d.y >= 0 && d.y < kHkv) {
            const int seg = d.x * kHkv + d.y;
            const int s0 = seg_ptr[seg], cnt = seg_ptr[seg + 1] - s0;
            if (cnt > 1 && s0 >= 0 && s0 <= capacity - cnt) {
              const int k = atomicAdd(list_len, 1);
              if (k < C::kList) list[k] = make_int4(seg, s0, cnt, 0);
            }
          }
        }
      }
      if (first_range && fuse) {
        // rows of empty sequences (no items): zeros, the segments spread over the warps
        for (int s0 = 0; vq + static_cast<int>(gridDim.x) * s0 < batch * kHkv; s0 += 32 * W) {
          const int64_t sg = vq + static_cast<int64_t>(gridDim.x) * (s0 + warp * 32 + lane);
          const bool none = sg < batch * kHkv && seg_ptr[sg + 1] == seg_ptr[sg];
          unsigned todo = __ballot_sync(0xffffffffu, none);
          while (todo != 0u) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            const int e = static_cast<int>(__shfl_sync(0xffffffffu, static_cast<int>(sg), src));
            for (int x = lane * 4; x < q_len * kGroup * kD; x += 128) {
              const int j = x / (kGroup * kD), y = x - j * kGroup * kD;
              store_out4(out, ((static_cast<int64_t>(e / kHkv) * q_len + j) * kHq + (e % kHkv) * kGroup) * kD + y,
                         0.f, 0.f, 0.f, 0.f, out_dtype);
            }
          }
        }
      }
      const uint32_t ring = base + warp * C::kRing;
      int split = 0;   // states handed over in this range
      int4 open = make_int4(-1, 0, 0, 0);
      int seg_items = 0;
      I4Warp<kNq> st;   // the queries and the state of the open piece
      // two states can wait there: this warp's lanes, 32 columns a query each
      const uint32_t tm = tmem_of(warp);
      if constexpr (kNq > 1) st.qa = base + C::kOffQ + warp * C::kQBytes;
      auto wait_slot = [&](int s) -> bool {   // (mostly it is there: one test, no look at the flag)
        if (__all_sync(0xffffffffu, mbar_try_wait(full_bar(warp, s), (n_slot / S) & 1))) return true;
        bool ok = !*abort_flag && mbar_wait(full_bar(warp, s), (n_slot / S) & 1, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) *abort_flag = 1;
        return ok;
      };
      auto release = [&](int s) {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(warp, s));
        ++n_slot;
      };
      while (true) {
        const int s = static_cast<int>(n_slot % S);
        if (!wait_slot(s)) break;
        const int4 m = *meta_of(warp, s);
        if (m.y & kI4Stop) {
          release(s);
          break;
        }
        if (m.y & kI4Open) {
          // a piece of an item begins: its queries, an empty state
          open = m;
          release(s);
          seg_items = 0;
          if (open.y & kI4Known) {
            const int h = open.y & kI4Head;
            if (fuse) {
              const int seg = open.z * kHkv + h;
              seg_items = seg_ptr[seg + 1] - seg_ptr[seg];
            }
            I4Row qr[kNq];
#pragma unroll
            for (int jn = 0; jn < kNq; ++jn)
              // (a query past q_len: the last one's, never stored)
              qr[jn].load(q + ((static_cast<int64_t>(open.z) * q_len + min(jn, q_len - 1)) * kHq +
                               h * kGroup + (lane >> 2)) * kD + 8 * (lane & 3));
            st.open(qr, scale_log2, lane);
          }
          st.reset();
          continue;
        }
        // a tile
        int nv[kNq];
        int most = 0;
#pragma unroll
        for (int jn = 0; jn < kNq; ++jn) {
          // (a query past q_len, never stored, sees all: no tile is partial for it)
          nv[jn] = jn < q_len ? m.w - (q_len - 1 - jn) : kPage;
          most = max(most, nv[jn]);
        }
        if ((m.y & kI4Ok) && most > 0) st.tile(ring + (n_tile % C::kStages) * kI4Record, nv, lane);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(free_bar(warp, n_tile % C::kStages));
          mbar_arrive(empty_bar(warp, s));
        }
        ++n_tile;
        ++n_slot;
        if (!(m.y & kI4Last)) continue;

        // ---- the piece is over
        st.finish();
        const int h = open.y & kI4Head;
        if ((open.y & kI4Start) && (m.y & kI4End)) {
          // the whole item: its partial, or its segment's only item: the output
          const bool direct = fuse && (open.y & kI4Known) && seg_items == 1;
          st.template rows<0, kNq>(lane, [&](int j, int hh, int d, float4 v, float, float l) {
            if (j >= q_len) return;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
            if (direct)
              store_out4(out, ((static_cast<int64_t>(open.z) * q_len + j) * kHq + h * kGroup + hh) * kD + d, v.x,
                         v.y, v.z, v.w, out_dtype);
            else
              *reinterpret_cast<float4*>(partial_o + ((static_cast<int64_t>(m.x) * q_len + j) * kGroup + hh) * kD + d) = v;
          });
          if (!direct)
            st.stats(lane, [&](int j, int hh, float mx, float l) {
              if (j < q_len) partial_lse[(static_cast<int64_t>(m.x) * q_len + j) * kGroup + hh] = lse_of(mx, l);
            });
        } else {
          // Shared with other warps: a state to hand over when the range is
          // done (a run has at most two, its first and its last piece).  Other
          // tiles may still stream through the ring, so O waits in tensor
          // memory.
          st.park(tm + 32u * kNq * split);
          float* sm = stats_of(warp, split);
          st.stats(lane, [&](int j, int hh, float mx, float l) {
            sm[j * 2 * kGroup + hh] = mx;
            sm[j * 2 * kGroup + kGroup + hh] = l;
          });
          if (lane == 0)
            pieces[warp * 2 + split] = make_int4(m.x, open.y | (m.y & kI4End), open.z, seg_items);
          ++split;
        }
      }
    }
    __syncthreads();
    if (*abort_flag) break;
    // ------------------------------------------------- shared items' states
    // Entries in the order of the range's tiles: runs, then a run's first and
    // second state.  An item's entries begin at one that starts it and end at
    // the next one that ends it; one warp per (item, query, head), a lane per
    // four elements, states in their fixed order, one or two queries a round.
    {
      const int4 mine = lane < 2 * W ? pieces[lane] : make_int4(-1, 0, 0, 0);
      const unsigned valid = __ballot_sync(0xffffffffu, mine.x >= 0);
      const unsigned starts = __ballot_sync(0xffffffffu, mine.x >= 0 && (mine.y & kI4Start));
      const unsigned ends = __ballot_sync(0xffffffffu, mine.x >= 0 && (mine.y & kI4End));
#pragma unroll 1
      for (int round = 0; valid != 0u && round * C::kRoundNq < q_len; ++round) {
        // this warp's states of the round's queries, from tensor memory to its
        // ring (no copy is in flight any more)
        if (round > 0) __syncthreads();
        if (warp < W) {
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            if (!(valid >> (2 * warp + k) & 1u)) break;
            I4Warp<kNq> back;
            back.unpark(tmem_of(warp) + 32u * kNq * k, round);
            float* so = reinterpret_cast<float*>(smem + warp * C::kRing + k * C::kState);
            back.template rows<0, C::kRoundNq>(lane, [&](int j, int hh, int d, float4 v, float, float) {
              *reinterpret_cast<float4*>(so + (j * kGroup + hh) * C::kOStride + d) = v;
            });
          }
        }
        __syncthreads();
        const int per_item = min(C::kRoundNq, q_len - round * C::kRoundNq) * kGroup;
#pragma unroll 1
        for (int task = warp; task < __popc(starts) * per_item; task += W + 1) {
          unsigned rest = starts;
          for (int k = task / per_item; k > 0; --k) rest &= rest - 1;
          const int e0 = __ffs(rest) - 1;
          const unsigned tail = ends >> e0;
          if (tail == 0u) continue;   // (an item always ends in its range)
          const int e1 = e0 + __ffs(tail) - 1;
          const int jr = task % per_item / kGroup, hh = task % kGroup, j = round * C::kRoundNq + jr;
          const int4 head = pieces[e0];
          // lane k: entry k's maximum and sum, then its weight
          const bool in = lane >= e0 && lane <= e1 && (valid >> lane & 1u);
          const float* sm = stats_of(lane >> 1, lane & 1) + j * 2 * kGroup + hh;
          const float mk = in ? sm[0] : -INFINITY, lk = in ? sm[kGroup] : 0.f;
          float M = mk;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
          const float Ms = M == -INFINITY ? 0.f : M;
          const float wk = exp2_ftz(mk - Ms);
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = e0; k <= e1; ++k) {
            const float w = __shfl_sync(0xffffffffu, wk, k), l = __shfl_sync(0xffffffffu, lk, k);
            if (!(valid >> k & 1u)) continue;
            const float4 v = *reinterpret_cast<const float4*>(
                smem + (k >> 1) * C::kRing + (k & 1) * C::kState + ((jr * kGroup + hh) * C::kOStride + 4 * lane) * 4);
            L += w * l;
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
          const int h = head.y & kI4Head;
          if (fuse && (head.y & kI4Known) && head.w == 1) {
            store_out4(out, ((static_cast<int64_t>(head.z) * q_len + j) * kHq + h * kGroup + hh) * kD + 4 * lane,
                       acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv, out_dtype);
          } else {
            const int64_t prow = (static_cast<int64_t>(head.x) * q_len + j) * kGroup + hh;
            *reinterpret_cast<float4*>(partial_o + prow * kD + 4 * lane) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (lane == 0) partial_lse[prow] = lse_of(Ms, L);
          }
        }
      }
    }
    if (fuse)
      i4_merge_segments<C::kList>(list, list_len, i0, i1, items4, seg_ptr, seg_done, batch, q_len, capacity, partial_o,
                                  partial_lse, out, out_dtype);
    fence_proxy_async_smem();   // the states lay where the next range's copies land
    __syncthreads();
    first_range = false;
  }
  // every warp is done with tensor memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W) tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(smem + C::kOffTmem), C::kTmemCols);
  if (threadIdx.x == 0) {
    finish_claims();
    if (cta_clock != nullptr) record_cta_clock(cta_clock, t_start);
  }
}

template <int kNq>
int launch_i4(const void* q, const void* kv_cache, int32_t num_blocks, const int32_t* block_table,
              int32_t max_blocks, const int32_t* seq_lens, int32_t batch, const hpc_attn_options& opts,
              const hpc_plan* plan, float* partial_o, float* partial_lse, float sm_scale, int32_t* status,
              unsigned long long* cta_clock, void* out, cudaStream_t stream) {
  using C = I4Cfg<kNq>;
  // once per device: the dynamic shared memory opt-in is a per-device setting
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return HPC_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      if (cudaFuncSetAttribute(decode_attn_i4_kernel<kNq>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::kSmemBytes) != cudaSuccess)
        return HPC_ERR_CUDA;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan->num_ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // Always a programmatic dependent: the kernel touches nothing global before
  // its wait for the previous kernel, whatever that is (the planner lets it
  // start at once: barriers and tensor memory are set up meanwhile).
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, decode_attn_i4_kernel<kNq>, static_cast<const uint8_t*>(kv_cache),
      static_cast<const uint16_t*>(q), block_table, max_blocks, num_blocks, seq_lens, batch, opts.q_len,
      static_cast<const hpc_work_item*>(plan->items), static_cast<const int32_t*>(plan->cta_ptr),
      static_cast<const int32_t*>(plan->home_end), plan->pool, plan->capacity, partial_o, partial_lse,
      sm_scale, status, cta_clock, static_cast<const int32_t*>(plan->seg_ptr), plan->seg_done, out,
      opts.out_dtype);
  return e == cudaSuccess ? HPC_OK : HPC_ERR_CUDA;
}

}  // namespace
}  // namespace hpc

int hpc::launch_decode_attn_i4(HPC_LAYOUT_LAUNCH_ARGS) {
  (void)kv_dtype;
  (void)kv_scale;
  (void)pdl;   // (it always is one)
  auto run = [&](auto launch) {
    return launch(q, kv_cache, num_blocks, block_table, max_blocks, seq_lens, batch, opts, plan, partial_o,
                  partial_lse, sm_scale, status, cta_clock, out, stream);
  };
  return opts.q_len == 1 ? run(hpc::launch_i4<1>) : opts.q_len == 2 ? run(hpc::launch_i4<2>) : run(hpc::launch_i4<4>);
}
