// Rows of the paged cache read back as values: the inverse of the prologue's
// K/V write, for every cache type (a row's transfer to another cache or to
// the host, and checks of what later steps read).
//
// One warp per (token, KV head), its halves K and V, a lane per 8 elements:
// 16-byte stores of a 16-bit output.  A block takes kGatherTokens tokens, all
// loads of a warp's rows before its stores.  Bound by the bytes written, once
// there are enough of them (8191 tokens to bf16: 11 us, 3.9 TB/s in and out).
#include "int4.cuh"

namespace hpc {
namespace {

constexpr int kGatherTokens = 4;

// Eight consecutive output elements (index a multiple of 8).
__device__ __forceinline__ void store_out8(void* out, int64_t idx, const float (&x)[8], int32_t out_dtype) {
  if (out_dtype == HPC_OUT_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + idx);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = out_dtype == HPC_OUT_FP16 ? pack_f16(x[2 * e], x[2 * e + 1]) : pack_bf16(x[2 * e], x[2 * e + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + idx) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int kKv>
__global__ void __launch_bounds__(32 * kHkv) kv_gather_kernel(
    const uint8_t* __restrict__ kv_cache, const float* __restrict__ kv_scale, int32_t num_blocks,
    const int64_t* __restrict__ slots, int32_t num_slots, int32_t per_block, void* __restrict__ k_out,
    void* __restrict__ v_out, int32_t out_dtype, int32_t* __restrict__ status) {
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv = lane >> 4, d = 8 * (lane & 15);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per_block;
  uint4 raw[kGatherTokens];   // the row's stored elements (E4M3: .x, .y; 4-bit: .x)
  float scale[kGatherTokens];
  bool have[kGatherTokens];
#pragma unroll
  for (int i = 0; i < kGatherTokens; ++i) {
    have[i] = false;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    if (i >= per_block || first + i >= num_slots) continue;
    const int64_t slot = slots[first + i];
    if (slot >= static_cast<int64_t>(num_blocks) * kPage) {
      if (threadIdx.x == 0) atomicOr(status, HPC_STATUS_BAD_SLOT);
      continue;
    }
    if (slot < 0) continue;
    have[i] = true;
    const int64_t blk = slot / kPage;
    const int t = static_cast<int>(slot % kPage);
    if constexpr (kKv == HPC_KV_INT4) {
      const uint8_t* rec = kv_cache + (blk * kHkv + h) * kI4Record;
      const int g = d / kI4Group;
      if (kv == 0)
        raw[i].x = *reinterpret_cast<const uint32_t*>(rec + i4_k_byte(t, d));
      else
        raw[i].x = *reinterpret_cast<const uint16_t*>(rec + i4_v_byte(t, d)) |
                   (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(rec + i4_v_byte(t, d + 4))) << 16);
      scale[i] = __bfloat162float(
          *reinterpret_cast<const __nv_bfloat16*>(rec + (kv == 0 ? i4_ks_byte(t, g) : i4_vs_byte(t, g))));
    } else {
      const int64_t row = ((blk * 2 + kv) * kHkv + h) * kPage + t;
      if constexpr (kKv == HPC_KV_BF16) {
        raw[i] = *reinterpret_cast<const uint4*>(kv_cache + (row * kD + d) * 2);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(kv_cache + row * kD + d);
        raw[i].x = w.x;
        raw[i].y = w.y;
        scale[i] = kv_scale[kv];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kGatherTokens; ++i) {
    if (i >= per_block || first + i >= num_slots) continue;
    float x[8];
    if constexpr (kKv == HPC_KV_BF16) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * e] = bf16_lo(w[e]), x[2 * e + 1] = bf16_hi(w[e]);
    } else if constexpr (kKv == HPC_KV_FP8_E4M3) {
      const uint32_t w[2] = {raw[i].x, raw[i].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t f16 = e4m3x2_to_f16x2(static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16));
        x[2 * e] = f.x * scale[i];
        x[2 * e + 1] = f.y * scale[i];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = have[i] ? i4_value(raw[i].x, e, scale[i]) : 0.f;
    }
    store_out8(kv == 0 ? k_out : v_out, ((first + i) * kHkv + h) * kD + d, x, out_dtype);
  }
}

}  // namespace
}  // namespace hpc

extern "C" int hpc_kv_gather(const void* kv_cache, int32_t kv_dtype, const float* kv_scale,
                             int32_t num_blocks, const int64_t* slots, int32_t num_slots, void* k_out,
                             void* v_out, int32_t out_dtype, int32_t* status, cudaStream_t stream) {
  HPC_CHECK_ARG(num_blocks > 0 && num_slots >= 0);
  HPC_CHECK_ARG(kv_cache && status && (num_slots == 0 || (slots && k_out && v_out)));
  if (kv_dtype != HPC_KV_BF16 && kv_dtype != HPC_KV_FP8_E4M3 && kv_dtype != HPC_KV_INT4)
    return HPC_ERR_UNSUPPORTED;
  if (out_dtype != HPC_OUT_BF16 && out_dtype != HPC_OUT_FP16 && out_dtype != HPC_OUT_FP32)
    return HPC_ERR_UNSUPPORTED;
  HPC_CHECK_ARG(kv_dtype != HPC_KV_FP8_E4M3 || kv_scale != nullptr);
  HPC_CHECK_ARG((reinterpret_cast<uintptr_t>(kv_cache) & 15) == 0 &&
                (reinterpret_cast<uintptr_t>(k_out) & 15) == 0 &&
                (reinterpret_cast<uintptr_t>(v_out) & 15) == 0);
  if (num_slots == 0) return HPC_OK;
  // few tokens: a block each, so that they spread over the SMs
  const int per_block = num_slots <= 512 ? 1 : hpc::kGatherTokens;
  auto launch = [&](auto kernel) {
    kernel<<<(num_slots - 1) / per_block + 1, 32 * hpc::kHkv, 0, stream>>>(
        static_cast<const uint8_t*>(kv_cache), kv_scale, num_blocks, slots, num_slots, per_block, k_out,
        v_out, out_dtype, status);
  };
  if (kv_dtype == HPC_KV_BF16) launch(hpc::kv_gather_kernel<HPC_KV_BF16>);
  else if (kv_dtype == HPC_KV_FP8_E4M3) launch(hpc::kv_gather_kernel<HPC_KV_FP8_E4M3>);
  else launch(hpc::kv_gather_kernel<HPC_KV_INT4>);
  return HPC_LAUNCH_STATUS();
}
