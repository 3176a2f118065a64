// Block tables and slot maps of a step, built on the device from the request
// lengths, and the return of pages to the pool.
//
// With h_b tokens of sequence b in the cache, n_b new ones, P = 64:
//   start_b = sum_{b' < b} n_b'                     packed position of b's first new token
//   need_b  = ceil((h_b + n_b) / P) - ceil(h_b / P)  pages it takes from the pool
//   before_b = sum_{b' < b} need_b'
// The pool is a stack: the k-th page taken in a call, in (sequence, page)
// order, is the k-th from its top, so the result does not depend on which
// thread comes first.  A fresh page holds exactly one new token at its first
// slot (it begins at or after h_b, and is taken for a new token), so the
// thread of that token writes the page's table entry and there is no pass
// over pages.  Tokens read table entries of old pages only, which the call
// does not write.
//
// The sizes are small (12 bytes per token, 20 per sequence): latency counts.
// One launch: every block makes both prefix sums over the whole batch for
// itself (at most 8192 lengths, through L2) and keeps them in shared memory,
// then takes its share of the packed tokens, each finding its sequence by
// bisection.  The last block to have read the pool's size writes the new one.
// A decode step of 256 sequences 8 us (64 threads go through four chains of
// dependent loads each), 1000 prompts of 300 tokens in a padded batch of 196608 rows
// 6 us; the release 2 and 4 us.
#include <mutex>

#include "common.cuh"
#include "plan_body.cuh"

namespace hpc {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabPer = 4;      // consecutive tokens per thread and step
constexpr int kTabBlockTokens = kTabThreads * kTabPer;

// Exclusive scan over the CTA of one 64-bit value per thread; *total the sum.
__device__ int64_t tab_scan64(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < kTabThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int64_t excl = x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
  *total = warp_sums[31];
  __syncthreads();
  return excl;
}

__device__ __forceinline__ int pages_for(int tokens) { return (tokens + kPage - 1) / kPage; }

// The last entry b of the nondecreasing starts[0 .. n-1] with starts[b] <= i
// (the one that holds i, as empty ranges start where the next one does).
__device__ __forceinline__ int tab_find(const int32_t* starts, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// pool[1] counts the blocks that have read the pool; the last one stores the
// new size and sets the count back.
__device__ __forceinline__ void tab_finish(int32_t* pool, int new_size) {
  __syncthreads();
  if (threadIdx.x == 0 && atomic_add_acq_rel_gpu(&pool[1], 1) == static_cast<int>(gridDim.x) - 1) {
    pool[0] = new_size;
    pool[1] = 0;
  }
}

__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(
    const int32_t* __restrict__ hist_lens, const int32_t* __restrict__ new_lens, int32_t batch,
    int32_t num_blocks, const int32_t* __restrict__ free_blocks, int32_t* pool,
    int32_t* block_table, int32_t max_blocks, int32_t* __restrict__ seq_lens,
    int32_t* __restrict__ query_start, int32_t* __restrict__ positions,
    int64_t* __restrict__ slot_mapping, int32_t max_tokens, int32_t* __restrict__ status) {
  extern __shared__ int32_t tab_smem[];
  int32_t* start = tab_smem;              // [batch] packed start of b
  int32_t* before = start + batch;        // [batch] pages taken before b, or -1: b sits out
  __shared__ int64_t sums64[32];
  __shared__ int sums32[32];
  __shared__ int taken_s;
  const int free_count = max(0, min(pool[0], num_blocks));
  const int per = (batch + kTabThreads - 1) / kTabThreads;
  const int b0 = min(batch, static_cast<int>(threadIdx.x) * per), b1 = min(batch, b0 + per);
  const bool first = blockIdx.x == 0;
  const int64_t limit = static_cast<int64_t>(max_blocks) * kPage;
  if (threadIdx.x == 0) taken_s = 0;

  int64_t local = 0;
  for (int b = b0; b < b1; ++b) local += max(new_lens[b], 0);
  int64_t total;
  int64_t run = tab_scan64(local, sums64, &total);
  // a sequence sits the step out when its lengths are bad or its tokens pass max_tokens
  auto fits = [&](int h, int n, int64_t at) {
    return h >= 0 && n >= 0 && static_cast<int64_t>(h) + n <= limit && at + n <= max_tokens;
  };
  int need = 0;
  const int64_t run0 = run;
  for (int b = b0; b < b1; ++b) {
    const int h = hist_lens[b], n = new_lens[b];
    if (fits(h, n, run)) need += pages_for(h + n) - pages_for(h);
    run += max(n, 0);
  }
  int pages;
  int page = cta_exclusive_scan<kTabThreads>(need, sums32, &pages);
  run = run0;
  for (int b = b0; b < b1; ++b) {
    const int h = hist_lens[b], n = new_lens[b];
    const bool ok = fits(h, n, run);
    const int want = ok ? pages_for(h + n) - pages_for(h) : 0;
    const bool served = ok && (want == 0 || page + want <= free_count);
    start[b] = static_cast<int32_t>(min(run, static_cast<int64_t>(INT32_MAX)));
    before[b] = served ? page : -1;
    if (served && want > 0) atomicMax(&taken_s, page + want);
    if (first) {
      seq_lens[b] = served ? h + n : 0;
      query_start[b] = start[b];
      if (!served) {
        const bool bad = h < 0 || n < 0 || static_cast<int64_t>(h) + n > limit;
        atomicOr(status, bad ? HPC_STATUS_BAD_SEQ_LEN
                             : ok ? HPC_STATUS_OUT_OF_BLOCKS : HPC_STATUS_PLAN_OVERFLOW);
      }
    }
    page += want;
    run += max(n, 0);
  }
  if (first && threadIdx.x == 0)
    query_start[batch] = static_cast<int32_t>(min(total, static_cast<int64_t>(INT32_MAX)));
  __syncthreads();

  const int live = static_cast<int>(min(total, static_cast<int64_t>(max_tokens)));
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kTabBlockTokens; base < max_tokens;
       base += static_cast<int64_t>(gridDim.x) * kTabBlockTokens) {
    const int64_t i0 = base + static_cast<int64_t>(threadIdx.x) * kTabPer;
    int b = i0 < live ? tab_find(start, batch, static_cast<int>(i0)) : batch;
#pragma unroll
    for (int k = 0; k < kTabPer; ++k) {
      const int64_t i = i0 + k;
      if (i >= max_tokens) break;
      int pos = 0;
      int64_t slot = -1;
      if (i < live) {
        while (b + 1 < batch && start[b + 1] <= i) ++b;
        const int h = hist_lens[b];
        pos = max(h, 0) + static_cast<int>(i - start[b]);
        if (before[b] >= 0) {
          const int j = pos / kPage, old = pages_for(h);
          const int64_t entry = static_cast<int64_t>(b) * max_blocks + j;
          const int id = j >= old ? free_blocks[free_count - 1 - (before[b] + j - old)] : block_table[entry];
          if (j >= old && pos % kPage == 0) block_table[entry] = id;
          if (id >= 0 && id < num_blocks) slot = static_cast<int64_t>(id) * kPage + pos % kPage;
          else atomicOr(status, HPC_STATUS_BAD_BLOCK);
        } else {
          pos = 0;
        }
      }
      positions[i] = pos;
      slot_mapping[i] = slot;
    }
  }
  tab_finish(pool, free_count - taken_s);
}

__global__ void __launch_bounds__(kTabThreads) block_release_kernel(
    const int32_t* __restrict__ lens, const int32_t* __restrict__ keep_lens, int32_t batch,
    const int32_t* __restrict__ block_table, int32_t max_blocks, int32_t num_blocks,
    int32_t* __restrict__ free_blocks, int32_t* pool, int32_t* __restrict__ status) {
  extern __shared__ int32_t tab_smem[];
  int32_t* before = tab_smem;   // [batch] pages given back before b's
  __shared__ int sums32[32];
  const int free_count = max(0, min(pool[0], num_blocks));
  const int per = (batch + kTabThreads - 1) / kTabThreads;
  const int b0 = min(batch, static_cast<int>(threadIdx.x) * per), b1 = min(batch, b0 + per);
  const int64_t limit = static_cast<int64_t>(max_blocks) * kPage;
  auto count = [&](int b) {
    const int n = lens[b], k = keep_lens[b];
    return n >= 0 && n <= limit && k >= 0 && k <= n ? pages_for(n) - pages_for(k) : -1;
  };
  int local = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = count(b);
    if (n < 0 && blockIdx.x == 0) atomicOr(status, HPC_STATUS_BAD_SEQ_LEN);
    local += max(n, 0);
  }
  int total;
  int run = cta_exclusive_scan<kTabThreads>(local, sums32, &total);
  for (int b = b0; b < b1; ++b) {
    before[b] = run;
    run += max(count(b), 0);
  }
  __syncthreads();
  const bool fits = free_count + static_cast<int64_t>(total) <= num_blocks;
  if (fits) {
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kTabThreads + threadIdx.x; k < total;
         k += static_cast<int64_t>(gridDim.x) * kTabThreads) {
      const int b = tab_find(before, batch, static_cast<int>(k));
      const int j = pages_for(keep_lens[b]) + static_cast<int>(k - before[b]);
      const int id = block_table[static_cast<int64_t>(b) * max_blocks + j];
      if (id < 0 || id >= num_blocks) atomicOr(status, HPC_STATUS_BAD_BLOCK);
      free_blocks[free_count + total - 1 - k] = id;
    }
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    atomicOr(status, HPC_STATUS_PLAN_OVERFLOW);
  }
  tab_finish(pool, fits ? free_count + total : free_count);
}

// The two prefix sums of a large batch pass 48 KB; opted in once per device.
cudaError_t tab_smem_optin() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(2 * sizeof(int32_t) * HPC_MAX_BATCH));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

// Blocks for `items` pieces of work, `per_block` each: at most one per SM.
int tab_grid(int64_t items, int64_t per_block, int* grid) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return HPC_ERR_CUDA;
  const int64_t want = (items + per_block - 1) / per_block;
  *grid = static_cast<int>(want < 1 ? 1 : want > sms ? sms : want);
  return HPC_OK;
}

}  // namespace
}  // namespace hpc

extern "C" int hpc_block_tables(const int32_t* hist_lens, const int32_t* new_lens, int32_t batch,
                                int32_t num_blocks, const int32_t* free_blocks, int32_t* pool,
                                int32_t* block_table, int32_t max_blocks, int32_t* seq_lens,
                                int32_t* query_start, int32_t* positions, int64_t* slot_mapping,
                                int32_t max_tokens, int32_t* status, cudaStream_t stream) {
  HPC_CHECK_ARG(batch >= 0 && num_blocks > 0 && max_blocks >= 1 && max_tokens >= 0);
  HPC_CHECK_ARG(free_blocks && pool && query_start && status);
  HPC_CHECK_ARG(batch == 0 || (hist_lens && new_lens && block_table && seq_lens && seq_lens != hist_lens &&
                               seq_lens != new_lens));
  HPC_CHECK_ARG(max_tokens == 0 || (positions && slot_mapping));
  if (batch > HPC_MAX_BATCH || num_blocks > HPC_MAX_NUM_BLOCKS) return HPC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * max_blocks >= (int64_t{1} << 31) ||
      static_cast<int64_t>(max_blocks) * hpc::kPage >= (int64_t{1} << 31))
    return HPC_ERR_UNSUPPORTED;
  int grid = 1;
  const int rc = hpc::tab_grid(max_tokens, hpc::kTabBlockTokens, &grid);
  if (rc != HPC_OK) return rc;
  const size_t smem = 2 * sizeof(int32_t) * batch;
  if (smem > 32 * 1024 && hpc::tab_smem_optin() != cudaSuccess)
    return HPC_ERR_CUDA;
  hpc::block_tables_kernel<<<grid, hpc::kTabThreads, smem, stream>>>(
      hist_lens, new_lens, batch, num_blocks, free_blocks, pool, block_table, max_blocks, seq_lens,
      query_start, positions, slot_mapping, max_tokens, status);
  return HPC_LAUNCH_STATUS();
}

extern "C" int hpc_block_release(const int32_t* lens, const int32_t* keep_lens, int32_t batch,
                                 const int32_t* block_table, int32_t max_blocks, int32_t num_blocks,
                                 int32_t* free_blocks, int32_t* pool, int32_t* status,
                                 cudaStream_t stream) {
  HPC_CHECK_ARG(batch >= 0 && num_blocks > 0 && max_blocks >= 1);
  HPC_CHECK_ARG(free_blocks && pool && status && (batch == 0 || (lens && keep_lens && block_table)));
  if (batch > HPC_MAX_BATCH || num_blocks > HPC_MAX_NUM_BLOCKS) return HPC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * max_blocks >= (int64_t{1} << 31) ||
      static_cast<int64_t>(max_blocks) * hpc::kPage >= (int64_t{1} << 31))
    return HPC_ERR_UNSUPPORTED;
  if (batch == 0) return HPC_OK;
  int grid = 1;
  const int64_t most = static_cast<int64_t>(batch) * max_blocks;   // pages that could come back
  const int rc = hpc::tab_grid(most < num_blocks ? most : num_blocks, 4 * hpc::kTabThreads, &grid);
  if (rc != HPC_OK) return rc;
  const size_t smem = sizeof(int32_t) * batch;
  hpc::block_release_kernel<<<grid, hpc::kTabThreads, smem, stream>>>(
      lens, keep_lens, batch, block_table, max_blocks, num_blocks, free_blocks, pool, status);
  return HPC_LAUNCH_STATUS();
}
