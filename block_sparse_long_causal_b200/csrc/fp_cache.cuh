// fp_cache.cuh -- what the key/value cache kernels share: the launch description of a cache, page
// look-up and the per-launch tables that turn a work index into (sequence, unit).
#pragma once
#include "fp_cache.h"
#include "fp_dev.cuh"
#include "fp_seq.cuh"

namespace fp {

// Programmatic dependent launch: a kernel that was launched with launch_pdl may start while the one before
// it on the stream still runs; pdl_wait returns once that one has ended and its writes are visible.
// pdl_trigger, in the earlier kernel, allows the start (at its end without it).
// So nothing here reads through ld.global.nc (__ldg), which is for data that no one writes while the kernel runs: a
// line that the SM holds from the kernel before would do for it. Plain loads see what pdl_wait waited for.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... K, typename... A>
cudaError_t launch_pdl(void (*kernel)(K...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// 3-D tiled load global -> shared (Q as tokens x heads x columns); tma_load_2d's rules.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// u / page_size by a multiplication (a division by a run-time number is some twenty instructions).
__device__ __forceinline__ int page_of(const CacheInfo& c, int u) {
  return (int)(__umulhi((unsigned)u, c.page_mul) >> c.page_shift);
}
// Row of the cache that holds slot u of sequence s, or -1 when the block table points outside the
// cache (callers flag FP_DEV_BAD_PROBLEM and treat the slot as not there). u < max_pages * page_size
// is the caller's duty (n <= max_len is checked before any slot is used).
__device__ __forceinline__ long long slot_row(const CacheInfo& c, int s, int u) {
  const int lp = page_of(c, u);
  const int page = c.block_table[(long long)s * c.max_pages + lp];
  if (page < 0 || page >= c.num_pages) return -1;
  return (long long)page * c.page_size + (u - lp * c.page_size);
}
// Index of (slot, kv-head) in the weights and positions arrays [num_pages, Hkv, page_size], or -1.
__device__ __forceinline__ long long slot_word(const CacheInfo& c, int s, int g, int u) {
  const int lp = page_of(c, u);
  const int page = c.block_table[(long long)s * c.max_pages + lp];
  if (page < 0 || page >= c.num_pages) return -1;
  return ((long long)page * c.hkv + g) * c.page_size + (u - lp * c.page_size);
}

// Exclusive prefix table over sequences: tab[s] = sum_{s' < s} count(s', L, n), tab[S] = the total.
// L: new tokens of the sequence, n = lens + L: its keys. Called by every thread of a block of
// kThreads threads; returns false (and flags FP_DEV_BAD_PROBLEM) when the device arrays disagree with
// the host's description, so that no later access can leave a buffer.
template <int kThreads, typename Count>
__device__ __forceinline__ bool cache_table(const CacheInfo& c, long long* tab, long long* s_warp, int* s_bad,
                                            int32_t* dev_status, Count count) {
  const int S = c.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (S + kThreads - 1) / kThreads;
  const int a = min(S, tid * per), b = min(S, a + per);
  if (tid == 0) *s_bad = 0;
  __syncthreads();
  long long sum = 0;
  bool bad = tid == 0 && (c.cu_seqlens[0] != 0 || c.cu_seqlens[S] != c.total_tokens);
  for (int s = a; s < b; ++s) {
    const int lo = c.cu_seqlens[s], hi = c.cu_seqlens[s + 1], len = c.lens[s];
    const bool ok = lo >= 0 && hi >= lo && hi <= c.total_tokens && len >= 0 && len <= c.max_len - (hi - lo);
    bad |= !ok;
    tab[s] = sum;
    if (ok) sum += count(s, hi - lo, len + hi - lo);
  }
  const long long incl = warp_incl_scan(sum);
  if (lane == 31) s_warp[warp] = incl;
  if (bad) *s_bad = 1;
  __syncthreads();
  long long base = incl - sum, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += s_warp[w];
    total += s_warp[w];
  }
  for (int s = a; s < b; ++s) tab[s] += base;
  if (tid == 0) tab[S] = total;
  __syncthreads();
  const bool ok = *s_bad == 0;
  if (!ok && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) dev_flag(dev_status, kDevBadProblem);
  return ok;
}

// A line of `total` tiles in equal shares, [at(i), at(i + 1)) for i < parts (at most `most`, and every one
// has a tile): the first `rem` shares are one tile longer.
struct Shares {
  long long q = 0;
  int rem = 0, parts = 0;
  Shares() = default;
  __device__ __forceinline__ Shares(long long total, int most) {
    parts = (int)min((long long)most, total);
    if (parts == 0) return;
    if (total < 0x7fffffffll) {  // the 32-bit division is several times shorter
      q = (unsigned)total / (unsigned)parts;
      rem = (int)((unsigned)total % (unsigned)parts);
    } else {
      q = total / parts;
      rem = (int)(total % parts);
    }
  }
  __device__ __forceinline__ long long at(int i) const { return i * q + min(i, rem); }
};

__device__ __forceinline__ bool nonfinite2(uint32_t x) {  // either of two bf16
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

// Largest s in [0, S) with tab[s] <= x < tab[s + 1] (sequences without work are passed over).
__device__ __forceinline__ int find_seq64(const long long* tab, int S, long long x) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace fp
