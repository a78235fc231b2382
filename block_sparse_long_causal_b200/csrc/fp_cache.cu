// fp_cache.cu -- writing to a paged key/value cache and keeping it within a budget: append, selection
// of the slots that stay by collected attention weight, compaction.
#include <cooperative_groups.h>

#include <mutex>
#include <type_traits>

#include "fp_cache.cuh"

namespace cg = cooperative_groups;

namespace fp {

constexpr unsigned kFullMask = 0xffffffffu;

// ------------------------------------------------------------------------ append ---------------
// One warp per new token: it finds its sequence (the number of s with cu_seqlens[s] <= t, counted 32 at
// a time, so that the look-up waits on one round trip and not on a chain), then copies the token's K
// and V rows in 16-byte pieces and sets weight 0 and the position of its slot in every kv-head. Bound by the
// copy: 39 thousand tokens of 8 kv-heads (318 MB moved) take 51.5 us, 6.2 TB/s; 64 single tokens 3.1 us.
constexpr int kAppend = 4;  // 16-byte pieces of K and of V that a lane has in flight
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const CacheInfo& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= c.total_tokens) return;
  int s = -1;
  for (int b = 0; b < c.num_seqs; b += 32) {
    const int x = b + lane;
    s += __popc(__ballot_sync(kFullMask, x < c.num_seqs && c.cu_seqlens[x] <= t));
  }
  bool ok = s >= 0;
  int u = 0;
  long long row = -1;
  if (ok) {
    const int lo = c.cu_seqlens[s], hi = c.cu_seqlens[s + 1], len = c.lens[s];
    ok = lo >= 0 && t >= lo && t < hi && len >= 0 && len <= c.max_len - (hi - lo);
    u = len + (int)(t - lo);
    if (ok) row = slot_row(c, s, u);
  }
  if (row < 0) {
    if (lane == 0) dev_flag(p.dev_status, kDevBadProblem);
    return;
  }
  const int chunks = c.hkv * (kHeadDim / 8);
  const uint4* ks = reinterpret_cast<const uint4*>(p.k + t * p.k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(p.v + t * p.v_stride);
  uint4* kd = reinterpret_cast<uint4*>(c.k) + row * chunks;
  uint4* vd = reinterpret_cast<uint4*>(c.v) + row * chunks;
  for (int i0 = lane; i0 < chunks; i0 += 32 * kAppend) {  // eight kv-heads at once, all their reads in flight
    uint4 x[kAppend], y[kAppend];
#pragma unroll
    for (int j = 0; j < kAppend; ++j)
      if (i0 + 32 * j < chunks) {
        x[j] = ks[i0 + 32 * j];
        y[j] = vs[i0 + 32 * j];
      }
#pragma unroll
    for (int j = 0; j < kAppend; ++j)
      if (i0 + 32 * j < chunks) {
        kd[i0 + 32 * j] = x[j];
        vd[i0 + 32 * j] = y[j];
      }
  }
  if (c.weights || c.positions) {
    const long long page = page_of(c, (int)row), off = row - page * c.page_size;  // a cache has less than 2^31 rows
    const int pos = (p.next_pos ? p.next_pos[s] : c.lens[s]) + (u - c.lens[s]);
    for (int g = lane; g < c.hkv; g += 32) {
      const long long w = (page * c.hkv + g) * c.page_size + off;
      if (c.weights) c.weights[w] = 0.f;
      if (c.positions) c.positions[w] = pos;
    }
  }
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
  return launch_pdl(append_kernel, dim3((p.c.total_tokens + 7) / 8), 256, 0, st, p);
}

// ------------------------------------------------------------------------ selection -------------
// Order-preserving 32-bit key of a weight (larger key = larger weight); -0 counts as 0, NaN ranks
// below everything, a protected slot above everything.
__device__ __forceinline__ uint32_t rank_key(float w, bool safe) {
  if (safe) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelCluster = 16;      // largest cluster
constexpr int kSelSpan = 8192;       // slots a CTA is meant to take (16 a thread)
// Keys that a CTA keeps in shared memory: with 36 KB of other arrays 226 KB where an SM holds one CTA, 112 KB where
// it holds two
constexpr int kSelKeys1 = 48640, kSelKeys2 = 19456;
constexpr int kSelBins = 2048;
constexpr int kSelCand = 6144;       // keys of the first digit's class that a CTA may list (24 KB)
static_assert(kSelBins == 4 * kSelThreads, "a thread sums four bins");

// One cluster per (sequence, kv-head); each of its CTAs takes a contiguous range of the slots, a
// contiguous part of it per warp. The slots are read once: their keys stay in shared memory (a range
// that they do not fit is read again in every pass). The key of rank `budget` is found by a radix select,
// three passes of 11, 11 and 10 bits over the keys that match the prefix so far; a CTA adds its
// occupied bins (few: weights cluster) to every CTA's sums through distributed shared memory, one cluster
// barrier a pass. After the first digit its class is usually small (a few percent): every CTA lists its
// keys of it, and the other passes run in each CTA over all lists, without a barrier across the cluster
// (128K slots and 8 heads: 43.6 -> 35.8 us). Then every warp counts its slots above and at the threshold, and
// after a scan over the cluster's warps writes its holes (evicted slots below the budget) and sources (kept
// slots at or past it) in ascending order.
// Bound by latency, not by its 8 bytes a slot: of 15 us for 16 sequences of 4.1K slots 4 go to the reads, 2 to 3
// to each pass, 2 to the list. The loops keep several slots a lane in flight. Clusters of 8 CTAs take 39 us for 128K
// slots of 8 heads where 16 take 36. Every write is bounded by itself: the passes over a range that is read again would
// disagree if another stream changed the weights meanwhile.
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const __grid_constant__ SelectParams p, const int keys_cap) {
  extern __shared__ uint32_t s_keys[];
  // the list is written once every CTA has added to the first pass's sums and this one has read them; from then on
  // no sums of the cluster are formed
  __shared__ __align__(16) union {
    unsigned sum[2][kSelBins];
    uint32_t list[kSelCand];
  } s_u;
  __shared__ __align__(16) unsigned s_hist[kSelBins];
  __shared__ unsigned s_tot[kSelWarps], s_pick[3], s_listed;
  __shared__ int4 s_cnt[kSelWarps];                // slots above / at the threshold, below / past the budget
  __shared__ int s_eq[kSelCluster * kSelWarps + 1], s_hole[kSelCluster * kSelWarps + 1], s_from[kSelCluster * kSelWarps + 1];
  __shared__ int s_part[3][8];
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
  const CacheInfo& c = p.c;
  const int sg = blockIdx.x / C, s = sg / c.hkv, g = sg % c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int lo = c.cu_seqlens[s], hi = c.cu_seqlens[s + 1], len = c.lens[s], L = hi - lo;
  int32_t* moves = p.moves + (long long)sg * p.budget * 2;
  auto fill = [&] {
    for (int i = rank * kSelThreads + tid; i < p.budget; i += C * kSelThreads)
      reinterpret_cast<int2*>(moves)[i] = make_int2(-1, -1);
  };
  const bool bad_seq = L < 0 || len < 0 || len > c.max_len - L;
  const int n = bad_seq ? 0 : len + L;
  if (tid == 0 && rank == 0) {
    if (bad_seq) dev_flag(p.dev_status, kDevBadProblem);
    if (g == 0) p.new_lens[s] = bad_seq ? len : min(n, p.budget);
  }
  if (n <= p.budget) {  // nothing to evict (or a sequence that is skipped: no moves, lens as it was)
    if (tid == 0 && rank == 0) p.move_counts[sg] = 0;
    fill();
    return;
  }
  // positions at or past `young` are protected (the difference cannot overflow: 64 bits)
  const long long young = (long long)(p.next_pos ? p.next_pos[s] : len) + L - p.recent;
  bool bad_page = false;
  const bool with_pos = c.positions != nullptr;  // (a branch in front of every read took 0.3 us)
  const int32_t* positions = with_pos ? c.positions : reinterpret_cast<const int32_t*>(c.weights);
  const int32_t* table = c.block_table + (long long)s * c.max_pages;
  // keys of slots u, u + 32, ... (K of them; past the last slot: anything), all their reads in flight together
  auto read_keys = [&](int u, uint32_t* out, auto count) {
    constexpr int K = decltype(count)::value;
    int page[K], pos[K];
    float val[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
      page[i] = table[page_of(c, min(u + 32 * i, n - 1))];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int v = min(u + 32 * i, n - 1);
      const bool bad = page[i] < 0 || page[i] >= c.num_pages;
      const long long w = ((long long)(bad ? 0 : page[i]) * c.hkv + g) * c.page_size + (v - page_of(c, v) * c.page_size);
      val[i] = c.weights[w];
      pos[i] = positions[w];  // (the weights where the cache has no positions)
      page[i] = bad;
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      bad_page |= page[i] != 0;
      const int at = with_pos ? pos[i] : u + 32 * i;
      out[i] = page[i] ? 0u : rank_key(val[i], at < p.sinks || at >= young);
    }
  };
  const int wspan = (int)((((long long)n + C * kSelWarps - 1) / (C * kSelWarps) + 31) & ~31ll);  // slots a warp
  const long long first = (long long)rank * kSelWarps * wspan;
  const int base = (int)min((long long)n, first);
  const int u0 = (int)min((long long)n, first + warp * wspan), u1 = min(n, u0 + wspan);
  const bool kept = kSelWarps * wspan <= keys_cap;
  *reinterpret_cast<uint4*>(&s_hist[4 * tid]) = make_uint4(0, 0, 0, 0);
  *reinterpret_cast<uint4*>(&s_u.sum[0][4 * tid]) = make_uint4(0, 0, 0, 0);
  if (kept) {
    auto read_all = [&](auto count) {
      constexpr int K = decltype(count)::value;
      for (int u = u0 + lane; u < u1; u += 32 * K) {
        uint32_t k[K];
        read_keys(u, k, count);
        if (u == u0 + lane) fill();  // the moves' places, while the reads are under way
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (u + 32 * i < u1) s_keys[u + 32 * i - base] = k[i];
      }
    };
    // slots a lane reads at once: of four and five what leaves the fewer look-ups past the range's end (16 sequences of
    // 4.1K slots, 9 a lane: 15.9 and 15.3 us; of 0.3K, 1 a lane: 8.6 and 8.9; 128K slots of 8 heads, 16 a lane: 35.2 and
    // 36.0; eight or ten at once 9.2 to 9.7 for 0.3K)
    const int per = wspan / 32;
    if ((per + 3) / 4 * 4 < (per + 4) / 5 * 5) read_all(std::integral_constant<int, 4>());
    else read_all(std::integral_constant<int, 5>());
    __syncwarp();  // a warp reads back its own keys only
  }
  if (!kept || u0 + lane >= u1) fill();  // the lanes that had nothing to read
  // f(slot of lane 0, key) for the warp's slots, 32 at a time in ascending order; lanes past u1 get any key
  auto each = [&](auto f) {
    for (int u = u0; u < u1; u += 128) {
      uint32_t k[4];
      if (kept) {
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = s_keys[min(u + 32 * i + lane, u1 - 1) - base];
      } else {
        read_keys(u + lane, k, std::integral_constant<int, 4>());
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (u + 32 * i < u1) f(u + 32 * i, k[i]);
    }
  };
  auto sync_all = [&] {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };
  sync_all();  // every CTA's sums are zero before another adds to them
  bool listed = false;
  if (tid == 0) s_listed = s_pick[0] = s_pick[1] = s_pick[2] = 0;
  unsigned prefix = 0, need = (unsigned)p.budget;  // `need` keys of the current prefix class stay
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const unsigned mask = (1u << bits) - 1u;
    if (listed) {
      const int per = kSelThreads / C, r = tid / per;  // threads per list, and this thread's list
      const unsigned num = min(*cluster.map_shared_rank(&s_listed, r), (unsigned)kSelCand);
      const uint32_t* list = cluster.map_shared_rank(s_u.list, r);
#pragma unroll 4
      for (unsigned j = tid % per; j < num; j += per) {
        const uint32_t k = list[j];
        if (pass == 1 || ((k >> 10) & 2047u) == (prefix & 2047u)) atomicAdd(&s_hist[(k >> shift) & mask], 1u);
      }
    } else {
      each([&](int u, uint32_t k) {
        // the warp's most likely run of equal digits (protected slots, ties) is added once: that of its first lane
        // that matches
        const bool match = u + lane < u1 && (pass == 0 || (k >> (shift + bits)) == prefix);
        const unsigned dig = (k >> shift) & mask;
        int from = 0;
        if (pass > 0) {
          const unsigned act = __ballot_sync(kFullMask, match);
          if (act == 0) return;
          from = __ffs(act) - 1;
        }
        const unsigned lead = __shfl_sync(kFullMask, dig, from);
        const unsigned same = __ballot_sync(kFullMask, match && dig == lead);
        if (match && dig != lead) atomicAdd(&s_hist[dig], 1u);
        if (lane == 0) atomicAdd(&s_hist[lead], (unsigned)__popc(same));
      });
    }
    __syncthreads();
    // thread t owns bins 2047 - 4 t and the three below, so that an inclusive scan counts the larger digits
    const int bin = kSelBins - 4 - 4 * tid;
    uint4 cnt = *reinterpret_cast<const uint4*>(&s_hist[bin]);
    *reinterpret_cast<uint4*>(&s_hist[bin]) = make_uint4(0, 0, 0, 0);
    if (C > 1 && !listed) {
      unsigned* sums = s_u.sum[pass & 1];
      // the other buffer is zeroed for the next pass, which no CTA begins before the barrier below
      *reinterpret_cast<uint4*>(&s_u.sum[(pass + 1) & 1][bin]) = make_uint4(0, 0, 0, 0);
      if (cnt.x | cnt.y | cnt.z | cnt.w)
        for (int r = 0; r < C; ++r) {
          unsigned* dst = cluster.map_shared_rank(&sums[bin], r);
          if (cnt.x) atomicAdd(dst, cnt.x);
          if (cnt.y) atomicAdd(dst + 1, cnt.y);
          if (cnt.z) atomicAdd(dst + 2, cnt.z);
          if (cnt.w) atomicAdd(dst + 3, cnt.w);
        }
      cluster.sync();
      cnt = *reinterpret_cast<const uint4*>(&sums[bin]);
    }
    const unsigned sum = cnt.x + cnt.y + cnt.z + cnt.w;
    unsigned incl = warp_incl_scan(sum);
    if (lane == 31) s_tot[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) incl += w < warp ? s_tot[w] : 0u;
    unsigned above = incl - sum;  // keys of larger bins
    if (incl >= need && above < need) {
      int at = bin + 3;
      if (above + cnt.w < need) {
        above += cnt.w;
        --at;
        if (above + cnt.z < need) {
          above += cnt.z;
          --at;
          if (above + cnt.y < need) {
            above += cnt.y;
            --at;
          }
        }
      }
      s_pick[0] = (unsigned)at;
      s_pick[2] = at == bin + 3 ? cnt.w : at == bin + 2 ? cnt.z : at == bin + 1 ? cnt.y : cnt.x;
      s_pick[1] = need - above;
    }
    __syncthreads();
    prefix = (prefix << bits) | s_pick[0];
    need = s_pick[1];
    if (pass == 0 && s_pick[2] <= kSelCand) {
      listed = true;
      each([&](int u, uint32_t k) {
        const bool match = u + lane < u1 && (k >> 21) == prefix;
        const unsigned m = __ballot_sync(kFullMask, match);
        unsigned at = 0;
        if (lane == 0 && m) at = atomicAdd(&s_listed, (unsigned)__popc(m));
        at = __shfl_sync(kFullMask, at, 0);
        at += __popc(m & ((1u << lane) - 1u));
        if (match && at < kSelCand) s_u.list[at] = k;
      });
      sync_all();
    }
  }
  const uint32_t thr = prefix;  // keys above thr stay, and the first `need` slots whose key is thr
  int4 cnt = make_int4(0, 0, 0, 0);
  each([&](int u, uint32_t k) {
    const bool in = u + lane < u1;
    const unsigned mg = __ballot_sync(kFullMask, in && k > thr), me = __ballot_sync(kFullMask, in && k == thr);
    // the lanes below the budget: all, none, or a run from lane 0
    const unsigned below = u + 32 <= p.budget ? kFullMask : u >= p.budget ? 0u : (1u << (p.budget - u)) - 1u;
    cnt.x += __popc(mg & below);
    cnt.y += __popc(mg & ~below);
    cnt.z += __popc(me & below);
    cnt.w += __popc(me & ~below);
  });
  if (lane == 0) s_cnt[warp] = cnt;
  sync_all();
  // ---- scans over the cluster's warps in slot order: slots at the threshold before a warp, then its
  // holes and sources (the kept slots at the threshold are the first `need` of them)
  const int W = C * kSelWarps;
  int4 mine = make_int4(0, 0, 0, 0);
  if (tid < W) mine = *cluster.map_shared_rank(&s_cnt[tid % kSelWarps], tid / kSelWarps);
  int eq = mine.z + mine.w, eqi = eq;
  if (tid < 256) {
    eqi = warp_incl_scan(eq);
    if (lane == 31) s_part[0][warp] = eqi;
  }
  __syncthreads();
  int hole = 0, from = 0, hi_ = 0, fi = 0;
  if (tid < 256) {
    for (int w = 0; w < warp; ++w) eqi += s_part[0][w];
    if (tid < W) {
      const int room = max(0, (int)need - (eqi - eq));
      const int k0 = min(mine.z, room), k1 = min(mine.w, room - k0);
      const long long wa = (long long)tid * wspan;
      const int a = (int)min((long long)n, wa), b = (int)min((long long)n, wa + wspan);
      hole = min(b, p.budget) - min(a, p.budget) - mine.x - k0;
      from = mine.y + k1;
    }
    hi_ = warp_incl_scan(hole);
    fi = warp_incl_scan(from);
    if (lane == 31) {
      s_part[1][warp] = hi_;
      s_part[2][warp] = fi;
    }
  }
  __syncthreads();
  if (tid < 256) {
    for (int w = 0; w < warp; ++w) {
      hi_ += s_part[1][w];
      fi += s_part[2][w];
    }
    s_eq[tid] = eqi - eq;
    s_hole[tid] = hi_ - hole;
    s_from[tid] = fi - from;
    if (tid == 255) s_from[256] = fi;
  }
  __syncthreads();
  const int me_w = rank * kSelWarps + warp;
  int eq_before = s_eq[me_w];
  hole = s_hole[me_w];
  from = s_from[me_w];
  const int total = s_from[256];
  each([&](int u, uint32_t k) {
    const bool in = u + lane < u1;
    const unsigned me = __ballot_sync(kFullMask, in && k == thr);
    const unsigned lt = (1u << lane) - 1u;
    const bool keep = in && (k > thr || (k == thr && eq_before + __popc(me & lt) < (int)need));
    eq_before += __popc(me);
    const bool low = u + lane < p.budget;
    if (u < p.budget) {
      const unsigned mh = __ballot_sync(kFullMask, in && low && !keep);
      const int at = hole + __popc(mh & lt);
      if (in && low && !keep && at < p.budget) moves[2ll * at + 1] = u + lane;
      hole += __popc(mh);
    }
    if (u + 32 > p.budget) {
      const unsigned ms = __ballot_sync(kFullMask, keep && !low);
      const int at = from + __popc(ms & lt);
      if (keep && !low && at < p.budget) moves[2ll * at] = u + lane;
      from += __popc(ms);
    }
  });
  if (tid == 0 && rank == 0) p.move_counts[sg] = total;
  if (bad_page) dev_flag(p.dev_status, kDevBadProblem);
  if (C > 1) cluster.sync();  // no CTA ends while another still reads its counts
}

// Clusters of 1, 2, 4, 8 and 16 CTAs that the device holds at once, with kSelKeys1 and with kSelKeys2 keys a CTA.
struct SelFit {
  int n[5][2];
};
static cudaLaunchConfig_t select_config(cudaLaunchAttribute (&at)[2], int grid, int C, int keys, cudaStream_t st) {
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)keys * 4;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;  // the cluster; the launch adds the other
  return cfg;
}
// Asked once per device and context (the kernel's attributes are set with it).
static cudaError_t select_fit(SelFit& fit) {
  static std::mutex mu;
  static unsigned long long known[kMaxCachedDevices] = {};
  static SelFit fits[kMaxCachedDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const bool cached = dev >= 0 && dev < kMaxCachedDevices;
  unsigned long long id = cached ? context_id() : 0;
  if (id != 0 && known[dev] == id) {
    fit = fits[dev];
    return cudaSuccess;
  }
  const void* fn = reinterpret_cast<const void*>(select_kernel);
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys1 * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 5; ++i)
    for (int two = 0; two < 2; ++two) {
      cudaLaunchAttribute at[2];
      const cudaLaunchConfig_t cfg = select_config(at, 1 << i, 1 << i, two ? kSelKeys2 : kSelKeys1, nullptr);
      if (cudaOccupancyMaxActiveClusters(&fit.n[i][two], select_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();  // a size that this device does not take
        fit.n[i][two] = 0;
      }
    }
  id = cached ? context_id() : 0;  // the calls above made the context current
  if (id != 0) {
    fits[dev] = fit;
    known[dev] = id;
  }
  return cudaSuccess;
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  SelFit fit;
  cudaError_t e = select_fit(fit);
  if (e != cudaSuccess) return e;
  // The longest sequence that there may be (max_len) sets the CTAs of a cluster and their buffers: the lengths are on
  // the device. In this order:
  //  - the largest cluster that leaves about kSelSpan slots a CTA, whose ranges' keys fit and of which the device holds
  //    all at once: two CTAs an SM with up to kSelKeys2 keys each, one with up to kSelKeys1 (32 heads of 128K slots, 17K
  //    a CTA: 54 us by two CTAs an SM, 109 by one in three waves);
  //  - a CTA a head with up to kSelKeys1, in several waves (160 heads of 20K slots: 81 us; read again in every pass, by
  //    two CTAs an SM, 91);
  //  - two CTAs an SM, in the largest clusters that the device holds at once; what does not fit is read again in every
  //    pass. 8 heads of 500K slots: 143 us, kept by one CTA an SM in two waves 133; but 16 sequences of 4.1K slots that may
  //    grow to 128K: 18 us, in two waves 27.
  const long long pairs = (long long)p.c.num_seqs * p.c.hkv;
  auto span = [&](int C) { return (((long long)p.c.max_len + C * kSelWarps - 1) / (C * kSelWarps) + 31) / 32 * 32 * kSelWarps; };
  int top = 0;
  while (top < 4 && (long long)(1 << top) * kSelSpan < p.c.max_len) ++top;
  int size = -1;
  long long keys = 0;
  for (int i = top; i >= 0 && size < 0; --i) {
    const long long k = span(1 << i);
    if (k <= kSelKeys1 && pairs <= fit.n[i][k <= kSelKeys2]) {
      size = i;
      keys = k;
    }
  }
  if (size < 0 && span(1) <= kSelKeys1) {
    size = 0;
    keys = span(1);
  }
  if (size < 0) {
    for (size = top; size > 0 && pairs > fit.n[size][1];) --size;
    keys = kSelKeys2;
  }
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = select_config(at, (int)(pairs << size), 1 << size, (int)keys, st);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel, p, (int)keys);
}

// ------------------------------------------------------------------------ compaction ------------
// A CTA takes 64 moves at a time. Two warps look up their rows, a lane to a move, and move the weights and
// positions, so that neighbouring slots of a head go together; then every warp moves the K and V rows of eight
// of them with all its loads in flight, lanes 0..15 the K row and lanes 16..31 the V row, 16 bytes each. (Words
// moved by the eight lanes of each warp that looked them up: 33.3 instead of 27.0 us for a cut from 128K to 16K
// slots.) Sources lie at or past the budget and destinations below it (checked), so no move reads what another
// one writes and the order of the moves does not matter.
constexpr int kMovesW = 8, kMovesC = 8 * kMovesW;
__global__ void __launch_bounds__(256, 4) compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ longlong2 s_rows[2][kMovesC];  // source and destination rows; source -1: none
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sg = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int s = sg / c.hkv, g = sg % c.hkv;
  pdl_wait();
  pdl_trigger();
  const int cnt = p.move_counts[sg];
  const int slots = (int)min((long long)c.max_len, (long long)c.max_pages * c.page_size);
  if (part == 0 && tid == 0) {
    if (cnt < 0 || cnt > p.budget) dev_flag(p.dev_status, kDevBadList);
    if (g == 0) {
      const int nl = p.new_lens[s];
      if (nl >= 0 && nl <= slots) c.lens[s] = nl;
      else dev_flag(p.dev_status, kDevBadProblem);
    }
  }
  const int2* moves = reinterpret_cast<const int2*>(p.moves) + (long long)sg * p.budget;
  const int n = min(cnt, p.budget);
  auto look_up = [&](long long i, int buf) {  // moves i .. i + 63, by the first 64 threads
    longlong2 r = make_longlong2(-1, -1);
    if (i + tid < n) {
      const int2 mv = moves[i + tid];
      if (mv.x < p.budget || mv.x >= slots || mv.y < 0 || mv.y >= p.budget || mv.y >= slots) {
        dev_flag(p.dev_status, kDevBadList);
      } else {
        r = make_longlong2(slot_row(c, s, mv.x), slot_row(c, s, mv.y));
        if (r.x < 0 || r.y < 0) {
          dev_flag(p.dev_status, kDevBadProblem);
          r.x = -1;
        }
      }
    }
    s_rows[buf][tid] = r;
    if (r.x < 0) return;
    const long long ps = page_of(c, (int)r.x), pd = page_of(c, (int)r.y);  // a cache has less than 2^31 rows
    const long long ws = (ps * c.hkv + g) * c.page_size + (r.x - ps * c.page_size);
    const long long wd = (pd * c.hkv + g) * c.page_size + (r.y - pd * c.page_size);
    float w = 0.f;
    int pos = 0;
    if (c.weights) w = c.weights[ws];
    if (c.positions) pos = c.positions[ws];
    if (c.weights) c.weights[wd] = w;
    if (c.positions) c.positions[wd] = pos;
  };
  long long i = (long long)part * kMovesC;
  const int step = p.parts * kMovesC;
  if (i < n && tid < kMovesC) look_up(i, 0);
  uint4* rows = reinterpret_cast<uint4*>(lane < 16 ? c.k : c.v) + (lane & 15);
  for (int buf = 0; i < n; i += step, buf ^= 1) {
    __syncthreads();
    uint4 v[kMovesW];
    const longlong2* r = s_rows[buf] + warp * kMovesW;
#pragma unroll
    for (int m = 0; m < kMovesW; ++m)
      if (r[m].x >= 0) v[m] = rows[(r[m].x * c.hkv + g) * 16];
    if (i + step < n && tid < kMovesC) look_up(i + step, buf ^ 1);  // the next ones, while these rows arrive
#pragma unroll
    for (int m = 0; m < kMovesW; ++m)
      if (r[m].x >= 0) rows[(r[m].y * c.hkv + g) * 16] = v[m];
  }
}

cudaError_t launch_compact(const CompactParams& in, int sms, cudaStream_t st) {
  CompactParams p = in;
  // about four CTAs an SM over all pairs, and no more than there are chunks of moves
  const long long pairs = (long long)p.c.num_seqs * p.c.hkv, most = ((long long)p.budget + kMovesC - 1) / kMovesC;
  const long long want = (4ll * sms + pairs - 1) / pairs;
  p.parts = (int)(want < most ? want : most);
  return launch_pdl(compact_kernel, dim3((unsigned)(pairs * p.parts)), 256, 0, st, p);
}

}  // namespace fp
