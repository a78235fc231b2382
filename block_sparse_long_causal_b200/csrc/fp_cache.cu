// fp_cache.cu -- writing to a paged key/value cache and keeping it within a budget: append, selection
// of the slots that stay by collected attention weight, compaction.
#include <cooperative_groups.h>

#include "fp_cache.cuh"

namespace cg = cooperative_groups;

namespace fp {

constexpr unsigned kFullMask = 0xffffffffu;

// ------------------------------------------------------------------------ append ---------------
// One warp per new token: it finds its sequence (the number of s with cu_seqlens[s] <= t, counted 32 at
// a time, so that the look-up waits on one round trip and not on a chain), then copies the token's K
// and V rows in 16-byte pieces and sets weight 0 and the position of its slot in every kv-head.
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  const CacheInfo& c = p.c;
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= c.total_tokens) return;
  int s = -1;
  for (int b = 0; b < c.num_seqs; b += 32) {
    const int x = b + lane;
    s += __popc(__ballot_sync(kFullMask, x < c.num_seqs && __ldg(c.cu_seqlens + x) <= t));
  }
  bool ok = s >= 0;
  int u = 0;
  long long row = -1;
  if (ok) {
    const int lo = __ldg(c.cu_seqlens + s), hi = __ldg(c.cu_seqlens + s + 1), len = c.lens[s];
    ok = t < hi && len >= 0 && len <= c.max_len - (hi - lo);
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
  for (int i = lane; i < chunks; i += 32) {
    kd[i] = __ldg(ks + i);
    vd[i] = __ldg(vs + i);
  }
  if (c.weights || c.positions) {
    const long long page = row / c.page_size, off = row - page * c.page_size;
    const int pos = (p.next_pos ? p.next_pos[s] : c.lens[s]) + (u - c.lens[s]);
    for (int g = lane; g < c.hkv; g += 32) {
      const long long w = (page * c.hkv + g) * c.page_size + off;
      if (c.weights) c.weights[w] = 0.f;
      if (c.positions) c.positions[w] = pos;
    }
  }
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
  append_kernel<<<(p.c.total_tokens + 7) / 8, 256, 0, st>>>(p);
  return cudaGetLastError();
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

constexpr int kSelThreads = 1024;

// One CTA per (sequence, kv-head). The key of rank `budget` is found by a radix select (four passes of
// eight bits over the keys, each a histogram of the keys that match the prefix so far); then every warp
// counts, over its own contiguous range of slots, the slots above and at the threshold, and after a
// scan writes its holes (evicted slots below the budget) and sources (kept slots at or past it) in
// ascending order.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  const CacheInfo& c = p.c;
  const int s = blockIdx.x / c.hkv, g = blockIdx.x % c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kSelThreads / 32;
  __shared__ unsigned s_hist[256];
  __shared__ unsigned s_prefix, s_need;
  __shared__ int s_gt[2][kWarps], s_eq[2][kWarps];
  const int lo = __ldg(c.cu_seqlens + s), hi = __ldg(c.cu_seqlens + s + 1), len = c.lens[s], L = hi - lo;
  int32_t* moves = p.moves + ((long long)s * c.hkv + g) * p.budget * 2;
  const bool bad_seq = L < 0 || len < 0 || len > c.max_len - L;
  const int n = bad_seq ? 0 : len + L;
  if (tid == 0 && bad_seq) dev_flag(p.dev_status, kDevBadProblem);
  if (tid == 0 && g == 0) p.new_lens[s] = bad_seq ? len : min(n, p.budget);
  if (n <= p.budget) {  // nothing to evict (or a sequence that is skipped: no moves, lens as it was)
    if (tid == 0) p.move_counts[(long long)s * c.hkv + g] = 0;
    for (int i = tid; i < 2 * p.budget; i += kSelThreads) moves[i] = -1;
    return;
  }
  // positions at or past `young` are protected (the difference cannot overflow: 64 bits)
  const long long young = (long long)(p.next_pos ? p.next_pos[s] : len) + L - p.recent;
  bool bad_page = false;
  auto key_of = [&](int u) -> uint32_t {
    const long long w = slot_word(c, s, g, u);
    if (w < 0) {
      bad_page = true;
      return 0u;
    }
    const int pos = c.positions ? c.positions[w] : u;
    return rank_key(c.weights[w], pos < p.sinks || pos >= young);
  };
  unsigned prefix = 0, need = (unsigned)p.budget;  // `need` keys of the current prefix class stay
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int u = tid; u < n; u += kSelThreads) {
      const uint32_t k = key_of(u);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      unsigned left = need;
      int b = 255;
      while (b > 0 && s_hist[b] < left) left -= s_hist[b--];
      s_prefix = (prefix << 8) | (unsigned)b;
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  const uint32_t thr = prefix;  // keys above thr stay, and the first `need` slots whose key is thr
  const int span = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int u0 = min(n, warp * span), u1 = min(n, u0 + span);
  int gt[2] = {0, 0}, eq[2] = {0, 0};  // below / at or past the budget
  for (int u = u0; u < u1; u += 32) {
    const bool in = u + lane < u1;
    const uint32_t k = in ? key_of(u + lane) : 0u;
    const unsigned below = __ballot_sync(kFullMask, in && u + lane < p.budget);
    const unsigned mg = __ballot_sync(kFullMask, in && k > thr), me = __ballot_sync(kFullMask, in && k == thr);
    gt[0] += __popc(mg & below);
    gt[1] += __popc(mg & ~below);
    eq[0] += __popc(me & below);
    eq[1] += __popc(me & ~below);
  }
  if (lane == 0)
    for (int i = 0; i < 2; ++i) {
      s_gt[i][warp] = gt[i];
      s_eq[i][warp] = eq[i];
    }
  __syncthreads();
  // kept slots at the threshold are the first `need` in slot order: walk the warps before this one
  int eq_before = 0, hole = 0, from = 0, total = 0;
  {
    int e = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int a = min(n, w * span), b = min(n, a + span);
      const int room = max(0, (int)need - e);
      const int k0 = min(s_eq[0][w], room), k1 = min(s_eq[1][w], room - k0);
      const int holes = max(0, min(b, p.budget) - min(a, p.budget)) - s_gt[0][w] - k0;
      const int stay = s_gt[1][w] + k1;
      if (w < warp) {
        hole += holes;
        from += stay;
        eq_before += s_eq[0][w] + s_eq[1][w];
      }
      total += stay;
      e += s_eq[0][w] + s_eq[1][w];
    }
  }
  for (int u = u0; u < u1; u += 32) {
    const bool in = u + lane < u1;
    const uint32_t k = in ? key_of(u + lane) : 0u;
    const unsigned me = __ballot_sync(kFullMask, in && k == thr);
    const unsigned lt = (1u << lane) - 1u;
    const bool keep = in && (k > thr || (k == thr && eq_before + __popc(me & lt) < (int)need));
    const bool low = u + lane < p.budget;
    const unsigned mh = __ballot_sync(kFullMask, in && low && !keep), ms = __ballot_sync(kFullMask, keep && !low);
    if (in && low && !keep) moves[2 * (hole + __popc(mh & lt)) + 1] = u + lane;
    if (keep && !low) moves[2 * (from + __popc(ms & lt))] = u + lane;
    hole += __popc(mh);
    from += __popc(ms);
    eq_before += __popc(me);
  }
  for (int i = 2 * total + tid; i < 2 * p.budget; i += kSelThreads) moves[i] = -1;
  if (tid == 0) p.move_counts[(long long)s * c.hkv + g] = total;
  if (bad_page) dev_flag(p.dev_status, kDevBadProblem);
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  select_kernel<<<p.c.num_seqs * p.c.hkv, kSelThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------ compaction ------------
// One warp per move: lanes 0..15 carry the K row, lanes 16..31 the V row, 16 bytes each. Sources lie at
// or past the budget and destinations below it (checked), so no move reads what another one writes
// and the order of the moves does not matter.
__global__ void __launch_bounds__(256) compact_kernel(const CompactParams p) {
  const CacheInfo& c = p.c;
  const int lane = threadIdx.x & 31, sg = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int s = sg / c.hkv, g = sg % c.hkv;
  const int cnt = p.move_counts[sg];
  const int slots = min((long long)c.max_len, (long long)c.max_pages * c.page_size);
  if (part == 0 && threadIdx.x == 0) {
    if (cnt < 0 || cnt > p.budget) dev_flag(p.dev_status, kDevBadList);
    if (g == 0) {
      const int nl = p.new_lens[s];
      if (nl >= 0 && nl <= slots) c.lens[s] = nl;
      else dev_flag(p.dev_status, kDevBadProblem);
    }
  }
  const int2* moves = reinterpret_cast<const int2*>(p.moves) + (long long)sg * p.budget;
  for (int i = part * 8 + (threadIdx.x >> 5); i < min(cnt, p.budget); i += p.parts * 8) {
    const int2 mv = moves[i];
    if (mv.x < p.budget || mv.x >= slots || mv.y < 0 || mv.y >= p.budget || mv.y >= slots) {
      if (lane == 0) dev_flag(p.dev_status, kDevBadList);
      continue;
    }
    const long long src = slot_row(c, s, mv.x), dst = slot_row(c, s, mv.y);
    if (src < 0 || dst < 0) {
      if (lane == 0) dev_flag(p.dev_status, kDevBadProblem);
      continue;
    }
    uint4* base = reinterpret_cast<uint4*>(lane < 16 ? c.k : c.v) + (lane & 15);
    base[(dst * c.hkv + g) * 16] = base[(src * c.hkv + g) * 16];
    if (lane < 2) {
      const long long ws = (src / c.page_size * c.hkv + g) * c.page_size + src % c.page_size;
      const long long wd = (dst / c.page_size * c.hkv + g) * c.page_size + dst % c.page_size;
      if (lane == 0 && c.weights) c.weights[wd] = c.weights[ws];
      if (lane == 1 && c.positions) c.positions[wd] = c.positions[ws];
    }
  }
}

cudaError_t launch_compact(const CompactParams& in, cudaStream_t st) {
  CompactParams p = in;
  p.parts = p.budget < 64 * 64 ? (p.budget + 63) / 64 : 64;
  compact_kernel<<<p.c.num_seqs * p.c.hkv * p.parts, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fp
