// fp_cache_weights.cu -- the attention weight that cached slots collect from a call of many rows:
//   w_ug = decay * w_ug + sum_{t, h in group g, u <= lens + t} 2^(scale_log2 q_th . k_u - lse2_th)
// after the attention has left -lse2.
//
// S^T = K Q^T on the tcgen05 tensor cores with the keys along the accumulator's lanes and a row tile's 128
// rows along its columns, so that a thread owns a key and its sum over rows needs no exchange. An item is 256
// keys of one (sequence, kv-head), 128 per warpgroup: the two share the row tiles and run freely beside each
// other. Bound by the exponentials (one per pair of row and key, 16 per SM and clock); with 128 keys an item,
// the two warpgroups sharing its columns and adding up at its end, a third of the time was spent on that.
//
// A step is one (item, row tile); the steps of all items form one line that the CTAs share out evenly, as in
// the attention: an item that several CTAs share leaves one partial sum per piece, added up in the order of
// the pieces by a second kernel, so the result does not depend on timing. Row tiles stay in shared memory over
// the items of a kv-head where they fit (kQ of them).
#include "fp_cache.cuh"

namespace fp {

namespace cw {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 384, kBK = 256;
constexpr int kQ = 2, kK = 2, kS = 2;  // row tiles, items of keys, pairs of accumulators
constexpr uint32_t kTile = 128 * 128 * 2, kSlab = 128 * 128;
constexpr uint32_t kOffQ = 0, kOffK = kQ * kTile, kOffBar = kOffK + kK * 2 * kTile;
// q_full[], q_empty[], k_full[], k_empty[], s_full[][2], s_empty[][2], z_full[], drain, never (the test hook's
// barrier that nothing arrives on)
constexpr int kNumBars = 2 * kQ + 2 * kK + 5 * kS + 2;
constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;                // tmem base, abort flag, bad flag
constexpr uint32_t kOffScan = (kOffMisc + 16 + 15) & ~15u;           // int64[12]
constexpr uint32_t kOffZ = kOffScan + 8 * 12;                        // float -lse2[kS][128]
constexpr uint32_t kOffTab = kOffZ + kS * 128 * 4;
constexpr uint32_t smem_bytes(int S) { return kOffTab + 8 * (S + 1) + 1024; }
static_assert(smem_bytes(kMaxSeqs) <= 227 * 1024, "shared memory per CTA");
constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, 0, 0);
constexpr uint64_t kDrainLimitNs = 1000000000ull;

// A place on the line: step (s, g, kt, rt).
struct Step {
  int s, g, kt, rt;
  int seq0, L, len, n;
  int R, kts;   // row tiles, items of 256 keys
  int rt0;      // the first row tile that sees a key of item kt
};
__device__ __forceinline__ int first_row_tile(int len, int kt, int TT) {
  const int past = kt * kBK - len;  // tokens before the first that sees the item's first key
  return past > 0 ? past / TT : 0;
}
// steps of one kv-head: items up to the one of slot len are seen by every row tile
__device__ __forceinline__ long long head_steps(int L, int n, int TT) {
  if (L <= 0) return 0;
  const int len = n - L, R = (L + TT - 1) / TT, kts = (n + kBK - 1) / kBK, full = min(kts, len / kBK + 1);
  long long sum = (long long)full * R;
  for (int kt = full; kt < kts; ++kt) sum += R - first_row_tile(len, kt, TT);
  return sum;
}
__device__ __forceinline__ void load_seq(Step& u, const CacheInfo& c, int s, int TT) {
  u.s = s;
  u.seq0 = c.cu_seqlens[s];
  u.L = c.cu_seqlens[s + 1] - u.seq0;
  u.len = c.lens[s];
  u.n = u.len + u.L;
  u.R = (u.L + TT - 1) / TT;
  u.kts = (u.n + kBK - 1) / kBK;
}
__device__ __forceinline__ Step step_at(const CacheInfo& c, const long long* tab, int TT, long long x) {
  Step u;
  load_seq(u, c, find_seq64(tab, c.num_seqs, x), TT);
  const long long per = (tab[u.s + 1] - tab[u.s]) / c.hkv;
  long long left = x - tab[u.s];
  u.g = (int)(left / per);
  left -= u.g * per;
  const int full = min(u.kts, u.len / kBK + 1);
  if (left < (long long)full * u.R) {
    u.kt = (int)(left / u.R);
    u.rt = (int)(left - (long long)u.kt * u.R);
    u.rt0 = 0;
    return u;
  }
  left -= (long long)full * u.R;
  for (u.kt = full;; ++u.kt) {
    u.rt0 = first_row_tile(u.len, u.kt, TT);
    if (left < u.R - u.rt0) break;
    left -= u.R - u.rt0;
  }
  u.rt = u.rt0 + (int)left;
  return u;
}
__device__ __forceinline__ void step_next(Step& u, const CacheInfo& c, int TT, bool more) {
  if (++u.rt < u.R || !more) return;
  if (++u.kt == u.kts) {
    u.kt = 0;
    if (++u.g == c.hkv) {
      u.g = 0;
      int s = u.s;
      do load_seq(u, c, ++s, TT);
      while (u.L <= 0 && s + 1 < c.num_seqs);
    }
  }
  u.rt = u.rt0 = first_row_tile(u.len, u.kt, TT);
}

__global__ void __launch_bounds__(kThreads, 1) cache_tiles_weights_kernel(const __grid_constant__ CacheAttnParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem), sQ = sbase + kOffQ, sK = sbase + kOffK, bar0 = sbase + kOffBar;
  auto b_q_full = [&](uint32_t i) { return bar0 + 8 * (i % kQ); };
  auto b_q_empty = [&](uint32_t i) { return bar0 + 8 * (kQ + i % kQ); };
  auto b_k_full = [&](uint32_t i) { return bar0 + 8 * (2 * kQ + i % kK); };
  auto b_k_empty = [&](uint32_t i) { return bar0 + 8 * (2 * kQ + kK + i % kK); };
  auto b_s_full = [&](uint32_t i, int h) { return bar0 + 8 * (2 * kQ + 2 * kK + 2 * (i % kS) + h); };
  auto b_s_empty = [&](uint32_t i, int h) { return bar0 + 8 * (2 * kQ + 2 * kK + 2 * kS + 2 * (i % kS) + h); };
  auto b_z_full = [&](uint32_t i) { return bar0 + 8 * (2 * kQ + 2 * kK + 4 * kS + i % kS); };
  const uint32_t b_drain = bar0 + 8 * (kNumBars - 2), b_never = b_drain + 8;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_bad = reinterpret_cast<int*>(smem + kOffMisc + 8);
  long long* s_scan = reinterpret_cast<long long*>(smem + kOffScan);
  float* s_z = reinterpret_cast<float*>(smem + kOffZ);
  long long* tab = reinterpret_cast<long long*>(smem + kOffTab);
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const int G = c.group, TT = p.tile_tokens;
  if (tid == 0) {
    for (int i = 0; i < kQ; ++i) {
      mbar_init(b_q_full(i), 1);
      mbar_init(b_q_empty(i), 1);
    }
    for (int i = 0; i < kK; ++i) {
      mbar_init(b_k_full(i), 1);
      mbar_init(b_k_empty(i), 1);
    }
    for (int i = 0; i < kS; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(b_s_full(i, h), 1);
        mbar_init(b_s_empty(i, h), 128);
      }
      mbar_init(b_z_full(i), 32);
    }
    mbar_init(b_drain, 1);
    mbar_init(b_never, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  pdl_wait();
  const bool ok = cache_table<kThreads>(c, tab, s_scan, s_bad, p.dev_status, [&](int, int L, int n) -> long long {
    return c.hkv * head_steps(L, n, TT);
  });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_trigger();
  const long long T = ok ? tab[c.num_seqs] : 0;
  const Shares sh(T, gridDim.x);
  const int me = blockIdx.x;
  const long long x0 = me < sh.parts ? sh.at(me) : 0, x1 = me < sh.parts ? sh.at(me + 1) : 0;
  if (x0 >= x1) {
    if (tid == 0) p.meta[(long long)me * kMetaWords] = 0;
  }
  Step u;
  if (x0 < x1) u = step_at(c, tab, TT, x0);
  auto all_wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(kAll, mbar_wait(bar, parity, p.wait_limit_ns));
  };
  bool fail = false;
  if (warp == 0) {
    // =========================================================== loads
    if (x0 < x1 && lane == 0) {
      int32_t* meta = p.meta + (long long)me * kMetaWords;
      const long long item0 = x0 - (u.rt - u.rt0), end = item0 + u.R - u.rt0;
      const bool inside = u.rt > u.rt0;
      meta[0] = inside && sh.at(me - 1) <= item0;
      if (inside) {
        int last = me;  // the last CTA whose share begins inside the item's steps
        while (last + 1 < sh.parts && sh.at(last + 1) < end) ++last;
        meta[1] = last;
        meta[2] = u.s;
        meta[3] = u.g;
        meta[4] = u.kt;
      }
    }
    uint32_t qit = 0, kit = 0;
    bool bad_page = false;
    const int bh = p.box_rows, lanes = kBK / bh;
    const uint32_t q_bytes = (uint32_t)(G * TT) * 128u;
    const int no_row = (int)min((long long)c.num_pages * c.page_size, 0x7fffffffll);
    auto load_q = [&](int rt) -> bool {
      if (qit >= kQ && !all_wait(b_q_empty(qit), ((qit / kQ) - 1) & 1)) return false;
      if (lane == 0) {
        const uint32_t dst = sQ + qit % kQ * kTile;
        mbar_arrive_expect_tx(b_q_full(qit), 2 * q_bytes);
        tma_load_3d(dst, &p.tm_q, b_q_full(qit), 0, u.g * G, u.seq0 + rt * TT);
        tma_load_3d(dst + kSlab, &p.tm_q, b_q_full(qit), 64, u.g * G, u.seq0 + rt * TT);
      }
      ++qit;
      return true;
    };
    bool head = true, tile = true;  // this step begins a kv-head / an item (within the share)
    for (long long x = x0; x < x1; ++x) {
      const bool resident = u.R <= kQ;
      if (head && resident) {
        for (int j = 0; j < u.R && !fail; ++j) fail = !load_q(j);
        if (fail) break;
      }
      if (tile) {
        const int key = u.kt * kBK + lane * bh;
        int row = no_row;  // a page outside the cache and slots past the sequence's end read as zeros
        if (lane < lanes && key < u.n) {
          const long long r = slot_row(c, u.s, key);
          bad_page |= r < 0;
          if (r >= 0) row = (int)r;
        }
        if (kit >= kK && !all_wait(b_k_empty(kit), ((kit / kK) - 1) & 1)) { fail = true; break; }
        if (lane == 0) mbar_arrive_expect_tx(b_k_full(kit), 2 * kTile);
        __syncwarp();
        if (lane < lanes) {
          const uint32_t dst = sK + kit % kK * 2 * kTile + lane * bh / 128 * kTile + lane * bh % 128 * 128;
          tma_load_2d(dst, &p.tm_k, b_k_full(kit), u.g * kHeadDim, row);
          tma_load_2d(dst + kSlab, &p.tm_k, b_k_full(kit), u.g * kHeadDim + 64, row);
        }
        ++kit;
      }
      if (!resident && !load_q(u.rt)) { fail = true; break; }
      const int g = u.g, kt = u.kt, s = u.s;
      step_next(u, c, TT, x + 1 < x1);
      head = u.g != g || u.s != s;
      tile = head || u.kt != kt;
      if (*s_abort) { fail = true; break; }
    }
    if (bad_page) dev_flag(p.dev_status, kDevBadProblem);
    if (fail && lane == 0) {
      *s_abort = 1;
      dev_flag(p.dev_status, kDevTimeout);
      for (uint32_t i = 0; i < kQ; ++i)  // copies in flight land before the CTA ends
        if (qit > i) mbar_wait(b_q_full(qit - 1 - i), ((qit - 1 - i) / kQ) & 1, kDrainLimitNs);
      for (uint32_t i = 0; i < kK; ++i)
        if (kit > i) mbar_wait(b_k_full(kit - 1 - i), ((kit - 1 - i) / kK) & 1, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // =========================================================== tcgen05 issue (one thread)
    if (lane == 0) {
      uint32_t qit = 0, kit = 0, it = 0;  // row tiles released, key tiles released, steps
      bool head = true, tile = true;
      for (long long x = x0; x < x1; ++x, ++it) {
        const bool resident = u.R <= kQ;
        if (head && resident) {
          for (int j = 0; j < u.R && !fail; ++j) fail = !mbar_wait(b_q_full(qit + j), ((qit + j) / kQ) & 1, p.wait_limit_ns);
          if (fail) break;
        }
        if (!resident && !mbar_wait(b_q_full(qit), (qit / kQ) & 1, p.wait_limit_ns)) { fail = true; break; }
        if (tile && !mbar_wait(b_k_full(kit), (kit / kK) & 1, p.wait_limit_ns)) { fail = true; break; }
        const uint32_t qslot = (resident ? qit + u.rt : qit) % kQ;
        const uint64_t qdesc = sdesc_sw128(sQ + qslot * kTile, 16, 1024);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!fail && it >= kS) fail = !mbar_wait(b_s_empty(it, h), ((it / kS) - 1) & 1, p.wait_limit_ns);
          if (fail) break;
          tc_fence_after();
          const uint64_t kdesc = sdesc_sw128(sK + (kit % kK * 2 + h) * kTile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
            mma_ss(tmem + 256 * (it % kS) + 128 * h, desc_advance(kdesc, off), desc_advance(qdesc, off), kIdesc,
                   kk > 0 ? 1u : 0u);
          }
          mma_commit(b_s_full(it, h));
        }
        if (fail) break;
        const int g = u.g, kt = u.kt, s = u.s, R = u.R;
        step_next(u, c, TT, x + 1 < x1);
        head = u.g != g || u.s != s || x + 1 == x1;
        tile = head || u.kt != kt;
        if (!resident) {
          mma_commit(b_q_empty(qit));
          ++qit;
        } else if (head) {
          for (int j = 0; j < R; ++j) mma_commit(b_q_empty(qit + j));
          qit += R;
        }
        if (tile) {
          mma_commit(b_k_empty(kit));
          ++kit;
        }
        if (*s_abort) { fail = true; break; }
      }
      if (fail) {
        *s_abort = 1;
        dev_flag(p.dev_status, kDevTimeout);
      }
      mma_commit(b_drain);  // every issued product completes before TMEM is released
      mbar_wait(b_drain, 0, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 2) {
    // =========================================================== -lse2 of the row tiles, copied as they are
    uint32_t it = 0;
    int tok_r[4], head_r[4];
    for (int j = 0; j < 4; ++j) {
      tok_r[j] = (lane + 32 * j) / G;
      head_r[j] = (lane + 32 * j) % G;
    }
    for (long long x = x0; x < x1; ++x, ++it) {
      if (it >= kS && (!all_wait(b_s_empty(it, 0), ((it / kS) - 1) & 1) || !all_wait(b_s_empty(it, 1), ((it / kS) - 1) & 1))) {
        fail = true;
        break;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (tok_r[j] < TT) {  // tokens past the sequence's end are masked: any value
          const int tok = min(u.rt * TT + tok_r[j], u.L - 1);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sbase + kOffZ + (it % kS * 128 + lane + 32 * j) * 4),
                       "l"(p.lse2 + (long long)(u.g * G + head_r[j]) * c.total_tokens + u.seq0 + tok)
                       : "memory");
        }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(b_z_full(it)) : "memory");
      step_next(u, c, TT, x + 1 < x1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (fail && lane == 0) {
      *s_abort = 1;
      dev_flag(p.dev_status, kDevTimeout);
    }
    __syncwarp();
  } else if (wg >= 1) {
    // =========================================================== exponentials: thread = key
    const int half = wg - 1, r = 128 * half + (warp & 3) * 32 + lane;  // the item's key
    const uint32_t col0 = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128 * half;
    const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
    uint32_t it = 0;
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
    bool first_part = x0 < x1 && u.rt > u.rt0;  // the share begins inside an item's steps
    bool fresh = true;
    long long at = -1;  // this thread's weight, looked up (and read) while the item's first step is under way
    float old = 0.f;
    if (p.test_unsignalled_wait && x0 < x1) fail = !all_wait(b_never, 0);
    for (long long x = x0; x < x1 && !fail; ++x, ++it) {
      if (fresh) {
        fresh = false;
        const int key = u.kt * kBK + r;
        at = key < u.n ? slot_word(c, u.s, u.g, key) : -1;
        old = at >= 0 && p.decay > 0.f ? c.weights[at] : 0.f;
      }
      if (!all_wait(b_z_full(it), (it / kS) & 1) || !all_wait(b_s_full(it, half), (it / kS) & 1)) { fail = true; break; }
      tc_fence_after();
      const float* z = s_z + it % kS * 128;
      // columns [cmin, cmax) hold rows that see the key
      const int past = u.kt * kBK + r - u.len - u.rt * TT;
      const int cmin = (past > 0 ? min(past, TT) : 0) * G;
      const bool part = (u.rt + 1) * TT > u.L;
      const int cmax = (part ? u.L - u.rt * TT : TT) * G;
      const bool edge = part || u.kt * kBK + kBK - 1 - u.len > u.rt * TT;  // the same for every thread
      // columns below it need no mask; the spare ones of a row tile, which nothing loads, always do
      const int plain = edge ? 0 : TT * G;
      const uint32_t col = col0 + 256 * (it % kS);
      uint32_t v[2][32];
      tmem_ld32(col, v[0]);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        tmem_wait_ld();
        reg_fence32(v[b & 1]);
        if (b < 3) tmem_ld32(col + 32 * (b + 1), v[(b + 1) & 1]);
        if (32 * (b + 1) <= plain) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 zz = *reinterpret_cast<const float4*>(z + 32 * b + e);
            float a0, a1, a2, a3;
            f2_split(ffma2(f2_bits(v[b & 1][e], v[b & 1][e + 1]), scale2, f2_make(zz.x, zz.y)), a0, a1);
            f2_split(ffma2(f2_bits(v[b & 1][e + 2], v[b & 1][e + 3]), scale2, f2_make(zz.z, zz.w)), a2, a3);
            acc[(e >> 1) & 2] = fadd2(acc[(e >> 1) & 2], f2_make(ex2_approx(a0), ex2_approx(a1)));
            acc[((e >> 1) & 2) + 1] = fadd2(acc[((e >> 1) & 2) + 1], f2_make(ex2_approx(a2), ex2_approx(a3)));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int col_e = 32 * b + e;
            const float2 zz = *reinterpret_cast<const float2*>(z + col_e);
            float a0, a1;
            f2_split(ffma2(f2_bits(v[b & 1][e], v[b & 1][e + 1]), scale2, f2_make(zz.x, zz.y)), a0, a1);
            a0 = col_e >= cmin && col_e < cmax ? ex2_approx(a0) : 0.f;
            a1 = col_e + 1 >= cmin && col_e + 1 < cmax ? ex2_approx(a1) : 0.f;
            acc[(e >> 1) & 3] = fadd2(acc[(e >> 1) & 3], f2_make(a0, a1));
          }
        }
      }
      tc_fence_before();
      mbar_arrive(b_s_empty(it, half));
      const bool ends = u.rt + 1 == u.R;
      if (ends || x + 1 == x1) {
        float a0, a1, b0, b1;
        f2_split(fadd2(acc[0], acc[1]), a0, a1);
        f2_split(fadd2(acc[2], acc[3]), b0, b1);
        const float w = (a0 + a1) + (b0 + b1);
        acc[0] = acc[1] = acc[2] = acc[3] = 0ull;
        if (ends && !first_part) {
          if (at >= 0) c.weights[at] = p.decay > 0.f ? fmaf(p.decay, old, w) : w;
        } else {
          p.part_ml[(2ll * me + (first_part ? 0 : 1)) * kBK + r] = w;
        }
        first_part = false;
        fresh = true;
      }
      step_next(u, c, TT, x + 1 < x1);
    }
    if (fail) {
      *s_abort = 1;
      dev_flag(p.dev_status, kDevTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Adds up the pieces of the items that several CTAs share (places as in the attention's join).
__global__ void __launch_bounds__(kBK) cache_weights_join_kernel(const __grid_constant__ CacheAttnParams p) {
  pdl_wait();
  const int b = blockIdx.x + 1;
  const int32_t* meta = p.meta + (long long)b * kMetaWords;
  if (meta[0] == 0) return;
  const CacheInfo& c = p.c;
  const int last = meta[1], s = meta[2], key = meta[4] * kBK + (int)threadIdx.x;
  const int n = c.lens[s] + c.cu_seqlens[s + 1] - c.cu_seqlens[s];
  if (key >= n) return;
  const long long at = slot_word(c, s, meta[3], key);
  if (at < 0) return;
  float w = 0.f;
  for (int k = b - 1; k <= last; ++k) w += p.part_ml[(2ll * k + (k == b - 1)) * kBK + threadIdx.x];
  c.weights[at] = p.decay > 0.f ? fmaf(p.decay, c.weights[at], w) : w;
}

}  // namespace cw

cudaError_t launch_cache_weights(const CacheAttnParams& p, int sms, cudaStream_t st) {
  static unsigned long long attr[2][kMaxCachedDevices] = {};
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(cw::cache_tiles_weights_kernel), cw::smem_bytes(kMaxSeqs),
                               attr[0]);
  if (e == cudaSuccess)
    e = set_max_smem_carveout(reinterpret_cast<const void*>(cw::cache_weights_join_kernel), 0, attr[1]);
  if (e == cudaSuccess)
    e = launch_pdl(cw::cache_tiles_weights_kernel, dim3(sms), cw::kThreads, cw::smem_bytes(p.c.num_seqs), st, p);
  if (e != cudaSuccess || sms < 2) return e;
  return launch_pdl(cw::cache_weights_join_kernel, dim3(sms - 1), cw::kBK, 0, st, p);
}

}  // namespace fp
