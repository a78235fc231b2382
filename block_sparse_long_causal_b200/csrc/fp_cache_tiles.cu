// fp_cache_tiles.cu -- attention of new tokens over a paged key/value cache on the tcgen05 tensor cores:
// the schedule for calls whose longest piece has more packed rows than the few-row kernel takes (32).
//
// A row tile is 128 / G whole tokens with the G q-heads of one kv-head (row r: token r / G, head r % G),
// so that a K/V tile is read once for all heads of its group. A unit is two neighbouring row tiles of one
// (sequence, kv-head), one per softmax warpgroup, over the same 128-key tiles; a unit with a single row
// tile (few new tokens) gives its key tiles to the two warpgroups in turn and joins the two results
// when it ends, so that one warpgroup's softmax overlaps the other's matrix products either way.
//
// The key tiles of all units form one line that is cut into equal parts, one per CTA, whatever the
// lengths; a part may begin or end inside a unit, and the pieces of such a unit are joined from the
// workspace by the join kernel. The line visits the units in an order (unit_at) that lets CTAs which
// run at the same time work on the same kv-heads, whose K/V then stay in the L2.
#include "fp_cache.cuh"

namespace fp {

namespace tiles {

constexpr int kThreads = 384;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kBK = 128;                  // keys of a tile
constexpr int kStages = 2;                // K ring and V ring
constexpr int kUnitRing = 4;
constexpr int kUnitReaders = 10;          // the MMA warp, the tail warp and the 8 softmax warps
constexpr int kRegsCtl = 104, kRegsSoftmax = 200;
static_assert(128 * kRegsCtl + 256 * kRegsSoftmax == kThreads * 168, "register split must equal the launch allocation");
constexpr uint64_t kDrainLimitNs = 1000000000ull;
constexpr float kFastSumLimit = 65536.f;  // largest row sum that an item without a max pass may have
constexpr uint32_t kTile = 128 * 128 * 2, kSlab = 128 * 128;
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = kOffK + kStages * kTile, kOffBar = kOffV + kStages * kTile;
// q_full, q_empty, k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], o_final[2], x_full, x_done,
// drain, v_tail[], unit_full[], unit_empty[], never (the test hook's barrier that nothing arrives on)
constexpr int kNumBars = 2 + 4 * kStages + 6 + 3 + kStages + 2 * kUnitRing + 1;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;                   // tmem base, abort flag, bad flag
constexpr uint32_t kOffScan = (kOffMisc + 16 + 15) & ~15u;              // int64[12]; the line's start (5 int64)
constexpr uint32_t kOffUnit = kOffScan + 8 * 12 + 8 * 6;                // unit descriptors
constexpr uint32_t kUnitBytes = 48;
constexpr uint32_t kOffX = kOffUnit + kUnitRing * kUnitBytes;           // float max[2][128], sum[2][128]
constexpr uint32_t kOffBad = kOffX + 2 * 2 * 128 * 4;                   // per unit entry: int key[3][128], then flags
constexpr uint32_t kOffTab = (kOffBad + kUnitRing * (3 * 128 + 1) * 4 + 15) & ~15u;
constexpr uint32_t smem_bytes(int S) { return kOffTab + 8 * (S + 1) + 1024; }
static_assert(smem_bytes(kMaxSeqs) <= 227 * 1024, "shared memory per CTA");
constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kBK, 0, 0), kIdescPV = idesc_bf16_f32(128, kHeadDim, 0, 1);

// What the roles need of a piece of a unit: key tiles [kt0, kt1) of its kts.
struct Piece {
  int seq0, L, len;   // first new token, new tokens, slots before them; -1 in seq0: the CTA's part is done
  int g, tok0;        // kv-head, first token of row tile 0
  int nslot;          // row tiles
  int kt0, kt1, kts;
  int kts0;           // key tiles that row tile 0 needs (kts: row tile 1)
  int slot;           // partial result's place, or -1: the whole unit
};
static_assert(sizeof(Piece) <= kUnitBytes, "unit ring entry");

struct Unit {
  int s, g, m;
  int seq0, L, len;
};
__device__ __forceinline__ int key_tiles(const Unit& u, int tokens) {
  return (u.len + min(u.L, tokens) + kBK - 1) / kBK;
}
// Unit x in kv-head order: per sequence kv-head outermost, then the row-tile pairs from the last (longest)
// to the first.
__device__ __forceinline__ Unit decode(const CacheInfo& c, const long long* tab, int TT, long long x) {
  Unit u;
  u.s = find_seq64(tab, c.num_seqs, x);
  u.seq0 = c.cu_seqlens[u.s];
  u.L = c.cu_seqlens[u.s + 1] - u.seq0;
  u.len = c.lens[u.s];
  const int pairs = ((u.L + TT - 1) / TT + 1) / 2;
  const int local = (int)(x - tab[u.s]);
  u.g = local / pairs;
  u.m = pairs - 1 - (local - u.g * pairs);
  return u;
}
__device__ __forceinline__ unsigned gcd32(unsigned a, unsigned b) {
  while (b) {
    const unsigned t = a % b;
    a = b;
    b = t;
  }
  return a;
}
// The line's i-th unit. A CTA's part covers about N / ctas units in a row, so unit i is reached after the
// fraction i * ctas / N (mod 1) of the run; ranking the units by that fraction gives the CTAs that
// run at the same time neighbouring units of the kv-head order. d = gcd(ctas, N): i and i + N / d have
// the same fraction and follow one another. (Calls of more units than that keep the kv-head order.)
constexpr long long kOrderMax = 1 << 22;
__device__ __forceinline__ long long unit_at(long long i, long long N, unsigned ctas, unsigned d) {
  if (N <= ctas || N > kOrderMax) return i;
  return (unsigned)i * ctas % (unsigned)N + (unsigned)i / ((unsigned)N / d);
}
// What a unit weighs on the line: its key tiles, more where two row tiles take part in each, and what
// beginning and ending it costs.
constexpr int kCost1 = 2, kCost2 = 3, kUnitCost = 6;
__device__ __forceinline__ int tile_cost(const Unit& u, int TT) { return (2 * u.m + 1) * TT < u.L ? kCost2 : kCost1; }
__device__ __forceinline__ int tiles_before(long long cost, int w) { return (int)((cost + w - 1) / w); }

__global__ void __launch_bounds__(kThreads, 1) cache_tiles_kernel(const __grid_constant__ CacheAttnParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + kOffQ, sK = sbase + kOffK, sV = sbase + kOffV, bar0 = sbase + kOffBar;
  const uint32_t b_q_full = bar0, b_q_empty = bar0 + 8;
  auto b_k_full = [&](int i) { return bar0 + 16 + 8 * i; };
  auto b_k_empty = [&](int i) { return bar0 + 16 + 8 * (kStages + i); };
  auto b_v_full = [&](int i) { return bar0 + 16 + 8 * (2 * kStages + i); };
  auto b_v_empty = [&](int i) { return bar0 + 16 + 8 * (3 * kStages + i); };
  const uint32_t b_s_full0 = bar0 + 16 + 32 * kStages, b_p_full0 = b_s_full0 + 16, b_o_final0 = b_p_full0 + 16;
  const uint32_t b_x_full = b_o_final0 + 16, b_x_done = b_x_full + 8, b_drain = b_x_done + 8;
  auto b_v_tail = [&](int i) { return b_drain + 8 + 8 * i; };
  auto b_u_full = [&](uint32_t i) { return b_drain + 8 + 8 * (kStages + i % kUnitRing); };
  auto b_u_empty = [&](uint32_t i) { return b_drain + 8 + 8 * (kStages + kUnitRing + i % kUnitRing); };
  const uint32_t b_never = bar0 + 8 * (kNumBars - 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_bad = reinterpret_cast<int*>(smem + kOffMisc + 8);
  long long* s_scan = reinterpret_cast<long long*>(smem + kOffScan);
  long long* s_start = s_scan + 12;  // T, unit index, its tile, its line position
  long long* tab = reinterpret_cast<long long*>(smem + kOffTab);
  // first key of the unit's unseen-by-some ones whose V is NaN, +inf, -inf in a column (see the tail warp)
  auto bad_keys = [&](uint32_t i) { return reinterpret_cast<int*>(smem + kOffBad) + (i % kUnitRing) * 3 * 128; };
  volatile int* s_bad_unit = reinterpret_cast<volatile int*>(smem + kOffBad + kUnitRing * 3 * 128 * 4);
  auto unit_entry = [&](uint32_t i) { return reinterpret_cast<Piece*>(smem + kOffUnit + (i % kUnitRing) * kUnitBytes); };

  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const int G = c.group, TT = p.tile_tokens;
  if (tid == 0) {
    mbar_init(b_q_full, 1);
    mbar_init(b_q_empty, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(b_k_full(i), 1);
      mbar_init(b_k_empty(i), 1);
      mbar_init(b_v_full(i), 1);
      mbar_init(b_v_empty(i), 1);
      mbar_init(b_v_tail(i), 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(b_s_full0 + 8 * k, 1);
      mbar_init(b_p_full0 + 8 * k, 128);
      mbar_init(b_o_final0 + 8 * k, 1);
    }
    mbar_init(b_x_full, 256);
    mbar_init(b_x_done, 256);
    mbar_init(b_drain, 1);
    mbar_init(b_never, 1);
    for (int i = 0; i < kUnitRing; ++i) {
      mbar_init(b_u_full(i), 1);
      mbar_init(b_u_empty(i), kUnitReaders);
    }
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  for (int e = tid; e < kUnitRing * 3 * 128; e += kThreads) bad_keys(0)[e] = 0x7fffffff;
  if (tid < kUnitRing) s_bad_unit[tid] = 0;
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  pdl_wait();
  const bool ok = cache_table<kThreads>(c, tab, s_scan, s_bad, p.dev_status, [&](int, int L, int) -> long long {
    return (long long)c.hkv * (((L + TT - 1) / TT + 1) / 2);
  });
  const long long N = ok ? tab[c.num_seqs] : 0;
  // ---- this CTA's part [x0, x1) of the line, and the unit that x0 falls into
  const unsigned d = N > gridDim.x && N <= kOrderMax ? gcd32((unsigned)N, gridDim.x) : 1u;
  long long x0 = 0, x1 = 0;
  {
    int kts = 0, w = 1;
    auto cost = [&](long long i, Unit& u) {
      u = decode(c, tab, TT, unit_at(i, N, gridDim.x, d));
      kts = key_tiles(u, (2 * u.m + 2) * TT);
      w = tile_cost(u, TT);
      return (long long)kts * w + kUnitCost;
    };
    const long long per = N <= kThreads ? 1 : (N + kThreads - 1) / kThreads, a = min(N, tid * per), b = min(N, a + per);
    long long sum = 0;
    Unit u;
    for (long long i = a; i < b; ++i) sum += cost(i, u);
    const long long incl = warp_incl_scan(sum);
    __syncthreads();  // cache_table is done with the scratch
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long base = incl - sum, T = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) base += s_scan[k];
      T += s_scan[k];
    }
    // a share is no shorter than a tile, so that every piece between two shares has one
    const Shares sh(T, (int)min((long long)gridDim.x, T / kCost2));
    const int me = blockIdx.x;
    int32_t* meta = p.meta + (long long)me * kMetaWords;
    if (me < sh.parts) {
      x0 = sh.at(me);
      x1 = sh.at(me + 1);
      if (base <= x0 && x0 < base + sum) {
        for (long long i = a; i < b; ++i) {
          const long long all = per > 1 ? cost(i, u) : (long long)kts * w + kUnitCost;
          if (x0 < base + all) {
            s_start[0] = i;
            s_start[1] = x0 - base;
            // a part that begins inside a unit: the first such CTA of the unit has the pieces joined
            const bool inside = x0 > base && tiles_before(x0 - base, w) < kts;
            meta[0] = inside && sh.at(me - 1) <= base;
            if (inside) {
              int last = me;  // the last CTA whose part begins inside the unit
              while (last + 1 < sh.parts && tiles_before(sh.at(last + 1) - base, w) < kts) ++last;
              meta[1] = last;
              meta[2] = u.seq0;
              meta[3] = u.g;
              meta[4] = 2 * u.m * TT;
              meta[5] = u.L;
            }
            break;
          }
          base += all;
        }
      }
    } else if (tid == 0) {
      meta[0] = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_trigger();
  auto t_s = [&](int k) { return tmem + 128u * k; };
  auto t_o = [&](int k) { return tmem + 256u + 128u * k; };

  if (wg == 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
  if (warp == 0) {
    // =========================================================== loads
    uint32_t kit = 0, vit = 0, uc = 0;
    int q_issued = 0;
    bool fail = false, bad_page = false;
    const int bh = p.box_rows, lanes = kBK / bh;
    const uint32_t q_bytes = (uint32_t)(G * TT) * 128u;
    const int no_row = (int)min((long long)c.num_pages * c.page_size, 0x7fffffffll);  // loads from here read zeros
    auto all_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(kAll, mbar_wait(bar, parity, p.wait_limit_ns));
    };
    long long i = x0 < x1 ? s_start[0] : 0;
    long long off = x0 < x1 ? s_start[1] : 0;
    for (long long x = x0; x < x1 && !fail; ++i, off = 0) {
      const Unit u = decode(c, tab, TT, unit_at(i, N, gridDim.x, d));
      const int w = tile_cost(u, TT);
      Piece pc;
      pc.kts = key_tiles(u, (2 * u.m + 2) * TT);
      pc.kt0 = (int)min((long long)pc.kts, (long long)tiles_before(off, w));
      pc.kt1 = (int)min((long long)pc.kts, (off + (x1 - x) + w - 1) / w);
      x += (long long)pc.kts * w + kUnitCost - off;
      if (pc.kt0 >= pc.kts) continue;  // the part begins in what ending the unit costs
      pc.seq0 = u.seq0;
      pc.L = u.L;
      pc.len = u.len;
      pc.g = u.g;
      pc.tok0 = 2 * u.m * TT;
      pc.nslot = pc.tok0 + TT < u.L ? 2 : 1;
      pc.kts0 = key_tiles(u, (2 * u.m + 1) * TT);
      pc.slot = pc.kt0 == 0 && pc.kt1 == pc.kts ? -1 : 2 * (int)blockIdx.x + (pc.kt0 == 0 ? 1 : 0);
      if (uc >= kUnitRing && !all_wait(b_u_empty(uc), ((uc / kUnitRing) - 1) & 1)) { fail = true; break; }
      if (lane == 0) {
        *unit_entry(uc) = pc;
        mbar_arrive(b_u_full(uc));
      }
      if (!all_wait(b_q_empty, (uc & 1) ^ 1)) { fail = true; break; }
      if (lane == 0) {
        mbar_arrive_expect_tx(b_q_full, 2 * pc.nslot * q_bytes);
        for (int k = 0; k < 2 * pc.nslot; ++k)
          tma_load_3d(sQ + (k >> 1) * kTile + (k & 1) * kSlab, &p.tm_q, b_q_full, 64 * (k & 1), u.g * G,
                      u.seq0 + pc.tok0 + (k >> 1) * TT);
      }
      ++q_issued;
      ++uc;
      const int n = u.len + u.L;
      // one lane per group of box_rows slots, which lie in one page; a page outside the cache and groups
      // past the sequence's end read as zeros
      auto row_of = [&](int t) -> int {
        const int key = t * kBK + lane * bh;
        if (lane >= lanes || key >= n) return no_row;
        const long long row = slot_row(c, u.s, key);
        bad_page |= row < 0;
        return row < 0 ? no_row : (int)row;
      };
      auto load = [&](uint32_t dst, const void* tm, uint32_t full, int row) {
        if (lane == 0) mbar_arrive_expect_tx(full, kTile);
        __syncwarp();
        if (lane < lanes) {
          tma_load_2d(dst + lane * bh * 128, tm, full, u.g * kHeadDim, row);
          tma_load_2d(dst + kSlab + lane * bh * 128, tm, full, u.g * kHeadDim + 64, row);
        }
      };
      // a tile with keys that the unit's first token does not see goes to the tail warp first
      const int tail0 = (u.len + pc.tok0 + 1) / kBK;
      auto load_v = [&](int t, int row) -> bool {
        const int vs = vit % kStages;
        if (!all_wait(b_v_empty(vs), ((vit / kStages) & 1) ^ 1)) return false;
        load(sV + vs * kTile, &p.tm_v, t >= tail0 ? b_v_tail(vs) : b_v_full(vs), row);
        ++vit;
        return true;
      };
      // V of a tile is loaded after K of the next one: its product comes later
      int row = row_of(pc.kt0), vrow = -1;
      for (int t = pc.kt0; t < pc.kt1; ++t) {
        const int ks = kit % kStages;
        const int next = t + 1 < pc.kt1 ? row_of(t + 1) : no_row;  // the table's answer arrives during the wait
        if (!all_wait(b_k_empty(ks), ((kit / kStages) & 1) ^ 1)) { fail = true; break; }
        load(sK + ks * kTile, &p.tm_k, b_k_full(ks), row);
        ++kit;
        if (t > pc.kt0 && !load_v(t - 1, vrow)) { fail = true; break; }
        vrow = row;
        row = next;
        if (*s_abort) { fail = true; break; }
      }
      if (!fail && !load_v(pc.kt1 - 1, vrow)) fail = true;
    }
    if (!fail && uc >= kUnitRing && !all_wait(b_u_empty(uc), ((uc / kUnitRing) - 1) & 1)) fail = true;
    if (!fail && lane == 0) {
      unit_entry(uc)->seq0 = -1;
      mbar_arrive(b_u_full(uc));
    }
    if (bad_page) dev_flag(p.dev_status, kDevBadProblem);
    if (fail && lane == 0) {
      *s_abort = 1;
      dev_flag(p.dev_status, kDevTimeout);
      for (int k = 0; k < kStages; ++k) {  // copies in flight land before the CTA ends
        if (kit > (uint32_t)k) mbar_wait(b_k_full((kit - 1 - k) % kStages), ((kit - 1 - k) / kStages) & 1, kDrainLimitNs);
        if (vit > (uint32_t)k) mbar_wait(b_v_full((vit - 1 - k) % kStages), ((vit - 1 - k) / kStages) & 1, kDrainLimitNs);
      }
      if (q_issued > 0) mbar_wait(b_q_full, (uint32_t)(q_issued - 1) & 1, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // =========================================================== tcgen05 issue (one thread)
    if (lane == 0) {
      uint32_t kit = 0, vit = 0, cnt[2] = {0, 0};
      bool fail = false;
      auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, p.wait_limit_ns); };
      // descriptors are built once: every instruction of this thread lies on the critical path
      const uint64_t q_desc = sdesc_sw128(sQ, 16, 1024), k_desc = sdesc_sw128(sK, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(sV, kSlab, 1024);
      for (uint32_t uc = 0; !fail; ++uc) {
        if (!wait(b_u_full(uc), (uc / kUnitRing) & 1)) { fail = true; break; }
        const Piece pc = *unit_entry(uc);
        mbar_arrive(b_u_empty(uc));
        if (pc.seq0 < 0) break;
        if (!wait(b_q_full, uc & 1)) { fail = true; break; }
        tc_fence_after();
        int prev_part = 0;
        bool had_pv[2] = {false, false};
        auto pv = [&](int k) -> bool {  // O_k += P_k V of the tile before
          if (!wait(b_p_full0 + 8 * k, (cnt[k] - 1) & 1)) return false;
          const int vs = vit % kStages;
          if (!wait(b_v_full(vs), (vit / kStages) & 1)) return false;
          tc_fence_after();
          const uint64_t vdesc = desc_advance(v_desc, vs * (kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            mma_ts(t_o(k), t_s(k) + kk * 8, desc_advance(vdesc, kk * (2048 >> 4)), kIdescPV,
                   had_pv[k] || kk > 0 ? 1u : 0u);
          had_pv[k] = true;
          return true;
        };
        const uint64_t q_desc1 = pc.nslot == 2 ? desc_advance(q_desc, kTile >> 4) : q_desc;
        auto qk = [&](int k, uint64_t kdesc) {
          const uint64_t qdesc = k == 0 ? q_desc : q_desc1;
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
            mma_ss(t_s(k), desc_advance(qdesc, off), desc_advance(kdesc, off), kIdescQK, kk > 0 ? 1u : 0u);
          }
          mma_commit(b_s_full0 + 8 * k);
          ++cnt[k];
        };
        for (int t = pc.kt0; t < pc.kt1; ++t) {
          const int part = pc.nslot == 2 ? (t < pc.kts0 ? 3 : 2) : 1 << ((t - pc.kt0) & 1);
          const int ks = kit % kStages;
          if (!wait(b_k_full(ks), (kit / kStages) & 1)) { fail = true; break; }
          tc_fence_after();
          const uint64_t kdesc = desc_advance(k_desc, ks * (kTile >> 4));
          // a slot that took part in the previous tile issues that tile's PV before this one's QK (S overwrites
          // P); the QK of one that did not goes first, so that its softmax overlaps the other's
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (((part & ~prev_part) >> k) & 1) qk(k, kdesc);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!fail && ((prev_part >> k) & 1)) {
              if (!pv(k)) { fail = true; break; }
              if ((part >> k) & 1) qk(k, kdesc);
            }
          if (fail) break;
          if (t > pc.kt0) {
            mma_commit(b_v_empty(vit % kStages));
            ++vit;
          }
          mma_commit(b_k_empty(ks));
          if (t + 1 == pc.kt1) mma_commit(b_q_empty);
          ++kit;
          prev_part = part;
          if (*s_abort) { fail = true; break; }
        }
        if (fail) break;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (!fail && ((prev_part >> k) & 1))
            if (!pv(k)) fail = true;
        if (fail) break;
        mma_commit(b_v_empty(vit % kStages));
        if (had_pv[0]) mma_commit(b_o_final0);
        if (had_pv[1]) mma_commit(b_o_final0 + 8);
        ++vit;
      }
      if (fail) {
        *s_abort = 1;
        dev_flag(p.dev_status, kDevTimeout);
      }
      mma_commit(b_drain);  // every issued product completes before TMEM is released
      mbar_wait(b_drain, 0, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp == 3) {
    // =========================================================== V rows that some row of the unit does not see
    // 0 * NaN is NaN, so what is masked has to be finite in V as well. Slots behind the sequence's last one may
    // hold anything: zeros. Non-finite values of new tokens become zeros too, and the first key that has one in
    // a column is noted for the epilogue, which adds it to the rows that do see the key (p > 0).
    uint32_t vit = 0, tails[2] = {0, 0};
    static_assert(kStages == 2, "tail barriers' phases");
    bool fail = false;
    auto all_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(kAll, mbar_wait(bar, parity, p.wait_limit_ns));
    };
    for (uint32_t uc = 0; !fail; ++uc) {
      if (!all_wait(b_u_full(uc), (uc / kUnitRing) & 1)) { fail = true; break; }
      const Piece pc = *unit_entry(uc);
      __syncwarp();
      if (pc.seq0 < 0) break;
      int* bad = bad_keys(uc);
      if (s_bad_unit[uc % kUnitRing]) {  // left by an earlier unit of this entry
        __syncwarp();
        for (int e = lane; e < 3 * 128; e += 32) bad[e] = 0x7fffffff;
        if (lane == 0) s_bad_unit[uc % kUnitRing] = 0;
        __syncwarp();
      }
      const int seen = pc.len + pc.tok0 + 1;  // keys below it are seen by every row
      for (int t = pc.kt0; t < pc.kt1; ++t, ++vit) {
        if (t < seen / kBK) continue;
        const int vs = vit % kStages;
        const uint32_t phase = vs ? tails[1]++ : tails[0]++;
        if (!all_wait(b_v_tail(vs), phase & 1)) { fail = true; break; }
        unsigned char* v = smem + kOffV + vs * kTile;
        const int live = min(kBK, pc.len + pc.L - t * kBK);  // rows of the sequence
        bool any = false;
        for (int e = max(0, seen - t * kBK) * 8 + lane; e < live * 8; e += 32)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 x = *reinterpret_cast<const uint4*>(v + h * kSlab + e * 16);
            any |= nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) || nonfinite2(x.w);
          }
        if (__any_sync(kAll, any)) {
          for (int e = max(0, seen - t * kBK) * 8 + lane; e < live * 8; e += 32)
            for (int h = 0; h < 2; ++h)
              for (int i = 0; i < 8; ++i) {
                uint16_t* x = reinterpret_cast<uint16_t*>(v + h * kSlab + e * 16) + i;
                if ((*x & 0x7f80) != 0x7f80) continue;
                const int col = 64 * h + (((e & 7) ^ ((e >> 3) & 7)) << 3) + i;  // 128-byte swizzle
                atomicMin(bad + ((*x & 0x7f) ? 0 : *x >> 15 ? 256 : 128) + col, t * kBK + (e >> 3));
                *x = 0;
              }
          if (lane == 0) s_bad_unit[uc % kUnitRing] = 1;
        }
        for (int e = live * 8 + lane; e < kBK * 8; e += 32) {
          *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(v + kSlab + e * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __threadfence_block();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_v_full(vs));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_u_empty(uc));
    }
    if (fail && lane == 0) {
      *s_abort = 1;
      dev_flag(p.dev_status, kDevTimeout);
    }
    __syncwarp();
  } else if (wg >= 1) {
    // =========================================================== softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int slot = wg - 1, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = t_s(slot) + lane_off, o_col = t_o(slot) + lane_off;
    const uint32_t b_s_full = b_s_full0 + 8 * slot, b_p_full = b_p_full0 + 8 * slot;
    float* s_xm = reinterpret_cast<float*>(smem + kOffX);
    float* s_xl = s_xm + 256;
    uint32_t cnt = 0, fc[2] = {0, 0}, xc = 0;
    bool fail = false;
    auto all_wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(kAll, mbar_wait(bar, parity, p.wait_limit_ns));
    };
    const uint64_t scale2 = f2_make(p.scale_log2, p.scale_log2);
    if (p.test_unsignalled_wait && x0 < x1) fail = !all_wait(b_never, 0);
    for (uint32_t uc = 0; !fail; ++uc) {
      if (!all_wait(b_u_full(uc), (uc / kUnitRing) & 1)) { fail = true; break; }
      const Piece pc = *unit_entry(uc);
      __syncwarp();
      if (pc.seq0 < 0) break;
      const bool dual = pc.nslot == 1;  // both warpgroups share the row tile
      const int tok = pc.tok0 + (dual ? 0 : slot) * TT + r / G;
      // rows without a token (the tile's spare rows, tokens past the sequence's end) hold anything: they take no
      // part in the votes and are not written
      const bool pad = r >= TT * G || tok >= pc.L;
      const int last = pad ? 0x7fffffff : pc.len + tok;  // the last key that the row sees
      const int t1 = dual || slot == 1 ? pc.kt1 : min(pc.kt1, pc.kts0), step = dual ? 2 : 1;
      float m_run = -INFINITY, l_run = 0.f;
      int n = 0;
      for (int t = pc.kt0 + (dual ? slot : 0); t < t1; t += step) {
        if (!all_wait(b_s_full, cnt & 1)) { fail = true; break; }
        tc_fence_after();
        const int valid = last - t * kBK;  // keys 0 .. valid of the tile are seen
        const bool masked = valid < kBK - 1;
        uint32_t pk[kBK / 2];
        bool done = false;
        // without a max pass, against the row's reference so far; a sum of at most 2^16 bounds every term
        if (__all_sync(kAll, pad || (!masked && m_run != -INFINITY))) {
          const uint64_t negm2 = f2_make(-m_run, -m_run);
          uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
          uint32_t cb[2][32];
          tmem_ld32(s_col, cb[0]);
#pragma unroll
          for (int b = 0; b < kBK / 32; ++b) {
            tmem_wait_ld();
            reg_fence32(cb[b & 1]);
            if (b + 1 < kBK / 32) tmem_ld32(s_col + 32 * (b + 1), cb[(b + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const int pr = 16 * b + e / 2;
              float v0, v1;
              f2_split(ffma2(f2_bits(cb[b & 1][e], cb[b & 1][e + 1]), scale2, negm2), v0, v1);
              v0 = ex2_approx(v0);
              v1 = ex2_approx(v1);
              acc[pr & 3] = fadd2(acc[pr & 3], f2_make(v0, v1));
              pk[pr] = pack_bf16x2(v0, v1);  // P goes to the tensor cores in bf16 (half a step: 2^-9 of a term)
            }
          }
          float a0, a1, b0, b1;
          f2_split(fadd2(acc[0], acc[1]), a0, a1);
          f2_split(fadd2(acc[2], acc[3]), b0, b1);
          const float sum = (a0 + a1) + (b0 + b1);
          done = __all_sync(kAll, pad || sum <= kFastSumLimit);
          if (done) l_run += sum;
        }
        if (!done) {
          uint32_t sr[kBK];
#pragma unroll
          for (int b = 0; b < kBK; b += 32) tmem_ld32(s_col + b, *reinterpret_cast<uint32_t(*)[32]>(&sr[b]));
          tmem_wait_ld();
#pragma unroll
          for (int b = 0; b < kBK; b += 32) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[b]));
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kBK; e += 8)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const float v0 = e + 2 * a <= valid ? __uint_as_float(sr[e + 2 * a]) : -INFINITY;
              const float v1 = e + 2 * a + 1 <= valid ? __uint_as_float(sr[e + 2 * a + 1]) : -INFINITY;
              sr[e + 2 * a] = __float_as_uint(v0);
              sr[e + 2 * a + 1] = __float_as_uint(v1);
              m4[a] = fmax3(m4[a], v0, v1);
            }
          const float m_new = fmaxf(m_run, fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * p.scale_log2);
          // the reference follows only when a score passes it by 2^8: the quotient does not depend on it
          const bool grow = m_new > m_run + 8.f;
          float alpha = 1.f;
          if (grow) {
            alpha = ex2_approx(m_run - m_new);
            m_run = m_new;
          }
          l_run *= alpha;
          if (n > 0 && __any_sync(kAll, grow)) {
            // this slot's earlier products are complete: S came after them. In a shared row tile they are those of
            // the slot's own last tile, whose PV was issued before the QK of this one
            const uint64_t a2 = f2_make(alpha, alpha);
#pragma unroll 1
            for (int b = 0; b < kHeadDim; b += 32) {
              uint32_t o[32];
              tmem_ld32(o_col + b, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float lo, hi;
                f2_split(fmul2(f2_bits(o[e], o[e + 1]), a2), lo, hi);
                o[e] = __float_as_uint(lo);
                o[e + 1] = __float_as_uint(hi);
              }
              tmem_st32(o_col + b, o);
            }
          }
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          const uint64_t negm2 = f2_make(-m_use, -m_use);
          uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
          for (int e = 0; e < kBK; e += 2) {
            float v0, v1;
            f2_split(ffma2(f2_bits(sr[e], sr[e + 1]), scale2, negm2), v0, v1);
            v0 = ex2_approx(v0);
            v1 = ex2_approx(v1);
            sum2[(e >> 1) & 1] = fadd2(sum2[(e >> 1) & 1], f2_make(v0, v1));
            pk[e / 2] = pack_bf16x2(v0, v1);
          }
          float a0, a1, b0, b1;
          f2_split(sum2[0], a0, a1);
          f2_split(sum2[1], b0, b1);
          l_run += (a0 + a1) + (b0 + b1);
        }
#pragma unroll
        for (int b = 0; b < kBK / 2; b += 32) tmem_st32(s_col + b, *reinterpret_cast<uint32_t(*)[32]>(&pk[b]));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(b_p_full);
        ++cnt;
        ++n;
      }
      if (__any_sync(kAll, fail || *s_abort)) { fail = true; break; }
      // ---- the piece is complete
      const int h = pc.g * G + r % G;
      const long long token = (long long)pc.seq0 + tok;
      float w0 = 1.f, w1 = 0.f;      // weights of O_0 and O_1 (of this slot's own O when not shared)
      bool use[2] = {n > 0, false};  // which accumulators hold something (the same for every thread)
      if (dual) {
        const bool two = pc.kt1 - pc.kt0 > 1;
        s_xm[slot * 128 + r] = m_run;
        s_xl[slot * 128 + r] = l_run;
        mbar_arrive(b_x_full);
        if (!all_wait(b_x_full, xc & 1)) { fail = true; break; }
        const float m0 = s_xm[r], l0 = s_xl[r], m1 = s_xm[128 + r], l1 = s_xl[128 + r];
        m_run = fmaxf(m0, m1);
        const float mu = m_run == -INFINITY ? 0.f : m_run;
        w0 = ex2_approx(m0 - mu);
        w1 = two ? ex2_approx(m1 - mu) : 0.f;
        l_run = two ? w0 * l0 + w1 * l1 : w0 * l0;
        use[0] = true;
        use[1] = two;
        if (!all_wait(b_o_final0, fc[0] & 1)) fail = true;
        if (two && !all_wait(b_o_final0 + 8, fc[1] & 1)) fail = true;
        fc[0] += 1;
        fc[1] += two;
      } else {
        if (n > 0 && !all_wait(b_o_final0 + 8 * slot, fc[slot] & 1)) fail = true;
        fc[0] += pc.kt0 < pc.kts0;  // both warpgroups count the phases of both barriers
        fc[1] += 1;
      }
      if (fail) break;
      tc_fence_after();
      const bool any = l_run > 0.f || l_run != l_run;
      if (pc.slot < 0) {
        const float inv = any ? 1.f / l_run : 0.f;
        w0 *= inv;
        w1 *= inv;
      }
      const long long part0 = (long long)pc.slot * 2 + (dual ? 0 : slot);  // this row tile's partial results
      uint16_t* orow = p.out + (token * c.hq + h) * kHeadDim;
      const int* bad = bad_keys(uc);
      // the notes are this unit's only where the piece has a tail tile: its V, and so its products, then waited for the
      // tail warp; in a piece without one the tail warp may still be clearing an earlier unit's
      const bool odd = pc.kt1 > (pc.len + pc.tok0 + 1) / kBK && s_bad_unit[uc % kUnitRing] != 0;
      const uint32_t col0 = t_o(dual ? 0 : slot) + lane_off, col1 = t_o(1) + lane_off;
      const int cb = dual ? 64 * slot : 0, ce = dual ? cb + 64 : kHeadDim;
      if (use[0] || pc.slot < 0) {
#pragma unroll 1
        for (int b = cb; b < ce; b += 32) {
          uint32_t o[32];
          if (use[0]) {
            tmem_ld32(col0 + b, o);
            tmem_wait_ld();
            reg_fence32(o);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = use[0] ? __float_as_uint(__uint_as_float(o[e]) * w0) : 0u;
          if (use[1]) {
            uint32_t o1[32];
            tmem_ld32(col1 + b, o1);
            tmem_wait_ld();
            reg_fence32(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
          }
          if (odd)  // rare: non-finite V of a key that this row sees and others do not
            for (int e = 0; e < 32; ++e) {
              float add = last >= bad[b + e] ? NAN : 0.f;
              if (last >= bad[128 + b + e]) add += INFINITY;
              if (last >= bad[256 + b + e]) add -= INFINITY;
              o[e] = __float_as_uint(__uint_as_float(o[e]) + add);
            }
          if (!pad && pc.slot < 0) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            if (p.out32) {  // a whole sector per thread
              st_global_v8(orow + b, w);
              st_global_v8(orow + b + 16, w + 8);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(orow + b);
#pragma unroll
              for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          } else if (!pad) {
            // [eight columns][row]: a warp's store is 1 KB in a row (a row of 512 bytes per thread took 2 us longer)
            float* dst = p.part_o + ((part0 * (kHeadDim / 8) + b / 8) * 128 + r) * 8;
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_v8(dst + e * 128, o + e);
          }
          __syncwarp();
        }
      }
      if (!pad && (!dual || slot == 0)) {
        if (pc.slot < 0) {
          const float mu = m_run == -INFINITY ? 0.f : m_run;
          const float z = any ? mu + log2f(l_run) : -INFINITY;
          const long long at = (long long)h * c.total_tokens + token;
          if (p.lse2) p.lse2[at] = any ? -z : -INFINITY;  // a row without a finite score adds no weight
          if (p.lse) p.lse[at] = z * 0.6931471805599453f;
        } else {  // a row tile without a key tile in this piece: sum 0, and its O is not read
          *reinterpret_cast<float2*>(p.part_ml + 2 * (part0 * 128 + r)) = make_float2(n > 0 || dual ? m_run : -INFINITY, l_run);
        }
      }
      tc_fence_before();
      if (dual) {  // neither warpgroup goes on to overwrite an accumulator or the exchange that the other still reads
        mbar_arrive(b_x_done);
        if (!all_wait(b_x_done, xc & 1)) { fail = true; break; }
        ++xc;
        tc_fence_after();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_u_empty(uc));  // the entry and its noted keys may be used again
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

// Joins the pieces of the units that several CTAs share. Entry b of meta describes the unit inside of which
// the part of CTA b begins and is set for the first such CTA of a unit: the unit's pieces are then the last
// one of CTA b - 1 (place 1) and the first one (place 0) of every CTA from b to meta[1].
// The time is one chain of dependent reads, so the work is laid out flat: every block lists the set entries, and a
// warp takes 32 rows (a lane each) and 16 columns of a unit, four pieces in flight at a time; where there are fewer
// such tasks than warps, up to eight warps of a block share a task's pieces.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinBatch = 4;
__global__ void __launch_bounds__(kJoinThreads) cache_tiles_join_kernel(const __grid_constant__ CacheAttnParams p, int ctas) {
  __shared__ int4 s_meta[kJoinThreads][2];  // set entries; word 0: the CTA
  __shared__ int s_first[kJoinThreads], s_num[kJoinWarps];  // tasks of the entries before an entry
  __shared__ float s_acc[kJoinWarps][18][32];               // maximum, sum and columns of a warp's pieces
  pdl_wait();
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = c.group, TT = p.tile_tokens;
  for (int b0 = 0; b0 < ctas; b0 += kJoinThreads) {  // one round on devices of up to 256 SMs
    __syncthreads();
    int4 e0 = make_int4(0, 0, 0, 0), e1 = e0;
    if (b0 + tid < ctas) {
      const int4* src = reinterpret_cast<const int4*>(p.meta + (long long)(b0 + tid) * kMetaWords);
      e0 = __ldcg(src);
      e1 = __ldcg(src + 1);
    }
    const unsigned set = __ballot_sync(kAll, e0.x != 0);
    int mine = 0;  // 32-row groups of the unit, times 8 column groups
    if (e0.x != 0) {
      const int toks = e1.y - e1.x, rows = toks > TT ? 128 + min(toks - TT, TT) * G : toks * G;
      mine = (rows + 31) / 32 * 8;
    }
    const int incl = warp_incl_scan(mine);
    if (lane == 31) s_num[warp] = incl << 6 | __popc(set);  // at most 32 * 64 tasks, 32 entries
    __syncthreads();
    int at = __popc(set & ((1u << lane) - 1u)), num = 0, first = incl - mine, tasks = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const int x = s_num[w];
      at += w < warp ? x & 63 : 0;
      num += x & 63;
      first += w < warp ? x >> 6 : 0;
      tasks += x >> 6;
    }
    if (e0.x != 0) {
      e0.x = b0 + tid;
      s_meta[at][0] = e0;
      s_meta[at][1] = e1;
      s_first[at] = first;
    }
    __syncthreads();
    int wr = 1;  // warps that share a task
    while (wr < kJoinWarps && 2ll * wr * tasks <= (long long)gridDim.x * kJoinWarps) wr *= 2;
    const int per = kJoinWarps / wr, slice = warp % wr;  // tasks a block takes at a time
    for (int task0 = blockIdx.x * per; task0 < tasks; task0 += gridDim.x * per) {
      const int task = min(task0 + warp / wr, tasks - 1);
      int unit = 0;
      for (int hi = num - 1; unit < hi;) {  // the entry that the task belongs to
        const int mid = (unit + hi + 1) >> 1;
        if (s_first[mid] <= task) unit = mid; else hi = mid - 1;
      }
      const int4 meta = s_meta[unit][0], meta2 = s_meta[unit][1];
      const int b = meta.x, P = meta.y - b + 2, seq0 = meta.z, g = meta.w, tok0 = meta2.x, L = meta2.y;
      const int cg = (task - s_first[unit]) & 7, row = ((task - s_first[unit]) >> 3) * 32 + lane;
      const int half = row >> 7, r = row & 127, tok = tok0 + half * TT + r / G;
      const bool in = task0 + warp / wr < tasks && r < TT * G && tok < L;
      float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = 0.f;
      // pieces slice, slice + wr, ...
      for (int k0 = in ? slice : P; k0 < P; k0 += kJoinBatch * wr) {
        float2 ml[kJoinBatch];
        float4 o[kJoinBatch][4];
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
          ml[j] = make_float2(-INFINITY, 0.f);
          const int k = k0 + j * wr;
          if (k < P) {
            const long long part0 = (2ll * (b - 1 + k) + (k == 0)) * 2 + half;
            ml[j] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + part0 * 128 + r);
            const float* src = p.part_o + ((part0 * (kHeadDim / 8) + 2 * cg) * 128 + r) * 8;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[j][e] = __ldcg(reinterpret_cast<const float4*>(src + (e >> 1) * 128 * 8) + (e & 1));
          }
        }
        float mn = m;
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) mn = fmaxf(mn, ml[j].x);
        const float mu = mn == -INFINITY ? 0.f : mn, a = ex2_approx(m - mu);
        l *= a;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= a;
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j)
          if (ml[j].y != 0.f) {  // sum 0: nothing of the row in this piece, and its O may be unwritten
            const float w = ex2_approx(ml[j].x - mu);
            l += w * ml[j].y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[4 * e] += w * o[j][e].x;
              acc[4 * e + 1] += w * o[j][e].y;
              acc[4 * e + 2] += w * o[j][e].z;
              acc[4 * e + 3] += w * o[j][e].w;
            }
          }
        m = mn;
      }
      if (wr > 1) {
        s_acc[warp][0][lane] = m;
        s_acc[warp][1][lane] = l;
#pragma unroll
        for (int e = 0; e < 16; ++e) s_acc[warp][2 + e][lane] = acc[e];
        __syncthreads();
        if (slice == 0) {
          float mt = m;
          for (int q = 1; q < wr; ++q) mt = fmaxf(mt, s_acc[warp + q][0][lane]);
          const float mu = mt == -INFINITY ? 0.f : mt, a = ex2_approx(m - mu);
          l *= a;
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] *= a;
          for (int q = 1; q < wr; ++q) {
            const float w = ex2_approx(s_acc[warp + q][0][lane] - mu);
            l += w * s_acc[warp + q][1][lane];
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] += w * s_acc[warp + q][2 + e][lane];
          }
          m = mt;
        }
        __syncthreads();
      }
      if (!in || slice != 0) continue;
      const bool any = l > 0.f || l != l;
      const float inv = any ? 1.f / l : 0.f;
      const long long t = (long long)seq0 + tok;
      const int h = g * G + r % G;
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      uint16_t* dst = p.out + (t * c.hq + h) * kHeadDim + 16 * cg;
      if (p.out32) {
        st_global_v8(dst, w);
      } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if (cg == 0) {
        const float z = any ? (m == -INFINITY ? 0.f : m) + log2f(l) : -INFINITY;
        const long long place = (long long)h * c.total_tokens + t;
        if (p.lse2) p.lse2[place] = any ? -z : -INFINITY;  // as in a whole unit
        if (p.lse) p.lse[place] = z * 0.6931471805599453f;
      }
    }
  }
}

}  // namespace tiles

cudaError_t launch_cache_tiles(const CacheAttnParams& p, int sms, cudaStream_t st) {
  static unsigned long long attr[2][kMaxCachedDevices] = {};
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(tiles::cache_tiles_kernel), tiles::smem_bytes(kMaxSeqs), attr[0]);
  if (e == cudaSuccess)
    e = set_max_smem_carveout(reinterpret_cast<const void*>(tiles::cache_tiles_join_kernel), 0, attr[1]);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tiles::cache_tiles_kernel, dim3(sms), tiles::kThreads, tiles::smem_bytes(p.c.num_seqs), st, p);
  if (e != cudaSuccess || sms < 2) return e;
  return launch_pdl(tiles::cache_tiles_join_kernel, dim3(2 * sms), tiles::kJoinThreads, 0, st, p, sms);
}

}  // namespace fp
