// fp_cache_attn.cu -- attention of new tokens over a paged key/value cache, with the attention weight
// that every cached slot collects: the schedule for few rows (single tokens, short drafts) with the join of
// its split units, and the entry that picks a schedule.
//
//   o_th = sum_u p_thu v_u,  p_thu = exp(scale q_th . k_u - lse_th),  u <= lens[s] + t
//   w_ug = decay * w_ug + sum_{t, h in group g} p_thu
//
// Bound by reading K and V once: a unit is one (sequence, kv-head) with all its rows (row r: token r / G,
// q-head r % G of the group), 8 NT of them at most, and its keys are cut into tiles of 64. All tiles of all
// units form one line that the CTAs share out evenly, whatever the lengths: a CTA's share may begin or end
// inside a unit, and the pieces of such a unit are joined from the workspace by a second kernel. Every
// warp takes 16 keys of a tile with its own ring of cp.async stages, its own running maximum, row sum and
// accumulator, so warps never wait for one another inside a unit. (A loop of the same copies alone takes 80 us for
// 537 MB on this GPU, in any order of the heads; this kernel takes 92 us for them, 4 of which find the share.)
//
// The products are formed transposed, keys and columns along the 16-row side of the matrix instruction and the
// unit's rows along its 8-column side (S^T = K Q^T, O^T = V^T P^T): with the four rows of a token over
// a group of four heads that halves the instructions and the accumulator registers.
#include <cmath>

#include "fp_cache.cuh"

namespace fp {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowsMax = 32;                // rows of a unit
constexpr int kKeysW = 16;                  // keys of a tile per warp
constexpr int kWarps = 4, kRowThreads = 32 * kWarps;
constexpr int kKeysT = kKeysW * kWarps;     // keys of a tile
constexpr int kStageBytes = 2 * kKeysW * kHeadDim * 2;  // K then V of one warp's 16 keys
// Up to 16 rows: twelve warps an SM with two stages each, Q in registers (fewer warps leave the schedulers waiting).
// Up to 32: the accumulators take the registers of eight warps, with three stages, and Q stays in shared memory.
constexpr int stages(int nt) { return nt <= 2 ? 2 : 3; }
constexpr int ctas_sm(int nt) { return nt <= 2 ? 3 : 2; }
constexpr bool q_shared(int nt) { return nt > 2; }
constexpr int row_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }  // of 8 rows: 1, 2 or 4 are built
constexpr int off_q(int nt) { return kWarps * stages(nt) * kStageBytes; }
constexpr int off_ml(int nt) { return off_q(nt) + (q_shared(nt) ? 8 * nt * 256 : 0); }  // float m[warp][32], l[warp][32]
constexpr int row_smem(int nt) { return off_ml(nt) + 2 * kWarps * kRowsMax * 4; }
static_assert(16 * kHeadDim * 4 <= kStageBytes, "a consumed stage holds 16 rows of the warp's result when a unit is joined");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {  // transposes an 8x8 matrix of 16-bit elements
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A place on the line.
struct Cursor {
  int s, g, kt;          // sequence, kv-head, tile
  int seq0, L, len, n;   // first new token, new tokens, slots before them, keys
  int kts;               // tiles of the sequence's units
};
__device__ __forceinline__ int unit_tiles(int L, int n) { return L > 0 ? (n + kKeysT - 1) / kKeysT : 0; }
__device__ __forceinline__ void load_seq(Cursor& u, const CacheInfo& c, int s) {
  u.s = s;
  u.seq0 = c.cu_seqlens[s];
  u.L = c.cu_seqlens[s + 1] - u.seq0;
  u.len = c.lens[s];
  u.n = u.len + u.L;
  u.kts = unit_tiles(u.L, u.n);
}
// Step to the next tile of the line. more: there is one.
__device__ __forceinline__ void cursor_next(Cursor& u, const CacheInfo& c, bool more) {
  if (++u.kt < u.kts || !more) return;
  u.kt = 0;
  if (++u.g < c.hkv) return;
  u.g = 0;
  int s = u.s;
  do load_seq(u, c, ++s);
  while (u.kts == 0 && s + 1 < c.num_seqs);
}
// Every warp by itself: lane i sums the tiles of a contiguous run of sequences, a scan gives the total, and
// the lane whose run holds the start of share `me` walks it. No shared memory and no barrier: this
// chain is most of what a short call waits for. The device arrays are checked against the host's
// description here, before any other access depends on them.
__device__ __forceinline__ bool find_share(const CacheInfo& c, Shares& sh, Cursor& u, int me, int parts, long long max_tiles,
                                           int32_t* dev_status) {
  const int lane = threadIdx.x & 31, S = c.num_seqs, per = (S + 31) / 32;
  const int a = min(S, lane * per), b = min(S, a + per);
  long long sum = 0;
  bool bad = lane == 0 && (c.cu_seqlens[0] != 0 || c.cu_seqlens[S] != c.total_tokens);
#pragma unroll 4
  for (int s = a; s < b; ++s) {
    const int lo = c.cu_seqlens[s], hi = c.cu_seqlens[s + 1], len = c.lens[s];
    const bool ok = lo >= 0 && hi >= lo && hi <= c.total_tokens && hi - lo <= c.max_new && len >= 0 &&
                    len <= c.max_len - (hi - lo);
    bad |= !ok;
    if (ok) sum += (long long)c.hkv * unit_tiles(hi - lo, len + hi - lo);
  }
  if (__any_sync(kAll, bad)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) dev_flag(dev_status, kDevBadProblem);
    return false;
  }
  const long long incl = warp_incl_scan(sum), total = __shfl_sync(kAll, incl, 31);
  if (total > max_tiles) {  // more tiles than the workspace has scores for: sequences share pages
    if (threadIdx.x == 0 && blockIdx.x == 0) dev_flag(dev_status, kDevBadProblem);
    return false;
  }
  sh = Shares(total, parts);
  if (me >= sh.parts) return false;
  const long long x0 = sh.at(me);
  const bool mine = incl - sum <= x0 && x0 < incl;
  if (mine) {
    long long left = x0 - (incl - sum);
    for (int s = a;; ++s) {
      load_seq(u, c, s);
      const long long tiles = (long long)c.hkv * u.kts;
      if (left < tiles) break;
      left -= tiles;
    }
    u.g = left < 0x7fffffffll ? (int)((unsigned)left / (unsigned)u.kts) : (int)(left / u.kts);
    u.kt = (int)(left - (long long)u.g * u.kts);
  }
  const int src = __ffs(__ballot_sync(kAll, mine)) - 1;
  u.s = __shfl_sync(kAll, u.s, src);
  u.g = __shfl_sync(kAll, u.g, src);
  u.kt = __shfl_sync(kAll, u.kt, src);
  u.seq0 = __shfl_sync(kAll, u.seq0, src);
  u.L = __shfl_sync(kAll, u.L, src);
  u.len = __shfl_sync(kAll, u.len, src);
  u.n = u.len + u.L;
  u.kts = unit_tiles(u.L, u.n);
  return true;
}

template <int NT>
__global__ void __launch_bounds__(kRowThreads, ctas_sm(NT)) cache_rows_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int kStages = stages(NT);
  constexpr bool kQs = q_shared(NT);
  extern __shared__ __align__(1024) unsigned char smem[];
  pdl_wait();
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Shares sh;
  Cursor cur;
  int32_t* meta = p.meta + (long long)blockIdx.x * kMetaWords;
  const bool work = find_share(c, sh, cur, blockIdx.x, gridDim.x, p.scores ? p.score_tiles : 0x7fffffffffffffffll, p.dev_status);
  pdl_trigger();
  if (!work) {
    if (tid == 0) meta[0] = 0;
    return;
  }
  const int me = blockIdx.x;
  const long long x0 = sh.at(me), x1 = sh.at(me + 1);
  Cursor ld = cur;
  if (tid == 0) {
    const long long unit0 = x0 - cur.kt, end = unit0 + cur.kts;  // the unit that the share begins in
    meta[0] = cur.kt > 0 && sh.at(me - 1) <= unit0;  // its first CTA but one: its pieces are joined in its name
    if (cur.kt > 0) {
      int last = me;  // the last CTA whose share begins inside the unit
      while (last + 1 < sh.parts && sh.at(last + 1) < end) ++last;
      meta[1] = last;
      meta[2] = cur.seq0;
      meta[3] = cur.g;
      meta[4] = 0;
      meta[5] = cur.L * c.group;
    }
  }
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  // ---- loads: tile x of the line into stage (x - x0) % kStages. The page of a tile is looked up one tile ahead.
  auto row_of = [&](const Cursor& u) -> long long {
    const int key0 = u.kt * kKeysT + warp * kKeysW;  // pages hold whole groups of 16 slots
    return key0 < u.n ? slot_row(c, u.s, key0) : -1;
  };
  long long row0 = row_of(ld);
  int put = 0;
  // a lane copies 16 bytes of rows lane / 16, + 2, ...; its places in a stage (128-byte swizzle)
  const long long lane_off = (long long)(lane >> 4) * c.hkv * kHeadDim + (lane & 15) * 8;
  const long long row_step = 2ll * c.hkv * kHeadDim;
  uint32_t put_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) put_off[i] = (lane >> 4) * 256 + (((lane & 15) ^ (2 * i + (lane >> 4))) << 4);
  auto load = [&](long long x) {
    if (x < x1) {
      const uint32_t st = ring + (uint32_t)put * kStageBytes;
      put = put + 1 == kStages ? 0 : put + 1;
      const int key0 = ld.kt * kKeysT + warp * kKeysW;
      if (key0 < ld.n && row0 < 0 && lane == 0) dev_flag(p.dev_status, kDevBadProblem);
      // a bad page and the slots past the sequence's end read as zeros
      const int live = row0 < 0 ? 0 : min(kKeysW, ld.n - key0);
      const long long base = ((row0 < 0 ? 0 : row0) * c.hkv + ld.g) * kHeadDim;
      if (live == kKeysW) {
        const uint16_t *ks = c.k + base + lane_off, *vs = c.v + base + lane_off;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cp_async16(st + i * 512 + put_off[i & 3], ks, true);
          cp_async16(st + i * 512 + put_off[i & 3] + kKeysW * 256, vs, true);
          ks += row_step;
          vs += row_step;
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int r = 2 * i + (lane >> 4);
          const long long off = r < live ? base + (long long)r * c.hkv * kHeadDim + (lane & 15) * 8 : 0;
          const uint32_t d = st + r * 256 + (((lane & 15) ^ (r & 7)) << 4);
          cp_async16(d, c.k + off, r < live);
          cp_async16(d + kKeysW * 256, c.v + off, r < live);
        }
      }
      cursor_next(ld, c, x + 1 < x1);
      if (x + 1 < x1) row0 = row_of(ld);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(x0 + i);

  uint32_t qf[kQs ? 1 : NT][8][2];
  // m: the reference maximum; mu: the same, 0 while the row has seen no key; thr: how far above mu a score may lie
  float o[8][NT][4], l[NT][2], m[NT][2], mu[NT][2], thr[NT][2];
  const int kr = lane >> 2, rc = (lane & 3) * 2;  // this thread's keys kr, kr + 8 and rows rc, rc + 1 (+ 8 t)
  float* s_m = reinterpret_cast<float*>(smem + off_ml(NT));
  float* s_l = s_m + kWarps * kRowsMax;
  // ldmatrix rows of this lane: K [key][column] as it lies, V transposed
  const int rk = (lane & 7) + (((lane >> 3) & 1) << 3), rv = (lane & 7) + ((lane >> 4) << 3);
  const uint32_t get_k = rk * 256 + (((lane >> 4) ^ (rk & 7)) << 4);
  const uint32_t get_v = rv * 256 + ((((lane >> 3) & 1) ^ (rv & 7)) << 4);
  // Q in shared memory: rows lane & 7 of two row tiles, both 8-column halves of a K step
  const int rq = ((lane >> 4) << 3) + (lane & 7);
  const uint32_t get_q = smem_u32(smem) + off_q(NT) + rq * 256 + ((((lane >> 3) & 1) ^ (rq & 7)) << 4);
  auto last_of = [&](int t, int i) { return cur.len + (8 * t + rc + i) / c.group; };  // the last key that a row sees
  bool fresh = true;
  int first_kt = 0, get = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
      first_kt = cur.kt;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
        l[t][0] = l[t][1] = 0.f;
        m[t][0] = m[t][1] = thr[t][0] = thr[t][1] = -INFINITY;
        mu[t][0] = mu[t][1] = 0.f;
        if (!kQs) {
          const int r = 8 * t + kr;
          const bool in = r < cur.L * c.group;
          const uint16_t* q0 = p.q + (long long)(cur.seq0 + (in ? r / c.group : 0)) * p.q_stride +
                               (cur.g * c.group + (in ? r % c.group : 0)) * kHeadDim + rc;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qf[kQs ? 0 : t][kk][0] = in ? *reinterpret_cast<const uint32_t*>(q0 + kk * 16) : 0u;
            qf[kQs ? 0 : t][kk][1] = in ? *reinterpret_cast<const uint32_t*>(q0 + kk * 16 + 8) : 0u;
          }
        }
      }
      if (kQs) {  // the last unit's join has ended for every warp
        for (int e = tid; e < 8 * NT * 16; e += kRowThreads) {
          const int r = e >> 4, ch = e & 15;
          uint4 y = make_uint4(0, 0, 0, 0);
          if (r < cur.L * c.group)
            y = reinterpret_cast<const uint4*>(p.q + (long long)(cur.seq0 + r / c.group) * p.q_stride +
                                               (cur.g * c.group + r % c.group) * kHeadDim)[ch];
          *reinterpret_cast<uint4*>(smem + off_q(NT) + r * 256 + ((ch ^ (r & 7)) << 4)) = y;
        }
        __syncthreads();
      }
    }
    load(x + kStages - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t sk = ring + (uint32_t)get * kStageBytes, sv = sk + kKeysW * 256;
    // S^T = K Q^T: 16 keys x 8 NT rows, in two chains
    float sc[NT][4];
    {
      float s2[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] = s2[t][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; kk += 2) {
        uint32_t a[4], b[4];
        ldsm4((sk + get_k) ^ (kk << 5), a);
        ldsm4((sk + get_k) ^ ((kk + 1) << 5), b);
        if (kQs) {
#pragma unroll
          for (int t = 0; t < NT; t += 2) {
            uint32_t q0[4], q1[4];
            ldsm4((get_q ^ (kk << 5)) + t * 8 * 256, q0);
            ldsm4((get_q ^ ((kk + 1) << 5)) + t * 8 * 256, q1);
            mma16816(sc[t], a, q0[0], q0[1]);
            mma16816(sc[t + 1], a, q0[2], q0[3]);
            mma16816(s2[t], b, q1[0], q1[1]);
            mma16816(s2[t + 1], b, q1[2], q1[3]);
          }
        } else {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816(sc[t], a, qf[kQs ? 0 : t][kk][0], qf[kQs ? 0 : t][kk][1]);
            mma16816(s2[t], b, qf[kQs ? 0 : t][kk + 1][0], qf[kQs ? 0 : t][kk + 1][1]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] += s2[t][e];
    }
    const int key0 = cur.kt * kKeysT + warp * kKeysW;
    // keys up to `len` are seen by every row; past it row r of token t sees keys up to len + t
    if (key0 + kKeysW - 1 > cur.len) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + kr + (e >> 1) * 8;
          if (key > last_of(t, e & 1) || key >= cur.n) sc[t][e] = -INFINITY;
        }
    }
    if (p.scores) {  // for the weights pass: [four rows][64 keys][4] of a tile, so that both sides go 128 bytes at a time
      float* dst = p.scores + (x * p.score_rows + rc / 4 * 4) * kKeysT + (warp * kKeysW + kr) * 4 + (rc & 2);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (8 * t + rc < p.score_rows) {
          *reinterpret_cast<float2*>(dst + 8 * t * kKeysT) = make_float2(sc[t][0] * p.scale_log2, sc[t][1] * p.scale_log2);
          *reinterpret_cast<float2*>(dst + 8 * t * kKeysT + 32) =
              make_float2(sc[t][2] * p.scale_log2, sc[t][3] * p.scale_log2);
        }
    }
    // the reference maximum follows only when a score passes it by 2^8 (any reference gives the same
    // quotient; 8 keeps every term finite and the sums exact enough in 32 bits)
    bool grow = false;
    float ex[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ex[t][e] = fmaf(sc[t][e], p.scale_log2, -mu[t][e & 1]);
        grow |= ex[t][e] > thr[t][e & 1];
      }
    if (__any_sync(kAll, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(sc[t][i], sc[t][2 + i]);
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
          const float mn = fmaxf(m[t][i], mx * p.scale_log2);
          const float a = mn == -INFINITY ? 1.f : ex2_approx(m[t][i] - mn);
          m[t][i] = mn;
          mu[t][i] = mn == -INFINITY ? 0.f : mn;
          thr[t][i] = mn == -INFINITY ? -INFINITY : 8.f;
          l[t][i] *= a;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j][t][i] *= a;
            o[j][t][2 + i] *= a;
          }
          ex[t][i] = fmaf(sc[t][i], p.scale_log2, -mu[t][i]);
          ex[t][2 + i] = fmaf(sc[t][2 + i], p.scale_log2, -mu[t][i]);
        }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float e0 = ex2_approx(ex[t][0]), e1 = ex2_approx(ex[t][1]);
      const float e2 = ex2_approx(ex[t][2]), e3 = ex2_approx(ex[t][3]);
      l[t][0] += e0 + e2;
      l[t][1] += e1 + e3;
      // the tensor cores take bf16 (half a step is 2^-9 of each term); [key][row] becomes [row][key]
      pf[t][0] = movmatrix(pack_bf16x2(e0, e1));
      pf[t][1] = movmatrix(pack_bf16x2(e2, e3));
    }
    // 0 * NaN is NaN, so what is masked has to be finite in V as well: non-finite values of new tokens go to the
    // rows that see them by themselves (p > 0) and become zeros for the product
    if (cur.L > 1 && key0 + kKeysW - 1 > cur.len) {
      unsigned char* v = smem + (sv - smem_u32(smem));
      bool any = false;
#pragma unroll 1
      for (int e = lane; e < kKeysW * 16; e += 32) {
        const uint4 y = *reinterpret_cast<const uint4*>(v + e * 16);
        any |= nonfinite2(y.x) || nonfinite2(y.y) || nonfinite2(y.z) || nonfinite2(y.w);
      }
      if (__any_sync(kAll, any)) {
        for (int k = 0; k < kKeysW; ++k)
#pragma unroll
          for (int j = 0; j < 16; ++j) {  // this thread's columns 8 j + kr: accumulators [j / 2][.][2 (j & 1)], [.. + 1]
            const uint32_t y = *reinterpret_cast<const uint16_t*>(v + k * 256 + ((j ^ (k & 7)) << 4) + kr * 2);
            if ((y & 0x7f80) != 0x7f80) continue;
            const float f = __uint_as_float(y << 16);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (key0 + k <= last_of(t, i)) o[j >> 1][t][2 * (j & 1) + i] += f;
          }
        __syncwarp();
        for (int e = lane; e < kKeysW * kHeadDim; e += 32) {
          uint16_t* y = reinterpret_cast<uint16_t*>(v) + e;
          if ((*y & 0x7f80) == 0x7f80) *y = 0;
        }
        __syncwarp();
      }
    }
    {  // O^T += V^T P^T: 16 columns at a time
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t a[4];
        ldsm4t((sv + get_v) ^ (j << 5), a);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[j][t], a, pf[t][0], pf[t][1]);
      }
    }
    __syncwarp();  // every lane has read the stage before it is loaded again
    const bool ends = cur.kt + 1 == cur.kts;
    if (ends || x + 1 == x1) {
      // ---- the unit's piece is complete: join the warps through the stages that they have just consumed
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[t][i] += __shfl_xor_sync(kAll, l[t][i], 4);
          l[t][i] += __shfl_xor_sync(kAll, l[t][i], 8);
          l[t][i] += __shfl_xor_sync(kAll, l[t][i], 16);
          if (kr == 0) {
            s_m[warp * kRowsMax + 8 * t + rc + i] = m[t][i];
            s_l[warp * kRowsMax + 8 * t + rc + i] = l[t][i];
          }
        }
      __syncthreads();
      float* s_o = reinterpret_cast<float*>(smem + (sk - smem_u32(smem)));  // [row of 16][128], columns swizzled
      const bool whole = ends && first_kt == 0;
      const long long slot = 2ll * blockIdx.x + (first_kt == 0 ? 1 : 0);  // a piece from a unit's start: place 1
#pragma unroll
      for (int r0 = 0; r0 < 8 * NT; r0 += 16) {
#pragma unroll
        for (int t = r0 / 8; t < NT && t < r0 / 8 + 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * t + rc + i;
            float mt = s_m[r];
            for (int k = 1; k < kWarps; ++k) mt = fmaxf(mt, s_m[k * kRowsMax + r]);
            const float w = ex2_approx(m[t][i] - (mt == -INFINITY ? 0.f : mt));
            const int swz = ((r >> 1) & 3) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              s_o[(r - r0) * kHeadDim + ((16 * j + kr) ^ swz)] = o[j][t][i] * w;
              s_o[(r - r0) * kHeadDim + ((16 * j + 8 + kr) ^ swz)] = o[j][t][2 + i] * w;
            }
          }
        __syncthreads();
        // thread: four columns of every fourth row
        const int cc = lane * 4;
        for (int r = r0 + warp; r < min(r0 + 16, cur.L * c.group); r += kWarps) {
          float mt = s_m[r];
          for (int k = 1; k < kWarps; ++k) mt = fmaxf(mt, s_m[k * kRowsMax + r]);
          const float mu_r = mt == -INFINITY ? 0.f : mt;
          float lt = 0.f;
          for (int k = 0; k < kWarps; ++k) lt += s_l[k * kRowsMax + r] * ex2_approx(s_m[k * kRowsMax + r] - mu_r);
          const float* src = reinterpret_cast<const float*>(smem + get * kStageBytes) + (r - r0) * kHeadDim +
                             (cc ^ (((r >> 1) & 3) * 8));
          float4 a = *reinterpret_cast<const float4*>(src);
          for (int k = 1; k < kWarps; ++k) {
            const float4 b = *reinterpret_cast<const float4*>(src + k * (kStages * kStageBytes / 4));
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
          }
          if (!whole) {
            *reinterpret_cast<float4*>(p.part_o + (slot * kRowsMax + r) * kHeadDim + cc) = a;
            if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * (slot * kRowsMax + r)) = make_float2(mt, lt);
          } else {
            const bool any = lt > 0.f || lt != lt;
            const float inv = any ? 1.f / lt : 0.f;
            const long long t = (long long)cur.seq0 + r / c.group;
            const int h = cur.g * c.group + r % c.group;
            *reinterpret_cast<uint2*>(p.out + (t * c.hq + h) * kHeadDim + cc) =
                make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
            if (lane == 0) {
              const float z = any ? mu_r + log2f(lt) : -INFINITY;
              const long long at = (long long)h * c.total_tokens + t;
              if (p.lse2) p.lse2[at] = z;
              if (p.lse) p.lse[at] = z * 0.6931471805599453f;
            }
          }
        }
        __syncthreads();
      }
      fresh = true;
    }
    get = get + 1 == kStages ? 0 : get + 1;
    cursor_next(cur, c, x + 1 < x1);
  }
  cp_async_wait<0>();
}

// Weights of the few-row schedule, from the scores that it left in the workspace (a hundredth of the
// bytes of K): the line of tiles again, shared out over the warps; a lane takes keys lane and lane + 32 of a tile.
__global__ void __launch_bounds__(256) cache_rows_weights_kernel(const __grid_constant__ CacheAttnParams p) {
  pdl_wait();
  const CacheInfo& c = p.c;
  Shares sh;
  Cursor u;
  const int me = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31, rs = p.score_rows;
  if (!find_share(c, sh, u, me, gridDim.x * (blockDim.x >> 5), p.score_tiles, nullptr)) return;
  const long long x0 = sh.at(me), x1 = sh.at(me + 1);
  float z = 0.f;  // lane r: lse2 of the unit's row r
  int s = -1, g = -1;
  for (long long x = x0; x < x1; ++x, cursor_next(u, c, x < x1)) {
    const int rows = u.L * c.group;
    if (u.s != s || u.g != g) {
      s = u.s;
      g = u.g;
      z = lane < rows ? __ldcg(p.lse2 + (long long)(g * c.group + lane % c.group) * c.total_tokens + u.seq0 +
                               lane / c.group)
                      : INFINITY;
      if (z == -INFINITY) z = INFINITY;  // a row without a finite score: 2^(-inf - z) is to be 0, not NaN
    }
    const float4* sc = reinterpret_cast<const float4*>(p.scores) + x * (rs / 4) * kKeysT + lane;
    long long at[2];
    int rmin[2];  // the first row that sees the key: masked scores are -inf, but a row's lse may be NaN
    float old[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = u.kt * kKeysT + 32 * i + lane;
      rmin[i] = max(key - u.len, 0) * c.group;
      at[i] = key < u.n ? slot_word(c, s, g, key) : -1;  // a bad page was flagged by the attention
      if (at[i] >= 0 && p.decay > 0.f) old[i] = c.weights[at[i]];
    }
#pragma unroll 2
    for (int r = 0; r < rows; r += 4, sc += kKeysT) {
      float zr[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) zr[j] = __shfl_sync(kAll, z, r + j);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = __ldcg(sc + 32 * i);
        if (r >= rmin[i]) w[i] += ex2_approx(v.x - zr[0]);
        if (r + 1 < rows && r + 1 >= rmin[i]) w[i] += ex2_approx(v.y - zr[1]);
        if (r + 2 < rows && r + 2 >= rmin[i]) w[i] += ex2_approx(v.z - zr[2]);
        if (r + 3 < rows && r + 3 >= rmin[i]) w[i] += ex2_approx(v.w - zr[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at[i] >= 0) c.weights[at[i]] = p.decay > 0.f ? fmaf(p.decay, old[i], w[i]) : w[i];
  }
}

// Joins the pieces of the units that several CTAs share. Entry b of meta describes the unit inside of which
// the share of CTA b begins and is set for the first such CTA of a unit: the unit's pieces are then the last
// one of CTA b - 1 (place 1) and the first one (place 0) of every CTA from b to meta[1].
// The time is one chain of dependent reads (meta, maxima, accumulators), so the work is laid out flat: every
// block lists the set entries, and the rows of all listed units go round the grid's warps, 32 maxima at
// once; where there are fewer rows than warps, up to 16 warps of a block share a row's pieces.
constexpr int kJoinWarps = 16, kJoinUnits = 512;
__global__ void __launch_bounds__(32 * kJoinWarps) cache_join_kernel(const __grid_constant__ CacheAttnParams p, int ctas) {
  __shared__ float4 s_acc[kJoinWarps][32];
  __shared__ int4 s_meta[kJoinUnits][2];  // set entries; word 0: the CTA
  __shared__ int s_num[kJoinWarps];
  pdl_wait();
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = c.group;
  for (int b0 = 0; b0 < ctas; b0 += kJoinUnits) {  // one round on devices of up to 256 SMs
    __syncthreads();
    int4 e0 = make_int4(0, 0, 0, 0), e1 = e0;
    if (b0 + tid < ctas) {
      const int4* src = reinterpret_cast<const int4*>(p.meta + (long long)(b0 + tid) * kMetaWords);
      e0 = __ldcg(src);
      e1 = __ldcg(src + 1);
    }
    const unsigned set = __ballot_sync(kAll, e0.x != 0);
    if (lane == 0) s_num[warp] = __popc(set);
    __syncthreads();
    int at = __popc(set & ((1u << lane) - 1u)), num = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const int x = s_num[w];
      at += w < warp ? x : 0;
      num += x;
    }
    const int tasks = num * min(kRowsMax, c.max_new * G);
    if (e0.x != 0) {
      e0.x = b0 + tid;
      s_meta[at][0] = e0;
      s_meta[at][1] = e1;
    }
    __syncthreads();
    if (num == 0) continue;
    int wr = 1;  // warps that share a row
    while (wr < kJoinWarps && 2ll * wr * tasks <= (long long)gridDim.x * kJoinWarps) wr *= 2;
    const int per = kJoinWarps / wr, slice = warp % wr;  // rows a block takes at a time
    for (int task0 = blockIdx.x * per; task0 < tasks; task0 += gridDim.x * per) {
      const int task = task0 + warp / wr;
      // rows outermost: the rows that no unit has come last
      const int row = task / num, unit = task < tasks ? task - row * num : 0;
      const int4 meta = s_meta[unit][0], meta2 = s_meta[unit][1];
      // meta2: first packed row and packed rows
      const int b = meta.x, P = meta.y - b + 2, seq0 = meta.z, g = meta.w;
      const int pr = meta2.x + row, tok = pr / G, head = pr % G;
      const bool in = task < tasks && pr < meta2.y;
      float l = 0.f, mu = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in) {
        auto place = [&](int k) { return (2ll * (b - 1 + k) + (k == 0)) * kRowsMax + row; };
        auto ml_of = [&](int k) {
          return k < P ? __ldcg(reinterpret_cast<const float2*>(p.part_ml + 2 * place(k))) : make_float2(-INFINITY, 0.f);
        };
        const float2 ml0 = ml_of(lane);
        float m = ml0.x;
        for (int k = lane + 32; k < P; k += 32) m = fmaxf(m, ml_of(k).x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        mu = m == -INFINITY ? 0.f : m;
        for (int k0 = 0; k0 < P; k0 += 32) {
          const float2 ml = k0 == 0 ? ml0 : ml_of(k0 + lane);
          const float w = ml.y != 0.f ? ex2_approx(ml.x - mu) : 0.f;  // sum 0: nothing of the row in this piece
          if (ml.y != 0.f) l += w * ml.y;
          const unsigned use = __ballot_sync(kAll, ml.y != 0.f);      // its O may be unwritten
          const int top = min(32, P - k0);
#pragma unroll 8
          for (int j = slice; j < top; j += wr) {
            const float wj = __shfl_sync(kAll, w, j);
            if ((use >> j) & 1) {
              const float4 a = __ldcg(reinterpret_cast<const float4*>(p.part_o + place(k0 + j) * kHeadDim) + lane);
              acc.x += wj * a.x; acc.y += wj * a.y; acc.z += wj * a.z; acc.w += wj * a.w;
            }
          }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
      }
      if (wr > 1) {
        s_acc[warp][lane] = acc;
        __syncthreads();
        if (slice == 0)
          for (int q = 1; q < wr; ++q) {
            const float4 a = s_acc[warp + q][lane];
            acc.x += a.x; acc.y += a.y; acc.z += a.z; acc.w += a.w;
          }
        __syncthreads();
      }
      if (!in || slice != 0) continue;
      const bool any = l > 0.f || l != l;
      const float inv = any ? 1.f / l : 0.f;
      const long long t = (long long)seq0 + tok;
      const int h = g * G + head;
      *reinterpret_cast<uint2*>(p.out + (t * c.hq + h) * kHeadDim + lane * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (lane == 0) {
        const float z = any ? mu + log2f(l) : -INFINITY;
        if (p.lse2) p.lse2[(long long)h * c.total_tokens + t] = z;
        if (p.lse) p.lse[(long long)h * c.total_tokens + t] = z * 0.6931471805599453f;
      }
    }
  }
}

}  // namespace

// Few rows: up to 32 packed rows a sequence. Where both schedules run, at 32 q-heads over 8 kv-heads, the call takes
// (this one / the 128-row one, us): one sequence of 2K keys, 4 rows 10.5 / 19.0, 16 rows 13.8 / 19.7, 32 rows 15.5 / 21.2;
// 32K keys, 16 rows 35.6 / 46.0, 32 rows 45.3 / 52.0; with weights 45.3 / 73.0 and 62.1 / 79.1; 32 sequences of 4K, 16 rows 97.9 /
// 105.1, 32 rows 109.5 / 106.6.
bool cache_attn_tiled(int32_t max_new, int32_t group) { return (int64_t)max_new * group > kRowsMax; }

CacheAttnLayout cache_attn_layout(int sms, bool tiled, const CacheInfo& c, bool scores) {
  auto up = [](int64_t x) { return (x + 255) & ~(int64_t)255; };
  const int64_t grid = tiled ? sms : ctas_sm(row_tiles((int64_t)c.max_new * c.group)) * sms;
  const int64_t rows = 2 * grid * (tiled ? 2 * kTileM : kRowsMax);
  CacheAttnLayout w;
  w.part_o = 0;
  w.part_ml = up(w.part_o + rows * kHeadDim * 4);
  w.meta = up(w.part_ml + rows * 2 * 4);
  w.lse2 = up(w.meta + grid * kMetaWords * 4);
  w.scores = up(w.lse2 + (int64_t)c.hq * c.total_tokens * 4);
  w.score_rows = (c.max_new * c.group + 3) / 4 * 4;
  // tiles of a call that writes weights: by the longest sequence that there may be, and by the pages, which no
  // two sequences share then
  const int64_t by_len = (int64_t)c.num_seqs * ((c.max_len + kKeysT - 1) / kKeysT);
  const int64_t by_page = ((int64_t)c.num_pages * c.page_size + kKeysT - 1) / kKeysT + c.num_seqs;
  w.score_tiles = (by_len < by_page ? by_len : by_page) * c.hkv;
  w.total = tiled || !scores ? w.scores : up(w.scores + w.score_tiles * kKeysT * w.score_rows * 4);
  return w;
}

// Every kernel of a call asks for the same split of the SM's memory (the largest shared part): between
// kernels that differ in it the SM has to drain first, which costs microseconds.
cudaError_t launch_cache_attn(const CacheAttnParams& p, bool tiled, int sms, cudaStream_t st) {
  static unsigned long long attr[2][kMaxCachedDevices] = {}, attr_rows[5][kMaxCachedDevices] = {};
  cudaError_t e;
  if (tiled) {
    if ((e = launch_cache_tiles(p, sms, st)) != cudaSuccess || !(p.decay >= 0.f)) return e;
    return launch_cache_weights(p, sms, st);
  }
  const int nt = row_tiles((int64_t)p.c.max_new * p.c.group), grid = ctas_sm(nt) * sms;
  void (*fn)(const CacheAttnParams) = nt == 1 ? cache_rows_kernel<1> : nt == 2 ? cache_rows_kernel<2> : cache_rows_kernel<4>;
  if ((e = set_max_smem_carveout(reinterpret_cast<const void*>(fn), row_smem(nt), attr_rows[nt])) != cudaSuccess) return e;
  if ((e = launch_pdl(fn, dim3(grid), kRowThreads, row_smem(nt), st, p)) != cudaSuccess) return e;
  if ((e = set_max_smem_carveout(reinterpret_cast<const void*>(cache_join_kernel), 0, attr[0])) != cudaSuccess) return e;
  e = launch_pdl(cache_join_kernel, dim3(sms), 32 * kJoinWarps, 0, st, p, grid);
  if (e != cudaSuccess || !(p.decay >= 0.f)) return e;
  if ((e = set_max_smem_carveout(reinterpret_cast<const void*>(cache_rows_weights_kernel), 0, attr[1])) != cudaSuccess)
    return e;
  return launch_pdl(cache_rows_weights_kernel, dim3(4 * sms), 256, 0, st, p);
}

}  // namespace fp
