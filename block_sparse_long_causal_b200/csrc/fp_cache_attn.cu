// fp_cache_attn.cu -- attention of new tokens over a paged key/value cache, with the attention weight
// that every cached slot collects.
//
//   o_th = sum_u p_thu v_u,  p_thu = exp(scale q_th . k_u - lse_th),  u <= lens[s] + t
//   w_ug = decay * w_ug + sum_{t, h in group g} p_thu
//
// A unit is 16 packed rows (token-major: row r is token r / G, q-head r % G of the group) of one
// (sequence, kv-head); its keys are cut into tiles of 64. All tiles of all units form one line that
// the CTAs share out evenly, whatever the lengths: a CTA's range may begin or end inside a unit, and the
// pieces of such a unit are joined from the workspace by a second kernel. Every warp takes 16 keys of a
// tile with its own ring of cp.async stages, its own running maximum, row sum and accumulator, so warps
// never wait for one another inside a unit.
#include <cmath>

#include "fp_cache.cuh"

namespace fp {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowsT = 16;                  // packed rows of a unit
constexpr int kKeysW = 16;                  // keys of a tile per warp
constexpr int kWarps = 4, kRowThreads = 32 * kWarps;
constexpr int kKeysT = kKeysW * kWarps;     // keys of a tile
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kKeysW * kHeadDim * 2;  // K then V of one warp's 16 keys
constexpr int kJoinCols = 32;               // output columns joined at a time
constexpr int kOffJoin = kWarps * kStages * kStageBytes;
constexpr int kOffMl = kOffJoin + kWarps * kRowsT * kJoinCols * 4;  // float m[warp][16], l[warp][16]
constexpr int kOffTabR = kOffMl + 2 * kWarps * kRowsT * 4 + 64;
constexpr int row_smem(int S) { return kOffTabR + 8 * (S + 1); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A unit and the tile of it that a cursor stands on.
struct Cursor {
  int s, g, rt;          // sequence, kv-head, row tile
  int seq0, L, len, n;   // first new token, new tokens, slots before them, keys
  int rts, kts;          // row tiles, key tiles of the sequence's units
  int kt;                // tile
  long long unit0;       // line position of the unit's first tile
};
__device__ __forceinline__ void load_seq(Cursor& u, const CacheInfo& c, int s) {
  u.s = s;
  u.seq0 = __ldg(c.cu_seqlens + s);
  u.L = __ldg(c.cu_seqlens + s + 1) - u.seq0;
  u.len = c.lens[s];
  u.n = u.len + u.L;
  u.rts = (u.L * c.group + kRowsT - 1) / kRowsT;
  u.kts = (u.n + kKeysT - 1) / kKeysT;
}
__device__ __forceinline__ Cursor cursor_at(const CacheInfo& c, const long long* tab, long long x) {
  Cursor u;
  load_seq(u, c, find_seq64(tab, c.num_seqs, x));
  const long long local = x - tab[u.s];
  const long long unit = local / u.kts;
  u.kt = (int)(local - unit * u.kts);
  u.g = (int)(unit / u.rts);
  u.rt = (int)(unit - (long long)u.g * u.rts);
  u.unit0 = x - u.kt;
  return u;
}
// Step to the next tile of the line; more: there is one.
__device__ __forceinline__ void cursor_next(Cursor& u, const CacheInfo& c, const long long* tab, bool more) {
  if (++u.kt < u.kts || !more) return;
  u.kt = 0;
  u.unit0 += u.kts;
  if (++u.rt < u.rts) return;
  u.rt = 0;
  if (++u.g < c.hkv) return;
  u.g = 0;
  load_seq(u, c, find_seq64(tab, c.num_seqs, u.unit0));
}

__global__ void __launch_bounds__(kRowThreads, 2) cache_rows_kernel(const __grid_constant__ CacheAttnParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long* tab = reinterpret_cast<long long*>(smem + kOffTabR);
  long long* s_scan = reinterpret_cast<long long*>(smem + kOffMl);  // before the ring is used
  int* s_bad = reinterpret_cast<int*>(smem + kOffMl + 64);
  const bool ok = cache_table<kRowThreads>(c, tab, s_scan, s_bad, p.dev_status, [&](int, int L, int n) -> long long {
    return (long long)c.hkv * ((L * c.group + kRowsT - 1) / kRowsT) * ((n + kKeysT - 1) / kKeysT);
  });
  pdl_trigger();
  const long long total = ok ? tab[c.num_seqs] : 0;
  const int ctas = (int)min((long long)gridDim.x, total);  // CTAs with work: every one has a tile
  const int me = blockIdx.x;
  const long long x0 = me < ctas ? total * me / ctas : 0, x1 = me < ctas ? total * (me + 1) / ctas : 0;
  int32_t* meta = p.meta + (long long)blockIdx.x * kMetaWords;
  if (x0 >= x1) {
    if (tid == 0) meta[0] = 0;
    return;
  }
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  Cursor ld = cursor_at(c, tab, x0);
  Cursor cur = ld;
  if (tid == 0) {
    // a range that begins inside a unit: its first CTA but one joins the unit's pieces
    const bool inside = cur.kt > 0;
    const long long prev0 = me > 0 ? total * (me - 1) / ctas : 0;
    meta[0] = inside && prev0 <= cur.unit0;
    if (inside) {
      // the last CTA whose range begins inside the unit
      const long long end = cur.unit0 + cur.kts;
      int last = me;
      while (last + 1 < ctas && total * (last + 1) / ctas < end) ++last;
      meta[1] = last;
      meta[2] = cur.seq0;
      meta[3] = cur.g;
      meta[4] = cur.rt * kRowsT;
      meta[5] = cur.L * c.group;
    }
  }

  // ---- loads: tile x of the line into stage (x - x0) % kStages
  auto load = [&](long long x) {
    if (x < x1) {
      const uint32_t st = ring + (uint32_t)((x - x0) % kStages) * kStageBytes;
      const int key0 = ld.kt * kKeysT + warp * kKeysW;  // pages hold whole groups of 16 slots
      const long long row0 = key0 < ld.n ? slot_row(c, ld.s, key0) : -1;
      if (key0 < ld.n && row0 < 0 && lane == 0) dev_flag(p.dev_status, kDevBadProblem);
      // a bad page and the slots past the sequence's end read as zeros
      const int live = row0 < 0 ? 0 : min(kKeysW, ld.n - key0);
      const long long base = ((row0 < 0 ? 0 : row0) * c.hkv + ld.g) * kHeadDim;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + (lane >> 4), ch = lane & 15;
        const long long off = r < live ? base + (long long)r * c.hkv * kHeadDim + ch * 8 : 0;
        const uint32_t d = st + r * 256 + ((ch ^ (r & 7)) << 4);
        cp_async16(d, c.k + off, r < live);
        cp_async16(d + kKeysW * 256, c.v + off, r < live);
      }
      cursor_next(ld, c, tab, x + 1 < x1);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(x0 + i);

  uint32_t qf[8][4];
  float o[16][4], l[2], m[2];
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  float* s_join = reinterpret_cast<float*>(smem + kOffJoin);
  float* s_m = reinterpret_cast<float*>(smem + kOffMl);
  float* s_l = s_m + kWarps * kRowsT;
  bool fresh = true;
  int first_kt = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
      first_kt = cur.kt;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      l[0] = l[1] = 0.f;
      m[0] = m[1] = -INFINITY;
      const uint16_t* q0[2];
      bool in[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = cur.rt * kRowsT + qr + 8 * i;
        in[i] = r < cur.L * c.group;
        q0[i] = p.q + (long long)(cur.seq0 + (in[i] ? r / c.group : 0)) * p.q_stride +
                (cur.g * c.group + (in[i] ? r % c.group : 0)) * kHeadDim + qc;
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qf[kk][i] = in[i] ? __ldg(reinterpret_cast<const uint32_t*>(q0[i] + kk * 16)) : 0u;
          qf[kk][2 + i] = in[i] ? __ldg(reinterpret_cast<const uint32_t*>(q0[i] + kk * 16 + 8)) : 0u;
        }
    }
    load(x + kStages - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t sk = ring + (uint32_t)((x - x0) % kStages) * kStageBytes, sv = sk + kKeysW * 256;
    // S = Q K^T: 16 rows x 16 keys
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const int r = (lane & 7) + ((lane >> 4) << 3), h = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t b0, b1, b2, b3;
        ldsm4(sk + r * 256 + (((2 * kk + h) ^ (r & 7)) << 4), b0, b1, b2, b3);
        mma16816(sc[0], qf[kk], b0, b1);
        mma16816(sc[1], qf[kk], b2, b3);
      }
    }
    const int key0 = cur.kt * kKeysT + warp * kKeysW;
    // keys up to `len` are seen by every row; past it row r of token t sees keys up to len + t
    const bool edge = key0 + kKeysW - 1 > cur.len;
    bool grow = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int last = edge ? min(cur.n - 1, cur.len + (cur.rt * kRowsT + qr + 8 * i) / c.group) : 0x7fffffff;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& v = sc[e >> 1][2 * i + (e & 1)];
        const int key = key0 + (e >> 1) * 8 + qc + (e & 1);
        v = key <= last ? v * p.scale_log2 : -INFINITY;
        grow |= v > m[i] + 8.f;
      }
    }
    // the reference maximum follows only when a score passes it by 2^8 (any reference gives the same
    // quotient; 8 keeps every term finite and the sums exact enough in 32 bits)
    if (__any_sync(kAll, grow)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
        const float mn = fmaxf(m[i], mx);
        const float a = mn == -INFINITY ? 1.f : ex2_approx(m[i] - mn);
        m[i] = mn;
        l[i] *= a;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j][2 * i] *= a;
          o[j][2 * i + 1] *= a;
        }
      }
    }
    uint32_t pf[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mu = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float e0 = ex2_approx(sc[j][2 * i] - mu), e1 = ex2_approx(sc[j][2 * i + 1] - mu);
        l[i] += e0 + e1;
        pf[2 * j + i] = pack_bf16x2(e0, e1);  // the tensor cores take bf16: half a step is 2^-9 of each term
      }
    }
    {
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), h = lane >> 4;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t b0, b1, b2, b3;
        ldsm4t(sv + r * 256 + (((2 * j + h) ^ (r & 7)) << 4), b0, b1, b2, b3);
        mma16816(o[2 * j], pf, b0, b1);
        mma16816(o[2 * j + 1], pf, b2, b3);
      }
    }
    __syncwarp();  // every lane has read the stage before it is loaded again
    const bool ends = cur.kt + 1 == cur.kts;
    if (!ends && x + 1 < x1) {
      cursor_next(cur, c, tab, true);
      continue;
    }
    // ---- the unit's piece is complete: join the warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(kAll, l[i], 1);
      l[i] += __shfl_xor_sync(kAll, l[i], 2);
      if ((lane & 3) == 0) {
        s_m[warp * kRowsT + qr + 8 * i] = m[i];
        s_l[warp * kRowsT + qr + 8 * i] = l[i];
      }
    }
    __syncthreads();
    const bool whole = ends && first_kt == 0;
    const long long slot = 2ll * blockIdx.x + (first_kt == 0 ? 1 : 0);  // a piece from a unit's start: slot 1
    float w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = qr + 8 * i;
      float mt = s_m[r];
      for (int k = 1; k < kWarps; ++k) mt = fmaxf(mt, s_m[k * kRowsT + r]);
      const float mu = mt == -INFINITY ? 0.f : mt;
      float lt = 0.f;
      for (int k = 0; k < kWarps; ++k) lt += s_l[k * kRowsT + r] * ex2_approx(s_m[k * kRowsT + r] - mu);
      w[i] = ex2_approx(m[i] - mu);
      if (whole) w[i] *= lt > 0.f || lt != lt ? 1.f / lt : 0.f;
      if (warp == 0 && (lane & 3) == 0) {
        if (!whole) {
          *reinterpret_cast<float2*>(p.part_ml + 2 * (slot * kRowsT + r)) = make_float2(mt, lt);
        } else {
          const int pr = cur.rt * kRowsT + r;
          if (pr < cur.L * c.group) {
            const long long at =
                (long long)(cur.g * c.group + pr % c.group) * c.total_tokens + cur.seq0 + pr / c.group;
            const float v = lt > 0.f || lt != lt ? mu + log2f(lt) : -INFINITY;
            if (p.lse2) p.lse2[at] = v;
            if (p.lse) p.lse[at] = v * 0.6931471805599453f;
          }
        }
      }
    }
    for (int cb = 0; cb < kHeadDim / kJoinCols; ++cb) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j / 4 == cb) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(s_join + (warp * kRowsT + qr + 8 * i) * kJoinCols + (j & 3) * 8 + qc) =
                make_float2(o[j][2 * i] * w[i], o[j][2 * i + 1] * w[i]);
        }
      __syncthreads();
      {
        const int r = tid >> 3, cc = (tid & 7) * 4;  // 16 rows x 8 groups of four columns
        float4 a = *reinterpret_cast<const float4*>(s_join + r * kJoinCols + cc);
        for (int k = 1; k < kWarps; ++k) {
          const float4 b = *reinterpret_cast<const float4*>(s_join + (k * kRowsT + r) * kJoinCols + cc);
          a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        if (!whole) {
          *reinterpret_cast<float4*>(p.part_o + (slot * kRowsT + r) * kHeadDim + cb * kJoinCols + cc) = a;
        } else {
          const int pr = cur.rt * kRowsT + r;
          if (pr < cur.L * c.group)
            *reinterpret_cast<uint2*>(p.out + ((long long)(cur.seq0 + pr / c.group) * c.hq + cur.g * c.group +
                                               pr % c.group) * kHeadDim + cb * kJoinCols + cc) =
                make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        }
      }
      __syncthreads();
    }
    fresh = true;
    cursor_next(cur, c, tab, x + 1 < x1);
  }
  cp_async_wait<0>();
}

// Joins the pieces of the units that several CTAs share. Block (b, y) looks at the unit inside of which the
// share of CTA b + 1 begins (meta) and works when that CTA is the first such of its unit: the pieces are
// the last one of CTA b (place 1) and the first one (place 0) of every CTA up to meta[1]. 16 rows a block.
// The time is one chain of dependent reads (meta, maxima, accumulators), so the pieces of a row are read
// side by side: 32 maxima a warp at once, and where rows are few the warps share a row's pieces.
template <bool kTiled>
__global__ void __launch_bounds__(512) cache_join_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int kRowsU = kTiled ? 2 * kTileM : kRowsT;  // rows of a piece
  __shared__ float4 s_acc[16][32];
  pdl_wait();
  const int b = blockIdx.x + 1;
  const int4 meta = *reinterpret_cast<const int4*>(p.meta + (long long)b * kMetaWords);
  const int2 meta2 = *reinterpret_cast<const int2*>(p.meta + (long long)b * kMetaWords + 4);
  if (meta.x == 0) return;
  const CacheInfo& c = p.c;
  const int P = meta.y - b + 2, seq0 = meta.z, g = meta.w, G = c.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // meta2: first token and tokens of the sequence (tiled), first packed row and packed rows (not)
  int wr = 1;  // warps that share a row
  if (!kTiled)
    while (wr < 16 && 16 / (2 * wr) >= meta2.y - meta2.x) wr *= 2;
  const int row = blockIdx.y * 16 + warp / wr, slice = warp % wr;
  int tok, head;
  bool in;
  if (kTiled) {
    const int r = row & 127, TT = p.tile_tokens;
    tok = meta2.x + (row >> 7) * TT + r / G;
    head = r % G;
    in = r < TT * G && tok < meta2.y;
  } else {
    const int pr = meta2.x + row;
    tok = pr / G;
    head = pr % G;
    in = pr < meta2.y && row < kRowsU;
  }
  if (wr == 1 && !in) return;
  auto place = [&](int k) { return (2ll * (b - 1 + k) + (k == 0)) * kRowsU + (in ? row : 0); };
  auto ml_of = [&](int k) {
    return k < P ? *reinterpret_cast<const float2*>(p.part_ml + 2 * place(k)) : make_float2(-INFINITY, 0.f);
  };
  float m = -INFINITY;
  for (int k = lane; k < P; k += 32) m = fmaxf(m, ml_of(k).x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < P; k0 += 32) {
    const float2 ml = ml_of(k0 + lane);
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
  if (wr > 1) {
    s_acc[warp][lane] = acc;
    __syncthreads();
    if (slice != 0 || !in) return;
    for (int q = 1; q < wr; ++q) {
      const float4 a = s_acc[warp + q][lane];
      acc.x += a.x; acc.y += a.y; acc.z += a.z; acc.w += a.w;
    }
  }
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

// ------------------------------------------------------------------------ collected weights -----
// Every warp takes 16 keys of one (sequence, kv-head) and walks the rows of its new tokens, 16 at a
// time: S again from Q and K, then p = 2^(S - lse2) summed over the rows. No two warps touch one
// weight, so the sum's order is fixed.
__global__ void __launch_bounds__(kRowThreads) cache_weights_kernel(const __grid_constant__ CacheAttnParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const CacheInfo& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t sk = smem_u32(smem) + warp * kKeysW * 256;
  long long* tab = reinterpret_cast<long long*>(smem + kWarps * kKeysW * 256 + 128);
  long long* s_scan = reinterpret_cast<long long*>(smem + kWarps * kKeysW * 256);
  int* s_bad = reinterpret_cast<int*>(s_scan + kWarps);
  const bool ok = cache_table<kRowThreads>(c, tab, s_scan, s_bad, p.dev_status, [&](int, int L, int n) -> long long {
    return L > 0 ? (long long)c.hkv * ((n + kKeysT - 1) / kKeysT) : 0ll;
  });
  const long long total = ok ? tab[c.num_seqs] : 0;
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  for (long long x = blockIdx.x; x < total; x += gridDim.x) {
    const int s = find_seq64(tab, c.num_seqs, x);
    const int seq0 = __ldg(c.cu_seqlens + s), L = __ldg(c.cu_seqlens + s + 1) - seq0, len = c.lens[s], n = len + L;
    const int kts = (n + kKeysT - 1) / kKeysT;
    const int g = (int)((x - tab[s]) / kts), kt = (int)((x - tab[s]) % kts);
    const int key0 = kt * kKeysT + warp * kKeysW;
    if (key0 >= n) continue;
    const long long row0 = slot_row(c, s, key0);
    if (row0 < 0) {
      if (lane == 0) dev_flag(p.dev_status, kDevBadProblem);
      continue;
    }
    const int live = min(kKeysW, n - key0);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 2 * i + (lane >> 4), ch = lane & 15;
      cp_async16(sk + r * 256 + ((ch ^ (r & 7)) << 4),
                 c.k + ((row0 + (r < live ? r : 0)) * c.hkv + g) * kHeadDim + ch * 8, r < live);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // [8-key half][column] of this thread's rows
    const int rows = L * c.group;
    // tokens before key0 - len do not see any key of this warp
    const int rt0 = key0 > len ? (key0 - len) * c.group / kRowsT : 0;
    for (int rt = rt0; rt * kRowsT < rows; ++rt) {
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const uint16_t* q0[2];
      float lse2[2];
      int last[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rt * kRowsT + qr + 8 * i;
        const bool in = r < rows;
        const int t = in ? r / c.group : 0, h = g * c.group + (in ? r % c.group : 0);
        q0[i] = p.q + (long long)(seq0 + t) * p.q_stride + h * kHeadDim + qc;
        lse2[i] = __ldg(p.lse2 + (long long)h * c.total_tokens + seq0 + t);
        last[i] = in ? len + t : -1;
      }
      const int r = (lane & 7) + ((lane >> 4) << 3), hh = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t a[4], b0, b1, b2, b3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = __ldg(reinterpret_cast<const uint32_t*>(q0[i] + kk * 16));
          a[2 + i] = __ldg(reinterpret_cast<const uint32_t*>(q0[i] + kk * 16 + 8));
        }
        ldsm4(sk + r * 256 + (((2 * kk + hh) ^ (r & 7)) << 4), b0, b1, b2, b3);
        mma16816(sc[0], a, b0, b1);
        mma16816(sc[1], a, b2, b3);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + (e >> 1) * 8 + qc + (e & 1);
          if (key <= last[i]) w[e >> 1][e & 1] += ex2_approx(fmaf(sc[e >> 1][2 * i + (e & 1)], p.scale_log2, -lse2[i]));
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = w[e >> 1][e & 1];
      v += __shfl_xor_sync(kAll, v, 4);
      v += __shfl_xor_sync(kAll, v, 8);
      v += __shfl_xor_sync(kAll, v, 16);
      const int k = (e >> 1) * 8 + qc + (e & 1);
      if (lane < 4 && k < live) {
        const long long page = row0 / c.page_size;
        float* dst = c.weights + (page * c.hkv + g) * c.page_size + (row0 - page * c.page_size) + k;
        *dst = p.decay > 0.f ? fmaf(p.decay, *dst, v) : v;
      }
    }
  }
}
constexpr int weights_smem(int S) { return kWarps * kKeysW * 256 + 128 + 8 * (S + 1); }

}  // namespace

bool cache_attn_tiled(int32_t max_new, int32_t group) { return (int64_t)max_new * group > kRowsT; }

CacheAttnLayout cache_attn_layout(int sms, bool tiled, int64_t hq, int64_t total_tokens) {
  auto up = [](int64_t x) { return (x + 255) & ~(int64_t)255; };
  const int64_t grid = tiled ? sms : 2 * sms, rows = 2 * grid * (tiled ? 2 * kTileM : kRowsT);
  CacheAttnLayout w;
  w.part_o = 0;
  w.part_ml = up(w.part_o + rows * kHeadDim * 4);
  w.meta = up(w.part_ml + rows * 2 * 4);
  w.lse2 = up(w.meta + grid * kMetaWords * 4);
  w.total = up(w.lse2 + hq * total_tokens * 4);
  return w;
}

// Every kernel of a call asks for the same split of the SM's memory (the largest shared part): between
// kernels that differ in it the SM has to drain first, which costs microseconds.
cudaError_t launch_cache_join(const CacheAttnParams& p, bool tiled, int ctas, cudaStream_t st) {
  if (ctas < 2) return cudaSuccess;
  void (*fn)(const CacheAttnParams) = tiled ? cache_join_kernel<true> : cache_join_kernel<false>;
  static unsigned long long attr[2][kMaxCachedDevices] = {};
  const cudaError_t e = set_max_smem(reinterpret_cast<const void*>(fn), 0, attr[tiled], true);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, dim3(ctas - 1, tiled ? 16 : 1), 512, 0, st, p);
}

cudaError_t launch_cache_attn(const CacheAttnParams& p, bool tiled, int sms, cudaStream_t st) {
  static unsigned long long attr[kMaxCachedDevices] = {}, attr_w[kMaxCachedDevices] = {};
  cudaError_t e;
  if (tiled) {
    if ((e = launch_cache_tiles(p, sms, st)) != cudaSuccess) return e;
  } else {
    e = set_max_smem(reinterpret_cast<const void*>(cache_rows_kernel), row_smem(kMaxSeqs), attr, true);
    if (e != cudaSuccess) return e;
    const int grid = 2 * sms;
    cache_rows_kernel<<<grid, kRowThreads, row_smem(p.c.num_seqs), st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_cache_join(p, false, grid, st)) != cudaSuccess) return e;
  }
  if (!(p.decay >= 0.f)) return cudaSuccess;
  if ((e = set_max_smem(reinterpret_cast<const void*>(cache_weights_kernel), weights_smem(kMaxSeqs), attr_w, true)) !=
      cudaSuccess)
    return e;
  cache_weights_kernel<<<8 * sms, kRowThreads, weights_smem(p.c.num_seqs), st>>>(p);
  return cudaGetLastError();
}

}  // namespace fp
