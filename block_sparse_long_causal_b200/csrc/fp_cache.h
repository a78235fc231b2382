// fp_cache.h -- what the host side of the key/value cache calls shares with their kernels: launch
// parameters, the workspace's layout and the launchers. (A header of its own: fp_internal.h belongs to the prefill
// kernels, whose recorded DRAM traffic holds for the sources that it was measured on.)
#pragma once
#include "fp_internal.h"

namespace fp {

// A key/value cache and the chunk of new tokens that a call works on (fp_kv_cache with fp_problem).
struct CacheInfo {
  const int32_t* cu_seqlens;  // device [S+1], the new tokens
  int32_t* lens;              // device [S], slots in use before the new tokens
  const int32_t* block_table; // device [S, max_pages]
  int32_t num_seqs, total_tokens;
  int32_t max_pages, page_size, num_pages;
  uint32_t page_mul, page_shift;  // u / page_size = (u * page_mul) >> (32 + page_shift) for 0 <= u < 2^31
  int32_t max_len;            // bound of lens[s] + L_s
  int32_t max_new;            // bound of L_s
  int32_t hq, hkv, group;
  uint16_t* k;                // [num_pages * page_size, Hkv, d] bf16 bits
  uint16_t* v;
  float* weights;             // [num_pages, Hkv, page_size] or null
  int32_t* positions;         // likewise
};

struct AppendParams {
  CacheInfo c;
  const uint16_t* k;          // [T, Hkv, d], rows k_stride elements apart
  const uint16_t* v;
  int64_t k_stride, v_stride;
  const int32_t* next_pos;    // device [S] or null (the slot is the position)
  int32_t* dev_status;
};

// Tensor maps first: they must be 64-byte aligned (rows schedule: unused).
struct __align__(64) CacheAttnParams {
  CUtensorMap tm_q;           // q as [T][Hq][128]: boxes of 64 columns x group heads x tile_tokens tokens
  CUtensorMap tm_k, tm_v;     // the cache's rows x Hkv * 128: boxes of 64 columns x box_rows rows
  int32_t tile_tokens;        // tokens of a 128-row tile: 128 / group
  int32_t box_rows;           // rows of a K/V copy: the largest power of two up to 128 that divides page_size
  CacheInfo c;
  const uint16_t* q;          // [T, Hq, d], rows q_stride elements apart
  int64_t q_stride;
  float scale_log2;           // softmax_scale * log2(e)
  uint16_t* out;              // [T, Hq, d] bf16 bits
  float* lse;                 // [Hq, T] or null (natural log)
  float* lse2;                // [Hq, T] workspace, log2 units (for the weights; negated by the 128-row schedule), or null
  bool out32;                 // out is 32-byte aligned
  float* part_o;              // workspace: partial outputs [2 * grid][rows][128] (row tiles: [..][16][128 rows][8])
  float* part_ml;             // workspace: their running max (log2 units) and row sum, 2 * grid * rows of each
  int32_t* meta;              // workspace: the unit that each CTA's range begins inside of [grid][kMetaWords]
  float* scores;              // workspace: scaled scores [tile of the line][score_rows / 4][64 keys][4] (few rows), or null
  int32_t score_rows;
  int64_t score_tiles;        // tiles that fit
  float decay;                // weights = decay * weights + this call's; < 0: weights are left alone
  int32_t* dev_status;
  uint64_t wait_limit_ns;
  int32_t test_unsignalled_wait;  // tests only: as in AttnParams (128-row schedule)
};

struct SelectParams {
  CacheInfo c;
  int32_t budget, sinks, recent;
  const int32_t* next_pos;    // device [S] or null
  int32_t* moves;             // [S, Hkv, budget, 2]
  int32_t* move_counts;       // [S, Hkv]
  int32_t* new_lens;          // [S]
  int32_t* dev_status;
};

struct CompactParams {
  CacheInfo c;
  int32_t budget;
  const int32_t* moves;
  const int32_t* move_counts;
  const int32_t* new_lens;
  int32_t parts;              // CTAs per (sequence, kv-head), set by the launcher
  int32_t* dev_status;
};

// set_max_smem that also asks for the largest shared part of the SM's memory at every launch.
cudaError_t set_max_smem_carveout(const void* func, int bytes, unsigned long long (&done)[kMaxCachedDevices]);

// Key/value cache (fp_cache.cu, fp_cache_attn.cu).
cudaError_t launch_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_select(const SelectParams& p, cudaStream_t st);
cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t st);
constexpr int kMetaWords = 8;               // ints per CTA that describe the unit its share begins inside of
// Schedule of the attention call: units of up to 32 rows (fp_cache_attn.cu) or 128-row tiles (fp_cache_tiles.cu).
bool cache_attn_tiled(int32_t max_new, int32_t group);
struct CacheAttnLayout {                    // byte offsets of its workspace
  int64_t part_o, part_ml, meta, lse2, scores, total;
  int64_t score_tiles;
  int32_t score_rows;
};
CacheAttnLayout cache_attn_layout(int sms, bool tiled, const CacheInfo& c, bool scores);
cudaError_t launch_cache_attn(const CacheAttnParams& p, bool tiled, int sms, cudaStream_t st);
cudaError_t launch_cache_tiles(const CacheAttnParams& p, int sms, cudaStream_t st);
cudaError_t launch_cache_weights(const CacheAttnParams& p, int sms, cudaStream_t st);

}  // namespace fp
