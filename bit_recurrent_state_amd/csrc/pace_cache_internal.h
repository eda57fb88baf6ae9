// Internal declarations of the attention-layer operators (include/pace_cache.h): the cache's
// byte layout, shared by host and kernels, and the parameter blocks passed by value.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pace_cache.h"

namespace pace {

// Sizes of one page's record of one head (include/pace_cache.h: CACHE LAYOUT).
struct CacheRecord {
  uint32_t codes, scales, total;   // bytes of one codes part, one scales part, the record
};

__host__ __device__ inline CacheRecord cache_record(int d, int group, int page, int bits) {
  CacheRecord r;
  r.codes = (uint32_t)(page * d * bits / 8);
  r.scales = (uint32_t)(page * (d / group) * 2);
  r.total = 2 * (r.codes + r.scales);
  return r;
}

struct RotaryParams {
  const int32_t* positions;
  const double* freqs;
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;   // elements
  float magnitude;
  int32_t n, Hq, Hk, d, rd, interleaved, inverse;
  int32_t copy_q, copy_k;   // channels from rd on have to be copied (not in place)
};

struct CacheIoParams {       // pace_cache_write / pace_cache_read
  uint8_t* cache;
  const int32_t* table;
  const int32_t* positions;
  const void* k_in;          // write: inputs
  const void* v_in;
  void* k_out;               // read: outputs
  void* v_out;
  int64_t k_stride, v_stride;   // elements
  int32_t B, T, Hkv, page_shift, num_pages, max_pages;
};

// Tiles of 16 tokens of a call of T (the first token of 16 or more may be at any place of its tile), and
// workgroups of four tiles.
inline int cache_io_tiles(int T) { return T < 16 ? 1 : (int)(((int64_t)T + 15 + 15) / 16); }
inline int64_t cache_io_blocks(int B, int T, int Hkv) { return ((int64_t)B * cache_io_tiles(T) * Hkv + 3) / 4; }

struct AttnParams {
  const uint8_t* cache;
  const int32_t* table;
  const void* q;
  int64_t q_stride;
  const int32_t* ctx_lens;
  const int32_t* draft_lens;   // may be null
  const uint32_t* tree;        // may be null (chain)
  int64_t tree_stride;         // words between sequences' trees
  void* o;
  float* lse;                  // may be null
  float* part_o;               // [nsplit][B][Hkv][R][d], used when nsplit > 1
  float* part_lse;             // [nsplit][B][Hkv][R], base-2 logarithms
  float scale_log2e;
  int32_t B, T, Hq, Hkv, gamma, R;   // R = T * gamma rows of one key/value head
  int32_t page_shift, num_pages, max_pages;
  int32_t nsplit, chunk;       // the context is cut into nsplit pieces of `chunk` tokens
  int32_t row_blocks;
};

constexpr int kMaxPieces = 1024;   // of one context (the join keeps their weights in LDS)

// 16-token tiles that a wave takes at once.  (Four cost registers, so waves, and gained nothing.)
constexpr int kTiles = 2;

// How pace_cache_attention cuts its work (a function of host-known sizes only).
struct AttnPlan {
  int32_t row_tiles;    // 16-row tiles a wave, and so a workgroup, holds
  int32_t waves;        // of a workgroup, on different tokens: 4 or 8
  int32_t row_blocks;   // workgroups over the rows
  int32_t step;         // tokens a workgroup takes at once
  int32_t nsplit, chunk;
};
AttnPlan attn_plan(const pace_cache_cfg& c, int T, int max_len);

// Launchers (defined next to their kernels).  They only enqueue work.
hipError_t launch_rotary(const RotaryParams& p, int io_bf16, bool wide, hipStream_t stream);
hipError_t launch_cache_write(const CacheIoParams& p, int kind, int d, int group, int io_bf16,
                              hipStream_t stream);
hipError_t launch_cache_read(const CacheIoParams& p, int kind, int d, int group, int io_bf16,
                             hipStream_t stream);
hipError_t launch_attention_int8(const AttnParams& p, const AttnPlan& plan, int d, int group, int io_bf16,
                                 hipStream_t stream);
hipError_t launch_attention_int4(const AttnParams& p, const AttnPlan& plan, int d, int group, int io_bf16,
                                 hipStream_t stream);
hipError_t launch_attention_fp8(const AttnParams& p, const AttnPlan& plan, int d, int group, int io_bf16,
                                hipStream_t stream);
hipError_t launch_attention(const AttnParams& p, const AttnPlan& plan, int kind, int d, int group,
                            int io_bf16, hipStream_t stream);

}  // namespace pace
