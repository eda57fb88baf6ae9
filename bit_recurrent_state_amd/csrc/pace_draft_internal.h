// Internal declarations of the operators that serve drafted tokens (include/pace_draft.h): the
// parameter blocks passed by value and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pace_draft.h"
#include "pace_internal.h"

namespace pace {

constexpr int kMaxDrafts = 64;        // T of pace_draft_step and pace_draft_commit: a row of tree bits is 64 bits
constexpr int kMaxNodes = 1024;       // T of pace_draft_verify
constexpr int kMaxVocab = 1 << 24;
constexpr int kMaxMoved = 1 << 30;    // T of pace_cache_move

struct DraftParams {
  DecodeParams l;               // the layer; q, k, v, a, beta [B][T].., o
  const int32_t* draft_lens;    // may be null
  const uint32_t* tree;         // may be null (a chain)
  int64_t tree_stride;          // words between sequences' trees
  int32_t T;
};

// 16-token tiles of the buffered and drafted tokens of one sequence.
inline int draft_tiles(int dP, int T) { return (dP - 1 + T + 15) / 16; }

struct CommitParams {
  DecodeParams l;               // the layer; k, v, a, beta [B][T]..
  const int32_t* nodes;         // [B][T]
  const int32_t* counts;
  const int32_t* done;          // [B][Hv] tokens that earlier rounds took (null: none), as kFilled says
  int32_t* done_out;            // [B][Hv]
  int32_t T, most;
};

struct VerifyParams {
  const void* target;
  const void* draft;            // may be null
  int64_t target_stride, draft_stride;   // elements
  const int32_t* tokens;
  const int32_t* parents;       // may be null (a chain)
  int64_t parents_stride;
  const float* uniforms;
  const int32_t* draft_lens;    // may be null
  int32_t* nodes;
  int32_t* counts;
  int32_t* next;
  uint8_t* workspace;
  int64_t scratch;              // bytes of a sequence there
  int32_t B, T, V, chunks;
};

// Tokens of a chunk: what a wave sums at once.
constexpr int kVerifyChunk = 2048;

// Workspace of a sequence: a double a chunk, the walk (48 bytes), its path and refused tokens.
inline int64_t verify_scratch(int T, int chunks) { return ((int64_t)chunks * 8 + 48 + 8 * (int64_t)T + 63) / 64 * 64; }

struct MoveParams {
  uint8_t* cache;
  const int32_t* src_table;
  const int32_t* dst_table;
  const int32_t* start;
  const int32_t* nodes;         // may be null: i itself
  int64_t nodes_stride;
  const int32_t* counts;
  int32_t B, T, Hkv, page_shift, num_pages, max_pages;
};

// Launchers (defined next to their kernels).  They only enqueue work.
hipError_t launch_draft_step(const DraftParams& p, int dk, int buf_kind, hipStream_t stream);
hipError_t launch_draft_append(const CommitParams& p, int dk, int buf_kind, hipStream_t stream);
hipError_t launch_draft_verify(const VerifyParams& p, int prob_bf16, hipStream_t stream);
hipError_t launch_cache_move(const MoveParams& p, int kind, int d, int group, hipStream_t stream);

}  // namespace pace
