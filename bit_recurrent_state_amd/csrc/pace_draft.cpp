// Host entry points of the operators that serve drafted tokens (include/pace_draft.h): validation,
// sizes, and the launches.  No call allocates, frees or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pace_draft_internal.h"
#include "pace_layer_host.h"

using namespace pace;

namespace {

constexpr int64_t kMaxSpan = INT64_C(1) << 48;   // bytes from the first row to the last

int rounds_of(const pace_layer_cfg* c, int32_t most) { return (most + c->dP - 1) / c->dP; }

size_t commit_bytes(const pace_layer_cfg* c, int32_t most) {
  return (size_t)(rounds_of(c, most) + 1) * c->B * c->Hv * sizeof(int32_t);
}

bool tokens_ok(const void* k, const void* v, const float* a, const float* beta) {
  return k && v && a && beta && aligned(k, 16) && aligned(v, 16) && aligned(a, 4) && aligned(beta, 4);
}

pace_status validate(const pace_verify_cfg* c) {
  if (!c || c->B < 1 || c->T < 1 || c->V < 1) return PACE_EINVAL;
  if (c->prob_dtype != PACE_IO_F32 && c->prob_dtype != PACE_IO_BF16) return PACE_EINVAL;
  if (c->B > 65535 || c->T > kMaxNodes || c->V > kMaxVocab) return PACE_EUNSUPPORTED;
  return PACE_OK;
}

int verify_chunks(const pace_verify_cfg* c) { return (c->V + kVerifyChunk - 1) / kVerifyChunk; }

size_t verify_bytes(const pace_verify_cfg* c) { return (size_t)c->B * verify_scratch(c->T, verify_chunks(c)); }

}  // namespace

extern "C" {

pace_status pace_draft_step(const pace_layer_cfg* cfg, const void* state, const void* buffer,
                            const void* q, const void* k, const void* v, const float* a,
                            const float* beta, int32_t T, const int32_t* draft_lens,
                            const uint32_t* tree, int64_t tree_stride, void* o, void* stream) {
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  if (T < 1) return PACE_EINVAL;
  if (T > kMaxDrafts) return PACE_EUNSUPPORTED;
  if (!state || !buffer || !q || !o || !aligned(state, 256) || !aligned(buffer, 256) || !aligned(q, 16) ||
      !aligned(o, 16) || !tokens_ok(k, v, a, beta) || !aligned(draft_lens, 4) || !aligned(tree, 4))
    return PACE_EINVAL;
  if (tree_stride < 0 || tree_stride > kMaxSpan / 4 / cfg->B) return PACE_EINVAL;
  DraftParams p{};
  p.l = layer_params(cfg, state, buffer);
  p.l.q = q; p.l.k = k; p.l.v = v; p.l.a = a; p.l.beta = beta; p.l.o = o;
  p.draft_lens = draft_lens;
  p.tree = tree;
  p.tree_stride = tree_stride;
  p.T = T;
  const hipError_t e = launch_draft_step(p, cfg->dk, cfg->buf_kind, (hipStream_t)stream);
  return e == hipSuccess ? PACE_OK : PACE_EHIP;
}

pace_status pace_draft_commit_workspace_bytes(const pace_layer_cfg* cfg, int32_t most,
                                              size_t* bytes_out) {
  if (!bytes_out) return PACE_EINVAL;
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  if (most < 1) return PACE_EINVAL;
  if (most > kMaxDrafts) return PACE_EUNSUPPORTED;
  *bytes_out = commit_bytes(cfg, most);
  return PACE_OK;
}

pace_status pace_draft_commit(const pace_layer_cfg* cfg, void* state, void* buffer, const void* k,
                              const void* v, const float* a, const float* beta, int32_t T,
                              const int32_t* nodes, const int32_t* counts, int32_t most,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  if (T < 1 || most < 1 || most > T) return PACE_EINVAL;
  if (T > kMaxDrafts) return PACE_EUNSUPPORTED;
  if (!state || !buffer || !aligned(state, 256) || !aligned(buffer, 256) || !tokens_ok(k, v, a, beta) || !nodes ||
      !counts || !aligned(nodes, 4) || !aligned(counts, 4))
    return PACE_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < commit_bytes(cfg, most)) return PACE_EINVAL;
  CommitParams p{};
  p.l = layer_params(cfg, state, buffer);
  p.l.k = k; p.l.v = v; p.l.a = a; p.l.beta = beta;
  p.nodes = nodes;
  p.counts = counts;
  p.T = T;
  p.most = most;
  // Tokens up to the end of the period, the fold of the buffers that it fills, and on.  At most dP - 1 tokens
  // are held before, so `most` more end at most ceil(most / dP) periods.
  DecodeParams fold = flush_params(cfg, state, buffer, 2);
  const int rounds = rounds_of(cfg, most);
  const size_t each = (size_t)cfg->B * cfg->Hv;
  for (int r = 0; r <= rounds; ++r) {
    p.done = r ? (const int32_t*)workspace + (r - 1) * each : nullptr;
    p.done_out = (int32_t*)workspace + r * each;
    if (launch_draft_append(p, cfg->dk, cfg->buf_kind, (hipStream_t)stream) != hipSuccess) return PACE_EHIP;
    if (r == rounds) break;
    fold.filled = p.done_out;
    if (launch_decode(fold, nullptr, cfg->dk, cfg->dv, cfg->buf_kind, (hipStream_t)stream) != hipSuccess) return PACE_EHIP;
  }
  return PACE_OK;
}

pace_status pace_draft_verify_workspace_bytes(const pace_verify_cfg* cfg, size_t* bytes_out) {
  if (!bytes_out) return PACE_EINVAL;
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  *bytes_out = verify_bytes(cfg);
  return PACE_OK;
}

pace_status pace_draft_verify(const pace_verify_cfg* cfg, const void* target, int64_t target_stride,
                              const void* draft, int64_t draft_stride, const int32_t* tokens,
                              const int32_t* parents, int64_t parents_stride,
                              const float* uniforms, const int32_t* draft_lens, int32_t* nodes,
                              int32_t* counts, int32_t* next, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  const size_t e = cfg->prob_dtype == PACE_IO_BF16 ? 2 : 4;
  const int64_t rows = (int64_t)cfg->B * cfg->T;
  if (!target || !aligned(target, e) || !aligned(draft, e) || !tokens || !aligned(tokens, 4) || !aligned(parents, 4) ||
      !uniforms || !aligned(uniforms, 4) || !aligned(draft_lens, 4) || !nodes || !aligned(nodes, 4) || !counts ||
      !aligned(counts, 4) || !next || !aligned(next, 4))
    return PACE_EINVAL;
  if (target_stride < cfg->V || (draft && draft_stride < cfg->V) || parents_stride < 0) return PACE_EINVAL;
  const int64_t longest = draft ? std::max(target_stride, draft_stride) : target_stride;
  if (longest > kMaxSpan / (int64_t)e / rows || parents_stride > kMaxSpan / 4 / cfg->B) return PACE_EUNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < verify_bytes(cfg)) return PACE_EINVAL;
  VerifyParams p{};
  p.target = target; p.target_stride = target_stride;
  p.draft = draft; p.draft_stride = draft_stride;
  p.tokens = tokens;
  p.parents = parents; p.parents_stride = parents_stride;
  p.uniforms = uniforms;
  p.draft_lens = draft_lens;
  p.nodes = nodes; p.counts = counts; p.next = next;
  p.workspace = (uint8_t*)workspace;
  p.B = cfg->B; p.T = cfg->T; p.V = cfg->V;
  p.chunks = verify_chunks(cfg);
  p.scratch = verify_scratch(cfg->T, p.chunks);
  const hipError_t err = launch_draft_verify(p, cfg->prob_dtype == PACE_IO_BF16, (hipStream_t)stream);
  return err == hipSuccess ? PACE_OK : PACE_EHIP;
}

pace_status pace_cache_move(const pace_cache_cfg* cfg, void* cache, const int32_t* src_table,
                            const int32_t* dst_table, const int32_t* start, const int32_t* nodes,
                            int64_t nodes_stride, const int32_t* counts, int32_t T, void* stream) {
  pace_cache_layout_info info;
  const pace_status st = pace_cache_layout(cfg, &info);
  if (st != PACE_OK) return st;
  if (T < 0) return PACE_EINVAL;
  if (T > kMaxMoved) return PACE_EUNSUPPORTED;
  if (T == 0) return PACE_OK;
  if (!cache || !aligned(cache, 256) || !src_table || !aligned(src_table, 4) || !dst_table || !aligned(dst_table, 4) ||
      !start || !aligned(start, 4) || !aligned(nodes, 4) || !counts || !aligned(counts, 4))
    return PACE_EINVAL;
  if (nodes && (nodes_stride < T || nodes_stride > kMaxSpan / 4 / cfg->B)) return PACE_EINVAL;
  MoveParams p{};
  p.cache = (uint8_t*)cache;
  p.src_table = src_table;
  p.dst_table = dst_table;
  p.start = start;
  p.nodes = nodes;
  p.nodes_stride = nodes_stride;
  p.counts = counts;
  p.B = cfg->B; p.T = T; p.Hkv = cfg->Hkv;
  while ((1 << p.page_shift) < cfg->page) ++p.page_shift;
  p.num_pages = cfg->num_pages;
  p.max_pages = cfg->max_pages;
  const hipError_t e = launch_cache_move(p, cfg->kind, cfg->d, cfg->group, (hipStream_t)stream);
  return e == hipSuccess ? PACE_OK : PACE_EHIP;
}

}  // extern "C"
