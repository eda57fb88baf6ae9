// Host entry points of the attention-layer operators (include/pace_cache.h): validation,
// sizes, rotary frequencies, tree bits, and the launches.  No call allocates, frees or
// synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "pace_cache_internal.h"

using namespace pace;

namespace {

constexpr int kMaxQueryHeads = 1024;
constexpr int kMaxRows = 1 << 24;
constexpr double kLog2e = 1.4426950408889634074;
constexpr int64_t kMaxThreads = INT64_C(0xFFFFFFFF);   // of a launch
constexpr int kRotaryTokens = 1 << 23;                 // of a launch (256 threads each at most)

int cache_bits(int kind) { return kind == PACE_CACHE_INT4 ? 4 : 8; }

size_t io_bytes(int io_dtype) { return io_dtype == PACE_IO_BF16 ? 2 : 4; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Finite in fp32, in which the kernels take it.
bool fits_f32(double x) { return std::fabs(x) <= (double)0x1.fffffep127f; }

// n steps of `stride` elements of e bytes stay within any address space.
bool spans(int64_t n, int64_t stride, int64_t e) { return stride <= (INT64_C(1) << 48) / e / std::max<int64_t>(n, 1); }

bool rows_ok(const void* p, int64_t n, int64_t stride, int64_t width, int io_dtype) {
  const int64_t e = (int64_t)io_bytes(io_dtype);
  return p && aligned(p, 16) && stride >= width && spans(n, stride, e) && (stride * e) % 16 == 0;
}

pace_status validate(const pace_cache_cfg* c) {
  if (!c) return PACE_EINVAL;
  if (c->B <= 0 || c->Hq <= 0 || c->Hkv <= 0 || c->d <= 0 || c->group <= 0 || c->page <= 0 ||
      c->num_pages <= 0 || c->max_pages <= 0)
    return PACE_EINVAL;
  if (c->Hq % c->Hkv != 0 || c->d % c->group != 0) return PACE_EINVAL;
  if (c->kind != PACE_CACHE_INT8 && c->kind != PACE_CACHE_INT4 && c->kind != PACE_CACHE_FP8) return PACE_EINVAL;
  if (c->io_dtype != PACE_IO_F32 && c->io_dtype != PACE_IO_BF16) return PACE_EINVAL;
  // kernel coverage
  if (c->d != 64 && c->d != 128 && c->d != 256) return PACE_EUNSUPPORTED;
  if (c->group != 32 && c->group != 64 && c->group != 128) return PACE_EUNSUPPORTED;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1))) return PACE_EUNSUPPORTED;
  if (c->B > 65535 || c->Hq > kMaxQueryHeads) return PACE_EUNSUPPORTED;
  if ((int64_t)c->max_pages * c->page > INT32_MAX) return PACE_EUNSUPPORTED;
  return PACE_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

pace_status attn_sizes(const pace_cache_cfg* c, int32_t T, int32_t max_len, AttnPlan* plan, size_t* bytes) {
  const pace_status st = validate(c);
  if (st != PACE_OK) return st;
  if (T < 1 || max_len < 1) return PACE_EINVAL;
  const int64_t R = (int64_t)T * (c->Hq / c->Hkv);
  if (R > kMaxRows) return PACE_EUNSUPPORTED;
  *plan = attn_plan(*c, T, max_len);
  // the kernel's grid, and the rows that the join counts (pieces are cut for 384 blocks of rows or fewer: its
  // own grid is small)
  const int64_t groups = (int64_t)plan->nsplit * plan->row_blocks * c->B * c->Hkv;
  if (groups * 64 * plan->waves > kMaxThreads || (int64_t)c->B * c->Hkv * R > INT32_MAX) return PACE_EUNSUPPORTED;
  *bytes = plan->nsplit > 1
               ? (size_t)plan->nsplit * c->B * c->Hkv * (size_t)R * (size_t)(c->d + 1) * sizeof(float)
               : 0;
  return PACE_OK;
}

}  // namespace

namespace pace {

AttnPlan attn_plan(const pace_cache_cfg& c, int T, int max_len) {
  AttnPlan a;
  const int64_t R = (int64_t)T * (c.Hq / c.Hkv);
  // Two row tiles a wave unpack every code once for 32 rows (d = 128, int8: a 512-token chunk over
  // 7680 tokens 240 us, with one tile 305).  Up to 32 rows that saves nothing and one tile leaves
  // more waves (16 trees of 5 to 8 tokens over 4096: 25 to 31 us, with two tiles 28 to 35); from there
  // to 100 rows either may be ahead by up to 22% (trees of 9 to 25 tokens, the three kinds: 36 to 73 us with one
  // tile, 37 to 62 with two, 2% apart on average).  fp32 with d = 128 has twice the operands: there the same
  // trees take 42 to 88 us with one tile and 48 to 82 with two (9% more on average), trees of 48 tokens 92 to
  // 113 against 89 to 113.  d = 256 has no registers for two.
  const int one_tile = c.io_dtype == PACE_IO_F32 && c.d == 128 ? 128 : 32;
  a.row_tiles = c.d <= 128 && R > one_tile ? 2 : 1;
  a.row_blocks = ceil_div(R, 16 * a.row_tiles);
  const int64_t base = (int64_t)a.row_blocks * c.B * c.Hkv;
  // Short contexts of few sequences.  Four waves take 256 tokens in one workgroup.  For some more, eight
  // do, and no second kernel has to be launched to join pieces: one sequence of 300 to 760 tokens, 8
  // heads, takes 8.2 to 10.3 us a call against 11.7.  (In a graph, where launches are cheap, 7.5 to 9.9 us
  // against 8.5 to 9.1: no slower to about 512 tokens, and faster to 1000 with 16 sequences.)
  a.waves = a.row_tiles == 1 && c.d <= 128 && base <= 256 && max_len > 256 && max_len <= 768 ? 8 : 4;
  a.step = 16 * kTiles * a.waves;
  // Otherwise pieces until the 256 compute units hold three workgroups each, at most one for every two steps
  // (rounded up to whole steps; the last piece is what is left).
  // (Twice as many cost 5% of three contexts of 131072 tokens and 14% of 16 trees of 25, and
  // gained 3% of 64 ragged ones: every workgroup waits for its first tokens, and its part is written
  // and read once more.)
  const int64_t want = a.waves == 8 ? 1 : std::max<int64_t>(1, 768 / base);
  const int most = ceil_div(max_len, 2 * a.step);
  const int n = (int)std::min<int64_t>(std::min<int64_t>(want, most), kMaxPieces);
  const int64_t chunk = (int64_t)ceil_div(ceil_div(max_len, n), a.step) * a.step;
  a.nsplit = ceil_div(max_len, chunk);
  a.chunk = (int)std::min<int64_t>(chunk, INT32_MAX / a.step * a.step);   // (one piece ends with the tokens)
  return a;
}

}  // namespace pace

extern "C" {

pace_status pace_rotary_freqs(int32_t rd, double base, int32_t scaling, double factor,
                              double original_len, double fast_turns, double slow_turns,
                              double* freqs, double* magnitude) {
  if (!freqs || !magnitude || rd < 2 || rd % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return PACE_EINVAL;
  if (scaling < PACE_ROPE_PLAIN || scaling > PACE_ROPE_BLEND) return PACE_EINVAL;
  if (scaling != PACE_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return PACE_EINVAL;
  double lo = 0.0, hi = 0.0;
  if (scaling == PACE_ROPE_BLEND) {
    if (factor < 1.0 || !(original_len > 0.0) || !(slow_turns > 0.0) || !(fast_turns > slow_turns) ||
        !std::isfinite(original_len) || !std::isfinite(fast_turns))
      return PACE_EINVAL;
    // the pair index at which a pair turns n times over the original length:
    // original_len base^(-2 i / rd) = 2 pi n
    auto pair_of = [&](double n) {
      return rd * std::log(original_len / (n * 2.0 * M_PI)) / (2.0 * std::log(base));
    };
    lo = std::max(0.0, std::floor(pair_of(fast_turns)));
    hi = std::min((double)rd - 1.0, std::ceil(pair_of(slow_turns)));
  }
  const double b = scaling == PACE_ROPE_NTK ? base * std::pow(factor, (double)rd / std::max(1, rd - 2)) : base;
  for (int i = 0; i < rd / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rd);
    if (scaling == PACE_ROPE_LINEAR) f /= factor;
    if (scaling == PACE_ROPE_BLEND) {
      const double r = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      f = f * (1.0 - r) + f / factor * r;
    }
    freqs[i] = f;
  }
  *magnitude = scaling == PACE_ROPE_BLEND ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return PACE_OK;
}

pace_status pace_rotary(const pace_rotary_cfg* cfg, int32_t n, const int32_t* positions,
                        const double* freqs, double magnitude, int32_t inverse, const void* q,
                        int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                        int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (!cfg || n < 0) return PACE_EINVAL;
  if (cfg->Hq < 0 || cfg->Hk < 0 || cfg->Hq + (int64_t)cfg->Hk < 1) return PACE_EINVAL;
  if (cfg->d < 2 || cfg->d % 2 || cfg->rd < 2 || cfg->rd % 2 || cfg->rd > cfg->d) return PACE_EINVAL;
  if (cfg->interleaved != 0 && cfg->interleaved != 1) return PACE_EINVAL;
  if (cfg->io_dtype != PACE_IO_F32 && cfg->io_dtype != PACE_IO_BF16) return PACE_EINVAL;
  if (!fits_f32(magnitude)) return PACE_EINVAL;
  if (cfg->d > 1024 || cfg->rd > 512 || cfg->Hq > kMaxQueryHeads || cfg->Hk > kMaxQueryHeads) return PACE_EUNSUPPORTED;
  if (n == 0) return PACE_OK;
  if (!positions || !freqs || !aligned(positions, 4) || !aligned(freqs, 8)) return PACE_EINVAL;
  const size_t e = io_bytes(cfg->io_dtype);
  // the wide form moves 8 channels at once
  bool wide = cfg->d % 8 == 0 && cfg->rd % (cfg->interleaved ? 8 : 16) == 0;
  struct Side {
    int32_t H;
    const void* in;
    int64_t s_in;
    void* out;
    int64_t s_out;
  } sides[2] = {{cfg->Hq, q, q_stride, q_out, q_out_stride}, {cfg->Hk, k, k_stride, k_out, k_out_stride}};
  for (const Side& s : sides) {
    if (s.H == 0) continue;
    const int64_t width = (int64_t)s.H * cfg->d;
    if (!s.in || !s.out || s.s_in < width || s.s_out < width) return PACE_EINVAL;
    if (!spans(n, s.s_in, (int64_t)e) || !spans(n, s.s_out, (int64_t)e)) return PACE_EINVAL;
    if (!aligned(s.in, e) || !aligned(s.out, e)) return PACE_EINVAL;
    if (s.in == s.out && s.s_in != s.s_out) return PACE_EINVAL;
    wide = wide && aligned(s.in, 16) && aligned(s.out, 16) && (s.s_in * e) % 16 == 0 && (s.s_out * e) % 16 == 0;
  }
  RotaryParams p{};
  p.positions = positions;
  p.freqs = freqs;
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.q_stride = q_stride; p.k_stride = k_stride;
  p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
  p.magnitude = (float)magnitude;
  p.n = n; p.Hq = cfg->Hq; p.Hk = cfg->Hk; p.d = cfg->d; p.rd = cfg->rd;
  p.interleaved = cfg->interleaved;
  p.inverse = inverse != 0;
  p.copy_q = q != q_out; p.copy_k = k != k_out;
  for (int32_t done = 0; done < n;) {
    p.n = std::min(n - done, kRotaryTokens);
    const hipError_t err = launch_rotary(p, cfg->io_dtype == PACE_IO_BF16, wide, (hipStream_t)stream);
    if (err != hipSuccess) return PACE_EHIP;
    if (p.n == n - done) break;
    done += p.n;
    p.positions += p.n;
    auto on = [&](const void* at, int64_t stride) { return (char*)at + (int64_t)p.n * stride * (int64_t)e; };
    if (cfg->Hq) p.q = on(p.q, q_stride), p.q_out = on(p.q_out, q_out_stride);
    if (cfg->Hk) p.k = on(p.k, k_stride), p.k_out = on(p.k_out, k_out_stride);
  }
  return PACE_OK;
}

pace_status pace_cache_layout(const pace_cache_cfg* cfg, pace_cache_layout_info* out) {
  if (!out) return PACE_EINVAL;
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  const int bits = cache_bits(cfg->kind);
  const CacheRecord r = cache_record(cfg->d, cfg->group, cfg->page, bits);
  out->record_bytes = r.total;
  out->page_bytes = (size_t)r.total * cfg->Hkv;
  out->cache_bytes = out->page_bytes * cfg->num_pages;
  out->bits_per_value = bits + 16.0 / cfg->group;
  return PACE_OK;
}

static void fill_io(CacheIoParams* p, const pace_cache_cfg* c, const int32_t* table, const int32_t* positions, int32_t T,
                    int64_t ks, int64_t vs) {
  p->table = table;
  p->positions = positions;
  p->k_stride = ks;
  p->v_stride = vs;
  p->B = c->B; p->T = T; p->Hkv = c->Hkv;
  p->page_shift = log2_of(c->page);
  p->num_pages = c->num_pages;
  p->max_pages = c->max_pages;
}

pace_status pace_cache_write(const pace_cache_cfg* cfg, void* cache, const int32_t* page_table,
                             const int32_t* positions, int32_t T, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, void* stream) {
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  if (T < 0) return PACE_EINVAL;
  if (T == 0) return PACE_OK;
  if (cache_io_blocks(cfg->B, T, cfg->Hkv) * 256 > kMaxThreads) return PACE_EUNSUPPORTED;
  const int64_t width = (int64_t)cfg->Hkv * cfg->d, n = (int64_t)cfg->B * T;
  if (!cache || !page_table || !positions || !aligned(cache, 256) || !aligned(page_table, 4) ||
      !aligned(positions, 4) || !rows_ok(k, n, k_stride, width, cfg->io_dtype) ||
      !rows_ok(v, n, v_stride, width, cfg->io_dtype))
    return PACE_EINVAL;
  CacheIoParams p{};
  fill_io(&p, cfg, page_table, positions, T, k_stride, v_stride);
  p.cache = (uint8_t*)cache;
  p.k_in = k;
  p.v_in = v;
  const hipError_t e = launch_cache_write(p, cfg->kind, cfg->d, cfg->group, cfg->io_dtype == PACE_IO_BF16,
                                          (hipStream_t)stream);
  return e == hipSuccess ? PACE_OK : PACE_EHIP;
}

pace_status pace_cache_read(const pace_cache_cfg* cfg, const void* cache,
                            const int32_t* page_table, const int32_t* positions, int32_t T,
                            void* k, int64_t k_stride, void* v, int64_t v_stride, void* stream) {
  const pace_status st = validate(cfg);
  if (st != PACE_OK) return st;
  if (T < 0) return PACE_EINVAL;
  if (T == 0) return PACE_OK;
  if (cache_io_blocks(cfg->B, T, cfg->Hkv) * 256 > kMaxThreads) return PACE_EUNSUPPORTED;
  const int64_t width = (int64_t)cfg->Hkv * cfg->d, n = (int64_t)cfg->B * T;
  if (!cache || !page_table || !positions || !aligned(cache, 256) || !aligned(page_table, 4) ||
      !aligned(positions, 4) || !rows_ok(k, n, k_stride, width, cfg->io_dtype) ||
      !rows_ok(v, n, v_stride, width, cfg->io_dtype))
    return PACE_EINVAL;
  CacheIoParams p{};
  fill_io(&p, cfg, page_table, positions, T, k_stride, v_stride);
  p.cache = (uint8_t*)const_cast<void*>(cache);
  p.k_out = k;
  p.v_out = v;
  const hipError_t e = launch_cache_read(p, cfg->kind, cfg->d, cfg->group, cfg->io_dtype == PACE_IO_BF16,
                                         (hipStream_t)stream);
  return e == hipSuccess ? PACE_OK : PACE_EHIP;
}

pace_status pace_tree_bits(const int32_t* parents, int32_t T, uint32_t* bits) {
  if (!parents || !bits || T < 1) return PACE_EINVAL;
  for (int i = 0; i < T; ++i)
    if (parents[i] < -1 || parents[i] >= i) return PACE_EINVAL;
  const size_t W = ((size_t)T + 31) / 32;
  for (int i = 0; i < T; ++i) {
    uint32_t* row = bits + (size_t)i * W;
    for (size_t w = 0; w < W; ++w) row[w] = parents[i] < 0 ? 0u : bits[(size_t)parents[i] * W + w];
    row[i / 32] |= 1u << (i % 32);
  }
  return PACE_OK;
}

pace_status pace_cache_attention_workspace_bytes(const pace_cache_cfg* cfg, int32_t T,
                                                 int32_t max_len, size_t* bytes_out) {
  if (!bytes_out) return PACE_EINVAL;
  AttnPlan plan;
  size_t need = 0;
  const pace_status st = attn_sizes(cfg, T, max_len, &plan, &need);
  if (st != PACE_OK) return st;
  *bytes_out = need;
  return PACE_OK;
}

pace_status pace_cache_attention(const pace_cache_cfg* cfg, const void* cache,
                                 const int32_t* page_table, const void* q, int64_t q_stride,
                                 int32_t T, const int32_t* ctx_lens, const int32_t* draft_lens,
                                 const uint32_t* tree, int64_t tree_stride, double scale,
                                 int32_t max_len, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  AttnPlan plan;
  size_t need = 0;
  const pace_status st = attn_sizes(cfg, T, max_len, &plan, &need);
  if (st != PACE_OK) return st;
  if (!cache || !page_table || !ctx_lens || !o || !aligned(cache, 256) || !aligned(page_table, 4) ||
      !aligned(ctx_lens, 4) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(draft_lens, 4) ||
      !aligned(tree, 4) || !rows_ok(q, (int64_t)cfg->B * T, q_stride, (int64_t)cfg->Hq * cfg->d, cfg->io_dtype))
    return PACE_EINVAL;
  if (tree_stride < 0 || !spans(cfg->B, tree_stride, 4) || !fits_f32(scale * kLog2e)) return PACE_EINVAL;
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return PACE_EINVAL;
  AttnParams p{};
  p.cache = (const uint8_t*)cache;
  p.table = page_table;
  p.q = q;
  p.q_stride = q_stride;
  p.ctx_lens = ctx_lens;
  p.draft_lens = draft_lens;
  p.tree = tree;
  p.tree_stride = tree_stride;
  p.o = o;
  p.lse = lse;
  p.scale_log2e = (float)(scale * kLog2e);
  p.B = cfg->B; p.T = T; p.Hq = cfg->Hq; p.Hkv = cfg->Hkv;
  p.gamma = cfg->Hq / cfg->Hkv;
  p.R = T * p.gamma;
  p.page_shift = log2_of(cfg->page);
  p.num_pages = cfg->num_pages;
  p.max_pages = cfg->max_pages;
  p.nsplit = plan.nsplit; p.chunk = plan.chunk;
  p.row_blocks = plan.row_blocks;
  if (need) {
    p.part_o = (float*)workspace;
    p.part_lse = p.part_o + (size_t)plan.nsplit * cfg->B * cfg->Hkv * (size_t)p.R * cfg->d;
  }
  const hipError_t e = launch_attention(p, plan, cfg->kind, cfg->d, cfg->group, cfg->io_dtype == PACE_IO_BF16,
                                        (hipStream_t)stream);
  return e == hipSuccess ? PACE_OK : PACE_EHIP;
}

}  // extern "C"
