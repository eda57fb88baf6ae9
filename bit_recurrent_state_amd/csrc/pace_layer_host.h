// Host-side view of a gated-delta layer, shared by the entry points that take a pace_layer_cfg: its
// validation, the geometry of its packed state, and the layer's part of a decode launch.
#pragma once

#include <hip/hip_runtime.h>

#include "pace_internal.h"

namespace pace {

// Structural validity (PACE_EINVAL) and kernel coverage (PACE_EUNSUPPORTED).
inline pace_status validate(const pace_layer_cfg* c) {
  if (!c) return PACE_EINVAL;
  const bool bf16_state = c->state_kind == PACE_STATE_BF16;
  if (c->B <= 0 || c->Hv <= 0 || c->Hk <= 0 || c->dk <= 0 || c->dv <= 0 || c->dP <= 0 || c->chunk <= 0)
    return PACE_EINVAL;
  if (c->Hv % c->Hk != 0) return PACE_EINVAL;
  if (c->state_kind != PACE_STATE_SYM && c->state_kind != PACE_STATE_ASYM && !bf16_state) return PACE_EINVAL;
  // a bf16 state has no scale groups and no per-head bit widths
  if (bf16_state && c->head_bits) return PACE_EINVAL;
  if (!bf16_state && (c->group <= 0 || c->dk % c->group != 0)) return PACE_EINVAL;
  if (c->buf_kind != PACE_BUF_INT8 && c->buf_kind != PACE_BUF_K4_VBF16) return PACE_EINVAL;
  if (c->io_dtype != PACE_IO_F32 && c->io_dtype != PACE_IO_BF16) return PACE_EINVAL;
  if (c->head_bits)
    for (int h = 0; h < c->Hv; ++h)
      if (c->head_bits[h] != 4 && c->head_bits[h] != 8) return PACE_EINVAL;
  // kernel coverage
  if (!((c->dk == 64 || c->dk == 128) && c->dv == c->dk)) return PACE_EUNSUPPORTED;
  if (!bf16_state && c->group != 32 && c->group != 64) return PACE_EUNSUPPORTED;
  if (c->dP > kMaxPeriod) return PACE_EUNSUPPORTED;
  if (c->Hv > kMaxHeads || c->B > 65535) return PACE_EUNSUPPORTED;
  // the prefill kernels round where a 64-token sub-block ends on a multiple of the period
  if (c->chunk % 64 != 0) return PACE_EUNSUPPORTED;
  // 4-bit zero points pack two groups of one column per byte
  if (c->state_kind == PACE_STATE_ASYM && (c->dk / c->group) % 2 != 0) return PACE_EUNSUPPORTED;
  // a bf16 state is served with the int8 decode buffer only
  if (bf16_state && c->buf_kind != PACE_BUF_INT8) return PACE_EUNSUPPORTED;
  return PACE_OK;
}

inline int head_bits_of(const pace_layer_cfg* c, int h) { return c->head_bits ? c->head_bits[h] : 4; }

struct StateGeom {
  RecordLayout r4, r8;
  uint64_t mask8 = 0;
  size_t seq_stride = 0;
};

inline StateGeom state_geom(const pace_layer_cfg* c) {
  StateGeom g;
  if (c->state_kind == PACE_STATE_BF16) {     // one dv x dk bf16 record per head
    const uint32_t rec = (uint32_t)((size_t)c->dk * c->dv * 2);
    g.r4 = RecordLayout{rec, 0u, 0u, rec};
    g.r8 = g.r4;
    g.seq_stride = (size_t)rec * c->Hv;
    return g;
  }
  const bool asym = c->state_kind == PACE_STATE_ASYM;
  g.r4 = record_layout(c->dk, c->dv, c->group, asym, 4);
  g.r8 = record_layout(c->dk, c->dv, c->group, asym, 8);
  for (int h = 0; h < c->Hv; ++h) {
    const bool is8 = head_bits_of(c, h) == 8;
    if (is8) g.mask8 |= 1ull << h;
    g.seq_stride += is8 ? g.r8.total : g.r4.total;
  }
  return g;
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The state, the buffer and the layer's sizes; tokens, masks and what the launch does are the caller's.
inline DecodeParams layer_params(const pace_layer_cfg* cfg, const void* state, const void* buffer) {
  const StateGeom g = state_geom(cfg);
  const BufferLayout bl = buffer_layout(*cfg);
  DecodeParams p{};
  p.state = (uint8_t*)const_cast<void*>(state);
  p.buffer = (uint8_t*)const_cast<void*>(buffer);
  p.mask8 = g.mask8;
  p.rec4 = g.r4.total; p.rec8 = g.r8.total;
  p.scales_off4 = g.r4.codes; p.zeros_off4 = g.r4.codes + g.r4.scales;
  p.scales_off8 = g.r8.codes; p.zeros_off8 = g.r8.codes + g.r8.scales;
  p.seq_stride = g.seq_stride;
  p.off_kc = bl.kc; p.off_ks = bl.ks; p.off_v = bl.v; p.off_vs = bl.vs;
  p.off_a = bl.a; p.off_beta = bl.beta;
  p.B = cfg->B; p.Hv = cfg->Hv; p.Hk = cfg->Hk; p.gamma = cfg->Hv / cfg->Hk;
  p.dP = cfg->dP; p.group = cfg->group; p.asym = cfg->state_kind == PACE_STATE_ASYM;
  p.bf16_state = cfg->state_kind == PACE_STATE_BF16;
  p.io_bf16 = cfg->io_dtype == PACE_IO_BF16;
  return p;
}

// A launch that folds buffered tokens into the state (flush_only as in DecodeParams).  There is no token: the
// kernel's unconditional token loads read the state instead (every index they form is below B * Hk * dk * 4
// bytes, which the state always exceeds) and never use the values.
inline DecodeParams flush_params(const pace_layer_cfg* cfg, void* state, void* buffer, int flush_only) {
  DecodeParams p = layer_params(cfg, state, buffer);
  p.flush_only = flush_only;
  p.q = p.k = p.v = state;
  p.a = p.beta = (const float*)state;
  return p;
}

}  // namespace pace
