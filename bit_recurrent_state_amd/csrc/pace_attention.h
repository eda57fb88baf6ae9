// Attention for drafted tokens over the quantised paged cache (include/pace_cache.h:
// pace_cache_attention; the cache's layout there).
//
// Mathematics.  The T * gamma rows of one key/value head (row r: token r div gamma, query head
// r mod gamma) are the columns of S^T = K Q^T, so a matrix instruction v_mfma_f32_16x16x32_f16
// takes 16 cached tokens against 16 rows.  Codes are exact in fp16: keys enter as they are
// stored and their scales multiply the fp32 scores of a token.  Scores leave the instruction
// with four consecutive tokens of one row in a lane, and the product O^T = V^T P^T takes
// its eight tokens a lane in any order, so with values stored by quads of tokens the weights go
// straight from registers back into the matrix unit: no LDS, no lane exchange but the row
// maximum.  Value scales multiply the weights (they belong to a token and a channel group),
// in units of a running power of two V >= every value scale seen, so that they fit fp16.
// The softmax keeps a running maximum that may lag by kLag octaves (weights up to
// 2^(kLift + kLag), which fp16 holds), so accumulators are rescaled only when it is exceeded.
//
// Work split: a workgroup's four waves take either different 16-row tiles of the same tokens
// (row_waves) or different tokens of the same rows, joined in LDS at the end; long contexts are
// also cut over workgroups, joined by a second kernel.
#pragma once

#include <hip/hip_runtime.h>

#include "pace_cache_internal.h"
#include "pace_lanes.h"
#include "pace_numerics.h"

namespace pace {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

constexpr int kStep = 32;        // tokens a wave takes at once

constexpr float kLift = 7.f;     // weights are 2^kLift exp(s - m): fp16 stays normal down to 2^-21
constexpr float kLag = 8.f;      // octaves the running maximum may lag behind
constexpr float kFloor = -1e30f; // running maximum before any token

__device__ inline half2_t h2(uint32_t x) { return __builtin_bit_cast(half2_t, x); }
__device__ inline uint32_t u2(half2_t x) { return __builtin_bit_cast(uint32_t, x); }
__device__ inline half8_t frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 w = {a, b, c, d};
  return __builtin_bit_cast(half8_t, w);
}
// Two fp32 -> packed fp16, round to nearest even.
__device__ inline uint32_t pk_f16(float a, float b) {
  const half2_t h = {(_Float16)a, (_Float16)b};
  return u2(h);
}
// The rest of (a, b) after their fp16 rounding `hi`.  hi goes through an empty statement first, so
// that the matrix operand and the subtraction see the same bits: without it the compiler forms the
// operand with a fused multiply-and-round and the subtrahend with two roundings, which differ
// by a unit where the product lies next to a tie.
__device__ inline uint32_t pk_rest(float a, float b, uint32_t& hi) {
  asm("" : "+v"(hi));
  return pk_f16(a - (float)h2(hi)[0], b - (float)h2(hi)[1]);
}
__device__ inline float4_t mfma(half8_t a, half8_t b, float4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Stored codes as fp16 operands, exactly.  int8: byte u next to 0x64 is the fp16 number 1024 + u,
// from which 1152 is taken.  int4: the low nibble likewise; 1024 + 16 n for the high one, of which
// a sixteenth less 72 is taken in one fused step.  One operation a code and a little.  (A field
// alone is a subnormal fp16 number, which would save the subtraction, but the matrix unit sums
// products of subnormals to 2^-15 only.)
template <int KIND>
struct Codes {
  // four 8-bit fields
  static __device__ void four(uint32_t x, uint32_t& a, uint32_t& b) {
    if constexpr (KIND == PACE_CACHE_FP8) {
      a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)x, 1.0f, false));
      b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)x, 1.0f, true));
    } else {
      const half2_t bias = {(_Float16)1152.f, (_Float16)1152.f};
      a = u2(h2(__builtin_amdgcn_perm(x, 0x64646464u, 0x00050004u)) - bias);
      b = u2(h2(__builtin_amdgcn_perm(x, 0x64646464u, 0x00070006u)) - bias);
    }
  }
  // the low nibbles of bytes 0, 2 and the high ones; magic: 0x64006400 in a vector register, so
  // that mask and exponent go in with one operation (it takes one scalar constant only)
  static __device__ void two(uint32_t x, uint32_t magic, uint32_t& lo, uint32_t& hi) {
    const half2_t b0 = {(_Float16)1032.f, (_Float16)1032.f}, b1 = {(_Float16)72.f, (_Float16)72.f};
    const half2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    lo = u2(h2((x & 0x000F000Fu) | magic) - b0);
    hi = u2(h2((x & 0x00F000F0u) | magic) * sixteenth - b1);
  }
  // channels 32 B + 8 g .. + 7 of a token
  static __device__ half8_t key(const uint32_t* k, int B, uint32_t magic) {
    uint32_t w[4];
    if constexpr (KIND == PACE_CACHE_INT4) {
      two(k[B], magic, w[0], w[1]);
      two(k[B] >> 8, magic, w[2], w[3]);
    } else {
      four(k[2 * B], w[0], w[1]);
      four(k[2 * B + 1], w[2], w[3]);
    }
    return frag(w[0], w[1], w[2], w[3]);
  }
  // channels 32 B + 2 n + {0, 1} of the lane's quads of both tiles
  static __device__ void values(const uint32_t* v0, const uint32_t* v1, int B, uint32_t magic, half8_t (&f)[2]) {
    if constexpr (KIND == PACE_CACHE_INT4) {
      uint32_t l[4], h[4];
      two(v0[B], magic, l[0], h[0]);
      two(v0[B] >> 8, magic, l[1], h[1]);
      two(v1[B], magic, l[2], h[2]);
      two(v1[B] >> 8, magic, l[3], h[3]);
      f[0] = frag(l[0], l[1], l[2], l[3]);
      f[1] = frag(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t w[4];
        four(v0[2 * B + e], w[0], w[1]);
        four(v1[2 * B + e], w[2], w[3]);
        f[e] = frag(w[0], w[1], w[2], w[3]);
      }
    }
  }
};

// One lane's share of the codes of a 16-token tile, or of its quads' values: LB bytes.
template <int LB>
struct Raw {
  uint32_t w[LB / 4];
};
template <int LB, int LANES>
__device__ inline Raw<LB> load_raw(const uint8_t* base, int lane) {
  Raw<LB> r;
  if constexpr (LB == 8) {
    const uint2 v = *(const uint2*)(base + lane * 8);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < LB / 16; ++i) {
      const uint4 v = *(const uint4*)(base + i * (LANES * 16) + lane * 16);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

// bf16 scales of a lane's quad, all groups.
template <int NG>
struct Scales {
  uint32_t w[NG][2];
  __device__ float get(int G, int t) const {
    const uint32_t x = w[G][t >> 1];
    return __uint_as_float((t & 1) ? (x & 0xFFFF0000u) : (x << 16));
  }
};
template <int NG>
__device__ inline Scales<NG> load_scales(const uint8_t* base) {
  Scales<NG> s;
  if constexpr (NG == 1) {
    const uint2 v = *(const uint2*)base;
    s.w[0][0] = v.x; s.w[0][1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      const uint4 v = *(const uint4*)(base + 16 * i);
      s.w[2 * i][0] = v.x; s.w[2 * i][1] = v.y; s.w[2 * i + 1][0] = v.z; s.w[2 * i + 1][1] = v.w;
    }
  }
  return s;
}

__device__ inline ushort2_t us2(uint32_t x) { return __builtin_bit_cast(ushort2_t, x); }
// Sum over a row's four lanes.
__device__ inline float rows_sum(float x) {
  LanePair a = pair16(__float_as_uint(x));
  x = __uint_as_float(a.lo) + __uint_as_float(a.hi);
  a = pair32(__float_as_uint(x));
  return __uint_as_float(a.lo) + __uint_as_float(a.hi);
}
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

template <int KIND, int D, int GROUP, bool BF16>
struct Shape {
  static constexpr int BITS = KIND == PACE_CACHE_INT4 ? 4 : 8;
  static constexpr int LB = D * BITS / 32;      // bytes of a lane's codes
  static constexpr int NB = D / 32;             // 32-channel blocks
  static constexpr int NG = D / GROUP;          // scale groups
  static constexpr int BPG = GROUP / 32;        // blocks a group
  static constexpr int PIECES = BF16 ? 1 : 2;   // fp16 pieces of q and of the weights
};

// Running state of one 16-row tile in a wave.
template <int D>
struct Tile {
  float4_t acc[D / 16];   // [32 G + 2 (4 g + i) + e] of row lane % 16, at index 2 G + e, element i
  float m, l;             // running maximum (base-2, all lanes of a row agree), sum of this lane
};

template <int KIND, int D, int GROUP, bool BF16, int RT, int NW>
__global__ __launch_bounds__(NW * 64) void attn_kernel(AttnParams p) {
  using S = Shape<KIND, D, GROUP, BF16>;
  using C = Codes<KIND>;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int split = id % p.nsplit;
  id /= p.nsplit;
  const int rb = id % p.row_blocks;
  id /= p.row_blocks;
  const int h = id % p.Hkv, b = id / p.Hkv;
  const int rw = wave % p.row_waves, tw = wave / p.row_waves, nt = NW / p.row_waves;
  const int row0 = (rb * p.row_waves + rw) * (RT * 16);

  const int page = 1 << p.page_shift;
  const CacheRecord rec = cache_record(D, GROUP, page, S::BITS);
  const int capacity = p.max_pages << p.page_shift;
  const int ctx = min(max(p.ctx_lens[b], 0), capacity);
  const int drafts = p.draft_lens ? min(max(p.draft_lens[b], 0), p.T) : p.T;
  // the last position any row of this workgroup can see, + 1
  const int last_row = min((rb + 1) * p.row_waves * RT * 16, p.R) - 1;
  const int seen = p.tree ? drafts : min(drafts, last_row / p.gamma + 1);
  const int end = uniform(drafts > 0 ? (int)min((int64_t)ctx + seen, (int64_t)capacity) : 0);
  const int lo = uniform(split * p.chunk), hi = uniform(split == p.nsplit - 1 ? end : min(end, lo + p.chunk));

  // ---- the step's two 16-token tiles; a tile past the end is replaced and masked
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  const int last_tile = uniform(max(end - 1, 0) >> 4);
  struct Where {
    const uint8_t* at[2];
    uint32_t off[2];
    bool there[2];
  };
  auto where = [&](int s0) {
    Where w;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tile = min((s0 >> 4) + u, last_tile);
      const int pg = uniform(table[(tile << 4) >> p.page_shift]);
      w.there[u] = pg >= 0 && pg < p.num_pages;
      w.at[u] = p.cache + ((int64_t)(w.there[u] ? pg : 0) * p.Hkv + h) * rec.total;
      w.off[u] = (uint32_t)((tile << 4) & (page - 1));
    }
    return w;
  };
  Raw<S::LB> kr[2], vr[2];
  Scales<S::NG> ks[2], vs[2];
  // use == 0 (no further step): every lane asks for the tile's first bytes, one cache line
  auto load_keys = [&](const Where& w, int use) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kr[u] = load_raw<S::LB, 64>(w.at[u] + w.off[u] * (D * S::BITS / 8), lane & use);
      ks[u] = load_scales<S::NG>(w.at[u] + rec.codes + (w.off[u] / 4 + (g & use)) * (S::NG * 8));
    }
  };
  auto load_values = [&](const Where& w, int use) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* v = w.at[u] + rec.codes + rec.scales;
      vr[u] = load_raw<S::LB, 16>(v + (w.off[u] / 4 + (g & use)) * (D * S::BITS / 2), n & use);
      vs[u] = load_scales<S::NG>(v + rec.codes + (w.off[u] / 4 + (g & use)) * (S::NG * 8));
    }
  };
  const int first = lo + tw * kStep, stride = nt * kStep;
  Where cur;
  if (first < hi) {
    cur = where(first);
    load_keys(cur, -1);
    load_values(cur, -1);
  }

  // ---- the rows' queries as fp16 operands, scaled by a power of two to [2^13, 2^14)
  half8_t qf[S::PIECES][RT][S::NB];
  float cs[RT];
  int tok[RT];                 // the row's token, or -1
  const uint32_t* bits[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = row0 + t * 16 + n, i = r / p.gamma;
    tok[t] = (r < p.R && i < drafts) ? i : -1;
    bits[t] = p.tree ? p.tree + (int64_t)b * p.tree_stride + (int64_t)max(tok[t], 0) * ((p.T + 31) / 32) : nullptr;
    float x[S::NB][8];
    float mx = 0.f;
    const int64_t at = ((int64_t)b * p.T + max(tok[t], 0)) * p.q_stride + (int64_t)(h * p.gamma + (r - i * p.gamma)) * D + 8 * g;
#pragma unroll
    for (int G = 0; G < S::NB; ++G) {
      if constexpr (BF16) {
        const uint4 v = tok[t] >= 0 ? *(const uint4*)((const uint16_t*)p.q + at + 32 * G) : uint4{0, 0, 0, 0};
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[G][2 * j] = __uint_as_float(w[j] << 16);
          x[G][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 v = tok[t] >= 0 ? *(const float4*)((const float*)p.q + at + 32 * G + 4 * j) : float4{0, 0, 0, 0};
          x[G][4 * j] = v.x; x[G][4 * j + 1] = v.y; x[G][4 * j + 2] = v.z; x[G][4 * j + 3] = v.w;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(x[G][j]));
    }
    mx = rows_max(mx);
    // exponent field e of the maximum: |x| < 2^(e - 126); 2^(140 - e) takes it under 2^14
    int e = (int)(__float_as_uint(mx) >> 23) & 255;
    e = min(max(e, 14), 254);
    float up = __uint_as_float((uint32_t)min(140 - e + 127, 254) << 23);
    // scores are cs * (K q); the scale's sign goes into q, so that cs > 0 and masks can be -inf
    cs[t] = p.scale_log2e == 0.f ? 1.f : fmaxf(fabsf(p.scale_log2e) / up, 0x1p-126f);
    up = p.scale_log2e == 0.f ? 0.f : copysignf(up, p.scale_log2e);
#pragma unroll
    for (int B = 0; B < S::NB; ++B) {
      uint32_t w[4], z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = x[B][2 * k] * up, c = x[B][2 * k + 1] * up;
        w[k] = pk_f16(a, c);
        if constexpr (!BF16) z[k] = pk_rest(a, c, w[k]);
      }
      qf[0][t][B] = frag(w[0], w[1], w[2], w[3]);
      if constexpr (!BF16) qf[1][t][B] = frag(z[0], z[1], z[2], z[3]);
    }
  }

  Tile<D> T[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) T[t].acc[j] = float4_t{0, 0, 0, 0};
    T[t].m = kFloor;
    T[t].l = 0.f;
  }
  uint32_t magic = 0x64006400u;
  asm("" : "+v"(magic));
  float vunit = 0.f, vinv = 0.f;   // the running power of two over the value scales, its inverse

  for (int s0 = first; s0 < hi; s0 += stride) {
    const bool more = s0 + stride < hi;
    const int use = more ? -1 : 0;
    const Where next = where(more ? s0 + stride : s0);

    // ---- scores over cs: s[t][u][i] of token s0 + 16 u + 4 g + i and row n of tile t
    float s[RT][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int G = 0; G < S::NG; ++G) {
        float4_t a[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) a[t] = float4_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < S::BPG; ++j) {
          const int B = G * S::BPG + j;
          const half8_t kf = C::key(kr[u].w, B, magic);
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int c = 0; c < S::PIECES; ++c) a[t] = mfma(kf, qf[c][t][B], a[t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float k = ks[u].get(G, i);
#pragma unroll
          for (int t = 0; t < RT; ++t) s[t][u][i] = G == 0 ? a[t][i] * k : fmaf(a[t][i], k, s[t][u][i]);
        }
      }
    }
    load_keys(next, use);

    // ---- masks, where some row may not see some token of the step
    if (s0 + kStep > ctx || !cur.there[0] || !cur.there[1]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int p0 = s0 + 16 * u + 4 * g;
        uint32_t keep = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = p0 + i;
          const bool held = cur.there[u] && pos < end;
          if (held) keep |= 0xFFu << (8 * i);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int j = pos - ctx;
            bool ok = held && tok[t] >= 0;
            if (ok && j >= 0) ok = p.tree ? (bits[t][j >> 5] >> (j & 31)) & 1u : j <= tok[t];
            s[t][u][i] = ok ? s[t][u][i] : -INFINITY;
          }
        }
        // old bytes may be NaN scales, or NaN codes of fp8, and 0 times NaN is NaN
        const uint32_t k01 = __builtin_amdgcn_perm(keep, keep, 0x01010000u), k23 = __builtin_amdgcn_perm(keep, keep, 0x03030202u);
#pragma unroll
        for (int G = 0; G < S::NG; ++G) {
          vs[u].w[G][0] &= k01;
          vs[u].w[G][1] &= k23;
        }
        if constexpr (KIND == PACE_CACHE_FP8) {
#pragma unroll
          for (int x = 0; x < S::LB / 4; ++x) vr[u].w[x] &= keep;
        }
      }
    }

    // ---- running maximum and value unit; rescale when either is exceeded
    // (scales are not negative: their bf16 patterns compare as integers, two at a time)
    ushort2_t top = us2(vs[0].w[0][0]);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int G = 0; G < S::NG; ++G)
#pragma unroll
        for (int i = 0; i < 2; ++i) top = __builtin_elementwise_max(top, us2(vs[u].w[G][i]));
    const float vmax = rows_max(__uint_as_float((uint32_t)max(top[0], top[1]) << 16));
    float mx[RT];
    bool grow = vmax > vunit;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float x = fmaxf(s[t][0][0], s[t][0][1]);
      x = fmaxf(fmaxf(x, s[t][0][2]), s[t][0][3]);
      x = fmaxf(fmaxf(x, s[t][1][0]), s[t][1][1]);
      mx[t] = rows_max(fmaxf(fmaxf(x, s[t][1][2]), s[t][1][3])) * cs[t];
      grow |= mx[t] > T[t].m + kLag;
    }
    if (__any(grow)) {
      float vf = 1.f;
      if (vmax > vunit) {
        // a power of two over vmax with two octaves to spare (value scales end at 2^125)
        const uint32_t e = min((__float_as_uint(vmax) >> 23) + 3u, 253u);
        const float now = __uint_as_float(e << 23);
        vinv = __uint_as_float((254u - e) << 23);
        vf = vunit * vinv;
        vunit = now;
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float now = fmaxf(T[t].m, mx[t]);
        const float f = __builtin_amdgcn_exp2f(T[t].m - now);
        T[t].m = now;
        T[t].l *= f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) T[t].acc[j][i] *= f * vf;
      }
    }

    // ---- weights, and O^T += V^T P^T
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float m = T[t].m - kLift;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][u][i] = __builtin_amdgcn_exp2f(fmaf(s[t][u][i], cs[t], -m));   // one rounding, of the difference
          T[t].l += s[t][u][i];
        }
    }
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      half8_t pf[S::PIECES][RT];
      float sc[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[u][i] = vs[u].get(G, i) * vinv;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        uint32_t w[4], z[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = s[t][u][i] * sc[u][i];
          // the token order in which the value codes unpack
          constexpr int o1 = KIND == PACE_CACHE_INT4 ? 2 : 1, o2 = 3 - o1;
          w[2 * u] = pk_f16(x[0], x[o1]);
          w[2 * u + 1] = pk_f16(x[o2], x[3]);
          if constexpr (!BF16) {
            z[2 * u] = pk_rest(x[0], x[o1], w[2 * u]);
            z[2 * u + 1] = pk_rest(x[o2], x[3], w[2 * u + 1]);
          }
        }
        pf[0][t] = frag(w[0], w[1], w[2], w[3]);
        if constexpr (!BF16) pf[1][t] = frag(z[0], z[1], z[2], z[3]);
      }
#pragma unroll
      for (int jb = 0; jb < S::BPG; ++jb) {
        const int B = G * S::BPG + jb;
        half8_t vf[2];
        C::values(vr[0].w, vr[1].w, B, magic, vf);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int c = 0; c < S::PIECES; ++c) T[t].acc[2 * B + e] = mfma(vf[e], pf[c][t], T[t].acc[2 * B + e]);
      }
    }
    load_values(next, use);
    cur = next;
  }

  // ---- this wave's result: o = acc V / l of its tokens, base-2 log of the sum
  float lse[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float l = rows_sum(T[t].l);
    if (tok[t] < 0) l = 0.f;     // a row past the drafted tokens saw what it should not have
    const float inv = l == 0.f ? 0.f : vunit / l;      // a NaN row stays NaN
    lse[t] = l == 0.f ? -INFINITY : T[t].m - kLift + __builtin_amdgcn_logf(l);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) T[t].acc[j][i] *= inv;
  }

  // ---- joined over the waves that took other tokens of the same rows
  if (nt > 1) {
    constexpr int REGS = D / 4;   // accumulator registers of a tile
    constexpr int SLOT = RT * (REGS + 1) * 64;
    if (tw > 0) {
      float* mine = lds + (size_t)((tw - 1) * p.row_waves + rw) * SLOT;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[(t * (REGS + 1) + 4 * j + i) * 64 + lane] = T[t].acc[j][i];
        mine[(t * (REGS + 1) + REGS) * 64 + lane] = lse[t];
      }
    }
    __syncthreads();
    if (tw > 0) return;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float top = lse[t];
      for (int w = 1; w < nt; ++w)
        top = fmaxf(top, lds[(size_t)((w - 1) * p.row_waves + rw) * SLOT + (t * (REGS + 1) + REGS) * 64 + lane]);
      const float base = top == -INFINITY ? 0.f : top;
      float f = __builtin_amdgcn_exp2f(lse[t] - base), sum = f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) T[t].acc[j][i] *= f;
      for (int w = 1; w < nt; ++w) {
        const float* from = lds + (size_t)((w - 1) * p.row_waves + rw) * SLOT + t * (REGS + 1) * 64 + lane;
        f = __builtin_amdgcn_exp2f(from[REGS * 64] - base);
        sum += f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) T[t].acc[j][i] = fmaf(from[(4 * j + i) * 64], f, T[t].acc[j][i]);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      lse[t] = sum == 0.f ? -INFINITY : base + __builtin_amdgcn_logf(sum);
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) T[t].acc[j][i] *= inv;
    }
  }

  // ---- out: final rows, or this piece's part
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = row0 + t * 16 + n;
    if (r >= p.R) continue;
    const int i = r / p.gamma;
    if (p.nsplit > 1) {
      const int64_t at = ((int64_t)(split * p.B + b) * p.Hkv + h) * p.R + r;
      if (g == 0) p.part_lse[at] = lse[t];
      if (lse[t] == -INFINITY) continue;
      float* o = p.part_o + at * D + 8 * g;
#pragma unroll
      for (int G = 0; G < S::NB; ++G) {
        const float4_t a = T[t].acc[2 * G], c = T[t].acc[2 * G + 1];
        *(float4*)(o + 32 * G) = float4{a[0], c[0], a[1], c[1]};
        *(float4*)(o + 32 * G + 4) = float4{a[2], c[2], a[3], c[3]};
      }
    } else {
      const int64_t at = ((int64_t)b * p.T + i) * p.Hq + h * p.gamma + (r - i * p.gamma);
      if (g == 0 && p.lse) p.lse[at] = lse[t] * 0.69314718055994530942f;
#pragma unroll
      for (int G = 0; G < S::NB; ++G) {
        const float4_t a = T[t].acc[2 * G], c = T[t].acc[2 * G + 1];
        if constexpr (BF16) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __bf16 x = (__bf16)a[k], y = (__bf16)c[k];
            w[k] = (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
          }
          *(uint4*)((uint16_t*)p.o + at * D + 32 * G + 8 * g) = uint4{w[0], w[1], w[2], w[3]};
        } else {
          float* o = (float*)p.o + at * D + 32 * G + 8 * g;
          *(float4*)o = float4{a[0], c[0], a[1], c[1]};
          *(float4*)(o + 4) = float4{a[2], c[2], a[3], c[3]};
        }
      }
    }
  }
}

template <int KIND, int D, int GROUP, bool BF16, int RT, int NW>
hipError_t launch_shape(const AttnParams& p, hipStream_t s) {
  const uint32_t grid = (uint32_t)((int64_t)p.nsplit * p.row_blocks * p.Hkv * p.B);
  const size_t lds = (size_t)(NW - p.row_waves) * RT * (D / 4 + 1) * 64 * sizeof(float);
  attn_kernel<KIND, D, GROUP, BF16, RT, NW><<<grid, NW * 64, lds, s>>>(p);
  return hipGetLastError();
}

template <int KIND, int D, int GROUP, bool BF16>
hipError_t launch_by_plan(const AttnParams& p, const AttnPlan& a, hipStream_t s) {
  if constexpr (D <= 128)
    if (a.row_tiles == 2) return launch_shape<KIND, D, GROUP, BF16, 2, 4>(p, s);
  if (a.waves == 8) return launch_shape<KIND, D, GROUP, BF16, 1, 8>(p, s);
  return launch_shape<KIND, D, GROUP, BF16, 1, 4>(p, s);
}

template <int KIND, int D>
hipError_t launch_by_group(const AttnParams& p, const AttnPlan& a, int group, int io_bf16, hipStream_t s) {
  if (group == 32) return io_bf16 ? launch_by_plan<KIND, D, 32, true>(p, a, s) : launch_by_plan<KIND, D, 32, false>(p, a, s);
  if (group == 64) return io_bf16 ? launch_by_plan<KIND, D, 64, true>(p, a, s) : launch_by_plan<KIND, D, 64, false>(p, a, s);
  if constexpr (D >= 128)
    return io_bf16 ? launch_by_plan<KIND, D, 128, true>(p, a, s) : launch_by_plan<KIND, D, 128, false>(p, a, s);
  return hipErrorInvalidValue;
}

}  // namespace

template <int KIND>
hipError_t launch_attention_kind(const AttnParams& p, const AttnPlan& a, int d, int group, int io_bf16, hipStream_t s) {
  if (d == 64) return launch_by_group<KIND, 64>(p, a, group, io_bf16, s);
  if (d == 128) return launch_by_group<KIND, 128>(p, a, group, io_bf16, s);
  return launch_by_group<KIND, 256>(p, a, group, io_bf16, s);
}

}  // namespace pace
