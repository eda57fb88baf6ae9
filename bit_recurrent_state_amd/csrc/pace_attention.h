// Attention for drafted tokens over the quantised paged cache (include/pace_cache.h:
// pace_cache_attention; the cache's layout there).
//
// Mathematics.  The T * gamma rows of one key/value head (row r: token r div gamma, query head
// r mod gamma) are the columns of S^T = K Q^T, so a matrix instruction v_mfma_f32_16x16x32_f16
// takes 16 cached tokens against 16 rows.  Codes are exact in fp16: keys enter as they are
// stored and their scales (over 2^kDown, see Rows) multiply the fp32 scores of a token.  Scores leave the instruction
// with four consecutive tokens of one row in a lane, and the product O^T = V^T P^T takes
// its eight tokens a lane in any order, so with values stored by quads of tokens the weights go
// straight from registers back into the matrix unit: no lane exchange but the row maximum.
// Value scales multiply the weights (they belong to a token and a channel group), in a running power of
// two of the row and group, so that they fit fp16 (see Sums).
// The softmax keeps a running maximum that may lag by kLag octaves (weights up to
// 2^(kLift + kLag), which fp16 holds), so accumulators are rescaled only when it is exceeded.
//
// Work split: a wave holds one or two 16-row tiles and takes 32 cached tokens at a time, straight
// from memory into registers, the next ones asked for while these are multiplied; the waves of a
// workgroup take different tokens of the same rows and are joined in LDS at the end; long
// contexts are also cut over workgroups, joined by a second kernel (pace_attention.hip); more rows
// are more workgroups over the same tokens.
//
// What bounds it (d = 128, bf16 rows, calls in a graph over three input sets; "busy" from the issue counters over
// the kernel's cycles).  Few rows, 8-bit codes: memory.  3 tokens over 131072, int8: 155 us, 5.3 TB/s, a large
// copy's rate.  Few rows, 4-bit codes: unpacking and latency.  64 tokens over 512 to 8192, g = 64: 87 us, 3.2 TB/s;
// vector unit 52% busy, waves wait a fifth of their time, 1.1 of them a SIMD on average since the
// contexts differ.  Many rows: the vector unit.  512 tokens of 2 sequences over 7680, int8: 223 us, 596
// TFLOP/s; vector unit 74% busy, matrix unit 26%; 22 vector operations a score, unpacking among them.
// Trees between the two: 16 of 25 tokens over 256 to 4096, fp8: 57 us, 220 TFLOP/s, vector unit 44% busy,
// 1.16 waves a SIMD.
//
// (A kernel that unpacked every token once a workgroup, into LDS, for waves on different rows was, before
// weights had units of their rows, 2 to 7% faster for that chunk in int8 and int4 with g >= 64 and in fp32,
// and slower elsewhere: 2% in fp8, 6% with d = 64, 16% with g = 32, 17 and 27% for chunks of 128 and 64
// tokens, 4% for the trees.)
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

constexpr float kLift = 7.f;     // weights are 2^kLift exp(s - m): fp16 stays normal down to 2^-21
constexpr float kLag = 8.f;      // octaves the running maximum may lag behind
constexpr float kFloor = -0x1.fffffep127f;   // running maximum before any token: no finite score is lower
constexpr int kDown = 22;        // key scales enter the scores over 2^kDown (see Rows)
constexpr float kFar = 0x1p20f;  // running maxima past this: scores are rounded before they are compared

__device__ inline half2_t h2(uint32_t x) { return __builtin_bit_cast(half2_t, x); }
__device__ inline ushort2_t us2(uint32_t x) { return __builtin_bit_cast(ushort2_t, x); }
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
  // channels 32 B + 2 n + {0, 1} of the lane's quads of two tiles
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
  // All of them over 2^n, `down` being n << 7 in both halves: exponent fields less n, 0 where that ends
  // under the normal numbers.
  __device__ void lower(uint32_t down) {
#pragma unroll
    for (int G = 0; G < NG; ++G)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[G][i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(us2(w[G][i]), us2(down)));
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

// The larger of two, as the median with `top`, +inf in a register that the compiler cannot look into: fmaxf passes
// lane swaps' words and merged values through a quieting step first (12 of 297 vector operations of a step of
// two row tiles).  Of two NaNs it is +inf: a row of them becomes NaN either way.
__device__ inline float larger(float a, float b, float top) { return __builtin_amdgcn_fmed3f(a, b, top); }
__device__ inline float opaque_top() {
  float top = INFINITY;
  asm("" : "+s"(top));
  return top;
}
// Maximum over a row's four lanes.
__device__ inline float rows_most(float x, float top) {
  LanePair a = pair16(__float_as_uint(x));
  x = larger(__uint_as_float(a.lo), __uint_as_float(a.hi), top);
  a = pair32(__float_as_uint(x));
  return larger(__uint_as_float(a.lo), __uint_as_float(a.hi), top);
}
// Sum over a row's four lanes.
__device__ inline float rows_sum(float x) {
  LanePair a = pair16(__float_as_uint(x));
  x = __uint_as_float(a.lo) + __uint_as_float(a.hi);
  a = pair32(__float_as_uint(x));
  return __uint_as_float(a.lo) + __uint_as_float(a.hi);
}
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
// A NaN row stays one: no sum of it is zero, no lse of it is that of an empty row.
__device__ inline bool is_zero(float x) { return __float_as_uint(x) == 0u; }
__device__ inline bool is_empty(float lse) { return __float_as_uint(lse) == 0xFF800000u; }

template <int KIND, int D, int GROUP, bool BF16>
struct Shape {
  static constexpr int BITS = KIND == PACE_CACHE_INT4 ? 4 : 8;
  static constexpr int LB = D * BITS / 32;      // bytes of a lane's codes of a tile
  static constexpr int NB = D / 32;             // 32-channel blocks
  static constexpr int NG = D / GROUP;          // scale groups
  static constexpr int BPG = GROUP / 32;        // blocks a group
  static constexpr int PIECES = BF16 ? 1 : 2;   // fp16 pieces of q and of the weights
};

// What a workgroup works on.
struct Span {
  int b, h, split, rb;   // sequence, key/value head, piece of the context, block of rows
  int ctx, drafts;       // cached and drafted tokens of the sequence
  int end;               // positions from here on are seen by no row of the workgroup
  int lo, hi;            // its piece
};
__device__ inline Span span_of(const AttnParams& p, int rows) {
  Span w;
  // Workgroups go round the eight XCDs in turn.  Blocks of rows that read the same tokens are put
  // on one XCD, whose L2 then reads them once: of the groups (sequence, head, piece), the first
  // multiple of eight in this way, the rest in order.
  int id = blockIdx.x, group = id;
  w.rb = 0;
  if (p.row_blocks > 1) {
    const int whole = (p.B * p.Hkv * p.nsplit) & ~7, main = whole * p.row_blocks;
    const int local = id < main ? id >> 3 : id - main;
    w.rb = local % p.row_blocks;
    group = id < main ? (local / p.row_blocks) * 8 + (id & 7) : whole + local / p.row_blocks;
  }
  w.split = group % p.nsplit;
  group /= p.nsplit;
  w.h = group % p.Hkv;
  w.b = group / p.Hkv;
  const int capacity = p.max_pages << p.page_shift;
  w.ctx = min(max(p.ctx_lens[w.b], 0), capacity);
  w.drafts = p.draft_lens ? min(max(p.draft_lens[w.b], 0), p.T) : p.T;
  const int last_row = min((w.rb + 1) * rows, p.R) - 1;
  const int seen = p.tree ? w.drafts : min(w.drafts, last_row / p.gamma + 1);
  w.end = uniform(w.drafts > 0 ? (int)min((int64_t)w.ctx + seen, (int64_t)capacity) : 0);
  // (contexts may end 16 tokens under 2^31: no sum of a position and a step is formed before it is known to be less)
  w.lo = uniform((int)min((int64_t)w.split * p.chunk, (int64_t)w.end));
  w.hi = uniform(w.split == p.nsplit - 1 ? w.end : min(w.end, w.lo + p.chunk));
  return w;
}

// A 16-token tile in memory; one past the end is replaced by the last (and masked).
struct Place {
  const uint8_t* at;   // the record
  uint32_t off;        // its first token in the page
  bool there;          // its page is one of the pool
};
__device__ inline int tile_at(const Span& w, int pos) { return min(pos, max(w.end - 1, 0)) & ~15; }
__device__ inline Place place_of(const AttnParams& p, const Span& w, uint32_t record, int tile, int pg) {
  Place r;
  r.there = pg >= 0 && pg < p.num_pages;
  r.at = p.cache + ((uint64_t)(r.there ? (uint32_t)pg : 0u) * (uint32_t)p.Hkv + (uint32_t)w.h) * record;
  r.off = (uint32_t)(tile & ((1 << p.page_shift) - 1));
  return r;
}

// A wave's rows: RT tiles of 16, row n = lane % 16 of each, as matrix operands.
template <class S, int RT>
struct Rows {
  half8_t q[S::PIECES][RT][S::NB];
  float cs[RT];           // scores are cs * (K q)
  int tok[RT];            // the row's token, or -1
  const uint32_t* bits[RT];
  // Scores are summed in units of cs, with queries of up to 2^14, 256 channels of them: a key of up to 2^127
  // would leave fp32 there although the score itself does not.  So key scales are taken over 2^kDown,
  // and cs makes up for it.  Scales under 2^(kDown - 126) then count as zero, which a query under 2^22
  // does not notice (2^-64 of a score); where every query of the wave is larger, scores are large before
  // sums are, and scales stay as they are.
  uint32_t down;          // what Scales::lower takes

  __device__ void load(const AttnParams& p, const Span& w, int row0, int lane) {
    const int n = lane & 15, g = lane >> 4;
    constexpr int D = S::NB * 32;
    float ups[RT];
    bool small = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = row0 + t * 16 + n, i = r / p.gamma;
      tok[t] = (r < p.R && i < w.drafts) ? i : -1;
      bits[t] = p.tree ? p.tree + (int64_t)w.b * p.tree_stride + (int64_t)max(tok[t], 0) * ((p.T + 31) / 32) : nullptr;
      float x[S::NB][8];
      float mx = 0.f;
      const int64_t at = ((int64_t)w.b * p.T + max(tok[t], 0)) * p.q_stride +
                         (int64_t)(w.h * p.gamma + (r - i * p.gamma)) * D + 8 * g;
#pragma unroll
      for (int B = 0; B < S::NB; ++B) {
        if constexpr (S::PIECES == 1) {
          const uint4 v = tok[t] >= 0 ? *(const uint4*)((const uint16_t*)p.q + at + 32 * B) : uint4{0, 0, 0, 0};
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[B][2 * j] = __uint_as_float(u[j] << 16);
            x[B][2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 v = tok[t] >= 0 ? *(const float4*)((const float*)p.q + at + 32 * B + 4 * j) : float4{0, 0, 0, 0};
            x[B][4 * j] = v.x; x[B][4 * j + 1] = v.y; x[B][4 * j + 2] = v.z; x[B][4 * j + 3] = v.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(x[B][j]));
      }
      mx = rows_max(mx);
      // scaled by a power of two to [2^13, 2^14): exponent field e of the maximum says
      // |x| < 2^(e - 126), and 2^(140 - e) takes it under 2^14
      int e = (int)(__float_as_uint(mx) >> 23) & 255;
      e = min(max(e, 14), 254);
      float up = __uint_as_float((uint32_t)min(140 - e + 127, 254) << 23);
      ups[t] = up;
      small |= mx > 0.f && e < 126 + 22;
      // the scale's sign goes into q, so that cs > 0 and masks can be -inf
      up = p.scale_log2e == 0.f ? 0.f : copysignf(up, p.scale_log2e);
      if (mx == INFINITY) up = __builtin_nanf("");   // or scores that are all -inf would pass for masked ones
#pragma unroll
      for (int B = 0; B < S::NB; ++B) {
        uint32_t u[4], z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = x[B][2 * k] * up, c = x[B][2 * k + 1] * up;
          u[k] = pk_f16(a, c);
          if constexpr (S::PIECES == 2) z[k] = pk_rest(a, c, u[k]);
        }
        q[0][t][B] = frag(u[0], u[1], u[2], u[3]);
        if constexpr (S::PIECES == 2) q[1][t][B] = frag(z[0], z[1], z[2], z[3]);
      }
    }
    const bool lowered = __any(small);
    down = lowered ? kDown * 0x00800080u : 0u;
    const float scale = fabsf(p.scale_log2e) * (lowered ? (float)(1 << kDown) : 1.f);
#pragma unroll
    for (int t = 0; t < RT; ++t)
      cs[t] = p.scale_log2e == 0.f ? 1.f : fminf(fmaxf(scale / ups[t], 0x1p-126f), 0x1.fffffep127f);
  }
};

// Running softmax and outputs of a wave's rows.
//
// A weight times a value scale has to fit fp16 and keep its bits there, so it is taken over a unit: a power
// of two for each row and channel group, set 2^3 under the largest such product that the row has met
// and grown only when one would pass 2^15.  It comes from what the row sees: a token that it does not see, or
// hardly weighs, costs it nothing, however large its values.
// Finding those products takes every weight, so steps are let through by bounds that cost less: scales of at
// most a unit (weights are at most 2^15), then the row's largest weight times the lane's largest scale.
// (Sums of weights over the least unit stay in fp32 up to 2^21 tokens, and products keep their bits
// down to value scales of 2^-118.)
constexpr float kMostProduct = 0x1p15f;
constexpr uint32_t kLeastUnit = (127u - 96u) << 23;     // 2^-96, as are units before any token
template <class S, int RT>
struct Sums {
  static constexpr int NJ = S::NB * 2;
  // One group: the exponential itself divides by the unit, which costs nothing.  Its argument grows by
  // the unit's octaves, so not for fp32, whose weights keep 22 bits.
  static constexpr bool FOLD = S::NG == 1 && S::PIECES == 1;
  float4_t acc[RT][NJ];   // [t][2 B + e][i]: channel 32 B + 2 (4 g + i) + e of row n, over its unit
  float m[RT], l[RT];     // running maximum (base 2, all lanes of a row agree), sum of this lane's weights
  float iu[RT][S::NG];    // one over the unit, in weights under the present m
  uint32_t room[S::NG];   // the smaller unit of the lane's rows, as bf16 in both halves
  float base[RT];         // weights are exp2(cs s + base)
  bool far;               // scores are rounded first (see weigh), by
  float far_cs[RT];       // this cs; cs is 1 then

  static __device__ float over(float pow2) { return __uint_as_float(0x7F000000u - __float_as_uint(pow2)); }

  __device__ void clear() {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[t][j] = float4_t{0, 0, 0, 0};
      m[t] = kFloor;
      l[t] = base[t] = 0.f;
#pragma unroll
      for (int G = 0; G < S::NG; ++G) iu[t][G] = over(__uint_as_float(kLeastUnit));
    }
#pragma unroll
    for (int G = 0; G < S::NG; ++G) room[G] = (kLeastUnit >> 16) * 0x10001u;
    far = false;
  }

  // log2 of what the weights of row tile t carry beside themselves.
  __device__ float carried(int t) const {
    return FOLD ? (float)((int)(__float_as_uint(iu[t][0]) >> 23) - 127) : 0.f;
  }
  template <int N>
  __device__ bool maxima(const float (&s)[RT][N], const float (&cs)[RT], float (&mx)[RT]) const {
    const float top = opaque_top();
    bool grow = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float x = larger(s[t][0], s[t][1], top);
#pragma unroll
      for (int i = 2; i < N; ++i) x = fmaxf(x, s[t][i]);
      mx[t] = rows_most(x, top) * cs[t];
      grow |= mx[t] > m[t] + kLag;
    }
    return grow;
  }

  // New maxima and units for a step: s[t] holds scores over cs, vs the value scales.
  template <int NT>
  __device__ void raise(float (&s)[RT][4 * NT], float (&cs)[RT], const Scales<S::NG> (&vs)[NT]) {
    float mx[RT];
    bool grow = maxima(s, cs, mx);
    // scales are not negative: their bf16 patterns compare as integers, two at a time
    ushort2_t top[S::NG];
    uint32_t past = 0u;
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      top[G] = us2(vs[0].w[G][0]);
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) top[G] = __builtin_elementwise_max(top[G], us2(vs[u].w[G][i]));
      past |= __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(top[G], us2(room[G])));
    }
    if (__builtin_expect(!__any(grow || past != 0u || far), 1)) return;
    if (far) {
      round_scores(s, far_cs);
      grow = maxima(s, cs, mx);
    }
    bool close = grow;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float w = __builtin_amdgcn_exp2f((mx[t] - (m[t] - kLift)) + carried(t));
#pragma unroll
      for (int G = 0; G < S::NG; ++G)
        close |= w * (FOLD ? 1.f : iu[t][G]) * __uint_as_float((uint32_t)max(top[G][0], top[G][1]) << 16) > kMostProduct;
    }
    if (__any(close)) refit(s, cs, vs, mx);
    if (far) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) s[t][i] -= m[t] - kLift;
    }
  }

  // Maxima and units from this step's scores, of which mx are the largest.
  template <int NT>
  __device__ void refit(float (&s)[RT][4 * NT], float (&cs)[RT], const Scales<S::NG> (&vs)[NT], const float (&mx)[RT]) {
    float f[RT];
    bool beyond = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      // whole octaves, so that nothing below rounds
      const float now = mx[t] > m[t] + kLag ? __builtin_ceilf(mx[t]) : m[t];
      f[t] = __builtin_amdgcn_ldexpf(1.f, (int)fmaxf(m[t] - now, -300.f));
      m[t] = now;
      if (!FOLD) l[t] *= f[t];
      beyond |= fabsf(now) > kFar && fabsf(now) < -kFloor;   // (an infinite query is its own row's affair)
    }
    if (!far && __any(beyond)) {
      far = true;
      round_scores(s, cs);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        far_cs[t] = cs[t];
        cs[t] = 1.f;
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float most[S::NG];                     // the largest products over 2^16, which would pass fp32 at 2^127
#pragma unroll
      for (int G = 0; G < S::NG; ++G) most[G] = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) {
        const float w = __builtin_amdgcn_exp2f(fmaf(s[t][i], cs[t], -m[t]) + (kLift - 16.f));
#pragma unroll
        for (int G = 0; G < S::NG; ++G) most[G] = fmaxf(most[G], w * vs[i / 4].get(G, i % 4));
      }
#pragma unroll
      for (int G = 0; G < S::NG; ++G) {
        const float x = rows_max(most[G]);
        const float old = over(iu[t][G]) * f[t];
        float unit = fmaxf(old, __uint_as_float(kLeastUnit));
        // (with the maximum the unit moves up as well, or the bounds above would stop every step from then on)
        if (x > unit * (f[t] < 1.f ? 0x1p-12f : kMostProduct * 0x1p-16f))
          unit = __uint_as_float(min((__float_as_uint(x) >> 23) + 13u, 253u) << 23);
        iu[t][G] = over(unit);
        const float turn = old * iu[t][G];
        if (FOLD) l[t] *= turn;
#pragma unroll
        for (int j = 2 * G * S::BPG; j < 2 * (G + 1) * S::BPG; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][j][i] *= turn;
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) base[t] = (far ? 0.f : kLift - m[t]) + carried(t);
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      float most = iu[0][G];
#pragma unroll
      for (int t = 1; t < RT; ++t) most = fmaxf(most, iu[t][G]);
      room[G] = (__float_as_uint(over(most)) >> 16) * 0x10001u;
    }
  }

  template <int N>
  static __device__ void round_scores(float (&s)[RT][N], const float (&cs)[RT]) {
#pragma clang fp contract(off)   // what is taken off them later stays a step of its own
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) s[t][i] *= cs[t];
  }

  // Scores become weights.  The maximum is a rounded score: up to kFar it is off by 2^-4 at most, and one
  // fused step takes it from exact products.  Past that the difference would keep the maximum's rounding,
  // which soon is more than its own distance to the row (and 2^32 is past any exponent).  So from the first
  // such maximum on the wave's products are rounded first, as the maximum was, and the maximum is
  // taken off them (raise): the row's largest weighs about 2^kLift whatever its size.
  template <int N>
  __device__ void weigh(float (&s)[RT][N], const float (&cs)[RT]) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], cs[t], base[t]));
        l[t] += s[t][i];
      }
  }

  // This wave's outputs o = acc / l and the base-2 logarithms of the sums.
  __device__ void finish(const int (&tok)[RT], float (&lse)[RT]) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float sum = rows_sum(l[t]);
      if (tok[t] < 0) sum = 0.f;     // a row past the drafted tokens saw what it should not have
      const float inv = is_zero(sum) ? 0.f : 1.f / sum;
      lse[t] = is_zero(sum) ? -INFINITY : (m[t] - kLift) + (__builtin_amdgcn_logf(sum) - carried(t));
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = acc[t][j][i] * inv * (FOLD ? 1.f : over(iu[t][j / (2 * S::BPG)]));
    }
  }

  // To memory: final rows, or this piece's part.
  __device__ void store(const AttnParams& p, const Span& w, int row0, int lane, const float (&lse)[RT]) const {
    constexpr int D = S::NB * 32;
    const int n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = row0 + t * 16 + n;
      if (r >= p.R) continue;
      const int i = r / p.gamma;
      if (p.nsplit > 1) {
        const int64_t at = ((int64_t)(w.split * p.B + w.b) * p.Hkv + w.h) * p.R + r;
        if (g == 0) p.part_lse[at] = lse[t];
        if (is_empty(lse[t])) continue;
        float* o = p.part_o + at * D + 8 * g;
#pragma unroll
        for (int B = 0; B < S::NB; ++B) {
          const float4_t a = acc[t][2 * B], c = acc[t][2 * B + 1];
          *(float4*)(o + 32 * B) = float4{a[0], c[0], a[1], c[1]};
          *(float4*)(o + 32 * B + 4) = float4{a[2], c[2], a[3], c[3]};
        }
      } else {
        const int64_t at = ((int64_t)w.b * p.T + i) * p.Hq + w.h * p.gamma + (r - i * p.gamma);
        if (g == 0 && p.lse) p.lse[at] = lse[t] * 0.69314718055994530942f;
#pragma unroll
        for (int B = 0; B < S::NB; ++B) {
          const float4_t a = acc[t][2 * B], c = acc[t][2 * B + 1];
          if constexpr (S::PIECES == 1) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __bf16 x = (__bf16)a[k], y = (__bf16)c[k];
              u[k] = (uint32_t)__builtin_bit_cast(uint16_t, x) | (uint32_t)__builtin_bit_cast(uint16_t, y) << 16;
            }
            *(uint4*)((uint16_t*)p.o + at * D + 32 * B + 8 * g) = uint4{u[0], u[1], u[2], u[3]};
          } else {
            float* o = (float*)p.o + at * D + 32 * B + 8 * g;
            *(float4*)o = float4{a[0], c[0], a[1], c[1]};
            *(float4*)(o + 4) = float4{a[2], c[2], a[3], c[3]};
          }
        }
      }
    }
  }
};

// -inf where row n of tile t may not see token pos = p0 + i (i < 4); held: the lane's tokens that
// are there at all.
template <class S, int RT, int N>
__device__ inline void mask_scores(float (&s)[RT][N], int at, const AttnParams& p, const Span& w, const Rows<S, RT>& rows,
                                   int p0, bool there) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = p0 + i, j = pos - w.ctx;
    const bool held = there && pos < w.end;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      bool ok = held && rows.tok[t] >= 0;
      if (ok && j >= 0) ok = p.tree ? (rows.bits[t][j >> 5] >> (j & 31)) & 1u : j <= rows.tok[t];
      s[t][at + i] = ok ? s[t][at + i] : -INFINITY;
    }
  }
}

// Bytes of the lane's quad from p0 on that belong to tokens that are there.
__device__ inline uint32_t held_bytes(const Span& w, int p0, bool there) {
  const int n = there ? min(max(w.end - p0, 0), 4) : 0;
  return n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
}

// Old bytes may be NaN scales, or NaN codes of fp8, and 0 times NaN is NaN: values and their scales
// of tokens that are not there become zero.
template <int KIND, int LB, int NG>
__device__ inline void drop_old(Raw<LB>& v, Scales<NG>& s, uint32_t keep) {
  const uint32_t k01 = __builtin_amdgcn_perm(keep, keep, 0x01010000u), k23 = __builtin_amdgcn_perm(keep, keep, 0x03030202u);
#pragma unroll
  for (int G = 0; G < NG; ++G) {
    s.w[G][0] &= k01;
    s.w[G][1] &= k23;
  }
  if constexpr (KIND == PACE_CACHE_FP8) {
#pragma unroll
    for (int x = 0; x < LB / 4; ++x) v.w[x] &= keep;
  }
}

// The weights of two tiles (scores at, at + 4) times their value scales in the rows' units, as matrix
// operands.  (iu first: a token that the row does not see has a weight of 0 and any scale.)
template <class S, int KIND, int RT, int N>
__device__ inline void weight_operands(const float (&s)[RT][N], int at, const float4_t (&sc)[2], const float (&iu)[RT],
                                       half8_t (&pf)[S::PIECES][RT]) {
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    uint32_t w[4], z[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = s[t][at + 4 * u + i] * iu[t] * sc[u][i];
      // the token order in which the value codes unpack
      constexpr int o1 = KIND == PACE_CACHE_INT4 ? 2 : 1, o2 = 3 - o1;
      w[2 * u] = pk_f16(x[0], x[o1]);
      w[2 * u + 1] = pk_f16(x[o2], x[3]);
      if constexpr (S::PIECES == 2) {
        z[2 * u] = pk_rest(x[0], x[o1], w[2 * u]);
        z[2 * u + 1] = pk_rest(x[o2], x[3], w[2 * u + 1]);
      }
    }
    pf[0][t] = frag(w[0], w[1], w[2], w[3]);
    if constexpr (S::PIECES == 2) pf[1][t] = frag(z[0], z[1], z[2], z[3]);
  }
}

// ------------------------------------------------------------------------------------ kernel

// Waves a SIMD that the registers have to allow: two for two row tiles with d = 128, where the compiler would stop a
// few registers short of them.  Those few then are in memory before and after the loop, not in it (a 512-token
// chunk, int8, g = 32: 318 us, with one wave 444).  Where they would reach into the loop, one wave it is.
template <int KIND, int D, int GROUP, bool BF16, int RT>
constexpr int least_waves() {
  return D == 128 && RT == 2 && !(GROUP == 32 && (!BF16 || KIND == PACE_CACHE_INT4)) ? 2 : 1;
}

template <int KIND, int D, int GROUP, bool BF16, int RT, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(least_waves<KIND, D, GROUP, BF16, RT>()))) void attn_kernel(AttnParams p) {
  using S = Shape<KIND, D, GROUP, BF16>;
  using C = Codes<KIND>;
  constexpr int NT = kTiles, STEP = 16 * NT;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  const Span w = span_of(p, RT * 16);
  const int row0 = w.rb * (RT * 16);
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, S::BITS);

  Raw<S::LB> kr[NT], vr[NT];
  Scales<S::NG> ks[NT], vs[NT];
  const int32_t* table = p.table + (int64_t)w.b * p.max_pages;
  struct Where {
    Place t[NT];
  };
  auto where = [&](int s0) {
    Where x;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int tile = tile_at(w, s0 + 16 * u);
      x.t[u] = place_of(p, w, rec.total, tile, uniform(table[tile >> p.page_shift]));
    }
    return x;
  };
  // use == 0 (no further step): every lane asks for the tile's first bytes, one cache line
  auto load_keys = [&](const Where& x, int use) {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      kr[u] = load_raw<S::LB, 64>(x.t[u].at + x.t[u].off * (D * S::BITS / 8), lane & use);
      ks[u] = load_scales<S::NG>(x.t[u].at + rec.codes + (x.t[u].off / 4 + (g & use)) * (S::NG * 8));
    }
  };
  auto load_values = [&](const Where& x, int use) {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const uint8_t* v = x.t[u].at + rec.codes + rec.scales;
      vr[u] = load_raw<S::LB, 16>(v + (x.t[u].off / 4 + (g & use)) * (D * S::BITS / 2), n & use);
      vs[u] = load_scales<S::NG>(v + rec.codes + (x.t[u].off / 4 + (g & use)) * (S::NG * 8));
    }
  };
  constexpr int stride = NW * STEP;
  const bool any = w.hi - w.lo > wave * STEP;
  const int first = any ? w.lo + wave * STEP : 0;
  Where cur;
  if (any) {
    cur = where(first);
    load_keys(cur, -1);
    load_values(cur, -1);
  }
  Rows<S, RT> rows;
  rows.load(p, w, row0, lane);
  Sums<S, RT> sums;
  sums.clear();
  uint32_t magic = 0x64006400u;
  asm("" : "+v"(magic));

  bool more = any;
  for (int s0 = first; more; s0 += stride) {
    more = w.hi - s0 > stride;
    const int use = more ? -1 : 0;
    const Where next = where(more ? s0 + stride : s0);

    // ---- scores over cs: s[t][4 u + i] of token s0 + 16 u + 4 g + i
    float s[RT][4 * NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      ks[u].lower(rows.down);
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
            for (int c = 0; c < S::PIECES; ++c) a[t] = mfma(kf, rows.q[c][t][B], a[t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float k = ks[u].get(G, i);
#pragma unroll
          for (int t = 0; t < RT; ++t) s[t][4 * u + i] = G == 0 ? a[t][i] * k : fmaf(a[t][i], k, s[t][4 * u + i]);
        }
      }
    }
    load_keys(next, use);

    bool there = true;
#pragma unroll
    for (int u = 0; u < NT; ++u) there = there && cur.t[u].there;
    if (w.ctx - s0 < STEP || !there) {
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const int p0 = s0 + 16 * u + 4 * g;
        mask_scores<S>(s, 4 * u, p, w, rows, p0, cur.t[u].there);
        drop_old<KIND>(vr[u], vs[u], held_bytes(w, p0, cur.t[u].there));
      }
    }

    sums.raise(s, rows.cs, vs);
    sums.weigh(s, rows.cs);

    // ---- O^T += V^T P^T
#pragma unroll
    for (int pr = 0; pr < NT / 2; ++pr)
#pragma unroll
      for (int G = 0; G < S::NG; ++G) {
        float4_t sc[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[u][i] = vs[2 * pr + u].get(G, i);
        float iu[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) iu[t] = sums.FOLD ? 1.f : sums.iu[t][G];
        half8_t pf[S::PIECES][RT];
        weight_operands<S, KIND>(s, 8 * pr, sc, iu, pf);
#pragma unroll
        for (int jb = 0; jb < S::BPG; ++jb) {
          const int B = G * S::BPG + jb;
          half8_t vf[2];
          C::values(vr[2 * pr].w, vr[2 * pr + 1].w, B, magic, vf);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
              for (int c = 0; c < S::PIECES; ++c) sums.acc[t][2 * B + e] = mfma(vf[e], pf[c][t], sums.acc[t][2 * B + e]);
        }
      }
    load_values(next, use);
    cur = next;
  }

  float lse[RT];
  sums.finish(rows.tok, lse);

  // ---- joined over the waves
  constexpr int REGS = D / 4;   // accumulator registers of a tile
  constexpr int SLOT = RT * (REGS + 1) * 64;
  if (wave > 0) {
    float* mine = lds + (size_t)(wave - 1) * SLOT;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(t * (REGS + 1) + 4 * j + i) * 64 + lane] = sums.acc[t][j][i];
      mine[(t * (REGS + 1) + REGS) * 64 + lane] = lse[t];
    }
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    float top = lse[t];
    for (int k = 1; k < NW; ++k) top = fmaxf(top, lds[(size_t)(k - 1) * SLOT + (t * (REGS + 1) + REGS) * 64 + lane]);
    const float base = is_empty(top) ? 0.f : top;
    float sum = __builtin_amdgcn_exp2f(lse[t] - base);
    for (int k = 1; k < NW; ++k) sum += __builtin_amdgcn_exp2f(lds[(size_t)(k - 1) * SLOT + (t * (REGS + 1) + REGS) * 64 + lane] - base);
    // shares that add up to 1: outputs of up to 2^127 stay finite
    const float inv = is_zero(sum) ? 0.f : 1.f / sum;
    float f = __builtin_amdgcn_exp2f(lse[t] - base) * inv;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums.acc[t][j][i] *= f;
    for (int k = 1; k < NW; ++k) {
      const float* from = lds + (size_t)(k - 1) * SLOT + t * (REGS + 1) * 64 + lane;
      f = __builtin_amdgcn_exp2f(from[REGS * 64] - base) * inv;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums.acc[t][j][i] = fmaf(from[(4 * j + i) * 64], f, sums.acc[t][j][i]);
    }
    lse[t] = is_zero(sum) ? -INFINITY : base + __builtin_amdgcn_logf(sum);
  }
  sums.store(p, w, row0, lane, lse);
}

// ------------------------------------------------------------------------------------ launch

template <int KIND, int D, int GROUP, bool BF16, int RT, int NW>
hipError_t launch_shape(const AttnParams& p, uint32_t grid, hipStream_t s) {
  const size_t lds = (size_t)(NW - 1) * RT * (D / 4 + 1) * 64 * sizeof(float);
  attn_kernel<KIND, D, GROUP, BF16, RT, NW><<<grid, NW * 64, lds, s>>>(p);
  return hipGetLastError();
}

template <int KIND, int D, int GROUP, bool BF16>
hipError_t launch_by_plan(const AttnParams& p, const AttnPlan& a, hipStream_t s) {
  const uint32_t grid = (uint32_t)((int64_t)p.nsplit * p.row_blocks * p.Hkv * p.B);
  if constexpr (D <= 128) {
    if (a.row_tiles == 2) return launch_shape<KIND, D, GROUP, BF16, 2, 4>(p, grid, s);
    if (a.waves == 8) return launch_shape<KIND, D, GROUP, BF16, 1, 8>(p, grid, s);
  }
  return launch_shape<KIND, D, GROUP, BF16, 1, 4>(p, grid, s);
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
