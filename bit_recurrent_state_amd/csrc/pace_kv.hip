// The quantised paged key/value cache: writing and reading back (include/pace_cache.h:
// pace_cache_write, pace_cache_read; layout and quantiser there).
//
// A wave takes 16 consecutive tokens of one head, keys or values (two rows of the grid), in the lanes
// that hold them in the cache, so that codes move as 16 bytes a lane, contiguous over the wave:
//   keys: lane 16 a + r holds the 8-channel units a, a + 4, .. of token r, all LB bytes of them;
//   values: lane 16 g + m holds channels 32 B + 2 m + {0, 1} of the four tokens of quad g.
// A group's maximum is found across the four lanes of a token (keys) or the 16 of a quad
// (values).  Runs of consecutive positions are cut at multiples of 16 positions, from any start;
// a quad that is not whole (single tokens, edges, holes) moves its values byte by byte.
// Inputs are read once, codes and scales written once.  Writing 4 x 4093 tokens, 8 heads of 128, int4, g =
// 32: 23 us, 3.7 TB/s; 15 vector operations a value keep that unit 67% busy and waves wait
// 39% of their time.  Reading them back: 17.6 us, 4.9 TB/s.  Reading 4 x 16384 tokens of int8: 95 us, 4.3
// TB/s; values leave in 4-byte stores, four rows of them a wave.  A token's write takes 3.8 us.
#include <hip/hip_runtime.h>

#include <utility>

#include "pace_cache_internal.h"
#include "pace_lanes.h"
#include "pace_numerics.h"

namespace pace {
namespace {

constexpr int kThreads = 256;

// N channels next to each other, as one load or store.
template <typename E, int N>
struct alignas(sizeof(E) * N < 16 ? sizeof(E) * N : 16) Run {
  E v[N];
};

__device__ inline float widen(float x) { return x; }
__device__ inline float widen(uint16_t x) { return bf16_to_f32(x); }
template <typename E>
__device__ inline E narrow(float x) {
  if constexpr (sizeof(E) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)x);
  else
    return x;
}

template <int KIND, int D, int GROUP>
struct Shape {
  static constexpr int BITS = KIND == PACE_CACHE_INT4 ? 4 : 8;
  static constexpr int LB = D * BITS / 32;          // bytes a lane holds
  static constexpr int W = LB < 16 ? LB : 16;       // in pieces of
  static constexpr int NB = D / 32, NG = D / GROUP, BPG = GROUP / 32;
  static __device__ uint32_t key_at(int r, int a, int i) {
    return (uint32_t)(r >> 4) * (64 * LB) + i * (64 * W) + (16 * a + (r & 15)) * W;
  }
  static __device__ uint32_t value_at(int r, int m, int i) {
    return (uint32_t)(r >> 2) * (16 * LB) + i * (16 * W) + m * W;
  }
  static __device__ uint32_t scale_at(int r, int G) { return 2u * (((uint32_t)(r >> 2) * NG + G) * 4 + (r & 3)); }
};

template <int KIND>
__host__ __device__ constexpr float levels() {
  return KIND == PACE_CACHE_INT8 ? 127.f : KIND == PACE_CACHE_INT4 ? 7.f : 448.f;
}

// Finite stand-in of an input (the cache holds finite values only).
__device__ inline float tame(float x) {
  const bool nan = (f32_bits(x) & 0x7FFFFFFFu) > 0x7F800000u;
  return nan ? 0.f : fminf(fmaxf(x, -0x1p127f), 0x1p127f);
}
constexpr uint32_t kTame = 0x7F000000u;   // the bits of 2^127: larger magnitudes need it

// Magnitudes compare as their bit patterns, which orders NaN last: one operation a value.
__device__ inline uint32_t magnitude(const Run<float, 2>& x) {
  return max(f32_bits(x.v[0]) & 0x7FFFFFFFu, f32_bits(x.v[1]) & 0x7FFFFFFFu);
}
__device__ inline uint32_t magnitude(const Run<float, 8>& x) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, f32_bits(x.v[i]) & 0x7FFFFFFFu);
  return m;
}
typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));
__device__ inline ushort2_t magnitudes(uint32_t x) { return __builtin_bit_cast(ushort2_t, x & 0x7FFF7FFFu); }
__device__ inline uint32_t magnitude(const Run<uint16_t, 2>& x) {
  const ushort2_t m = magnitudes(__builtin_bit_cast(uint32_t, x));
  return (uint32_t)max(m[0], m[1]) << 16;
}
__device__ inline uint32_t magnitude(const Run<uint16_t, 8>& x) {
  const uint4 w = __builtin_bit_cast(uint4, x);
  const ushort2_t m = __builtin_elementwise_max(__builtin_elementwise_max(magnitudes(w.x), magnitudes(w.y)),
                                                __builtin_elementwise_max(magnitudes(w.z), magnitudes(w.w)));
  return (uint32_t)max(m[0], m[1]) << 16;
}

// Scale and reciprocal of a group from its largest magnitude.
template <int KIND>
__device__ inline void scale_of(float m, float& s, float& r) {
  constexpr float L = levels<KIND>();
  s = bf16_ceil_div(m, L, 1.0f / L);
  if (s < 0x1p-126f) s = 0.f;
  r = s > 0.f ? rcp_bf16(s) : 0.f;
}

// x / s, correctly rounded (r is the correctly rounded reciprocal, the residual exact; for scales under
// 2^-108 the residual ends below the subnormal numbers and the quotient may be a unit off).  At most
// L in magnitude, since s >= max|x| / L.
__device__ inline float quotient(float x, float s, float r) {
  const float a = x * r, e = fmaf(-a, s, x);
  return fmaf(e, r, a);
}

// The stored field of an int quotient above kField: adding 1.5 2^23 + offset rounds to the nearest
// integer, ties to even (the offset is even), and leaves it in the low mantissa bits.
constexpr uint32_t kField = 0x4B400000u;
template <int KIND>
__device__ inline uint32_t int_field(float x, float s, float r) {
  return f32_bits(quotient(x, s, r) + (12582912.0f + (KIND == PACE_CACHE_INT8 ? 128.f : 8.f)));
}
// Two e4m3 bytes.  The quotient's correction turns -0 into +0: e4m3 keeps the quotient's sign.
__device__ inline uint32_t fp8_pair(float x, float y, float s, float r) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(copysignf(quotient(x, s, r), x), copysignf(quotient(y, s, r), y), 0, false);
}
// Four bytes from the low bytes of four fields.
__device__ inline uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}

template <int KIND>
__device__ inline float value_of(uint32_t f) {
  if constexpr (KIND == PACE_CACHE_FP8)
    return __builtin_amdgcn_cvt_f32_fp8((int)f, 0);
  else
    return (float)((int)f - (KIND == PACE_CACHE_INT8 ? 128 : 8));
}

// Lane exchanges inside a row of 16.
template <int CTRL>
__device__ inline uint32_t row_move(uint32_t x) { return __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, true); }
constexpr int kMirror = 0x140, kHalfMirror = 0x141, kSwap2 = 0x4E, kSwap1 = 0xB1, kFromLane = 0x150;

// One step of a reduce-scatter of N maxima over a row: lanes whose `upper` is set keep the upper half
// of the array, their partners (CTRL) the lower; a single value is combined.
template <int N, int CTRL>
__device__ inline void scatter_step(uint32_t* v, bool upper) {
  if constexpr (N == 1) {
    v[0] = max(v[0], row_move<CTRL>(v[0]));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t keep = upper ? v[i + N / 2] : v[i], give = upper ? v[i] : v[i + N / 2];
      v[i] = max(keep, row_move<CTRL>(give));
    }
  }
}
// f(0), f(1), .. with compile-time indexes (lane numbers have to be).
template <int... K, typename F>
__device__ inline void for_each(std::integer_sequence<int, K...>, F f) {
  (f(std::integral_constant<int, K>{}), ...);
}
constexpr int half_of(int n) { return n > 1 ? n / 2 : 1; }
// Maxima of N values over the 16 lanes of a row.  Lane m ends with value(s) m N / 16, or
// m div (16 / N) where N < 16.
template <int N>
__device__ inline void scatter_max(uint32_t* v, int m) {
  scatter_step<N, kMirror>(v, m & 8);
  scatter_step<half_of(N), kHalfMirror>(v, m & 4);
  scatter_step<half_of(half_of(N)), kSwap2>(v, m & 2);
  scatter_step<half_of(half_of(half_of(N))), kSwap1>(v, m & 1);
}

// What a wave works on: sequence, head, and the token index of its first position.
struct Item {
  int b, h, t0;   // t0 may be negative
  bool in;
};
__device__ inline Item item_of(const CacheIoParams& p, int ntile) {
  const int64_t id = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (kThreads / 64) + threadIdx.x / 64));
  Item w;
  w.h = (int)(id % p.Hkv);
  const int64_t bt = id / p.Hkv;
  w.b = (int)(bt / ntile);
  w.in = w.b < p.B;
  if (!w.in) w.b = 0;
  // (fewer than 16 tokens fill no tile: no use in waiting for the first position)
  const int first = p.T >= 16 ? p.positions[(int64_t)w.b * p.T] : 0;
  w.t0 = (int)(bt % ntile) * 16 - (first >= 0 ? (first & 15) : 0);
  return w;
}

// Record of token t's position, or null where it is skipped; r: its place in the page.
__device__ inline uint8_t* record_of(const CacheIoParams& p, const Item& w, int t, uint32_t rec, int& pos, int& r) {
  pos = -1;
  r = 0;
  if (!w.in || t < 0 || t >= p.T) return nullptr;
  pos = p.positions[(int64_t)w.b * p.T + t];
  const int entry = pos >> p.page_shift;
  if (pos < 0 || entry >= p.max_pages) return nullptr;
  const int page = p.table[(int64_t)w.b * p.max_pages + entry];
  if (page < 0 || page >= p.num_pages) return nullptr;
  r = pos & ((1 << p.page_shift) - 1);
  return p.cache + ((int64_t)page * p.Hkv + w.h) * rec;
}

// The positions of a quad of values: whole if they are the four of one stored quad.
struct Quad {
  uint8_t* at[4];
  int r[4];
  bool whole;
  __device__ void find(const CacheIoParams& p, const Item& w, int t, uint32_t rec) {
    int pos[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = record_of(p, w, t + j, rec, pos[j], r[j]);
    whole = at[0] && at[1] && at[2] && at[3] && (pos[0] & 3) == 0 && pos[1] == pos[0] + 1 && pos[2] == pos[0] + 2 &&
            pos[3] == pos[0] + 3;
  }
};

template <int W>
__device__ inline void store_piece(uint8_t* to, const uint32_t* w) {
  if constexpr (W == 16)
    *(uint4*)to = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *(uint2*)to = make_uint2(w[0], w[1]);
}
template <int W>
__device__ inline void load_piece(const uint8_t* from, uint32_t* w) {
  if constexpr (W == 16) {
    const uint4 v = *(const uint4*)from;
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *(const uint2*)from;
    w[0] = v.x; w[1] = v.y;
  }
}

template <int KIND, int D, int GROUP, typename E>
__device__ inline void write_keys(const CacheIoParams& p, const Item& w, int lane) {
  using S = Shape<KIND, D, GROUP>;
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, S::BITS);
  const int a = lane >> 4, t = w.t0 + (lane & 15);
  const bool in = w.in && t >= 0 && t < p.T;
  Run<E, 8> raw[S::NB];
  const E* from = (const E*)p.k_in + ((int64_t)w.b * p.T + (in ? t : 0)) * p.k_stride + w.h * D + 8 * a;
#pragma unroll
  for (int B = 0; B < S::NB; ++B) raw[B] = *(const Run<E, 8>*)(from + 32 * B);
  int pos, r;
  uint8_t* const at = record_of(p, w, t, rec.total, pos, r);
  float x[S::NB][8];
#pragma unroll
  for (int B = 0; B < S::NB; ++B)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[B][i] = widen(raw[B].v[i]);
  uint32_t top[S::NG], most = 0u;
#pragma unroll
  for (int G = 0; G < S::NG; ++G) {
    top[G] = 0u;
#pragma unroll
    for (int j = 0; j < S::BPG; ++j) top[G] = max(top[G], magnitude(raw[G * S::BPG + j]));
    most = max(most, top[G]);
  }
  if (__any(most > kTame)) {
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      top[G] = 0u;
#pragma unroll
      for (int j = 0; j < S::BPG; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& y = x[G * S::BPG + j][i];
          y = tame(y);
          top[G] = max(top[G], f32_bits(y) & 0x7FFFFFFFu);
        }
    }
  }
  uint32_t word[S::LB / 4];
  float s[S::NG];
#pragma unroll
  for (int G = 0; G < S::NG; ++G) {
    LanePair pr = pair16(top[G]);
    pr = pair32(max(pr.lo, pr.hi));
    float inv;
    scale_of<KIND>(bits_f32(max(pr.lo, pr.hi)), s[G], inv);
#pragma unroll
    for (int j = 0; j < S::BPG; ++j) {
      const int B = G * S::BPG + j;
      if constexpr (KIND == PACE_CACHE_FP8) {
        const uint32_t live = s[G] > 0.f ? 0xFFFFFFFFu : 0u;   // a zero group is +0
#pragma unroll
        for (int k = 0; k < 2; ++k)
          word[2 * B + k] = live & ((fp8_pair(x[B][4 * k], x[B][4 * k + 1], s[G], inv) & 0xFFFFu) |
                                    fp8_pair(x[B][4 * k + 2], x[B][4 * k + 3], s[G], inv) << 16);
      } else {
        uint32_t f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = int_field<KIND>(x[B][i], s[G], inv);
        if constexpr (KIND == PACE_CACHE_INT4) {
          // channel e in nibble e / 2 + 4 (e mod 2); kField's own bits, shifted and summed, come off
          uint32_t w = f[0] - (kField + (kField << 4) + (kField << 8));
          w += (f[2] << 4) + (f[4] << 8) + (f[6] << 12);
          word[B] = w + (f[1] << 16) + (f[3] << 20) + (f[5] << 24) + (f[7] << 28);
        } else {
          word[2 * B] = four_bytes(f[0], f[1], f[2], f[3]);
          word[2 * B + 1] = four_bytes(f[4], f[5], f[6], f[7]);
        }
      }
    }
  }
  if (!at) return;
#pragma unroll
  for (int i = 0; i < S::LB / S::W; ++i) store_piece<S::W>(at + S::key_at(r, a, i), word + i * (S::W / 4));
  if (a == 0) {
#pragma unroll
    for (int G = 0; G < S::NG; ++G)
      *(uint16_t*)(at + rec.codes + S::scale_at(r, G)) = (uint16_t)(f32_bits(s[G]) >> 16);
  }
}

template <int KIND, int D, int GROUP, typename E>
__device__ inline void write_values(const CacheIoParams& p, const Item& w, int lane) {
  using S = Shape<KIND, D, GROUP>;
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, S::BITS);
  const int m = lane & 15, t = w.t0 + 4 * (lane >> 4);
  Run<E, 2> raw[4][S::NB];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = w.in && t + j >= 0 && t + j < p.T;
    const E* from = (const E*)p.v_in + ((int64_t)w.b * p.T + (in ? t + j : 0)) * p.v_stride + w.h * D + 2 * m;
#pragma unroll
    for (int B = 0; B < S::NB; ++B) raw[j][B] = *(const Run<E, 2>*)(from + 32 * B);
  }
  Quad q;
  q.find(p, w, t, rec.total);
  // ---- the groups' maxima, j NG + G; each found by the lanes of the row together, its scale by
  // the lane (or lanes) that end with it, from which every lane reads scale and reciprocal
  constexpr int N = 4 * S::NG;
  float x[4][S::NB][2];
  uint32_t top[N], most = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      uint32_t& v = top[j * S::NG + G];
      v = 0u;
#pragma unroll
      for (int k = 0; k < S::BPG; ++k) {
        const int B = G * S::BPG + k;
        x[j][B][0] = widen(raw[j][B].v[0]);
        x[j][B][1] = widen(raw[j][B].v[1]);
        v = max(v, magnitude(raw[j][B]));
      }
      most = max(most, v);
    }
  if (__any(most > kTame)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int G = 0; G < S::NG; ++G) {
        uint32_t& v = top[j * S::NG + G];
        v = 0u;
#pragma unroll
        for (int k = 0; k < S::BPG; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& y = x[j][G * S::BPG + k][e];
            y = tame(y);
            v = max(v, f32_bits(y) & 0x7FFFFFFFu);
          }
      }
  }
  scatter_max<N>(top, m);
  constexpr int PER = N > 16 ? N / 16 : 1;   // values a lane ends with
  float sc[PER], inv[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) scale_of<KIND>(bits_f32(top[i]), sc[i], inv[i]);

  // word 2 B + e (8 bits) or B (4 bits): one byte a token
  uint32_t f[4][S::NB][2];
  uint16_t s[4][S::NG];
  for_each(std::make_integer_sequence<int, N>{}, [&](auto index) {   // group K = j NG + G
    constexpr int K = decltype(index)::value;
    constexpr int j = K / S::NG, G = K % S::NG, from = N >= 16 ? K * 16 / N : K * (16 / N), at = N > 16 ? K % PER : 0;
    const float a = bits_f32(row_move<kFromLane + from>(f32_bits(sc[at]))), r = bits_f32(row_move<kFromLane + from>(f32_bits(inv[at])));
    s[j][G] = (uint16_t)(f32_bits(a) >> 16);
#pragma unroll
    for (int k = 0; k < S::BPG; ++k) {
      const int B = G * S::BPG + k;
      if constexpr (KIND == PACE_CACHE_FP8) {
        const uint32_t w = a > 0.f ? fp8_pair(x[j][B][0], x[j][B][1], a, r) : 0u;   // a zero group is +0
        f[j][B][0] = w;
        f[j][B][1] = w >> 8;
      } else {
        f[j][B][0] = int_field<KIND>(x[j][B][0], a, r);
        f[j][B][1] = int_field<KIND>(x[j][B][1], a, r);
      }
    }
  });
  uint32_t word[S::LB / 4];
#pragma unroll
  for (int B = 0; B < S::NB; ++B) {
    if constexpr (KIND == PACE_CACHE_INT4) {
      uint32_t y[4];                         // both nibbles in the low byte
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = f[j][B][0] + (f[j][B][1] << 4);
      word[B] = four_bytes(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) word[2 * B + e] = four_bytes(f[0][B][e], f[1][B][e], f[2][B][e], f[3][B][e]);
    }
  }
  const uint32_t codes_at = rec.codes + rec.scales, scales_at = codes_at + rec.codes;
  if (q.whole) {
#pragma unroll
    for (int i = 0; i < S::LB / S::W; ++i) store_piece<S::W>(q.at[0] + codes_at + S::value_at(q.r[0], m, i), word + i * (S::W / 4));
#pragma unroll
    for (int G = 0; G < S::NG; ++G)
      if (m == G)
        *(uint2*)(q.at[0] + scales_at + S::scale_at(q.r[0], G)) =
            make_uint2(s[0][G] | (uint32_t)s[1][G] << 16, s[2][G] | (uint32_t)s[3][G] << 16);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!q.at[j]) continue;
#pragma unroll
    for (int i = 0; i < S::LB / 4; ++i)
      q.at[j][codes_at + S::value_at(q.r[j], m, 4 * i / S::W) + 4 * i % S::W + (q.r[j] & 3)] = (uint8_t)(word[i] >> (8 * j));
#pragma unroll
    for (int G = 0; G < S::NG; ++G)
      if (m == G) *(uint16_t*)(q.at[j] + scales_at + S::scale_at(q.r[j], G)) = s[j][G];
  }
}

template <int KIND, int D, int GROUP, typename E>
__device__ inline void read_keys(const CacheIoParams& p, const Item& w, int lane) {
  using S = Shape<KIND, D, GROUP>;
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, S::BITS);
  const int a = lane >> 4, t = w.t0 + (lane & 15);
  int pos, r;
  const uint8_t* const at = record_of(p, w, t, rec.total, pos, r);
  uint32_t word[S::LB / 4];
  float s[S::NG];
#pragma unroll
  for (int i = 0; i < S::LB / 4; ++i) word[i] = 0u;
#pragma unroll
  for (int G = 0; G < S::NG; ++G) s[G] = 0.f;
  if (at) {
#pragma unroll
    for (int i = 0; i < S::LB / S::W; ++i) load_piece<S::W>(at + S::key_at(r, a, i), word + i * (S::W / 4));
#pragma unroll
    for (int G = 0; G < S::NG; ++G) s[G] = bf16_to_f32(*(const uint16_t*)(at + rec.codes + S::scale_at(r, G)));
  }
  if (!w.in || t < 0 || t >= p.T) return;
  E* to = (E*)p.k_out + ((int64_t)w.b * p.T + t) * p.k_stride + w.h * D + 8 * a;
#pragma unroll
  for (int B = 0; B < S::NB; ++B) {
    Run<E, 8> y;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t f = KIND == PACE_CACHE_INT4 ? (word[B] >> (4 * (i / 2 + 4 * (i & 1)))) & 15u
                                                 : (word[2 * B + i / 4] >> (8 * (i & 3))) & 255u;
      y.v[i] = at ? narrow<E>(value_of<KIND>(f) * s[B / S::BPG]) : narrow<E>(0.f);
    }
    *(Run<E, 8>*)(to + 32 * B) = y;
  }
}

template <int KIND, int D, int GROUP, typename E>
__device__ inline void read_values(const CacheIoParams& p, const Item& w, int lane) {
  using S = Shape<KIND, D, GROUP>;
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, S::BITS);
  const int m = lane & 15, t = w.t0 + 4 * (lane >> 4);
  Quad q;
  q.find(p, w, t, rec.total);
  const uint32_t codes_at = rec.codes + rec.scales, scales_at = codes_at + rec.codes;
  uint32_t word[S::LB / 4];
  float s[4][S::NG];
#pragma unroll
  for (int i = 0; i < S::LB / 4; ++i) word[i] = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int G = 0; G < S::NG; ++G) s[j][G] = 0.f;
  if (q.whole) {
#pragma unroll
    for (int i = 0; i < S::LB / S::W; ++i) load_piece<S::W>(q.at[0] + codes_at + S::value_at(q.r[0], m, i), word + i * (S::W / 4));
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      const uint2 v = *(const uint2*)(q.at[0] + scales_at + S::scale_at(q.r[0], G));
      s[0][G] = bits_f32(v.x << 16);
      s[1][G] = bits_f32(v.x & 0xFFFF0000u);
      s[2][G] = bits_f32(v.y << 16);
      s[3][G] = bits_f32(v.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!q.at[j]) continue;
#pragma unroll
      for (int i = 0; i < S::LB / 4; ++i)
        word[i] |= (uint32_t)q.at[j][codes_at + S::value_at(q.r[j], m, 4 * i / S::W) + 4 * i % S::W + (q.r[j] & 3)] << (8 * j);
#pragma unroll
      for (int G = 0; G < S::NG; ++G) s[j][G] = bf16_to_f32(*(const uint16_t*)(q.at[j] + scales_at + S::scale_at(q.r[j], G)));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!w.in || t + j < 0 || t + j >= p.T) continue;
    E* to = (E*)p.v_out + ((int64_t)w.b * p.T + t + j) * p.v_stride + w.h * D + 2 * m;
#pragma unroll
    for (int B = 0; B < S::NB; ++B) {
      Run<E, 2> y;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t f = KIND == PACE_CACHE_INT4 ? (word[B] >> (8 * j + 4 * e)) & 15u : (word[2 * B + e] >> (8 * j)) & 255u;
        y.v[e] = q.at[j] ? narrow<E>(value_of<KIND>(f) * s[j][B / S::BPG]) : narrow<E>(0.f);
      }
      *(Run<E, 2>*)(to + 32 * B) = y;
    }
  }
}

template <int KIND, int D, int GROUP, typename E>
__global__ __launch_bounds__(kThreads) void write_kernel(CacheIoParams p, int ntile) {
  const Item w = item_of(p, ntile);
  if (blockIdx.y == 0)
    write_keys<KIND, D, GROUP, E>(p, w, threadIdx.x & 63);
  else
    write_values<KIND, D, GROUP, E>(p, w, threadIdx.x & 63);
}

template <int KIND, int D, int GROUP, typename E>
__global__ __launch_bounds__(kThreads) void read_kernel(CacheIoParams p, int ntile) {
  const Item w = item_of(p, ntile);
  if (blockIdx.y == 0)
    read_keys<KIND, D, GROUP, E>(p, w, threadIdx.x & 63);
  else
    read_values<KIND, D, GROUP, E>(p, w, threadIdx.x & 63);
}

template <bool WRITE, int KIND, int D, int GROUP, typename E>
hipError_t launch(const CacheIoParams& p, hipStream_t s) {
  const int ntile = cache_io_tiles(p.T);
  const dim3 grid((uint32_t)cache_io_blocks(p.B, p.T, p.Hkv), 2);
  if constexpr (WRITE)
    write_kernel<KIND, D, GROUP, E><<<grid, kThreads, 0, s>>>(p, ntile);
  else
    read_kernel<KIND, D, GROUP, E><<<grid, kThreads, 0, s>>>(p, ntile);
  return hipGetLastError();
}

template <bool WRITE, int KIND, int D, int GROUP>
hipError_t by_io(const CacheIoParams& p, int io_bf16, hipStream_t s) {
  return io_bf16 ? launch<WRITE, KIND, D, GROUP, uint16_t>(p, s) : launch<WRITE, KIND, D, GROUP, float>(p, s);
}

template <bool WRITE, int KIND, int D>
hipError_t by_group(const CacheIoParams& p, int group, int io_bf16, hipStream_t s) {
  if (group == 32) return by_io<WRITE, KIND, D, 32>(p, io_bf16, s);
  if (group == 64) return by_io<WRITE, KIND, D, 64>(p, io_bf16, s);
  if constexpr (D >= 128) return by_io<WRITE, KIND, D, 128>(p, io_bf16, s);
  return hipErrorInvalidValue;
}

template <bool WRITE, int KIND>
hipError_t by_d(const CacheIoParams& p, int d, int group, int io_bf16, hipStream_t s) {
  if (d == 64) return by_group<WRITE, KIND, 64>(p, group, io_bf16, s);
  if (d == 128) return by_group<WRITE, KIND, 128>(p, group, io_bf16, s);
  return by_group<WRITE, KIND, 256>(p, group, io_bf16, s);
}

template <bool WRITE>
hipError_t by_kind(const CacheIoParams& p, int kind, int d, int group, int io_bf16, hipStream_t s) {
  if (kind == PACE_CACHE_INT8) return by_d<WRITE, PACE_CACHE_INT8>(p, d, group, io_bf16, s);
  if (kind == PACE_CACHE_INT4) return by_d<WRITE, PACE_CACHE_INT4>(p, d, group, io_bf16, s);
  return by_d<WRITE, PACE_CACHE_FP8>(p, d, group, io_bf16, s);
}

}  // namespace

hipError_t launch_cache_write(const CacheIoParams& p, int kind, int d, int group, int io_bf16, hipStream_t stream) {
  return by_kind<true>(p, kind, d, group, io_bf16, stream);
}
hipError_t launch_cache_read(const CacheIoParams& p, int kind, int d, int group, int io_bf16, hipStream_t stream) {
  return by_kind<false>(p, kind, d, group, io_bf16, stream);
}

}  // namespace pace
