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
// Bound by memory: inputs read once, codes and scales written once, about 15 operations a value.
#include <hip/hip_runtime.h>

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

// Scale and reciprocal of a group from its largest magnitude.
template <int KIND>
__device__ inline void scale_of(float m, float& s, float& r) {
  constexpr float L = levels<KIND>();
  s = bf16_ceil_div(m, L, 1.0f / L);
  if (s < 0x1p-126f) s = 0.f;
  r = s > 0.f ? rcp_bf16(s) : 0.f;
}

// The stored field of x: x / s, correctly rounded (r is the correctly rounded reciprocal, the
// residual exact), then to the nearest code.
template <int KIND>
__device__ inline float quotient(float x, float s, float r) {
  constexpr float L = levels<KIND>();
  const float a = x * r, e = fmaf(-a, s, x);
  return fminf(fmaxf(fmaf(e, r, a), -L), L);
}
template <int KIND>
__device__ inline void fields_of(float x, float y, float s, float r, uint32_t& f, uint32_t& h) {
  float a = quotient<KIND>(x, s, r), b = quotient<KIND>(y, s, r);
  if constexpr (KIND == PACE_CACHE_FP8) {
    // the correction above turns -0 into +0: e4m3 keeps the quotient's sign (a zero group is +0)
    a = s > 0.f ? copysignf(a, x) : 0.f;
    b = s > 0.f ? copysignf(b, y) : 0.f;
    const uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    f = w & 0xFFu;
    h = (w >> 8) & 0xFFu;
  } else {
    constexpr int offset = KIND == PACE_CACHE_INT8 ? 128 : 8;
    f = (uint32_t)((int)rintf(a) + offset);
    h = (uint32_t)((int)rintf(b) + offset);
  }
}

template <int KIND>
__device__ inline float value_of(uint32_t f) {
  if constexpr (KIND == PACE_CACHE_FP8)
    return __builtin_amdgcn_cvt_f32_fp8((int)f, 0);
  else
    return (float)((int)f - (KIND == PACE_CACHE_INT8 ? 128 : 8));
}

// Maximum over the 16 lanes of a row, in every lane of it.
__device__ inline float row_max(float x) {
  x = fmaxf(x, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x128, 0xF, 0xF, true)));   // rotated by 8
  x = fmaxf(x, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x124, 0xF, 0xF, true)));
  x = fmaxf(x, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x122, 0xF, 0xF, true)));
  return fmaxf(x, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x121, 0xF, 0xF, true)));
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
  uint32_t word[S::LB / 4];
  float s[S::NG];
#pragma unroll
  for (int G = 0; G < S::NG; ++G) {
    float m = 0.f, inv;
#pragma unroll
    for (int j = 0; j < S::BPG; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(tame(widen(raw[G * S::BPG + j].v[i]))));
    scale_of<KIND>(rows_max(m), s[G], inv);
#pragma unroll
    for (int j = 0; j < S::BPG; ++j) {
      const int B = G * S::BPG + j;
      uint32_t f[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        fields_of<KIND>(tame(widen(raw[B].v[i])), tame(widen(raw[B].v[i + 1])), s[G], inv, f[i], f[i + 1]);
      if constexpr (KIND == PACE_CACHE_INT4) {
        word[B] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) word[B] |= f[i] << (4 * (i / 2 + 4 * (i & 1)));
      } else {
        word[2 * B] = f[0] | f[1] << 8 | f[2] << 16 | f[3] << 24;
        word[2 * B + 1] = f[4] | f[5] << 8 | f[6] << 16 | f[7] << 24;
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
  // word 2 B + e (8 bits) or B (4 bits): one byte a token
  uint32_t word[S::LB / 4];
#pragma unroll
  for (int i = 0; i < S::LB / 4; ++i) word[i] = 0u;
  uint16_t s[4][S::NG];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int G = 0; G < S::NG; ++G) {
      float mx = 0.f, sc, inv;
#pragma unroll
      for (int k = 0; k < S::BPG; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) mx = fmaxf(mx, fabsf(tame(widen(raw[j][G * S::BPG + k].v[e]))));
      scale_of<KIND>(row_max(mx), sc, inv);
      s[j][G] = (uint16_t)(f32_bits(sc) >> 16);
#pragma unroll
      for (int k = 0; k < S::BPG; ++k) {
        const int B = G * S::BPG + k;
        uint32_t f, h;
        fields_of<KIND>(tame(widen(raw[j][B].v[0])), tame(widen(raw[j][B].v[1])), sc, inv, f, h);
        if constexpr (KIND == PACE_CACHE_INT4) {
          word[B] |= (f | h << 4) << (8 * j);
        } else {
          word[2 * B] |= f << (8 * j);
          word[2 * B + 1] |= h << (8 * j);
        }
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
  // tiles of 16 tokens; the first token of 16 or more may be at any place of its tile
  const int ntile = p.T < 16 ? 1 : (int)(((int64_t)p.T + 15 + 15) / 16);
  const int64_t waves = (int64_t)p.B * ntile * p.Hkv;
  if (waves > 0x7FFFFFFF - 4) return hipErrorInvalidValue;
  const int64_t blocks = (waves + 3) / 4;
  const dim3 grid((uint32_t)blocks, 2);
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
