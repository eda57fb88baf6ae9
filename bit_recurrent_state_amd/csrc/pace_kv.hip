// The quantised paged key/value cache: writing and reading back (include/pace_cache.h:
// pace_cache_write, pace_cache_read; layout and quantiser there).
//
// A thread takes 8 channels of up to four consecutive tokens of one head (16-byte loads of
// bf16 inputs); the g / 8 threads of a scale group find its maximum with lane exchanges.
// Values lie interleaved by four tokens, so a thread that holds a whole quad of positions
// stores (loads) 8 bytes a lane where one token alone would store bytes; quads are cut at
// the sequence's first position, so that a run of positions fills whole quads from any start.
// Bound by memory: inputs read once, codes and scales written once; the arithmetic is about
// 12 operations a value.  Keys and values are two rows of the grid.
#include <hip/hip_runtime.h>

#include "pace_cache_internal.h"
#include "pace_numerics.h"

namespace pace {
namespace {

constexpr int kThreads = 256;

template <typename E>
struct alignas(16) Eight {
  E v[8];
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

// Byte offsets inside a record of the 8-channel unit u (channels 8 u .. 8 u + 7).
template <int KIND, int D, int GROUP>
struct Place {
  static constexpr int BITS = KIND == PACE_CACHE_INT4 ? 4 : 8;
  static constexpr int LB = D * BITS / 32;          // bytes a lane holds
  static constexpr int W = LB < 16 ? LB : 16;
  static constexpr int NG = D / GROUP;
  static constexpr int UB = BITS;                   // bytes of one unit of 8 codes
  // keys: the unit of token r
  static __device__ uint32_t key(int r, int u) {
    const int x = (u >> 2) * UB, a = u & 3;
    return (uint32_t)(r >> 4) * (64 * LB) + (x / W) * (64 * W) + (16 * a + (r & 15)) * W + x % W;
  }
  // values: the two channels 8 u + 2 i, + 1 of the quad that holds token r; UB bytes:
  // 8 bits: [2 channels][4 tokens], 4 bits: [4 tokens] (both channels in a byte)
  static __device__ uint32_t value(int r, int u, int i) {
    const int x = (u >> 2) * UB, m = 4 * (u & 3) + i;
    return (uint32_t)(r >> 2) * (16 * LB) + (x / W) * (16 * W) + m * W + x % W;
  }
  static __device__ uint32_t scale(int r, int u) {
    return 2u * (((uint32_t)(r >> 2) * NG + u * 8 / GROUP) * 4 + (r & 3));
  }
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

// Stored fields of 8 values: 8 bits in two words, channel order; 4 bits one byte a value too.
template <int KIND, int GROUP>
__device__ inline float quantise(const float (&x)[8], uint32_t (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
  for (int s = 1; s < GROUP / 8; s *= 2) m = fmaxf(m, __shfl_xor(m, s));
  constexpr float L = levels<KIND>();
  float s = bf16_ceil_div(m, L, 1.0f / L);
  if (s < 0x1p-126f) s = 0.f;
  const float r = s > 0.f ? rcp_bf16(s) : 0.f;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // x / s, correctly rounded: r is the correctly rounded reciprocal, the residual exact
    const float a = x[i] * r, e = fmaf(-a, s, x[i]);
    q[i] = fminf(fmaxf(fmaf(e, r, a), -L), L);
  }
  if constexpr (KIND == PACE_CACHE_FP8) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // the correction above turns -0 into +0: e4m3 keeps the quotient's sign (a zero group is +0)
      const float a = s > 0.f ? copysignf(q[i], x[i]) : 0.f, b = s > 0.f ? copysignf(q[i + 1], x[i + 1]) : 0.f;
      const uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
      f[i] = w & 0xFFu;
      f[i + 1] = (w >> 8) & 0xFFu;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (uint32_t)((int)rintf(q[i]) + (KIND == PACE_CACHE_INT8 ? 128 : 8));
  }
  return s;
}

template <int KIND>
__device__ inline float value_of(uint32_t f) {
  if constexpr (KIND == PACE_CACHE_FP8)
    return __builtin_amdgcn_cvt_f32_fp8((int)f, 0);
  else
    return (float)((int)f - (KIND == PACE_CACHE_INT8 ? 128 : 8));
}

// The key unit of 8 fields as stored words.
template <int KIND>
__device__ inline uint2 key_words(const uint32_t (&f)[8]) {
  uint2 w = {0u, 0u};
  if constexpr (KIND == PACE_CACHE_INT4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w.x |= f[i] << (4 * (i / 2 + 4 * (i & 1)));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w.x |= f[i] << (8 * i);
      w.y |= f[i + 4] << (8 * i);
    }
  }
  return w;
}

template <int KIND>
__device__ inline void key_fields(uint2 w, uint32_t (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = KIND == PACE_CACHE_INT4 ? (w.x >> (4 * (i / 2 + 4 * (i & 1)))) & 15u
                                   : ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 255u;
}

// What a thread works on: sequence, head, unit, and its four token indexes.
struct Item {
  int b, h, u, t0;   // t0: token index of the quad's first position (may be negative)
  bool in;
};

template <int D>
__device__ inline Item item_of(const CacheIoParams& p, int nquad) {
  constexpr int U = D / 8;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  Item w;
  w.u = (int)(id % U);
  const int64_t r = id / U;
  w.h = (int)(r % p.Hkv);
  const int64_t bq = r / p.Hkv;
  w.b = (int)(bq / nquad);
  w.in = w.b < p.B;
  if (!w.in) w.b = 0;
  const int first = p.positions[(int64_t)w.b * p.T];
  w.t0 = (int)(bq % nquad) * 4 - (first >= 0 ? (first & 3) : 0);
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

template <int KIND, int D, int GROUP, typename E>
__global__ __launch_bounds__(kThreads) void write_kernel(CacheIoParams p, int nquad) {
  using L = Place<KIND, D, GROUP>;
  const Item w = item_of<D>(p, nquad);
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, L::BITS);
  const bool isv = blockIdx.y != 0;
  const E* in = (const E*)(isv ? p.v_in : p.k_in);
  const int64_t stride = isv ? p.v_stride : p.k_stride;
  uint8_t* at[4];
  int pos[4], r[4];
  Eight<E> raw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    at[j] = record_of(p, w, w.t0 + j, rec.total, pos[j], r[j]);
    raw[j] = {};
    if (at[j]) raw[j] = *(const Eight<E>*)(in + ((int64_t)w.b * p.T + w.t0 + j) * stride + w.h * D + w.u * 8);
  }
  uint32_t f[4][8];
  uint16_t s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = tame(widen(raw[j].v[i]));
    s[j] = (uint16_t)(f32_bits(quantise<KIND, GROUP>(x, f[j])) >> 16);
  }
  const uint32_t codes_at = isv ? rec.codes + rec.scales : 0u, scales_at = codes_at + rec.codes;
  const bool leads = w.u % (GROUP / 8) == 0;
  // a whole quad of one page: positions r0 .. r0 + 3 with r0 a multiple of 4
  const bool quad = at[0] && at[1] && at[2] && at[3] && (pos[0] & 3) == 0 && pos[1] == pos[0] + 1 &&
                    pos[2] == pos[0] + 2 && pos[3] == pos[0] + 3;
  if (quad) {
    if (leads)
      *(uint2*)(at[0] + scales_at + L::scale(r[0], w.u)) =
          make_uint2(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16);
    if (isv) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo = 0u, hi = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (KIND == PACE_CACHE_INT4) {
            lo |= (f[j][2 * i] | f[j][2 * i + 1] << 4) << (8 * j);
          } else {
            lo |= f[j][2 * i] << (8 * j);
            hi |= f[j][2 * i + 1] << (8 * j);
          }
        }
        uint8_t* to = at[0] + codes_at + L::value(r[0], w.u, i);
        if constexpr (KIND == PACE_CACHE_INT4)
          *(uint32_t*)to = lo;
        else
          *(uint2*)to = make_uint2(lo, hi);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!at[j]) continue;
    if (leads && !quad) *(uint16_t*)(at[j] + scales_at + L::scale(r[j], w.u)) = s[j];
    if (isv) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint8_t* to = at[j] + codes_at + L::value(r[j], w.u, i) + (r[j] & 3);
        if constexpr (KIND == PACE_CACHE_INT4) {
          *to = (uint8_t)(f[j][2 * i] | f[j][2 * i + 1] << 4);
        } else {
          to[0] = (uint8_t)f[j][2 * i];
          to[4] = (uint8_t)f[j][2 * i + 1];
        }
      }
    } else {
      const uint2 k = key_words<KIND>(f[j]);
      uint8_t* to = at[j] + L::key(r[j], w.u);
      if constexpr (KIND == PACE_CACHE_INT4)
        *(uint32_t*)to = k.x;
      else
        *(uint2*)to = k;
    }
  }
}

template <int KIND, int D, int GROUP, typename E>
__global__ __launch_bounds__(kThreads) void read_kernel(CacheIoParams p, int nquad) {
  using L = Place<KIND, D, GROUP>;
  const Item w = item_of<D>(p, nquad);
  const CacheRecord rec = cache_record(D, GROUP, 1 << p.page_shift, L::BITS);
  const bool isv = blockIdx.y != 0;
  E* out = (E*)(isv ? p.v_out : p.k_out);
  const int64_t stride = isv ? p.v_stride : p.k_stride;
  const uint32_t codes_at = isv ? rec.codes + rec.scales : 0u, scales_at = codes_at + rec.codes;
  uint8_t* at[4];
  int pos[4], r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) at[j] = record_of(p, w, w.t0 + j, rec.total, pos[j], r[j]);
  const bool quad = at[0] && at[1] && at[2] && at[3] && (pos[0] & 3) == 0 && pos[1] == pos[0] + 1 &&
                    pos[2] == pos[0] + 2 && pos[3] == pos[0] + 3;
  uint32_t f[4][8];
  uint16_t s[4] = {0, 0, 0, 0};
  if (quad) {
    const uint2 sw = *(const uint2*)(at[0] + scales_at + L::scale(r[0], w.u));
    s[0] = (uint16_t)sw.x; s[1] = (uint16_t)(sw.x >> 16);
    s[2] = (uint16_t)sw.y; s[3] = (uint16_t)(sw.y >> 16);
  }
  if (isv && quad) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* from = at[0] + codes_at + L::value(r[0], w.u, i);
      uint2 y;
      if constexpr (KIND == PACE_CACHE_INT4)
        y.x = *(const uint32_t*)from, y.y = 0u;
      else
        y = *(const uint2*)from;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (KIND == PACE_CACHE_INT4) {
          f[j][2 * i] = (y.x >> (8 * j)) & 15u;
          f[j][2 * i + 1] = (y.x >> (8 * j + 4)) & 15u;
        } else {
          f[j][2 * i] = (y.x >> (8 * j)) & 255u;
          f[j][2 * i + 1] = (y.y >> (8 * j)) & 255u;
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!at[j]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] = 0u;
        continue;
      }
      if (!quad) s[j] = *(const uint16_t*)(at[j] + scales_at + L::scale(r[j], w.u));
      if (isv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* from = at[j] + codes_at + L::value(r[j], w.u, i) + (r[j] & 3);
          if constexpr (KIND == PACE_CACHE_INT4) {
            f[j][2 * i] = *from & 15u;
            f[j][2 * i + 1] = *from >> 4;
          } else {
            f[j][2 * i] = from[0];
            f[j][2 * i + 1] = from[4];
          }
        }
      } else {
        const uint8_t* from = at[j] + L::key(r[j], w.u);
        uint2 y;
        if constexpr (KIND == PACE_CACHE_INT4)
          y.x = *(const uint32_t*)from, y.y = 0u;
        else
          y = *(const uint2*)from;
        key_fields<KIND>(y, f[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = w.t0 + j;
    if (!w.in || t < 0 || t >= p.T) continue;
    const float sc = bf16_to_f32(s[j]);
    Eight<E> y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y.v[i] = at[j] ? narrow<E>(value_of<KIND>(f[j][i]) * sc) : narrow<E>(0.f);
    *(Eight<E>*)(out + ((int64_t)w.b * p.T + t) * stride + w.h * D + w.u * 8) = y;
  }
}

template <bool WRITE, int KIND, int D, int GROUP, typename E>
hipError_t launch(const CacheIoParams& p, hipStream_t s) {
  const int nquad = (int)(((int64_t)p.T + 3 + 3) / 4);   // T tokens, the first at any place of its quad
  const int64_t threads = (int64_t)p.B * nquad * p.Hkv * (D / 8);
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)blocks, 2);
  if constexpr (WRITE)
    write_kernel<KIND, D, GROUP, E><<<grid, kThreads, 0, s>>>(p, nquad);
  else
    read_kernel<KIND, D, GROUP, E><<<grid, kThreads, 0, s>>>(p, nquad);
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
