// Rotary positions (include/pace_cache.h: pace_rotary).
//
// One workgroup takes kTok tokens: its threads first form the kTok * rd / 2 cosines and
// sines in LDS (the angle's turn count in fp64, its fraction in fp32), then walk the tokens'
// heads in units of 8 channels, 16 bytes a lane.  Bound by memory: every element is read and
// written once; the trigonometry is shared by all heads of a token.  32768 tokens of 40 heads of 128,
// bf16: 126 us, 5.3 TB/s, a large copy's rate.  1021 tokens of 20 heads of 256, fp32: 9.4 us, 4.4 TB/s.
// 64 tokens: 3.1 us, of which an empty launch is half.
#include <hip/hip_runtime.h>

#include "pace_cache_internal.h"
#include "pace_numerics.h"

namespace pace {
namespace {

constexpr int kThreads = 256;
constexpr double kInv2Pi = 0.15915494309189533577;

template <typename E>
struct Io;
template <>
struct Io<float> {
  static __device__ float get(float x) { return x; }
  static __device__ float put(float x) { return x; }
};
template <>
struct Io<uint16_t> {
  static __device__ float get(uint16_t x) { return bf16_to_f32(x); }
  static __device__ uint16_t put(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};

template <typename E>
struct alignas(16) Eight {
  E v[8];
};

// (cos, sin) of the kTok tokens' angles, times the magnitude; inverse flips the sine.
__device__ inline void angles(const RotaryParams& p, int tok0, int ntok, float2* cs) {
  const int half = p.rd / 2;
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const double turns = (double)p.positions[tok0 + t] * (p.freqs[j] * kInv2Pi);
    const float f = (float)(turns - rint(turns));   // [-1/2, 1/2]: 2 f pi is the angle
    const float c = cospif(2.f * f) * p.magnitude, s = sinpif(2.f * f) * p.magnitude;
    cs[i] = make_float2(c, p.inverse ? -s : s);
  }
  __syncthreads();
}

// Units of 8 channels; in the half layout a unit of the first half takes its partner along.
template <typename E, bool IL>
__global__ __launch_bounds__(kThreads) void rotary_wide(RotaryParams p, int tok_per_wg) {
  extern __shared__ float2 cs[];
  const int tok0 = blockIdx.x * tok_per_wg, ntok = min(tok_per_wg, p.n - tok0), half = p.rd / 2;
  angles(p, tok0, ntok, cs);
  const int rot = IL ? p.rd / 8 : p.rd / 16, tail = (p.d - p.rd) / 8, per = rot + tail;
  const int heads = p.Hq + p.Hk, total = ntok * heads * per;
  for (int u = threadIdx.x; u < total; u += kThreads) {
    const int th = u / per, c = u - th * per, t = th / heads, h = th - t * heads;
    const bool isq = h < p.Hq;
    const int hh = isq ? h : h - p.Hq;
    const E* in = (const E*)(isq ? p.q : p.k) + (int64_t)(tok0 + t) * (isq ? p.q_stride : p.k_stride) + hh * p.d;
    E* out = (E*)(isq ? p.q_out : p.k_out) + (int64_t)(tok0 + t) * (isq ? p.q_out_stride : p.k_out_stride) + hh * p.d;
    if (c >= rot) {
      if (isq ? p.copy_q : p.copy_k) {
        const int at = p.rd + (c - rot) * 8;
        *(Eight<E>*)(out + at) = *(const Eight<E>*)(in + at);
      }
    } else if constexpr (IL) {
      const Eight<E> x = *(const Eight<E>*)(in + c * 8);
      Eight<E> y;
      const float2* w = cs + t * half + c * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = Io<E>::get(x.v[2 * i]), b = Io<E>::get(x.v[2 * i + 1]);
        y.v[2 * i] = Io<E>::put(a * w[i].x - b * w[i].y);
        y.v[2 * i + 1] = Io<E>::put(b * w[i].x + a * w[i].y);
      }
      *(Eight<E>*)(out + c * 8) = y;
    } else {
      const Eight<E> x = *(const Eight<E>*)(in + c * 8), z = *(const Eight<E>*)(in + half + c * 8);
      Eight<E> y0, y1;
      const float2* w = cs + t * half + c * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = Io<E>::get(x.v[i]), b = Io<E>::get(z.v[i]);
        y0.v[i] = Io<E>::put(a * w[i].x - b * w[i].y);
        y1.v[i] = Io<E>::put(b * w[i].x + a * w[i].y);
      }
      *(Eight<E>*)(out + c * 8) = y0;
      *(Eight<E>*)(out + half + c * 8) = y1;
    }
  }
}

// Any even d and rd, any stride and alignment: one pair (or one copied channel pair) a step.
template <typename E>
__global__ __launch_bounds__(kThreads) void rotary_pairs(RotaryParams p) {
  extern __shared__ float2 cs[];
  const int tok = blockIdx.x, half = p.rd / 2, pairs = p.d / 2, heads = p.Hq + p.Hk;
  angles(p, tok, 1, cs);
  for (int u = threadIdx.x; u < heads * pairs; u += kThreads) {
    const int h = u / pairs, c = u - h * pairs;
    const bool isq = h < p.Hq;
    const int hh = isq ? h : h - p.Hq;
    const E* in = (const E*)(isq ? p.q : p.k) + (int64_t)tok * (isq ? p.q_stride : p.k_stride) + hh * p.d;
    E* out = (E*)(isq ? p.q_out : p.k_out) + (int64_t)tok * (isq ? p.q_out_stride : p.k_out_stride) + hh * p.d;
    if (c < half) {
      const int i = p.interleaved ? 2 * c : c, j = p.interleaved ? 2 * c + 1 : c + half;
      const float a = Io<E>::get(in[i]), b = Io<E>::get(in[j]);
      out[i] = Io<E>::put(a * cs[c].x - b * cs[c].y);
      out[j] = Io<E>::put(b * cs[c].x + a * cs[c].y);
    } else if (isq ? p.copy_q : p.copy_k) {
      out[2 * c] = in[2 * c];
      out[2 * c + 1] = in[2 * c + 1];
    }
  }
}

template <typename E>
void launch(const RotaryParams& p, bool wide, hipStream_t s) {
  if (!wide) {
    rotary_pairs<E><<<p.n, kThreads, p.rd / 2 * sizeof(float2), s>>>(p);
    return;
  }
  // four tokens a workgroup where that still leaves eight workgroups a compute unit, so that the angles'
  // barrier is paid once for four; one below
  const int tok = p.n >= 4 * 2048 ? 4 : 1;
  const int grid = (p.n + tok - 1) / tok;
  const size_t lds = (size_t)tok * (p.rd / 2) * sizeof(float2);
  if (p.interleaved)
    rotary_wide<E, true><<<grid, kThreads, lds, s>>>(p, tok);
  else
    rotary_wide<E, false><<<grid, kThreads, lds, s>>>(p, tok);
}

}  // namespace

hipError_t launch_rotary(const RotaryParams& p, int io_bf16, bool wide, hipStream_t stream) {
  if (io_bf16)
    launch<uint16_t>(p, wide, stream);
  else
    launch<float>(p, wide, stream);
  return hipGetLastError();
}

}  // namespace pace
