// The decode buffer's quantiser on tokens held 8 channels a lane (include/pace.h: DECODE BUFFER LAYOUT):
// code c = rne(x / s) in fp32, s = fp32(max|x| / 127), or / 7 for 4-bit keys.  D / 8 neighbouring lanes hold a token.
// The same operations as in the decode kernel, so that the codes and scales are the same bits.
#pragma once

#include <hip/hip_runtime.h>

#include "pace_numerics.h"

namespace pace {

// Lane permutations inside rows of 16 lanes (DPP).
template <int CTRL>
__device__ inline float row_shuffle(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}

// Maximum over the 8 or 16 lanes of a token; every one of them ends with it.
template <int LANES>
__device__ inline float token_max(float x) {
  x = fmaxf(x, row_shuffle<0xB1>(x));
  x = fmaxf(x, row_shuffle<0x4E>(x));
  x = fmaxf(x, row_shuffle<0x141>(x));
  if constexpr (LANES == 16) x = fmaxf(x, row_shuffle<0x140>(x));
  return x;
}

// Eight neighbouring elements of a q, k or v row, as they lie in memory.
template <bool BF16>
struct Raw8 {
  uint32_t w[BF16 ? 4 : 8];
  __device__ void load(const void* p) {
    const uint4* from = (const uint4*)p;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
      const uint4 v = from[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
  __device__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (BF16) x[i] = bits_f32(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      else x[i] = bits_f32(w[i]);
    }
  }
};
template <bool BF16>
__device__ inline void load8(const void* p, int64_t at, float (&x)[8]) {
  Raw8<BF16> r;
  r.load((const uint8_t*)p + at * (BF16 ? 2 : 4));
  r.values(x);
}

// Codes (whole numbers) and scale of a token.  x / s is formed in three operations from the correctly rounded reciprocal
// (q = fl(x r) is within an ulp, its residual exact in a fused step, and one more rounds correctly: Markstein), the same
// fp32 quotient as the decode's division in a quarter of its operations.  Its rounding needs no clamp, since s is at most an
// ulp under max|x| / top.  A scale whose reciprocal would leave fp32's normal range takes the division.
template <int LANES>
__device__ inline float quantise8(const float (&x)[8], bool four_bits, float (&c)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  m = token_max<LANES>(m);
  const float s = div_rn(m, four_bits ? 7.f : 127.f, four_bits ? 1.0f / 7.0f : 1.0f / 127.0f);
  const float r = 1.0f / s;
  if (__builtin_expect(__any(s < 0x1p-100f), 0)) {
    const float top = four_bits ? 7.f : 127.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s > 0.f ? fminf(fmaxf(rintf(x[i] / s), -top), top) : 0.f;
    return s;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * r;
    c[i] = rintf(fmaf(fmaf(-q, s, x[i]), r, q));
  }
  return s;
}

// Two fp32 values rounded to nearest-even bf16, packed (a in the low half).
__device__ inline uint32_t two_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

}  // namespace pace
