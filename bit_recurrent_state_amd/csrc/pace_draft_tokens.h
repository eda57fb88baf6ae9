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

// Eight neighbouring elements of a q, k or v row.
template <bool BF16>
__device__ inline void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 w = *(const uint4*)((const uint16_t*)p + at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bits_f32(u[i] << 16);
      x[2 * i + 1] = bits_f32(u[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *(const float4*)((const float*)p + at), b = *(const float4*)((const float*)p + at + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// Codes (whole numbers) and scale of a token.
template <int LANES>
__device__ inline float quantise8(const float (&x)[8], bool four_bits, float (&c)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  m = token_max<LANES>(m);
  const float top = four_bits ? 7.f : 127.f;
  const float s = div_rn(m, top, four_bits ? 1.0f / 7.0f : 1.0f / 127.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = s > 0.f ? fminf(fmaxf(rintf(x[i] / s), -top), top) : 0.f;
  return s;
}

// Two fp32 values rounded to nearest-even bf16, packed (a in the low half).
__device__ inline uint32_t two_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

}  // namespace pace
