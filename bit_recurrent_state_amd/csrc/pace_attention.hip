// Attention for drafted tokens over the quantised paged cache: the join of a context's pieces,
// and the choice of the kernel (pace_attention.h, one source per cache kind).
#include <hip/hip_runtime.h>

#include "pace_cache_internal.h"

namespace pace {
namespace {

constexpr int kJoinWaves = 4;

// Joins the pieces of a row: one wave a row, D / 64 channels a lane, pieces in order.
template <int D, bool BF16>
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(AttnParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kJoinWaves + (threadIdx.x >> 6);   // (b, h, r)
  const int64_t rows = (int64_t)p.B * p.Hkv * p.R;
  if (row >= rows) return;
  constexpr int C = D / 64;
  float top = -INFINITY;
  for (int s = 0; s < p.nsplit; ++s) top = fmaxf(top, p.part_lse[s * rows + row]);
  if (top == -INFINITY) top = 0.f;      // nothing seen (or NaN everywhere)
  float acc[C] = {}, sum = 0.f;
  for (int s = 0; s < p.nsplit; ++s) {
    const float l = p.part_lse[s * rows + row];
    if (l == -INFINITY) continue;       // an empty piece wrote no output
    const float f = __builtin_amdgcn_exp2f(l - top);
    sum += f;
    const float* o = p.part_o + (s * rows + row) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(f, o[c], acc[c]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int r = (int)(row % p.R), i = r / p.gamma;
  const int64_t bh = row / p.R, b = bh / p.Hkv, h = bh % p.Hkv;
  const int64_t at = (b * p.T + i) * p.Hq + h * p.gamma + (r - i * p.gamma);
  if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float x = acc[c] * inv;
    if constexpr (BF16)
      ((uint16_t*)p.o)[at * D + lane * C + c] = __builtin_bit_cast(uint16_t, (__bf16)x);
    else
      ((float*)p.o)[at * D + lane * C + c] = x;
  }
}

template <bool BF16>
hipError_t join(const AttnParams& p, int d, hipStream_t s) {
  const int64_t rows = (int64_t)p.B * p.Hkv * p.R;
  const uint32_t grid = (uint32_t)((rows + kJoinWaves - 1) / kJoinWaves);
  if (d == 64)
    join_kernel<64, BF16><<<grid, kJoinWaves * 64, 0, s>>>(p);
  else if (d == 128)
    join_kernel<128, BF16><<<grid, kJoinWaves * 64, 0, s>>>(p);
  else
    join_kernel<256, BF16><<<grid, kJoinWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnParams& p, const AttnPlan& plan, int kind, int d, int group, int io_bf16,
                            hipStream_t stream) {
  const hipError_t e = kind == PACE_CACHE_INT8   ? launch_attention_int8(p, plan, d, group, io_bf16, stream)
                       : kind == PACE_CACHE_INT4 ? launch_attention_int4(p, plan, d, group, io_bf16, stream)
                                                 : launch_attention_fp8(p, plan, d, group, io_bf16, stream);
  if (e != hipSuccess || p.nsplit == 1) return e;
  return io_bf16 ? join<true>(p, d, stream) : join<false>(p, d, stream);
}

}  // namespace pace
