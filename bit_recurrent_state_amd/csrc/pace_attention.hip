// Attention for drafted tokens over the quantised paged cache: the join of a context's pieces,
// and the choice of the kernel (pace_attention.h, one source per cache kind).
#include <hip/hip_runtime.h>

#include "pace_cache_internal.h"

namespace pace {
namespace {

constexpr int kJoin = 256;       // threads of a joining workgroup
constexpr int kFewPieces = 16;

// Four channels of a row and its lse to where the caller wants them.
template <int D, bool BF16>
__device__ inline void store_row(const AttnParams& p, int64_t row, int c, float4 acc, float top, float sum) {
  const int r = (int)(row % p.R), i = r / p.gamma;
  const int64_t bh = row / p.R, b = bh / p.Hkv, h = bh % p.Hkv;
  const int64_t at = (b * p.T + i) * p.Hq + h * p.gamma + (r - i * p.gamma);
  if (c == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
  if constexpr (BF16) {
    auto pack = [&](float x, float y) {
      return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)y) << 16;
    };
    *(uint2*)((uint16_t*)p.o + at * D + 4 * c) = make_uint2(pack(acc.x, acc.y), pack(acc.z, acc.w));
  } else {
    *(float4*)((float*)p.o + at * D + 4 * c) = acc;
  }
}

// Pieces are summed by their shares of the weight, which add up to 1: outputs of up to 2^127 stay finite.

// Few pieces, usually of many rows: D / 4 threads a row, four channels each, which walk the pieces
// themselves.  (A workgroup a row took 38 us for the 32768 rows of 2 pieces of a 512-token chunk.)
template <int D, bool BF16>
__global__ __launch_bounds__(kJoin) void join_few_kernel(AttnParams p) {
  constexpr int C = D / 4;
  const int64_t rows = (int64_t)p.B * p.Hkv * p.R, row = (int64_t)blockIdx.x * (kJoin / C) + threadIdx.x / C;
  const int c = threadIdx.x % C;
  if (row >= rows) return;
  float l[kFewPieces];
  float4 o[4];
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int s = 0; s < kFewPieces; ++s) {
    l[s] = s < p.nsplit ? p.part_lse[s * rows + row] : -INFINITY;
    top = fmaxf(top, l[s]);
  }
  if (top == -INFINITY) top = 0.f;      // nothing seen (or NaN everywhere)
#pragma unroll
  for (int s = 0; s < kFewPieces; ++s) {
    l[s] = __builtin_amdgcn_exp2f(l[s] - top);
    sum += l[s];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s0 = 0; s0 < kFewPieces; s0 += 4) {
    if (s0 >= p.nsplit) break;
#pragma unroll
    for (int k = 0; k < 4; ++k)         // an empty piece wrote no output
      o[k] = l[s0 + k] != 0.f ? *(const float4*)(p.part_o + ((s0 + k) * rows + row) * D + 4 * c) : float4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = l[s0 + k] * inv;
      acc.x = fmaf(f, o[k].x, acc.x);
      acc.y = fmaf(f, o[k].y, acc.y);
      acc.z = fmaf(f, o[k].z, acc.z);
      acc.w = fmaf(f, o[k].w, acc.w);
    }
  }
  store_row<D, BF16>(p, row, c, acc, top, sum);
}

// Many pieces.  One workgroup a row: D / 4 threads hold its channels, four each, and
// the 256 / (D / 4) groups of them take every so many-th piece, so that many pieces' loads are
// in flight at once (one wave walking the pieces one by one took over 1 us a piece).  Weights
// first, once, in LDS; sums in a fixed order.
template <int D, bool BF16>
__global__ __launch_bounds__(kJoin) void join_kernel(AttnParams p) {
  constexpr int C = D / 4, NGRP = kJoin / C;
  __shared__ float weight[kMaxPieces];
  __shared__ float4 part[kJoin];
  __shared__ float red[kJoin / 64][2];
  const int64_t row = blockIdx.x, rows = (int64_t)p.B * p.Hkv * p.R;   // (b, h, r)
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < p.nsplit; s += kJoin) {
    const float l = p.part_lse[s * rows + row];
    weight[s] = l;
    top = fmaxf(top, l);
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) top = fmaxf(top, __shfl_xor(top, k));
  if (lane == 0) red[wave][0] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
  if (top == -INFINITY) top = 0.f;      // nothing seen (or NaN everywhere)
  float sum = 0.f;
  for (int s = threadIdx.x; s < p.nsplit; s += kJoin) {
    const float f = __builtin_amdgcn_exp2f(weight[s] - top);
    weight[s] = f;
    sum += f;
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) sum += __shfl_xor(sum, k);
  if (lane == 0) red[wave][1] = sum;
  __syncthreads();
  sum = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  const int c = threadIdx.x % C, grp = threadIdx.x / C;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = grp; s < p.nsplit; s += NGRP) {
    const float f = weight[s] * inv;
    if (f != 0.f) {                     // an empty piece wrote no output
      const float4 o = *(const float4*)(p.part_o + (s * rows + row) * D + 4 * c);
      acc.x = fmaf(f, o.x, acc.x);
      acc.y = fmaf(f, o.y, acc.y);
      acc.z = fmaf(f, o.z, acc.z);
      acc.w = fmaf(f, o.w, acc.w);
    }
  }
  part[threadIdx.x] = acc;
  __syncthreads();
  if (grp > 0) return;
  for (int k = 1; k < NGRP; ++k) {
    const float4 o = part[k * C + c];
    acc.x += o.x;
    acc.y += o.y;
    acc.z += o.z;
    acc.w += o.w;
  }
  store_row<D, BF16>(p, row, c, acc, top, sum);
}

template <int D, bool BF16>
hipError_t join_d(const AttnParams& p, hipStream_t s) {
  const int64_t rows = (int64_t)p.B * p.Hkv * p.R;
  constexpr int per = kJoin / (D / 4);
  if (p.nsplit <= kFewPieces)
    join_few_kernel<D, BF16><<<(uint32_t)((rows + per - 1) / per), kJoin, 0, s>>>(p);
  else
    join_kernel<D, BF16><<<(uint32_t)rows, kJoin, 0, s>>>(p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t join(const AttnParams& p, int d, hipStream_t s) {
  return d == 64 ? join_d<64, BF16>(p, s) : d == 128 ? join_d<128, BF16>(p, s) : join_d<256, BF16>(p, s);
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
