// Accepted drafts into the decode buffer (include/pace_draft.h: pace_draft_commit).
//
// One workgroup per (sequence, value head) takes the head's share of the path: tokens in D / 8 lanes each, 8 channels a lane,
// through the buffer quantiser and into the slots from the head's count on, up to the end of the period.  The rounding
// of the buffers that this fills is the decode kernel's own fold, launched after this one; a further launch of
// this one goes on with the tokens that are left.  Bound by latency: counts -> nodes -> tokens -> slots.
//
// Measured, 64 sequences of up to 8 tokens, 32/16 heads of 128: launches of 5.0 us, 3.6 (fold) and 2.4 (mostly
// nothing left), 11.4 us together in a graph, 24.5 where every sequence ends its period; a launch that finds nothing to do takes
// 2.4.  Tokens of the next period need a launch behind the fold, since the value heads of a key head share its key slots.
#include <hip/hip_runtime.h>

#include "pace_draft_internal.h"
#include "pace_draft_tokens.h"

namespace pace {
namespace {

constexpr int kThreads = 128;

template <int D, bool BF16, bool MIXED>
__global__ __launch_bounds__(kThreads) void append_kernel(CommitParams p) {
  constexpr int LANES = D / 8, ROWS = kThreads / LANES;
  const DecodeParams& l = p.l;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int kh = h / l.gamma;
  const size_t bh = (size_t)b * l.Hv + h;
  int32_t* const countp = (int32_t*)l.buffer + bh;
  const int n = min(max(*countp, 0), l.dP - 1);
  const int done = p.done ? p.done[bh] & kTakenMask : 0;
  int m = min(max(p.counts[b], 0), p.most);
  // the path ends at its first index that is no node (T <= 64: one lane each)
  const int node_l = lane < p.T ? p.nodes[(size_t)b * p.T + lane] : -1;
  const uint64_t bad = __ballot(lane < m && (node_l < 0 || node_l >= p.T));
  if (bad) m = min(m, __builtin_ctzll(bad));
  const int take = min(m - done, l.dP - n);
  if (tid == 0) p.done_out[bh] = (done + max(take, 0)) | (take > 0 && n + take == l.dP ? kFilled : 0);
  if (take <= 0) return;

  const int c0 = 8 * (tid % LANES);
  const size_t kslot = ((size_t)b * l.Hk + kh) * l.dP + n, vslot = bh * l.dP + n;
  const bool keys = h % l.gamma == 0;
  for (int i0 = 0; i0 < take; i0 += ROWS) {
    const int i = i0 + tid / LANES;
    const bool in = i < take;
    const int node = __shfl(node_l, done + (in ? i : 0));
    const size_t tok = (size_t)b * p.T + node;
    float x[8], c[8];
    if (keys) {
      load8<BF16>(l.k, (int64_t)((tok * l.Hk + kh) * D + c0), x);
      const float s = quantise8<LANES>(x, MIXED, c);
      if (in) {
        if constexpr (MIXED) {
          // byte w of a unit: channel w in the low nibble, 4 + w in the high, each plus 8
          uint32_t w = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) w |= (uint32_t)((int)c[j] + 8 + (((int)c[4 + j] + 8) << 4)) << (8 * j);
          *(uint32_t*)(l.buffer + l.off_kc + (kslot + i) * (D / 2) + c0 / 2) = w;
        } else {
          uint32_t w[2] = {0u, 0u};
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j / 4] |= ((uint32_t)(int)c[j] & 255u) << (8 * (j % 4));
          *(uint2*)(l.buffer + l.off_kc + (kslot + i) * D + c0) = make_uint2(w[0], w[1]);
        }
        if (c0 == 0) ((float*)(l.buffer + l.off_ks))[kslot + i] = s;
      }
    }
    load8<BF16>(l.v, (int64_t)((tok * l.Hv + h) * D + c0), x);
    if constexpr (MIXED) {
      if (in)
        *(uint4*)(l.buffer + l.off_v + ((vslot + i) * D + c0) * 2) =
            make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]), two_bf16(x[4], x[5]), two_bf16(x[6], x[7]));
    } else {
      const float s = quantise8<LANES>(x, false, c);
      if (in) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j / 4] |= ((uint32_t)(int)c[j] & 255u) << (8 * (j % 4));
        *(uint2*)(l.buffer + l.off_v + (vslot + i) * D + c0) = make_uint2(w[0], w[1]);
        if (c0 == 0) ((float*)(l.buffer + l.off_vs))[vslot + i] = s;
      }
    }
    if (in && c0 == 0) {
      ((float*)(l.buffer + l.off_a))[vslot + i] = l.a[tok * l.Hv + h];
      ((float*)(l.buffer + l.off_beta))[vslot + i] = l.beta[tok * l.Hv + h];
    }
  }
  __syncthreads();   // every wave has read the count
  if (tid == 0) *countp = n + take;
}

template <int D, bool BF16>
hipError_t launch(const CommitParams& p, int buf_kind, hipStream_t s) {
  const dim3 grid((unsigned)p.l.Hv, (unsigned)p.l.B);
  if (buf_kind == PACE_BUF_INT8)
    append_kernel<D, BF16, false><<<grid, kThreads, 0, s>>>(p);
  else
    append_kernel<D, BF16, true><<<grid, kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_draft_append(const CommitParams& p, int dk, int buf_kind, hipStream_t stream) {
  if (dk == 128) return p.l.io_bf16 ? launch<128, true>(p, buf_kind, stream) : launch<128, false>(p, buf_kind, stream);
  return p.l.io_bf16 ? launch<64, true>(p, buf_kind, stream) : launch<64, false>(p, buf_kind, stream);
}

}  // namespace pace
