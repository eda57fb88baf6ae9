// Verification of drafted tokens (include/pace_draft.h: pace_draft_verify).
//
// One workgroup per sequence.  The probabilities of every node's token in its parent's rows are gathered at once; one wave
// then walks the tree, 64 nodes a ballot.  With A the sum of the W's so far, what is left of a row after its refused children
// is w = max(p - A q, 0) (the same as taking W q off each time, as q >= 0), so that a row's state is two numbers.
// A row is read only where its sum is asked for: after a refusal with the draft's probabilities, and to draw the following
// token.  It is summed in chunks of 2048 tokens, one a wave; the token is found by the chunks' sums and then inside its
// chunk.  All in fp64: the fp32 (bf16) inputs are exact, and a sum of 2^24 of them is off by 2^-29 of a step of fp32.
#include <hip/hip_runtime.h>

#include "pace_draft_internal.h"
#include "pace_numerics.h"

namespace pace {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kPer = kVerifyChunk / 64;   // tokens of a chunk a lane holds, eight neighbouring ones at a time

template <typename E>
struct alignas(sizeof(E)) Eight {
  E v[8];
};

// What a probability counts: 0 for what is none.
__device__ inline double weight(float x) { return x > 0.f && x <= 3.402823466e38f ? (double)x : 0.0; }
__device__ inline double weight(uint16_t x) { return weight(bf16_to_f32(x)); }
__device__ inline double uniform(float u) { return u > 0.f ? fmin((double)u, 1.0) : 0.0; }

__device__ inline double lane_double(double x, int lane) {
  const uint64_t u = f64_bits(x);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return bits_f64((uint64_t)hi << 32 | lo);
}

// Inclusive sums over the lanes of a wave.
__device__ inline double wave_scan(double x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

struct Shared {
  double pt[kMaxNodes], qt[kMaxNodes];   // of a node's token, in its parent's rows of target and draft
  int32_t parent[kMaxNodes], token[kMaxNodes], path[kMaxNodes];
  int32_t gone[kMaxNodes];               // draft NULL: tokens of the refused children of x
  double A, W, u0;
  int32_t x, at, length, ngone;          // the node, the last child looked at, accepted nodes
  int32_t sum;                           // the walk waits for the sum of its row
};

// Goes on with the walk; returns at its end (sum = 0) or where a row's sum is needed (sum = 1).  One wave.
__device__ inline void walk(const VerifyParams& p, Shared& s, int b, int len, int lane) {
  const bool drawn = p.draft != nullptr;
  int x = s.x, at = s.at, length = s.length, ngone = s.ngone;
  double A = s.A, W = s.W;
  int sum = 0;
  for (int blk = (at + 1) / 64; blk * 64 < len && !sum; ++blk) {
    const int c = blk * 64 + lane;
    const bool in = c < len;
    const int parent = in ? s.parent[c] : -1, token = in ? s.token[c] : -1;
    const double pt = in ? s.pt[c] : 0.0, qt = in ? s.qt[c] : 0.0;
    const double u = in ? uniform(p.uniforms[(int64_t)b * p.T + c]) : 0.0;
    for (;;) {
      const uint64_t mask = __ballot(c > at && parent == x && token >= 0);
      if (!mask) break;
      const int l = __builtin_ctzll(mask);
      at = blk * 64 + l;
      const double uc = lane_double(u, l);
      const int t = __builtin_amdgcn_readlane(token, l);
      double w = lane_double(pt, l);
      bool accept;
      if (drawn) {
        const double q = lane_double(qt, l);
        w = fmax(w - A * q, 0.0);
        accept = uc * W * q < w;
      } else {
        for (int i = 0; i < ngone; i += 64)
          if (__any(i + lane < ngone && s.gone[i + lane] == t)) w = 0.0;
        accept = uc * W < w;
      }
      if (accept) {
        x = at;
        if (lane == 0) s.path[length] = at;
        ++length;
        A = 0.0;
        W = 1.0;
        ngone = 0;
      } else if (drawn) {
        A += W;
        sum = 1;
        break;
      } else {
        W = fmax(W - w, 0.0);
        if (lane == 0) s.gone[ngone] = t;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        ++ngone;
      }
    }
  }
  if (lane == 0) {
    s.x = x; s.at = at; s.length = length; s.ngone = ngone;
    s.A = A; s.W = W;
    s.sum = sum;
  }
}

// Weights of eight neighbouring tokens of row x.
template <typename E>
__device__ inline void weights(const VerifyParams& p, const Shared& s, const E* pr, const E* qr, double A, int ngone, int v0,
                               double (&w)[8]) {
  Eight<E> a, q;
  if (v0 + 8 <= p.V) {
    a = *(const Eight<E>*)(pr + v0);
    if (qr) q = *(const Eight<E>*)(qr + v0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.v[i] = v0 + i < p.V ? pr[v0 + i] : E(0);
      if (qr) q.v[i] = v0 + i < p.V ? qr[v0 + i] : E(0);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = qr ? fmax(weight(a.v[i]) - A * weight(q.v[i]), 0.0) : weight(a.v[i]);
  for (int k = 0; k < ngone; ++k) {
    const int d = s.gone[k] - v0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (d == i) w[i] = 0.0;
  }
}

template <typename E>
__device__ inline double chunk_sum(const VerifyParams& p, const Shared& s, const E* pr, const E* qr, double A, int ngone,
                                   int chunk, int lane) {
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < kPer / 8; ++j) {
    double w[8];
    weights(p, s, pr, qr, A, ngone, chunk * kVerifyChunk + j * 512 + lane * 8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += w[i];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  return sum;
}

// Sum of n values, the same in every lane.
__device__ inline double total_of(const double* sums, int n, int lane) {
  double t = 0.0;
  for (int i = lane; i < n; i += 64) t += sums[i];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) t += __shfl_xor(t, d);
  return t;
}

template <typename E>
__global__ __launch_bounds__(kThreads) void verify_kernel(VerifyParams p) {
  __shared__ Shared s;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int len = p.draft_lens ? min(max(p.draft_lens[b], 0), p.T) : p.T;
  if (len == 0) {
    for (int i = tid; i < p.T; i += kThreads) p.nodes[(int64_t)b * p.T + i] = -1;
    if (tid == 0) {
      p.counts[b] = 0;
      p.next[b] = -1;
    }
    return;
  }
  const E* const target = (const E*)p.target + (int64_t)b * p.T * p.target_stride;
  const E* const draft = p.draft ? (const E*)p.draft + (int64_t)b * p.T * p.draft_stride : nullptr;
  double* const sums = p.sums + (int64_t)b * p.chunks;
  for (int c = tid; c < len; c += kThreads) {
    const int parent = p.parents ? p.parents[b * p.parents_stride + c] : c - 1;
    const int token = p.tokens[(int64_t)b * p.T + c];
    const bool ok = parent >= 0 && parent < c && token >= 0 && token < p.V;
    s.parent[c] = ok ? parent : -1;
    s.token[c] = ok ? token : -1;
    s.pt[c] = ok ? weight(target[parent * p.target_stride + token]) : 0.0;
    s.qt[c] = ok && draft ? weight(draft[parent * p.draft_stride + token]) : 0.0;
    s.path[c] = 0;
  }
  if (tid == 0) {
    s.x = 0; s.at = 0; s.length = 1; s.ngone = 0;
    s.A = 0.0; s.W = 1.0;
    s.u0 = uniform(p.uniforms[(int64_t)b * p.T]);
  }
  __syncthreads();
  double total = 0.0;
  bool have = false;                  // the sums are those of the walk's row as it is left
  for (;;) {
    if (wave == 0) walk(p, s, b, len, lane);
    __syncthreads();
    const bool again = s.sum;
    if (again || !have || s.A == 0.0) {
      // (a row that was summed has A > 0, and the walk comes to another row with A = 0)
      const E* const pr = target + s.x * p.target_stride;
      const E* const qr = draft && s.A > 0.0 ? draft + s.x * p.draft_stride : nullptr;
      for (int i = wave; i < p.chunks; i += kWaves) {
        const double t = chunk_sum(p, s, pr, qr, s.A, s.ngone, i, lane);
        if (lane == 0) sums[i] = t;
      }
      __syncthreads();
      total = total_of(sums, p.chunks, lane);
    }
    have = true;
    if (!again) break;
    if (tid == 0) s.W = total;
    __syncthreads();
  }
  if (total == 0.0 && (s.A > 0.0 || s.ngone > 0)) {      // nothing is left: the row itself
    __syncthreads();
    if (tid == 0) {
      s.A = 0.0;
      s.ngone = 0;
    }
    __syncthreads();
    for (int i = wave; i < p.chunks; i += kWaves) {
      const double t = chunk_sum(p, s, target + s.x * p.target_stride, (const E*)nullptr, 0.0, 0, i, lane);
      if (lane == 0) sums[i] = t;
    }
    __syncthreads();
    total = total_of(sums, p.chunks, lane);
  }
  for (int i = tid; i < p.T; i += kThreads) p.nodes[(int64_t)b * p.T + i] = i < s.length ? s.path[i] : -1;
  if (tid == 0) p.counts[b] = s.length;
  if (wave != 0) return;
  if (total == 0.0) {
    if (lane == 0) p.next[b] = -1;
    return;
  }
  // the first chunk whose end passes r, or the last of any weight
  double r = s.u0 * total, before = 0.0, found = 0.0;
  int chunk = -1, last = 0;
  for (int i = 0; i < p.chunks && chunk < 0; i += 64) {
    const double t = i + lane < p.chunks ? sums[i + lane] : 0.0;
    const double upto = before + wave_scan(t, lane);
    const uint64_t over = __ballot(upto > r), any = __ballot(t > 0.0);
    if (over) {
      const int l = __builtin_ctzll(over);
      chunk = i + l;
      found = l ? lane_double(upto, l - 1) : before;
    } else {
      if (any) last = i + 63 - __builtin_clzll(any);
      before = lane_double(upto, 63);
    }
  }
  if (chunk < 0) {
    chunk = last;
    r = HUGE_VAL;
  }
  // the first token whose end passes r, or the last of any weight
  const E* const pr = target + s.x * p.target_stride;
  const E* const qr = draft && s.A > 0.0 ? draft + s.x * p.draft_stride : nullptr;
  int token = -1, tail = 0;
  before = found;
  for (int j = 0; j < kPer / 8 && token < 0; ++j) {
    const int v0 = chunk * kVerifyChunk + j * 512 + lane * 8;
    double w[8];
    weights(p, s, pr, qr, s.A, s.ngone, v0, w);
    double t = 0.0;
    int high = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t += w[i];
      if (w[i] > 0.0) high = i;
    }
    const double upto = before + wave_scan(t, lane);
    double from = __shfl_up(upto, 1);
    if (lane == 0) from = before;
    int mine = -1;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      // sums from the left
      double e = from;
#pragma unroll
      for (int k = 0; k <= i; ++k) e += w[k];
      if (e > r && w[i] > 0.0) mine = i;
    }
    const uint64_t over = __ballot(mine >= 0), any = __ballot(high >= 0);
    if (over) {
      const int l = __builtin_ctzll(over);
      token = chunk * kVerifyChunk + j * 512 + l * 8 + __builtin_amdgcn_readlane(mine, l);
    } else if (any) {
      const int l = 63 - __builtin_clzll(any);
      tail = chunk * kVerifyChunk + j * 512 + l * 8 + __builtin_amdgcn_readlane(high, l);
    }
    before = lane_double(upto, 63);
  }
  if (lane == 0) p.next[b] = token >= 0 ? token : tail;
}

}  // namespace

hipError_t launch_draft_verify(const VerifyParams& p, int prob_bf16, hipStream_t stream) {
  if (prob_bf16)
    verify_kernel<uint16_t><<<p.B, kThreads, 0, stream>>>(p);
  else
    verify_kernel<float><<<p.B, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace pace
