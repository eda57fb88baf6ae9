// Verification of drafted tokens (include/pace_draft.h: pace_draft_verify).
//
// The probabilities of every node's token in its parent's rows are gathered at once; one wave then walks the tree, 64 nodes
// a ballot.  With A the sum of the W's so far, what is left of a row after its refused children
// is w = max(p - A q, 0) (the same as taking W q off each time, as q >= 0), so that a row's state is A and W.  Where
// little is left, A q is nearly p: A is kept whole, in as many doubles as it takes, and w is as good as if W q had been taken off
// each time.
// A row is read only where its sum is asked for: after a refusal with the draft's probabilities, and to draw the following
// token.  It is summed in chunks of 2048 tokens, one a wave; the token is found by the chunks' sums and then inside its
// chunk.  All in fp64: the fp32 (bf16) inputs are exact.  A weight passes 7 additions in its lane, 6 over the lanes, one for
// every 64 chunks and 6 over those, so that a sum of 2^24 weights is off by 147 roundings of 2^-53 at most, 2^-45.8 of itself;
// with the draft's probabilities a weight is besides off by a rounding for each part of A (one up to two refusals, mostly).
//
// Bound by memory for large batches and by latency for small ones.  Measured (graph): 64 chains of 8 over 131072 tokens,
// fp32, drawn: 18.8 us, of which the sums 14.7 (4.6 TB/s; a large copy 5.1) and the rest 4.1; 16 trees of 25 over
// 100003 tokens, bf16, not drawn: 10.3 us (7.4 and 4.3 by themselves): parents -> probabilities -> walk -> row; one chain of 5 over
// 32768: 9.4 us.
//
// Few sequences over a large vocabulary: the first row that is asked for is summed by several workgroups a sequence, each
// of which walks there by itself; a second kernel goes on from there.  Otherwise one workgroup a sequence does it all.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pace_draft_internal.h"
#include "pace_numerics.h"

namespace pace {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kLdsChunks = 128;          // sums that a workgroup keeps to itself
constexpr int kPer = kVerifyChunk / 64;   // tokens of a chunk a lane holds, eight neighbouring ones at a time

template <typename E>
struct alignas(sizeof(E)) Eight {
  E v[8];
};

// What a probability counts: 0 for what is none.
__device__ inline double weight(float x) {
  const float y = fmaxf(x, 0.f);         // (of a NaN, too)
  return (double)(y <= 3.402823466e38f ? y : 0.f);
}
__device__ inline double weight(uint16_t x) { return weight(bf16_to_f32(x)); }
__device__ inline double uniform(float u) { return u > 0.f ? fmin((double)u, 1.0) : 0.0; }

__device__ inline double lane_double(double x, int lane) {
  const uint64_t u = f64_bits(x);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return bits_f64((uint64_t)hi << 32 | lo);
}

// Sums over the lanes of a wave, by lane moves on the vector unit: rows of 16 first (shifts by 1, 2, 4, 8), then the sums of
// the rows before them.
template <int CTRL, int ROWS>
__device__ inline double moved(double x) {   // 0 where nothing is moved to
  const uint64_t u = f64_bits(x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
  return bits_f64((uint64_t)hi << 32 | lo);
}
// (lane l: of lanes 0 .. l)
__device__ inline double wave_scan(double x) {
  x += moved<0x111, 0xF>(x);
  x += moved<0x112, 0xF>(x);
  x += moved<0x114, 0xF>(x);
  x += moved<0x118, 0xF>(x);
  x += moved<0x142, 0xA>(x);                  // lane 15 of a row to the next one's lanes: rows 1 and 3
  x += moved<0x143, 0xC>(x);                  // lane 31 to rows 2 and 3
  return x;
}
__device__ inline double wave_sum(double x) { return lane_double(wave_scan(x), 63); }

// The walk's state, and what of it a second kernel needs (which begins behind one refusal at most: A = 1 without a rest).
struct Walk {
  double A, W;                           // A and the parts of `rest`
  int32_t x, at, length, ngone;          // the node, the last child looked at, accepted nodes, refused ones (draft NULL)
  int32_t sum, more;                     // the row's sum is waited for; children of x are left behind `at`
  int32_t parts;                         // of `rest`
};

static_assert(sizeof(Walk) <= 48, "verify_scratch");

// Parts follow one another by 53 bits or more, down to the smallest double.
constexpr int kParts = 21;

template <int NODES>
struct Shared {
  double pt[NODES], qt[NODES], u[NODES]; // of a node's token, in its parent's rows of target and draft; its uniform
  int32_t parent[NODES], token[NODES], path[NODES];
  int32_t gone[NODES];                   // draft NULL: tokens of the refused children of x
  double rest[kParts];                   // what A has beyond its first 53 bits, the largest part first
  double part[kParts + 1];               // (at work)
  double sums[kLdsChunks];
  Walk w;
};

// A sequence's part of the workspace: chunk sums, the walk, its path, refused tokens.
struct Scratch {
  double* sums;
  Walk* w;
  int32_t *path, *gone;
};
__device__ inline Scratch scratch_of(const VerifyParams& p, int b) {
  uint8_t* const at = p.workspace + (int64_t)b * p.scratch;
  double* const sums = (double*)at;
  Walk* const w = (Walk*)(sums + p.chunks);
  int32_t* const path = (int32_t*)(w + 1);
  return {sums, w, path, path + p.T};
}

// Gathers what the walk needs of the nodes, and begins it.
template <typename E, int NODES>
__device__ inline int begin(const VerifyParams& p, Shared<NODES>& s, int b, const E* target, const E* draft) {
  const int tid = threadIdx.x;
  const int len = p.draft_lens ? min(max(p.draft_lens[b], 0), p.T) : p.T;
  for (int c = tid; c < p.T; c += blockDim.x) {
    const int parent = p.parents ? p.parents[b * p.parents_stride + c] : c - 1;
    const int token = p.tokens[(int64_t)b * p.T + c];
    const float u = p.uniforms[(int64_t)b * p.T + c];
    const bool ok = c < len && parent >= 0 && parent < c && token >= 0 && token < p.V;
    s.parent[c] = ok ? parent : -1;
    s.token[c] = ok ? token : -1;
    s.pt[c] = ok ? weight(target[parent * p.target_stride + token]) : 0.0;
    s.qt[c] = ok && draft ? weight(draft[parent * p.draft_stride + token]) : 0.0;
    s.u[c] = uniform(u);
    s.path[c] = 0;
  }
  if (tid == 0) s.w = Walk{0.0, 1.0, 0, 0, 1, 0, 0, 0, 0};
  __syncthreads();
  return len;
}

// A sum of two doubles and what its rounding loses, exactly.
__device__ inline double two_sum(double a, double b, double& lost) {
  const double s = a + b, t = s - a;
  lost = (a - (s - t)) + (b - t);
  return s;
}

// A + rest[0] + .. + rest[n - 1] gains x, and none of it is lost; the number of parts afterwards.  part: n + 1 at work.
__device__ inline int gain(double& A, double* rest, int n, double x, double* part) {
  for (int i = n - 1; i >= 0; --i) x = two_sum(rest[i], x, part[i + 1]);
  A = two_sum(A, x, part[0]);
  // each part as large as the ones behind it make it
  int k = -1;
  double top = A;
  for (int i = 0; i <= n; ++i) {
    double lost;
    const double s = two_sum(top, part[i], lost);
    if (lost != 0.0) {
      if (k < 0) A = s;
      else rest[k] = s;
      if (++k == kParts) return kParts;
      top = lost;
    } else {
      top = s;
    }
  }
  if (k < 0) A = top;
  else if (top != 0.0) rest[k++] = top;
  return max(k, 0);
}

// What the refused children leave of p.
__device__ inline double left(double p, double q, double A, const double* rest, int parts) {
  double w = fma(-A, q, p);
  for (int i = 0; i < parts; ++i) w = fma(-rest[i], q, w);
  return fmax(w, 0.0);
}

// Goes on with the walk; returns at its end (sum = 0) or where a row's sum is needed (sum = 1).  One wave.
template <int NODES>
__device__ inline void walk(Shared<NODES>& s, int len, bool drawn, int lane) {
  int x = s.w.x, at = s.w.at, length = s.w.length, ngone = s.w.ngone;
  double A = s.w.A, W = s.w.W;
  int sum = 0, more = 0, parts = s.w.parts;
  for (int blk = (at + 1) / 64; blk * 64 < len && !more; ++blk) {
    const int c = blk * 64 + lane;
    const bool in = c < len;
    const int parent = in ? s.parent[c] : -1, token = in ? s.token[c] : -1;
    const double pt = in ? s.pt[c] : 0.0, qt = in ? s.qt[c] : 0.0, u = in ? s.u[c] : 0.0;
    for (;;) {
      const uint64_t mask = __ballot(c > at && parent == x);
      if (!mask) break;
      if (sum) {                         // (a refusal waits for its row's sum: the next child needs it)
        more = 1;
        break;
      }
      const int l = __builtin_ctzll(mask);
      at = blk * 64 + l;
      const double uc = lane_double(u, l);
      const int t = __builtin_amdgcn_readlane(token, l);
      double w = lane_double(pt, l);
      bool accept;
      if (drawn) {
        const double q = lane_double(qt, l);
        w = left(w, q, A, s.rest, parts);
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
        parts = 0;
        ngone = 0;
      } else if (drawn) {
        sum = 1;                         // (the last one that this call looks at)
      } else {
        W = fmax(W - w, 0.0);
        if (lane == 0) s.gone[ngone] = t;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        ++ngone;
      }
    }
  }
  if (lane == 0) {
    if (sum) parts = gain(A, s.rest, parts, W, s.part);
    s.w = Walk{A, W, x, at, length, ngone, sum, more, parts};
  }
}

// A row of target, less what was refused of it.
template <typename E>
struct Row {
  const E *p, *q;                        // q null: nothing drawn was refused
  double A;
  const double* rest;
  int parts;
  const int32_t* gone;
  int ngone, V;
};

// Weights of eight neighbouring tokens.  What a row has decides once for a chunk, so that the loads of all its tokens may be on
// their way together.
enum { kWhole, kLess, kLessRest };         // no q; A alone; A with parts beyond it

template <int HAS, typename E>
__device__ inline void weights(const Row<E>& r, int v0, double (&w)[8]) {
  Eight<E> a, q;
  if (v0 + 8 <= r.V) {
    a = *(const Eight<E>*)(r.p + v0);
    if constexpr (HAS != kWhole) q = *(const Eight<E>*)(r.q + v0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.v[i] = v0 + i < r.V ? r.p[v0 + i] : E(0);
      if constexpr (HAS != kWhole) q.v[i] = v0 + i < r.V ? r.q[v0 + i] : E(0);
    }
  }
  double y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = weight(a.v[i]);
    if constexpr (HAS != kWhole) {         // (as `left`)
      y[i] = weight(q.v[i]);
      w[i] = fma(-r.A, y[i], w[i]);
    }
  }
  if constexpr (HAS == kLessRest)
    for (int k = 0; k < r.parts; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = fma(-r.rest[k], y[i], w[i]);
  if constexpr (HAS != kWhole)
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fmax(w[i], 0.0);
  for (int k = 0; k < r.ngone; ++k) {
    const int d = r.gone[k] - v0;
    if (__any(d >= 0 && d < 8)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (d == i) w[i] = 0.0;
    }
  }
}
template <typename E, typename F>
__device__ inline void by_row(const Row<E>& r, F f) {
  if (!r.q) f(std::integral_constant<int, kWhole>{});
  else if (!r.parts) f(std::integral_constant<int, kLess>{});
  else f(std::integral_constant<int, kLessRest>{});
}

template <typename E>
__device__ inline double chunk_sum(const Row<E>& r, int chunk, int lane) {
  double sum = 0.0;
  by_row(r, [&](auto has) {
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j) {
      double w[8];
      weights<decltype(has)::value>(r, chunk * kVerifyChunk + j * 512 + lane * 8, w);
      sum += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
    }
  });
  return wave_sum(sum);
}

// Sum of n values, the same in every lane.
__device__ inline double total_of(const double* sums, int n, int lane) {
  double t = 0.0;
  for (int i = lane; i < n; i += 64) t += sums[i];
  return wave_sum(t);
}

// The sums of a row's chunks by the waves of a workgroup, and their total.
template <typename E>
__device__ inline double row_sums(const VerifyParams& p, const Row<E>& r, double* sums) {
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < p.chunks; i += blockDim.x / 64) {
    const double t = chunk_sum(r, i, lane);
    if (lane == 0) sums[i] = t;
  }
  __syncthreads();
  return total_of(sums, p.chunks, lane);
}

// The first token whose sum from the row's start passes u total, or the last of any weight; total > 0.  All waves find the
// chunk; four of them look at a quarter of it each.  Written to *next by one thread.
template <typename E>
__device__ inline void token_at(const VerifyParams& p, const Row<E>& row, const double* sums, double u, double total, int32_t* next) {
  constexpr int PARTS = kPer / 8;
  __shared__ double part_sum[PARTS];
  __shared__ int32_t part_last[PARTS], hit[PARTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave >= PARTS && blockDim.x > 64 * PARTS) {
    __syncthreads();
    __syncthreads();
    return;
  }
  // (no sum exceeds all of the total, but one that is formed in another order may)
  double r = u < 1.0 ? u * total : HUGE_VAL, before = 0.0, found = 0.0;
  int chunk = -1, last = 0;
  for (int i = 0; i < p.chunks && chunk < 0; i += 64) {
    const double t = i + lane < p.chunks ? sums[i + lane] : 0.0;
    const double upto = before + wave_scan(t);
    // Sums up to neighbouring chunks are formed in other orders: behind a chunk without weight one may be larger than
    // before it, by a rounding.  The token lies in a chunk of some weight.
    const uint64_t any = __ballot(t > 0.0), over = __ballot(upto > r) & any;
    if (over) {
      const int l = __builtin_ctzll(over);
      chunk = i + l;
      found = l ? lane_double(upto, l - 1) : before;
    } else {
      if (any) last = i + 63 - __builtin_clzll(any);
      before = lane_double(upto, 63);
    }
  }
  if (chunk < 0) {                       // (u = 1, or a last sum that rounded below the total)
    chunk = last;
    r = HUGE_VAL;
  }
  const int v0 = chunk * kVerifyChunk + wave * 512 + lane * 8;
  double w[8];
  by_row(row, [&](auto has) { weights<decltype(has)::value>(row, v0, w); });
  double t = 0.0;
  int high = -1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t += w[i];
    if (w[i] > 0.0) high = i;
  }
  const double upto = wave_scan(t);
  if (lane == 63) part_sum[wave] = upto;
  __syncthreads();
  double e = found;                      // the sums from the left: of the parts before, of the lanes before, of the tokens
#pragma unroll
  for (int j = 0; j < PARTS; ++j)
    if (j < wave) e += part_sum[j];
  const double left = moved<0x138, 0xF>(upto);   // lane l - 1's
  e += lane ? left : 0.0;
  int mine = -1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    e += w[i];
    if (mine < 0 && e > r && w[i] > 0.0) mine = i;
  }
  const uint64_t over = __ballot(mine >= 0), any = __ballot(high >= 0);
  const int lo = over ? __builtin_ctzll(over) : 0, la = any ? 63 - __builtin_clzll(any) : 0;
  const int base = chunk * kVerifyChunk + wave * 512;
  const int hit_at = __builtin_amdgcn_readlane(mine, lo), last_at = __builtin_amdgcn_readlane(high, la);
  if (lane == 0) {
    hit[wave] = over ? base + lo * 8 + hit_at : -1;
    part_last[wave] = any ? base + la * 8 + last_at : -1;
  }
  __syncthreads();
  if (threadIdx.x > 0) return;
  int token = -1;
#pragma unroll
  for (int j = PARTS - 1; j >= 0; --j)
    if (hit[j] >= 0) token = hit[j];
#pragma unroll
  for (int j = PARTS - 1; j >= 0; --j)
    if (token < 0) token = part_last[j];
  *next = token;
}

template <typename E>
__device__ inline const E* target_of(const VerifyParams& p, int b) { return (const E*)p.target + (int64_t)b * p.T * p.target_stride; }
template <typename E>
__device__ inline const E* draft_of(const VerifyParams& p, int b) {
  return p.draft ? (const E*)p.draft + (int64_t)b * p.T * p.draft_stride : nullptr;
}
template <typename E>
__device__ inline Row<E> row_of(const VerifyParams& p, int b, const Walk& w, const double* rest, const int32_t* gone) {
  const E* const draft = draft_of<E>(p, b);
  return {target_of<E>(p, b) + w.x * p.target_stride, draft && w.A > 0.0 ? draft + w.x * p.draft_stride : nullptr, w.A, rest, w.parts,
          gone, w.ngone, p.V};
}

// The results from the walk's end.  total: of the row as it is left, chunk by chunk in sums.
template <typename E>
__device__ inline void finish(const VerifyParams& p, int b, const Walk& w, const int32_t* path, Row<E> row, double* sums, double total) {
  const int tid = threadIdx.x;
  for (int i = tid; i < p.T; i += blockDim.x) p.nodes[(int64_t)b * p.T + i] = i < w.length ? path[i] : -1;
  if (tid == 0) p.counts[b] = w.length;
  if (total == 0.0 && (row.q || row.ngone > 0)) {      // nothing is left: the row itself
    row.q = nullptr;
    row.ngone = 0;
    __syncthreads();
    total = row_sums(p, row, sums);
  }
  if (total > 0.0)
    token_at(p, row, sums, uniform(p.uniforms[(int64_t)b * p.T]), total, p.next + b);
  else if (tid == 0)
    p.next[b] = -1;
}

// The walk from where it stands to its end, and the results.  One workgroup.  total: of the row that the walk waits for.
template <typename E, int NODES>
__device__ inline void go_on(const VerifyParams& p, Shared<NODES>& s, int b, int len, double* sums, double total) {
  const int tid = threadIdx.x;
  for (;;) {
    // (the walk stops for the sum of a row of which A > 0, and ends there or at a row of which A = 0)
    const bool waited = s.w.sum;
    __syncthreads();
    if (waited && !s.w.more) break;
    if (tid == 0 && waited) s.w.W = total;
    __syncthreads();
    if (tid < 64) walk(s, len, p.draft != nullptr, tid);
    __syncthreads();
    total = row_sums(p, row_of<E>(p, b, s.w, s.rest, s.gone), sums);
    if (!s.w.sum) break;
  }
  finish(p, b, s.w, s.path, row_of<E>(p, b, s.w, s.rest, s.gone), sums, total);
}

// A sequence without drafts.
__device__ inline void nothing(const VerifyParams& p, int b) {
  for (int i = threadIdx.x; i < p.T; i += blockDim.x) p.nodes[(int64_t)b * p.T + i] = -1;
  if (threadIdx.x == 0) {
    p.counts[b] = 0;
    p.next[b] = -1;
  }
}

template <typename E, int NODES>
__global__ __launch_bounds__(kThreads) void verify_kernel(VerifyParams p) {
  __shared__ Shared<NODES> s;
  const int b = blockIdx.x;
  const int len = begin(p, s, b, target_of<E>(p, b), draft_of<E>(p, b));
  if (len == 0) return nothing(p, b);
  go_on<E>(p, s, b, len, p.chunks <= kLdsChunks ? s.sums : scratch_of(p, b).sums, 0.0);
}

// In two kernels: the walk to the first row that is summed, and that row's sums ...
constexpr int kSumThreads = 256;

template <typename E, int NODES>
__global__ __launch_bounds__(kSumThreads) void sums_kernel(VerifyParams p) {
  __shared__ Shared<NODES> s;
  const int b = blockIdx.y, tid = threadIdx.x;
  const int len = begin(p, s, b, target_of<E>(p, b), draft_of<E>(p, b));
  if (len == 0) return;
  if (tid < 64) walk(s, len, p.draft != nullptr, tid);
  __syncthreads();
  const Scratch to = scratch_of(p, b);
  Row<E> row = row_of<E>(p, b, s.w, s.rest, s.gone);
  row.parts = 0;                         // (one refusal: A is 1)
  const int waves = gridDim.x * (kSumThreads / 64);
  for (int i = blockIdx.x * (kSumThreads / 64) + tid / 64; i < p.chunks; i += waves) {
    const double t = chunk_sum(row, i, tid & 63);
    if ((tid & 63) == 0) to.sums[i] = t;
  }
  if (blockIdx.x > 0) return;
  for (int i = tid; i < s.w.length; i += kSumThreads) to.path[i] = s.path[i];
  for (int i = tid; i < s.w.ngone; i += kSumThreads) to.gone[i] = s.gone[i];
  if (tid == 0) *to.w = s.w;
}

// ... and the results, or the rest of the walk where more than one row is summed.
template <typename E, int NODES>
__global__ __launch_bounds__(kThreads) void finish_kernel(VerifyParams p) {
  __shared__ Shared<NODES> s;
  const int b = blockIdx.x, tid = threadIdx.x;
  const Scratch from = scratch_of(p, b);
  const Walk w = *from.w;                // (of a sequence without drafts: whatever lay there, not used)
  if (p.draft_lens && p.draft_lens[b] <= 0) return nothing(p, b);
  const double total = total_of(from.sums, p.chunks, tid & 63);
  if (!w.more) {
    Row<E> row = row_of<E>(p, b, w, nullptr, from.gone);
    row.parts = 0;                       // (one refusal: A is 1)
    finish(p, b, w, from.path, row, from.sums, total);
    return;
  }
  const int len = begin(p, s, b, target_of<E>(p, b), draft_of<E>(p, b));
  for (int i = tid; i < w.length; i += kThreads) s.path[i] = from.path[i];
  if (tid == 0) s.w = w;
  __syncthreads();
  go_on<E>(p, s, b, len, from.sums, total);
}

template <typename E, int NODES>
void launch(const VerifyParams& p, hipStream_t s) {
  // Two kernels where one workgroup a sequence leaves much of the chip idle for long: few sequences, rows of more than a chunk a
  // wave.  Chains of 8, drawn, fp32, in one kernel and in two: V = 131072: 1 sequence 21.5 and 8.1 us, 64 28.3 and 18.8, 128
  // 35.3 and 31.5, 192 45.0 and 47.8; V = 65536: 16 14.5 and 10.4, 256 28.3 and 30.7; V = 32768: 32 10.2 and 10.4, 128 12.6 and
  // 14.3.  One chain of 5 over 32768: 9.4 and 8.0 in a graph, 9.8 and 11.1 to 12.9 called eagerly: a second launch costs an eager
  // call as much as it saves a captured one, or more, and from few sequences on it saves nothing there.
  if (p.chunks <= kWaves || p.B > std::min(2 * p.chunks, 128)) {
    verify_kernel<E, NODES><<<p.B, kThreads, 0, s>>>(p);
    return;
  }
  // (about four workgroups a compute unit read the rows)
  const int slices = std::min(1024 / p.B, (p.chunks + kSumThreads / 64 - 1) / (kSumThreads / 64));
  sums_kernel<E, NODES><<<dim3((unsigned)slices, (unsigned)p.B), kSumThreads, 0, s>>>(p);
  finish_kernel<E, NODES><<<p.B, kThreads, 0, s>>>(p);
}

}  // namespace

hipError_t launch_draft_verify(const VerifyParams& p, int prob_bf16, hipStream_t stream) {
  // (LDS for 64 nodes or for 1024: 64 chains of 8 over 131072 tokens 18.8 us, with the larger 22.2)
  if (p.T <= 64) {
    if (prob_bf16) launch<uint16_t, 64>(p, stream);
    else launch<float, 64>(p, stream);
  } else {
    if (prob_bf16) launch<uint16_t, kMaxNodes>(p, stream);
    else launch<float, kMaxNodes>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace pace
