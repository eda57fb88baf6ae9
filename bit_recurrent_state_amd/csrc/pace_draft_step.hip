// Gated-delta outputs of drafted tokens (include/pace_draft.h: pace_draft_step) -- gfx950, wave64.
//
// One workgroup of two or four waves per (sequence, value head) tile; nothing is written but o.  With S_0 the dequantised state and
// tokens 0 .. N-1 the n buffered ones and then the drafts, D_ij the product of the decays behind token j up to i along
// the path of i, and Gamma_i the product of all of them (from S_0 on),
//     u_i = beta_i (v_i - Gamma_i S_0^T k_i - sum_{j before i} D_ij (k_j . k_i) u_j)
//     o_i = Gamma_i S_0^T q_i + sum_{j before i, or i} D_ij (k_j . q_i) u_j,
// so the state of no node is ever formed: the tile's codes are read once, for all tokens.
//
//   tokens       buffered codes and quantised drafts as bf16 (exact) in LDS, in the order of the state's units
//   Gram         k_j . k_i and k_j . q_i on the bf16 matrix cores, times the decays: products along i's path, from its end back
//   projections  tokens (A) times state columns (B), 32 keys an instruction.  A 4-bit code c becomes the bf16 number 16 + c by
//                a shift and a mask-and-or of two codes; the offset and the zero point are taken off by the tokens' block
//                sums.  In fp32 codes enter less their zero points: an offset is rounded at its own size, which
//                outputs in bf16 do not show, but 64 chains of 8 were off by 4.5e-7 of their norm in fp32, now 1.5e-7, in
//                the same 21.1 us.  One scale a (column, 32 keys).
//   solve        16 tokens at a time in the matrix unit's layout (4 tokens x 4 columns a lane), four at a time within them
// Queries enter as they are in bf16, as three bf16 pieces (exact) in fp32.  Everything else is fp32.
//
// Measured (graph), 32/16 heads of 128, int4 state: 64 chains of up to 8 14.0 us, 2.1 TB/s (a large copy: 5.1).  All 2048
// workgroups are on the chip at once: their loads take 6 us together, so that the last quarter waits for its tokens, and
// then takes the 6 us of a workgroup; vector unit and LDS are busy half of the time each, the matrix unit 23%, waves wait for
// their turn 44% of theirs.  16 trees of up to 25 (mixed heads and buffer): 13.3 us, two workgroups a compute unit, vector
// unit 42%: latency of one tile after another.  One sequence's five tokens: 5.6 us, a workgroup's chain of loads, tokens,
// Gram, projections, solve, outputs 4.6 of them.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "pace_draft_internal.h"
#include "pace_draft_tokens.h"
#include "pace_lanes.h"

namespace pace {
namespace {

// Waves of a workgroup: two where one tile holds all tokens (eight such workgroups a compute unit), four beyond it
// (LDS leaves four, or fewer).  32/16 heads of 128, in a graph, in two waves and in four: 64 chains of 8 14.0 and 15.8 us, 32 9.6
// and 10.0, 16 7.5 and 6.6, one sequence's five 5.6 and 5.0; 16 trees of 25 16.9 and 13.4.  (Four for one tile of few
// sequences would be one more kernel of each kind for those 10%.)  At d = 64 each of four waves would have one strip of
// columns, and strips are taken in pairs.
template <int D, int NKT>
constexpr int waves_of() {
  return NKT == 1 || D == 64 ? 2 : 4;
}

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ inline v4f mfma(v8bf a, v8bf b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

__device__ inline v8bf as_operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 w = make_uint4(a, b, c, d);
  return __builtin_bit_cast(v8bf, w);
}

// NKT: 16-token tiles of the buffered and drafted tokens.  PIECES: of a query.  KPS: 32-key blocks that share a scale.
template <int D, int NKT, int PIECES, int KPS>
struct alignas(16) Smem {
  static constexpr int NK = 16 * NKT;
  static constexpr int TS = D + 8;              // row stride of tokens (bf16): 16 rows on distinct banks
  alignas(16) uint16_t k[NK][TS];               // key codes
  alignas(16) uint16_t q[16 * PIECES][TS];      // queries of one tile of tokens
  alignas(16) float u[NK][D];                   // v^, then u
  struct Gram {                                 // of one tile of tokens i and those before them
    alignas(16) float a[NK][16];                // [j][i]: beta_i D_ij (k_j . k_i), 0 for j >= i
    alignas(16) float c[NK][16];                // [j][i]: D_ij (k_j . q_i)
  };
  struct Scales {                               // of (32 keys, or 64, column), bf16
    alignas(16) uint16_t s[D / 32 / KPS][D];
    alignas(16) uint16_t z[D / 32 / KPS][D];    // minus what the operand's codes are too large by
  };
  // The Gram products are formed first, while the state is on its way.  With one tile and 32-key blocks that would leave
  // room for seven workgroups a compute unit at D = 128, not eight: there the tile is projected first, and both use one place.
  static constexpr bool kGramFirst = NKT > 1 || KPS > 1;
  struct Both {
    Gram g;
    Scales s;
  };
  union Either {
    Gram g;
    Scales s;
  };
  alignas(16) std::conditional_t<kGramFirst, Both, Either> m;
  alignas(16) float ks[NK], decay[NK], beta[NK], gamma[16];
  uint64_t row[NK < kMaxDrafts ? NK : kMaxDrafts];   // tree bits
};

// The wave's own LDS accesses in order.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Eight token elements in the order of the state operand, as four words: packed states keep the order in
// which nibbles come out of a unit, bf16 states the natural one.
template <bool BFS>
__device__ inline uint4 in_order(const float (&x)[8]) {
  if constexpr (BFS) return make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]), two_bf16(x[4], x[5]), two_bf16(x[6], x[7]));
  return make_uint4(two_bf16(x[0], x[2]), two_bf16(x[1], x[3]), two_bf16(x[4], x[6]), two_bf16(x[5], x[7]));
}

// HB: 4 = every head 4-bit, 0 = by the head map.  KPS: 32-key blocks that are sure to share a scale (group / 32, or 1).
template <int D, int NKT, bool BF16, bool MIXED, int HB, int KPS, bool BFS>
__global__ __launch_bounds__((64 * waves_of<D, NKT>())) __attribute__((amdgpu_waves_per_eu(BF16 && !BFS ? 4 : 1)))
void step_kernel(DraftParams p) {
  constexpr int kWaves = waves_of<D, NKT>(), kThreads = 64 * kWaves;
  constexpr int PIECES = BF16 ? 1 : 3;
  using SM = Smem<D, NKT, PIECES, KPS>;
  constexpr int KB = D / 32;                   // matrix instructions along the keys
  constexpr int SPW = D / 16 / kWaves;         // 16-column strips a wave
  constexpr int CW = D / kWaves;               // columns a wave
  constexpr int LANES = D / 8, ROWS = kThreads / LANES, PASS = 16 / ROWS;   // passes over 16 tokens
  __shared__ SM sm;
  const DecodeParams& l = p.l;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, qq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.y;
  // the value heads of one key head on one XCD, as in the decode
  int h = blockIdx.x;
  if (l.gamma > 1 && (l.gamma & (l.gamma - 1)) == 0 && l.Hv % (8 * l.gamma) == 0) {
    const int lg = __builtin_ctz(l.gamma);
    const int r = h & (8 * l.gamma - 1);
    h = ((((h >> (3 + lg)) << 3) + (r & 7)) << lg) | (r >> 3);
  }
  const int kh = h / l.gamma, T = p.T;
  const size_t bh = (size_t)b * l.Hv + h, tok0 = (size_t)b * T;
  // Every load up to the barrier is unconditional with an in-bounds index, so that all are on their way
  // before the first is waited for.
  const int count = ((const int32_t*)l.buffer)[bh];
  const int len_raw = p.draft_lens ? p.draft_lens[b] : T;

  // ------------------------------------------------- 16 tokens at a time, 8 channels a lane
  const int e0 = 8 * (tid % LANES), row0 = tid / LANES;
  struct Slots {                               // buffered
    uint32_t k[PASS][2], v[PASS][MIXED ? 4 : 2];
    float ks[PASS], vs[PASS], a[PASS], beta[PASS];
  };
  // (bases are the workgroup's: scalar registers; lanes add 32 bits)
  const size_t kslot0 = ((size_t)b * l.Hk + kh) * l.dP, vslot0 = bh * l.dP;
  const uint8_t* const buf_k = l.buffer + l.off_kc + kslot0 * (MIXED ? D / 2 : D);
  const uint8_t* const buf_v = l.buffer + l.off_v + vslot0 * (MIXED ? 2 * D : D);
  const float* const buf_ks = (const float*)(l.buffer + l.off_ks) + kslot0;
  const float* const buf_vs = (const float*)(l.buffer + l.off_vs) + vslot0;
  const float* const buf_a = (const float*)(l.buffer + l.off_a) + vslot0;
  const float* const buf_beta = (const float*)(l.buffer + l.off_beta) + vslot0;
  auto load_slots = [&](int g, Slots& s) {
#pragma unroll
    for (int e = 0; e < PASS; ++e) {
      if (16 * g + ROWS * e >= l.dP - 1) continue;       // (at most dP - 1 are held)
      const uint32_t i = min(16 * g + ROWS * e + row0, l.dP - 1);
      if constexpr (MIXED) {
        s.k[e][0] = *(const uint32_t*)(buf_k + (i * (D / 2) + e0 / 2));
        const uint4 w = *(const uint4*)(buf_v + (i * D + e0) * 2);
        s.v[e][0] = w.x; s.v[e][1] = w.y; s.v[e][2] = w.z; s.v[e][3] = w.w;
      } else {
        const uint2 w = *(const uint2*)(buf_k + (i * D + e0)), x = *(const uint2*)(buf_v + (i * D + e0));
        s.k[e][0] = w.x; s.k[e][1] = w.y;
        s.v[e][0] = x.x; s.v[e][1] = x.y;
        s.vs[e] = buf_vs[i];
      }
      s.ks[e] = buf_ks[i];
      s.a[e] = buf_a[i];
      s.beta[e] = buf_beta[i];
    }
  };
  struct Drafts {
    Raw8<BF16> k[PASS], v[PASS];
    float a[PASS], beta[PASS];
  };
  constexpr int E = BF16 ? 2 : 4;
  const uint8_t* const in_k = (const uint8_t*)l.k + (tok0 * l.Hk + kh) * D * E;
  const uint8_t* const in_q = (const uint8_t*)l.q + (tok0 * l.Hk + kh) * D * E;
  const uint8_t* const in_v = (const uint8_t*)l.v + (tok0 * l.Hv + h) * D * E;
  const float* const in_a = l.a + tok0 * l.Hv + h;
  const float* const in_beta = l.beta + tok0 * l.Hv + h;
  const uint32_t next_k = (uint32_t)l.Hk * D * E, next_v = (uint32_t)l.Hv * D * E;   // (of a token; T of them: under 2^22)
  auto load_drafts = [&](int g, Drafts& s) {
#pragma unroll
    for (int e = 0; e < PASS; ++e) {
      if (16 * g + ROWS * e >= T) continue;
      const uint32_t t = min(16 * g + ROWS * e + row0, T - 1);
      s.k[e].load(in_k + (t * next_k + e0 * E));
      s.v[e].load(in_v + (t * next_v + e0 * E));
      s.a[e] = in_a[t * (uint32_t)l.Hv];
      s.beta[e] = in_beta[t * (uint32_t)l.Hv];
    }
  };
  // (queries of drafts first + 0 .. 15)
  auto load_queries = [&](int first, Raw8<BF16> (&x)[PASS]) {
#pragma unroll
    for (int e = 0; e < PASS; ++e) {
      if (first + ROWS * e >= T) continue;
      x[e].load(in_q + ((uint32_t)min(max(first + ROWS * e + row0, 0), T - 1) * next_k + e0 * E));
    }
  };
  Slots slots;
  load_slots(0, slots);
  Drafts drafts, more;
  load_drafts(0, drafts);
  if constexpr (NKT > 1) load_drafts(1, more);
  Raw8<BF16> queries[PASS];
  if constexpr (NKT == 1) load_queries(0, queries);
  const int words = (T + 31) / 32;
  const uint32_t* const bits_at = p.tree ? p.tree + b * p.tree_stride + min(tid, T - 1) * words : (const uint32_t*)l.buffer;
  const uint32_t bits_lo = bits_at[0], bits_hi = bits_at[words - 1];   // (a chain: whatever the buffer begins with, not used)

  // ------------------------------------------------------------------ state
  const bool is8 = HB != 4 && !BFS && ((l.mask8 >> h) & 1ull) != 0, asym = l.asym != 0;
  const int bits = BFS ? 16 : is8 ? 8 : 4;
  const uint64_t below = HB != 4 && h ? (l.mask8 & ((1ull << h) - 1ull)) : 0ull;
  const uint8_t* rec = l.state + (uint64_t)b * l.seq_stride + (uint64_t)h * l.rec4 + (uint64_t)__popcll(below) * (l.rec8 - l.rec4);
  // a thread's column of scales and zero points (groups of 32 keys, or 64); ahead of the
  // state, as they are waited for with the tokens
  const int wide = l.group == 64;
  uint16_t column_s[KB / KPS];
  uint8_t column_z[KB / KPS];
  const int column = min(tid, D - 1);
  if constexpr (!BFS) {
    const int NG = KPS > 1 ? KB / KPS : KB >> wide;
    const uint16_t* scales = (const uint16_t*)(rec + (is8 ? l.scales_off8 : l.scales_off4));
    const uint8_t* zeros = rec + (is8 ? l.zeros_off8 : l.zeros_off4);
#pragma unroll
    for (int kb = 0; kb < KB / KPS; ++kb) {
      const int i = column * NG + (KPS > 1 ? kb : kb >> wide);
      column_s[kb] = scales[i];
      if (asym) column_z[kb] = zeros[is8 ? i : i >> 1];
    }
  }
  // a lane's columns: c0 .. c0 + SPW - 1, one a strip; their codes of keys 8 qq .. + 7 of every 32 (one unit each)
  const int c0 = wave * CW + SPW * l16;
  constexpr int AW = BFS ? 4 * KB : HB == 4 ? KB : 2 * KB;
  uint32_t raw[SPW][AW];
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const uint8_t* col = rec + (uint32_t)((c0 + s) * (D * bits / 8));
    if constexpr (BFS) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const uint4 v = *(const uint4*)(col + 2 * (32 * kb + 8 * qq));
        raw[s][4 * kb] = v.x; raw[s][4 * kb + 1] = v.y; raw[s][4 * kb + 2] = v.z; raw[s][4 * kb + 3] = v.w;
      }
    } else if (is8) {
      if constexpr (HB != 4) {
#pragma unroll
        for (int kb = 0; kb < KB; kb += 2) {
          const uint4 v = *(const uint4*)(col + 8 * (qq * KB + kb));
          raw[s][2 * kb] = v.x; raw[s][2 * kb + 1] = v.y; raw[s][2 * kb + 2] = v.z; raw[s][2 * kb + 3] = v.w;
        }
      }
    } else if constexpr (KB == 4) {
      const uint4 v = *(const uint4*)(col + 16 * qq);
      raw[s][0] = v.x; raw[s][1] = v.y; raw[s][2] = v.z; raw[s][3] = v.w;
    } else {
      const uint2 v = *(const uint2*)(col + 8 * qq);
      raw[s][0] = v.x; raw[s][1] = v.y;
    }
  }
  // ----------------------------------------------------------------- tokens
  const int len = __builtin_amdgcn_readfirstlane(min(max(len_raw, 0), T));
  const int n = __builtin_amdgcn_readfirstlane(min(max(count, 0), l.dP - 1)), N = n + len;
  const int NT = (N + 15) / 16, NR = 16 * NT;        // tiles and rows in use
  uint8_t* const out = (uint8_t*)l.o + (tok0 * l.Hv + h) * D * E;
  auto store_rows = [&](int t, const float (&x)[SPW]) {
    uint8_t* const at = out + ((uint32_t)t * next_v + c0 * E);
    if constexpr (BF16) {
      uint32_t w[SPW / 2];
#pragma unroll
      for (int s = 0; s < SPW / 2; ++s) w[s] = two_bf16(x[2 * s], x[2 * s + 1]);
      if constexpr (SPW == 4) *(uint2*)at = make_uint2(w[0], w[1]);
      else *(uint32_t*)at = w[0];
    } else {
      if constexpr (SPW == 4) *(float4*)at = make_float4(x[0], x[1], x[2], x[3]);
      else *(float2*)at = make_float2(x[0], x[1]);
    }
  };
  if (len < T) {
    const float none[SPW] = {};
    for (int t = len + qq; t < T; t += 4) store_rows(t, none);
    if (len == 0) return;
  }
  auto put = [&](int i, const float (&kx)[8], const float (&vx)[8], float ks, float a, float beta) {
    *(uint4*)&sm.k[i][e0] = in_order<BFS>(kx);
    *(float4*)&sm.u[i][e0] = make_float4(vx[0], vx[1], vx[2], vx[3]);
    *(float4*)&sm.u[i][e0 + 4] = make_float4(vx[4], vx[5], vx[6], vx[7]);
    if (e0 == 0) {
      sm.ks[i] = ks;
      sm.decay[i] = a;
      sm.beta[i] = beta;
    }
  };
  auto take_slots = [&](int g, const Slots& s) {
#pragma unroll
    for (int e = 0; e < PASS; ++e) {
      const int i = 16 * g + ROWS * e + row0;
      if (16 * g + ROWS * e >= n) continue;              // (of the workgroup: nothing is computed for nobody)
      float kx[8], vx[8];
      if constexpr (MIXED) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          kx[j] = (float)((int)((s.k[e][0] >> (8 * j)) & 15u) - 8);
          kx[4 + j] = (float)((int)((s.k[e][0] >> (8 * j + 4)) & 15u) - 8);
          vx[2 * j] = bits_f32(s.v[e][j] << 16);
          vx[2 * j + 1] = bits_f32(s.v[e][j] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          kx[j] = (float)(int8_t)(s.k[e][j / 4] >> (8 * (j & 3)));
          vx[j] = (float)(int8_t)(s.v[e][j / 4] >> (8 * (j & 3))) * s.vs[e];
        }
      }
      if (i < n) put(i, kx, vx, s.ks[e], s.a[e], s.beta[e]);
    }
  };
  auto take_drafts = [&](int g, const Drafts& s) {
#pragma unroll
    for (int e = 0; e < PASS; ++e) {
      const int t = 16 * g + ROWS * e + row0;
      if (16 * g + ROWS * e >= len) continue;
      float x[8], kx[8], vx[8];
      s.k[e].values(x);
      const float ks = quantise8<LANES>(x, MIXED, kx);
      s.v[e].values(x);
      if constexpr (MIXED) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t w = two_bf16(x[j], x[j + 1]);
          vx[j] = bits_f32(w << 16);
          vx[j + 1] = bits_f32(w & 0xFFFF0000u);
        }
      } else {
        const float vs = quantise8<LANES>(x, false, vx);
#pragma unroll
        for (int j = 0; j < 8; ++j) vx[j] *= vs;
      }
      if (t < len) put(n + t, kx, vx, ks, s.a[e], s.beta[e]);
    }
  };
  // of drafts first + 0 .. 15 into rows row + 0 .. 15 of the tile, as far as they are in it
  auto take_queries = [&](int first, int row, const Raw8<BF16> (&in)[PASS]) {
#pragma unroll
    for (int e = 0; e < PASS; ++e) {
      const int i = row + ROWS * e + row0;
      if (first + ROWS * e >= len) continue;
      if (i < 0 || i >= 16) continue;
      if constexpr (BF16) {                    // (exact as they are)
        const uint32_t* const w = in[e].w;
        uint4 y = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (!BFS) {
          y.x = __builtin_amdgcn_perm(w[1], w[0], 0x05040100u);
          y.y = __builtin_amdgcn_perm(w[1], w[0], 0x07060302u);
          y.z = __builtin_amdgcn_perm(w[3], w[2], 0x05040100u);
          y.w = __builtin_amdgcn_perm(w[3], w[2], 0x07060302u);
        }
        *(uint4*)&sm.q[i][e0] = y;
        continue;
      }
      float x[8];
      in[e].values(x);
#pragma unroll
      for (int c = 0; c < PIECES; ++c) {
        *(uint4*)&sm.q[16 * c + i][e0] = in_order<BFS>(x);
        if (c + 1 < PIECES) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const uint32_t w = two_bf16(x[j], x[j + 1]);
            x[j] -= bits_f32(w << 16);
            x[j + 1] -= bits_f32(w & 0xFFFF0000u);
          }
        }
      }
    }
  };
  take_slots(0, slots);
  take_drafts(0, drafts);
  if constexpr (NKT == 1) {
    take_queries(0, n, queries);                          // (every token is in the one tile)
  } else {
    load_queries(-n, queries);
    take_drafts(1, more);
    take_queries(-n, 0, queries);
    load_queries(16 - n, queries);                     // (the next tile's)
    for (int g = 1; 16 * g < n; ++g) {
      load_slots(g, slots);
      take_slots(g, slots);
    }
    for (int g = 2; 16 * g < len; ++g) {
      load_drafts(g, drafts);
      take_drafts(g, drafts);
    }
  }
  for (int i = N + row0; i < NR; i += ROWS) {        // rows behind the last token hold zeros
    *(uint4*)&sm.k[i][e0] = make_uint4(0, 0, 0, 0);
    *(float4*)&sm.u[i][e0] = make_float4(0.f, 0.f, 0.f, 0.f);
    *(float4*)&sm.u[i][e0 + 4] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e0 == 0) sm.ks[i] = sm.decay[i] = sm.beta[i] = 0.f;
  }
  if (tid < len) sm.row[tid] = p.tree ? bits_lo | (words > 1 ? (uint64_t)bits_hi << 32 : 0ull) : ~0ull;
  if constexpr (!BFS) {
    if (tid < D) {
#pragma unroll
      for (int kb = 0; kb < KB / KPS; ++kb) {
        sm.m.s.s[kb][tid] = column_s[kb];
        const int odd = (KPS > 1 ? tid * (KB / KPS) + kb : tid * (KB >> wide) + (kb >> wide)) & 1;   // (4 bits: two zero points a byte)
        const int zp = is8 ? column_z[kb] : (column_z[kb] >> (4 * odd)) & 15;
        const float z = asym ? (float)zp : (float)(1 << (bits - 1));
        sm.m.s.z[kb][tid] = (uint16_t)two_bf16(-((!BF16 || is8 ? 0.f : 16.f) + z), 0.f);
      }
    }
  }
  __syncthreads();

  auto operand = [&](const uint16_t* row) { return *(const v8bf*)(row + 8 * qq); };
  // Projections of a tile's keys and queries on the wave's columns: [s] of strip s, tokens 4 qq + r.  What the operand's codes
  // are too large by comes first (in fp32 nothing): sums of the tokens' 32-key blocks (A) times offset and scale of the columns'
  // blocks (B), one fp32 product a strip.  Then turns of 32 keys and two strips, a turn's sums scaled while the next one's products are
  // formed; all at once, the operands and sums are some 100 registers more.
  auto project = [&](auto eight_bits, const uint16_t* rows, v4f (&xk)[SPW], v4f (&xq)[SPW]) {
    constexpr bool E8 = decltype(eight_bits)::value;
    constexpr int PAIRS = SPW / 2;
    constexpr v4f none = {0.f, 0.f, 0.f, 0.f};
    v8bf tk[2], tq[2][PIECES];                 // of 32 keys, the next ones ahead
    auto fetch = [&](int kb) {
      int own = l16;                           // (not earlier than its turn)
      asm volatile("" : "+v"(own));
      tk[kb & 1] = operand(rows + (size_t)own * SM::TS + 32 * kb);
#pragma unroll
      for (int e = 0; e < PIECES; ++e) tq[kb & 1][e] = operand(&sm.q[16 * e + own][32 * kb]);
    };
    auto queries_times = [&](int kb, v8bf x, v4f acc) {
#pragma unroll
      for (int e = 0; e < PIECES; ++e) acc = mfma(tq[kb & 1][e], x, acc);
      return acc;
    };
    if constexpr (BFS) {
#pragma unroll
      for (int s = 0; s < SPW; ++s) xk[s] = xq[s] = none;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        fetch(kb);
#pragma unroll
        for (int s = 0; s < SPW; ++s) {
          const v8bf st = as_operand(raw[s][4 * kb], raw[s][4 * kb + 1], raw[s][4 * kb + 2], raw[s][4 * kb + 3]);
          xk[s] = mfma(tk[kb & 1], st, xk[s]);
          xq[s] = queries_times(kb, st, xq[s]);
        }
      }
      return;
    }
    if constexpr (!BF16) {
#pragma unroll
      for (int s = 0; s < SPW; ++s) xk[s] = xq[s] = none;
    } else {
      constexpr uint32_t one = 0x3F803F80u;
      const v8bf ones = as_operand(one, one, one, one);
      float sum_k = 0.f, sum_q = 0.f;          // of token l16's block qq
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        fetch(kb);
        const float k = mfma(ones, tk[kb & 1], none)[0];
        v4f acc = none;
#pragma unroll
        for (int e = 0; e < PIECES; ++e) acc = mfma(ones, tq[kb & 1][e], acc);
        sum_k = qq == kb ? k : sum_k;
        sum_q = qq == kb ? acc[0] : sum_q;
      }
      const int kb = (KB == 4 ? qq : qq & 1) / KPS;      // (two blocks: the sums of the others are zeros)
#pragma unroll
      for (int s = 0; s < SPW; s += 2) {
        const uint32_t sc = *(const uint32_t*)&sm.m.s.s[kb][c0 + s], zp = *(const uint32_t*)&sm.m.s.z[kb][c0 + s];
        const float f0 = bits_f32(sc << 16) * bits_f32(zp << 16), f1 = bits_f32(sc & 0xFFFF0000u) * bits_f32(zp & 0xFFFF0000u);
        xk[s] = __builtin_amdgcn_mfma_f32_16x16x4f32(sum_k, f0, none, 0, 0, 0);
        xq[s] = __builtin_amdgcn_mfma_f32_16x16x4f32(sum_q, f0, none, 0, 0, 0);
        xk[s + 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(sum_k, f1, none, 0, 0, 0);
        xq[s + 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(sum_q, f1, none, 0, 0, 0);
      }
    }
    v4f ak[2][2], aq[2][2];                    // [turn][strip of the pair]
    uint32_t sc[2], zp = 0u;
    auto add = [&](int turn) {
      const int s0 = 2 * (turn % PAIRS);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const float scale = bits_f32(s ? sc[turn & 1] & 0xFFFF0000u : sc[turn & 1] << 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          xk[s0 + s][r] = fmaf(scale, ak[turn & 1][s][r], xk[s0 + s][r]);
          xq[s0 + s][r] = fmaf(scale, aq[turn & 1][s][r], xq[s0 + s][r]);
        }
        asm volatile("" : "+v"(xk[s0 + s]), "+v"(xq[s0 + s]));
      }
    };
    // (a mask in a vector register and a constant in a scalar one: one operation for both)
    uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
    asm volatile("" : "+v"(mask), "+s"(sixteen));
    constexpr int TURNS = PAIRS * KB / KPS;
    if constexpr (KPS == 1) fetch(0);
#pragma unroll
    for (int turn = 0; turn < TURNS; ++turn) {
      const int kb0 = turn / PAIRS * KPS, s0 = 2 * (turn % PAIRS);
      if (s0 == 0) {
        if constexpr (KPS == 1) {
          if (kb0 + 1 < KB) fetch(kb0 + 1);
        } else {
          fetch(kb0);
          fetch(kb0 + 1);
        }
      }
#pragma unroll
      for (int s = s0; s < s0 + 2; ++s)
#pragma unroll
        for (int i = 0; i < (E8 ? 2 : 1) * KPS; ++i) asm volatile("" : "+v"(raw[s][E8 ? 2 * kb0 + i : kb0 + i]));
      sc[turn & 1] = *(const uint32_t*)&sm.m.s.s[kb0 / KPS][c0 + s0];
      if constexpr (!BF16) zp = *(const uint32_t*)&sm.m.s.z[kb0][c0 + s0];
#pragma unroll
      for (int kb = kb0; kb < kb0 + KPS; ++kb)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          v8bf st;
          if constexpr (!BF16) {
            const float z = bits_f32(s ? zp & 0xFFFF0000u : zp << 16);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t y = E8 ? raw[s0 + s][2 * kb + e] : (raw[s0 + s][kb] >> (4 * e)) & 0x0F0F0F0Fu;
              asm volatile("" : "+v"(y));      // (bytes from here on: one operation takes and converts one)
              w[2 * e] = two_bf16((float)(y & 255u) + z, (float)((y >> 16) & 255u) + z);
              w[2 * e + 1] = two_bf16((float)((y >> 8) & 255u) + z, (float)(y >> 24) + z);
            }
            st = as_operand(w[0], w[1], w[2], w[3]);
          } else if constexpr (E8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t y = raw[s0 + s][2 * kb + e];
              w[2 * e] = two_bf16((float)(y & 255u), (float)((y >> 16) & 255u));
              w[2 * e + 1] = two_bf16((float)((y >> 8) & 255u), (float)(y >> 24));
            }
            st = as_operand(w[0], w[1], w[2], w[3]);
          } else {
            const uint32_t y = raw[s0 + s][kb];
            st = as_operand(((y << 3) & mask) | sixteen, ((y >> 5) & mask) | sixteen, ((y >> 1) & mask) | sixteen,
                            ((y >> 9) & mask) | sixteen);
          }
          ak[turn & 1][s] = mfma(tk[kb & 1], st, kb > kb0 ? ak[turn & 1][s] : none);
          aq[turn & 1][s] = queries_times(kb, st, kb > kb0 ? aq[turn & 1][s] : none);
        }
      if (turn > 0) add(turn - 1);
    }
    add(TURNS - 1);
  };
  // The decays and Gram products of a tile with the tokens before it, in the matrix unit's layout: token i = 16 t + l16 a lane,
  // tokens j 4 qq + r of 16 jt.  From the tile's own end back to the first token: D_ij is the product of the decays on i's path
  // behind j, i's own among them: those behind in the lane's four, in the rows of lanes above, and in the tiles behind.
  // With four waves, two of them each take every other tile of j.
  auto gram = [&](auto of_queries, int t) {
    constexpr bool Q = decltype(of_queries)::value;
    const int i = 16 * t + l16;
    const uint64_t path = i >= n && i < N ? sm.row[i - n] : ~0ull;
    const uint32_t lo = (uint32_t)path, hi = (uint32_t)(path >> 32);
    // bit j of the three words: token j is on i's path (buffered ones are)
    const uint32_t w0 = n ? lo << n | ((1u << n) - 1u) : lo, w1 = n ? hi << n | lo >> (32 - n) : hi, w2 = n ? hi >> (32 - n) : 0u;
    const uint32_t v0 = i < n ? ~0u : w0, v1 = i < n ? ~0u : w1, v2 = i < n ? ~0u : w2;
    const float own = Q ? 1.f : sm.beta[i] * sm.ks[i];
    float behind = 1.f;
    for (int jt = t; jt >= 0; --jt) {
      const bool mine = kWaves == 2 || ((t - jt) & 1) == wave / 2;
      v4f acc = {0.f, 0.f, 0.f, 0.f};
      if (mine) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const v8bf kj = operand(&sm.k[16 * jt + l16][32 * kb]);
          if constexpr (Q) {
#pragma unroll
            for (int e = 0; e < PIECES; ++e) acc = mfma(kj, operand(&sm.q[16 * e + l16][32 * kb]), acc);
          } else {
            acc = mfma(kj, operand(&sm.k[16 * t + l16][32 * kb]), acc);
          }
        }
      }
      const int j = 16 * jt + 4 * qq;
      const uint32_t nibble = (jt < 2 ? v0 : jt < 4 ? v1 : v2) >> (16 * (jt & 1) + 4 * qq);
      const float4 dj = *(const float4*)&sm.decay[j], kj = *(const float4*)&sm.ks[j];
      const float d[4] = {dj.x, dj.y, dj.z, dj.w}, ks[4] = {kj.x, kj.y, kj.z, kj.w};
      bool on[4];
      float f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        on[r] = i < N && j + r < i && ((nibble >> r) & 1u);
        f[r] = on[r] || j + r == i ? d[r] : 1.f;
        if (Q) on[r] = on[r] || (i < N && j + r == i);
      }
      const float f32_ = f[3] * f[2], f321 = f32_ * f[1];
      uint32_t rows[4];
      rows_gather(f32_bits(f321 * f[0]), 4, rows);
      const float g1 = bits_f32(rows[1]), g2 = bits_f32(rows[2]), g3 = bits_f32(rows[3]), g32_ = g3 * g2, g321 = g32_ * g1;
      const float above = behind * (qq == 0 ? g321 : qq == 1 ? g32_ : qq == 2 ? g3 : 1.f);
      const float p[4] = {f321, f32_, f[3], 1.f};
      float (*to)[16] = Q ? sm.m.g.c : sm.m.g.a;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (mine) to[j + r][l16] = on[r] ? above * p[r] * (own * ks[r]) * acc[r] : 0.f;
      behind *= g321 * bits_f32(rows[0]);
    }
    if (!Q && qq == 0 && wave == 0) sm.gamma[l16] = behind;
  };
  auto columns = [&](const float* row, float (&y)[SPW]) {
    if constexpr (SPW == 4) {
      const float4 v = *(const float4*)(row + c0);
      y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
    } else {
      const float2 v = *(const float2*)(row + c0);
      y[0] = v.x; y[1] = v.y;
    }
  };
  // x += what the tokens below `end` add, four an instruction (fp32): weights at[j][l16], times sign
  auto add_tokens = [&](int end, const float (*at)[16], float sign, v4f (&x)[SPW]) {
    for (int j0 = 0; j0 < end; j0 += 16) {     // (rows behind the last token are zeros)
      float w[4], u[4][SPW];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        w[f] = sign * at[j0 + 4 * f + qq][l16];
        columns(sm.u[j0 + 4 * f + qq], u[f]);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (j0 + 4 * f >= end) break;
#pragma unroll
        for (int s = 0; s < SPW; ++s) x[s] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[f], u[f][s], x[s], 0, 0, 0);
      }
    }
  };

  for (int t = 0; t < (NKT == 1 ? 1 : NT); ++t) {
    if constexpr (NKT > 1) {
      if (t > 0) {
        __syncthreads();                       // the tile before is done with its queries and products
        take_queries(16 * t - n, 0, queries);
        load_queries(16 * (t + 1) - n, queries);
        __syncthreads();
      }
    }
    auto grams = [&] {
      if (wave % 2 == 0) gram(std::false_type{}, t);
      else gram(std::true_type{}, t);
    };
    if constexpr (SM::kGramFirst) grams();
    v4f xk[SPW], xq[SPW];
    if (!is8) project(std::false_type{}, &sm.k[16 * t][0], xk, xq);
    else if constexpr (HB != 4) project(std::true_type{}, &sm.k[16 * t][0], xk, xq);
    if constexpr (!SM::kGramFirst) {
      __syncthreads();                         // the scales have been read: the Gram products take their place
      grams();
    }
    __syncthreads();

    // ---------------------------------------------------------------- solve
    const int i0 = 16 * t + 4 * qq;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float be = sm.beta[i0 + r], f = be * sm.gamma[4 * qq + r] * sm.ks[i0 + r];
      float v[SPW];
      columns(sm.u[i0 + r], v);
#pragma unroll
      for (int s = 0; s < SPW; ++s) xk[s][r] = be * v[s] - f * xk[s][r];
    }
    if (NKT > 1 && t > 0) add_tokens(16 * t, sm.m.g.a, -1.f, xk);
    // four tokens at a time: they are in the lanes of one row, which solve their triangle; what they add to those behind them
    // is one product a strip
    float4 a0[4], a1[4];
    float a23[4], w[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const float (*a)[16] = sm.m.g.a + 16 * t + 4 * f;
      a0[f] = *(const float4*)&a[0][4 * f];
      a1[f] = *(const float4*)&a[1][4 * f];
      a23[f] = a[2][4 * f + 3];
      w[f] = -a[qq][l16];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      float y[4][SPW];
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        y[0][s] = xk[s][0];
        y[1][s] = xk[s][1] - a0[f].y * y[0][s];
        y[2][s] = xk[s][2] - a0[f].z * y[0][s] - a1[f].z * y[1][s];
        y[3][s] = xk[s][3] - a0[f].w * y[0][s] - a1[f].w * y[1][s] - a23[f] * y[2][s];
      }
      if (qq == f)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float* row = &sm.u[i0 + r][c0];
          if constexpr (SPW == 4) *(float4*)row = make_float4(y[r][0], y[r][1], y[r][2], y[r][3]);
          else *(float2*)row = make_float2(y[r][0], y[r][1]);
        }
      wave_sync();
      if (f == 3 || 16 * t + 4 * f + 4 >= N) break;      // (zeros from there on, and nobody asks for them)
      float u[SPW];
      columns(sm.u[16 * t + 4 * f + qq], u);
#pragma unroll
      for (int s = 0; s < SPW; ++s) xk[s] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[f], u[s], xk[s], 0, 0, 0);
    }

    // -------------------------------------------------------------- outputs
    if (16 * t + 16 <= n) continue;            // buffered tokens only
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float g = sm.gamma[4 * qq + r];
#pragma unroll
      for (int s = 0; s < SPW; ++s) xq[s][r] *= g;
    }
    add_tokens(min(N, 16 * t + 16), sm.m.g.c, 1.f, xq);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float y[SPW];
#pragma unroll
      for (int s = 0; s < SPW; ++s) y[s] = xq[s][r];
      if (i0 + r >= n && i0 + r < N) store_rows(i0 + r - n, y);
    }
  }
}

template <int D, int NKT, bool BF16>
hipError_t launch(const DraftParams& p, int buf_kind, hipStream_t s) {
  const dim3 grid((unsigned)p.l.Hv, (unsigned)p.l.B);
  constexpr int kThreads = 64 * waves_of<D, NKT>();
  const bool mixed = buf_kind == PACE_BUF_K4_VBF16;
  if (p.l.bf16_state) {                        // (int8 buffer only: checked by the caller)
    step_kernel<D, NKT, BF16, false, 4, 1, true><<<grid, kThreads, 0, s>>>(p);
  } else if (BF16 && p.l.mask8 == 0 && !mixed && p.l.group == 64) {
    // All heads in 4 bits, the symmetric layout's groups: fewer registers, no second way through the projections, half
    // as many scalings.  64 chains of 8 take 14.0 us, by the general kernel 14.8; one sequence's five 5.6 and 6.1.  (The
    // layout that batches are served in; not tried for fp32, the mixed buffer or some heads in 8 bits.)
    if constexpr (BF16) step_kernel<D, NKT, true, false, 4, 2, false><<<grid, kThreads, 0, s>>>(p);
  } else if (mixed) {
    step_kernel<D, NKT, BF16, true, 0, 1, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    step_kernel<D, NKT, BF16, false, 0, 1, false><<<grid, kThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <int D, bool BF16>
hipError_t by_tiles(const DraftParams& p, int buf_kind, hipStream_t s) {
  // (LDS goes by the tiles: 64 chains of 8 in the one tile that they need 14.0 us, in the kernel for two 17.6)
  const int t = draft_tiles(p.l.dP, p.T);
  if (t <= 1) return launch<D, 1, BF16>(p, buf_kind, s);
  if (t <= 2) return launch<D, 2, BF16>(p, buf_kind, s);
  if (t <= 3) return launch<D, 3, BF16>(p, buf_kind, s);
  if (t <= 4) return launch<D, 4, BF16>(p, buf_kind, s);
  return launch<D, 6, BF16>(p, buf_kind, s);
}

}  // namespace

hipError_t launch_draft_step(const DraftParams& p, int dk, int buf_kind, hipStream_t stream) {
  if (dk == 128) return p.l.io_bf16 ? by_tiles<128, true>(p, buf_kind, stream) : by_tiles<128, false>(p, buf_kind, stream);
  return p.l.io_bf16 ? by_tiles<64, true>(p, buf_kind, stream) : by_tiles<64, false>(p, buf_kind, stream);
}

}  // namespace pace
