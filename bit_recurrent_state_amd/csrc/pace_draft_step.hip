// Gated-delta outputs of drafted tokens (include/pace_draft.h: pace_draft_step) -- gfx950, wave64.
//
// One workgroup of two waves per (sequence, value head) tile; nothing is written but o.  With S_0 the dequantised state and
// tokens 0 .. N-1 the n buffered ones and then the drafts, D_ij the product of the decays behind token j up to i along
// the path of i, and Gamma_i the product of all of them (from S_0 on),
//     u_i = beta_i (v_i - Gamma_i S_0^T k_i - sum_{j before i} D_ij (k_j . k_i) u_j)
//     o_i = Gamma_i S_0^T q_i + sum_{j before i, or i} D_ij (k_j . q_i) u_j,
// so the state of no node is ever formed: the tile's codes are read once, for all tokens.
//
//   tokens       buffered codes and quantised drafts as bf16 (exact) in LDS, in the order of the state's units
//   decays       row i's products by one lane, walking its path back
//   Gram         k_j . k_i and k_j . q_i on the bf16 matrix cores, times the decays
//   projections  tokens (A) times state columns (B), 32 keys an instruction.  A 4-bit code c becomes the bf16 number 16 + c by
//                a shift and a mask-and-or of two codes; a second product with -(16 + z) takes the offset and the zero
//                point off, so that the sums are exact for key codes.  One scale a (column, group).
//   solve        16 tokens at a time: what the tokens before them add in the matrix unit's layout (4 tokens x 4 columns
//                a lane), then the 16 x 16 triangle, one column a lane
//   outputs      16 queries at a time, the same way
// Queries enter as they are in bf16, as three bf16 pieces (exact) in fp32.  Everything else is fp32.
#include <hip/hip_runtime.h>

#include "pace_draft_internal.h"
#include "pace_draft_tokens.h"

namespace pace {
namespace {

constexpr int kWaves = 2, kThreads = 64 * kWaves;

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ inline v4f mfma(v8bf a, v8bf b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

__device__ inline v8bf as_operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 w = make_uint4(a, b, c, d);
  return __builtin_bit_cast(v8bf, w);
}

// NKT: 16-token tiles of the buffered and drafted tokens.  PIECES: of a query.
template <int D, int NKT, int PIECES>
struct alignas(16) Smem {
  static constexpr int NK = 16 * NKT;
  static constexpr int TS = D + 8;              // row stride of tokens (bf16): 16 rows on distinct banks
  alignas(16) uint16_t k[NK][TS];               // key codes
  alignas(16) uint16_t q[16 * PIECES][TS];      // one tile of queries
  alignas(16) float u[NK][D];                   // v^, then u
  alignas(16) float a[NK][NK];                  // [j][i]: beta_i D_ij (k_j . k_i), 0 for j >= i
  alignas(16) float c[NK][16];                  // [j][i]: D_ij (k_j . q_i) of one tile of queries
  float scale[4][D], zero[4][D];                // of (group, column)
  alignas(16) float ks[NK], decay[NK], beta[NK], gamma[NK];
  uint64_t row[kMaxDrafts];                     // tree bits
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

template <int D, int NKT, bool BF16, bool BFS>
__global__ __launch_bounds__(kThreads) void step_kernel(DraftParams p, int mixed) {
  constexpr int PIECES = BF16 ? 1 : 3;
  using SM = Smem<D, NKT, PIECES>;
  constexpr int KB = D / 32;                   // matrix instructions along the keys
  constexpr int SPW = D / 16 / kWaves;         // 16-column strips a wave
  constexpr int CW = D / kWaves;               // columns a wave
  constexpr int LANES = D / 8, ROWS = kThreads / LANES;
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
  const int len = p.draft_lens ? min(max(p.draft_lens[b], 0), T) : T;
  const size_t bh = (size_t)b * l.Hv + h, tok0 = (size_t)b * T;
  const int n = min(max(((const int32_t*)l.buffer)[bh], 0), l.dP - 1), N = n + len;
  // a lane's columns: c0 .. c0 + SPW - 1, one a strip
  const int c0 = wave * CW + SPW * l16;

  auto store_rows = [&](int t, const float (&x)[SPW]) {
    const size_t at = ((tok0 + t) * l.Hv + h) * D + c0;
    if constexpr (BF16) {
      uint32_t w[SPW / 2];
#pragma unroll
      for (int s = 0; s < SPW / 2; ++s) w[s] = two_bf16(x[2 * s], x[2 * s + 1]);
      if constexpr (SPW == 4) *(uint2*)((uint16_t*)l.o + at) = make_uint2(w[0], w[1]);
      else *(uint32_t*)((uint16_t*)l.o + at) = w[0];
    } else {
      if constexpr (SPW == 4) *(float4*)((float*)l.o + at) = make_float4(x[0], x[1], x[2], x[3]);
      else *(float2*)((float*)l.o + at) = make_float2(x[0], x[1]);
    }
  };
  {
    const float none[SPW] = {};
    for (int t = len + qq; t < T; t += 4) store_rows(t, none);
  }
  if (len == 0) return;

  // ------------------------------------------------------------------ state
  const bool is8 = !BFS && ((l.mask8 >> h) & 1ull) != 0, asym = l.asym != 0;
  const int bits = BFS ? 16 : is8 ? 8 : 4;
  const uint64_t below = h ? (l.mask8 & ((1ull << h) - 1ull)) : 0ull;
  const uint8_t* rec = l.state + (uint64_t)b * l.seq_stride + (uint64_t)h * l.rec4 + (uint64_t)__popcll(below) * (l.rec8 - l.rec4);
  const int group = BFS ? D : l.group, NG = D / group, kpg = group / 32;
  // the wave's codes: of strip s, column c0 + s, keys 8 qq .. + 7 of every 32 (one unit each)
  constexpr int AW = BFS ? 4 * KB : 2 * KB;
  uint32_t raw[SPW][AW];
#pragma unroll
  for (int s = 0; s < SPW; ++s) {
    const uint8_t* col = rec + (size_t)(c0 + s) * (D * bits / 8);
    if constexpr (BFS) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const uint4 v = *(const uint4*)(col + 2 * (32 * kb + 8 * qq));
        raw[s][4 * kb] = v.x; raw[s][4 * kb + 1] = v.y; raw[s][4 * kb + 2] = v.z; raw[s][4 * kb + 3] = v.w;
      }
    } else if (is8) {
#pragma unroll
      for (int kb = 0; kb < KB; kb += 2) {
        const uint4 v = *(const uint4*)(col + 8 * (qq * KB + kb));
        raw[s][2 * kb] = v.x; raw[s][2 * kb + 1] = v.y; raw[s][2 * kb + 2] = v.z; raw[s][2 * kb + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) raw[s][kb] = ((const uint32_t*)(col + 4 * qq * KB))[kb];
    }
  }
  if constexpr (!BFS) {
    const uint16_t* scales = (const uint16_t*)(rec + (is8 ? l.scales_off8 : l.scales_off4));
    const uint8_t* zeros = rec + (is8 ? l.zeros_off8 : l.zeros_off4);
    for (int i = tid; i < D * NG; i += kThreads) {
      const int c = i / NG, g = i - c * NG;
      sm.scale[g][c] = bf16_to_f32(scales[i]);
      sm.zero[g][c] = !asym ? (float)(1 << (bits - 1)) : is8 ? (float)zeros[i] : (float)((zeros[i >> 1] >> (4 * (i & 1))) & 15);
    }
  }

  // ----------------------------------------------------------------- tokens
  const int e0 = 8 * (tid % LANES);
  for (int i0 = 0; i0 < N; i0 += ROWS) {
    const int i = i0 + tid / LANES;
    if (i >= N) continue;
    float kx[8], vx[8], ks;
    if (i < n) {
      const size_t kslot = ((size_t)b * l.Hk + kh) * l.dP + i, vslot = bh * l.dP + i;
      if (mixed) {
        const uint32_t w = *(const uint32_t*)(l.buffer + l.off_kc + kslot * (D / 2) + e0 / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          kx[j] = (float)((int)((w >> (8 * j)) & 15u) - 8);
          kx[4 + j] = (float)((int)((w >> (8 * j + 4)) & 15u) - 8);
        }
        load8<true>(l.buffer + l.off_v, (int64_t)(vslot * D + e0), vx);
      } else {
        const uint2 w = *(const uint2*)(l.buffer + l.off_kc + kslot * D + e0);
        const uint2 x = *(const uint2*)(l.buffer + l.off_v + vslot * D + e0);
        const float vs = ((const float*)(l.buffer + l.off_vs))[vslot];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          kx[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
          vx[j] = (float)(int8_t)((j < 4 ? x.x : x.y) >> (8 * (j & 3))) * vs;
        }
      }
      ks = ((const float*)(l.buffer + l.off_ks))[kslot];
      if (e0 == 0) {
        sm.decay[i] = ((const float*)(l.buffer + l.off_a))[vslot];
        sm.beta[i] = ((const float*)(l.buffer + l.off_beta))[vslot];
      }
    } else {
      const size_t tok = tok0 + (i - n);
      float x[8];
      load8<BF16>(l.k, (int64_t)((tok * l.Hk + kh) * D + e0), x);
      ks = quantise8<LANES>(x, mixed, kx);
      load8<BF16>(l.v, (int64_t)((tok * l.Hv + h) * D + e0), x);
      if (mixed) {
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
      if (e0 == 0) {
        sm.decay[i] = l.a[tok * l.Hv + h];
        sm.beta[i] = l.beta[tok * l.Hv + h];
      }
    }
    if (e0 == 0) sm.ks[i] = ks;
    *(uint4*)&sm.k[i][e0] = in_order<BFS>(kx);
    *(float4*)&sm.u[i][e0] = make_float4(vx[0], vx[1], vx[2], vx[3]);
    *(float4*)&sm.u[i][e0 + 4] = make_float4(vx[4], vx[5], vx[6], vx[7]);
  }
  const int NT = (N + 15) / 16, NR = 16 * NT;        // tiles and rows in use
  for (int i = N + tid / LANES; i < NR; i += ROWS) { // rows behind the last token hold zeros
    *(uint4*)&sm.k[i][e0] = make_uint4(0, 0, 0, 0);
    *(float4*)&sm.u[i][e0] = make_float4(0.f, 0.f, 0.f, 0.f);
    *(float4*)&sm.u[i][e0 + 4] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e0 == 0) sm.ks[i] = sm.decay[i] = sm.beta[i] = 0.f;
  }
  if (tid < len) {
    uint64_t bitsrow = ~0ull;
    if (p.tree) {
      const int words = (T + 31) / 32;
      const uint32_t* t = p.tree + b * p.tree_stride + (int64_t)tid * words;
      bitsrow = t[0];
      if (words > 1) bitsrow |= (uint64_t)t[1] << 32;
    }
    sm.row[tid] = bitsrow;
  }
  __syncthreads();

  // ----------------------------------------------------------------- decays
  // a[j][i] = D_ij of the tokens before i on its path, 0 elsewhere
  if (tid < NR) {
    const int i = tid;
    float prod = sm.decay[i];
    const uint64_t bitsrow = i >= n && i < N ? sm.row[i - n] : ~0ull;
    for (int j = NR - 1; j >= 0; --j) {
      const bool on = i < N && j < i && (j < n || ((bitsrow >> (j - n)) & 1ull));
      sm.a[j][i] = on ? prod : 0.f;
      if (on) prod *= sm.decay[j];
    }
    sm.gamma[i] = prod;
  }
  __syncthreads();

  // ------------------------------------------------------------------- Gram
  auto operand = [&](const uint16_t* row) { return *(const v8bf*)(row + 8 * qq); };
  for (int t = wave; t < NT * NT; t += kWaves) {
    const int it = t / NT, jt = t % NT;               // rows (A) i, columns (B) j
    if (jt > it) continue;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) acc = mfma(operand(&sm.k[16 * it + l16][32 * kb]), operand(&sm.k[16 * jt + l16][32 * kb]), acc);
    const int j = 16 * jt + l16, i = 16 * it + 4 * qq;
    float4* at = (float4*)&sm.a[j][i];
    const float4 d = *at, ksi = *(const float4*)&sm.ks[i], be = *(const float4*)&sm.beta[i];
    const float kj = sm.ks[j];
    *at = make_float4(d.x * be.x * ksi.x * kj * acc[0], d.y * be.y * ksi.y * kj * acc[1], d.z * be.z * ksi.z * kj * acc[2],
                      d.w * be.w * ksi.w * kj * acc[3]);
  }

  // State operand of strip s, instruction kb, and the offset it carries.
  auto state_operand = [&](int s, int kb) {
    if constexpr (BFS) return as_operand(raw[s][4 * kb], raw[s][4 * kb + 1], raw[s][4 * kb + 2], raw[s][4 * kb + 3]);
    if (!is8) {
      const uint32_t x = raw[s][kb];
      return as_operand(((x << 3) & 0x00780078u) | 0x41804180u, ((x >> 5) & 0x00780078u) | 0x41804180u,
                        ((x >> 1) & 0x00780078u) | 0x41804180u, ((x >> 9) & 0x00780078u) | 0x41804180u);
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t x = raw[s][2 * kb + e];
      w[2 * e] = two_bf16((float)(x & 255u), (float)((x >> 16) & 255u));
      w[2 * e + 1] = two_bf16((float)((x >> 8) & 255u), (float)(x >> 24));
    }
    return as_operand(w[0], w[1], w[2], w[3]);
  };
  // Projections of 16 tokens (PIECES operands a 32-key block) on the wave's columns: x[s][r] of token 4 qq + r.
  auto project = [&](auto pieces, const uint16_t* rows, float (&x)[SPW][4]) {
    constexpr int P = decltype(pieces)::value;
    v8bf tok[P][KB];
#pragma unroll
    for (int e = 0; e < P; ++e)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) tok[e][kb] = operand(rows + (size_t)(16 * e + l16) * SM::TS + 32 * kb);
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
      v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 4; ++r) x[s][r] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const v8bf st = state_operand(s, kb);
        const int g = kb / kpg;
        if constexpr (!BFS) {
          const float off = -((is8 ? 0.f : 16.f) + sm.zero[g][c0 + s]);
          const uint32_t w = two_bf16(off, off);
          const v8bf z = as_operand(w, w, w, w);
#pragma unroll
          for (int e = 0; e < P; ++e) acc = mfma(tok[e][kb], z, acc);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) acc = mfma(tok[e][kb], st, acc);
        if constexpr (!BFS) {
          if ((kb + 1) % kpg == 0) {
            const float sc = sm.scale[g][c0 + s];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[s][r] += sc * acc[r];
            acc = v4f{0.f, 0.f, 0.f, 0.f};
          }
        }
      }
      if constexpr (BFS)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[s][r] = acc[r];
    }
  };
  auto add_columns = [&](const float* row, float (&y)[SPW]) {
    if constexpr (SPW == 4) {
      const float4 v = *(const float4*)(row + c0);
      y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
    } else {
      const float2 v = *(const float2*)(row + c0);
      y[0] = v.x; y[1] = v.y;
    }
  };
  __syncthreads();

  // ------------------------------------------------------------------ solve
  for (int t = 0; t < NT; ++t) {
    float x[SPW][4];
    project(std::integral_constant<int, 1>{}, &sm.k[16 * t][0], x);
    const int i0 = 16 * t + 4 * qq;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float be = sm.beta[i0 + r], f = be * sm.gamma[i0 + r] * sm.ks[i0 + r];
      float v[SPW];
      add_columns(sm.u[i0 + r], v);
#pragma unroll
      for (int s = 0; s < SPW; ++s) x[s][r] = be * v[s] - f * x[s][r];
    }
    for (int j = 0; j < 16 * t; ++j) {
      const float4 a = *(const float4*)&sm.a[j][i0];
      float u[SPW];
      add_columns(sm.u[j], u);
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        x[s][0] -= a.x * u[s];
        x[s][1] -= a.y * u[s];
        x[s][2] -= a.z * u[s];
        x[s][3] -= a.w * u[s];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float* row = &sm.u[i0 + r][c0];
      if constexpr (SPW == 4) *(float4*)row = make_float4(x[0][r], x[1][r], x[2][r], x[3][r]);
      else *(float2*)row = make_float2(x[0][r], x[1][r]);
    }
    wave_sync();
    if (lane < CW) {
      const int c = wave * CW + lane;
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = sm.u[16 * t + i][c];
#pragma unroll
      for (int j = 0; j < 15; ++j) {
        const float* a = &sm.a[16 * t + j][16 * t];
#pragma unroll
        for (int i = j + 1; i < 16; ++i) y[i] -= a[i] * y[j];
      }
#pragma unroll
      for (int i = 1; i < 16; ++i) sm.u[16 * t + i][c] = y[i];
    }
    wave_sync();
  }

  // ---------------------------------------------------------------- outputs
  for (int t0 = 0; t0 < len; t0 += 16) {
    __syncthreads();
    for (int i = tid / LANES; i < 16; i += ROWS) {
      float x[8] = {};
      if (t0 + i < len) load8<BF16>(l.q, (int64_t)(((tok0 + t0 + i) * l.Hk + kh) * D + e0), x);
#pragma unroll
      for (int e = 0; e < PIECES; ++e) {
        *(uint4*)&sm.q[16 * e + i][e0] = in_order<BFS>(x);
        if (e + 1 < PIECES) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const uint32_t w = two_bf16(x[j], x[j + 1]);
            x[j] -= bits_f32(w << 16);
            x[j + 1] -= bits_f32(w & 0xFFFF0000u);
          }
        }
      }
    }
    // decays of these rows, themselves included
    if (tid < 16) {
      const int i = n + t0 + tid;
      const bool in = t0 + tid < len;
      const uint64_t bitsrow = in ? sm.row[t0 + tid] : 0ull;
      float prod = 1.f;
      for (int j = NR - 1; j >= 0; --j) {
        const bool on = in && (j == i || (j < i && (j < n || ((bitsrow >> (j - n)) & 1ull))));
        sm.c[j][tid] = on ? prod : 0.f;
        if (on) prod *= sm.decay[j];
      }
    }
    __syncthreads();
    const int jt_end = min(NT, (n + t0 + 16 + 15) / 16);
    for (int jt = wave; jt < jt_end; jt += kWaves) {
      v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < PIECES; ++e)
          acc = mfma(operand(&sm.q[16 * e + l16][32 * kb]), operand(&sm.k[16 * jt + l16][32 * kb]), acc);
      const int j = 16 * jt + l16;
      float4* at = (float4*)&sm.c[j][4 * qq];
      const float4 d = *at;
      const float kj = sm.ks[j];
      *at = make_float4(d.x * kj * acc[0], d.y * kj * acc[1], d.z * kj * acc[2], d.w * kj * acc[3]);
    }
    float x[SPW][4];
    project(std::integral_constant<int, PIECES>{}, &sm.q[0][0], x);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + 4 * qq + r;
      const float g = t < len ? sm.gamma[n + t] : 0.f;
#pragma unroll
      for (int s = 0; s < SPW; ++s) x[s][r] *= g;
    }
    const int j_end = min(N, n + t0 + 16);
    for (int j = 0; j < j_end; ++j) {
      const float4 c = *(const float4*)&sm.c[j][4 * qq];
      float u[SPW];
      add_columns(sm.u[j], u);
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        x[s][0] += c.x * u[s];
        x[s][1] += c.y * u[s];
        x[s][2] += c.z * u[s];
        x[s][3] += c.w * u[s];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + 4 * qq + r;
      float y[SPW];
#pragma unroll
      for (int s = 0; s < SPW; ++s) y[s] = x[s][r];
      if (t < len) store_rows(t, y);
    }
  }
}

template <int D, int NKT, bool BF16>
hipError_t launch(const DraftParams& p, int buf_kind, hipStream_t s) {
  const dim3 grid((unsigned)p.l.Hv, (unsigned)p.l.B);
  const int mixed = buf_kind == PACE_BUF_K4_VBF16;
  if (p.l.bf16_state)
    step_kernel<D, NKT, BF16, true><<<grid, kThreads, 0, s>>>(p, mixed);
  else
    step_kernel<D, NKT, BF16, false><<<grid, kThreads, 0, s>>>(p, mixed);
  return hipGetLastError();
}

template <int D, bool BF16>
hipError_t by_tiles(const DraftParams& p, int buf_kind, hipStream_t s) {
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
