// Cached entries to other places (include/pace_draft.h: pace_cache_move; layout in include/pace_cache.h).
//
// A workgroup takes one piece (16, or 8, bytes of every lane) of the keys or of the values of one head and sequence, and
// walks the destinations from the first on, 64 tokens a step, in the lanes that hold them in the cache: every step's
// entries are in registers before any is stored, and what a later step reads lies behind all that was stored, as
// nodes[i] >= i.  Keys move as whole pieces; values are put together from the bytes of four tokens.
#include <hip/hip_runtime.h>

#include "pace_cache_internal.h"
#include "pace_draft_internal.h"

namespace pace {
namespace {

constexpr int kThreads = 256, kStep = 64;

struct Entry {
  const uint8_t* from;   // record of the entry (null: left out)
  uint8_t* to;
  int r_from, r_to;      // places in their pages
};

struct Walk {
  int64_t start;
  int count, h, b;
  uint32_t rec;
};

__device__ inline int page_of(const MoveParams& p, const int32_t* table, int b, int64_t pos) {
  const int64_t entry = pos >> p.page_shift;
  if (pos < 0 || entry >= p.max_pages) return -1;
  const int page = table[(int64_t)b * p.max_pages + entry];
  return page < p.num_pages ? page : -1;
}

// The entry that destination `pos` takes.
__device__ inline Entry entry_of(const MoveParams& p, const Walk& w, int64_t pos) {
  Entry e{nullptr, nullptr, 0, 0};
  const int64_t i = pos - w.start;
  if (i < 0 || i >= w.count) return e;
  const int node = p.nodes ? p.nodes[w.b * p.nodes_stride + i] : (int)i;
  if (node < 0) return e;
  const int64_t src = w.start + node;
  const int from = page_of(p, p.src_table, w.b, src), to = page_of(p, p.dst_table, w.b, pos);
  const int mask = (1 << p.page_shift) - 1;
  e.r_from = (int)(src & mask);
  e.r_to = (int)(pos & mask);
  if (from < 0 || to < 0 || (from == to && e.r_from == e.r_to)) return e;
  e.from = p.cache + ((int64_t)from * p.Hkv + w.h) * w.rec;
  e.to = p.cache + ((int64_t)to * p.Hkv + w.h) * w.rec;
  return e;
}

template <int W>
struct Piece {
  uint32_t w[W / 4];
};
template <int W>
__device__ inline Piece<W> load_piece(const uint8_t* at) {
  Piece<W> x;
  if constexpr (W == 16) {
    const uint4 v = *(const uint4*)at;
    x.w[0] = v.x; x.w[1] = v.y; x.w[2] = v.z; x.w[3] = v.w;
  } else {
    const uint2 v = *(const uint2*)at;
    x.w[0] = v.x; x.w[1] = v.y;
  }
  return x;
}
template <int W>
__device__ inline void store_piece(uint8_t* at, const Piece<W>& x) {
  if constexpr (W == 16)
    *(uint4*)at = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  else
    *(uint2*)at = make_uint2(x.w[0], x.w[1]);
}

// Every load of the step has arrived in every wave.
__device__ inline void all_loaded() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

template <int W>
__global__ __launch_bounds__(kThreads) void move_kernel(MoveParams p, int LB, int ng, uint32_t codes, uint32_t scales) {
  const int pieces = LB / W, tid = threadIdx.x;
  const int piece = blockIdx.x % pieces, kv = blockIdx.x / pieces % 2;
  Walk w;
  w.h = blockIdx.x / (2 * pieces);
  w.b = blockIdx.y;
  w.rec = 2 * (codes + scales);
  w.start = p.start[w.b];
  w.count = min(max(p.counts[w.b], 0), p.T);
  const int64_t end = min(w.start + w.count, (int64_t)p.max_pages << p.page_shift);
  const uint32_t part = kv ? codes + scales : 0u;
  auto scale_at = [&](int r, int g) { return part + codes + 2u * (((uint32_t)(r >> 2) * ng + g) * 4 + (r & 3)); };
  for (int64_t base = (w.start > 0 ? w.start : 0) & ~(int64_t)(kStep - 1); base < end; base += kStep) {
    // scales: one token a lane, by the workgroups of the first pieces
    Entry es{nullptr, nullptr, 0, 0};
    if (piece == 0 && tid < kStep) es = entry_of(p, w, base + tid);
    uint16_t sc[8];                              // (at most 256 channels in groups of 32)
    if (es.from) {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g < ng) sc[g] = *(const uint16_t*)(es.from + scale_at(es.r_from, g));
    }
    if (kv == 0) {
      const int a = (tid >> 4) & 3;
      const Entry e = entry_of(p, w, base + 16 * (tid >> 6) + (tid & 15));
      auto at = [&](int r) { return (uint32_t)(r >> 4) * (64 * LB) + piece * (64 * W) + (16 * a + (r & 15)) * W; };
      Piece<W> x;
      if (e.from) x = load_piece<W>(e.from + at(e.r_from));
      all_loaded();
      if (e.from) store_piece<W>(e.to + at(e.r_to), x);
    } else {
      const int m = tid & 15;
      auto at = [&](int r) { return part + (uint32_t)(r >> 2) * (16 * LB) + piece * (16 * W) + m * W; };
      Entry e[4];
      Piece<W> x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = entry_of(p, w, base + 4 * (tid >> 4) + j);
        if (e[j].from) x[j] = load_piece<W>(e[j].from + at(e[j].r_from));
      }
      all_loaded();
      Piece<W> y;
#pragma unroll
      for (int k = 0; k < W / 4; ++k) {
        y.w[k] = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e[j].from) y.w[k] |= ((x[j].w[k] >> (8 * (e[j].r_from & 3))) & 255u) << (8 * j);
      }
      if (e[0].from && e[1].from && e[2].from && e[3].from) {
        store_piece<W>(e[0].to + at(e[0].r_to), y);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e[j].from)
#pragma unroll
            for (int k = 0; k < W / 4; ++k) e[j].to[at(e[j].r_to) + 4 * k + (e[j].r_to & 3)] = (uint8_t)(y.w[k] >> (8 * j));
      }
    }
    if (es.from) {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g < ng) *(uint16_t*)(es.to + scale_at(es.r_to, g)) = sc[g];
    }
  }
}

}  // namespace

hipError_t launch_cache_move(const MoveParams& p, int kind, int d, int group, hipStream_t stream) {
  const int bits = kind == PACE_CACHE_INT4 ? 4 : 8, LB = d * bits / 32, W = LB < 16 ? LB : 16;
  const CacheRecord r = cache_record(d, group, 1 << p.page_shift, bits);
  const dim3 grid((unsigned)(p.Hkv * 2 * (LB / W)), (unsigned)p.B);
  if (W == 16)
    move_kernel<16><<<grid, kThreads, 0, stream>>>(p, LB, d / group, r.codes, r.scales);
  else
    move_kernel<8><<<grid, kThreads, 0, stream>>>(p, LB, d / group, r.codes, r.scales);
  return hipGetLastError();
}

}  // namespace pace
