// Cached entries to other places (include/pace_draft.h: pace_cache_move; layout in include/pace_cache.h).
//
// With nodes, a workgroup takes one piece (16, or 8, bytes of every lane) of the keys or of the values of one head and
// sequence, and walks the destinations from the first on in the lanes that hold them in the cache.  Every step's entries
// are in registers, in every wave, before any is stored; and what a later step reads lies behind all that was stored, as
// nodes[i] >= i, so that the next step's entries are on their way meanwhile, and their addresses (node -> pages) a step
// ahead of those.  Keys move as whole pieces; values are put together from the bytes of four tokens.
// Measured (graph): half of 4 x 16384 entries, int8, 8 heads of 128: 45.4 us, 2.6 TB/s of entries; those kept lie among those
// dropped, so that nearly every line of the old contexts is read, 3.8 TB/s of lines (a large copy: 5.1).  Waves wait for
// memory 60% of their time; a second step in flight made it no faster (46 us).  64 accepted paths of 25: 6.0 us, latency of
// counts -> nodes -> pages -> entries.
// Without nodes nothing shifts: pages are copied record by record, all at once, and the tokens of the first and
// last page that are not asked for are left out by masks.  8 forks of 4093 tokens, int4: 11.4 us, 3.7 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pace_cache_internal.h"
#include "pace_draft_internal.h"
#include "pace_move_range.h"

namespace pace {
namespace {

struct Layout {
  int LB, ng;                     // bytes a lane holds of a token (keys) or quad (values), scales a token
  uint32_t codes, scales, rec;    // bytes of the parts and of the record
};

__device__ inline int page_of(const MoveParams& p, const int32_t* table, int b, int64_t pos) {
  const int64_t entry = pos >> p.page_shift;
  if (pos < 0 || entry >= p.max_pages) return -1;
  const int page = table[(int64_t)b * p.max_pages + entry];
  return page < p.num_pages ? page : -1;
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

// ------------------------------------------------------------------------------- with nodes

// An entry's record and its place in the page: byte offset times 1024 plus the place; -1: left out.
constexpr int kPlaceBits = 10;   // pages hold 1024 tokens at most
__device__ inline uint8_t* record(const MoveParams& p, int64_t e) { return p.cache + (e >> kPlaceBits); }
__device__ inline int place(int64_t e) { return (int)(e & ((1 << kPlaceBits) - 1)); }

// What the loop has in flight is loaded without conditions (entries that are left out read the cache's first bytes), into
// variables that change their part from step to step: a copy would wait for the loads.
template <int W, int NT, int SPLIT, bool VALUES>
__device__ inline void walk(const MoveParams& p, const Layout& y, int piece, int split, int h) {
  constexpr int KL = 4 / SPLIT, VL = 16 / SPLIT;   // lanes of a token's piece (keys), of a quad's (values)
  constexpr int STEP = NT / KL;                // tokens a step
  __shared__ int64_t from[4][STEP], to[4][STEP];
  const int tid = threadIdx.x, b = blockIdx.y;
  MoveRange range;
  if (!move_range(p.start[b], p.counts[b], p.T, (int64_t)p.max_pages << p.page_shift, range)) return;
  const int64_t start = range.start, end = range.end, base = range.base;
  const int steps = (int)((end - base + STEP - 1) / STEP);
  const int32_t* const nodes = p.nodes + b * p.nodes_stride;
  const int32_t* const src_table = p.src_table + (int64_t)b * p.max_pages;
  const int32_t* const dst_table = p.dst_table + (int64_t)b * p.max_pages;
  const uint32_t part = VALUES ? y.codes + y.scales : 0u;
  const int64_t mine = base + tid;             // this thread's destination, where it finds one: of step 0

  // The entry that destination mine + s STEP takes, in three parts a step apart: its node, its pages, its place.
  auto entry = [&](int64_t pos) { return (int)min(max(pos >> p.page_shift, (int64_t)0), (int64_t)p.max_pages - 1); };
  auto load_node = [&](int s, int& node) {
    if (tid < STEP) node = nodes[node_place(range, mine + (int64_t)s * STEP)];
  };
  struct Pages {
    int node, from, to;
  };
  auto load_pages = [&](int s, int node, Pages& g) {
    if (tid >= STEP) return;
    g.node = node;
    g.from = src_table[entry(start + node)];
    g.to = dst_table[entry(mine + (int64_t)s * STEP)];
  };
  auto put_entry = [&](int s, const Pages& g) {
    if (tid >= STEP) return;
    const int64_t pos = mine + (int64_t)s * STEP, src = start + g.node, limit = (int64_t)p.max_pages << p.page_shift;
    const int mask = (1 << p.page_shift) - 1, r = (int)(src & mask), r_to = (int)(pos & mask);
    const bool in = pos >= start && pos < end && g.node >= 0 && src >= 0 && src < limit && g.from >= 0 &&
                    g.from < p.num_pages && g.to >= 0 && g.to < p.num_pages && !(g.from == g.to && r == r_to);
    from[s & 3][tid] = in ? (((int64_t)g.from * p.Hkv + h) * y.rec << kPlaceBits) + r : -1;
    to[s & 3][tid] = in ? (((int64_t)g.to * p.Hkv + h) * y.rec << kPlaceBits) + r_to : -1;
  };

  // What a thread moves in a step: a piece of a token's key, or of a quad's four values; and a token's scales.
  struct Data {
    Piece<W> x0, x1, x2, x3;
    uint32_t scale[8];                         // (at most 256 channels in groups of 32)
  };
  auto scale_at = [&](int r, int g) { return part + y.codes + 2u * (((uint32_t)(r >> 2) * y.ng + g) * 4 + (r & 3)); };
  const bool with_scales = piece == 0 && split == 0 && tid < STEP;
  const int token = 16 * (tid / (16 * KL)) + (tid & 15), a = split * KL + (tid >> 4) % KL;
  const int quad = tid / VL, m = split * VL + tid % VL;
  auto at = [&](int r) {
    return VALUES ? part + (uint32_t)(r >> 2) * (16 * y.LB) + piece * (16 * W) + m * W
                  : (uint32_t)(r >> 4) * (64 * y.LB) + piece * (64 * W) + (16 * a + (r & 15)) * W;
  };
  auto load_one = [&](int64_t e) { return load_piece<W>(e < 0 ? p.cache : record(p, e) + at(place(e))); };
  auto load = [&](int s, Data& d) {
    const int64_t* const f = from[s & 3];
    if constexpr (VALUES) {
      d.x0 = load_one(f[4 * quad]);
      d.x1 = load_one(f[4 * quad + 1]);
      d.x2 = load_one(f[4 * quad + 2]);
      d.x3 = load_one(f[4 * quad + 3]);
    } else {
      d.x0 = load_one(f[token]);
    }
    if (with_scales) {
      const int64_t e = f[tid];
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g < y.ng) d.scale[g] = *(const uint16_t*)(e < 0 ? p.cache : record(p, e) + scale_at(place(e), g));
    }
  };
  auto arrive = [&](Data& d) {
    auto one = [](Piece<W>& x) {
      if constexpr (W == 16) asm volatile("" : "+v"(x.w[0]), "+v"(x.w[1]), "+v"(x.w[2]), "+v"(x.w[3]));
      else asm volatile("" : "+v"(x.w[0]), "+v"(x.w[1]));
    };
    one(d.x0);
    if constexpr (VALUES) {
      one(d.x1);
      one(d.x2);
      one(d.x3);
    }
    if (with_scales) {
#pragma unroll
      for (int g = 0; g < 8; ++g)
        if (g < y.ng) asm volatile("" : "+v"(d.scale[g]));
    }
  };
  auto store = [&](int s, const Data& d) {
    const int64_t* const f = from[s & 3];
    const int64_t* const t = to[s & 3];
    if constexpr (!VALUES) {
      const int64_t e = t[token];
      if (e >= 0) store_piece<W>(record(p, e) + at(place(e)), d.x0);
    } else {
      const int64_t e0 = t[4 * quad], e1 = t[4 * quad + 1], e2 = t[4 * quad + 2], e3 = t[4 * quad + 3];
      const int k0 = 8 * (place(f[4 * quad]) & 3), k1 = 8 * (place(f[4 * quad + 1]) & 3), k2 = 8 * (place(f[4 * quad + 2]) & 3),
                k3 = 8 * (place(f[4 * quad + 3]) & 3);
      Piece<W> z;
#pragma unroll
      for (int k = 0; k < W / 4; ++k)
        z.w[k] = ((d.x0.w[k] >> k0) & 255u) | ((d.x1.w[k] >> k1) & 255u) << 8 | ((d.x2.w[k] >> k2) & 255u) << 16 |
                 (d.x3.w[k] >> k3) << 24;
      if ((e0 | e1 | e2 | e3) >= 0) {
        store_piece<W>(record(p, e0) + at(place(e0)), z);
      } else {
        auto bytes = [&](int64_t e, int j) {   // (a destination's place in its quad is j)
          if (e < 0) return;
          uint8_t* const q = record(p, e) + at(place(e)) + j;
#pragma unroll
          for (int k = 0; k < W / 4; ++k) q[4 * k] = (uint8_t)(z.w[k] >> (8 * j));
        };
        bytes(e0, 0);
        bytes(e1, 1);
        bytes(e2, 2);
        bytes(e3, 3);
      }
    }
    if (with_scales) {
      const int64_t e = t[tid];
      if (e >= 0)
#pragma unroll
        for (int g = 0; g < 8; ++g)
          if (g < y.ng) *(uint16_t*)(record(p, e) + scale_at(place(e), g)) = (uint16_t)d.scale[g];
    }
  };

  if (steps == 1) {
    Data d;
    Pages g;
    int n;
    load_node(0, n);
    load_pages(0, n, g);
    put_entry(0, g);
    __syncthreads();
    load(0, d);
    arrive(d);
    __syncthreads();
    store(0, d);
    return;
  }
  // In flight ahead of step s: its data, step s + 1's entries, step s + 2's pages, step s + 3's nodes.
  Data d0, d1;
  Pages g0, g1;
  int n0, n1;
  load_node(0, n0);
  load_node(1, n1);
  load_pages(0, n0, g0);
  load_node(2, n0);
  put_entry(0, g0);
  load_pages(1, n1, g1);
  load_node(3, n1);
  put_entry(1, g1);
  load_pages(2, n0, g0);
  __syncthreads();
  load(0, d0);
  auto step = [&](int s, Data& now, Data& next, Pages& here, Pages& there, int& node_here, int& node_there) {
    // (steps past the last have no entries)
    load(s + 1, next);
    load_pages(s + 3, node_there, there);
    load_node(s + 4, node_here);
    put_entry(s + 2, here);
    arrive(now);
    // every wave's loads of this step have arrived, and what the next entries overwrite has been read
    __syncthreads();
    store(s, now);
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, d0, d1, g0, g1, n0, n1);
    step(s + 1, d1, d0, g1, g0, n1, n0);
  }
}

template <int W, int NT, int SPLIT>
__global__ __launch_bounds__(NT) void move_kernel(MoveParams p, Layout y) {
  const int pieces = y.LB / W, split = blockIdx.x / 2 % SPLIT, x = blockIdx.x / (2 * SPLIT);
  if (blockIdx.x & 1) walk<W, NT, SPLIT, true>(p, y, x % pieces, split, x / pieces);
  else walk<W, NT, SPLIT, false>(p, y, x % pieces, split, x / pieces);
}

// ---------------------------------------------------------------------------- without nodes

constexpr int kCopyThreads = 256;

template <int W>
__global__ __launch_bounds__(kCopyThreads) void copy_kernel(MoveParams p, Layout y, int64_t entries) {
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t start = p.start[b], end = min(start + min(max(p.counts[b], 0), p.T), (int64_t)p.max_pages << p.page_shift);
  const int64_t begin = max(start, (int64_t)0);
  if (begin >= end) return;
  const int64_t first = begin >> p.page_shift;
  for (int64_t i = blockIdx.x; i < entries * p.Hkv; i += gridDim.x) {
    const int64_t e = first + i / p.Hkv, pos = e << p.page_shift;
    const int h = (int)(i % p.Hkv);
    if (pos >= end) return;
    const int from = page_of(p, p.src_table, b, pos), to = page_of(p, p.dst_table, b, pos);
    if (from < 0 || to < 0 || from == to) continue;
    const uint8_t* const src = p.cache + ((int64_t)from * p.Hkv + h) * y.rec;
    uint8_t* const dst = p.cache + ((int64_t)to * p.Hkv + h) * y.rec;
    // tokens [r0, r1) of the page
    const int P = 1 << p.page_shift, r0 = (int)max(begin - pos, (int64_t)0), r1 = (int)min(end - pos, (int64_t)P);
    if (r0 == 0 && r1 == P) {
      const int n = y.rec / 16;                // (a record is a multiple of 16 bytes)
      for (int v = tid; v < n; v += 4 * kCopyThreads) {
        Piece<16> x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = load_piece<16>(src + 16 * (int64_t)min(v + k * kCopyThreads, n - 1));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (v + k * kCopyThreads < n) store_piece<16>(dst + 16 * (int64_t)(v + k * kCopyThreads), x[k]);
      }
      continue;
    }
    const int n = y.codes / W, tile = 64 * y.LB / W, quad = 16 * y.LB / W;
    const uint32_t values = y.codes + y.scales;
    for (int v = tid; v < n; v += kCopyThreads) {
      const int r = 16 * (v / tile) + (v & 15);          // a key's piece
      if (r >= r0 && r < r1) store_piece<W>(dst + v * W, load_piece<W>(src + v * W));
      const int q = 4 * (v / quad);                      // a quad's
      if (q + 4 <= r0 || q >= r1) continue;
      const Piece<W> x = load_piece<W>(src + values + v * W);
      if (q >= r0 && q + 4 <= r1) {
        store_piece<W>(dst + values + v * W, x);
      } else {
#pragma unroll
        for (int k = 0; k < W / 4; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (q + j >= r0 && q + j < r1) dst[values + v * W + 4 * k + j] = (uint8_t)(x.w[k] >> (8 * j));
      }
    }
    for (int v = tid; v < P * y.ng; v += kCopyThreads) {
      const int r = 4 * (v / (4 * y.ng)) + (v & 3);
      if (r < r0 || r >= r1) continue;
      ((uint16_t*)(dst + y.codes))[v] = ((const uint16_t*)(src + y.codes))[v];
      ((uint16_t*)(dst + values + y.codes))[v] = ((const uint16_t*)(src + values + y.codes))[v];
    }
  }
}

template <int W>
void launch(const MoveParams& p, const Layout& y, hipStream_t s) {
  if (!p.nodes) {
    // pages that T tokens from any place on lie in; beyond 2^22 workgroups they take several each
    const int64_t entries = std::min(((int64_t)p.T + (1 << p.page_shift) - 2) / (1 << p.page_shift) + 1, (int64_t)p.max_pages);
    const int64_t most = std::max<int64_t>(1, (1 << 22) / p.B);
    copy_kernel<W><<<dim3((unsigned)std::min(entries * p.Hkv, most), (unsigned)p.B), kCopyThreads, 0, s>>>(p, y, entries);
    return;
  }
  // (1024 heads in 16 parts of 1024 threads: 2^24 threads along x at most)
  const unsigned parts = (unsigned)(p.Hkv * 2 * (y.LB / W));
  // A workgroup's steps follow one another: 64 tokens each, or 512 where there are too few workgroups to fill the
  // chip with the small ones.  int8, 8 heads of 128, half of T kept, the small and the large: 4 x 16384 150 and 45.6 us, 4 x 300
  // 7.6 and 3.8, 8 x 8192 84 and 48, 16 x 8192 105 and 94, 64 x 1000 47.5 and 65.9, 64 x 300 19.3 and 44.
  if (p.T <= 64 || (int64_t)parts * p.B > 256)
    move_kernel<W, 256, 1><<<dim3(parts, (unsigned)p.B), 256, 0, s>>>(p, y);
  else
    move_kernel<W, 1024, 2><<<dim3(2 * parts, (unsigned)p.B), 1024, 0, s>>>(p, y);
}

}  // namespace

hipError_t launch_cache_move(const MoveParams& p, int kind, int d, int group, hipStream_t stream) {
  const int bits = kind == PACE_CACHE_INT4 ? 4 : 8, LB = d * bits / 32;
  const CacheRecord r = cache_record(d, group, 1 << p.page_shift, bits);
  const Layout y{LB, d / group, r.codes, r.scales, r.total};
  if (LB >= 16)
    launch<16>(p, y, stream);
  else
    launch<8>(p, y, stream);
  return hipGetLastError();
}

}  // namespace pace
