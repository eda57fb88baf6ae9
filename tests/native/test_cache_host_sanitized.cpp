// Host entry points of the attention-layer operators (csrc/pace_cache.cpp) built for the CPU
// with AddressSanitizer and UndefinedBehaviorSanitizer, linked against recording stand-ins of
// the kernel launchers.  Checks that refused calls launch nothing, that the launch parameters
// follow from the arguments, and that the work split covers every size without overlap.
// Built and run by tests/test_cache_sanitized.py; prints "OK <checks>" on success.
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../../bit_recurrent_state_amd/csrc/pace_cache_internal.h"

using namespace pace;

static int fails = 0;
static long checks = 0;
#define EXPECT(c)                                        \
  do {                                                   \
    ++checks;                                            \
    if (!(c) && fails++ < 30) printf("FAIL line %d: %s\n", __LINE__, #c); \
  } while (0)

namespace pace {
static int launches = 0;
static RotaryParams rot;
static bool rot_wide = false;
static CacheIoParams io;
static AttnParams at;
static AttnPlan at_plan;
hipError_t launch_rotary(const RotaryParams& p, int, bool wide, hipStream_t) {
  ++launches; rot = p; rot_wide = wide;
  return hipSuccess;
}
hipError_t launch_cache_write(const CacheIoParams& p, int, int, int, int, hipStream_t) {
  ++launches; io = p;
  return hipSuccess;
}
hipError_t launch_cache_read(const CacheIoParams& p, int, int, int, int, hipStream_t) {
  ++launches; io = p;
  return hipErrorInvalidValue;
}
hipError_t launch_attention(const AttnParams& p, const AttnPlan& a, int, int, int, int, hipStream_t) {
  ++launches; at = p; at_plan = a;
  return hipSuccess;
}
}  // namespace pace

int main() {
  void* X = (void*)0x100000;
  const int32_t* I = (const int32_t*)0x200000;
  std::mt19937 rng(5);
  auto pick = [&](std::vector<int> v) { return v[rng() % v.size()]; };
  for (int trial = 0; trial < 4000; ++trial) {
    pace_cache_cfg c{};
    c.B = 1 + rng() % 70; c.Hkv = 1 + rng() % 16; c.Hq = c.Hkv * (1 + rng() % 9);
    c.d = pick({64, 128, 256}); c.kind = rng() % 3; c.group = pick({32, 64});
    c.page = pick({16, 32, 64, 1024}); c.num_pages = 1 + rng() % 100000; c.max_pages = 1 + rng() % 20000;
    c.io_dtype = rng() % 2;
    const int T = 1 + rng() % 700, max_len = 1 + rng() % 300000;
    pace_cache_layout_info info;
    EXPECT(pace_cache_layout(&c, &info) == PACE_OK);
    EXPECT(info.record_bytes % 16 == 0 && info.cache_bytes == info.page_bytes * (size_t)c.num_pages);
    size_t need = 0;
    EXPECT(pace_cache_attention_workspace_bytes(&c, T, max_len, &need) == PACE_OK);
    const int before = launches;
    const pace_status st = pace_cache_attention(&c, X, I, X, (int64_t)c.Hq * c.d, T, I, nullptr, nullptr, 0, 0.1, max_len,
                                                X, nullptr, need ? X : nullptr, need, nullptr);
    EXPECT(st == PACE_OK && launches == before + 1);
    // every row is in exactly one workgroup, every token in exactly one piece
    const int64_t rows = 16 * at_plan.row_tiles;
    EXPECT(at_plan.row_blocks * rows >= at.R && (at_plan.row_blocks - 1) * rows < at.R && at.row_blocks == at_plan.row_blocks);
    EXPECT(at_plan.row_tiles == 1 || (at_plan.row_tiles == 2 && c.d <= 128));
    EXPECT(at_plan.waves == 4 || (at_plan.waves == 8 && at_plan.row_tiles == 1 && c.d <= 128));
    EXPECT(at_plan.step == 16 * kTiles * at_plan.waves);
    EXPECT(at.nsplit >= 1 && at.nsplit <= kMaxPieces && at.chunk % at_plan.step == 0);
    EXPECT((int64_t)at.nsplit * at.chunk >= max_len && (int64_t)(at.nsplit - 1) * at.chunk < max_len);
    EXPECT((need != 0) == (at.nsplit > 1));
    if (need) {
      const size_t rowsAll = (size_t)at.nsplit * c.B * c.Hkv * at.R;
      EXPECT((char*)(at.part_lse + rowsAll) <= (char*)X + need && (char*)at.part_lse == (char*)(at.part_o + rowsAll * c.d));
    }
    EXPECT((1 << at.page_shift) == c.page && at.gamma * c.Hkv == c.Hq);
    EXPECT(pace_cache_write(&c, X, I, I, T, X, (int64_t)c.Hkv * c.d, X, (int64_t)c.Hkv * c.d + 8, nullptr) == PACE_OK);
    EXPECT(io.cache == X && io.k_in == X && io.v_stride == (int64_t)c.Hkv * c.d + 8 && (1 << io.page_shift) == c.page);
    EXPECT(pace_cache_read(&c, X, I, I, T, X, (int64_t)c.Hkv * c.d, X, (int64_t)c.Hkv * c.d, nullptr) == PACE_EHIP);
    const int n = launches;
    EXPECT(pace_cache_write(&c, X, I, I, T, X, (int64_t)c.Hkv * c.d - 1, X, (int64_t)c.Hkv * c.d, nullptr) == PACE_EINVAL);
    EXPECT(pace_cache_write(&c, X, I, I, 0, nullptr, 0, nullptr, 0, nullptr) == PACE_OK);
    c.group = 48;
    EXPECT(pace_cache_write(&c, X, I, I, T, X, (int64_t)c.Hkv * c.d, X, (int64_t)c.Hkv * c.d, nullptr) == PACE_EINVAL);
    EXPECT(launches == n);
  }
  // rotary: which calls run in units of 8 channels
  struct { int d, rd, il; int64_t s; uintptr_t p; bool wide; } R[] = {
      {128, 64, 0, 512, 0x1000, true}, {128, 40, 0, 512, 0x1000, false}, {128, 40, 1, 512, 0x1000, true},
      {128, 64, 0, 513, 0x1000, false}, {128, 64, 0, 512, 0x1002, false}, {70, 32, 1, 512, 0x1000, false}};
  for (const auto& r : R) {
    pace_rotary_cfg c{2, 2, r.d, r.rd, r.il, PACE_IO_BF16};
    EXPECT(pace_rotary(&c, 3, I, (const double*)I, 1.0, 2, (void*)r.p, r.s, (void*)r.p, r.s, X, 512, (void*)r.p, r.s, nullptr) ==
           PACE_OK);
    EXPECT(rot_wide == r.wide && rot.copy_q == 1 && rot.copy_k == 0 && rot.inverse == 1);
  }
  // tree bits and frequencies write exactly what they say
  for (int T = 1; T < 140; ++T) {
    std::vector<int32_t> par(T);
    for (int i = 0; i < T; ++i) par[i] = (int)(rng() % (i + 1)) - 1;
    std::vector<uint32_t> bits((size_t)T * ((T + 31) / 32), 0xFFFFFFFFu);
    EXPECT(pace_tree_bits(par.data(), T, bits.data()) == PACE_OK);
    for (int i = 0; i < T; ++i)
      for (int j = 0; j < (T + 31) / 32 * 32; ++j) {
        bool anc = false;
        for (int a = i; a >= 0; a = par[a]) anc |= a == j;
        EXPECT((((bits[(size_t)i * ((T + 31) / 32) + j / 32] >> (j % 32)) & 1) != 0) == anc);
      }
  }
  for (int rd = 2; rd <= 512; rd += 2)
    for (int s = 0; s < 4; ++s) {
      std::vector<double> f(rd / 2, -1.0);
      double m = 0;
      EXPECT(pace_rotary_freqs(rd, 1e4, s, 4.0, 4096.0, 32.0, 1.0, f.data(), &m) == PACE_OK);
      for (double x : f) EXPECT(x > 0.0 && x <= 1.0);
      EXPECT(m >= 1.0);
    }
  if (fails) return printf("%d failures\n", fails), 1;
  printf("OK %ld\n", checks);
  return 0;
}
