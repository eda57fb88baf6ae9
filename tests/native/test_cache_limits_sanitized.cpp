// Host entry points of the attention-layer operators (csrc/pace_cache.cpp) at the ends of their ranges, built for the
// CPU with AddressSanitizer and UndefinedBehaviorSanitizer and linked against recording stand-ins of the kernel
// launchers.  Built and run by tests/test_cache_limits.py; prints "OK <checks>" on success.
#include <climits>
#include <cmath>
#include <cstdio>
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
static std::vector<RotaryParams> rot;
static CacheIoParams io;
static AttnParams at;
static AttnPlan at_plan;
hipError_t launch_rotary(const RotaryParams& p, int, bool, hipStream_t) {
  ++launches; rot.push_back(p);
  return hipSuccess;
}
hipError_t launch_cache_write(const CacheIoParams& p, int, int, int, int, hipStream_t) {
  ++launches; io = p;
  return hipSuccess;
}
hipError_t launch_cache_read(const CacheIoParams& p, int, int, int, int, hipStream_t) {
  ++launches; io = p;
  return hipSuccess;
}
hipError_t launch_attention(const AttnParams& p, const AttnPlan& a, int, int, int, int, hipStream_t) {
  ++launches; at = p; at_plan = a;
  return hipSuccess;
}
}  // namespace pace

static void* const X = (void*)0x100000;
static const int32_t* const I = (const int32_t*)0x200000;

// Any max_len that fits its type plans whole pieces that cover it.
static void plans() {
  std::mt19937 rng(9);
  auto pick = [&](std::vector<int> v) { return v[rng() % v.size()]; };
  const std::vector<int> ends = {INT_MAX, INT_MAX - 1, INT_MAX - 127, INT_MAX - 128, INT_MAX - 255, INT_MAX - 256, INT_MAX - 4096,
                                 1 << 30, (1 << 30) + 1};
  for (int trial = 0; trial < 4000; ++trial) {
    pace_cache_cfg c{};
    c.B = pick({1, 2, 3, 64, 97, 128, 768, 1000}); c.Hkv = pick({1, 2, 8}); c.Hq = c.Hkv * (1 + rng() % 9);
    c.d = pick({64, 128, 256}); c.kind = rng() % 3; c.group = pick({32, 64});
    c.page = pick({16, 64, 1024}); c.num_pages = 1 + rng() % 100000; c.max_pages = 1 + rng() % 20000;
    c.io_dtype = rng() % 2;
    const int T = 1 + rng() % 40, max_len = rng() % 2 ? pick(ends) : 1 + (int)(rng() % INT_MAX);
    size_t need = 0;
    EXPECT(pace_cache_attention_workspace_bytes(&c, T, max_len, &need) == PACE_OK);
    const int before = launches;
    EXPECT(pace_cache_attention(&c, X, I, X, (int64_t)c.Hq * c.d, T, I, nullptr, nullptr, 0, 0.1, max_len, X, nullptr,
                                need ? X : nullptr, need, nullptr) == PACE_OK);
    EXPECT(launches == before + 1);
    EXPECT(at.nsplit >= 1 && at.nsplit <= kMaxPieces && at.chunk > 0 && at.chunk % at_plan.step == 0);
    // (one piece takes all there is, whatever its length)
    EXPECT(at.nsplit == 1 || ((int64_t)at.nsplit * at.chunk >= max_len && (int64_t)(at.nsplit - 1) * at.chunk < max_len));
    EXPECT((need != 0) == (at.nsplit > 1));
  }
}

// Token strides as wide as a long prompt, up to 2^48 bytes for all tokens.
static void strides() {
  pace_cache_cfg c{};
  c.B = 4; c.Hq = 32; c.Hkv = 32; c.d = 128; c.kind = PACE_CACHE_INT8; c.group = 128; c.page = 64;
  c.num_pages = 64; c.max_pages = 64; c.io_dtype = PACE_IO_BF16;
  pace_rotary_cfg r{32, 32, 128, 128, 0, PACE_IO_BF16};
  for (int T : {1, 5}) {
    const int64_t most = (INT64_C(1) << 48) / 2 / (4 * T) / 8 * 8;
    for (int64_t s : {INT64_C(4096), INT64_C(8388608), INT64_C(16777216), INT64_C(1) << 31, most}) {
      EXPECT(pace_cache_write(&c, X, I, I, T, X, s, X, s, nullptr) == PACE_OK && io.k_stride == s && io.v_stride == s);
      EXPECT(pace_cache_read(&c, X, I, I, T, X, s, X, s, nullptr) == PACE_OK && io.k_stride == s && io.v_stride == s);
      EXPECT(pace_cache_attention(&c, X, I, X, s, T, I, nullptr, nullptr, 0, 0.1, 16, X, nullptr, nullptr, 0, nullptr) == PACE_OK &&
             at.q_stride == s);
      rot.clear();
      EXPECT(pace_rotary(&r, 4 * T, I, (const double*)I, 1.0, 0, X, s, X, s, (char*)X + 64, s, (char*)X + 64, s, nullptr) == PACE_OK);
      EXPECT(rot.size() == 1 && rot[0].q_stride == s && rot[0].k_out_stride == s);
    }
    const int n = launches;
    for (int64_t s : {most + 8, INT64_C(1) << 60, INT64_MAX / 8 * 8, INT64_C(-4096)}) {
      EXPECT(pace_cache_write(&c, X, I, I, T, X, s, X, 4096, nullptr) == PACE_EINVAL);
      EXPECT(pace_cache_read(&c, X, I, I, T, X, 4096, X, s, nullptr) == PACE_EINVAL);
      EXPECT(pace_cache_attention(&c, X, I, X, s, T, I, nullptr, nullptr, 0, 0.1, 16, X, nullptr, nullptr, 0, nullptr) == PACE_EINVAL);
      EXPECT(pace_rotary(&r, 4 * T, I, (const double*)I, 1.0, 0, X, s, X, 4096, (char*)X + 64, 4096, (char*)X + 64, 4096, nullptr) ==
             PACE_EINVAL);
    }
    EXPECT(launches == n);
  }
  // trees of 16384 drafts a sequence: 2^23 words
  c.Hkv = 32;
  const int T = 16384;
  const int64_t words = (int64_t)T * (T / 32);
  EXPECT(pace_cache_attention(&c, X, I, X, 4096, T, I, nullptr, (const uint32_t*)X, words, 0.1, 16, X, nullptr, nullptr, 0, nullptr) ==
             PACE_OK && at.tree_stride == words);
  EXPECT(pace_cache_attention(&c, X, I, X, 4096, T, I, nullptr, (const uint32_t*)X, INT64_C(1) << 45, 0.1, 16, X, nullptr, nullptr, 0,
                              nullptr) == PACE_EINVAL);
}

// Factors that are finite in fp64 and not in fp32, in which the kernels take them.
static void factors() {
  pace_cache_cfg c{};
  c.B = 1; c.Hq = 2; c.Hkv = 1; c.d = 64; c.kind = PACE_CACHE_FP8; c.group = 64; c.page = 16; c.num_pages = 4; c.max_pages = 4;
  pace_rotary_cfg r{2, 1, 64, 64, 0, PACE_IO_F32};
  auto attend = [&](double scale) {
    return pace_cache_attention(&c, X, I, X, 128, 1, I, nullptr, nullptr, 0, scale, 16, X, nullptr, nullptr, 0, nullptr);
  };
  auto rotate = [&](double m) {
    return pace_rotary(&r, 3, I, (const double*)I, m, 0, X, 128, X, 64, (char*)X + 4096, 128, (char*)X + 8192, 64, nullptr);
  };
  const int n = launches;
  for (double x : {1e39, -1e39, 3.5e38, 1e300, -1e300}) {
    EXPECT(attend(x) == PACE_EINVAL);
    EXPECT(rotate(x) == PACE_EINVAL);
  }
  EXPECT(attend(2.4e38) == PACE_EINVAL);   // finite itself, not as the base-2 factor
  EXPECT(launches == n);
  for (double x : {0.0, 1e-300, -0.125, 2.3e38}) EXPECT(attend(x) == PACE_OK && std::isfinite(at.scale_log2e));
  for (double x : {0.0, 1e-300, -1.0, 3.4e38}) EXPECT(rotate(x) == PACE_OK && std::isfinite(rot.back().magnitude));
}

// A launch holds fewer than 2^32 threads: longer calls are cut or refused before any launch.
static void launch_sizes() {
  for (int wide : {0, 1})
    for (int n : {1, 8191, 8192, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 24) + 3, (1 << 26) + 5, INT_MAX}) {
      pace_rotary_cfg r{1, 1, wide ? 16 : 2, wide ? 16 : 2, 0, PACE_IO_BF16};
      const int64_t s = wide ? 16 : 5;
      rot.clear();
      char *q = (char*)((uintptr_t)1 << 40), *k = (char*)((uintptr_t)1 << 41), *qo = (char*)((uintptr_t)1 << 42);
      EXPECT(pace_rotary(&r, n, I, (const double*)I, 1.0, 0, q, s, k, s, qo, s, k, s, nullptr) == PACE_OK);
      int64_t done = 0;
      for (const RotaryParams& p : rot) {
        EXPECT(p.n > 0 && (int64_t)p.n * 256 < (INT64_C(1) << 32));
        EXPECT(p.positions == I + done && p.q == q + done * s * 2 && p.q_out == qo + done * s * 2);
        EXPECT(p.k == k + done * s * 2 && p.k_out == p.k && p.copy_q == 1 && p.copy_k == 0);
        done += p.n;
      }
      EXPECT(done == n);
    }
  pace_cache_cfg c{};
  c.B = 65535; c.Hq = 1024; c.Hkv = 1024; c.d = 64; c.kind = PACE_CACHE_INT4; c.group = 64; c.page = 16;
  c.num_pages = 64; c.max_pages = 64; c.io_dtype = PACE_IO_BF16;
  auto io_call = [&](int T) {
    const pace_status a = pace_cache_write(&c, X, I, I, T, X, 65536, X, 65536, nullptr);
    EXPECT(pace_cache_read(&c, X, I, I, T, X, 65536, X, 65536, nullptr) == a);
    return a;
  };
  auto attend = [&](int T) {
    size_t need = 1;
    const pace_status a = pace_cache_attention_workspace_bytes(&c, T, 64, &need);
    EXPECT(pace_cache_attention(&c, X, I, X, 65536, T, I, nullptr, nullptr, 0, 0.1, 64, X, nullptr, X, need, nullptr) == a);
    return a;
  };
  EXPECT(io_call(1) == PACE_OK && io_call(15) == PACE_OK && io_call(16) == PACE_EUNSUPPORTED);
  EXPECT(attend(1) == PACE_EUNSUPPORTED);
  c.B = 16383;
  EXPECT(attend(1) == PACE_OK && attend(16) == PACE_OK && attend(17) == PACE_EUNSUPPORTED);   // rows by 16
  c.B = 16384;
  EXPECT(attend(1) == PACE_EUNSUPPORTED);
  c.B = 1; c.Hq = c.Hkv = 8;
  EXPECT(io_call(INT_MAX) == PACE_EUNSUPPORTED && io_call(1 << 26) == PACE_OK);
}

int main() {
  plans();
  strides();
  factors();
  launch_sizes();
  if (fails) return printf("%d failures\n", fails), 1;
  printf("OK %ld\n", checks);
  return 0;
}
