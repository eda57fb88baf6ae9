// Host entry points of the operators that serve drafted tokens (csrc/pace_draft.cpp) over random and extreme arguments,
// built for the CPU with AddressSanitizer and UndefinedBehaviorSanitizer and linked against recording stand-ins of the
// kernel launchers.  Built and run by tests/test_draft_sanitized.py; prints "OK <checks>" on success.
#include <climits>
#include <cstdio>
#include <random>
#include <vector>

#include "../../bit_recurrent_state_amd/csrc/pace_cache_internal.h"
#include "../../bit_recurrent_state_amd/csrc/pace_draft_internal.h"

using namespace pace;

static int fails = 0;
static long checks = 0;
#define EXPECT(c)                                        \
  do {                                                   \
    ++checks;                                            \
    if (!(c) && fails++ < 30) printf("FAIL line %d: %s\n", __LINE__, #c); \
  } while (0)

namespace pace {
static int launches = 0, folds = 0;
static hipError_t answer = hipSuccess;
static std::vector<CommitParams> appended;
static DraftParams step_p;
static VerifyParams verify_p;
static MoveParams move_p;
static DecodeParams fold_p;
hipError_t launch_draft_step(const DraftParams& p, int, int, hipStream_t) { ++launches; step_p = p; return answer; }
hipError_t launch_draft_append(const CommitParams& p, int, int, hipStream_t) { ++launches; appended.push_back(p); return answer; }
hipError_t launch_draft_verify(const VerifyParams& p, int, hipStream_t) { ++launches; verify_p = p; return answer; }
hipError_t launch_cache_move(const MoveParams& p, int, int, int, hipStream_t) { ++launches; move_p = p; return answer; }
hipError_t launch_decode(const DecodeParams& p, const SeqOrder*, int, int, int, hipStream_t) { ++folds; fold_p = p; return answer; }
hipError_t launch_prefill(const PrefillParams&, int, int, int, hipStream_t) { return hipErrorUnknown; }
size_t prefill_workspace_bytes(int, int, int, int, int, int) { return 0; }
hipError_t launch_bf16_decode(const Bf16Params&, int, int, int, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_calib(const CalibParams&, int, int, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_rotary(const RotaryParams&, int, bool, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_cache_write(const CacheIoParams&, int, int, int, int, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_cache_read(const CacheIoParams&, int, int, int, int, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_attention(const AttnParams&, const AttnPlan&, int, int, int, int, hipStream_t) { return hipErrorUnknown; }
}  // namespace pace

static void* const X = (void*)0x100000;
static const int32_t* const I = (const int32_t*)0x200000;
static int32_t* const O = (int32_t*)0x300000;
static const float* const F = (const float*)0x400000;
static const uint32_t* const U = (const uint32_t*)0x500000;
static std::mt19937 rng(5);
static int pick(const std::vector<int>& v) { return v[rng() % v.size()]; }
static const std::vector<int> ends = {INT_MIN, INT_MIN + 1, -1, 0, 1, 2, 63, 64, 65, 1024, 1025, 65535, 65536, 1 << 24, (1 << 24) + 1, 1 << 30, INT_MAX};

static pace_layer_cfg layer() {
  pace_layer_cfg c{};
  c.B = pick({1, 3, 65535}); c.Hk = pick({1, 4, 16}); c.Hv = c.Hk * pick({1, 2, 4});
  c.dk = c.dv = pick({64, 128}); c.group = pick({32, 64}); c.dP = pick({1, 8, 32}); c.chunk = 64;
  c.buf_kind = rng() % 2 ? PACE_BUF_INT8 : PACE_BUF_K4_VBF16; c.io_dtype = rng() % 2;
  return c;
}

// What is taken fits the launch; everything else is refused, whatever the sizes, with nothing launched.
static void layers() {
  for (int trial = 0; trial < 4000; ++trial) {
    const pace_layer_cfg c = layer();
    const int T = rng() % 2 ? 1 + (int)(rng() % 64) : pick(ends), most = rng() % 2 ? 1 + (int)(rng() % 64) : pick(ends);
    const int64_t stride = rng() % 4 ? (int64_t)(rng() % 1000) : (int64_t)(rng() | (uint64_t)rng() << 32);
    const bool fits = T >= 1 && T <= kMaxDrafts;
    int before = launches;
    pace_status st = pace_draft_step(&c, X, X, X, X, X, F, F, T, I, U, stride, X, nullptr);
    EXPECT((st == PACE_OK) == (launches == before + 1));
    EXPECT((st == PACE_OK) == (fits && stride >= 0 && stride <= (INT64_C(1) << 46) / c.B));
    if (st == PACE_OK) {
      EXPECT(step_p.T == T && step_p.tree_stride == stride);
      EXPECT(draft_tiles(c.dP, T) >= 1 && draft_tiles(c.dP, T) <= 6 && 16 * draft_tiles(c.dP, T) >= c.dP - 1 + T);
    }
    size_t need = 7;
    st = pace_draft_commit_workspace_bytes(&c, most, &need);
    EXPECT((st == PACE_OK) == (most >= 1 && most <= kMaxDrafts));
    if (st != PACE_OK) {
      EXPECT(need == 7);
      need = 1 << 30;
    }
    before = launches;
    const int rounded = folds;
    appended.clear();
    st = pace_draft_commit(&c, X, X, X, X, F, F, T, I, I, most, X, need, nullptr);
    EXPECT((st == PACE_OK) == (fits && most >= 1 && most <= T));
    const int rounds = st == PACE_OK ? (most + c.dP - 1) / c.dP : -1;
    EXPECT(launches - before == rounds + 1 && folds - rounded == (st == PACE_OK ? rounds : 0));
    // every launch reads what the one before wrote, and all lists lie in the workspace
    for (size_t r = 0; r < appended.size(); ++r) {
      EXPECT(appended[r].done == (r ? appended[r - 1].done_out : nullptr));
      EXPECT((char*)(appended[r].done_out + (size_t)c.B * c.Hv) <= (char*)X + need);
    }
    if (st == PACE_OK && rounds > 0) EXPECT(fold_p.flush_only == 2);
    if (st == PACE_OK) EXPECT(pace_draft_commit(&c, X, X, X, X, F, F, T, I, I, most, X, need - 1, nullptr) == PACE_EINVAL);
  }
}

static void verification() {
  for (int trial = 0; trial < 4000; ++trial) {
    pace_verify_cfg c{rng() % 3 ? 1 + (int)(rng() % 65535) : pick(ends), rng() % 3 ? 1 + (int)(rng() % 1024) : pick(ends),
                      rng() % 3 ? 1 + (int)(rng() % (1 << 24)) : pick(ends), (int)(rng() % 2)};
    size_t need = 7;
    const bool ok = c.B >= 1 && c.T >= 1 && c.V >= 1 && c.B <= 65535 && c.T <= 1024 && c.V <= 1 << 24;
    EXPECT((pace_draft_verify_workspace_bytes(&c, &need) == PACE_OK) == ok);
    EXPECT(ok || need == 7);
    const int64_t ts = rng() % 2 ? c.V : (int64_t)(rng() | (uint64_t)rng() << 32), ds = rng() % 2 ? c.V : (int64_t)rng();
    const int64_t ps = rng() % 2 ? c.T : (int64_t)(rng() | (uint64_t)rng() << 32);
    const bool drawn = rng() % 2;
    const int before = launches;
    const pace_status st = pace_draft_verify(&c, X, ts, drawn ? X : nullptr, ds, I, I, ps, F, I, O, O, O, X, need, nullptr);
    EXPECT((st == PACE_OK) == (launches == before + 1));
    if (!ok) {
      EXPECT(st != PACE_OK);
      continue;
    }
    if (st == PACE_OK) {
      // the last row's end and every part of the workspace
      EXPECT((__int128)ts * c.B * c.T <= (__int128)1 << 48 && (__int128)ps * c.B <= (__int128)1 << 46);
      EXPECT((size_t)verify_p.scratch * c.B <= need && verify_p.scratch >= verify_p.chunks * 8 + 48 + 8 * (int64_t)c.T);
      EXPECT((int64_t)verify_p.chunks * kVerifyChunk >= c.V && (int64_t)(verify_p.chunks - 1) * kVerifyChunk < c.V);
      EXPECT(pace_draft_verify(&c, X, ts, drawn ? X : nullptr, ds, I, I, ps, F, I, O, O, O, X, need - 1, nullptr) == PACE_EINVAL);
    }
  }
}

static void moves() {
  for (int trial = 0; trial < 4000; ++trial) {
    pace_cache_cfg c{};
    c.B = pick({1, 2, 1000, 65535}); c.Hkv = pick({1, 2, 8, 1024}); c.Hq = c.Hkv; c.d = pick({64, 128, 256});
    c.kind = rng() % 3; c.group = pick({32, 64}); c.page = pick({16, 64, 1024}); c.num_pages = 1 + rng() % 100000;
    c.max_pages = 1 + rng() % 20000; c.io_dtype = rng() % 2;
    const int T = rng() % 2 ? 1 + (int)(rng() % (1 << 30)) : pick(ends);
    const bool with = rng() % 2;
    const int64_t stride = rng() % 2 ? (int64_t)T : (int64_t)(rng() | (uint64_t)rng() << 32);
    const int before = launches;
    const pace_status st = pace_cache_move(&c, X, I, I, I, with ? I : nullptr, stride, I, T, nullptr);
    const bool ok = T >= 0 && T <= kMaxMoved && (T == 0 || !with || (stride >= T && stride <= (INT64_C(1) << 46) / c.B));
    EXPECT((st == PACE_OK) == ok);
    EXPECT(launches - before == (ok && T > 0 ? 1 : 0));
    if (ok && T > 0) EXPECT((1 << move_p.page_shift) == c.page && move_p.T == T);
  }
}

// An error of a launch is reported, and nothing is launched behind it.
static void errors() {
  const pace_layer_cfg c = layer();
  answer = hipErrorUnknown;
  const int before = launches, rounded = folds;
  EXPECT(pace_draft_commit(&c, X, X, X, X, F, F, 9, I, I, 9, X, 1 << 30, nullptr) == PACE_EHIP);
  EXPECT(launches == before + 1 && folds == rounded);
  EXPECT(pace_draft_step(&c, X, X, X, X, X, F, F, 9, nullptr, nullptr, 0, X, nullptr) == PACE_EHIP);
  const pace_verify_cfg v{2, 3, 100, 0};
  EXPECT(pace_draft_verify(&v, X, 100, nullptr, 0, I, nullptr, 0, F, nullptr, O, O, O, X, 1 << 20, nullptr) == PACE_EHIP);
  answer = hipSuccess;
}

int main() {
  layers();
  verification();
  moves();
  errors();
  if (fails) {
    printf("%d of %ld failed\n", fails, checks);
    return 1;
  }
  printf("OK %ld\n", checks);
  return 0;
}
