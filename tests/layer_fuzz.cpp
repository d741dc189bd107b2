// Host fuzz driver for csrc/layer_plan.cpp, built by tests/test_layer_cpu.py with g++ and the address
// and undefined-behaviour sanitizers (no HIP, no GPU).
//
//   layer_fuzz <seed> <iterations>
//
// Draws decay problems over their ranges, their edges and far beyond, checks that a refusal has a
// message and that the plan of an accepted problem is consistent, and checks the slots of packed
// sequences: for any ascending offsets no two sequences share a slot, every segment has one, and
// all lie inside the planned count; for arbitrary offsets, clamped as in the kernels, every
// segment's slot still lies inside.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <string>
#include <vector>

#include "decay_slots.h"
#include "kata.h"
#include "layer_plan.h"

namespace {
uint64_t g_state;
uint64_t next_u64() {
  uint64_t z = (g_state += 0x9e3779b97f4a7c15ull);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  return z ^ (z >> 31);
}
int64_t uniform(int64_t lo, int64_t hi) { return lo + int64_t(next_u64() % uint64_t(hi - lo + 1)); }
int64_t log_uniform(int64_t hi) {
  int64_t x = hi;
  for (uint64_t n = next_u64() % 24; n; --n) x /= 2;
  return uniform(1, std::max<int64_t>(1, x));
}
int32_t odd32() {
  const int32_t xs[] = {0, -1, 1, 65535, 65536, 1 << 26, (1 << 26) + 1,
                        std::numeric_limits<int32_t>::max(), std::numeric_limits<int32_t>::min()};
  return xs[next_u64() % 9];
}
#define CHECK(c)                                                    \
  do {                                                              \
    if (!(c)) {                                                     \
      std::fprintf(stderr, "FAIL %s line %d\n", #c, __LINE__);      \
      std::exit(1);                                                 \
    }                                                               \
  } while (0)

void fill(int64_t (&s)[3], int64_t T, int64_t H, int64_t w) {
  s[0] = int64_t(uint64_t(T) * uint64_t(H) * uint64_t(w));
  s[1] = H * w;
  s[2] = w;
  if (next_u64() % 8 == 0) s[next_u64() % 3] = 0;
  if (next_u64() % 50 == 0) s[next_u64() % 3] = int64_t(next_u64());
}

void slots(const kata_decay_problem& pr, const kata::DecayPlan& p) {
  const int SL = kata::kDecayChunk * p.L, n = std::min(pr.n_seq, 50);
  if (n != pr.n_seq) return;
  std::vector<int> cu(n + 1);
  for (int& x : cu) x = int(uniform(0, pr.T));
  const bool wild = next_u64() % 3 == 0;
  if (!wild) std::sort(cu.begin(), cu.end());
  if (!wild && next_u64() % 2) cu[0] = 0;
  int next_free = 0;
  for (int i = 0; i <= n; ++i) {                     // i == n: the rows behind
    const int first = cu[i], end = i < n ? cu[i + 1] : pr.T;
    const int len = std::max(end - first, 0), segs = std::max(1, (len + SL - 1) / SL);
    const int s0 = kata::decay_first_slot(first, i, SL);
    CHECK(s0 >= 0 && s0 + segs <= p.n_slots);
    if (!wild) {
      CHECK(s0 >= next_free);
      next_free = s0 + segs;
    }
  }
}
}  // namespace

int main(int argc, char** argv) {
  g_state = argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 1;
  const long n = argc > 2 ? std::strtol(argv[2], nullptr, 10) : 1000;
  long valid = 0, refused = 0;
  for (long it = 0; it < n; ++it) {
    kata_decay_problem pr{};
    pr.packed = int(next_u64() % 2);
    pr.n_seq = int(log_uniform(65535));
    pr.H = int(log_uniform(256));
    pr.T = int(log_uniform(int64_t(1) << 26));
    pr.dtype = int(next_u64() % 2);
    pr.dk = 8 * int(uniform(1, 16));
    pr.dv = 8 * int(uniform(1, 16));
    pr.scale = 0.5f;
    int32_t* fields[] = {&pr.n_seq, &pr.H, &pr.T, &pr.dk, &pr.dv, &pr.packed, &pr.dtype};
    if (next_u64() % 4 == 0) *fields[next_u64() % 7] = odd32();
    if (next_u64() % 64 == 0) pr.scale = std::numeric_limits<float>::quiet_NaN();
    fill(pr.sq, pr.T, pr.H, pr.dk);
    fill(pr.sk, pr.T, pr.H, pr.dk);
    fill(pr.sv, pr.T, pr.H, pr.dv);
    fill(pr.sdo, pr.T, pr.H, pr.dv);
    pr.so[0] = int64_t(uint64_t(int64_t(pr.T)) * uint64_t(int64_t(pr.H)) * uint64_t(int64_t(pr.dv)));
    pr.so[1] = int64_t(pr.H) * pr.dv;
    pr.so[2] = pr.dv;
    for (int backward = 0; backward < 2; ++backward) {
      std::string why;
      const kata_status s = kata::validate_decay(&pr, backward != 0, &why);
      if (s != KATA_OK) {
        CHECK(s == KATA_ERR_INVALID_ARGUMENT || s == KATA_ERR_UNSUPPORTED);
        CHECK(!why.empty());
        ++refused;
        continue;
      }
      ++valid;
      CHECK(pr.T >= 1 && pr.T <= 1 << 26 && pr.n_seq >= 1 && pr.n_seq <= 65535 && pr.H >= 1);
      CHECK(pr.dk <= 128 && pr.dv <= 128 && pr.dk * (pr.dtype ? 2 : 4) % 16 == 0);
      const kata::DecayPlan p = kata::plan_decay(&pr, backward ? 3 : 1);
      const int64_t chunks = (int64_t(pr.T) + 63) / 64;
      CHECK(p.L >= 1 && p.n_seg >= 1 && p.n_slots >= 1);
      CHECK(int64_t(p.L) * p.n_seg >= chunks && int64_t(p.L) * (p.n_seg - 1) < chunks);
      CHECK(p.scan == (p.n_seg > 1));
      if (p.scan) {
        const unsigned __int128 need = (unsigned __int128)p.n_slots * pr.H * pr.dk * pr.dv * 4;
        CHECK(p.role_bytes >= need && p.role_bytes < need + 256);
      }
      if (pr.packed) slots(pr, p);
      else CHECK(p.n_slots == int64_t(pr.n_seq) * p.n_seg);
    }
  }
  std::printf("ok %ld valid %ld refused %ld\n", n, valid, refused);
  return 0;
}
