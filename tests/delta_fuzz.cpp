// Host fuzz driver for csrc/delta_plan.cpp, built by tests/test_delta_cpu.py with g++ and the address and
// undefined-behaviour sanitizers (no HIP, no GPU).
//
//   delta_fuzz <seed> <iterations>
//
// Draws problems over their ranges, their edges and far beyond, checks that a refusal has a message and that
// the plan of an accepted problem is consistent: segments cover the chunks, the workspace's parts hold what
// the kernels put there and do not overlap, and for packed sequences (ascending offsets, and arbitrary ones,
// clamped as in the kernels) every segment's and every chunk's slot lies inside the planned count.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <string>
#include <vector>

#include "decay_slots.h"
#include "delta_plan.h"
#include "kata.h"

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

// Segments and chunks of packed sequences; SL: rows of a part, n_slots: the planned count.
void slots(const kata_delta_problem& pr, int SL, int n_slots, const std::vector<int>& cu, bool wild) {
  int next_free = 0;
  for (int i = 0; i <= pr.n_seq; ++i) {              // i == n_seq: the rows behind
    const int first = cu[i], end = i < pr.n_seq ? cu[i + 1] : pr.T;
    const int len = std::max(end - first, 0), parts = std::max(1, (len + SL - 1) / SL);
    const int s0 = kata::decay_first_slot(first, i, SL);
    CHECK(s0 >= 0 && s0 + parts <= n_slots);
    if (!wild) {
      CHECK(s0 >= next_free);
      next_free = s0 + parts;
    }
  }
}
}  // namespace

int main(int argc, char** argv) {
  g_state = argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 1;
  const long n = argc > 2 ? std::strtol(argv[2], nullptr, 10) : 1000;
  long valid = 0, refused = 0;
  for (long it = 0; it < n; ++it) {
    kata_delta_problem pr{};
    pr.packed = int(next_u64() % 2);
    pr.n_seq = int(log_uniform(65535));
    pr.Hk = int(log_uniform(64));
    pr.H = int(std::min<int64_t>(256, pr.Hk * log_uniform(8)));
    pr.T = int(log_uniform(int64_t(1) << 26));
    pr.dtype = int(next_u64() % 2);
    pr.dk = 8 * int(uniform(1, 16));
    pr.dv = 8 * int(uniform(1, 16));
    pr.scale = 0.5f;
    int32_t* fields[] = {&pr.n_seq, &pr.H, &pr.Hk, &pr.T, &pr.dk, &pr.dv, &pr.packed, &pr.dtype};
    if (next_u64() % 4 == 0) *fields[next_u64() % 8] = odd32();
    if (next_u64() % 64 == 0) pr.scale = std::numeric_limits<float>::quiet_NaN();
    fill(pr.sq, pr.T, pr.Hk, pr.dk);
    fill(pr.sk, pr.T, pr.Hk, pr.dk);
    fill(pr.sv, pr.T, pr.H, pr.dv);
    fill(pr.sdo, pr.T, pr.H, pr.dv);
    fill(pr.sbeta, pr.T, pr.H, 1);
    fill(pr.sdecay, pr.T, pr.H, 1);
    pr.so[0] = int64_t(uint64_t(int64_t(pr.T)) * uint64_t(int64_t(pr.H)) * uint64_t(int64_t(pr.dv)));
    pr.so[1] = int64_t(pr.H) * pr.dv;
    pr.so[2] = pr.dv;
    for (int backward = 0; backward < 2; ++backward) {
      std::string why;
      const kata_status s = kata::validate_delta(&pr, backward != 0, &why);
      if (s != KATA_OK) {
        CHECK(s == KATA_ERR_INVALID_ARGUMENT || s == KATA_ERR_UNSUPPORTED);
        CHECK(!why.empty());
        ++refused;
        continue;
      }
      ++valid;
      CHECK(pr.T >= 1 && pr.T <= 1 << 26 && pr.n_seq >= 1 && pr.n_seq <= 65535 && pr.H % pr.Hk == 0);
      CHECK(pr.dk <= 128 && pr.dv <= 128 && pr.dk * (pr.dtype ? 2 : 4) % 16 == 0);
      const kata::DeltaPlan p = kata::plan_delta(&pr, backward != 0);
      const int64_t chunks = (int64_t(pr.T) + 63) / 64;
      CHECK(p.L >= 1 && p.n_seg >= 1 && p.n_slots >= 1 && p.n_chunks == chunks);
      CHECK(int64_t(p.L) * p.n_seg >= chunks && int64_t(p.L) * (p.n_seg - 1) < chunks);
      if (p.groups >= int64_t(1) << 31) continue;    // refused by the entry points
      if (!pr.packed) {
        CHECK(p.n_slots == int64_t(pr.n_seq) * p.n_seg);
        CHECK(p.c_slots == int64_t(pr.n_seq) * chunks);
      } else if (pr.n_seq <= 50) {
        std::vector<int> cu(pr.n_seq + 1);
        for (int& x : cu) x = int(uniform(0, pr.T));
        const bool wild = next_u64() % 3 == 0;
        if (!wild) std::sort(cu.begin(), cu.end());
        if (!wild && next_u64() % 2) cu[0] = 0;
        slots(pr, 64 * p.L, p.n_slots, cu, wild);
        slots(pr, 64, p.c_slots, cu, wild);
      }
      using wide = unsigned __int128;
      const wide c = (wide)p.c_slots * pr.H, seg = (wide)p.n_slots * pr.H, state = (wide)pr.dk * pr.dv * 4;
      const wide rows = pr.dk <= 32 && !pr.dtype ? 32 : pr.dk <= 64 ? 64 : 128;
      const wide chunk = rows * 16 * ((pr.dv + 15) / 16) * 4;
      struct Part {
        size_t at;
        wide bytes;
      };
      std::vector<Part> parts = {{p.vec, c * 1280}, {p.inv, c * 10240}};
      if (p.n_seg > 1) {
        parts.push_back({p.sums, seg * state});
        parts.push_back({p.trans, seg * pr.dk * pr.dk * 4});
        if (backward) parts.push_back({p.rsums, seg * state});
      }
      if (backward) {
        parts.push_back({p.cstates, c * chunk});
        parts.push_back({p.u, c * 4096 * ((pr.dv + 15) / 16)});
        parts.push_back({p.x, c * 4096 * ((pr.dv + 15) / 16)});
        parts.push_back({p.rstates, c * chunk});
        if (p.by_heads)
          for (const size_t at : {p.pq, p.pk}) parts.push_back({at, (wide)(pr.packed ? 1 : pr.n_seq) * pr.T * pr.H * pr.dk * 4});
        parts.push_back({p.fstates, (wide)pr.n_seq * pr.H * chunk});
      }
      std::sort(parts.begin(), parts.end(), [](const Part& a, const Part& b) { return a.at < b.at; });
      wide end = 0;
      for (const Part& x : parts) {
        CHECK(x.at % 256 == 0 && x.at >= end);
        end = x.at + x.bytes;
      }
      CHECK(p.bytes >= end && p.bytes < end + 256);
    }
  }
  std::printf("ok %ld valid %ld refused %ld\n", n, valid, refused);
  return 0;
}
