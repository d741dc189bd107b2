// Host-side argument validation and launch planning of the gated delta rule (pure C++, no HIP).
#include "delta_plan.h"

#include <algorithm>
#include <cmath>

#include "decay_slots.h"
#include "layer_plan.h"
#include "plan.h"

namespace kata {

namespace {

kata_status fail(std::string* why, kata_status s, const std::string& msg) {
  if (why) *why = msg;
  return s;
}

// most: sequences that the form takes.
kata_status check_delta_problem(const kata_delta_problem* pr, int most, bool backward, std::string* why) {
  if (!pr) return fail(why, KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  if (pr->n_seq < 1 || pr->H < 1 || pr->Hk < 1 || pr->T < 1)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "n_seq, H, Hk and T must be >= 1");
  if (pr->T > kMaxT) return fail(why, KATA_ERR_UNSUPPORTED, "T exceeds 2^26");
  if (pr->n_seq > most || pr->H > kDecayMaxHeads)
    return fail(why, KATA_ERR_UNSUPPORTED, "n_seq or H exceeds 65535");
  if (pr->H % pr->Hk) return fail(why, KATA_ERR_INVALID_ARGUMENT, "H must be a multiple of Hk");
  if (pr->dtype != KATA_F32 && pr->dtype != KATA_BF16)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "dtype must be fp32 or bf16");
  if (pr->packed != 0 && pr->packed != 1)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "packed must be 0 or 1");
  if (pr->dk < 1 || pr->dv < 1)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "dk and dv must be >= 1");
  const int V = pr->dtype == KATA_BF16 ? 8 : 4;
  if (pr->dk > kDecayMaxWidth || pr->dv > kDecayMaxWidth || pr->dk % V || pr->dv % V)
    return fail(why, KATA_ERR_UNSUPPORTED,
                "dk and dv must be at most 128 and a multiple of 16 bytes");
  if (!std::isfinite(pr->scale)) return fail(why, KATA_ERR_INVALID_ARGUMENT, "scale must be finite");
  const int64_t B = pr->packed ? 1 : pr->n_seq;
  const int64_t sizes[3] = {B, pr->T, pr->H}, shared[3] = {B, pr->T, pr->Hk};
  kata_status s;
  if ((s = check_strides("q", pr->sq, shared, pr->dk, false, why)) != KATA_OK) return s;
  if ((s = check_strides("k", pr->sk, shared, pr->dk, false, why)) != KATA_OK) return s;
  if ((s = check_strides("v", pr->sv, sizes, pr->dv, false, why)) != KATA_OK) return s;
  if ((s = check_strides("beta", pr->sbeta, sizes, 1, false, why)) != KATA_OK) return s;
  if ((s = check_strides("log_decay", pr->sdecay, sizes, 1, false, why)) != KATA_OK) return s;
  if (backward) return check_strides("dO", pr->sdo, sizes, pr->dv, false, why);
  return check_strides("o", pr->so, sizes, pr->dv, true, why);
}

static_assert(kDecayChunk == kDeltaChunk, "one chunk for both layers' slots");
constexpr size_t kVecBytes = kDeltaVec * 4, kInvBytes = kInvFloats * 4;   // of a chunk and head

}  // namespace

kata_status validate_delta(const kata_delta_problem* pr, bool backward, std::string* why) {
  return check_delta_problem(pr, kDecayMaxSeqs, backward, why);
}

kata_status validate_delta_decode(const kata_delta_problem* pr, std::string* why) {
  const kata_status s = check_delta_problem(pr, INT32_MAX, false, why);
  if (s == KATA_OK && pr->packed) return fail(why, KATA_ERR_INVALID_ARGUMENT, "decode takes no packed sequences");
  return s;
}

DeltaPlan plan_delta(const kata_delta_problem* pr, bool backward) {
  DeltaPlan p;
  const bool bf16 = pr->dtype == KATA_BF16;
  const int64_t chunks = (int64_t(pr->T) + kDecayChunk - 1) / kDecayChunk;
  const int cols = decay_columns(bf16, pr->dv);
  const int64_t v_blocks = (pr->dv + cols - 1) / cols, k_blocks = (pr->dk + cols - 1) / cols;
  // Segments that a sequence (packed: all tokens together) is cut into to fill the card.  Of the bf16 walks of heads of
  // up to 64 two workgroups fit on a CU, of the others one: 131072 tokens of 16 heads of 64 take 1040 us in 512
  // segments and 1275 in 256, 4 x 16384 of 16 heads of 128 1278 in 256 and 1350 in 512.  Backward both directions
  // run side by side; where whole sequences fill the CUs once they stay whole (8 x 4096, 16 heads of 64: 1025 us, cut
  // in two 1164; 4 x 4096: cut into four 655, into two 729).
  const int64_t units = pr->H * v_blocks * (backward ? 2 : 1) * (pr->packed ? 1 : pr->n_seq);
  const int64_t fill = bf16 && pr->dk <= 64 && pr->dv <= 64 && !(backward && units >= 256) ? 512 : 256;
  const int64_t want = std::max<int64_t>(1, fill / units);
  // A cut costs two more launches, and a step of the join for each segment: a sequence of up to six chunks stays whole
  // (256 tokens 31 us, cut 38; 512 tokens 44 cut, 48 whole), and few chunks are cut into segments of about half their
  // number's square root, four at most (1024 tokens: segments of 2 51 us, of 4 59; 2048: of 3 64, of 2 or 4 66;
  // 4096: of 4 83, of 2 101).
  int64_t least = 1;
  while (least < 4 && 4 * least * least < chunks) ++least;
  const int64_t L = chunks <= 6 ? chunks : std::max(least, (chunks + want - 1) / want);
  p.L = int(L);
  p.n_chunks = int(chunks);
  const int64_t SL = L * kDecayChunk;
  p.n_seg = int((chunks + L - 1) / L);
  p.n_slots = pr->packed ? decay_slot_count(pr->T, pr->n_seq, int(SL)) : pr->n_seq * p.n_seg;
  p.c_slots = pr->packed ? decay_slot_count(pr->T, pr->n_seq, kDecayChunk) : int(std::min<int64_t>(pr->n_seq * chunks, INT32_MAX));
  const int64_t H = pr->H;
  p.groups = std::max<int64_t>((pr->packed ? int64_t(p.c_slots) : pr->n_seq * chunks) * H,
                               (int64_t(p.n_slots) * H + 7) / 8 * 8 * (2 * v_blocks + k_blocks + 1));
  size_t at = 0;
  const auto part = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~size_t(255);
    return here;
  };
  const size_t c = size_t(p.c_slots) * H, s = size_t(p.n_slots) * H, state = size_t(pr->dk) * pr->dv * 4;
  p.vec = part(c * kVecBytes);
  p.inv = part(c * kInvBytes);
  if (p.n_seg > 1) {
    p.sums = part(s * state);
    p.trans = part(s * pr->dk * pr->dk * 4);
  }
  if (backward) {
    if (p.n_seg > 1) p.rsums = part(s * state);
    const size_t rows = delta_state_rows(bf16, pr->dk), tiles = (pr->dv + kTileColumns - 1) / kTileColumns;
    const size_t chunk_state = rows * kTileColumns * tiles * 4, chunk_u = kDeltaChunk * kTileColumns * tiles * 4;
    p.cstates = part(c * chunk_state);
    p.rstates = part(c * chunk_state);
    p.u = part(c * chunk_u);
    p.x = part(c * chunk_u);
    // Few chunks and heads of q and k leave CUs idle: each value head by itself, then their sums (2 x 1001 tokens, three
    // fp32 heads of 40 and 72 on one of q and k: 78 us, the heads by themselves 31 and 5 for the sums).
    p.by_heads = pr->H > pr->Hk && int64_t(p.c_slots) * pr->Hk < kDeltaGradBlocks;
    if (p.by_heads) {
      const size_t heads = size_t(pr->packed ? 1 : pr->n_seq) * pr->T * H * pr->dk * 4;
      p.pq = part(heads);
      p.pk = part(heads);
    }
    p.fstates = part(size_t(pr->n_seq) * H * chunk_state);
  }
  p.bytes = at;
  return p;
}

}  // namespace kata
