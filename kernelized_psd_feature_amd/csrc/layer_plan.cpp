// Host-side argument validation and launch planning (pure C++, no HIP).
#include "layer_plan.h"

#include <algorithm>
#include <cmath>

#include "decay_slots.h"
#include "plan.h"

namespace kata {

namespace {

kata_status fail(std::string* why, kata_status s, const std::string& msg) {
  if (why) *why = msg;
  return s;
}

// most: sequences that the form takes.
kata_status check_decay_problem(const kata_decay_problem* pr, int most, bool backward, std::string* why) {
  if (!pr) return fail(why, KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  if (pr->n_seq < 1 || pr->H < 1 || pr->T < 1)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "n_seq, H and T must be >= 1");
  if (pr->T > kMaxT) return fail(why, KATA_ERR_UNSUPPORTED, "T exceeds 2^26");
  if (pr->n_seq > most || pr->H > kDecayMaxHeads)
    return fail(why, KATA_ERR_UNSUPPORTED, "n_seq or H exceeds 65535");
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
  const int64_t sizes[3] = {pr->packed ? 1 : pr->n_seq, pr->T, pr->H};
  kata_status s;
  if ((s = check_strides("q", pr->sq, sizes, pr->dk, false, why)) != KATA_OK) return s;
  if ((s = check_strides("k", pr->sk, sizes, pr->dk, false, why)) != KATA_OK) return s;
  if ((s = check_strides("v", pr->sv, sizes, pr->dv, false, why)) != KATA_OK) return s;
  if (backward) return check_strides("dO", pr->sdo, sizes, pr->dv, false, why);
  if ((s = check_strides("o", pr->so, sizes, pr->dv, true, why)) != KATA_OK) return s;
  return KATA_OK;
}

}  // namespace

kata_status check_strides(const char* name, const int64_t st[3], const int64_t sizes[3], int64_t width,
                          bool output, std::string* why) {
  const int64_t kMax = int64_t(1) << 60;
  int64_t extent = width;
  for (int a = 0; a < 3; ++a) {
    const int64_t s = sizes[a] > 1 ? st[a] : 0;
    if (s < 0) return fail(why, KATA_ERR_INVALID_ARGUMENT, std::string(name) + ": negative stride");
    if (sizes[a] > 1 && s < width && (output || s != 0))
      return fail(why, KATA_ERR_INVALID_ARGUMENT,
                  std::string(name) + ": stride smaller than the row length");
    if (sizes[a] > 1 && s > (kMax - extent) / (sizes[a] - 1))
      return fail(why, KATA_ERR_INVALID_ARGUMENT,
                  std::string(name) + ": strides address more than 2^60 elements");
    if (sizes[a] > 1) extent += (sizes[a] - 1) * s;
  }
  return KATA_OK;
}

kata_status validate_rows(const void* p, const int64_t st[3], const int64_t sizes[3], size_t esize,
                          const char* name, std::string* why) {
  int64_t used[3];
  for (int a = 0; a < 3; ++a) used[a] = sizes[a] > 1 ? st[a] : 0;
  return validate_tensor(p, used, esize, name, why);
}

kata_status validate_decay(const kata_decay_problem* pr, bool backward, std::string* why) {
  return check_decay_problem(pr, kDecayMaxSeqs, backward, why);
}

kata_status validate_decay_decode(const kata_decay_problem* pr, std::string* why) {
  const kata_status s = check_decay_problem(pr, INT32_MAX, false, why);
  if (s == KATA_OK && pr->packed) return fail(why, KATA_ERR_INVALID_ARGUMENT, "decode takes no packed sequences");
  return s;
}

DecayPlan plan_decay(const kata_decay_problem* pr, int n_roles) {
  DecayPlan p;
  const int64_t chunks = (int64_t(pr->T) + kDecayChunk - 1) / kDecayChunk;
  const int wide = n_roles > 1 ? std::max(pr->dk, pr->dv) : pr->dv;
  const int cols = decay_columns(pr->dtype == KATA_BF16, wide);
  // Workgroups that the card holds at once: two of four waves a CU, or one of eight, or of four that
  // keep an fp32 state of more than 64 rows (2 x 1001, 3 heads of 128: 55 us backward, 74 with 512
  // of them, 83 with 128).  Half as many leave it idle (8 x 4096, 16 bf16 heads of width 64: 93 us
  // for 82), twice as many add segment states and their scan (103 us).
  const bool deep = pr->dtype == KATA_F32 && (n_roles > 1 ? wide : pr->dk) > 64;
  const int64_t target = cols == 128 || deep ? 256 : 512;
  const auto col_blocks = [&](int width) { return int64_t((width + cols - 1) / cols); };
  const int64_t blocks = pr->H * (n_roles > 1 ? 2 * col_blocks(pr->dk) + col_blocks(pr->dv) : col_blocks(pr->dv));
  // segments that a sequence (packed: all tokens together) is cut into to fill the card
  const int64_t want = std::max<int64_t>(1, target / (pr->packed ? blocks : blocks * pr->n_seq));
  // Short sequences stay whole, and a segment has a few chunks at least: the state pass costs a launch,
  // and the scan another.  512 tokens of 16 bf16 heads: 20 us whole, 24 in segments of 3; 1024: 25 in
  // segments of 3, 28 of 4, 34 of 8.  A chunk in fp32 takes three times as long (512 tokens of 4
  // heads: 25 us in segments of 1, 46 whole).
  const bool bf16 = pr->dtype == KATA_BF16;
  const int64_t L = chunks <= (bf16 ? 8 : 2) ? chunks
                    : std::max<int64_t>(bf16 ? 3 : 1, (chunks + want - 1) / want);
  p.L = int(L);
  const int64_t SL = L * kDecayChunk;
  p.n_seg = int((chunks + L - 1) / L);
  p.n_slots = pr->packed ? decay_slot_count(pr->T, pr->n_seq, int(SL)) : pr->n_seq * p.n_seg;
  // as the kernel deals them out: slots and heads in eights, `blocks / H` column blocks each
  p.groups = (int64_t(p.n_slots) * pr->H + 7) / 8 * 8 * (blocks / pr->H);
  p.scan = p.n_seg > 1;
  // With few segments each walk adds up the sums before its own, for one launch less.  8 x 4096, 16 bf16
  // heads (4 segments): 76 us, 81 with the scan; 2 x 16384 backward (6): 207, 214; 2048 (11): 20.3,
  // 20.7, backward 27.3, 31.1; 4096 (22): 28.9, 28.6; 8192 (32): 40.4, 36.4.
  p.join = p.scan && p.n_seg <= 12;
  // Operands that do not stay in the Infinity Cache (256 MB) until the walk reads them again are loaded
  // past it; three sets of inputs in turn, q, k, v and o together, 16 bf16 heads of width 64: 512 MB 149 us, 158 through the cache
  // (64 x 1024: 107, 121; 131072 tokens: 337, 375), 448 MB 144, 146, 384 MB 140, 137, 256 MB
  // 83, 75.  The gradients' three roles share what they read, and take it through the cache (32 x
  // 2048: 278 us, 308 past it; with only the operands of one role past it 289).
  const double rows = double(pr->T) * (pr->packed ? 1 : pr->n_seq) * pr->H;
  p.stream = n_roles == 1 && rows * 2 * (pr->dk + pr->dv) * (bf16 ? 2 : 4) > 384 * 1048576.;
  const size_t states = size_t(p.n_slots) * pr->H * pr->dk * pr->dv * 4;
  p.role_bytes = p.scan ? (states + 255) & ~size_t(255) : 0;
  return p;
}

kata_status validate_rotary(const kata_rotary_problem* pr, std::string* why) {
  if (!pr) return fail(why, KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  if (pr->B < 1 || pr->T < 1 || pr->H < 1 || pr->Hk < 0)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "B, T and H must be >= 1, Hk >= 0");
  if (pr->D < 1 || pr->rot < 0 || pr->rot > pr->D || pr->rot % 2)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "rot must be even and between 0 and D");
  if (pr->D > 1024) return fail(why, KATA_ERR_UNSUPPORTED, "D exceeds 1024");
  if (pr->H > 4096 || pr->Hk > 4096) return fail(why, KATA_ERR_UNSUPPORTED, "more than 4096 heads");
  if (int64_t(pr->B) * pr->T >= int64_t(1) << 31)
    return fail(why, KATA_ERR_UNSUPPORTED, "B*T exceeds 2^31");
  if (pr->dtype != KATA_F32 && pr->dtype != KATA_BF16)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "dtype must be fp32 or bf16");
  if (!std::isfinite(pr->magnitude))
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "magnitude must be finite");
  if (pr->pos_b < 0 || pr->pos_t < 0)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "negative stride of positions");
  const int64_t sizes[3] = {pr->B, pr->T, pr->H}, sizes_k[3] = {pr->B, pr->T, pr->Hk};
  kata_status s;
  if ((s = check_strides("q", pr->sq, sizes, pr->D, false, why)) != KATA_OK) return s;
  if ((s = check_strides("out q", pr->soq, sizes, pr->D, true, why)) != KATA_OK) return s;
  if (!pr->Hk) return KATA_OK;
  if ((s = check_strides("k", pr->sk, sizes_k, pr->D, false, why)) != KATA_OK) return s;
  return check_strides("out k", pr->sok, sizes_k, pr->D, true, why);
}

kata_status validate_qk_norm(const kata_qk_norm_problem* pr, bool backward, std::string* why) {
  if (!pr) return fail(why, KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  kata_rotary_problem r{};
  r.B = pr->B; r.T = pr->T; r.H = pr->H; r.Hk = pr->Hk; r.D = pr->D; r.rot = pr->rot;
  r.dtype = pr->dtype;
  r.magnitude = pr->magnitude;
  r.pos_b = pr->pos_b; r.pos_t = pr->pos_t;
  std::copy_n(pr->sq, 3, r.sq); std::copy_n(pr->sk, 3, r.sk);
  std::copy_n(pr->soq, 3, r.soq); std::copy_n(pr->sok, 3, r.sok);
  if (pr->D > 256) return fail(why, KATA_ERR_UNSUPPORTED, "D exceeds 256");
  kata_status s = validate_rotary(&r, why);
  if (s != KATA_OK) return s;
  if (pr->w_dtype != KATA_F32 && !(pr->w_dtype == KATA_BF16 && pr->dtype == KATA_BF16))
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "weights must be fp32, or bf16 with bf16 rows");
  if (!std::isfinite(pr->eps) || pr->eps < 0.f)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (pr->pos_a < 0) return fail(why, KATA_ERR_INVALID_ARGUMENT, "negative stride of positions");
  if (!backward) return KATA_OK;
  const int64_t sizes[3] = {pr->B, pr->T, pr->H}, sizes_k[3] = {pr->B, pr->T, pr->Hk};
  if ((s = check_strides("dq", pr->sdq, sizes, pr->D, false, why)) != KATA_OK) return s;
  return pr->Hk ? check_strides("dk", pr->sdk, sizes_k, pr->D, false, why) : KATA_OK;
}

kata_status validate_norm(const kata_norm_problem* pr, bool backward, std::string* why) {
  if (!pr) return fail(why, KATA_ERR_INVALID_ARGUMENT, "problem pointer is null");
  if (pr->rows < 1 || pr->N < 1) return fail(why, KATA_ERR_INVALID_ARGUMENT, "rows and N must be >= 1");
  if (pr->N > 1 << 24 || pr->rows > int64_t(1) << 40)
    return fail(why, KATA_ERR_UNSUPPORTED, "N exceeds 2^24 or rows 2^40");
  if (pr->dtype != KATA_F32 && pr->dtype != KATA_BF16)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "dtype must be fp32 or bf16");
  if (pr->w_dtype != KATA_F32 && !(pr->w_dtype == KATA_BF16 && pr->dtype == KATA_BF16))
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "weights must be fp32, or bf16 with bf16 rows");
  if (!std::isfinite(pr->eps) || pr->eps < 0.f)
    return fail(why, KATA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  const int64_t strides[4] = {pr->sx, pr->sy, pr->sdy, pr->sdx};
  const char* names[4] = {"x", "y", "dy", "dx"};
  for (int i = 0; i < (backward ? 4 : 2); ++i) {
    const int64_t s = strides[i];
    if (s < 0) return fail(why, KATA_ERR_INVALID_ARGUMENT, std::string(names[i]) + ": negative stride");
    if (pr->rows > 1 && s < pr->N && (i % 2 || s != 0))   // an input may repeat its row
      return fail(why, KATA_ERR_INVALID_ARGUMENT,
                  std::string(names[i]) + ": stride smaller than the row length");
    if (pr->rows > 1 && s > (int64_t(1) << 60) / pr->rows)
      return fail(why, KATA_ERR_INVALID_ARGUMENT,
                  std::string(names[i]) + ": strides address more than 2^60 elements");
  }
  return KATA_OK;
}

size_t norm_workspace_bytes(const kata_norm_problem* pr) {
  // one pair of partial rows a workgroup
  const int64_t blocks = std::min<int64_t>(pr->rows, pr->N > kNormInRegisters ? kNormLoopBlocks : kNormBlocks);
  return (size_t(blocks) * 2 * pr->N * 4 + 255) & ~size_t(255);
}

}  // namespace kata
