// Host-side argument validation and launch planning of the decayed linear attention, the rotary
// positions and the layer norm.  Pure C++ (no HIP), like plan.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include "kata.h"

namespace kata {

constexpr int kDecayChunk = 64;           // tokens of a chunk
constexpr int kDecayMaxWidth = 128;       // dk and dv
constexpr int kDecayMaxHeads = 65535;
constexpr int kDecayMaxSeqs = 65535;      // of the chunked forms

// Segments of the chunked form (see decay.hip).
struct DecayPlan {
  int L = 1;                              // chunks of a segment
  int n_seg = 1;                          // batch form: segments of a sequence
  int n_slots = 1;                        // segment slots over all sequences
  int scan = 0;                           // 1: a state pass and a scan run before the walk
  int stream = 0;                         // 1: q, k and v are loaded past the caches
  int join = 0;                           // 1: the walk does the scan's work itself
  int64_t groups = 1;                     // workgroups of a chunk launch
  size_t role_bytes = 0;                  // workspace of one role's segment states
};

kata_status validate_decay(const kata_decay_problem* pr, bool backward, std::string* why);
kata_status validate_decay_decode(const kata_decay_problem* pr, std::string* why);
// A tensor's pointer and (b, t, h) strides: 16-byte aligned rows.  The stride of an axis of one
// entry means nothing.
kata_status validate_rows(const void* p, const int64_t st[3], const int64_t sizes[3], size_t esize,
                          const char* name, std::string* why);
// pr must have passed validate_decay.
DecayPlan plan_decay(const kata_decay_problem* pr, int n_roles);

kata_status validate_rotary(const kata_rotary_problem* pr, std::string* why);
// The strides of the gradients' rows count in the backward pass only.
kata_status validate_norm(const kata_norm_problem* pr, bool backward, std::string* why);
// Workgroups whose partial sums of dw and db the backward pass keeps at most: of rows in registers, and
// of wider ones than kNormInRegisters elements (layer_norm.hip).
constexpr int kNormBlocks = 768, kNormLoopBlocks = 64, kNormInRegisters = 8192;
size_t norm_workspace_bytes(const kata_norm_problem* pr);

}  // namespace kata
