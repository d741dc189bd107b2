// Host-side argument validation and launch planning of the gated delta rule.  Pure C++ (no HIP), like plan.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include "kata.h"

namespace kata {

constexpr int kDeltaGradBlocks = 256;     // workgroups of the gradients' kernel, one a CU

// Segments of the chunked form, and where the workspace's parts begin (delta.h).
struct DeltaPlan {
  int L = 1;                              // chunks of a segment
  int n_seg = 1, n_chunks = 1;            // batch form: segments and chunks of a sequence; packed: of all rows
  int n_slots = 1, c_slots = 1;           // segment and chunk slots over all sequences
  int64_t groups = 1;                     // workgroups of the largest launch
  size_t vec = 0, inv = 0, sums = 0, trans = 0, rsums = 0, cstates = 0, rstates = 0, u = 0, x = 0, fstates = 0, pq = 0, pk = 0;
  bool by_heads = false;                  // backward: dq and dk by value heads first
  size_t bytes = 0;
};

kata_status validate_delta(const kata_delta_problem* pr, bool backward, std::string* why);
kata_status validate_delta_decode(const kata_delta_problem* pr, std::string* why);
// pr must have passed validate_delta.
DeltaPlan plan_delta(const kata_delta_problem* pr, bool backward);

}  // namespace kata
