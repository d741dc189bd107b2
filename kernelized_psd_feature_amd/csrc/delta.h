// Arguments of the gated delta rule's kernels (delta.hip, delta_bwd.hip) and of their launchers.
#pragma once

#include <hip/hip_runtime.h>

namespace kata {

// The sequences of a call and how they are cut: chunks of 64 tokens, segments of L chunks.  A chunk
// slot holds what a chunk keeps in the workspace, a segment slot a segment's; batch form: sequence *
// n_chunks + chunk and sequence * n_seg + segment, packed form: decay_slots.h.
struct DeltaMap {
  const int* cu;                          // packed: [n_seq + 1] first rows of the sequences
  int packed, n_seq, T;
  int H, Hk;                              // heads of v, beta, log_decay and o; of q and k
  int dk, dv;
  int L, n_seg, n_chunks;                 // chunks of a segment; batch form: segments and chunks of a sequence
  int n_slots, c_slots;                   // segment slots and chunk slots over all sequences
};

struct DeltaArgs {
  DeltaMap m;
  const void *q, *k, *v, *beta, *dO;
  const float* log_decay;                 // null: no decay
  void* o;
  long long sq[3], sk[3], sv[3], so[3], sdo[3], sb[3], sl[3];   // element strides of (b, t, h)
  float scale;
  int zero_tail;
  // workspace
  float* vec;                             // [c_slots][H][kDeltaVec]
  float* inv;                             // [c_slots][H][kInvFloats] inverses
  float* sums;                            // [n_slots][H][dk][dv] sums of the segments, then their entry states
  float* trans;                           // [n_slots][H][dk][dk] transitions of the segments
  float* rsums;                           // backward: [n_slots][H][dk][dv], the same of the gradient of the state
  float* cstates;                         // backward: [c_slots][H][DK][DV] entry states of the chunks, in registers' order
  float* rstates;                         // backward: the gradient of the state behind each chunk
  float *pq, *pk;                         // backward, or null: [b][t][H][dk], dq and dk by value heads
  float *u, *x;                           // backward: [c_slots][H][DV][64] U of the chunks, and X (dv = b X), in registers' order
  float* fstates;                         // bf16 backward with dfin, or null: [n_seq][H], as cstates, the final states
  // states
  const float *init, *dfin;               // [n_seq][H][dk][dv] or null
  float *fin, *dinit;
  // gradients, contiguous [b][t][heads][width]
  void *dq, *dk, *dv, *dbeta;
  float* dlog;
};

hipError_t launch_delta_prep(const DeltaArgs& a, bool bf16, hipStream_t st);
// The segments' sums and transitions; their sums become entry states; the outputs.
hipError_t launch_delta_segments(const DeltaArgs& a, bool bf16, hipStream_t st);
hipError_t launch_delta_join(const DeltaArgs& a, bool backward, hipStream_t st);
hipError_t launch_delta_walk(const DeltaArgs& a, bool bf16, hipStream_t st);
// Backward: the states before every chunk and the gradients of the states behind them (sums: the segments'
// sums of both, and the transitions); then the gradients.
hipError_t launch_delta_bwd_walk(const DeltaArgs& a, bool bf16, bool sums, hipStream_t st);
hipError_t launch_delta_grads(const DeltaArgs& a, bool bf16, hipStream_t st);
hipError_t launch_delta_decode(const DeltaArgs& a, bool bf16, float* state, hipStream_t st);

}  // namespace kata
