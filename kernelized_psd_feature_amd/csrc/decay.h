// Arguments of the decayed linear attention kernels (decay.hip) and of their launchers.
#pragma once

#include <hip/hip_runtime.h>

namespace kata {

// One recurrence over the tokens of every sequence, in the role's own time order (rev: last
// token first):
//     out_t = out_scale ( g^t a_t . E + kv_scale sum_{s<=t} g^(t-s) (a_t . b_s) c_s )
// where E is the entry state, that is the state before the first token already decayed to it
// (forward: g times the initial state; reversed: the given state itself).  The forward pass is
// (a, b, c) = (q, k, v); the gradients are the same form with other operands:
//     dq: (dO, v, k) forward,  dk: (v, dO, q) reversed,  dv: (k, q, dO) reversed.
struct DecayRole {
  const void *a, *b, *c;
  void* out;
  long long sa[3], sb[3], sc[3], so[3];   // element strides of (b, t, h)
  const float* init;                      // [n_seq][H][dk][dv] (trans: [dv][dk]) or null
  float* fin;                             // [n_seq][H][dk][dv] or null: the state behind the last token
  float* states;                          // workspace [n_slots][H][dk][dv]
  int dk, dv;                             // widths of a and b, and of c and out
  int init_trans, rev;
  float out_scale, kv_scale;
};

struct DecayArgs {
  DecayRole role[3];
  const float* log_decay;                 // [H]
  const int* cu;                          // packed: [n_seq + 1] first rows of the sequences
  int n_roles, n_seq, H, T;
  int packed, zero_tail;
  int stream;                             // q, k and v are loaded past the caches
  int L;                                  // chunks of 64 tokens in a segment
  int n_seg;                              // batch form: segments of a sequence
  int n_slots;                            // segment slots over all sequences
  int blocks;                             // value-column blocks, those of all roles
  int scan;                               // a state pass runs before the walk, and then the scan, which writes fin
  int join;                               // with scan: no scan kernel, the walk adds the sums itself and writes fin
};

// exact_state: the terms of fin are added without rounding a factor to bf16.
// state_pass: only the sums over each sequence's segments, into role.states (the last one's where
// fin is wanted).
hipError_t launch_decay_chunks(DecayArgs& a, bool bf16, bool exact_state, bool state_pass,
                               hipStream_t st);
// The segments' sums in role.states become their entry states, and fin is written.
hipError_t launch_decay_scan(const DecayArgs& a, hipStream_t st);
hipError_t launch_decay_decode(bool bf16, int B, int T, int H, int dk, int dv,
                               const long long sq[3], const long long sk[3],
                               const long long sv[3], const long long so[3], const void* q,
                               const void* k, const void* v, const float* log_decay,
                               float scale, float* state, void* o, hipStream_t st);

}  // namespace kata
