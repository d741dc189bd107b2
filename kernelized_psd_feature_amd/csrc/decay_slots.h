// What the planner, the kernels and the planner's CPU test share.
//
// Sequence i with first row `first` takes the slots from first / SL + i on (SL rows a segment).
// With ascending first rows c_0 <= c_1 <= ... the next sequence's first slot is
//     floor(c_{i+1} / SL) + i + 1 >= floor(c_i / SL) + i + ceil((c_{i+1} - c_i) / SL)
// and at least one more, so every sequence has room for its segments without any sum over the
// lengths; T rows and n sequences, and one more for the rows behind them, need
// floor(T / SL) + n + 1 slots.
#pragma once

#ifdef __HIP__
#include <hip/hip_runtime.h>
#define KATA_HD __host__ __device__ inline
#else
#define KATA_HD inline
#endif

namespace kata {

KATA_HD int decay_first_slot(int first, int i, int SL) { return first / SL + i; }
KATA_HD int decay_slot_count(int T, int n_seq, int SL) { return T / SL + n_seq + 1; }

// Value columns of a workgroup, 16 a wave: four waves, or eight that share the staged rows and the
// scores of a wider head.
KATA_HD int decay_columns(bool bf16, int dv) { return bf16 && dv > 64 ? 128 : 64; }

}  // namespace kata
