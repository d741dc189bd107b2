// What the gated delta rule's kernels share: where a chunk lies, what the workspace holds of it, and
// products whose operands are kept in two bf16 terms.
#pragma once

#include "decay_slots.h"
#include "delta.h"
#include "tiles.h"

namespace kata {

// Floats that a chunk and head keep in the workspace: exp(c), exp(c_63 - c), beta and c itself (double)
// of every token, c being the sum of the log decays from the chunk's first token on.
constexpr int kDeltaVec = 3 * kC + 2 * kC;

// bf16 operands that come out of fp32 sums are kept as two terms, hi + lo, which hold 2^-18 of the value:
// the recurrence passes a rounding on from chunk to chunk, and states are fp32.  fp32: one term.
template <typename T>
constexpr int kTerms = sizeof(T) == 2 ? 2 : 1;

template <typename T>
struct Op {
  typename Elem<T>::frag t[kTerms<T>];
};

__device__ __forceinline__ void split_terms(const f32x4& a, const f32x4& b, Op<__bf16>& out) {
  const uint2 x = quad(a, __bf16()), y = quad(b, __bf16());
  out.t[0] = __builtin_bit_cast(bf16x8, uint4{x.x, x.y, y.x, y.y});
  out.t[1] = pack_frag(a - unquad(x), b - unquad(y), __bf16());
}
__device__ __forceinline__ void split_terms(const f32x4& a, const f32x4& b, Op<float>& out) {
  out.t[0] = pack_frag(a, b, float());
}

// c + a b with an exact a, and with both in terms (what two second terms give is left out)
template <typename T>
__device__ __forceinline__ f32x4 mul(const typename Elem<T>::frag& a, const Op<T>& b, f32x4 c) {
#pragma unroll
  for (int i = kTerms<T> - 1; i >= 0; --i) c = mma(a, b.t[i], c);
  return c;
}
template <typename T>
__device__ __forceinline__ f32x4 mul(const Op<T>& a, const typename Elem<T>::frag& b, f32x4 c) {
#pragma unroll
  for (int i = kTerms<T> - 1; i >= 0; --i) c = mma(a.t[i], b, c);
  return c;
}
template <typename T>
__device__ __forceinline__ f32x4 mul(const Op<T>& a, const Op<T>& b, f32x4 c) {
  if constexpr (kTerms<T> == 2) {
    c = mma(a.t[1], b.t[0], c);
    c = mma(a.t[0], b.t[1], c);
  }
  return mma(a.t[0], b.t[0], c);
}

// Split slots of column i (the lane's place in its group of 16) of columns 16 tile .. of 32 rows of LD elements
// at p, whose rows are kept in split places.
template <int LD>
__device__ __forceinline__ bf16x8 split_column_frag(const __bf16* p, int tile, int lane) {
  const __bf16* at = p + (4 * (lane >> 4) + ((lane & 15) >> 2)) * LD + 32 * (tile >> 1) + 8 * (lane & 3) + 4 * (tile & 1);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * LD));
  const uint2 ul = __builtin_bit_cast(uint2, lo), uh = __builtin_bit_cast(uint2, hi);
  return __builtin_bit_cast(bf16x8, uint4{ul.x, ul.y, uh.x, uh.y});
}
template <int LD>
__device__ __forceinline__ f32x8 split_column_frag(const float* p, int tile, int lane) {
  const float* at = p + 4 * (lane >> 4) * LD + split_place(16 * tile + (lane & 15));
  f32x8 x;
#pragma unroll
  for (int r = 0; r < 8; ++r) x[r] = at[(16 * (r / 4) + r % 4) * LD];
  return x;
}

__device__ __forceinline__ f32x4 half_of(const bf16x8& x, int half) {
  const uint4 u = __builtin_bit_cast(uint4, x);
  return half ? unquad(uint2{u.z, u.w}) : unquad(uint2{u.x, u.y});
}
__device__ __forceinline__ f32x4 half_of(const f32x8& x, int half) {
  return half ? f32x4{x[4], x[5], x[6], x[7]} : f32x4{x[0], x[1], x[2], x[3]};
}

// Operands of the inverse [row tile it][K step m] (its K step 32 m .. of the columns; of the transpose the rows)
// that are not all zero, in the order in which the workspace holds them: kTerms planes of one fragment a lane.
constexpr int kInvFrags = 6;
__device__ __forceinline__ constexpr int inv_frag(int it, int m) { return it < 2 ? it : 2 * (it - 1) + m; }
__device__ __forceinline__ constexpr int inv_t_frag(int it, int m) { return it < 2 ? 2 * it + m : 2 + it; }
template <typename T>
constexpr int kInvElems = kInvFrags * kTerms<T> * 64 * 8;

template <typename T>
__device__ __forceinline__ void load_inv(const T* base, int frag, int lane, Op<T>& out) {
#pragma unroll
  for (int t = 0; t < kTerms<T>; ++t) out.t[t] = row_frag(base + ((frag * kTerms<T> + t) * 64 + lane) * 8);
}

// exp(x), the exponent held in 64 bits: its fp32 rounding would cost |x| 2^-24.
__device__ __forceinline__ float exp64(double x) {
  const double y = x * 1.4426950408889634;
  const float hi = (float)y;
  return exp2f(hi) * (1.f + 0.69314718f * (float)(y - hi));
}

// ---- sequences -------------------------------------------------------------------------------
struct DeltaPart {
  int seq, b, start, len;                 // the sequence, its batch row, first row and length
  int part;                               // which segment (chunk) of it
  int c_slot;                             // its first chunk's slot
};

__device__ __forceinline__ int cu_at(const DeltaMap& m, int i) { return min(max(m.cu[i], 0), m.T); }

// The part of `len` chunks in `slot`; false where there is none.  seq == n_seq: rows behind the last sequence.
// sh: one int of LDS.  Every thread calls it.
__device__ __forceinline__ bool find_part(const DeltaMap& m, int slot, int chunks, int per_seq, int n_slots, int* sh,
                                          DeltaPart& s) {
  if (!m.packed) {
    const int seq = slot / per_seq;
    s = DeltaPart{seq, seq, 0, m.T, slot - seq * per_seq, seq * m.n_chunks};
    return true;
  }
  const int SL = kC * chunks;
  if (threadIdx.x == 0) *sh = -1;
  __syncthreads();
  for (int i = threadIdx.x; i <= m.n_seq; i += blockDim.x) {
    const int lo = decay_first_slot(cu_at(m, i), i, SL);
    const int hi = i < m.n_seq ? decay_first_slot(cu_at(m, i + 1), i + 1, SL) : n_slots;
    if (lo <= slot && slot < hi) *sh = i;
  }
  __syncthreads();
  const int i = *sh;
  if (i < 0) return false;
  const int first = cu_at(m, i), end = i < m.n_seq ? cu_at(m, i + 1) : m.T;
  s = DeltaPart{i, 0, first, max(end - first, 0), slot - decay_first_slot(first, i, SL), decay_first_slot(first, i, kC)};
  return true;
}

// A chunk's rows of an operand as they are staged (Stage in tiles.h), n of them.
template <typename S>
__device__ __forceinline__ void fetch_rows(S& s, long long st, int n) {
  if (n < kC) s.fetch(st, n);
  else s.template fetch<false>(st);
}

}  // namespace kata
