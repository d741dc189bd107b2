// What the gated delta rule's kernels share: where a chunk lies, what the workspace holds of it, and
// products whose operands are kept in two or three bf16 terms.
#pragma once

#include "decay_slots.h"
#include "delta.h"
#include "tiles.h"

namespace kata {

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const __bf16* p) { return unquad(*reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ f32x4 unquad(const f32x4& x) { return x; }

// What a chunk and head keep in the workspace.  Vectors: exp(c), exp(c_63 - c), beta, and c log2(e) as the sum
// of two floats, of every token, c being the sum of the log decays from the chunk's first token on.
// Inverse: its 16 x 16 blocks on and below the diagonal, by rows of blocks.  Their sizes: decay_slots.h, which the planner
// lays the workspace out by, too.
static_assert(kDeltaChunk == kC, "the planner's chunks are the kernels'");

// 2^(hi + lo) of the difference of two such sums
__device__ __forceinline__ float exp2_diff(float hi, float lo, float hj, float lj) {
  return __builtin_amdgcn_exp2f((hi - hj) + (lo - lj));
}

// bf16 operands that come out of fp32 sums are kept as N bf16 terms that add up to them: the recurrence passes
// a rounding on from chunk to chunk, and states are fp32.  Two terms hold 2^-18 of a value, three 2^-27.
// fp32: one.  The differences are of the rounded sums: contracted with the product that a sum ended with, they would
// depend on what the compiler makes of the path to them, and so a column on its neighbours' infinities.
template <typename T, int N>
struct Op {
  typename Elem<T>::frag t[N];
};

template <int N>
__device__ __forceinline__ void split_terms(f32x4 a, f32x4 b, Op<__bf16, N>& out) {
#pragma clang fp contract(off)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint2 x = quad(a, __bf16()), y = quad(b, __bf16());
    out.t[i] = __builtin_bit_cast(bf16x8, uint4{x.x, x.y, y.x, y.y});
    if (i + 1 < N) {
      a -= unquad(x);
      b -= unquad(y);
    }
  }
}
__device__ __forceinline__ void split_terms(const f32x4& a, const f32x4& b, Op<float, 1>& out) {
  out.t[0] = pack_frag(a, b, float());
}

// c + a b with an exact operand, and with both in terms (products of order max(N, K) and above are left out)
template <typename F, typename T, int N>
__device__ __forceinline__ f32x4 mul(const F& a, const Op<T, N>& b, f32x4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mma(a, b.t[i], c);
  return c;
}
template <typename F, typename T, int N>
__device__ __forceinline__ f32x4 mul(const Op<T, N>& a, const F& b, f32x4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mma(a.t[i], b, c);
  return c;
}
template <typename T, int N, int K>
__device__ __forceinline__ f32x4 mul(const Op<T, N>& a, const Op<T, K>& b, f32x4 c) {
  constexpr int most = N > K ? N : K;
#pragma unroll
  for (int order = most - 1; order >= 0; --order)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (order - i >= 0 && order - i < K) c = mma(a.t[i], b.t[order - i], c);
  return c;
}

// The pairs of terms (i, k) of a product of N by K of them, smallest first.  f adds that pair's product to several tiles
// in turn: a product that waits for the one just issued costs its whole latency.
template <int N, int K, typename F>
__device__ __forceinline__ void each_term(F f) {
  constexpr int most = N > K ? N : K;
#pragma unroll
  for (int order = most - 1; order >= 0; --order)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (order - i >= 0 && order - i < K) f(i, order - i);
}

// Four neighbouring elements of a row as N planes of them, `plane` elements apart.
template <int N, typename T>
__device__ __forceinline__ void put_terms(T* at, int plane, f32x4 x) {
#pragma clang fp contract(off)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Quad<T> u = quad(x, T());
    *reinterpret_cast<Quad<T>*>(at + i * plane) = u;
    if constexpr (sizeof(T) == 2)
      if (i + 1 < N) x -= unquad(u);
  }
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

// The N planes of a row's or (rows in split places) a column tile's operand, planes `plane` elements apart.
template <int N, typename T>
__device__ __forceinline__ Op<T, N> row_op(const T* p, int plane) {
  Op<T, N> x;
#pragma unroll
  for (int i = 0; i < N; ++i) x.t[i] = row_frag(p + i * plane);
  return x;
}
template <int N, int LD, typename T>
__device__ __forceinline__ Op<T, N> split_column_op(const T* p, int plane, int tile, int lane) {
  Op<T, N> x;
#pragma unroll
  for (int i = 0; i < N; ++i) x.t[i] = split_column_frag<LD>(p + i * plane, tile, lane);
  return x;
}

// The inverse of a chunk from the workspace into N planes [64][LD] of LDS, rows of split places.  zeros(): the
// two blocks above the diagonal that share a K step with one below it, written once.
template <typename T, int N, int LD, int kThr>
struct StageInv {
  static constexpr int kVecs = kInvFloats / 4, R = (kVecs + kThr - 1) / kThr;
  f32x4 x[R];
  template <bool kAlways = true>                    // (see fetch_rows)
  __device__ __forceinline__ void fetch(const float* p) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int v = threadIdx.x + i * kThr;
      if constexpr (kAlways || kVecs % kThr == 0) x[i] = reinterpret_cast<const f32x4*>(p)[min(v, kVecs - 1)];
      else if (v < kVecs) x[i] = reinterpret_cast<const f32x4*>(p)[v];
    }
  }
  __device__ __forceinline__ static void zeros(T* tile) {
    for (int v = threadIdx.x; v < 128; v += kThr)
      put_terms<N>(tile + (32 * (v >> 6) + ((v >> 2) & 15)) * LD + split_place(32 * (v >> 6) + 16 + 4 * (v & 3)), kC * LD, zero4());
  }
  __device__ __forceinline__ void put(T* tile) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int v = threadIdx.x + i * kThr, block = v >> 6, row = (v >> 2) & 15;
      const int bi = (block >= 1) + (block >= 3) + (block >= 6), bj = block - bi * (bi + 1) / 2;
      if (kVecs % kThr == 0 || v < kVecs)
        put_terms<N>(tile + (16 * bi + row) * LD + split_place(16 * bj + 4 * (v & 3)), kC * LD, x[i]);
    }
  }
};

// Products q . k of a wave's strip (transposed: lane's row 16 rt + l16, keys 16 (j0 + j) + 4 g + r) become its part
// of P, times `scale`; zero by selection where the key is later.  c: the logarithms' two floats.  Rows of
// split places, N planes.
template <typename T, int LP, int J, int N>
__device__ __forceinline__ void put_weights(T* sP, f32x4 (&p)[J], const float* c, int rt, int j0, int lane, float scale) {
  const int g = lane >> 4, l16 = lane & 15;
  const float hi = c[16 * rt + l16], lo = c[kC + 16 * rt + l16];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    f32x4 x = zero4();
    if (j0 + j <= rt) {                             // uniform
      const f32x4 hj = *reinterpret_cast<const f32x4*>(c + 16 * (j0 + j) + 4 * g);
      const f32x4 lj = *reinterpret_cast<const f32x4*>(c + kC + 16 * (j0 + j) + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = 16 * (j0 + j) + 4 * g + r > 16 * rt + l16 ? 0.f : p[j][r] * (exp2_diff(hi, lo, hj[r], lj[r]) * scale);
    }
    put_terms<N>(sP + (16 * rt + l16) * LP + split_place(16 * (j0 + j) + 4 * g), kC * LP, x);
  }
}
template <typename T, int DK, int LK, int LP, int J, int N>
__device__ __forceinline__ void put_scores(T* sP, const T* sQ, const T* sK, const float* c, int rt, int j0, int lane,
                                           float scale) {
  constexpr int M = DK / 32;
  const int g = lane >> 4, l16 = lane & 15;
  f32x4 p[J];
#pragma unroll
  for (int j = 0; j < J; ++j) p[j] = zero4();
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const auto q = row_frag(sQ + (16 * rt + l16) * LK + 32 * i + 8 * g);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j0 + j <= rt) p[j] = mma(row_frag(sK + (16 * (j0 + j) + l16) * LK + 32 * i + 8 * g), q, p[j]);
  }
  put_weights<T, LP, J, N>(sP, p, c, rt, j0, lane, scale);
}

// State tiles of columns col (the lane's): S[i] has rows 16 i + 4 g + r; zeros behind the state's rows and columns.
// (Loads from clamped places and a selection: under a condition each they cost the registers of as many branches.)
template <int NS>
__device__ __forceinline__ void load_state(f32x4 (&S)[NS], const float* p, int rows, int cols, int col, int g) {
  const float* const at = p + min(col, cols - 1);
  const bool live = col < cols;
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * i + 4 * g + r;
      const float x = at[min(row, rows - 1) * cols];
      S[i][r] = live && row < rows ? x : 0.f;
    }
}

// ---- sequences -------------------------------------------------------------------------------
struct DeltaPart {
  int seq, b, start, len;                 // the sequence, its batch row, first row and length
  int part;                               // which segment (chunk) of it
  int c_slot;                             // its first chunk's slot
};

__device__ __forceinline__ int cu_at(const DeltaMap& m, int i) { return min(max(m.cu[i], 0), m.T); }

// The part of `len` chunks in `slot`; false where there is none.  seq == n_seq: rows behind the last sequence.
// sh: one int of LDS.  Each of the `threads` threads calls it.
__device__ __forceinline__ bool find_part(const DeltaMap& m, int slot, int chunks, int per_seq, int n_slots, int* sh,
                                          int threads, DeltaPart& s) {
  if (!m.packed) {
    const int seq = slot / per_seq;
    s = DeltaPart{seq, seq, 0, m.T, slot - seq * per_seq, seq * m.n_chunks};
    return true;
  }
  const int SL = kC * chunks;
  if (threadIdx.x == 0) *sh = -1;
  __syncthreads();
  for (int i = threadIdx.x; i <= m.n_seq; i += threads) {
    const int lo = decay_first_slot(cu_at(m, i), i, SL);
    const int hi = i < m.n_seq ? decay_first_slot(cu_at(m, i + 1), i + 1, SL) : n_slots;
    if (lo <= slot && slot < hi) *sh = i;
  }
  __syncthreads();
  const int i = __builtin_amdgcn_readfirstlane(*sh);
  if (i < 0) return false;
  const int first = cu_at(m, i), end = i < m.n_seq ? cu_at(m, i + 1) : m.T;
  s = DeltaPart{i, 0, first, max(end - first, 0), slot - decay_first_slot(first, i, SL), decay_first_slot(first, i, kC)};
  return true;
}

// A workgroup's unit (segment and head) and block: the blocks of one unit read the same rows, so they get ids
// congruent mod 8, one XCD.
struct UnitBlock {
  unsigned unit;
  int sub;
};
__device__ __forceinline__ UnitBlock unit_block(int blocks) {
  const unsigned x = block_number(), per = blocks, y = x / 8 / per;
  return UnitBlock{8 * y + x % 8, int(x / 8 - y * per)};
}

// A chunk's rows of an operand as they are staged (Stage in tiles.h), n >= 1 of them.  kAlways: the last one is read
// for those behind it, which keep_rows() makes zeros before they are put, so that no load stands under a condition:
// before the next one's zeros are written the compiler waits for it, and with it for all others.  That serves a
// workgroup alone on its CU (the backward walks of 8 x 4096: 384 us, 320 so); two share the wait, and lack the
// registers (131072 tokens: sums 407 us, 515 so; outputs 490 and 537).
template <bool kAlways = true, typename S>
__device__ __forceinline__ void fetch_rows(S& s, long long st, int n) {
  if (kAlways && n < kC) {                          // uniform
    const int row = threadIdx.x / S::PER;
#pragma unroll
    for (int i = 0; i < S::N; ++i)
      s.x[i] = *reinterpret_cast<const uint4*>(s.p + (min(row + i * S::kRows, n - 1) - row) * st);
    s.p += kC * st;
  } else if (n < kC) {
    s.fetch(st, n);
  } else {
    s.template fetch<false>(st);
  }
}
template <typename S>
__device__ __forceinline__ void keep_rows(S& s, int n) {
  if (n < kC)                                       // uniform
#pragma unroll
    for (int i = 0; i < S::N; ++i)
      if (int(threadIdx.x / S::PER) + i * S::kRows >= n) s.x[i] = uint4{0u, 0u, 0u, 0u};
}
// The vectors of a chunk: a thread's four of them, and into LDS.
__device__ __forceinline__ uint4 fetch_vec(const float* p) {
  return reinterpret_cast<const uint4*>(p)[min((int)threadIdx.x, kDeltaVec / 4 - 1)];
}
__device__ __forceinline__ void put_vec(float* vec, const uint4& x) {
  if (threadIdx.x < kDeltaVec / 4) reinterpret_cast<uint4*>(vec)[threadIdx.x] = x;
}

}  // namespace kata
