// MFMA operands and staging of 64-token chunks, for bf16 and fp32 elements, shared by the kernels of the
// linear attention forms with a state (decay.hip, delta.hip, delta_bwd.hip).  Tiles are 16 x 16, K steps
// 32 wide; fragment conventions as in mfma_util.h.  Both operands of a product enumerate its K step in one
// order, of two: "straight" (slot r of lane group g is index 8 g + r) or "split" (slots 0..3 are 4 g + r,
// slots 4..7 are 16 + 4 g + r - 4, the order in which two accumulator tiles hold their rows).
#pragma once

#include <type_traits>

#include "device.h"
#include "mfma_util.h"

namespace kata {

constexpr int kC = 64;                    // tokens of a chunk

typedef __attribute__((__vector_size__(8 * sizeof(float)))) float f32x8;

template <typename T>
struct Elem;
template <>
struct Elem<__bf16> {
  using frag = bf16x8;
  static constexpr int V = 8;             // elements of a 16-byte vector
};
template <>
struct Elem<float> {
  using frag = f32x8;
  static constexpr int V = 4;
};

__device__ __forceinline__ f32x4 mma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return mfma32(a, b, c);
}
__device__ __forceinline__ f32x4 mma(const f32x8& a, const f32x8& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// Straight slots of a row: eight neighbouring elements.
__device__ __forceinline__ bf16x8 row_frag(const __bf16* p) {
  return __builtin_bit_cast(bf16x8, ld16(p));
}
__device__ __forceinline__ f32x8 row_frag(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// Rows that are read in split slots are kept so that these are neighbours: run u of four elements
// of every 32 (0..7) lies at place 2 (u % 4) + u / 4, and row_frag reads split slots.  (As two 8-byte
// reads 16 elements apart, which the compiler makes one instruction, they met each bank twice.)
__device__ __forceinline__ constexpr int split_place(int col) {
  return (col & ~31) + 8 * ((col >> 2) & 3) + 4 * ((col >> 4) & 1) + (col & 3);
}
// Straight slots 8 g .. 8 g + 7 of 32 columns of such a row.
__device__ __forceinline__ bf16x8 straight_frag(const __bf16* p, int g) {
  const uint2 a = *reinterpret_cast<const uint2*>(p + split_place(8 * g));
  const uint2 b = *reinterpret_cast<const uint2*>(p + split_place(8 * g + 4));
  return __builtin_bit_cast(bf16x8, uint4{a.x, a.y, b.x, b.y});
}
__device__ __forceinline__ f32x8 straight_frag(const float* p, int g) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p + split_place(8 * g));
  const f32x4 b = *reinterpret_cast<const f32x4*>(p + split_place(8 * g + 4));
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// Split slots of column i, i the lane's place in its group of 16, of 32 rows of LD elements at p.
// bf16 by the transposing read (v_frag in mfma_util.h).
template <int LD>
__device__ __forceinline__ bf16x8 column_frag(const __bf16* p, int lane) {
  const __bf16* at = p + (4 * (lane >> 4) + ((lane & 15) >> 2)) * LD + 4 * (lane & 3);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * LD));
  const uint2 ul = __builtin_bit_cast(uint2, lo), uh = __builtin_bit_cast(uint2, hi);
  return __builtin_bit_cast(bf16x8, uint4{ul.x, ul.y, uh.x, uh.y});
}
template <int LD>
__device__ __forceinline__ f32x8 column_frag(const float* p, int lane) {
  const float* at = p + 4 * (lane >> 4) * LD + (lane & 15);
  f32x8 x;
#pragma unroll
  for (int r = 0; r < 8; ++r) x[r] = at[(16 * (r / 4) + r % 4) * LD];
  return x;
}

__device__ __forceinline__ bf16x8 pack_frag(const f32x4& a, const f32x4& b, __bf16) {
  return __builtin_bit_cast(bf16x8, uint4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                          pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])});
}
__device__ __forceinline__ f32x8 pack_frag(const f32x4& a, const f32x4& b, float) {
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Adds 0 x to t for every element: t becomes nan where one is an infinity or nan.
__device__ __forceinline__ float poison(const bf16x8& x, float t) {
  const uint4 u = __builtin_bit_cast(uint4, x);
  typedef __attribute__((ext_vector_type(2))) __bf16 b2;
  const b2 z = __builtin_bit_cast(b2, 0u);
  t = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, u.x), z, t, false);
  t = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, u.y), z, t, false);
  t = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, u.z), z, t, false);
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, u.w), z, t, false);
}
__device__ __forceinline__ float poison(const f32x8& x, float t) {
#pragma unroll
  for (int r = 0; r < 8; ++r) t = fmaf(x[r], 0.f, t);
  return t;
}

// LDS reads above this line in the source stay above it, and what uses them below.  fp32 fragments
// are twice as large: there the compiler keeps its own order.
template <typename T>
__device__ __forceinline__ void reads_above() {
  if constexpr (sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);
}

// Four neighbouring elements as they are stored.
template <typename T>
using Quad = std::conditional_t<sizeof(T) == 2, uint2, f32x4>;
__device__ __forceinline__ uint2 quad(const f32x4& x, __bf16) {
  return uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}
__device__ __forceinline__ f32x4 quad(const f32x4& x, float) { return x; }
__device__ __forceinline__ f32x4 unquad(const uint2& u) {
  return f32x4{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y)};
}
__device__ __forceinline__ void store4(__bf16* p, const f32x4& x) {
  *reinterpret_cast<uint2*>(p) = quad(x, __bf16());
}
__device__ __forceinline__ void store4(float* p, const f32x4& x) {
  *reinterpret_cast<f32x4*>(p) = x;
}

// ---- staging -------------------------------------------------------------------------------
// A chunk of one operand: 64 rows of W columns, W / (4 V) 16-byte vectors a thread (the rows behind n
// zero).  A thread behind the operand's `width` columns reads the row's first vector again and
// writes it behind the tile's columns, into the row's padding: no load or write depends on the
// width, and the tile's columns behind the width keep the zeros that they start with (4 x 8192, 8 bf16
// heads of 72: 81 us, backward 251; with loads under a mask 96 and 334).
template <typename T, int W, int kThr>
struct Stage {
  static constexpr int V = Elem<T>::V, PER = W / V, N = kC * PER / kThr, kRows = kThr / PER;
  static_assert(N >= 1 && kC % kRows == 0, "whole rows a step");
  const T* p;                             // the thread's first vector of the next chunk
  int to, to2;                            // its columns in the tile; in split order of each half
  uint4 x[N];
  // row 0 at base, rows st elements apart (negative in reversed time)
  __device__ __forceinline__ Stage(const T* base, long long st, int width, bool split) {
    const int col = (threadIdx.x % PER) * V;
    const bool live = col < width;
    p = base + (long long)(threadIdx.x / PER) * st + (live ? col : 0);
    to = !live ? W : split ? split_place(col) : col;
    to2 = !live ? W + 4 : split_place(col + 4);
  }
  // 64 whole rows; kStream: nothing of them is kept in the caches
  template <bool kStream>
  __device__ __forceinline__ void fetch(long long st) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
      const u32x4* at = reinterpret_cast<const u32x4*>(p + i * kRows * st);
      x[i] = __builtin_bit_cast(uint4, kStream ? __builtin_nontemporal_load(at) : *at);
    }
    p += kC * st;
  }
  __device__ __forceinline__ void fetch(long long st, int n) {
    const int row = threadIdx.x / PER;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = uint4{0u, 0u, 0u, 0u};
      if (row + i * kRows < n) x[i] = *reinterpret_cast<const uint4*>(p + i * kRows * st);
    }
    p += kC * st;
  }
  template <int LD>
  __device__ __forceinline__ void put(T* tile) const {
    static_assert(LD - W >= V, "padding for a vector");
    T* at = tile + threadIdx.x / PER * LD + to;
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<uint4*>(at + i * kRows * LD) = x[i];
  }
  // the rows' runs of four elements at their split places
  template <int LD>
  __device__ __forceinline__ void put_split(T* tile) const {
    static_assert(LD - W >= V, "padding for a vector");
    T* at = tile + threadIdx.x / PER * LD;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (V == 8) {
        *reinterpret_cast<uint2*>(at + i * kRows * LD + to) = uint2{x[i].x, x[i].y};
        *reinterpret_cast<uint2*>(at + i * kRows * LD + to2) = uint2{x[i].z, x[i].w};
      } else {
        *reinterpret_cast<uint4*>(at + i * kRows * LD + to) = x[i];
      }
    }
  }
};

}  // namespace kata
