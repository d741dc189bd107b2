// Angles of rotary positions and 16-byte accesses to rows of any alignment, shared by the kernels that turn
// queries and keys (rotary.hip, qk_norm.hip).
#pragma once

#include "device.h"
#include "mfma_util.h"

namespace kata {

// 16 bytes of elements; kEdge: at any element, which this card's global memory allows.
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Unaligned {
  u32x4 u;
};
template <typename T, bool kEdge>
__device__ __forceinline__ u32x4 get(const T* p) {
  return kEdge ? reinterpret_cast<const Unaligned<T>*>(p)->u : *reinterpret_cast<const u32x4*>(p);
}
template <typename T, bool kEdge>
__device__ __forceinline__ void put(T* p, const u32x4& u) {
  if (kEdge) reinterpret_cast<Unaligned<T>*>(p)->u = u;
  else *reinterpret_cast<u32x4*>(p) = u;
}
__device__ __forceinline__ void unpack(const u32x4& u, float (&x)[8]) {
  x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
  x[4] = bf_lo(u.z); x[5] = bf_hi(u.z); x[6] = bf_lo(u.w); x[7] = bf_hi(u.w);
}
__device__ __forceinline__ void unpack(const u32x4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ u32x4 pack(const float (&x)[8]) {
  return u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
}
__device__ __forceinline__ u32x4 pack(const float (&x)[4]) {
  return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}

// m (cos, sin) of the angles of `tokens` tokens from `first` on, cs[token][pair]; with several axes a pair has its
// own axis's position (an axis that is not there is taken as the nearest one).
template <typename Args>
__device__ __forceinline__ void put_turns(const Args& A, float2* cs, unsigned first, int tokens, int threads) {
  const int half = A.rot / 2;
  for (int i = threadIdx.x; i < tokens * half; i += threads) {
    const unsigned token = first + i / half, b = token / (unsigned)A.T, t = token - b * (unsigned)A.T;
    const int pair = i % half;
    long long pos = A.offset + (long long)t;
    if (A.positions) {
      long long at = (long long)b * A.pos_b + (long long)t * A.pos_t;
      if (A.axes) at += min(max(A.axes[pair], 0), A.n_axes - 1) * A.pos_a;
      pos = A.pos64 ? reinterpret_cast<const long long*>(A.positions)[at]
                    : (long long)reinterpret_cast<const int*>(A.positions)[at];
    }
    double turn = (double)pos * A.rates[pair] * 0.15915494309189535;   // 1 / (2 pi)
    turn -= rint(turn);
    float s, c;
    sincospif((float)(2.0 * turn), &s, &c);
    cs[i] = float2{A.magnitude * c, A.inverse ? -A.magnitude * s : A.magnitude * s};
  }
}

}  // namespace kata
