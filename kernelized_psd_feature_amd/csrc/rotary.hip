// Rotary positions of q and k, gfx950.
//
// The first `rot` coordinates of a head form rot / 2 pairs (a, b) -- neighbours, or the two halves
// -- and the pair i of a token at position x becomes
//     m (a cos x r_i - b sin x r_i),  m (a sin x r_i + b cos x r_i)
// (inverse: angle -x r_i, which is the gradient); the other coordinates are copied.
//
// Angles grow with the position, so x r_i is formed and reduced to a fraction of a turn in 64
// bits: in fp32 an angle of 10^5 is known to 0.004 only.  All heads of q and k share the angles of
// a token, so a workgroup takes a few tokens, leaves their rot / 2 cosines and sines in LDS, and
// then streams every head through 16-byte accesses.  One launch for q and k.
// Bound: HBM, each element read and written once.
#include "device.h"
#include "layer.h"
#include "mfma_util.h"

namespace kata {
namespace {

constexpr int kThreads = 256;

template <typename T, int V>
struct Vec {
  float x[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      x[0] = to_f32(p[0]);
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      if constexpr (sizeof(T) == 2) {
        x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
        x[4] = bf_lo(u.z); x[5] = bf_hi(u.z); x[6] = bf_lo(u.w); x[7] = bf_hi(u.w);
      } else {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 1) {
      p[0] = from_f32<T>(x[0]);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(p) = uint4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    } else {
      *reinterpret_cast<float4*>(p) = float4{x[0], x[1], x[2], x[3]};
    }
  }
};

// V elements of a vector (1: element by element), IL: pairs of neighbours.
template <typename T, int V, bool IL>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs A) {
  extern __shared__ float2 cs[];                    // [tokens of the block][rot / 2]
  const int half = A.rot / 2, tid = threadIdx.x;
  const unsigned first = blockIdx.x * (unsigned)A.TT, total = (unsigned)A.B * (unsigned)A.T;   // < 2^31
  const int tokens = (int)min((unsigned)A.TT, total - first);
  for (int i = tid; i < tokens * half; i += kThreads) {
    const unsigned token = first + i / half, b = token / (unsigned)A.T, t = token - b * (unsigned)A.T;
    long long pos = A.offset + (long long)t;
    if (A.positions) {
      const long long at = (long long)b * A.pos_b + (long long)t * A.pos_t;
      pos = A.pos64 ? reinterpret_cast<const long long*>(A.positions)[at]
                    : (long long)reinterpret_cast<const int*>(A.positions)[at];
    }
    double turn = (double)pos * A.rates[i % half] * 0.15915494309189535;   // 1 / (2 pi)
    turn -= rint(turn);
    float s, c;
    sincospif((float)(2.0 * turn), &s, &c);
    cs[i] = float2{A.magnitude * c, A.inverse ? -A.magnitude * s : A.magnitude * s};
  }
  __syncthreads();
  // items of a head: NR that turn (V pairs in halves; V / 2 or one of neighbours), NC that are copied
  const int NR = IL ? A.rot / (V == 1 ? 2 : V) : half / V, NC = (A.D - A.rot) / V, NI = NR + NC;
  const int heads = A.H + A.Hk, per = heads * NI;
  for (int i = tid; i < tokens * per; i += kThreads) {
    const int tt = i / per, y = i % per, it = y % NI;
    int h = y / NI;
    const unsigned token = first + tt;
    const int b = int(token / (unsigned)A.T), t = int(token - (unsigned)b * (unsigned)A.T);
    const bool is_k = h >= A.H;
    h -= is_k ? A.H : 0;
    const T* src = reinterpret_cast<const T*>(is_k ? A.k : A.q) + row_off(is_k ? A.sk : A.sq, b, t, h);
    T* dst = reinterpret_cast<T*>(is_k ? A.ok : A.oq) + row_off(is_k ? A.sok : A.soq, b, t, h);
    if (it >= NR) {
      const int e = A.rot + (it - NR) * V;
      Vec<T, V> x;
      x.load(src + e);
      x.store(dst + e);
    } else if constexpr (!IL) {
      const int e = it * V;
      Vec<T, V> a, c, ya, yc;
      a.load(src + e);
      c.load(src + half + e);
#pragma unroll
      for (int r = 0; r < V; ++r) {
        const float2 w = cs[tt * half + e + r];
        ya.x[r] = a.x[r] * w.x - c.x[r] * w.y;
        yc.x[r] = a.x[r] * w.y + c.x[r] * w.x;
      }
      ya.store(dst + e);
      yc.store(dst + half + e);
    } else if constexpr (V == 1) {
      const float a = to_f32(src[2 * it]), c = to_f32(src[2 * it + 1]);
      const float2 w = cs[tt * half + it];
      dst[2 * it] = from_f32<T>(a * w.x - c * w.y);
      dst[2 * it + 1] = from_f32<T>(a * w.y + c * w.x);
    } else {
      const int e = it * V;
      Vec<T, V> x, z;
      x.load(src + e);
#pragma unroll
      for (int r = 0; r < V; r += 2) {
        const float2 w = cs[tt * half + (e + r) / 2];
        z.x[r] = x.x[r] * w.x - x.x[r + 1] * w.y;
        z.x[r + 1] = x.x[r] * w.y + x.x[r + 1] * w.x;
      }
      z.store(dst + e);
    }
  }
}

template <typename T, int V>
hipError_t launch_t(RotaryArgs& a, bool interleaved, hipStream_t st) {
  const int half = a.rot / 2;
  const int NR = interleaved ? a.rot / (V == 1 ? 2 : V) : half / V;
  const int per = (a.H + a.Hk) * (NR + (a.D - a.rot) / V);
  // about four items a thread, fewer where that leaves CUs without a workgroup, and the cosines of
  // the block within 32 KB
  const long long tokens = (long long)a.B * a.T;
  a.TT = 4 * kThreads / per;
  if (a.TT > tokens / 512) a.TT = (int)(tokens / 512);
  if (a.TT * half > 4096) a.TT = 4096 / half;
  if (a.TT < 1) a.TT = 1;
  const long long blocks = (tokens + a.TT - 1) / a.TT;
  const size_t lds = sizeof(float2) * a.TT * half;
  if (interleaved)
    launch_kernel(rotary_kernel<T, V, true>, dim3((unsigned)blocks), kThreads, lds, st, a);
  else
    launch_kernel(rotary_kernel<T, V, false>, dim3((unsigned)blocks), kThreads, lds, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(RotaryArgs& a, bool bf16, bool aligned, bool interleaved, hipStream_t st) {
  const int V = bf16 ? 8 : 4;
  // 16-byte accesses where rows, the turned part and (in halves) its half consist of whole vectors
  const bool vec = aligned && a.D % V == 0 && a.rot % V == 0 && (interleaved || a.rot / 2 % V == 0);
  if (bf16) return vec ? launch_t<__bf16, 8>(a, interleaved, st) : launch_t<__bf16, 1>(a, interleaved, st);
  return vec ? launch_t<float, 4>(a, interleaved, st) : launch_t<float, 1>(a, interleaved, st);
}

}  // namespace kata
