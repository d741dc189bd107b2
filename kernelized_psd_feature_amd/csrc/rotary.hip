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
// Bound: HBM, each element read and written once: 131072 tokens of 16 + 16 bf16 heads of width 64 in
// 194 us, 5.5 TB/s.  Parts that are not whole vectors cost the elements at their end: 4 x 8192 tokens of
// 16 + 4 heads, 24 of 64 coordinates turned, 61 us (133 element by element), 62 of 64 125 (135).
#include "device.h"
#include "layer.h"
#include "mfma_util.h"
#include "turns.h"

namespace kata {
namespace {

constexpr int kThreads = 256;

// IL: pairs of neighbours.  kEdge: rows of any alignment, and parts that end inside a vector, whose
// last elements go one by one.
template <typename T, bool IL, bool kEdge>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs A) {
  extern __shared__ float2 cs[];                    // [tokens of the block][rot / 2]
  const int half = A.rot / 2, tid = threadIdx.x;
  const unsigned first = block_number() * (unsigned)A.TT, total = (unsigned)A.B * (unsigned)A.T;   // < 2^31
  if (first >= total) return;                       // behind the last of several grid rows
  const int tokens = (int)min((unsigned)A.TT, total - first);
  put_turns(A, cs, first, tokens, kThreads);
  __syncthreads();
  // items of a head, of V elements: NR that turn (in halves with as many of the second half), then
  // those that are copied
  constexpr int V = 16 / sizeof(T);
  const int turned = IL ? A.rot : half;
  const int NR = (turned + V - 1) / V, NI = NR + (A.D - A.rot + V - 1) / V;
  const int heads = A.H + A.Hk, per = heads * NI;
  for (int i = tid; i < tokens * per; i += kThreads) {
    const int tt = i / per, y = i - tt * per, hh = y / NI, it = y - hh * NI;
    const unsigned token = first + tt;
    const int b = int(token / (unsigned)A.T), t = int(token - (unsigned)b * (unsigned)A.T);
    const bool is_k = hh >= A.H, turns = it < NR;
    const int h = hh - (is_k ? A.H : 0);
    const int e = turns ? it * V : A.rot + (it - NR) * V;
    const T* src = reinterpret_cast<const T*>(is_k ? A.k : A.q) + row_off(is_k ? A.sk : A.sq, b, t, h) + e;
    T* dst = reinterpret_cast<T*>(is_k ? A.ok : A.oq) + row_off(is_k ? A.sok : A.soq, b, t, h) + e;
    const float2* w = cs + tt * half + (IL ? e / 2 : e);
    if (kEdge) {
      const int n = (turns ? turned : A.D) - e;     // elements left
      if (n < V) {
        T u[V], v[V];
#pragma unroll
        for (int r = 0; r < V; ++r)
          if (r < n) u[r] = src[r];
#pragma unroll
        for (int r = 0; r < V; ++r)
          if (!IL && turns && r < n) v[r] = src[half + r];
#pragma unroll
        for (int r = 0; r < V; ++r) {
          if (r >= n) break;
          if (!turns) {
            dst[r] = u[r];
          } else if constexpr (!IL) {
            const float x = to_f32(u[r]), z = to_f32(v[r]);
            dst[r] = from_f32<T>(x * w[r].x - z * w[r].y);
            dst[half + r] = from_f32<T>(x * w[r].y + z * w[r].x);
          } else if (r % 2 == 0) {                  // rot is even: a whole pair
            const float x = to_f32(u[r]), z = to_f32(u[r + 1]);
            dst[r] = from_f32<T>(x * w[r / 2].x - z * w[r / 2].y);
            dst[r + 1] = from_f32<T>(x * w[r / 2].y + z * w[r / 2].x);
          }
        }
        continue;
      }
    }
    // Both loads are issued before the branch (a copy's second one repeats the first); the empty asm
    // keeps the compiler from moving the second one into it, behind the wait for the first (194 us
    // for 207 at 131072 tokens).
    const u32x4 u = get<T, kEdge>(src);
    u32x4 v = u;
    if constexpr (!IL) {
      v = get<T, kEdge>(src + (turns ? half : 0));
      asm volatile("" : "+v"(v));
    }
    float x[V], z[V], p[V], s[V];
    unpack(u, x);
    if (!turns) {
      put<T, kEdge>(dst, u);
    } else if constexpr (!IL) {
      unpack(v, z);
#pragma unroll
      for (int r = 0; r < V; ++r) {
        p[r] = x[r] * w[r].x - z[r] * w[r].y;
        s[r] = x[r] * w[r].y + z[r] * w[r].x;
      }
      put<T, kEdge>(dst, pack(p));
      put<T, kEdge>(dst + half, pack(s));
    } else {
#pragma unroll
      for (int r = 0; r < V; r += 2) {
        p[r] = x[r] * w[r / 2].x - x[r + 1] * w[r / 2].y;
        p[r + 1] = x[r] * w[r / 2].y + x[r + 1] * w[r / 2].x;
      }
      put<T, kEdge>(dst, pack(p));
    }
  }
}

template <typename T, bool kEdge>
hipError_t launch_t(RotaryArgs& a, bool interleaved, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int half = a.rot / 2;
  const int per = (a.H + a.Hk) * (((interleaved ? a.rot : half) + V - 1) / V + (a.D - a.rot + V - 1) / V);
  // About four vector loads a thread (an item of halves has two), fewer where that leaves CUs without
  // a workgroup, and the cosines of the block within 32 KB.  131072 tokens, 16 + 16 bf16 heads of
  // width 64, halves: two items 194 us, one 190, four 203, six 210; neighbours: four items 190, one
  // 243, two 197, six 196.  8 x 4096 tokens, halves: 40.4, 40.3, 42.7, 43.8.
  const long long tokens = (long long)a.B * a.T;
  a.TT = (interleaved ? 4 : 2) * kThreads / per;
  if (a.TT > tokens / 512) a.TT = (int)(tokens / 512);
  if (a.TT * half > 4096) a.TT = 4096 / half;
  if (a.TT < 1) a.TT = 1;
  const long long blocks = (tokens + a.TT - 1) / a.TT;
  const size_t lds = sizeof(float2) * a.TT * half;
  if (interleaved)
    launch_kernel(rotary_kernel<T, true, kEdge>, grid_rows(blocks), kThreads, lds, st, a);
  else
    launch_kernel(rotary_kernel<T, false, kEdge>, grid_rows(blocks), kThreads, lds, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(RotaryArgs& a, bool bf16, bool aligned, bool interleaved, hipStream_t st) {
  const int V = bf16 ? 8 : 4;
  // aligned rows whose turned part, its half (in halves) and the rest consist of whole vectors
  const bool whole = aligned && a.D % V == 0 && a.rot % V == 0 && (interleaved || a.rot / 2 % V == 0);
  if (bf16) return whole ? launch_t<__bf16, false>(a, interleaved, st) : launch_t<__bf16, true>(a, interleaved, st);
  return whole ? launch_t<float, false>(a, interleaved, st) : launch_t<float, true>(a, interleaved, st);
}

}  // namespace kata
