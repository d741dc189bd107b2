// Norms of the queries and keys of every head with the position rotation in the same pass, gfx950.
//
//   z = x r w,  r = 1 / sqrt(sum(x^2) / n + eps)  (n: the head's width, or 1 for rows of unit length)
//   y = the first `rot` coordinates of z turned by their positions (rotary.hip), the others as they are
//   backward: dz = the same turn back of dy, t = dz w,
//   dx = r (t - x r^2 sum(t x) / n),  dw = sum over tokens and heads of dz x r
//
// R lanes have a row, an item each (or two): V neighbouring elements of the part that is turned as pairs of
// neighbours or not at all, or V of the first half and their partners of the second.  So pairs meet in one
// lane, a row is read once, stays in registers over its sum, and is written once; the sums of a row go
// through the lanes by shuffles, in fp32.  The tokens' angles are shared by all heads and lie in LDS, formed
// in fp64.  The weight's gradients stay in a lane's registers over its rows (an item's place in the row is the
// same in all of them), are added up over the workgroup, and the partial sums of the workgroups by a second
// kernel, in a fixed order.
//
// Bound by HBM: 131072 tokens, 16 + 16 bf16 heads of 64, 200 us, 5.4 TB/s (the next rows' loads are issued before this
// row is computed; without that 263); 8 x 4096 with 16 + 8 heads, forward 47 us and backward 66 + 5 (4.3 and 4.6 TB/s).
#include "device.h"
#include "layer.h"
#include "layer_plan.h"
#include "mfma_util.h"
#include "turns.h"

namespace kata {
namespace {

constexpr int kThreads = 256;

// IL: pairs of neighbours.  kEdge: rows of any alignment, and parts that end inside a vector.  K: items a lane.
template <typename T, bool IL, bool kEdge, int K>
struct Lane {
  static constexpr int V = 16 / sizeof(T);
  int e[K], n[K];                                   // first element and how many (0: none)
  bool turns[K];
  int half;
  __device__ __forceinline__ Lane(const QkNormArgs& A, int l) {
    half = A.rot / 2;
    const int turned = IL ? A.rot : half, NR = (turned + V - 1) / V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int it = l + k * A.R;
      turns[k] = it < NR;
      e[k] = turns[k] ? it * V : A.rot + (it - NR) * V;
      n[k] = max(0, min(V, (turns[k] ? turned : A.D) - e[k]));
    }
  }
  // the item's vector, and (halves) its partners' (both loads without a branch: a lane without an item, and an
  // item without partners, repeat one); kEdge: whole vectors only
  __device__ __forceinline__ void fetch(const T* row, int k, u32x4& u, u32x4& v) const {
    const bool whole = n[k] == V;
    if (kEdge && !whole) return;
    const T* const at = row + (whole ? e[k] : 0);
    u = get<T, kEdge>(at);
    if (!IL) v = get<T, kEdge>(at + (whole && turns[k] ? half : 0));
  }
  // the elements and partners, zeros behind them
  __device__ __forceinline__ void load(const T* row, int k, const u32x4& u, const u32x4& v, float (&x)[V], float (&z)[V]) const {
    if (kEdge && n[k] < V) {
#pragma unroll
      for (int r = 0; r < V; ++r) {
        x[r] = r < n[k] ? to_f32(row[e[k] + r]) : 0.f;
        z[r] = !IL && turns[k] && r < n[k] ? to_f32(row[e[k] + half + r]) : 0.f;
      }
      return;
    }
    unpack(u, x);
    unpack(v, z);
#pragma unroll
    for (int r = 0; r < V; ++r) {
      x[r] = n[k] ? x[r] : 0.f;
      z[r] = !IL && n[k] && turns[k] ? z[r] : 0.f;
    }
  }
  __device__ __forceinline__ void store(T* row, int k, const float (&x)[V], const float (&z)[V]) const {
    if (kEdge && n[k] < V) {
#pragma unroll
      for (int r = 0; r < V; ++r)
        if (r < n[k]) {
          row[e[k] + r] = from_f32<T>(x[r]);
          if (!IL && turns[k]) row[e[k] + half + r] = from_f32<T>(z[r]);
        }
      return;
    }
    if (n[k] == 0) return;
    put<T, kEdge>(row + e[k], pack(x));
    if (!IL && turns[k]) put<T, kEdge>(row + e[k] + half, pack(z));
  }
  // turned by the token's angles, cs[pair]
  __device__ __forceinline__ void turn(const float2* cs, int k, float (&x)[V], float (&z)[V]) const {
    if (!turns[k]) return;
    if constexpr (IL) {
#pragma unroll
      for (int r = 0; r < V; r += 2)
        if (!kEdge || r < n[k]) {
          const float2 w = cs[(e[k] + r) / 2];
          const float a = x[r], b = x[r + 1];
          x[r] = a * w.x - b * w.y;
          x[r + 1] = a * w.y + b * w.x;
        }
    } else {
#pragma unroll
      for (int r = 0; r < V; ++r)
        if (!kEdge || r < n[k]) {
          const float2 w = cs[e[k] + r];
          const float a = x[r], b = z[r];
          x[r] = a * w.x - b * w.y;
          z[r] = a * w.y + b * w.x;
        }
    }
  }
  // the item's elements of a weight
  __device__ __forceinline__ void weight(const float* w, int k, float (&x)[V], float (&z)[V]) const {
#pragma unroll
    for (int r = 0; r < V; ++r) {
      x[r] = r < n[k] ? w[e[k] + r] : 1.f;
      z[r] = !IL && turns[k] && r < n[k] ? w[e[k] + half + r] : 1.f;
    }
  }
};

template <typename T, bool IL, bool kEdge, int K, bool kBackward>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(QkNormArgs A) {
  using L = Lane<T, IL, kEdge, K>;
  constexpr int V = L::V;
  extern __shared__ __align__(16) float2 cs[];      // [tokens of the block][rot / 2] and the weights; then (backward) the sums
  const int tid = threadIdx.x, G = kThreads / A.R, group = tid / A.R, half = A.rot / 2;
  const unsigned total = (unsigned)A.B * (unsigned)A.T;                // < 2^31
  const unsigned n_blocks = (total + A.TT - 1) / A.TT, mine = block_number();
  if (mine >= n_blocks) return;                     // behind the last of several grid rows
  const L lane(A, tid % A.R);
  // the weights as fp32 through LDS: a lane's elements of them one by one from memory, for each workgroup, cost a
  // fifth of the pass
  float* const sw = reinterpret_cast<float*>(cs + A.TT * half);        // [2][D]
  for (int i = tid; i < 2 * A.D; i += kThreads) {
    const void* const p = i < A.D ? A.wq : A.wk;
    const int at = i < A.D ? i : i - A.D;
    sw[i] = !p ? 1.f : A.w_bf16 ? to_f32(reinterpret_cast<const __bf16*>(p)[at]) : reinterpret_cast<const float*>(p)[at];
  }
  float w[2][K][2][V];
  float sum[2][K][2][V];
  if constexpr (kBackward)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int r = 0; r < V; ++r) sum[0][k][0][r] = sum[0][k][1][r] = sum[1][k][0][r] = sum[1][k][1][r] = 0.f;
  const int heads = A.H + A.Hk;
  const float inv_n = 1.f / A.count;

  // A row on its way.  Forward its loads are issued before the angles are formed, or while the row before it is
  // computed (8 x 4096, 16 and 8 heads of 64: 45 us for 49; backward the registers would cost more, 81 us for 69).
  struct Row {
    int tt;
    bool live, is_k;
    const T *src, *grad;
    T* dst;
    u32x4 x[K], z[K], dx[K], dz[K];
  };
  // (forward: one turn of the loop)
  for (unsigned block = mine; block < n_blocks; block += kBackward ? (unsigned)A.blocks : n_blocks) {
    const unsigned first = block * (unsigned)A.TT;
    const int tokens = (int)min((unsigned)A.TT, total - first), rows = tokens * heads;
    auto fetch = [&](int row, Row& R) {
      R.live = row < rows;
      const int y = R.live ? row : rows - 1;        // (others read the last row again)
      R.tt = y / heads;
      const int hh = y - R.tt * heads;
      R.is_k = hh >= A.H;
      const int h = hh - (R.is_k ? A.H : 0);
      const unsigned token = first + R.tt;
      const int b = int(token / (unsigned)A.T), t = int(token - (unsigned)b * (unsigned)A.T);
      R.src = reinterpret_cast<const T*>(R.is_k ? A.k : A.q) + row_off(R.is_k ? A.sk : A.sq, b, t, h);
      R.dst = reinterpret_cast<T*>(R.is_k ? A.ok : A.oq) + row_off(R.is_k ? A.sok : A.soq, b, t, h);
#pragma unroll
      for (int k = 0; k < K; ++k) lane.fetch(R.src, k, R.x[k], R.z[k]);
      if constexpr (kBackward) {
        R.grad = reinterpret_cast<const T*>(R.is_k ? A.dk : A.dq) + row_off(R.is_k ? A.sdk : A.sdq, b, t, h);
#pragma unroll
        for (int k = 0; k < K; ++k) lane.fetch(R.grad, k, R.dx[k], R.dz[k]);
      }
    };
    Row next{};
    if constexpr (!kBackward) fetch(group, next);
    if (kBackward && block != mine) __syncthreads();
    put_turns(A, cs, first, tokens, kThreads);
    __syncthreads();
    if (block == mine)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        lane.weight(sw, k, w[0][k][0], w[0][k][1]);
        lane.weight(sw + A.D, k, w[1][k][0], w[1][k][1]);
      }
    for (int row0 = 0; row0 < rows; row0 += G) {
      if constexpr (kBackward) fetch(row0 + group, next);
      const Row row = next;
      if constexpr (!kBackward)
        if (row0 + G < rows) fetch(row0 + G + group, next);
      const float2* at = cs + row.tt * half;
      float x[K][V], z[K][V], dx[K][V], dz[K][V];
      float ss = 0.f, st = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        lane.load(row.src, k, row.x[k], row.z[k], x[k], z[k]);
        if constexpr (kBackward) {
          lane.load(row.grad, k, row.dx[k], row.dz[k], dx[k], dz[k]);
          lane.turn(at, k, dx[k], dz[k]);
        }
#pragma unroll
        for (int r = 0; r < V; ++r) {
          ss = fmaf(x[k][r], x[k][r], ss);
          ss = fmaf(z[k][r], z[k][r], ss);
          if constexpr (kBackward) {
            st = fmaf(dx[k][r] * (row.is_k ? w[1][k][0][r] : w[0][k][0][r]), x[k][r], st);
            st = fmaf(dz[k][r] * (row.is_k ? w[1][k][1][r] : w[0][k][1][r]), z[k][r], st);
          }
        }
      }
      for (int d = 1; d < A.R; d <<= 1) {
        ss += __shfl_xor(ss, d);
        if constexpr (kBackward) st += __shfl_xor(st, d);
      }
      const float r_ = 1.f / sqrtf(fmaf(ss, inv_n, A.eps)), c = r_ * r_ * st * inv_n;
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int r = 0; r < V; ++r) {
          const float wx = row.is_k ? w[1][k][0][r] : w[0][k][0][r], wz = row.is_k ? w[1][k][1][r] : w[0][k][1][r];
          if constexpr (kBackward) {
            if (row.live) {
              const float ax = dx[k][r] * (x[k][r] * r_), az = dz[k][r] * (z[k][r] * r_);
              sum[0][k][0][r] += row.is_k ? 0.f : ax;
              sum[0][k][1][r] += row.is_k ? 0.f : az;
              sum[1][k][0][r] += row.is_k ? ax : 0.f;
              sum[1][k][1][r] += row.is_k ? az : 0.f;
            }
            x[k][r] = r_ * (dx[k][r] * wx - x[k][r] * c);
            z[k][r] = r_ * (dz[k][r] * wz - z[k][r] * c);
          } else {
            x[k][r] *= r_ * wx;
            z[k][r] *= r_ * wz;
          }
        }
        if constexpr (!kBackward) lane.turn(at, k, x[k], z[k]);
        if (row.live) lane.store(row.dst, k, x[k], z[k]);
      }
    }
  }
  if constexpr (kBackward) {
    if (!A.part) return;
    float* const red = reinterpret_cast<float*>(cs);                   // [group][2][D]
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int r = 0; r < V; ++r)
          if (r < lane.n[k]) {
            float* at = red + (group * 2 + side) * A.D + lane.e[k] + r;
            at[0] = sum[side][k][0][r];
            if (!IL && lane.turns[k]) at[half] = sum[side][k][1][r];
          }
    __syncthreads();
    for (int i = tid; i < 2 * A.D; i += kThreads) {
      float s = 0.f;
      for (int j = 0; j < G; ++j) s += red[j * 2 * A.D + i];
      A.part[(size_t)mine * 2 * A.D + i] = s;
    }
  }
}

// Sixteen columns of the partial sums: sixteen slices of the workgroups' rows, each in order with many loads on
// their way, then the slices.
__global__ __launch_bounds__(kThreads) void qk_norm_sum_kernel(QkNormArgs A) {
  __shared__ float slice[16][17];
  const int c = threadIdx.x & 15, s = threadIdx.x >> 4, i = blockIdx.x * 16 + c, n = 2 * A.D;
  const int per = (A.blocks + 15) / 16, end = min(A.blocks, (s + 1) * per);
  float x = 0.f;
  if (i < n) {
    const float* p = A.part + (size_t)s * per * n + i;
    int j = s * per;
    for (; j + 16 <= end; j += 16, p += (size_t)16 * n) {
      float y[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) y[r] = p[(size_t)r * n];
#pragma unroll
      for (int r = 0; r < 16; ++r) x += y[r];
    }
    for (; j < end; ++j, p += n) x += *p;
  }
  slice[s][c] = x;
  __syncthreads();
  if (s || i >= n) return;
  x = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) x += slice[r][c];
  void* const to = i < A.D ? A.dwq : A.dwk;
  if (!to) return;
  const int at = i < A.D ? i : i - A.D;
  if (A.w_bf16) reinterpret_cast<__bf16*>(to)[at] = (__bf16)x;
  else reinterpret_cast<float*>(to)[at] = x;
}

template <typename T, bool IL, bool kEdge>
hipError_t launch_t(QkNormArgs& a, bool backward, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int half = a.rot / 2, heads = a.H + a.Hk;
  const int items = ((IL ? a.rot : half) + V - 1) / V + (a.D - a.rot + V - 1) / V;
  a.R = 1;
  while (a.R < items && a.R < 64) a.R *= 2;
  const int K = items > a.R ? 2 : 1;
  const long long tokens = (long long)a.B * a.T;
  // Eight rows a group of lanes (backward four, of many such blocks in turn), fewer where that leaves CUs without a
  // workgroup, and the angles within 32 KB.  131072 tokens, 16 + 16 bf16 heads of 64: 222 us, two rows 266, four
  // 231, sixteen 222.
  a.TT = (backward ? 4 : 8) * (kThreads / a.R) / heads;
  if (a.TT > tokens / 512) a.TT = (int)(tokens / 512);
  if (half && a.TT * half > 4096) a.TT = 4096 / half;
  if (a.TT < 1) a.TT = 1;
  const long long n_blocks = (tokens + a.TT - 1) / a.TT;
  size_t lds = sizeof(float2) * a.TT * half + sizeof(float) * 2 * a.D;
  constexpr bool kMore = kEdge && sizeof(T) == 4;    // more items than a wave has lanes: at most 66
  auto run = [&](auto kernel, dim3 grid) {
    launch_kernel(kernel, grid, kThreads, lds, st, a);
    return hipGetLastError();
  };
  if (!backward) {
    a.blocks = 0;
    return K == 1 ? run(qk_norm_kernel<T, IL, kEdge, 1, false>, grid_rows(n_blocks))
                  : run(qk_norm_kernel<T, IL, kEdge, kMore ? 2 : 1, false>, grid_rows(n_blocks));
  }
  a.blocks = (int)(n_blocks < kQkNormBlocks ? n_blocks : kQkNormBlocks);
  const size_t red = sizeof(float) * (kThreads / a.R) * 2 * a.D;       // at most 32 KB (two items a lane: 16)
  lds = lds > red ? lds : red;
  hipError_t e = K == 1 ? run(qk_norm_kernel<T, IL, kEdge, 1, true>, dim3(a.blocks))
                        : run(qk_norm_kernel<T, IL, kEdge, kMore ? 2 : 1, true>, dim3(a.blocks));
  if (e != hipSuccess || !a.part) return e;
  launch_kernel(qk_norm_sum_kernel, dim3((2 * a.D + 15) / 16), kThreads, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm(QkNormArgs& a, bool bf16, bool aligned, bool interleaved, bool backward, hipStream_t st) {
  const int V = bf16 ? 8 : 4;
  // aligned rows whose turned part, its half (in halves) and the rest consist of whole vectors
  const bool whole = aligned && a.D % V == 0 && a.rot % V == 0 && (interleaved || a.rot / 2 % V == 0);
  auto go = [&](auto t) {
    using T = decltype(t);
    if (interleaved) return whole ? launch_t<T, true, false>(a, backward, st) : launch_t<T, true, true>(a, backward, st);
    return whole ? launch_t<T, false, false>(a, backward, st) : launch_t<T, false, true>(a, backward, st);
  };
  return bf16 ? go(__bf16()) : go(float());
}

}  // namespace kata
