// Layer norm over the last axis, forward and backward, gfx950.
//
//   hat = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  y = hat w + b
//   dx = rstd (t - sum(t) / N - hat sum(t hat) / N),  t = dy w
//   dw = sum over rows of dy hat,  db = sum over rows of dy
//
// A row stays in the registers of R lanes (K vectors of V elements each) between its statistics
// and its result, so every element is read once and written once; the variance is the second
// pass over those registers, of differences from the mean.  All sums are fp32.  A workgroup
// walks over many rows: w and b are read once, and the backward pass keeps its sums of dw and
// db in registers over its rows, adds them up across its lanes and leaves one partial row pair, which a
// second kernel adds in block order (no atomics: the same result every time).
// Bound: HBM.  32768 x 1024 bf16, calls in a row: forward 24 us (5.6 TB/s, part of it from the Infinity
// Cache; 30 us and 4.4 TB/s for rows that are not there), backward 39 us and 5 us of sums (5.2 TB/s).
// 512 x 1024: 3.3 us forward, latency.  Rows that are not whole, aligned vectors take unaligned 16-byte
// accesses and single elements at their end (kEdge; 8192 x 4097: 33 and 101 us, element by element 63
// and 110; 16384 x 2047: 38 and 66, 65 and 142).  Rows wider than the widest register form (8192
// elements) go through the loop kernels, which read a row again for each pass (from the L2 cache
// where it fits).
#include "device.h"
#include "layer.h"
#include "layer_plan.h"
#include "mfma_util.h"

namespace kata {
namespace {

constexpr int kThreads = 256;

// The 16 bytes of V elements; kEdge: at any element, which this card's global memory allows.
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Unaligned {
  u32x4 u;
};

// V elements from column c on; kEdge: rows of any length and alignment, zeros behind N.
template <typename T, int V, bool kEdge>
__device__ __forceinline__ void load_vec(float (&x)[V], const T* p, int c, int N) {
  if (kEdge && c + V > N) {
#pragma unroll
    for (int r = 0; r < V; ++r) x[r] = c + r < N ? to_f32(p[c + r]) : 0.f;
    return;
  }
  const u32x4 u = kEdge ? reinterpret_cast<const Unaligned<T>*>(p + c)->u
                        : *reinterpret_cast<const u32x4*>(p + c);
  if constexpr (sizeof(T) == 2) {
    x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
    x[4] = bf_lo(u.z); x[5] = bf_hi(u.z); x[6] = bf_lo(u.w); x[7] = bf_hi(u.w);
  } else {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
}
template <typename T, int V, bool kEdge>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V], int c, int N) {
  if (kEdge && c + V > N) {
#pragma unroll
    for (int r = 0; r < V; ++r)
      if (c + r < N) p[c + r] = from_f32<T>(x[r]);
    return;
  }
  u32x4 u;
  if constexpr (sizeof(T) == 2)
    u = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  else
    u = u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  if (kEdge) reinterpret_cast<Unaligned<T>*>(p + c)->u = u;
  else *reinterpret_cast<u32x4*>(p + c) = u;
}

__device__ __forceinline__ float param(const void* p, int bf16, int i, float none) {
  if (!p) return none;
  return bf16 ? (float)reinterpret_cast<const __bf16*>(p)[i] : reinterpret_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_param(void* p, int bf16, int i, float x) {
  if (!p) return;
  if (bf16) reinterpret_cast<__bf16*>(p)[i] = (__bf16)x;
  else reinterpret_cast<float*>(p)[i] = x;
}

// V neighbouring parameters from column c on; `none` where there are none or behind N.
template <int V, bool kEdge>
__device__ __forceinline__ void load_params(float (&x)[V], const void* p, int bf16, int c, int N, float none) {
#pragma unroll
  for (int r = 0; r < V; ++r) x[r] = none;
  if (!p || c >= N) return;
  if (kEdge && c + V > N) {
#pragma unroll
    for (int r = 0; r < V; ++r)
      if (c + r < N) x[r] = param(p, bf16, c + r, none);
  } else if (bf16) {
    const __bf16* b = reinterpret_cast<const __bf16*>(p) + c;
#pragma unroll
    for (int r = 0; r < V; ++r) x[r] = (float)b[r];
  } else {
    const float* f = reinterpret_cast<const float*>(p) + c;
#pragma unroll
    for (int r = 0; r < V; ++r) x[r] = f[r];
  }
}

// Sum over the R lanes of a row, in every one of them.  R = 256: over the workgroup, through
// `sh` (4 floats; every thread calls it, twice in a row with two buffers).
template <int R>
__device__ __forceinline__ float row_sum(float x, float* sh) {
#pragma unroll
  for (int m = (R < 64 ? R : 64) / 2; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  if constexpr (R == 256) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (sh[0] + sh[1]) + (sh[2] + sh[3]);
    __syncthreads();
  }
  return x;
}

template <typename T, int V, int R, int K, bool kEdge>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs A) {
  __shared__ float sh[4];
  constexpr int RPB = kThreads / R;                 // rows at a time
  const int l = threadIdx.x % R, N = A.N;
  float w[K][V], b[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_params<V, kEdge>(w[k], A.w, A.w_bf16, (k * R + l) * V, N, 1.f);
    load_params<V, kEdge>(b[k], A.b, A.w_bf16, (k * R + l) * V, N, 0.f);
  }
  const float n = (float)N;
  // R = 256: one row at a time, so all threads leave the loop together
  for (long long row = (long long)blockIdx.x * RPB + threadIdx.x / R; row < A.rows;
       row += (long long)gridDim.x * RPB) {
    const T* px = reinterpret_cast<const T*>(A.x) + row * A.sx;
    float x[K][V], sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * R + l) * V;
#pragma unroll
      for (int r = 0; r < V; ++r) x[k][r] = 0.f;
      if (c < N) load_vec<T, V, kEdge>(x[k], px, c, N);
#pragma unroll
      for (int r = 0; r < V; ++r) sum += x[k][r];
    }
    const float mean = row_sum<R>(sum, sh) / n;   // a division: a constant row has its value as mean
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int r = 0; r < V; ++r) {
        x[k][r] = (k * R + l) * V + (kEdge ? r : 0) < N ? x[k][r] - mean : 0.f;
        sq = fmaf(x[k][r], x[k][r], sq);
      }
    const float rstd = 1.f / sqrtf(row_sum<R>(sq, sh) / n + A.eps);
    T* py = reinterpret_cast<T*>(A.y) + row * A.sy;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * R + l) * V;
#pragma unroll
      for (int r = 0; r < V; ++r) x[k][r] = fmaf(x[k][r] * rstd, w[k][r], b[k][r]);
      if (c < N) store_vec<T, V, kEdge>(py, x[k], c, N);
    }
    if (l == 0 && A.mean) {
      A.mean[row] = mean;
      A.rstd[row] = rstd;
    }
  }
}

template <typename T, int V, int R, int K, bool kEdge>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs A) {
  constexpr int RPB = kThreads / R, W = R < 64 ? R : 64;
  __shared__ float sh[4];
  __shared__ float cross[R == 256 ? 1 : 4 * W * V];
  const int tid = threadIdx.x, l = tid % R, N = A.N;
  float w[K][V], gw[K][V], gb[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_params<V, kEdge>(w[k], A.w, A.w_bf16, (k * R + l) * V, N, 1.f);
#pragma unroll
    for (int r = 0; r < V; ++r) gw[k][r] = gb[k][r] = 0.f;
  }
  const float n = (float)N;
  for (long long row = (long long)blockIdx.x * RPB + tid / R; row < A.rows;
       row += (long long)gridDim.x * RPB) {
    const T* px = reinterpret_cast<const T*>(A.x) + row * A.sx;
    const T* pg = reinterpret_cast<const T*>(A.dy) + row * A.sdy;
    const float mean = A.mean[row], rstd = A.rstd[row];
    float hat[K][V], t[K][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * R + l) * V;
#pragma unroll
      for (int r = 0; r < V; ++r) hat[k][r] = t[k][r] = 0.f;
      if (c < N) {
        load_vec<T, V, kEdge>(hat[k], px, c, N);
        load_vec<T, V, kEdge>(t[k], pg, c, N);
#pragma unroll
        for (int r = 0; r < V; ++r) hat[k][r] = !kEdge || c + r < N ? (hat[k][r] - mean) * rstd : 0.f;
      }
#pragma unroll
      for (int r = 0; r < V; ++r) {
        gw[k][r] = fmaf(t[k][r], hat[k][r], gw[k][r]);
        gb[k][r] += t[k][r];
        t[k][r] *= w[k][r];
        s1 += t[k][r];
        s2 = fmaf(t[k][r], hat[k][r], s2);
      }
    }
    s1 = row_sum<R>(s1, sh) / n;
    s2 = row_sum<R>(s2, sh) / n;
    if (A.dx) {
      T* pd = reinterpret_cast<T*>(A.dx) + row * A.sdx;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * R + l) * V;
#pragma unroll
        for (int r = 0; r < V; ++r) t[k][r] = (t[k][r] - s1 - hat[k][r] * s2) * rstd;
        if (c < N) store_vec<T, V, kEdge>(pd, t[k], c, N);
      }
    }
  }
  if (!A.part) return;
  float* part = A.part + (long long)blockIdx.x * 2 * N;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float y[V];
#pragma unroll
      for (int r = 0; r < V; ++r) y[r] = which ? gb[k][r] : gw[k][r];
      if constexpr (R < 256) {                      // add up the rows taken side by side
#pragma unroll
        for (int r = 0; r < V; ++r)
#pragma unroll
          for (int m = R; m < 64; m <<= 1) y[r] += __shfl_xor(y[r], m);
        __syncthreads();
        if ((tid & 63) < W)
#pragma unroll
          for (int r = 0; r < V; ++r) cross[((tid >> 6) * W + (tid & 63)) * V + r] = y[r];
        __syncthreads();
        if (tid < W)
#pragma unroll
          for (int r = 0; r < V; ++r)
            y[r] = (cross[tid * V + r] + cross[(W + tid) * V + r]) +
                   (cross[(2 * W + tid) * V + r] + cross[(3 * W + tid) * V + r]);
      }
      if (R == 256 || tid < W)
#pragma unroll
        for (int r = 0; r < V; ++r) {
          const int c = (k * R + l) * V + r;
          if (c < N) {
            if (gridDim.x > 1) part[(long long)which * N + c] = y[r];
            else store_param(which ? A.db : A.dw, A.w_bf16, c, y[r]);
          }
        }
    }
}

// dw and db from the blocks' partial sums: 32 columns of a workgroup, 32 slices of the blocks, each
// added in order with eight loads in flight (one at a time took 19 us for 1024 blocks of 1024
// columns, all of it latency).
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormArgs A) {
  __shared__ float sh[32][33];
  const int col = threadIdx.x & 31, s = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
  const int which = blockIdx.y, per = (A.blocks + 31) / 32;
  const int i0 = s * per, i1 = min(A.blocks, i0 + per);
  float sum = 0.f;
  if (c < A.N) {
    const float* p = A.part + (long long)which * A.N + c;
    const long long step = 2LL * A.N;
    for (int i = i0; i < i1; i += 8) {
      float x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) x[r] = i + r < i1 ? p[(i + r) * step] : 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) sum += x[r];
    }
  }
  sh[s][col] = sum;
  __syncthreads();
  if (s == 0 && c < A.N) {
    for (int i = 1; i < 32; ++i) sum += sh[i][col];
    store_param(which ? A.db : A.dw, A.w_bf16, c, sum);
  }
}

// ---- rows of any width ------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_fwd_loop_kernel(NormArgs A) {
  __shared__ float sh[4];
  const int N = A.N;
  const float n = (float)N;
  for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const T* px = reinterpret_cast<const T*>(A.x) + row * A.sx;
    T* py = reinterpret_cast<T*>(A.y) + row * A.sy;
    float sum = 0.f, sq = 0.f;
    for (int c = threadIdx.x; c < N; c += kThreads) sum += to_f32(px[c]);
    const float mean = row_sum<256>(sum, sh) / n;
    for (int c = threadIdx.x; c < N; c += kThreads) {
      const float d = to_f32(px[c]) - mean;
      sq = fmaf(d, d, sq);
    }
    const float rstd = 1.f / sqrtf(row_sum<256>(sq, sh) / n + A.eps);
    for (int c = threadIdx.x; c < N; c += kThreads)
      py[c] = from_f32<T>(fmaf((to_f32(px[c]) - mean) * rstd, param(A.w, A.w_bf16, c, 1.f),
                               param(A.b, A.w_bf16, c, 0.f)));
    if (threadIdx.x == 0 && A.mean) {
      A.mean[row] = mean;
      A.rstd[row] = rstd;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_dx_loop_kernel(NormArgs A) {
  __shared__ float sh[4];
  const int N = A.N;
  const float n = (float)N;
  for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const T* px = reinterpret_cast<const T*>(A.x) + row * A.sx;
    const T* pg = reinterpret_cast<const T*>(A.dy) + row * A.sdy;
    T* pd = reinterpret_cast<T*>(A.dx) + row * A.sdx;
    const float mean = A.mean[row], rstd = A.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < N; c += kThreads) {
      const float t = to_f32(pg[c]) * param(A.w, A.w_bf16, c, 1.f);
      s1 += t;
      s2 = fmaf(t, (to_f32(px[c]) - mean) * rstd, s2);
    }
    s1 = row_sum<256>(s1, sh) / n;
    s2 = row_sum<256>(s2, sh) / n;
    for (int c = threadIdx.x; c < N; c += kThreads) {
      const float t = to_f32(pg[c]) * param(A.w, A.w_bf16, c, 1.f);
      pd[c] = from_f32<T>((t - s1 - (to_f32(px[c]) - mean) * rstd * s2) * rstd);
    }
  }
}

// Partial sums of dw and db: a column a thread, the rows of block y.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_dw_loop_kernel(NormArgs A) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= A.N) return;
  float gw = 0.f, gb = 0.f;
  for (long long row = blockIdx.y; row < A.rows; row += gridDim.y) {
    const float g = to_f32(reinterpret_cast<const T*>(A.dy)[row * A.sdy + c]);
    const float x = to_f32(reinterpret_cast<const T*>(A.x)[row * A.sx + c]);
    gw = fmaf(g, (x - A.mean[row]) * A.rstd[row], gw);
    gb += g;
  }
  float* part = A.part + (long long)blockIdx.y * 2 * A.N + c;
  part[0] = gw;
  part[A.N] = gb;
}

template <typename T, bool kEdge, bool kBwd>
bool launch_rows(NormArgs& a, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (a.N > kNormInRegisters) return false;
  const int nv = (a.N + V - 1) / V;
  auto run = [&](auto fwd, auto bwd, int rpb, int held) {
    const long long want = (a.rows + rpb - 1) / rpb;
    // Backward: three workgroups a CU, as one or two leave less in flight and four more partial rows to
    // add (32768 x 1024 bf16: 39.9 us; 1024 workgroups 41.3, 512 40.4, 256 60; 65536 x 512: 40.8, 40.9,
    // 45.9, 76), two where their rows are few (4096 x 1024: 13.6 us with 512, 16.7 with 768, 18.6
    // with 1024) and where no more fit (32 elements a thread in registers).
    const int most = !kBwd ? 2048 : want < 4 * kNormBlocks || held >= 32 ? 512 : kNormBlocks;
    // A few rows: one workgroup, whose sums are the gradients, instead of a second kernel (8 x 1024, two
    // turns: 7.6 us for 8.1 and a launch less; four turns: 9.8).
    a.blocks = kBwd && want <= 2 ? 1 : (int)(want < most ? want : most);
    launch_kernel(kBwd ? bwd : fwd, dim3(a.blocks), kThreads, 0, st, a);
    return true;
  };
#define KATA_NORM(R_, K_)                                                                       \
  if (nv <= R_ * K_)                                                                            \
    return run(norm_fwd_kernel<T, V, R_, K_, kEdge>, norm_bwd_kernel<T, V, R_, K_, kEdge>, kThreads / R_, K_ * V);
  KATA_NORM(8, 1) KATA_NORM(16, 1) KATA_NORM(32, 1) KATA_NORM(64, 1) KATA_NORM(64, 2)
  KATA_NORM(64, 3) KATA_NORM(64, 4) KATA_NORM(256, 2) KATA_NORM(256, 3) KATA_NORM(256, 4)
  if constexpr (V == 4) KATA_NORM(256, 8)           // 32 elements a thread, as of bf16 rows
#undef KATA_NORM
  static_assert(kNormInRegisters == 256 * (V == 4 ? 8 : 4) * V, "the widest of them");
  return false;
}

template <typename T>
hipError_t fwd_t(NormArgs& a, bool whole, hipStream_t st) {
  if (whole ? launch_rows<T, false, false>(a, st) : launch_rows<T, true, false>(a, st)) return hipGetLastError();
  launch_kernel(norm_fwd_loop_kernel<T>, dim3((unsigned)(a.rows < 2048 ? a.rows : 2048)), kThreads, 0, st, a);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_t(NormArgs& a, bool whole, hipStream_t st) {
  const bool rows = whole ? launch_rows<T, false, true>(a, st) : launch_rows<T, true, true>(a, st);
  if (!rows) {
    // dw and db first: dx may overwrite dy
    a.blocks = (int)(a.rows < kNormLoopBlocks ? a.rows : kNormLoopBlocks);
    if (a.part)
      launch_kernel(norm_dw_loop_kernel<T>, dim3((a.N + kThreads - 1) / kThreads, a.blocks), kThreads, 0, st, a);
    if (a.dx)
      launch_kernel(norm_dx_loop_kernel<T>, dim3((unsigned)(a.rows < 2048 ? a.rows : 2048)), kThreads, 0, st, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part || (rows && a.blocks == 1)) return e;
  launch_kernel(norm_sum_kernel, dim3((a.N + 31) / 32, 2), 1024, 0, st, a);
  return hipGetLastError();
}

// Rows of whole, aligned vectors.
bool vectors(const NormArgs& a, bool bf16, bool aligned) { return aligned && a.N % (bf16 ? 8 : 4) == 0; }

}  // namespace

hipError_t launch_norm_fwd(NormArgs& a, bool bf16, bool aligned, hipStream_t st) {
  return bf16 ? fwd_t<__bf16>(a, vectors(a, bf16, aligned), st) : fwd_t<float>(a, vectors(a, bf16, aligned), st);
}
hipError_t launch_norm_bwd(NormArgs& a, bool bf16, bool aligned, hipStream_t st) {
  return bf16 ? bwd_t<__bf16>(a, vectors(a, bf16, aligned), st) : bwd_t<float>(a, vectors(a, bf16, aligned), st);
}

}  // namespace kata
