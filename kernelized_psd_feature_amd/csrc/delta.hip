// Gated delta rule, gfx950: chunked form and recurrent form.
//
//   S_t = g_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   o_t = scale S_t^T q_t
//
// Chunk of 64 tokens with entry state S (the state behind the token before it), c_i the sum of the log
// decays of its tokens 0 .. i, y_i = exp(c_i):
//   A_ij = b_i exp(c_i - c_j) (k_i . k_j) for j < i, else 0
//   U = (I + A)^-1 diag(b) (V - diag(y) K S)
//   o = scale (diag(y) Q S + P U),  P_ij = exp(c_i - c_j) (q_i . k_j) for j <= i
//   S <- y_63 S + sum_j exp(c_63 - c_j) k_j u_j^T
// The inverses need no state: the first pass forms them for all chunks at once (delta_prep_kernel).
// The walk then runs the chunks of a sequence one after the other; everything in it that depends on S
// belongs to single columns of the values, so a wave takes 16 of them and passes S, X = b (V - y K S) and U
// from product to product in registers.
//
// A chunk maps S to M S + N.  Where sequences and heads do not fill the card, a sequence is cut into
// segments of L chunks: a pass over each of them gives its N (the recurrence from a state of zero) and its
// M (the recurrence from the unit matrix, without values), delta_join_kernel turns them into entry states,
// and the walk runs the segments side by side.
//
// Where the time goes (131072 tokens, 16 bf16 heads of 64): inverses 178 us, sums 393, joining 27, walk 476, for
// 215 us of reading q, k, v and writing o once.  A chunk is a chain of products (K S, T X, K^T U), each of operands
// that are split anew into bf16 terms out of the last one's fp32 sums, with LDS reads and two or three barriers
// between; two workgroups a CU hide part of each other's (sums: VALU 70 % of the cycles, LDS 60, MFMA 44; walk 51, 46,
// 27).  The terms are the price of a chain: one of them is 2^-8 of a value, which the recurrence would carry from chunk
// to chunk; with three the final state is off by 1.6e-7 of its norm, plain fp32 by 2.1e-7.
#include <type_traits>

#include "delta.h"
#include "delta_tiles.h"
#include "delta_walk.h"
#include "device.h"
#include "mfma_util.h"

namespace kata {
namespace {

constexpr int kThreads = 256;             // of the kernels other than the walk

// ---- inverses --------------------------------------------------------------------------------
// 178 us for 131072 tokens of 16 heads of 64 (reads k, writes 11.5 KB a chunk and head: 3.6 TB/s).  The
// substitution is exact to rounding for keys of any length; powers of A, which MFMA could take, grow with them.
// One workgroup for a chunk and head.  A wave forms a strip of 16 rows of A (fp32 sums on MFMA); the four
// blocks on the diagonal are inverted by substitution, 16 lanes a block, a column each; below them
// T_ij = -D_i sum_{j <= k < i} A_ik T_kj, a wave a block column, on the fp32 MFMA.
template <typename T, int DK>
struct PrepTiles {
  static constexpr int LK = DK + 16 / (int)sizeof(T), LD = 20;
  static constexpr int kHead = 16 + 3 * kC * 4;                        // an int, c in two floats, beta
  static constexpr int kKeys = kC * LK * (int)sizeof(T);               // then the diagonal's inverses
  static constexpr int bytes = kHead + kKeys + kInvBlocks * 16 * LD * 4;
  static_assert(kC * LD * 4 <= kKeys, "the inverses lie where the keys were");
};

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void delta_prep_kernel(DeltaArgs A) {
  using TL = PrepTiles<T, DK>;
  using frag = typename Elem<T>::frag;
  constexpr int M = DK / 32, LK = TL::LK, LD = TL::LD;
  extern __shared__ __align__(16) char lds[];
  int* const sh = reinterpret_cast<int*>(lds);
  float* const sc = reinterpret_cast<float*>(lds + 16);
  float* const sb = sc + 2 * kC;
  T* const sK = reinterpret_cast<T*>(lds + TL::kHead);
  float* const sD = reinterpret_cast<float*>(lds + TL::kHead);
  float* const sA = reinterpret_cast<float*>(lds + TL::kHead + TL::kKeys);   // blocks [16][LD], row by row of them
  auto block = [&](int i, int j) __attribute__((always_inline)) { return sA + (i * (i + 1) / 2 + j) * 16 * LD; };

  const DeltaMap& m = A.m;
  const unsigned unit = block_number();
  if (unit >= (unsigned)m.c_slots * (unsigned)m.H) return;
  const int slot = int(unit / (unsigned)m.H), h = int(unit - (unsigned)slot * (unsigned)m.H);
  DeltaPart s;
  if (!find_part(m, slot, 1, m.n_chunks, m.c_slots, sh, kThreads, s) || s.seq == m.n_seq) return;
  const int row0 = s.start + kC * s.part, n = min(kC, s.len - kC * s.part);
  if (n <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

  Stage<T, DK, kThreads> rk(reinterpret_cast<const T*>(A.k) + s.b * A.sk[0] + row0 * A.sk[1] + (h / (m.H / m.Hk)) * A.sk[2],
                            A.sk[1], m.dk, true);
  fetch_rows(rk, A.sk[1], n);
  if (m.dk < DK)
    for (int i = tid; i < kC * LK * (int)sizeof(T) / 16; i += kThreads)
      reinterpret_cast<uint4*>(sK)[i] = uint4{0u, 0u, 0u, 0u};
  float* const vec = A.vec + (long long)unit * kDeltaVec;
  if (w == 0) {
    float ld = 0.f, b = 0.f;
    if (lane < n) {
      b = to_f32(reinterpret_cast<const T*>(A.beta)[row_off(A.sb, s.b, row0 + lane, h)]);
      if (A.log_decay) ld = A.log_decay[row_off(A.sl, s.b, row0 + lane, h)];
      if (ld < -256.f) ld = -256.f;                 // exp of it is zero in fp32; sums of 64 stay finite
    }
    double c = ld * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(c, d);
      if (lane >= d) c += up;
    }
    const double left = __shfl(c, 63) - c;
    const float hi = (float)c, lo = hi - hi == 0.f ? (float)(c - hi) : hi;
    sc[lane] = hi;
    sc[kC + lane] = lo;
    sb[lane] = b;
    vec[lane] = exp2_diff(hi, lo, 0.f, 0.f);
    vec[kC + lane] = exp2_diff((float)left, (float)(left - (float)left), 0.f, 0.f);
    vec[2 * kC + lane] = b;
    vec[3 * kC + lane] = hi;
    vec[4 * kC + lane] = lo;
  }
  if (m.dk < DK) __syncthreads();
  keep_rows(rk, n);
  rk.template put_split<LK>(sK);
  __syncthreads();

  // A: rows 16 w + 4 g + r, columns 16 j + l16
  frag ka[M];
#pragma unroll
  for (int i = 0; i < M; ++i) ka[i] = row_frag(sK + (16 * w + l16) * LK + 32 * i + 8 * g);
  f32x4 sick = zero4();
  for (int j = 0; j <= w; ++j) {                    // uniform
    f32x4 acc = zero4();
#pragma unroll
    for (int i = 0; i < M; ++i) acc = mma(ka[i], row_frag(sK + (16 * j + l16) * LK + 32 * i + 8 * g), acc);
    const int col = 16 * j + l16;
    const float hj = sc[col], lj = sc[kC + col];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r;
      const float a = col < row ? sb[row] * exp2_diff(sc[row], sc[kC + row], hj, lj) * acc[r] : 0.f;
      sick[r] = fmaf(a, 0.f, sick[r]);
      block(w, j)[(4 * g + r) * LD + l16] = a;
    }
  }
  // A row with an infinity or nan would leave nan in earlier rows of the inverse: it is taken as zeros, and
  // its beta as nan, which makes the row's correction nan in the walk.
  if (__any(sick[0] + sick[1] + sick[2] + sick[3] != 0.f))
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) sick[r] += __shfl_xor(sick[r], d);
      if (sick[r] != 0.f) {
        for (int j = 0; j <= w; ++j) block(w, j)[(4 * g + r) * LD + l16] = 0.f;
        if (l16 == 0) vec[2 * kC + 16 * w + 4 * g + r] = __builtin_nanf("");
      }
    }
  __syncthreads();
  if (w == 0) {                                     // block g, column l16: x = e - A x
    float x[16];
    const float* a = block(g, g);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) y = fmaf(-a[i * LD + j], x[j], y);
      x[i] = y;
      sD[(16 * g + i) * LD + l16] = y;
    }
  }
  __syncthreads();
  // block column w
  float* const inv = A.inv + (long long)unit * kInvFloats;
  f32x4 t[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) t[0][r] = sD[(16 * w + 4 * g + r) * LD + l16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                     // block row w + i
    if (w + i > 3) break;                           // uniform
    const int bi = w + i;
    if (i > 0) {
      f32x4 acc = zero4();
#pragma unroll
      for (int k = 0; k < i; ++k) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(block(bi, w + k) + l16 * LD + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], t[k][r], acc, 0, 0, 0);
      }
      const f32x4 d = *reinterpret_cast<const f32x4*>(sD + (16 * bi + l16) * LD + 4 * g);
      // (a sum that overflows would meet the zeros above D's diagonal: it enters its own row alone)
      f32x4 over;
      t[i] = zero4();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool fits = fabsf(acc[r]) < __builtin_huge_valf();
        over[r] = fits ? 0.f : __builtin_nanf("");
        acc[r] = fits ? acc[r] : 0.f;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) t[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(-d[r], acc[r], t[i], 0, 0, 0);
      t[i] += over;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) inv[(bi * (bi + 1) / 2 + w) * 256 + (4 * g + r) * 16 + l16] = t[i][r];
  }
}

template <typename T, int DK, int W, int NT, Walk kWhat>
__global__ __launch_bounds__(64 * W, (WalkTiles<T, DK, W, NT, kWhat == Walk::output>::occupancy)) void delta_walk_kernel(
    DeltaArgs A, int blocks) {
  extern __shared__ __align__(16) char lds[];
  const UnitBlock u = unit_block(blocks);
  delta_walk<T, DK, W, NT, kWhat>(A, u.unit, u.sub, 0, lds);
}

// ---- joining segments ---------------------------------------------------------------------------
// Per (sequence, head) and 16 columns, over the segments in order: E_{j+1} = M_j E_j + N_j; the sum in slot
// j is replaced by the entry state E_j.  Backward also in reversed time: D_{j-1} = M_j^T D_j + N'_j, the
// sum in slot j replaced by D_j, the gradient of the state behind the segment.  On the fp32 MFMA; the rows are
// split over the waves, which pass the state through LDS, and kAhead steps' transitions are on their way (0.8 us a
// step at 64, where one launch a step would be 4; with loads under conditions 1.4).
template <int DK, bool kRev>
__device__ __forceinline__ void join(const DeltaArgs& A, int sub, int h, int seq, float (&sS)[2][16 * (DK + 4)]) {
  constexpr int M = DK / 32, NS = DK / 16, R = (NS + 3) / 4, LS = DK + 4, kAhead = DK > 64 ? 2 : 4;
  const DeltaMap& m = A.m;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), SL = kC * m.L;
  int slot = seq * m.n_seg, len = m.T;
  if (m.packed) {
    const int first = cu_at(m, seq);
    slot = decay_first_slot(first, seq, SL);
    len = max(cu_at(m, seq + 1) - first, 0);
  }
  const int n = (len + SL - 1) / SL;
  if (n < 2) return;
  const int col = 16 * sub + l16, SE = m.dk * m.dv, ME = m.dk * m.dk;
  float* const sums = kRev ? A.rsums : A.sums;
  const float* given = kRev ? A.dfin : A.init;
  const bool live = col < m.dv;
  auto place = [&](int j) __attribute__((always_inline)) { return (long long)(slot + (kRev ? n - 1 - j : j)) * m.H + h; };
  f32x4 S[R], N[kAhead][R];
  f32x8 a[kAhead][R][M];
  // No load under a condition (see fetch_rows), so places behind the state's ends are others' again.
  auto fetch = [&](int j, int to) __attribute__((always_inline)) {     // `to`: known where this is unrolled
    const long long at = place(min(j, n - 2));      // the last segment's are not used
    const float* const here = sums + at * SE + min(col, m.dv - 1);
    const float* const tr = A.trans + at * ME;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int tile = w * R + i, row = min(16 * tile + l16, m.dk - 1);
#pragma unroll
      for (int r = 0; r < 4; ++r) N[to][i][r] = here[min(16 * tile + 4 * g + r, m.dk - 1) * m.dv];
#pragma unroll
      for (int k = 0; k < M; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int q = min(32 * k + 16 * half + 4 * g, m.dk - 4);     // widths are multiples of four
          f32x4 x;
          if constexpr (kRev)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = tr[(q + r) * m.dk + row];
          else
            x = *reinterpret_cast<const f32x4*>(tr + row * m.dk + q);
#pragma unroll
          for (int r = 0; r < 4; ++r) a[to][i][k][4 * half + r] = x[r];
        }
    }
  };
  const float* const entry = (given ? given + ((long long)seq * m.H + h) * SE : sums + place(0) * SE) + min(col, m.dv - 1);
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[i][r] = entry[min(16 * (w * R + i) + 4 * g + r, m.dk - 1) * m.dv];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) fetch(j, j);
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!given || !live || 16 * (w * R + i) + 4 * g + r >= m.dk) S[i][r] = 0.f;
  for (int j0 = 0; j0 < n; j0 += kAhead)
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int j = j0 + s;
      if (j >= n) break;                            // uniform
      float* const here = sums + place(j) * SE;
      float* const buf = sS[j & 1];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int tile = w * R + i;
        if (tile < NS) *reinterpret_cast<f32x4*>(buf + l16 * LS + split_place(16 * tile + 4 * g)) = S[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int y = 16 * tile + 4 * g + r;
          if (live && y < m.dk) here[y * m.dv + col] = S[i][r];
        }
      }
      if (j + 1 >= n) break;
      __syncthreads();
      f32x4 odd[R];
#pragma unroll
      for (int i = 0; i < R; ++i) odd[i] = zero4();
      if (j > 0 || given)                           // else the state is zero, and the transition is not there
#pragma unroll
        for (int k = 0; k < M; ++k) {
          const f32x8 b = row_frag(buf + l16 * LS + 32 * k + 8 * g);
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int r = 0; r < 8; r += 2) {
              N[s][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s][i][k][r], b[r], N[s][i], 0, 0, 0);
              odd[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s][i][k][r + 1], b[r + 1], odd[i], 0, 0, 0);
            }
        }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        S[i] = N[s][i] + odd[i];
        before_branch(S[i]);
        if (m.dk < DK)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * (w * R + i) + 4 * g + r >= m.dk) S[i][r] = 0.f;
      }
      fetch(j + kAhead, s);
    }
}

template <int DK>
__global__ __launch_bounds__(kThreads) void delta_join_kernel(DeltaArgs A, int blocks) {
  __shared__ __align__(16) float sS[2][16 * (DK + 4)];
  unsigned x = blockIdx.x;                          // sequences: blockIdx.y
  const int sub = int(x % (unsigned)blocks);
  x /= (unsigned)blocks;
  const int h = int(x % (unsigned)A.m.H);
  if (x / (unsigned)A.m.H) join<DK, true>(A, sub, h, blockIdx.y, sS);
  else join<DK, false>(A, sub, h, blockIdx.y, sS);
}

// ---- recurrent form ------------------------------------------------------------------------
// One workgroup per (column block, head, sequence) keeps its part of the state in registers over the call's
// tokens: thread (row group, lane group) has 4 neighbouring columns of the rows row group + RG i.  Both
// products with the state are taken of the one before the token, in one pass over the rows:
//   a = S^T k, z = S^T q, u = b (v - g a), o = scale (g z + (q . k) u), S <- g S + k u^T.
// Bound by the state's two ways through HBM: 512 sequences of 16 heads of 64 x 64, 54.5 us, 5.0 TB/s, what a copy
// reaches.  One sequence: 4.7 us, a launch and one pass of loads.  Of 128 x 128 the
// state takes 192 registers a lane, which leaves too few waves to keep the loads going: 256 sequences 167 us, 3.2 TB/s.
struct TokenArgs {
  int T, H, share, dk, dv;
  long long sq[3], sk[3], sv[3], so[3], sb[3], sl[3];
  float scale;
};

template <typename T, int LC, int RI>
__global__ __launch_bounds__(kThreads) void delta_decode_kernel(
    TokenArgs A, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const T* __restrict__ beta, const float* __restrict__ log_decay, float* __restrict__ state, T* __restrict__ o) {
  constexpr int RG = kThreads / LC;
  __shared__ f32x4 part[2][4][2][LC];
  __shared__ float dots[2][4];
  const int tid = threadIdx.x, rg = tid / LC, col = 4 * (blockIdx.x * LC + tid % LC);
  const int h = blockIdx.y, b = blockIdx.z, w = tid >> 6, hk = h / A.share;
  const bool live = col < A.dv;
  float* st = state + ((long long)b * A.H + h) * A.dk * A.dv + col;
  f32x4 S[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = rg + RG * i;
    S[i] = zero4();
    if (live && row < A.dk) S[i] = load4(st + row * A.dv);
  }
  for (int t = 0; t < A.T; ++t) {
    const T* qt = q + row_off(A.sq, b, t, hk);
    const T* kt = k + row_off(A.sk, b, t, hk);
    const f32x4 vt = live ? load4(v + row_off(A.sv, b, t, h) + col) : zero4();
    const float bt = to_f32(beta[row_off(A.sb, b, t, h)]);
    const float gt = log_decay ? expf(log_decay[row_off(A.sl, b, t, h)]) : 1.f;
    f32x4 a = zero4(), z = zero4();
    float kr[RI], qk = 0.f;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int row = rg + RG * i;
      kr[i] = 0.f;
      if (row < A.dk) {
        kr[i] = to_f32(kt[row]);
        const float qr = to_f32(qt[row]);
        qk = fmaf(qr, kr[i], qk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          a[r] = fmaf(kr[i], S[i][r], a[r]);
          z[r] = fmaf(qr, S[i][r], z[r]);
        }
      }
    }
#pragma unroll
    for (int s = LC; s < 64; s <<= 1) {
      qk += __shfl_xor(qk, s);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a[r] += __shfl_xor(a[r], s);
        z[r] += __shfl_xor(z[r], s);
      }
    }
    const int p = t & 1;                            // two buffers: one barrier a token
    if ((tid & 63) < LC) {
      part[p][w][0][tid % LC] = a;
      part[p][w][1][tid % LC] = z;
      if ((tid & 63) == 0) dots[p][w] = qk;
    }
    __syncthreads();
    a = part[p][0][0][tid % LC] + part[p][1][0][tid % LC] + part[p][2][0][tid % LC] + part[p][3][0][tid % LC];
    const f32x4 u = bt * (vt - gt * a);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = fmaf(kr[i], u[r], gt * S[i][r]);
    if (tid < LC && live) {
      z = part[p][0][1][tid] + part[p][1][1][tid] + part[p][2][1][tid] + part[p][3][1][tid];
      qk = dots[p][0] + dots[p][1] + dots[p][2] + dots[p][3];
      store4(o + row_off(A.so, b, t, h) + col, A.scale * (gt * z + qk * u));
    }
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = rg + RG * i;
    if (live && row < A.dk) *reinterpret_cast<f32x4*>(st + row * A.dv) = S[i];
  }
}

template <typename F>
hipError_t with_lds(F kernel, int bytes) {
  return ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes);
}

template <typename T, int DK>
hipError_t launch_prep_t(const DeltaArgs& a, hipStream_t st) {
  using TL = PrepTiles<T, DK>;
  hipError_t e = with_lds(delta_prep_kernel<T, DK>, TL::bytes);
  if (e != hipSuccess) return e;
  launch_kernel(delta_prep_kernel<T, DK>, grid_rows((long long)a.m.c_slots * a.m.H), kThreads, TL::bytes, st, a);
  return hipGetLastError();
}

template <typename T, int DK, int W, int NT, Walk kWhat>
hipError_t launch_walk_t(const DeltaArgs& a, hipStream_t st) {
  using TL = WalkTiles<T, DK, W, NT, kWhat == Walk::output>;
  hipError_t e = with_lds(delta_walk_kernel<T, DK, W, NT, kWhat>, TL::bytes);
  if (e != hipSuccess) return e;
  const int tiles = (a.m.dv + 15) / 16 + (kWhat == Walk::sums ? (a.m.dk + 15) / 16 : 0), blocks = (tiles + W - 1) / W;
  const long long units = (long long)a.m.n_slots * a.m.H;
  launch_kernel(delta_walk_kernel<T, DK, W, NT, kWhat>, grid_rows((units + 7) / 8 * 8 * blocks), 64 * W, TL::bytes, st, a,
                blocks);
  return hipGetLastError();
}

template <Walk kWhat, int NT>
hipError_t launch_walk_bf16(const DeltaArgs& a, hipStream_t st) {
  const int dk = a.m.dk;
  if constexpr (kWhat == Walk::sums) {              // values and transition side by side
    if (dk <= 32 && a.m.dv <= 32) return launch_walk_t<__bf16, 32, 4, NT, kWhat>(a, st);
    return dk <= 64 ? launch_walk_t<__bf16, 64, 8, NT, kWhat>(a, st) : launch_walk_t<__bf16, 128, 8, NT, kWhat>(a, st);
  } else {
    if (decay_columns(true, a.m.dv) == 128)
      return dk <= 64 ? launch_walk_t<__bf16, 64, 8, NT, kWhat>(a, st) : launch_walk_t<__bf16, 128, 8, NT, kWhat>(a, st);
    return dk <= 32 ? launch_walk_t<__bf16, 32, 4, NT, kWhat>(a, st)
           : dk <= 64 ? launch_walk_t<__bf16, 64, 4, NT, kWhat>(a, st) : launch_walk_t<__bf16, 128, 4, NT, kWhat>(a, st);
  }
}

// States that the caller keeps are computed with three terms.
template <Walk kWhat>
hipError_t launch_walk_d(const DeltaArgs& a, bool bf16, hipStream_t st) {
  const int dk = a.m.dk;
  if (!bf16) return dk <= 32 ? launch_walk_t<float, 32, 4, 1, kWhat>(a, st)
                  : dk <= 64 ? launch_walk_t<float, 64, 4, 1, kWhat>(a, st) : launch_walk_t<float, 128, 4, 1, kWhat>(a, st);
  return a.fin ? launch_walk_bf16<kWhat, 3>(a, st) : launch_walk_bf16<kWhat, 2>(a, st);
}

}  // namespace

hipError_t launch_delta_prep(const DeltaArgs& a, bool bf16, hipStream_t st) {
  const int dk = a.m.dk;
  if (bf16) return dk <= 32 ? launch_prep_t<__bf16, 32>(a, st)
                 : dk <= 64 ? launch_prep_t<__bf16, 64>(a, st) : launch_prep_t<__bf16, 128>(a, st);
  return dk <= 32 ? launch_prep_t<float, 32>(a, st)
         : dk <= 64 ? launch_prep_t<float, 64>(a, st) : launch_prep_t<float, 128>(a, st);
}

hipError_t launch_delta_segments(const DeltaArgs& a, bool bf16, hipStream_t st) {
  return launch_walk_d<Walk::sums>(a, bf16, st);
}

hipError_t launch_delta_walk(const DeltaArgs& a, bool bf16, hipStream_t st) {
  return launch_walk_d<Walk::output>(a, bf16, st);
}

hipError_t launch_delta_join(const DeltaArgs& a, bool backward, hipStream_t st) {
  const int blocks = (a.m.dv + 15) / 16;
  const dim3 grid(blocks * a.m.H * (backward ? 2 : 1), a.m.n_seq);
  if (a.m.dk <= 32) launch_kernel(delta_join_kernel<32>, grid, kThreads, 0, st, a, blocks);
  else if (a.m.dk <= 64) launch_kernel(delta_join_kernel<64>, grid, kThreads, 0, st, a, blocks);
  else launch_kernel(delta_join_kernel<128>, grid, kThreads, 0, st, a, blocks);
  return hipGetLastError();
}

hipError_t launch_delta_decode(const DeltaArgs& x, bool bf16, float* state, hipStream_t st) {
  const DeltaMap& m = x.m;
  TokenArgs a;
  a.T = m.T; a.H = m.H; a.share = m.H / m.Hk; a.dk = m.dk; a.dv = m.dv; a.scale = x.scale;
  for (int i = 0; i < 3; ++i) {
    a.sq[i] = x.sq[i]; a.sk[i] = x.sk[i]; a.sv[i] = x.sv[i]; a.so[i] = x.so[i]; a.sb[i] = x.sb[i]; a.sl[i] = x.sl[i];
  }
  constexpr int LC = 16, kMost = 65535;             // sequences that a grid axis holds
  auto run = [&](auto t, auto ri) {
    using T_ = decltype(t);
    hipError_t e = hipSuccess;
    for (long long b = 0; b < m.n_seq && e == hipSuccess; b += kMost) {
      const dim3 grid((m.dv + 4 * LC - 1) / (4 * LC), m.H, (unsigned)(m.n_seq - b < kMost ? m.n_seq - b : kMost));
      launch_kernel(delta_decode_kernel<T_, LC, decltype(ri)::value>, grid, kThreads, 0, st, a,
                    (const T_*)x.q + b * a.sq[0], (const T_*)x.k + b * a.sk[0], (const T_*)x.v + b * a.sv[0],
                    (const T_*)x.beta + b * a.sb[0], x.log_decay ? x.log_decay + b * a.sl[0] : nullptr,
                    state + b * m.H * m.dk * m.dv, (T_*)x.o + b * a.so[0]);
      e = hipGetLastError();
    }
    return e;
  };
  auto rows = [&](auto t) {
    if (m.dk <= 32) return run(t, std::integral_constant<int, 2>());
    if (m.dk <= 64) return run(t, std::integral_constant<int, 4>());
    return run(t, std::integral_constant<int, 8>());
  };
  return bf16 ? rows(__bf16()) : rows(float());
}

}  // namespace kata
