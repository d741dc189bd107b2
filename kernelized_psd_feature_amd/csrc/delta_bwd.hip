// Gradients of the gated delta rule (delta.hip), gfx950.
//
// With the notation there, S the state before a chunk and D the gradient of the one behind it:
//   Z = P^T dO scale + diag(exp(c_63 - c)) K D          (the gradient of U)
//   X = (I + A)^-T Z,  dv = diag(b) X
//   the gradient of S:  y_63 D + scale (diag(y) Q)^T dO - (diag(y) K)^T dv
//   dbeta_i = X_i . (v_i - y_i S^T k_i - sum_{j < i} exp(c_i - c_j) (k_i . k_j) u_j), which needs no division by b
//   dlog_t = sum_{i >= t in the chunk} (dO_i . o_i - dv_i . v_i) + <D, S'>,  S' the state behind the chunk; or
//   dlog_t = sum_{i >= t > j} F_ij + sum_{i >= t} R_i + sum_{j < t} W_j + y_63 <D, S>,  where
//     F_ij = PO_ij (q_i . k_j) + PV_ij (k_i . k_j),  R_i = y_i (scale dO_i . S^T q_i - dv_i . S^T k_i),
//     W_j = exp(c_63 - c_j) (u_j . D^T k_j)
//   PO_ij = scale exp(c_i - c_j) (dO_i . u_j) for j <= i,  PV_ij = -exp(c_i - c_j) (dv_i . u_j) for j < i
//   dq = scale diag(y) dO S^T + PO K
//   dk = diag(exp(c_63 - c)) U D^T - diag(y) dv S^T + PO^T Q + PV^T K + PV K
// (dlog: what <D, S> changes by at a token is known from its products with the gradients, dv . v - dO . o; and
// dO . o is q . dq, a head's part of it.  The second form is what reaches over the token's decay, from the tokens and the state
// before it to those behind, every term with that decay for a factor.  Of a strong decay the first one's terms, which have it
// not, leave only their roundings: mean log decays of -1, -5, -10, -20 are off by 2e-6, 3e-5, 4e-4, 0.3 of the norm in bf16 (fp32 2e-6,
// 6e-5, 1e-3, 0.4), by the second form by 4e-7 to 7e-7 (fp32 2e-7 to 4e-7).  In bf16 weak ones are as good by the first (-0.02: 9e-7,
// by the second 3e-6, of operands in two terms), and for less work: a training step of 8 x 4096 tokens 948 us, 1016 where
// all chunks take the second.  So in bf16 the second is for chunks in which any token's decay is below exp(-1/2); in fp32, where it is the better one of
// all (-0.02: 3e-7 to 5e-7 for 6e-7 to 1e-6) and both together lack the registers (2 x 1001: 147 us, 152), for every chunk.)
//
// S and U, and D and X, come from two walks like the forward pass's, one of them in reversed time, which keep
// them for every chunk; all the rest is then computed for all chunks at once (delta_grads_kernel).
//
// 8 x 4096 tokens of 16 bf16 heads of 64: inverses 48 us, both walks 304, gradients 390; the bytes that the three
// exchange, 1.9 GB, are 380 us of HBM's time.  The walks are a chain as forward, 64 chunks of 4.6 us where 256
// workgroups have a CU each (VALU 33 % of the cycles, LDS 34, MFMA 20).  Four waves more, forming P^T dO and
// Q^T diag(y) dO a chunk ahead, did not shorten it (330 for 305): the waves share their SIMDs.
#include <type_traits>

#include "delta.h"
#include "delta_plan.h"
#include "delta_tiles.h"
#include "delta_walk.h"
#include "device.h"
#include "mfma_util.h"

namespace kata {
namespace {

constexpr int kThreads = 512;             // of the gradients' kernel

// ---- the walk in reversed time ------------------------------------------------------------------
template <typename T, int DK, int W>
struct ReverseTiles {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int DV = 16 * W;
  static constexpr int LK = DK + 16 / (int)sizeof(T), LV = DV + (kBf ? 16 : 4), LP = kC + 16 / (int)sizeof(T);
  static constexpr int kHead = 16 + kDeltaVec * 4;
  static constexpr int NT = kBf ? 3 : 1, NI = kBf ? 2 : 1, NP = NT;     // terms of the recurrence's operands, of the inverse, of P
  static constexpr int kTiles = kC * (2 * LK + LV);
  static constexpr int bytes = kHead + (kTiles + (NI + NP) * kC * LP) * (int)sizeof(T);
};

// kSums: of the segments, from a gradient of zero behind them.
template <typename T, int DK, int W, bool kSums>
__device__ __forceinline__ void delta_reverse(const DeltaArgs& A, unsigned unit, int sub, char* lds) {
  using TL = ReverseTiles<T, DK, W>;
  using frag = typename Elem<T>::frag;
  constexpr int kThr = 64 * W, DV = TL::DV, M = DK / 32, NS = DK / 16, LK = TL::LK, LV = TL::LV, LP = TL::LP;
  constexpr int NT = TL::NT, NI = TL::NI, NP = TL::NP;
  int* const sh = reinterpret_cast<int*>(lds);
  float* const vec = reinterpret_cast<float*>(lds + 16);
  T* const sK = reinterpret_cast<T*>(lds + TL::kHead);
  T* const sQ = sK + kC * LK;
  T* const sO = sQ + kC * LK;
  T* const sT = sK + TL::kTiles;
  T* const sP = sT + NI * kC * LP;

  const DeltaMap& m = A.m;
  // (locals: what lambdas read out of the arguments ended in scratch, whose loads wait for all others)
  const float scale = A.scale;
  const float* const at_vec = A.vec;
  const float* const at_inv = A.inv;
  float* const at_x = A.x;
  float* const at_states = A.rstates;
  const int tid = threadIdx.x;
  int lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  auto forget = [&]() __attribute__((always_inline)) {                 // (see the walk)
    if constexpr (M > 2 && TL::kBf) {
      asm volatile("" : "+v"(lane));
      g = lane >> 4;
      l16 = lane & 15;
    }
  };
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (unit >= (unsigned)m.n_slots * (unsigned)m.H) return;
  const int slot = int(unit / (unsigned)m.H), h = int(unit - (unsigned)slot * (unsigned)m.H);
  const int c0 = sub * DV;
  DeltaPart s;
  if (!find_part(m, slot, m.L, m.n_seg, m.n_slots, sh, kThr, s) || s.seq == m.n_seq) return;
  const int L = m.L, n_chunks = (s.len + kC - 1) / kC, n_seg = (n_chunks + L - 1) / L;
  const long long SE = (long long)m.dk * m.dv, st_off = ((long long)s.seq * m.H + h) * SE;
  if (s.part >= n_seg) {
    if (!kSums && s.len == 0 && s.part == 0 && A.dinit)   // an empty sequence
      for (int i = tid; i < m.dk * DV; i += kThr) {
        const int r = i / DV, c = c0 + i % DV;
        if (c < m.dv) A.dinit[st_off + (long long)r * m.dv + c] = A.dfin ? A.dfin[st_off + (long long)r * m.dv + c] : 0.f;
      }
    return;
  }
  if (kSums && s.part == 0) return;                 // enters no other segment
  const bool last_seg = s.part == n_seg - 1;
  const int first = s.part * L, behind = min(first + L, n_chunks);
  const int n_last = min(kC, s.len - kC * (behind - 1));
  const int hk = h / (m.H / m.Hk);
  const long long row0 = s.start + (long long)kC * (behind - 1);
  // (Stage steps to the next chunk by 64 rows; here the next one is the one before)
  const T* pk = reinterpret_cast<const T*>(A.k) + s.b * A.sk[0] + row0 * A.sk[1] + hk * A.sk[2];
  const T* pq = reinterpret_cast<const T*>(A.q) + s.b * A.sq[0] + row0 * A.sq[1] + hk * A.sq[2];
  const T* po = reinterpret_cast<const T*>(A.dO) + s.b * A.sdo[0] + row0 * A.sdo[1] + h * A.sdo[2] + c0;
  Stage<T, DK, kThr> rk(pk, A.sk[1], m.dk, true), rq(pq, A.sq[1], m.dk, true);
  Stage<T, DV, kThr> ro(po, A.sdo[1], m.dv - c0, false);
  StageInv<T, NI, LP, kThr> ri;
  uint4 vec_next;
  const long long chunk0 = (long long)s.c_slot * m.H + h;              // [c_slots][H]
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int n = c == behind - 1 ? n_last : kC;
    fetch_rows(rk, A.sk[1], n);
    fetch_rows(rq, A.sq[1], n);
    fetch_rows(ro, A.sdo[1], n);
    rk.p -= 2 * kC * A.sk[1];
    rq.p -= 2 * kC * A.sq[1];
    ro.p -= 2 * kC * A.sdo[1];
    ri.fetch(at_inv + (chunk0 + (long long)c * m.H) * kInvFloats);
    vec_next = fetch_vec(at_vec + (chunk0 + (long long)c * m.H) * kDeltaVec);
  };
  fetch(behind - 1);

  const int wc = 16 * w, col = c0 + wc + l16;
  const float* given = kSums ? nullptr : !last_seg ? A.rsums + ((long long)slot * m.H + h) * SE : A.dfin ? A.dfin + st_off : nullptr;
  f32x4 D[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) D[i] = zero4();
  if (given) load_state(D, given, m.dk, m.dv, col, g);                 // uniform
  if (m.dk < DK || m.dv - c0 < DV) {
    uint4* const z = reinterpret_cast<uint4*>(sK);
    for (int i = tid; i < TL::kTiles * (int)sizeof(T) / 16; i += kThr) z[i] = uint4{0u, 0u, 0u, 0u};
  }
  ri.zeros(sT);
  const int ct = (m.dv + 15) / 16;
  const bool live_tile = c0 / 16 + w < ct;          // uniform
#pragma unroll 1
  for (int c = behind - 1; c >= first; --c) {
    __syncthreads();                                // the last chunk's tiles have been read
    const int n = c == behind - 1 ? n_last : kC;
    keep_rows(rk, n);
    keep_rows(rq, n);
    keep_rows(ro, n);
    rk.template put_split<LK>(sK);
    rq.template put_split<LK>(sQ);
    ro.template put<LV>(sO);
    ri.put(sT);
    put_vec(vec, vec_next);
    if (!kSums && live_tile) {
      float* dst = at_states + ((chunk0 + (long long)c * m.H) * ct + c0 / 16 + w) * (DK * 16) + lane * 4;
#pragma unroll
      for (int i = 0; i < NS; ++i) *reinterpret_cast<f32x4*>(dst + i * 256) = D[i];
    }
    if (c > first) fetch(c - 1);
    __syncthreads();
    // reads in batches, as in the walk
    forget();
    f32x4 Z[4], X[4];
    frag of[2];
    {
      constexpr int J = 16 / W;
      const int rt = w & 3, j0 = J * (w >> 2);
      frag kr[4][M], qr[M];
#pragma unroll
      for (int i = 0; i < M; ++i) qr[i] = row_frag(sQ + (16 * rt + l16) * LK + 32 * i + 8 * g);
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int i = 0; i < M; ++i) kr[it][i] = row_frag(sK + (16 * it + l16) * LK + 32 * i + 8 * g);
      reads_above<T>();
      f32x4 p[J];
#pragma unroll
      for (int j = 0; j < J; ++j) p[j] = zero4();
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) p[j] = mma(W == 8 && j0 ? kr[(j + J) & 3][i] : kr[j][i], qr[i], p[j]);
      Op<T, NT> df[M];
#pragma unroll
      for (int i = 0; i < M; ++i) split_terms(D[2 * i], D[2 * i + 1], df[i]);
#pragma unroll
      for (int it = 0; it < 4; ++it) Z[it] = zero4();
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int t = NT - 1; t >= 0; --t)
#pragma unroll
          for (int it = 0; it < 4; ++it) Z[it] = mma(kr[it][i], df[i].t[t], Z[it]);
      put_weights<T, LP, J, NP>(sP, p, vec + 3 * kC, rt, j0, lane, scale);
    }
    forget();
#pragma unroll
    for (int i = 0; i < 2; ++i) of[i] = column_frag<LV>(sO + 32 * i * LV + wc, lane);
    Op<T, NI> inv[6];                               // (row tile, K step): (0, 0), (0, 1), (1, 0), (1, 1), (2, 1), (3, 1)
#pragma unroll
    for (int f = 0; f < 6; ++f)
      inv[f] = split_column_op<NI, LP>(sT + 32 * (f < 4 ? f & 1 : 1) * LP, kC * LP, f < 4 ? f >> 1 : f - 2, lane);
#pragma unroll
    for (int it = 0; it < 4; ++it) Z[it] *= *reinterpret_cast<const f32x4*>(vec + kC + 16 * it + 4 * g);
    __syncthreads();                                // P is there
    forget();
    {
      Op<T, NP> pf[6];
#pragma unroll
      for (int f = 0; f < 6; ++f)
        pf[f] = split_column_op<NP, LP>(sP + 32 * (f < 4 ? f & 1 : 1) * LP, kC * LP, f < 4 ? f >> 1 : f - 2, lane);
      reads_above<T>();
#pragma unroll
      for (int t = NP - 1; t >= 0; --t)
#pragma unroll
        for (int it = 0; it < 4; ++it) Z[it] = mma(pf[it < 2 ? 2 * it : it + 2].t[t], of[it >> 1], Z[it]);
#pragma unroll
      for (int t = NP - 1; t >= 0; --t)
#pragma unroll
        for (int it = 0; it < 2; ++it) Z[it] = mma(pf[2 * it + 1].t[t], of[1], Z[it]);
    }
    forget();
    frag qt[2][NS];                                 // Q transposed, 32 tokens each, then K
    auto read_t = [&](const T* tile, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NS; ++i) qt[j][i] = split_column_frag<LK>(tile + 32 * j * LK, i, lane);
    };
    if constexpr (M <= 2) read_t(sQ, 0);
    if constexpr (M <= 2) read_t(sQ, 1);
    reads_above<T>();
    {
      Op<T, NT> zf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_terms(Z[2 * i], Z[2 * i + 1], zf[i]);
#pragma unroll
      for (int it = 0; it < 4; ++it) X[it] = zero4();
      each_term<NI, NT>([&](int n, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int it = 0; it < 4; ++it) X[it] = mma(inv[it < 2 ? 2 * it : it + 2].t[n], zf[it >> 1].t[k], X[it]);
      });
      each_term<NI, NT>([&](int n, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int it = 0; it < 2; ++it) X[it] = mma(inv[2 * it + 1].t[n], zf[1].t[k], X[it]);
      });
    }
    Op<T, NT> kw[2], qw[2];
    if (!kSums && live_tile) {
      float* const px = at_x + ((chunk0 + (long long)c * m.H) * ct + c0 / 16 + w) * 1024 + lane * 4;
#pragma unroll
      for (int it = 0; it < 4; ++it) *reinterpret_cast<f32x4*>(px + it * 256) = X[it];
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f32x4 yv = *reinterpret_cast<const f32x4*>(vec + 16 * it + 4 * g);
      X[it] *= -yv * *reinterpret_cast<const f32x4*>(vec + 2 * kC + 16 * it + 4 * g);
      Z[it] = half_of(of[it >> 1], it & 1) * yv * scale;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      split_terms(X[2 * i], X[2 * i + 1], kw[i]);
      split_terms(Z[2 * i], Z[2 * i + 1], qw[i]);
    }
    const float whole = vec[kC - 1];
#pragma unroll
    for (int i = 0; i < NS; ++i) D[i] *= whole;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (M > 2) read_t(sQ, j);
      reads_above<T>();
#pragma unroll
      for (int t = NT - 1; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < NS; ++i) D[i] = mma(qt[j][i], qw[j].t[t], D[i]);
      read_t(sK, j);
    }
    reads_above<T>();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = NT - 1; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < NS; ++i) D[i] = mma(qt[j][i], kw[j].t[t], D[i]);
  }
  float* dst = kSums ? A.rsums + ((long long)slot * m.H + h) * SE : first == 0 && A.dinit ? A.dinit + st_off : nullptr;
  if (!dst || col >= m.dv) return;
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (16 * i + 4 * g + r < m.dk) dst[(long long)(16 * i + 4 * g + r) * m.dv + col] = D[i][r];
}

// Both walks side by side.  kSums: sums and transitions of the segments.
template <typename T, int DK, int W>
constexpr int kBothBytes = WalkTiles<T, DK, W, 3, false>::bytes > ReverseTiles<T, DK, W>::bytes ? WalkTiles<T, DK, W, 3, false>::bytes
                                                                                              : ReverseTiles<T, DK, W>::bytes;
template <typename T, int DK, int W, bool kSums>
__global__ __launch_bounds__(64 * W, (sizeof(T) == 4 && DK == 128 ? 1 : 2)) void delta_both_kernel(DeltaArgs A, int blocks, int forward) {
  extern __shared__ __align__(16) char lds[];
  const UnitBlock u = unit_block(blocks);
  if (u.sub < forward) delta_walk<T, DK, W, sizeof(T) == 2 ? 3 : 1, kSums ? Walk::sums : Walk::states>(A, u.unit, u.sub, 1, lds);
  else delta_reverse<T, DK, W, kSums>(A, u.unit, u.sub - forward, lds);
}

// ---- the gradients ------------------------------------------------------------------------------
// One workgroup of eight waves for a chunk and a head of q and k, over the value heads that share it (few chunks: for
// each value head) and blocks of 64 value columns, then for another chunk.  U, X and the states, which the walks
// have left in tiles of 16 columns, go through LDS, [column][token] and [column][row of the state]; a wave has 16
// tokens, four of the waves P's gradient and half of the columns of dq and dk, the others that of the system's
// matrix and the other half.
// 390 us for 8 x 4096 tokens of 16 heads of 64, 136 KB a chunk and head, 2.9 TB/s: a CU holds one workgroup (122 KB of
// LDS), its loads run a chunk ahead, and five barriers part phases of some hundred cycles of LDS and VALU each (VALU
// 38 % of the cycles, LDS 30, MFMA 10; without any load 290 us).
template <typename T, int DK>
struct GradTiles {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int PAD = 16 / (int)sizeof(T);
  static constexpr int LK = DK + PAD, LP = kC + PAD, LS = DK + PAD;
  static constexpr int kHead = 16 + kDeltaVec * 4 + (6 + 8) * kC * 4 + 16;                     // an int, vec, sums of the waves
  // Terms of U, X, S and PO, and how many of them enter dk, as of D and PV.  The dots dO . o and dv . v cancel in
  // dlog: with two terms it was off by 2e-6 to 1e-5 of its norm, with three by 5e-7 to 1.6e-6.
  static constexpr int N = kBf ? 3 : 1, N2 = kBf ? 2 : 1;
  static constexpr int kPlane = 64 * LP, kState = 64 * LS;
  // The next chunk's operands are loaded ahead, and D has a place of its own, where registers and LDS are there.
  static constexpr bool kAhead = DK <= 64;
  // dlog always by what is carried over the decays, with <D, S>; else with <D, S'> but for chunks of strong decays.
  static constexpr bool kCarried = !kBf;
  // K and Q; U and X, then PO and PV; S (and D)
  static constexpr int bytes = kHead + (2 * kC * LK + 2 * N * kPlane + (N + (kAhead ? N2 : 0)) * kState) * (int)sizeof(T);
};
template <int K, typename T, int N>
__device__ __forceinline__ Op<T, K> leading(const Op<T, N>& x) {
  Op<T, K> y;
#pragma unroll
  for (int i = 0; i < K; ++i) y.t[i] = x.t[i];
  return y;
}

// A row's operand over 32 value columns from `col` on, of `width` columns at p (the last ones again behind them), and
// the same order of columns of 32 rows of LD elements: bf16 straight (one load of 16 bytes), fp32 split (two).
__device__ __forceinline__ bf16x8 value_row(const __bf16* p, int col, int width, int g) {
  return row_frag(p + min(col + 8 * g, width - 8));
}
__device__ __forceinline__ f32x8 value_row(const float* p, int col, int width, int g) {
  return pack_frag(load4(p + min(col + 4 * g, width - 4)), load4(p + min(col + 16 + 4 * g, width - 4)), float());
}
__device__ __forceinline__ void keep_columns(bf16x8& x, bool row, int width, int g) {
  if (!row || 8 * g >= width) x = bf16x8{};
}
__device__ __forceinline__ void keep_columns(f32x8& x, bool row, int width, int g) {
  x = pack_frag(row && 4 * g < width ? half_of(x, 0) : zero4(), row && 16 + 4 * g < width ? half_of(x, 1) : zero4(), float());
}
__device__ __forceinline__ void store_row(__bf16* p, int width, int g, const bf16x8& x) {
  if (8 * g < width) *reinterpret_cast<uint4*>(p + 8 * g) = __builtin_bit_cast(uint4, x);
}
__device__ __forceinline__ void store_row(float* p, int width, int g, const f32x8& x) {
  if (4 * g < width) store4(p + 4 * g, half_of(x, 0));
  if (16 + 4 * g < width) store4(p + 16 + 4 * g, half_of(x, 1));
}
template <int LD>
__device__ __forceinline__ bf16x8 value_column(const __bf16* p, int lane) {
  const __bf16* at = p + (8 * (lane >> 4) + ((lane & 15) >> 2)) * LD + 4 * (lane & 3);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * LD));
  const uint2 ul = __builtin_bit_cast(uint2, lo), uh = __builtin_bit_cast(uint2, hi);
  return __builtin_bit_cast(bf16x8, uint4{ul.x, ul.y, uh.x, uh.y});
}
template <int LD>
__device__ __forceinline__ f32x8 value_column(const float* p, int lane) {
  return column_frag<LD>(p, lane);
}
template <int N, int LD, typename T>
__device__ __forceinline__ Op<T, N> value_op(const T* p, int plane, int lane) {
  Op<T, N> x;
#pragma unroll
  for (int i = 0; i < N; ++i) x.t[i] = value_column<LD>(p + i * plane, lane);
  return x;
}
// x of the lane whose number differs in bit 4 (5)
__device__ __forceinline__ float other_16(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(threadIdx.x & 16 ? p[0] : p[1]);
}
__device__ __forceinline__ float other_32(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(threadIdx.x & 32 ? p[0] : p[1]);
}
// the sum over the 16 lanes of a row of them
__device__ __forceinline__ float sum_16(float x) {
  const auto turned = [](float y, auto by) __attribute__((always_inline)) {              // row_ror
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, y), 0x120 + decltype(by)::value, 0xf, 0xf, true));
  };
  x += turned(x, std::integral_constant<int, 8>());
  x += turned(x, std::integral_constant<int, 4>());
  x += turned(x, std::integral_constant<int, 2>());
  return x + turned(x, std::integral_constant<int, 1>());
}
// the sum of the products of two operands' elements
template <typename F>
__device__ __forceinline__ float dot(const F& a, const F& b) {
  const f32x4 x = half_of(a, 0) * half_of(b, 0) + half_of(a, 1) * half_of(b, 1);
  return x[0] + x[1] + x[2] + x[3];
}

template <typename T, int DK>
__global__ __launch_bounds__(kThreads, 2) void delta_grads_kernel(DeltaArgs A) {
  using TL = GradTiles<T, DK>;
  using frag = typename Elem<T>::frag;
  constexpr int NS = DK / 16, NH = NS / 2, LK = TL::LK, LP = TL::LP, LS = TL::LS, N = TL::N, N2 = TL::N2;
  constexpr int PL = TL::kPlane, PS = TL::kState;
  constexpr bool kAhead = TL::kAhead, kCarried = TL::kCarried;
  constexpr int G = NH < 2 || (sizeof(T) == 4 && DK > 64) ? 1 : 2;     // tiles of dq and dk in turn (each_term), by the registers
  extern __shared__ __align__(16) char lds[];
  int* const sh = reinterpret_cast<int*>(lds);
  float* const vec = reinterpret_cast<float*>(lds + 16);
  const float* const sc = vec + 3 * kC;
  const float* const sb = vec + 2 * kC;
  float* const sE = vec + kDeltaVec;                // [2][64] each, in two parts: q . dq - dv . v (or R), dbeta, W
  float* const sG = sE + 6 * kC;                    // [2][4][64] by the halves' waves: the sums of F
  float* const sF = sG + 8 * kC;                    // [4] <D, S'> (or <D, S>)
  T* const sK = reinterpret_cast<T*>(lds + TL::kHead);
  T* const sQ = sK + kC * LK;
  T* const sU = sQ + kC * LK;                       // N planes each of U and X, then of PO and (N2) PV
  T* const sZ = sU + N * PL;
  T* const sS = sZ + N * PL;                        // N planes of S, N2 of D
  T* const sD = kAhead ? sS + N * PS : sS;

  const DeltaMap& m = A.m;
  const int tid = threadIdx.x;
  int lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  // The places in LDS that a phase uses are computed there: kept from phase to phase they would cost a hundred
  // registers, and scratch.
  auto forget = [&]() __attribute__((always_inline)) {
    asm volatile("" : "+v"(lane));
    g = lane >> 4;
    l16 = lane & 15;
  };
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
  const bool first_half = wave < 4;
  // A.pq: a workgroup has one value head, and leaves its dq and dk there, in fp32 rows of H heads
  const int shared = m.H / m.Hk, share = A.pq ? 1 : shared, heads = A.pq ? m.H : m.Hk;
  const int ct = (m.dv + 15) / 16, v_blocks = (m.dv + 63) / 64;
  const unsigned units = (unsigned)m.c_slots * (unsigned)heads;

  // where the workgroup is: a chunk and its value head h0 + hh, its `vb`th block of columns
  struct Place {
    unsigned unit;
    int slot, h0, hh, vb, n;
    DeltaPart s;
    long long row0;
  };
  auto put_grads = [&](long long at, const f32x4& q, const f32x4& k) __attribute__((always_inline)) {
    if (A.pq) {
      store4(A.pq + at, q);
      store4(A.pk + at, k);
    } else {
      store4(reinterpret_cast<T*>(A.dq) + at, q);
      store4(reinterpret_cast<T*>(A.dk) + at, k);
    }
  };
  auto clear = [&](const Place& p, int from, int rows) __attribute__((always_inline)) {
    const long long at_k = (long long)p.s.b * m.T * heads + p.h0 / share, lead = (long long)p.s.b * m.T * m.H + p.h0;
    for (long long i = tid; i < (long long)rows * (m.dk / 4); i += kThreads)
      put_grads((at_k + (from + i / (m.dk / 4)) * heads) * m.dk + i % (m.dk / 4) * 4, zero4(), zero4());
    const int per = share * m.dv / 4;
    for (long long i = tid; i < (long long)rows * per; i += kThreads)
      store4(reinterpret_cast<T*>(A.dv) + (lead + (from + i / per) * m.H) * m.dv + i % per * 4, zero4());
    for (long long i = tid; i < (long long)rows * share; i += kThreads) {
      const long long at = lead + (from + i / share) * m.H + i % share;
      reinterpret_cast<T*>(A.dbeta)[at] = T(0.f);
      if (A.dlog) A.dlog[at] = 0.f;
    }
  };
  // a lane's part (of four) of its token's dot with a row of K or Q: 16 columns, x the four of them at 4 g
  auto row_dot = [&](const T* tile, int columns, const f32x4& x) __attribute__((always_inline)) {
    const f32x4 y = unquad(*reinterpret_cast<const Quad<T>*>(tile + (16 * w + l16) * LK + split_place(16 * columns + 4 * g))) * x;
    return y[0] + y[1] + y[2] + y[3];
  };
  // The first unit from p.unit on that has tokens; those before it are zeros' rows, or nothing.
  auto find = [&](Place& p) __attribute__((always_inline)) {
    for (; p.unit < units; p.unit += gridDim.x) {
      p.slot = int(p.unit / (unsigned)heads);
      p.h0 = int(p.unit - (unsigned)p.slot * (unsigned)heads) * share;
      p.hh = p.vb = 0;
      if (m.packed) __syncthreads();                // the last answer has been read
      if (!find_part(m, p.slot, 1, m.n_chunks, m.c_slots, sh, kThreads, p.s)) continue;
      p.n = min(kC, p.s.len - kC * p.s.part);
      p.row0 = p.s.start + (long long)kC * p.s.part;
      if (p.s.seq == m.n_seq) {                     // rows behind the last sequence
        if (p.n > 0) clear(p, (int)p.row0, p.n);
        continue;
      }
      if (m.packed && p.s.seq == 0 && p.s.part == 0) clear(p, 0, p.s.start);   // before the first
      if (p.n > 0) return true;
    }
    return false;
  };

  // What is loaded for a place: a wave's 16 columns of U and S, or of X, D and S' (the state behind the chunk; kCarried: S); its 16
  // tokens' dO and (half of the columns) v; all together the chunk's rows and vectors.
  Stage<T, DK, kThreads> rk(nullptr, 0, m.dk, true), rq(nullptr, 0, m.dk, true);
  f32x4 x[4], S[NS], Sn[kAhead ? NS : 1];
  frag od[2], vd;
  uint4 vec_next;
  float frob_next = 0.f;
  auto load = [&](const Place& p) __attribute__((always_inline)) {
    const int h = p.h0 + p.hh, hk = h / shared, c0 = 64 * p.vb, row = 16 * w + l16;
    const bool last = kC * (p.s.part + 1) >= p.s.len, live_tile = 4 * p.vb + w < ct;   // uniform
    const int block_tile = live_tile ? 4 * p.vb + w : ct - 1;
    const long long cs = (long long)p.slot * m.H + h, tile = cs * ct + block_tile;
    if (p.hh == 0 && p.vb == 0) {
      rk = Stage<T, DK, kThreads>(reinterpret_cast<const T*>(A.k) + p.s.b * A.sk[0] + p.row0 * A.sk[1] + hk * A.sk[2], A.sk[1],
                                  m.dk, true);
      rq = Stage<T, DK, kThreads>(reinterpret_cast<const T*>(A.q) + p.s.b * A.sq[0] + p.row0 * A.sq[1] + hk * A.sq[2], A.sq[1],
                                  m.dk, true);
      fetch_rows(rk, A.sk[1], p.n);
      fetch_rows(rq, A.sq[1], p.n);
    }
    vec_next = fetch_vec(A.vec + cs * kDeltaVec);
    {
      const float* const fx = (first_half ? A.u : A.x) + tile * 1024 + lane * 4;
      const float* const fs = (first_half ? A.cstates : A.rstates) + tile * (DK * 16) + lane * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = load4(fx + i * 256);
#pragma unroll
      for (int i = 0; i < NS; ++i) S[i] = load4(fs + i * 256);
    }
    {
      const long long at = p.row0 + min(row, p.n - 1);
      const T* const po = reinterpret_cast<const T*>(A.dO) + p.s.b * A.sdo[0] + at * A.sdo[1] + h * A.sdo[2];
      const T* const pv = reinterpret_cast<const T*>(A.v) + p.s.b * A.sv[0] + at * A.sv[1] + h * A.sv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) od[i] = value_row(po, c0 + 32 * i, m.dv, g);
      vd = value_row(pv, c0 + (first_half ? 0 : 32), m.dv, g);
    }
    // (behind the last chunk without a gradient D is zero)
    const bool given = kCarried || !last || A.fstates;
    const float* const next = first_half || kCarried ? A.cstates + tile * (DK * 16) + lane * 4     // (first half: not used)
                              : !last ? A.cstates + (tile + (long long)m.H * ct) * (DK * 16) + lane * 4
                              : given ? A.fstates + (((long long)p.s.seq * m.H + h) * ct + block_tile) * (DK * 16) + lane * 4
                                      : A.rstates + tile * (DK * 16) + lane * 4;
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < NS; ++i) Sn[i] = load4(next + i * 256);
    } else {
      frob_next = 0.f;
      if (given && !first_half && live_tile)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const f32x4 y = S[i] * load4(next + i * 256);
          frob_next += y[0] + y[1] + y[2] + y[3];
        }
    }
  };

  Place now;
  now.unit = blockIdx.x;
  bool more = find(now);
  if (!more) return;
  if (m.dk < DK)                                    // columns that no operand has: zeros all along
    for (int i = tid; i < 2 * kC * LK * (int)sizeof(T) / 16; i += kThreads)
      reinterpret_cast<uint4*>(sK)[i] = uint4{0u, 0u, 0u, 0u};
  if constexpr (kAhead) load(now);

  f32x4 dqa[NH], dka[NH];                           // [row 16 (i0 + i) + 4 g + r][token 16 w + l16]
  f32x4 Wt[4], dqh[NH];                             // the strip of dO U^T (second half: X U^T), transposed; the head's dq
  float frob = 0.f, xv = 0.f, xe = 0.f;             // X . v, and dbeta without it, in parts
  float frob_in = 0.f, write = 0.f;                 // strong decays: <D, S> and W in parts
  const int i0 = first_half ? 0 : NH;
#pragma unroll 1
  while (more) {
    if constexpr (!kAhead) load(now);
    const int h = now.h0 + now.hh, c0 = 64 * now.vb, row = 16 * w + l16;
    const long long lead = ((long long)now.s.b * m.T + now.row0) * m.H + h;    // of [b][t][H]
    const bool live_row = row < now.n;
    if (now.vb == 0) {
      frob = xv = xe = frob_in = write = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) Wt[i] = zero4();
#pragma unroll
      for (int i = 0; i < NH; ++i) dqh[i] = zero4();
      if (now.hh == 0)
#pragma unroll
        for (int i = 0; i < NH; ++i) dqa[i] = dka[i] = zero4();
    }
    forget();
    __syncthreads();                                // the last block's tiles have been read
    if (now.vb == 0) put_vec(vec, vec_next);
    if (4 * now.vb + w >= ct) {                     // no such columns (uniform)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = zero4();
#pragma unroll
      for (int i = 0; i < NS; ++i) S[i] = zero4();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) keep_columns(od[i], live_row, m.dv - c0 - 32 * i, g);
    keep_columns(vd, live_row, m.dv - c0 - (first_half ? 0 : 32), g);
    if (now.hh == 0 && now.vb == 0) {
      keep_rows(rk, now.n);
      keep_rows(rq, now.n);
      rk.template put_split<LK>(sK);
      rq.template put_split<LK>(sQ);
    }
    {
      T* const at = (first_half ? sU : sZ) + row * LP + 4 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) put_terms<N>(at + 16 * i, PL, x[i]);
    }
    auto put_d = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NS; ++i) put_terms<N2>(sD + (16 * w + l16) * LS + 16 * i + 4 * g, PS, S[i]);
    };
    if (first_half) {
#pragma unroll
      for (int i = 0; i < NS; ++i) put_terms<N>(sS + (16 * w + l16) * LS + 16 * i + 4 * g, PS, S[i]);
    } else if constexpr (kAhead) {
      put_d();
      if (kCarried || kC * (now.s.part + 1) < now.s.len || A.fstates)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const f32x4 y = S[i] * Sn[i];
          frob += y[0] + y[1] + y[2] + y[3];
        }
    }
    frob += frob_next;
    const frag oc[2] = {od[0], od[1]}, vc = vd;
    Place next = now;
    if (++next.vb == v_blocks) {
      next.vb = 0;
      if (++next.hh == share) {
        next.unit += gridDim.x;
        more = find(next);
      }
    }
    if constexpr (kAhead)
      if (more) load(next);
    __syncthreads();

    // a wave's 16 tokens
    forget();
    float log2_decay = 0.f;
    if constexpr (!kCarried) log2_decay = sc[lane] - (lane ? sc[lane - 1] : 0.f);
    Op<T, N> z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) z[i] = value_op<N, LP>(sZ + 32 * i * LP + 16 * w, PL, lane);
    if (live_row) {                                 // dv, half of the columns each
      T* const dst = reinterpret_cast<T*>(A.dv) + (lead + (long long)row * m.H) * m.dv + c0;
      auto store = [&](const Op<T, N>& x, int to) __attribute__((always_inline)) {
        f32x4 lo = zero4(), hi = zero4();
#pragma unroll
        for (int t = N - 1; t >= 0; --t) {
          lo += half_of(x.t[t], 0);
          hi += half_of(x.t[t], 1);
        }
        store_row(dst + to, m.dv - c0 - to, g, pack_frag(sb[row] * lo, sb[row] * hi, T()));
      };
      if (first_half) store(z[0], 0);
      else store(z[1], 32);
    }
#pragma unroll
    for (int t = 0; t < N; ++t) xv += first_half ? dot(z[0].t[t], vc) : dot(z[1].t[t], vc);
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += 2)
      if (j0 <= w)                                  // uniform (a tile above the diagonal is not looked at)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const T* const at = sU + 32 * i * LP + 16 * j0;
          if (first_half) {
            const Op<T, N> ua = value_op<N, LP>(at, PL, lane), ub = value_op<N, LP>(at + 16, PL, lane);
#pragma unroll
            for (int t = N - 1; t >= 0; --t) {
              Wt[j0] = mma(ua.t[t], oc[i], Wt[j0]);
              Wt[j0 + 1] = mma(ub.t[t], oc[i], Wt[j0 + 1]);
            }
          } else {
            const Op<T, N2> ua = value_op<N2, LP>(at, PL, lane), ub = value_op<N2, LP>(at + 16, PL, lane);
            each_term<N2, N2>([&](int n, int k) __attribute__((always_inline)) {
              Wt[j0] = mma(ua.t[n], z[i].t[k], Wt[j0]);
              Wt[j0 + 1] = mma(ub.t[n], z[i].t[k], Wt[j0 + 1]);
            });
          }
        }
    forget();
    {
      const float yr = vec[16 * w + l16], yo = yr * A.scale, yb = yr * sb[16 * w + l16];
#pragma unroll
      for (int ia = 0; ia < NH; ia += G) {
        f32x4 a[G], b[G];
#pragma unroll
        for (int p = 0; p < G; ++p) a[p] = b[p] = zero4();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          Op<T, N> st[G];
#pragma unroll
          for (int p = 0; p < G; ++p) st[p] = value_op<N, LS>(sS + 32 * j * LS + 16 * (i0 + ia + p), PS, lane);
#pragma unroll
          for (int t = N - 1; t >= 0; --t)
#pragma unroll
            for (int p = 0; p < G; ++p) a[p] = mma(st[p].t[t], oc[j], a[p]);
          each_term<N2, N2>([&](int n, int k) __attribute__((always_inline)) {
#pragma unroll
            for (int p = 0; p < G; ++p) b[p] = mma(st[p].t[n], z[j].t[k], b[p]);
          });
        }
#pragma unroll
        for (int p = 0; p < G; ++p) {
          dqh[ia + p] += a[p] * yo;
          dka[ia + p] -= b[p] * yb;
          xe -= yr * row_dot(sK, i0 + ia + p, b[p]);
        }
      }
    }
    Op<T, N2> u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = value_op<N2, LP>(sU + 32 * i * LP + 16 * w, PL, lane);
    if constexpr (!kAhead) {
      __syncthreads();                              // S has been read
      if (!first_half) put_d();
      __syncthreads();
    }
    forget();
    // the rest, by how dlog is formed
    auto finish = [&](auto strong) __attribute__((always_inline)) {
      constexpr bool kStrong = decltype(strong)::value;
      if (kStrong && !kCarried && !first_half && 4 * now.vb + w < ct) {
        const long long tile = (((long long)now.slot * m.H + h) * ct + 4 * now.vb + w) * (DK * 16) + lane * 4;
#pragma unroll 1
        for (int i = 0; i < NS; ++i) {
          const f32x4 y = load4(A.cstates + tile + i * 256) * load4(A.rstates + tile + i * 256);
          frob_in += y[0] + y[1] + y[2] + y[3];
        }
      }
      const float left = vec[kC + 16 * w + l16];
#pragma unroll
      for (int ia = 0; ia < NH; ia += G) {
        f32x4 a[G];
#pragma unroll
        for (int p = 0; p < G; ++p) a[p] = zero4();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          Op<T, N2> st[G];
#pragma unroll
          for (int p = 0; p < G; ++p) st[p] = value_op<N2, LS>(sD + 32 * j * LS + 16 * (i0 + ia + p), PS, lane);
          each_term<N2, N2>([&](int n, int k) __attribute__((always_inline)) {
#pragma unroll
            for (int p = 0; p < G; ++p) a[p] = mma(st[p].t[n], u[j].t[k], a[p]);
          });
        }
#pragma unroll
        for (int p = 0; p < G; ++p) {
          a[p] *= left;
          dka[ia + p] += a[p];
          if (kStrong) write += row_dot(sK, i0 + ia + p, a[p]);
        }
      }
      if (now.vb + 1 < v_blocks) return;
      if constexpr (kAhead) __syncthreads();          // U and X have been read
      // PO or PV, the wave's strip of rows
      forget();
      const float b_row = first_half ? 1.f : sb[16 * w + l16];
      float e = 0.f;
      if (kStrong) {
        e = sb[16 * w + l16] * xe;
#pragma unroll
        for (int i = 0; i < NH; ++i) e += row_dot(sQ, i0 + i, dqh[i]);
      }
      {
        const float hi = sc[16 * w + l16], lo = sc[kC + 16 * w + l16], factor = first_half ? A.scale : -1.f;
        const int end = 16 * w + l16 + (first_half ? 1 : 0);             // the first key that it does not reach
        T* const at = (first_half ? sU : sZ) + (16 * w + l16) * LP;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4 p = zero4();
          if (j <= w) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int key = 16 * j + 4 * g + r;
              p[r] = key >= end ? 0.f : Wt[j][r] * (exp2_diff(hi, lo, sc[key], sc[kC + key]) * factor);
            }
          }
          Wt[j] = p;
          p *= b_row;
          if (first_half) put_terms<N>(at + split_place(16 * j + 4 * g), PL, p);
          else put_terms<N2>(at + split_place(16 * j + 4 * g), PL, p);
        }
      }
      if (!first_half) {
        if (kStrong && !kCarried) frob = frob_in;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) frob += __shfl_xor(frob, d);
        if (lane == 0) sF[w] = frob;
      }
      __syncthreads();
      if (!first_half || kStrong) {                    // F, of which dbeta wants the sums over the keys
        const T* const mine = (first_half ? sQ : sK) + (16 * w + l16) * LK + 8 * g;
        float before = 0.f;                           // F of the row's keys before the tile
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j > w) break;                           // uniform
          f32x4 f = zero4();
#pragma unroll
          for (int i = 0; i < DK / 32; ++i) f = mma(row_frag(sK + (16 * j + l16) * LK + 32 * i + 8 * g), row_frag(mine + 32 * i), f);
          f *= Wt[j];
          const float whole = f[0] + f[1] + f[2] + f[3];
          if (!first_half) xe += whole;
          if (kStrong) {
            // the row's sums over the keys before each key, then for each key those over the rows from it on
            const float near = other_16(whole), pair = whole + near, far = other_32(pair);
            f32x4 sum;
            sum[0] = before + (g & 1 ? near : 0.f) + (g & 2 ? far : 0.f);
            sum[1] = sum[0] + f[0];
            sum[2] = sum[1] + f[1];
            sum[3] = sum[2] + f[2];
            before += pair + far;
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] = sum_16(j == w && l16 < 4 * g + r ? 0.f : sum[r] * b_row);
            if (l16 == 0) *reinterpret_cast<f32x4*>(sG + (w + (first_half ? 0 : 4)) * kC + 16 * j + 4 * g) = sum;
          }
        }
      }
#pragma unroll
      for (int ia = 0; ia < NH; ia += G)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          frag kt[G];
#pragma unroll
          for (int p = 0; p < G; ++p) kt[p] = split_column_frag<LK>(sK + 32 * j * LK, i0 + ia + p, lane);
          if (j <= w >> 1) {                          // uniform
            const Op<T, N> po = row_op<N>(sU + (16 * w + l16) * LP + 32 * j + 8 * g, PL);
            const Op<T, N2> pv = row_op<N2>(sZ + (16 * w + l16) * LP + 32 * j + 8 * g, PL);
#pragma unroll
            for (int t = N - 1; t >= 0; --t)
#pragma unroll
              for (int p = 0; p < G; ++p) {
                dqh[ia + p] = mma(kt[p], po.t[t], dqh[ia + p]);
                if (t < N2) dka[ia + p] = mma(kt[p], pv.t[t], dka[ia + p]);
              }
          }
          if (j >= w >> 1) {
            const Op<T, N2> po = split_column_op<N2, LP>(sU + 32 * j * LP, PL, w, lane);
            const Op<T, N2> pv = split_column_op<N2, LP>(sZ + 32 * j * LP, PL, w, lane);
            frag qt[G];
#pragma unroll
            for (int p = 0; p < G; ++p) qt[p] = split_column_frag<LK>(sQ + 32 * j * LK, i0 + ia + p, lane);
#pragma unroll
            for (int t = N2 - 1; t >= 0; --t) {
#pragma unroll
              for (int p = 0; p < G; ++p) dka[ia + p] = mma(qt[p], po.t[t], dka[ia + p]);
#pragma unroll
              for (int p = 0; p < G; ++p) dka[ia + p] = mma(kt[p], pv.t[t], dka[ia + p]);
            }
          }
        }
      for (int i = 0; i < NH; ++i) {
        dqa[i] += dqh[i];
      }
      if (!kStrong) {                                  // dO . o = q . dq of this head
        e = -sb[row] * xv;
#pragma unroll
        for (int i = 0; i < NH; ++i) e += row_dot(sQ, i0 + i, dqh[i]);
      }
      e = sum_xor32(sum_xor16(e));
      xe = sum_xor32(sum_xor16(xe + xv));
      if (kStrong) write = sum_xor32(sum_xor16(write));
      if (lane < 16) {
        float* const at = sE + (first_half ? 0 : kC) + 16 * w + lane;
        at[0] = e;
        at[2 * kC] = xe;
        if (kStrong) at[4 * kC] = write;
      }
      __syncthreads();
      if (wave == 0) {
        const long long at = lead + (long long)lane * m.H;
        if (lane < now.n) reinterpret_cast<T*>(A.dbeta)[at] = from_f32<T>(sE[2 * kC + lane] + sE[3 * kC + lane]);
        if (kStrong) {
          float y = sE[lane] + sE[kC + lane], z = sE[4 * kC + lane] + sE[5 * kC + lane];
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) {
            const float down = __shfl_down(y, d), up = __shfl_up(z, d);
            if (lane + d < 64) y += down;
            if (lane >= d) z += up;
          }
          z = __shfl_up(z, 1);                        // of the tokens before
          y += (lane ? z : 0.f) + vec[kC - 1] * (sF[0] + sF[1] + sF[2] + sF[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i >= lane >> 4) y += sG[i * kC + lane] + sG[(4 + i) * kC + lane];
          if (A.dlog && lane < now.n) A.dlog[at] = y;
        } else if (A.dlog) {
          double y = (double)sE[lane] + sE[kC + lane];
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) {
            const double up = __shfl_down(y, d);
            if (lane + d < 64) y += up;
          }
          y += (double)sF[0] + sF[1] + sF[2] + sF[3];
          const bool none = now.s.part == 0 && lane == 0 && !A.init;     // a decay of nothing has no gradient
          if (lane < now.n) A.dlog[at] = none ? 0.f : (float)y;
        }
      }
      if (now.hh + 1 == share && live_row) {
        const long long at = (((long long)now.s.b * m.T + now.row0 + row) * heads + now.h0 / share) * m.dk + 4 * g;
#pragma unroll
        for (int i = 0; i < NH; ++i)
          if (16 * (i0 + i) + 4 * g < m.dk) put_grads(at + 16 * (i0 + i), dqa[i], dka[i]);
      }
    };
    if constexpr (!kCarried) {
      if (A.dlog && __any(log2_decay < -0.72f)) finish(std::true_type());       // uniform: log2 of exp(-1/2)
      else finish(std::false_type());
    } else {
      finish(std::true_type());
    }
    now = next;
  }
}

// dq and dk of the heads of q and k: the sums over the value heads that share them, in their order.
template <typename T>
__global__ __launch_bounds__(256) void delta_share_kernel(const float* __restrict__ pq, const float* __restrict__ pk, T* __restrict__ dq,
                                                          T* __restrict__ dk, long long quads, int width, int share) {
  const long long i = (long long)block_number() * 256 + threadIdx.x;   // [row and head][width / 4]
  if (i >= quads) return;
  const long long head = i / (width / 4), from = head * share * width + i % (width / 4) * 4;
  f32x4 q = load4(pq + from), k = load4(pk + from);
  for (int j = 1; j < share; ++j) {
    q += load4(pq + from + (long long)j * width);
    k += load4(pk + from + (long long)j * width);
  }
  store4(dq + 4 * i, q);
  store4(dk + 4 * i, k);
}

template <typename T, int DK, int W, bool kSums>
hipError_t launch_both_t(const DeltaArgs& a, hipStream_t st) {
  if (delta_state_rows(sizeof(T) == 2, a.m.dk) != DK) return hipErrorInvalidValue;   // the workspace is laid out for others
  constexpr int bytes = kBothBytes<T, DK, W>;
  const auto kernel = delta_both_kernel<T, DK, W, kSums>;
  hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes);
  if (e != hipSuccess) return e;
  const int reverse = (a.m.dv + 16 * W - 1) / (16 * W);
  const int forward = ((a.m.dv + 15) / 16 + (kSums ? (a.m.dk + 15) / 16 : 0) + W - 1) / W;
  const long long units = (long long)a.m.n_slots * a.m.H;
  launch_kernel(kernel, grid_rows((units + 7) / 8 * 8 * (forward + reverse)), 64 * W, bytes, st, a, forward + reverse, forward);
  return hipGetLastError();
}

template <bool kSums>
hipError_t launch_both_d(const DeltaArgs& a, bool bf16, hipStream_t st) {
  const int dk = a.m.dk;
  if (!bf16) return dk <= 32 ? launch_both_t<float, 32, 4, kSums>(a, st)
                  : dk <= 64 ? launch_both_t<float, 64, 4, kSums>(a, st) : launch_both_t<float, 128, 4, kSums>(a, st);
  if (decay_columns(true, a.m.dv) == 128)
    return dk <= 64 ? launch_both_t<__bf16, 64, 8, kSums>(a, st) : launch_both_t<__bf16, 128, 8, kSums>(a, st);
  return dk <= 64 ? launch_both_t<__bf16, 64, 4, kSums>(a, st)
                  : launch_both_t<__bf16, 128, 4, kSums>(a, st);
}

template <typename T, int DK>
hipError_t launch_grads_t(const DeltaArgs& a, hipStream_t st) {
  using TL = GradTiles<T, DK>;
  if (delta_state_rows(sizeof(T) == 2, a.m.dk) != DK) return hipErrorInvalidValue;
  const auto kernel = delta_grads_kernel<T, DK>;
  hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), TL::bytes);
  if (e != hipSuccess) return e;
  const long long units = (long long)a.m.c_slots * (a.pq ? a.m.H : a.m.Hk);
  launch_kernel(kernel, dim3(unsigned(units < kDeltaGradBlocks ? units : kDeltaGradBlocks)), kThreads, TL::bytes, st, a);
  if (a.pq) {
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const long long quads = (a.m.packed ? 1ll : a.m.n_seq) * a.m.T * a.m.Hk * (a.m.dk / 4);
    launch_kernel(delta_share_kernel<T>, grid_rows((quads + 255) / 256), 256, 0, st, a.pq, a.pk, (T*)a.dq, (T*)a.dk, quads, a.m.dk,
                  a.m.H / a.m.Hk);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_bwd_walk(const DeltaArgs& a, bool bf16, bool sums, hipStream_t st) {
  return sums ? launch_both_d<true>(a, bf16, st) : launch_both_d<false>(a, bf16, st);
}

hipError_t launch_delta_grads(const DeltaArgs& a, bool bf16, hipStream_t st) {
  const int dk = a.m.dk;
  if (bf16) return dk <= 64 ? launch_grads_t<__bf16, 64>(a, st) : launch_grads_t<__bf16, 128>(a, st);
  return dk <= 32 ? launch_grads_t<float, 32>(a, st)
         : dk <= 64 ? launch_grads_t<float, 64>(a, st) : launch_grads_t<float, 128>(a, st);
}

}  // namespace kata
