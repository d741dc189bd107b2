// Gradients of the gated delta rule (delta.hip), gfx950.
//
// With the notation there, S the state before a chunk and D the gradient of the one behind it:
//   Z = P^T dO scale + diag(exp(c_63 - c)) K D          (the gradient of U)
//   X = (I + A)^-T Z,  dv = diag(b) X
//   the gradient of S:  y_63 D + scale (diag(y) Q)^T dO - (diag(y) K)^T dv
//   dbeta_i = X_i . U_i / b_i
//   dlog_t = sum_{i >= t in the chunk} (dO_i . o_i - dv_i . v_i) + <D, S'>,  S' the state behind the chunk
//   PO_ij = scale exp(c_i - c_j) (dO_i . u_j) for j <= i,  PV_ij = -exp(c_i - c_j) (dv_i . u_j) for j < i
//   dq = scale diag(y) dO S^T + PO K
//   dk = diag(exp(c_63 - c)) U D^T - diag(y) dv S^T + PO^T Q + PV^T K + PV K
// (the second last line but two: what S_t loses or gains from token t on is known from its products with
// the gradients, d<dS_t, S_t> = dv_t . v_t - dO_t . o_t.)
//
// S and D of every chunk come from two walks like the forward pass's, one of them in reversed time, which
// keep nothing else; all the rest is then computed for all chunks at once (delta_grads_kernel).
#include <type_traits>

#include "delta.h"
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
  static constexpr int NT = kBf ? 3 : 1, NI = kBf ? 2 : 1, NP = NI;     // terms of the recurrence's operands, of the inverse, of P
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
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (unit >= (unsigned)m.n_slots * (unsigned)m.H) return;
  const int slot = int(unit / (unsigned)m.H), h = int(unit - (unsigned)slot * (unsigned)m.H);
  const int c0 = sub * DV;
  DeltaPart s;
  if (!find_part(m, slot, m.L, m.n_seg, m.n_slots, sh, s) || s.seq == m.n_seq) return;
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
  const T* px = reinterpret_cast<const T*>(A.dO) + s.b * A.sdo[0] + row0 * A.sdo[1] + h * A.sdo[2] + c0;
  Stage<T, DK, kThr> rk(pk, A.sk[1], m.dk, true), rq(pq, A.sq[1], m.dk, true);
  Stage<T, DV, kThr> ro(px, A.sdo[1], m.dv - c0, false);
  StageInv<T, NI, LP, kThr> ri;
  uint4 vec_next;
  const long long chunk0 = (long long)s.c_slot * m.H + h;              // [c_slots][H]
  auto fetch = [&](int c) {
    const int n = c == behind - 1 ? n_last : kC;
    fetch_rows(rk, A.sk[1], n);
    fetch_rows(rq, A.sq[1], n);
    fetch_rows(ro, A.sdo[1], n);
    rk.p -= 2 * kC * A.sk[1];
    rq.p -= 2 * kC * A.sq[1];
    ro.p -= 2 * kC * A.sdo[1];
    ri.fetch(A.inv + (chunk0 + (long long)c * m.H) * kInvFloats);
    if (tid < kDeltaVec / 4)
      vec_next = reinterpret_cast<const uint4*>(A.vec + (chunk0 + (long long)c * m.H) * kDeltaVec)[tid];
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
#pragma unroll 1
  for (int c = behind - 1; c >= first; --c) {
    __syncthreads();                                // the last chunk's tiles have been read
    rk.template put_split<LK>(sK);
    rq.template put_split<LK>(sQ);
    ro.template put<LV>(sO);
    ri.put(sT);
    if (tid < kDeltaVec / 4) reinterpret_cast<uint4*>(vec)[tid] = vec_next;
    if (!kSums && c0 / 16 + w < (m.dv + 15) / 16) {
      float* dst = A.rstates + ((chunk0 + (long long)c * m.H) * ((m.dv + 15) / 16) + c0 / 16 + w) * (DK * 16) + lane * 4;
#pragma unroll
      for (int i = 0; i < NS; ++i) *reinterpret_cast<f32x4*>(dst + i * 256) = D[i];
    }
    if (c > first) fetch(c - 1);
    __syncthreads();
    // reads in batches, as in the walk
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
        for (int it = 0; it < 4; ++it) Z[it] = mul(kr[it][i], df[i], Z[it]);
      put_weights<T, LP, J, NP>(sP, p, vec + 3 * kC, rt, j0, lane, A.scale);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) of[i] = column_frag<LV>(sO + 32 * i * LV + wc, lane);
    Op<T, NI> inv[6];                               // (row tile, K step): (0, 0), (0, 1), (1, 0), (1, 1), (2, 1), (3, 1)
#pragma unroll
    for (int f = 0; f < 6; ++f)
      inv[f] = split_column_op<NI, LP>(sT + 32 * (f < 4 ? f & 1 : 1) * LP, kC * LP, f < 4 ? f >> 1 : f - 2, lane);
#pragma unroll
    for (int it = 0; it < 4; ++it) Z[it] *= *reinterpret_cast<const f32x4*>(vec + kC + 16 * it + 4 * g);
    __syncthreads();                                // P is there
    {
      Op<T, NP> pf[6];
#pragma unroll
      for (int f = 0; f < 6; ++f)
        pf[f] = split_column_op<NP, LP>(sP + 32 * (f < 4 ? f & 1 : 1) * LP, kC * LP, f < 4 ? f >> 1 : f - 2, lane);
      reads_above<T>();
      Z[0] = mul(pf[0], of[0], Z[0]);
      Z[1] = mul(pf[2], of[0], Z[1]);
      Z[2] = mul(pf[4], of[1], Z[2]);
      Z[3] = mul(pf[5], of[1], Z[3]);
      Z[0] = mul(pf[1], of[1], Z[0]);
      Z[1] = mul(pf[3], of[1], Z[1]);
    }
    frag qt[2][NS];                                 // Q transposed, 32 tokens each, then K
    auto read_t = [&](const T* tile, int j) {
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
      X[0] = mul(inv[0], zf[0], zero4());
      X[1] = mul(inv[2], zf[0], zero4());
      X[2] = mul(inv[4], zf[1], zero4());
      X[3] = mul(inv[5], zf[1], zero4());
      X[0] = mul(inv[1], zf[1], X[0]);
      X[1] = mul(inv[3], zf[1], X[1]);
    }
    Op<T, NT> kw[2];
    Op<T, NI> qw[2];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f32x4 yv = *reinterpret_cast<const f32x4*>(vec + 16 * it + 4 * g);
      X[it] *= -yv * *reinterpret_cast<const f32x4*>(vec + 2 * kC + 16 * it + 4 * g);
      Z[it] = half_of(of[it >> 1], it & 1) * yv * A.scale;
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
      for (int i = 0; i < NS; ++i) D[i] = mul(qt[j][i], qw[j], D[i]);
      read_t(sK, j);
    }
    reads_above<T>();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < NS; ++i) D[i] = mul(qt[j][i], kw[j], D[i]);
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
template <typename T, int DK, int W, bool kSums>
constexpr int kBothBytes = WalkTiles<T, DK, W, 3, false>::bytes > ReverseTiles<T, DK, W>::bytes ? WalkTiles<T, DK, W, 3, false>::bytes
                                                                                              : ReverseTiles<T, DK, W>::bytes;
template <typename T, int DK, int W, bool kSums>
__global__ __launch_bounds__(64 * W, sizeof(T) == 4 && DK == 128 ? 1 : 8 / W) void delta_both_kernel(DeltaArgs A, int blocks,
                                                                                                  int forward) {
  extern __shared__ __align__(16) char lds[];
  const UnitBlock u = unit_block(blocks);
  if (u.sub < forward) delta_walk<T, DK, W, sizeof(T) == 2 ? 3 : 1, kSums ? Walk::sums : Walk::states>(A, u.unit, u.sub, 1, lds);
  else delta_reverse<T, DK, W, kSums>(A, u.unit, u.sub - forward, lds);
}

// ---- the gradients ------------------------------------------------------------------------------
// One workgroup of eight waves for a chunk and a head of q and k, over the value heads that share it and
// blocks of 64 value columns.  As in the walks a wave has 16 columns, four of them S, U and the outputs, the
// others D, Z, X and dv; then these go through LDS, [column][token] and [column][row of the state], and a wave
// has 16 tokens of dq and dk, half of the columns each.
template <typename T, int DK>
struct GradTiles {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int PAD = 16 / (int)sizeof(T);
  static constexpr int LK = DK + PAD, LO = 64 + PAD, LV = 64 + (kBf ? 16 : 4), LP = kC + PAD, LS = DK + PAD;
  static constexpr int kHead = 16 + kDeltaVec * 4 + 9 * kC * 4 + 16;   // an int, vec, dots and sums of the waves
  static constexpr int NT = kBf ? 3 : 1, NI = kBf ? 2 : 1, NP = NI;     // terms of the recurrence's operands, of the inverse, of P
  static constexpr int kStateTile = 64 * LS, kPair = 2 * 64 * LP;
  // scores, then (bf16) the second terms of U and dv, or (fp32) a state, then PO and PV
  static constexpr int kA = kBf || kPair > kStateTile ? kPair : kStateTile;
  // bf16: both states, and the inverse's terms
  static constexpr int bytes = kHead + (kC * (2 * LK + LO) + kA + kPair + (kBf ? 2 * kStateTile + NI * kC * LP : 0)) * (int)sizeof(T);
  static_assert(64 * LV <= (kBf ? kPair : kPair / 2), "V lies where U (bf16: and dv) come, the inverse (fp32) where dv comes");
};

__device__ __forceinline__ float sum16(float x) {   // over the 16 lanes of a group
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) x += __shfl_xor(x, s);
  return x;
}

template <typename T, int DK>
__global__ __launch_bounds__(kThreads, 1) void delta_grads_kernel(DeltaArgs A) {
  using TL = GradTiles<T, DK>;
  using frag = typename Elem<T>::frag;
  constexpr int M = DK / 32, NS = DK / 16, NH = NS / 2, LK = TL::LK, LO = TL::LO, LV = TL::LV, LP = TL::LP, LS = TL::LS;
  constexpr int NT = TL::NT, NI = TL::NI, NP = TL::NP;
  constexpr bool kBf = TL::kBf;
  extern __shared__ __align__(16) char lds[];
  int* const sh = reinterpret_cast<int*>(lds);
  float* const vec = reinterpret_cast<float*>(lds + 16);
  const float* const sc = vec + 3 * kC;
  float* const sE = vec + kDeltaVec;                // [8][64] dO . o, -dv . v; then [64] dv . U
  float* const sF = sE + 9 * kC;                    // [4] <D, S'>
  T* const sK = reinterpret_cast<T*>(lds + TL::kHead);
  T* const sQ = sK + kC * LK;
  T* const sO = sQ + kC * LK;
  T* const sA = sO + kC * LO;
  T* const sU = sA + TL::kA;                        // V, then U and dv
  T* const sZ = sU + 64 * LP;
  T* const sS = kBf ? sZ + 64 * LP : sA;
  T* const sD = kBf ? sS + TL::kStateTile : sA;
  T* const sT = kBf ? sD + TL::kStateTile : sZ;

  const DeltaMap& m = A.m;
  const int tid = threadIdx.x;
  int lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  // The places in LDS that a phase uses are computed there: kept from phase to phase they would cost a hundred
  // registers, and scratch.
  auto forget = [&] {
    asm volatile("" : "+v"(lane));
    g = lane >> 4;
    l16 = lane & 15;
  };
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
  const bool first_half = wave < 4;
  const unsigned unit = block_number();
  if (unit >= (unsigned)m.c_slots * (unsigned)m.Hk) return;
  const int slot = int(unit / (unsigned)m.Hk), hk = int(unit - (unsigned)slot * (unsigned)m.Hk);
  const int share = m.H / m.Hk;
  DeltaPart s;
  if (!find_part(m, slot, 1, m.n_chunks, m.c_slots, sh, s)) return;

  T* const gq = reinterpret_cast<T*>(A.dq) + ((long long)s.b * m.T * m.Hk + hk) * m.dk;   // row stride Hk dk
  T* const gk = reinterpret_cast<T*>(A.dk) + ((long long)s.b * m.T * m.Hk + hk) * m.dk;
  const long long lead = (long long)s.b * m.T * m.H + hk * share;      // of [b][t][H], the first shared head
  auto clear = [&](int from, int rows) {
    for (long long i = tid; i < (long long)rows * (m.dk / 4); i += kThreads) {
      const long long at = (from + i / (m.dk / 4)) * m.Hk * m.dk + i % (m.dk / 4) * 4;
      store4(gq + at, zero4());
      store4(gk + at, zero4());
    }
    const int per = share * m.dv / 4;
    for (long long i = tid; i < (long long)rows * per; i += kThreads)
      store4(reinterpret_cast<T*>(A.dv) + (lead + (from + i / per) * m.H) * m.dv + i % per * 4, zero4());
    for (long long i = tid; i < (long long)rows * share; i += kThreads) {
      const long long at = lead + (from + i / share) * m.H + i % share;
      reinterpret_cast<T*>(A.dbeta)[at] = T(0.f);
      if (A.dlog) A.dlog[at] = 0.f;
    }
  };
  const int n = min(kC, s.len - kC * s.part);
  if (s.seq == m.n_seq) {                           // rows behind the last sequence
    if (n > 0) clear(s.start + kC * s.part, n);
    return;
  }
  if (m.packed && s.seq == 0 && s.part == 0) clear(0, s.start);        // before the first
  if (n <= 0) return;
  const bool last = kC * (s.part + 1) >= s.len;
  const long long row0 = s.start + (long long)kC * s.part;
  const int ct = (m.dv + 15) / 16, v_blocks = (m.dv + 63) / 64;

  // tiles' columns that no operand has: zeros all along (V's place is written over: cleared each time)
  if (m.dk < DK || m.dv % 64)
    for (int i = tid; i < kC * (2 * LK + LO) * (int)sizeof(T) / 16; i += kThreads)
      reinterpret_cast<uint4*>(sK)[i] = uint4{0u, 0u, 0u, 0u};
  {
    Stage<T, DK, kThreads> rk(reinterpret_cast<const T*>(A.k) + s.b * A.sk[0] + row0 * A.sk[1] + hk * A.sk[2], A.sk[1], m.dk, true);
    Stage<T, DK, kThreads> rq(reinterpret_cast<const T*>(A.q) + s.b * A.sq[0] + row0 * A.sq[1] + hk * A.sq[2], A.sq[1], m.dk, true);
    fetch_rows(rk, A.sk[1], n);
    fetch_rows(rq, A.sq[1], n);
    if (m.dk < DK || m.dv % 64) __syncthreads();
    rk.template put_split<LK>(sK);
    rq.template put_split<LK>(sQ);
  }

  f32x4 dqa[NH], dka[NH];                           // [row 16 (i0 + i) + 4 g + r][token 16 w + l16]
  const int i0 = first_half ? 0 : NH;
#pragma unroll
  for (int i = 0; i < NH; ++i) dqa[i] = dka[i] = zero4();

#pragma unroll 1
  for (int hh = 0; hh < share; ++hh) {
    const int h = hk * share + hh;
    const long long cs = (long long)slot * m.H + h;                    // [c_slots][H]
    f32x4 Wt[4], e[4];                              // the strip of dO U^T (second half: dv U^T), transposed
    float frob = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) Wt[i] = e[i] = zero4();
#pragma unroll 1
    for (int vb = 0; vb < v_blocks; ++vb) {
      const int c0 = 64 * vb;
      forget();
      Stage<T, 64, kThreads> ro(reinterpret_cast<const T*>(A.dO) + s.b * A.sdo[0] + row0 * A.sdo[1] + h * A.sdo[2] + c0,
                                A.sdo[1], m.dv - c0, true);
      Stage<T, 64, kThreads> rv(reinterpret_cast<const T*>(A.v) + s.b * A.sv[0] + row0 * A.sv[1] + h * A.sv[2] + c0,
                                A.sv[1], m.dv - c0, false);
      fetch_rows(ro, A.sdo[1], n);
      fetch_rows(rv, A.sv[1], n);
      StageInv<T, NI, LP, kThreads> ri;
      ri.fetch(A.inv + cs * kInvFloats);
      f32x4 S[NS];                                  // (second half: D)
      const bool live_tile = 4 * vb + w < ct;       // uniform
#pragma unroll
      for (int i = 0; i < NS; ++i) S[i] = zero4();
      if (live_tile) {
        const long long tile = (cs * ct + 4 * vb + w) * (DK * 16) + lane * 4;
        const float* const from = (first_half ? A.cstates : A.rstates) + tile;
#pragma unroll
        for (int i = 0; i < NS; ++i) S[i] = *reinterpret_cast<const f32x4*>(from + i * 256);
        if (!first_half && !(last && !A.fstates)) {  // (behind the last chunk without a gradient D is zero)
          const float* const next = last ? A.fstates + (((long long)s.seq * m.H + h) * ct + 4 * vb + w) * (DK * 16) + lane * 4
                                         : A.cstates + tile + (long long)m.H * ct * (DK * 16);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(next + i * 256);
#pragma unroll
            for (int r = 0; r < 4; ++r) frob = fmaf(S[i][r], x[r], frob);
          }
        }
      }
      __syncthreads();                              // the last block's and head's tiles have been read
      if (vb == 0 && tid < kDeltaVec / 4)
        reinterpret_cast<uint4*>(vec)[tid] = reinterpret_cast<const uint4*>(A.vec + cs * kDeltaVec)[tid];
      if (m.dv - c0 < 64) {
        for (int i = tid; i < 64 * LV * (int)sizeof(T) / 16; i += kThreads)
          reinterpret_cast<uint4*>(sU)[i] = uint4{0u, 0u, 0u, 0u};
        if (vb > 0)
          for (int i = tid; i < kC * LO * (int)sizeof(T) / 16; i += kThreads)
            reinterpret_cast<uint4*>(sO)[i] = uint4{0u, 0u, 0u, 0u};
        __syncthreads();
      }
      ro.template put_split<LO>(sO);
      rv.template put<LV>(sU);
      ri.put(sT);
      ri.zeros(sT);
      __syncthreads();

      // a wave's 16 columns: x becomes U (X), y the outputs (Z)
      put_scores<T, DK, LK, LP, 2, NP>(sA, sQ, sK, sc, w, first_half ? 0 : 2, lane, A.scale);
      forget();
      const int wc = 16 * w;
      f32x4 x[4], y[4];
      frag of[2], vf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        vf[i] = column_frag<LV>(sU + 32 * i * LV + wc, lane);
        of[i] = split_column_frag<LO>(sO + 32 * i * LO, w, lane);
      }
      {
        Op<T, NT> sf[M];
#pragma unroll
        for (int i = 0; i < M; ++i) split_terms(S[2 * i], S[2 * i + 1], sf[i]);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          x[it] = y[it] = zero4();
#pragma unroll
          for (int i = 0; i < M; ++i) x[it] = mul(row_frag(sK + (16 * it + l16) * LK + 32 * i + 8 * g), sf[i], x[it]);
        }
        if (first_half)
#pragma unroll
          for (int it = 0; it < 4; ++it) {
#pragma unroll
            for (int i = 0; i < M; ++i) y[it] = mul(row_frag(sQ + (16 * it + l16) * LK + 32 * i + 8 * g), sf[i], y[it]);
            const f32x4 yv = *reinterpret_cast<const f32x4*>(vec + 16 * it + 4 * g);
            y[it] *= yv * A.scale;
            x[it] = *reinterpret_cast<const f32x4*>(vec + 2 * kC + 16 * it + 4 * g) * (half_of(vf[it >> 1], it & 1) - yv * x[it]);
          }
        else
#pragma unroll
          for (int it = 0; it < 4; ++it) y[it] = x[it] * *reinterpret_cast<const f32x4*>(vec + kC + 16 * it + 4 * g);
      }
      reads_above<T>();
      Op<T, NT> f[2];
      if (first_half) {
#pragma unroll
        for (int i = 0; i < 2; ++i) split_terms(x[2 * i], x[2 * i + 1], f[i]);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          x[it] = zero4();
#pragma unroll
          for (int i = 0; i <= it >> 1; ++i)
            x[it] = mul(row_op<NI>(sT + (16 * it + l16) * LP + 32 * i + 8 * g, kC * LP), f[i], x[it]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) split_terms(x[2 * i], x[2 * i + 1], f[i]);
      }
      __syncthreads();                              // P is there
      forget();
      if (first_half) {
#pragma unroll
        for (int it = 0; it < 4; ++it) {
#pragma unroll
          for (int i = 0; i <= it >> 1; ++i)
            y[it] = mul(row_op<NP>(sA + (16 * it + l16) * LP + 32 * i + 8 * g, kC * LP), f[i], y[it]);
          e[it] += y[it] * half_of(of[it >> 1], it & 1);
        }
      } else {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int i = it >> 1; i < 2; ++i)
            y[it] = mul(split_column_op<NP, LP>(sA + 32 * i * LP, kC * LP, it, lane), of[i], y[it]);
#pragma unroll
        for (int i = 0; i < 2; ++i) split_terms(y[2 * i], y[2 * i + 1], f[i]);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          x[it] = zero4();
#pragma unroll
          for (int i = it >> 1; i < 2; ++i)
            x[it] = mul(split_column_op<NI, LP>(sT + 32 * i * LP, kC * LP, it, lane), f[i], x[it]);
          x[it] *= *reinterpret_cast<const f32x4*>(vec + 2 * kC + 16 * it + 4 * g);      // dv
          e[it] -= x[it] * half_of(vf[it >> 1], it & 1);
        }
      }
      __syncthreads();                              // P, V and the inverse have been read
      // U, dv and the states through LDS
      forget();
      {
        T* const mine = (first_half ? sU : sZ) + (wc + l16) * LP + 4 * g;
        T* const rest = sA + ((first_half ? 0 : 64) + wc + l16) * LP + 4 * g;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const Quad<T> u = quad(x[it], T());
          *reinterpret_cast<Quad<T>*>(mine + 16 * it) = u;
          if constexpr (kBf) store4(rest + 16 * it, x[it] - unquad(u));
        }
        if (kBf || first_half)
#pragma unroll
          for (int i = 0; i < NS; ++i) store4((first_half ? sS : sD) + (wc + l16) * LS + 16 * i + 4 * g, S[i]);
      }
      __syncthreads();

      // a wave's 16 tokens
      forget();
      frag ur[2], zr[2], ot[2];
      {
        constexpr int NW = kBf ? 2 : 1;             // terms of U and dv
        Op<T, NW> zt[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          zt[i].t[0] = zr[i] = column_frag<LP>(sZ + 32 * i * LP + 16 * w, lane);
          if constexpr (kBf) zt[i].t[1] = column_frag<LP>(sA + (64 + 32 * i) * LP + 16 * w, lane);
          ot[i] = row_frag(sO + (16 * w + l16) * LO + 32 * i + 8 * g);
          ur[i] = column_frag<LP>(sU + 32 * i * LP + 16 * w, lane);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j <= w)                               // uniform
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              Op<T, NW> ut;
              ut.t[0] = column_frag<LP>(sU + 32 * i * LP + 16 * j, lane);
              if constexpr (kBf) ut.t[1] = column_frag<LP>(sA + 32 * i * LP + 16 * j, lane);
              if (first_half) Wt[j] = mul(ut, ot[i], Wt[j]);
              else Wt[j] = mul(ut, zt[i], Wt[j]);
            }
        forget();
        const float yr = vec[16 * w + l16], yo = yr * A.scale;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          f32x4 a = zero4(), b = zero4();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const frag st = column_frag<LS>(sS + 32 * j * LS + 16 * (i0 + i), lane);
            a = mma(st, ot[j], a);
            b = mma(st, zr[j], b);
          }
          dqa[i] += a * yo;
          dka[i] -= b * yr;
        }
        // dv: tokens 16 w + l16, columns 32 i + 16 half + 4 g, half of them each
        if (16 * w + l16 < n) {
          T* const dst = reinterpret_cast<T*>(A.dv) + ((lead + hh) + (row0 + 16 * w + l16) * m.H) * m.dv + c0 + 4 * g;
          const int i = first_half ? 0 : 1;
          const frag z = first_half ? zr[0] : zr[1];
#pragma unroll
          for (int half = 0; half < 2; ++half)
            if (c0 + 32 * i + 16 * half + 4 * g < m.dv) store4(dst + 32 * i + 16 * half, half_of(z, half));
        }
      }
      if constexpr (!kBf) {
        __syncthreads();                            // S has been read
        if (!first_half)
#pragma unroll
          for (int i = 0; i < NS; ++i) store4(sD + (wc + l16) * LS + 16 * i + 4 * g, S[i]);
        __syncthreads();
      }
      forget();
      const float left = vec[kC + 16 * w + l16];
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        f32x4 a = zero4();
#pragma unroll
        for (int j = 0; j < 2; ++j) a = mma(column_frag<LS>(sD + 32 * j * LS + 16 * (i0 + i), lane), ur[j], a);
        dka[i] += a * left;
      }
    }
    // dots: over a wave's 16 columns, then over the waves
    forget();
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float a = sum16(e[it][r]);
        if (l16 == 0) sE[wave * kC + 16 * it + 4 * g + r] = a;
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) frob += __shfl_xor(frob, d);
    if (lane == 0 && !first_half) sF[w] = frob;
    if (!first_half) {                              // the diagonal of dv U^T
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j == w && 4 * g + r == l16) d = Wt[j][r];
      if (l16 >> 2 == g) sE[8 * kC + 16 * w + l16] = d;
    }
    __syncthreads();                                // (the second terms and D have been read, too)
    // PO or PV, the wave's strip of rows
    {
      const float hi = sc[16 * w + l16], lo = sc[kC + 16 * w + l16], factor = first_half ? A.scale : -1.f;
      const int row = 16 * w + l16 + (first_half ? 1 : 0);             // the first key that it does not reach
      T* const at = sA + ((first_half ? 0 : kC) + 16 * w + l16) * LP;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 p = zero4();
        if (j <= w)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = 16 * j + 4 * g + r;
            p[r] = key >= row ? 0.f : Wt[j][r] * (exp2_diff(hi, lo, sc[key], sc[kC + key]) * factor);
          }
        store4(at + split_place(16 * j + 4 * g), p);
      }
    }
    if (wave == 0) {
      const long long at = lead + hh + (row0 + lane) * m.H;
      const float b = vec[2 * kC + lane];
      if (lane < n) reinterpret_cast<T*>(A.dbeta)[at] = from_f32<T>(sE[8 * kC + lane] / (b * b));
      if (A.dlog) {
        double x = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) x += (double)sE[i * kC + lane];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const double up = __shfl_down(x, d);
          if (lane + d < 64) x += up;
        }
        x += (double)sF[0] + sF[1] + sF[2] + sF[3];
        // a decay of nothing, and one of zero (in fp32), have no gradient
        const bool none = (s.part == 0 && lane == 0 && !A.init) || sc[lane] - (lane ? sc[lane - 1] : 0.f) < -150.f;
        if (lane < n) A.dlog[at] = none ? 0.f : (float)x;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const frag kt = split_column_frag<LK>(sK + 32 * j * LK, i0 + i, lane);
        if (j <= w >> 1) {                          // uniform
          dqa[i] = mma(kt, row_frag(sA + (16 * w + l16) * LP + 32 * j + 8 * g), dqa[i]);
          dka[i] = mma(kt, row_frag(sA + (kC + 16 * w + l16) * LP + 32 * j + 8 * g), dka[i]);
        }
        if (j >= w >> 1) {
          dka[i] = mma(split_column_frag<LK>(sQ + 32 * j * LK, i0 + i, lane), split_column_frag<LP>(sA + 32 * j * LP, w, lane), dka[i]);
          dka[i] = mma(kt, split_column_frag<LP>(sA + (kC + 32 * j) * LP, w, lane), dka[i]);
        }
      }
  }
  if (16 * w + l16 < n) {
    const long long at = (row0 + 16 * w + l16) * m.Hk * m.dk + 4 * g;
#pragma unroll
    for (int i = 0; i < NH; ++i)
      if (16 * (i0 + i) + 4 * g < m.dk) {
        store4(gq + at + 16 * (i0 + i), dqa[i]);
        store4(gk + at + 16 * (i0 + i), dka[i]);
      }
  }
}

template <typename T, int DK, int W, bool kSums>
hipError_t launch_both_t(const DeltaArgs& a, hipStream_t st) {
  constexpr int bytes = kBothBytes<T, DK, W, kSums>;
  const auto kernel = delta_both_kernel<T, DK, W, kSums>;
  hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes);
  if (e != hipSuccess) return e;
  const int v = (a.m.dv + 16 * W - 1) / (16 * W), forward = v + (kSums ? (a.m.dk + 16 * W - 1) / (16 * W) : 0);
  const long long units = (long long)a.m.n_slots * a.m.H;
  launch_kernel(kernel, grid_rows((units + 7) / 8 * 8 * (forward + v)), 64 * W, bytes, st, a, forward + v, forward);
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
  const auto kernel = delta_grads_kernel<T, DK>;
  hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), TL::bytes);
  if (e != hipSuccess) return e;
  launch_kernel(kernel, grid_rows((long long)a.m.c_slots * a.m.Hk), kThreads, TL::bytes, st, a);
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
